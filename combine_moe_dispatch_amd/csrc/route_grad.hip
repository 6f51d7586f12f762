// Gradient of a token's chosen weights to its logits (the backward pass of
// moe_topk_route).
//
// Without renormalisation w_k = p[idx_k], p the softmax over all experts:
//   dz_e = p_e (g_e - G),  g_e = sum of dw_k over idx_k = e,  G = sum of p[idx_k] dw_k.
// With it, w is the softmax over the chosen logits alone, and so is the
// gradient: dz_e = w_e (g_e - sum of w_k dw_k) for those, 0 for the others.
//
// LANES lanes have a token: its logits in registers, read once, the chosen
// experts' g in LDS, where each lane finds its own experts'.
#include <algorithm>
#include <cmath>

#include "moe_kernels.h"
#include "moe_ops.h"
#include "ops_common.h"

namespace moe {
namespace ops {
namespace {

template <int LANES>
__device__ inline float lanes_max(float v)
{
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1)
        v = fmaxf(v, __shfl_xor(v, d, LANES));
    return v;
}
template <int LANES>
__device__ inline float lanes_sum(float v)
{
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1)
        v += __shfl_xor(v, d, LANES);
    return v;
}

// exp(z - top): 0 for a masked logit (minus infinity, or NaN), 1 for plus infinity.
__device__ inline float weight_of(float z, float top)
{
    if (!(z > -INFINITY))
        return 0.0f;
    return z == top ? 1.0f : exp_of(z - top);
}

template <bool BF16>
__device__ inline float logit(const void* z, int64_t i)
{
    const float v = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)z)[i] << 16) : ((const float*)z)[i];
    return v == v ? v : -INFINITY;
}

// VALS logits per lane in groups of W consecutive ones.
template <int LANES, int VALS, int W, bool BF16>
__global__ __launch_bounds__(256) void topk_route_grad_kernel(const RouteGrad a)
{
    extern __shared__ __align__(16) float chosen[];     // [tokens of the workgroup][LANES * VALS]
    constexpr int TOKENS = 256 / LANES;
    const int lane = threadIdx.x % LANES;
    float* const add = chosen + threadIdx.x / LANES * (LANES * VALS);
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t t = block * TOKENS + threadIdx.x / LANES;
    const bool live = t < a.tokens;
    const int64_t row = live ? t * a.E : 0;
    auto expert = [&](int i) { return (i / W * LANES + lane) * W + i % W; };
#pragma unroll
    for (int i = 0; i < VALS; ++i)
        add[expert(i)] = 0.0f;
    float z[VALS];
    float top = -INFINITY, sum = 0.0f;
    if (!a.renorm) {
#pragma unroll
        for (int i = 0; i < VALS; i += W) {
            const int e = expert(i);
            if constexpr (W == 4) {
                z[i] = z[i + 1] = z[i + 2] = z[i + 3] = -INFINITY;
                if (e < a.E) {
                    if constexpr (BF16) {
                        const v2u u = *(const v2u*)((const uint16_t*)a.logits + row + e);
                        z[i] = bf16_lo(u.x);
                        z[i + 1] = bf16_hi(u.x);
                        z[i + 2] = bf16_lo(u.y);
                        z[i + 3] = bf16_hi(u.y);
                    } else {
                        const v4f u = *(const v4f*)((const float*)a.logits + row + e);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            z[i + c] = u[c];
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        z[i + c] = z[i + c] == z[i + c] ? z[i + c] : -INFINITY;
                }
            } else {
                z[i] = e < a.E ? logit<BF16>(a.logits, row + e) : -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < VALS; ++i)
            top = fmaxf(top, z[i]);
        top = lanes_max<LANES>(top);
#pragma unroll
        for (int i = 0; i < VALS; ++i) {
            z[i] = weight_of(z[i], top);
            sum += z[i];
        }
        sum = lanes_sum<LANES>(sum);
    }
    // the chosen experts, LANES at a time
    const int64_t first = live ? t * a.K : 0;
    if (a.renorm) {
        for (int k = lane; k < a.K; k += LANES) {
            const int e = a.idx[first + k];
            if ((uint32_t)e < (uint32_t)a.E)
                top = fmaxf(top, logit<BF16>(a.logits, row + e));
        }
        top = lanes_max<LANES>(top);
        for (int k = lane; k < a.K; k += LANES) {
            const int e = a.idx[first + k];
            if ((uint32_t)e < (uint32_t)a.E)
                sum += weight_of(logit<BF16>(a.logits, row + e), top);
        }
        sum = lanes_sum<LANES>(sum);
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    float G = 0.0f;
    for (int k = lane; k < a.K; k += LANES) {
        const int e = a.idx[first + k];
        if ((uint32_t)e < (uint32_t)a.E) {
            const float p = weight_of(logit<BF16>(a.logits, row + e), top) * inv;
            G += p > 0.0f ? p * a.dw[first + k] : 0.0f;
        }
    }
    G = lanes_sum<LANES>(G);
    __syncthreads();
    for (int k = lane; k < a.K; k += LANES) {
        const int e = a.idx[first + k];
        if ((uint32_t)e >= (uint32_t)a.E)
            continue;
        const float p = weight_of(logit<BF16>(a.logits, row + e), top) * inv;
        float g = 0.0f;                       // in the order of k, whichever lane it is
        for (int j = 0; j < a.K; ++j)
            if (a.idx[first + j] == e)
                g += a.dw[first + j];
        if (p > 0.0f)
            add[e] = a.renorm ? p * (g - G) : p * g;
    }
    __syncthreads();
    if (!live)
        return;
#pragma unroll
    for (int i = 0; i < VALS; i += W) {
        const int e = expert(i);
        if (e >= a.E)
            continue;
        float d[W];
#pragma unroll
        for (int c = 0; c < W; ++c) {
            d[c] = add[e + c];
            if (!a.renorm) {
                const float p = z[i + c] * inv;
                d[c] = p > 0.0f ? d[c] - p * G : 0.0f;
            }
        }
        if (a.out_bf16) {
            uint16_t* o = (uint16_t*)a.dlogits + row + e;
            if constexpr (W == 4)
                *(v2u*)o = v2u{bf16_pack(d[0], d[1]), bf16_pack(d[2], d[3])};
            else
                *o = (uint16_t)bf16_pack(d[0], 0.0f);
        } else {
            float* o = (float*)a.dlogits + row + e;
            if constexpr (W == 4)
                *(v4f*)o = v4f{d[0], d[1], d[2], d[3]};
            else
                *o = d[0];
        }
    }
}

template <int LANES, int VALS>
hipError_t launch(const RouteGrad& a, hipStream_t stream)
{
    constexpr int TOKENS = 256 / LANES;
    constexpr int64_t ROW = 1 << 20;              // a grid dimension times the threads stays below 2^32
    const int64_t blocks = (a.tokens + TOKENS - 1) / TOKENS;
    const dim3 grid((uint32_t)std::min(blocks, ROW), (uint32_t)((blocks + ROW - 1) / ROW));
    const int bytes = 256 * VALS * 4;
    const bool wide = a.E % 4 == 0;
    if constexpr (VALS % 4 == 0)
        if (wide) {
            if (a.bf16)
                topk_route_grad_kernel<LANES, VALS, 4, true><<<grid, dim3(256), bytes, stream>>>(a);
            else
                topk_route_grad_kernel<LANES, VALS, 4, false><<<grid, dim3(256), bytes, stream>>>(a);
            return hipGetLastError();
        }
    if (a.bf16)
        topk_route_grad_kernel<LANES, VALS, 1, true><<<grid, dim3(256), bytes, stream>>>(a);
    else
        topk_route_grad_kernel<LANES, VALS, 1, false><<<grid, dim3(256), bytes, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_topk_route_grad(const RouteGrad& a, hipStream_t stream)
{
    if (a.E <= 16)
        return launch<4, 4>(a, stream);
    if (a.E <= 64)
        return launch<16, 4>(a, stream);
    if (a.E <= 256)
        return launch<16, 16>(a, stream);
    return launch<64, 16>(a, stream);
}

}  // namespace ops
}  // namespace moe
