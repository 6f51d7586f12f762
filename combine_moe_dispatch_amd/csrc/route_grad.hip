// Gradient of a token's chosen weights to its logits (the backward pass of
// moe_topk_route).
//
// Without renormalisation w_k = p[idx_k], p the softmax over all experts:
//   dz_e = p_e (g_e - G),  g_e = sum of dw_k over idx_k = e,  G = sum of p[idx_k] dw_k.
// With it, w is the softmax over the chosen logits alone, and so is the
// gradient: dz_e = w_e (g_e - n_e sum of w_k dw_k) for those, 0 for the others,
// n_e how many of the choices are e (1, unless a caller's own choices repeat).
//
// LANES lanes have a token: its logits in registers, read once, and a row of
// LDS through which the exponentials reach the lanes that have the chosen
// experts, and those lanes' gradients the lanes that store them.  Bound by HBM:
// 131072 tokens, 256 experts, top 8, fp32 in and out 50 us, 5.6 TB/s, on logits
// that no cache holds (44 us where it does); 128 tokens 2.8 us, the launch's
// latency.
#include <algorithm>
#include <cmath>
#include <type_traits>

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

// What exp(z - top) is formed of: with a top of plus infinity the logits that are it share all, as
// zeros under a top of zero.  Masked logits (minus infinity, or NaN) give exp_of what is zero there,
// also under a top of minus infinity.
__device__ inline float under(float z, float top)
{
    return top == INFINITY ? (z == INFINITY ? 0.0f : -INFINITY) : z - top;
}

template <bool BF16>
__device__ inline float logit(const void* z, int64_t i)
{
    return BF16 ? __uint_as_float((uint32_t)((const uint16_t*)z)[i] << 16) : ((const float*)z)[i];
}

// VALS logits per lane in groups of W consecutive ones; LANES * 4 >= top_k
// (LANES, where that is 64).
template <int LANES, int VALS, int W, bool BF16>
__global__ __launch_bounds__(256) void topk_route_grad_kernel(const RouteGrad a)
{
    extern __shared__ __align__(16) float rows[];       // [tokens of the workgroup][LANES * VALS]
    constexpr int TOKENS = 256 / LANES, PER = LANES == WAVE ? 1 : 4;
    const int lane = threadIdx.x % LANES;
    float* const mine = rows + threadIdx.x / LANES * (LANES * VALS);
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t t = block * TOKENS + threadIdx.x / LANES;
    const bool live = t < a.tokens;
    const int64_t row = live ? t * a.E : 0;
    auto expert = [&](int i) { return (i / W * LANES + lane) * W + i % W; };
    // a row's lanes are of one wave: what they wrote is seen once the wave's writes are done
    auto meet = [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); };
    // the chosen experts, LANES at a time
    int e[PER];
    float dw[PER], p[PER];
    const int64_t first = live ? t * a.K : 0;
#pragma unroll
    for (int c = 0; c < PER; ++c) {
        const int k = c * LANES + lane;
        e[c] = -1;
        dw[c] = p[c] = 0.0f;
        if (k < a.K) {
            const int id = a.idx[first + k];
            dw[c] = a.dw[first + k];
            e[c] = (uint32_t)id < (uint32_t)a.E ? id : -1;
        }
    }
    float z[VALS];
    float top = -INFINITY, sum = 0.0f;
    if (!a.renorm) {
#pragma unroll
        for (int i = 0; i < VALS; i += W) {
            const int at = expert(i);
            if constexpr (W == 1) {
                z[i] = at < a.E ? logit<BF16>(a.logits, row + at) : -INFINITY;
            } else {
#pragma unroll
                for (int c = 0; c < W; ++c)
                    z[i + c] = -INFINITY;
                if (at < a.E) {
                    if constexpr (BF16) {
                        typedef uint32_t vu __attribute__((ext_vector_type(W / 2)));
                        const vu u = *(const vu*)((const uint16_t*)a.logits + row + at);
#pragma unroll
                        for (int c = 0; c < W / 2; ++c) {
                            z[i + 2 * c] = bf16_lo(u[c]);
                            z[i + 2 * c + 1] = bf16_hi(u[c]);
                        }
                    } else {
                        typedef float vf __attribute__((ext_vector_type(W)));
                        const vf u = *(const vf*)((const float*)a.logits + row + at);
#pragma unroll
                        for (int c = 0; c < W; ++c)
                            z[i + c] = u[c];
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VALS; ++i)
            top = fmaxf(top, z[i]);
        top = lanes_max<LANES>(top);
        if (top < INFINITY) {
#pragma unroll
            for (int i = 0; i < VALS; ++i)
                z[i] = exp_of(z[i] - top);
        } else {
#pragma unroll
            for (int i = 0; i < VALS; ++i)
                z[i] = exp_of(under(z[i], top));
        }
#pragma unroll
        for (int i = 0; i < VALS; ++i) {
            sum += z[i];
            mine[expert(i)] = z[i];
        }
        meet();
#pragma unroll
        for (int c = 0; c < PER; ++c)
            if (e[c] >= 0)
                p[c] = mine[e[c]];
        meet();
    } else {
#pragma unroll
        for (int c = 0; c < PER; ++c) {
            p[c] = e[c] >= 0 ? logit<BF16>(a.logits, row + e[c]) : -INFINITY;
            top = fmaxf(top, p[c]);
        }
        top = lanes_max<LANES>(top);
#pragma unroll
        for (int c = 0; c < PER; ++c) {
            p[c] = exp_of(under(p[c], top));
            sum += p[c];
        }
    }
    sum = lanes_sum<LANES>(sum);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    float G = 0.0f;
#pragma unroll
    for (int c = 0; c < PER; ++c) {
        p[c] *= inv;
        G += p[c] > 0.0f ? p[c] * dw[c] : 0.0f;
    }
    G = lanes_sum<LANES>(G);
    // what an expert's choices sent, in their order, whichever lane has them
    float g[PER], times[PER];
#pragma unroll
    for (int c = 0; c < PER; ++c) {
        g[c] = 0.0f;
        times[c] = 1.0f;
    }
    if (a.renorm) {
#pragma unroll
        for (int c = 0; c < PER; ++c)
            times[c] = 0.0f;
#pragma unroll
        for (int cj = 0; cj < PER; ++cj)
            for (int j = 0; j < LANES && cj * LANES + j < a.K; ++j) {
                const int ej = __shfl(e[cj], j, LANES);
#pragma unroll
                for (int c = 0; c < PER; ++c)
                    times[c] += ej == e[c] ? 1.0f : 0.0f;
            }
    }
#pragma unroll
    for (int cj = 0; cj < PER; ++cj)
        for (int j = 0; j < LANES && cj * LANES + j < a.K; ++j) {
            const int ej = __shfl(e[cj], j, LANES);
            const float dj = __shfl(dw[cj], j, LANES);
#pragma unroll
            for (int c = 0; c < PER; ++c)
                g[c] += ej == e[c] ? dj : 0.0f;
        }
#pragma unroll
    for (int i = 0; i < VALS; ++i) {
        const float q = a.renorm ? 0.0f : z[i] * inv;
        mine[expert(i)] = q > 0.0f ? -q * G : 0.0f;
    }
    meet();
#pragma unroll
    for (int c = 0; c < PER; ++c)
        if (p[c] > 0.0f)
            mine[e[c]] = p[c] * g[c] - p[c] * (times[c] * G);
    meet();
    if (!live)
        return;
#pragma unroll
    for (int i = 0; i < VALS; i += W) {
        const int at = expert(i);
        if (at >= a.E)
            continue;
        float d[W];
#pragma unroll
        for (int c = 0; c < W; ++c)
            d[c] = mine[at + c];
        if (a.out_bf16) {
            uint16_t* o = (uint16_t*)a.dlogits + row + at;
            if constexpr (W == 4)
                *(v2u*)o = v2u{bf16_pack(d[0], d[1]), bf16_pack(d[2], d[3])};
            else if constexpr (W == 2)
                *(uint32_t*)o = bf16_pack(d[0], d[1]);
            else
                *o = (uint16_t)bf16_pack(d[0], 0.0f);
        } else {
            float* o = (float*)a.dlogits + row + at;
            if constexpr (W == 1) {
                *o = d[0];
            } else {
                typedef float vf __attribute__((ext_vector_type(W)));
                vf v;
#pragma unroll
                for (int c = 0; c < W; ++c)
                    v[c] = d[c];
                *(vf*)o = v;
            }
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
    auto run = [&](auto w) {
        if (a.bf16)
            topk_route_grad_kernel<LANES, VALS, w, true><<<grid, dim3(256), bytes, stream>>>(a);
        else
            topk_route_grad_kernel<LANES, VALS, w, false><<<grid, dim3(256), bytes, stream>>>(a);
    };
    // rows start where the vectors of their loads may
    if (a.E % 4 == 0)
        run(std::integral_constant<int, 4>{});
    else if (a.E % 2 == 0)
        run(std::integral_constant<int, 2>{});
    else
        run(std::integral_constant<int, 1>{});
    return hipGetLastError();
}

}  // namespace

hipError_t launch_topk_route_grad(const RouteGrad& a, hipStream_t stream)
{
    if (a.E <= 16)
        return launch<4, 4>(a, stream);
    if (a.E <= 64)
        return launch<16, 4>(a, stream);
    if (a.E <= 128)
        return launch<16, 8>(a, stream);
    if (a.E <= 256)
        return launch<16, 16>(a, stream);
    if (a.E <= 512)
        return launch<64, 8>(a, stream);
    return launch<64, 16>(a, stream);
}

}  // namespace ops
}  // namespace moe
