// A whole expert layer for a few tokens, in two kernels.
//
//   x       -> codec (e4m3, scale per 128)
//   g, u    =  block-scaled products with the chosen expert's gate / up rows
//   h       =  silu(g) * u, fp32 in the workspace -> codec
//   y       =  block-scaled product with the expert's down rows, fp32
//   out[t]  =  bf16(sum over the token's experts of w * y)
//
// With a few tokens every weight is used once or a few times, so the layer is
// a stream of the distinct chosen experts' weights; everything else (x, h,
// scales) is small and stays in L2.  Weights go from HBM straight to the
// matrix instruction's registers, 16 rows by 128 bytes per instruction; the
// tokens of an expert (16 columns at a time) are coded on the way in by every
// wave for itself, which costs the vector unit less than the wait for the
// weights, and saves a launch and a pass.
//
// Both kernels work out who needs an expert from topk_idx alone: lane t of a
// wave looks through token t's K ids (at most 64 tokens).  A token that names
// an expert twice is one column with the sum of its weights.
#include "moe_ops.h"
#include "ops_common.h"

namespace moe {
namespace ops {
namespace {

constexpr int MAX_E_WORDS = 1024 / 32;

// The ids of all tokens in LDS, -1 where outside [0, E), and the set of
// experts they name.  Contains barriers.
__device__ inline void read_ids(const FewTokens& p, int32_t* ids, uint32_t* used)
{
    for (int i = threadIdx.x; i < MAX_E_WORDS; i += blockDim.x)
        used[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * p.K; i += blockDim.x) {
        const int e = p.idx[i];
        const bool ok = (unsigned)e < (unsigned)p.E;
        ids[i] = ok ? e : -1;
        if (ok)
            atomicOr(&used[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
}

// The u-th (from 0) expert of the set, -1 past the last; every wave finds it
// for itself.
__device__ inline int nth_expert(const uint32_t* used, int u)
{
    const int lane = threadIdx.x & (WAVE - 1);
    const uint32_t word = lane < MAX_E_WORDS ? used[lane] : 0;
    int incl = __popc(word);
#pragma unroll
    for (int d = 1; d < MAX_E_WORDS; d <<= 1) {
        const int o = __shfl_up(incl, d, WAVE);
        if (lane >= d)
            incl += o;
    }
    const uint64_t upto = __ballot(incl > u);
    if (upto == 0)
        return -1;
    const int src = __ffsll((unsigned long long)upto) - 1;
    uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)word, src);
    const int before = __builtin_amdgcn_readlane(incl, src) - __popc(w);
    for (int i = before; i < u; ++i)
        w &= w - 1;
    return src * 32 + __ffs((int)w) - 1;
}

__device__ inline int count_experts(const uint32_t* used)
{
    int n = 0;
    for (int i = 0; i < MAX_E_WORDS; ++i)
        n += __popc(used[i]);
    return n;
}

// Lane t: whether token t names expert e, the first of its K places that does,
// and the sum of the weights of all that do.
struct Member {
    bool is;
    int k;
    float w;
};

__device__ inline Member member(const FewTokens& p, const int32_t* ids, int e)
{
    const int t = threadIdx.x & (WAVE - 1);
    Member m{false, 0, 0.0f};
    if (t < p.T)
        for (int k = p.K - 1; k >= 0; --k)
            if (ids[t * p.K + k] == e) {
                m.is = true;
                m.k = k;
            }
    return m;
}

// Column c's token: the c-th set bit of the members' mask (lanes past the
// last take the last one; what they compute is dropped).
__device__ inline int nth_bit(uint64_t mask, int c)
{
    for (int i = 0; i < c; ++i) {
        const uint64_t rest = mask & (mask - 1);
        mask = rest ? rest : mask;
    }
    return __ffsll((unsigned long long)mask) - 1;
}

// 32 fp32 values of one token's block of 128 held by four lanes (l, l+16,
// l+32, l+48): their codes' values as fp16 (the codec's rounding, then an
// exact conversion for the matrix instruction), and the block scale.
__device__ inline void encode32(const float (&f)[32], v8h (&q)[4], float& scale)
{
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        top = fmaxf(top, fabsf(f[i]));
    top = fmaxf(top, __shfl_xor(top, 16, WAVE));
    top = fmaxf(top, __shfl_xor(top, 32, WAVE));
    float inv;
    block_scale(top, inv, scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float* v = f + 8 * i;
        q[i] = e4m3_to_f16(e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                           e4m3_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    }
}

// A lane's two 16-byte pieces of a weight row as fp16.
__device__ inline void convert32(v4u lo, v4u hi, v8h (&w)[4])
{
    w[0] = e4m3_to_f16(lo.x, lo.y);
    w[1] = e4m3_to_f16(lo.z, lo.w);
    w[2] = e4m3_to_f16(hi.x, hi.y);
    w[3] = e4m3_to_f16(hi.z, hi.w);
}

// The block's products of 16 weight rows and 16 columns, in fp32 from zero.
__device__ inline v4f product(const v8h (&a)[4], const v8h (&b)[4])
{
    v4f t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        t = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[i], b[i], t, 0, 0, 0);
    return t;
}

__device__ inline v4u ld_nt(const uint8_t* p) { return __builtin_nontemporal_load((const v4u*)p); }

// Lane (row r = l & 15, group g = l >> 4) of a 16 x 128 block holds the
// 16-byte pieces g and g + 4 of row r; the token's codes use the same order.
constexpr int GATE_WAVES = 4;
constexpr int DOWN_WAVES = 8;

// h[t*K+k][f]: one workgroup per (distinct expert, 16 columns f); its waves
// share the blocks of H and add up through LDS.  NC: 16-token columns sets.
template <int NC>
__global__ __launch_bounds__(GATE_WAVES* WAVE) void few_gate_up_kernel(const FewTokens p, float* hbuf)
{
    extern __shared__ int32_t ids[];
    __shared__ uint32_t used[MAX_E_WORDS];
    __shared__ float part[GATE_WAVES][2][NC * 16][17];
    read_ids(p, ids, used);
    const int e = nth_expert(used, blockIdx.y);
    if (e < 0)
        return;
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int r = lane & 15, g = lane >> 4;
    const Member me = member(p, ids, e);
    const uint64_t mask = __ballot(me.is);
    const int n = __popcll(mask);
    int tok[NC], item[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        tok[c] = nth_bit(mask, c * 16 + r);
        item[c] = tok[c] * p.K + __shfl(me.k, tok[c], WAVE);
    }
    const int KB = p.H / SCALE_BLOCK;
    const int f0 = blockIdx.x * 16;
    const uint8_t* gate = p.w13 + ((int64_t)e * 2 * p.F + f0 + r) * p.H + g * 16;
    const uint8_t* up = gate + (int64_t)p.F * p.H;
    const float* sg = p.s13 + ((int64_t)e * (2 * p.F / SCALE_BLOCK) + f0 / SCALE_BLOCK) * KB;
    const float* su = sg + (int64_t)(p.F / SCALE_BLOCK) * KB;
    v4f ag[NC], au[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        ag[c] = au[c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int k0 = KB * wave / GATE_WAVES, k1 = KB * (wave + 1) / GATE_WAVES;
    for (int kb = k0; kb < k1; ++kb) {
        const int64_t o = (int64_t)kb * SCALE_BLOCK;
        v8h wg[4], wu[4];
        convert32(ld_nt(gate + o), ld_nt(gate + o + 64), wg);
        convert32(ld_nt(up + o), ld_nt(up + o + 64), wu);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (c * 16 >= n)
                break;
            const uint16_t* xr = p.x + (int64_t)tok[c] * p.H + o + g * 16;
            const v4u a[4] = {((const v4u*)xr)[0], ((const v4u*)xr)[1], ((const v4u*)(xr + 64))[0],
                              ((const v4u*)(xr + 64))[1]};
            float f[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                f[2 * i] = bf16_lo(a[i / 4][i % 4]);
                f[2 * i + 1] = bf16_hi(a[i / 4][i % 4]);
            }
            float xs;
            v8h q[4];
            encode32(f, q, xs);
            const v4f tg = product(wg, q), tu = product(wu, q);
            const float a0 = xs * sg[kb], a1 = xs * su[kb];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ag[c][i] = fmaf(tg[i], a0, ag[c][i]);
                au[c][i] = fmaf(tu[i], a1, au[c][i]);
            }
        }
    }
    // lane (r, g) has rows 4g .. 4g+3 of column r
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            part[wave][0][c * 16 + r][g * 4 + i] = ag[c][i];
            part[wave][1][c * 16 + r][g * 4 + i] = au[c][i];
        }
    __shared__ int items[NC * 16];
    if (wave == 0 && g == 0)
#pragma unroll
        for (int c = 0; c < NC; ++c)
            items[c * 16 + r] = item[c];
    __syncthreads();
    for (int v = threadIdx.x; v < n * 16; v += GATE_WAVES * WAVE) {
        const int col = v >> 4, f = v & 15;
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int w = 0; w < GATE_WAVES; ++w) {
            a += part[w][0][col][f];
            b += part[w][1][col][f];
        }
        hbuf[(int64_t)items[col] * p.F + f0 + f] = a / (1.0f + __expf(-a)) * b;
    }
}

// out[t][n0 .. n0+15] of every token: the waves share the (expert, block of F)
// pairs in order; a wave adds an expert's finished part, times the router
// weight, to its own copy of the tile, and the copies are added in order.
template <int NC>
__global__ __launch_bounds__(DOWN_WAVES* WAVE) void few_down_kernel(const FewTokens p, const float* hbuf)
{
    extern __shared__ int32_t ids[];
    __shared__ uint32_t used[MAX_E_WORDS];
    __shared__ float tile[DOWN_WAVES][NC * 16][17];
    for (int i = threadIdx.x; i < DOWN_WAVES * NC * 16 * 17; i += DOWN_WAVES * WAVE)
        (&tile[0][0][0])[i] = 0.0f;
    read_ids(p, ids, used);
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int r = lane & 15, g = lane >> 4;
    const int FB = p.F / SCALE_BLOCK;
    const int n0 = blockIdx.x * 16;
    const int pairs = count_experts(used) * FB;
    const int q0 = (int)((int64_t)pairs * wave / DOWN_WAVES), q1 = (int)((int64_t)pairs * (wave + 1) / DOWN_WAVES);
    for (int q = q0; q < q1;) {
        const int u = q / FB;
        const int kb0 = q - u * FB, kb1 = min(FB, kb0 + q1 - q);
        const int e = nth_expert(used, u);
        const Member me = member(p, ids, e);
        const uint64_t mask = __ballot(me.is);
        const int n = __popcll(mask);
        float mine = 0.0f;                      // the token's weight for this expert
        if (me.is)
            for (int k = 0; k < p.K; ++k)
                if (ids[lane * p.K + k] == e)
                    mine += p.w[lane * p.K + k];
        int tok[NC], item[NC];
        v4f acc[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            tok[c] = nth_bit(mask, c * 16 + r);
            item[c] = tok[c] * p.K + __shfl(me.k, tok[c], WAVE);
            acc[c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const uint8_t* down = p.w2 + ((int64_t)e * p.H + n0 + r) * p.F + g * 16;
        const float* sd = p.s2 + ((int64_t)e * (p.H / SCALE_BLOCK) + n0 / SCALE_BLOCK) * FB;
        for (int kb = kb0; kb < kb1; ++kb) {
            const int64_t o = (int64_t)kb * SCALE_BLOCK;
            v8h wd[4];
            convert32(ld_nt(down + o), ld_nt(down + o + 64), wd);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (c * 16 >= n)
                    break;
                const float* hr = hbuf + (int64_t)item[c] * p.F + o + g * 16;
                float f[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const v4f v = ((const v4f*)(hr + (i < 4 ? 0 : 64)))[i % 4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        f[4 * i + j] = v[j];
                }
                float hs;
                v8h hq[4];
                encode32(f, hq, hs);
                const v4f t = product(wd, hq);
                const float s = hs * sd[kb];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[c][i] = fmaf(t[i], s, acc[c][i]);
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float w = __shfl(mine, tok[c], WAVE);
            if (c * 16 + r < n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tile[wave][tok[c]][g * 4 + i] += w * acc[c][i];
        }
        q += kb1 - kb0;
    }
    __syncthreads();
    for (int v = threadIdx.x; v < p.T * 8; v += DOWN_WAVES * WAVE) {
        const int t = v >> 3, n = (v & 7) * 2;
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int w = 0; w < DOWN_WAVES; ++w) {
            a += tile[w][t][n];
            b += tile[w][t][n + 1];
        }
        *(uint32_t*)(p.out + (int64_t)t * p.H + n0 + n) = bf16_pack(a, b);
    }
}

template <int NC>
hipError_t few(const FewTokens& p, hipStream_t stream)
{
    float* hbuf = (float*)p.workspace;
    const int experts = p.T * p.K < p.E ? p.T * p.K : p.E;     // distinct ones, at most
    const uint32_t ids = (uint32_t)(p.T * p.K) * 4;
    few_gate_up_kernel<NC><<<dim3(p.F / 16, experts), dim3(GATE_WAVES * WAVE), ids, stream>>>(p, hbuf);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    few_down_kernel<NC><<<dim3(p.H / 16), dim3(DOWN_WAVES * WAVE), ids, stream>>>(p, hbuf);
    return hipGetLastError();
}

}  // namespace

size_t few_token_workspace(int T, int K, int H, int F)
{
    (void)H;
    return (size_t)T * K * F * sizeof(float);
}

hipError_t launch_few_token_layer(const FewTokens& p, hipStream_t stream)
{
    if (p.T == 0)
        return hipSuccess;
    if (p.T <= 16)
        return few<1>(p, stream);
    if (p.T <= 32)
        return few<2>(p, stream);
    return few<4>(p, stream);
}

}  // namespace ops
}  // namespace moe
