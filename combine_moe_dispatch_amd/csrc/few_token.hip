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
constexpr int MOE_TOKENS = WAVE;          // most tokens: a wave's lanes

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

// Lane t: whether token t names expert e, and the first of its K places that
// does.
struct Member {
    bool is;
    int k;
};

__device__ inline Member member(const FewTokens& p, const int32_t* ids, int e)
{
    const int t = threadIdx.x & (WAVE - 1);
    Member m{false, 0};
    if (t < p.T)
        for (int k = p.K - 1; k >= 0; --k)
            if (ids[t * p.K + k] == e) {
                m.is = true;
                m.k = k;
            }
    return m;
}

// The columns of one expert: entry c of `cols` is the item t*K+k (k the
// token's first place that names the expert) of the c-th token, in token
// order.  Written by one wave, lane t for token t.
__device__ inline int list_columns(const FewTokens& p, const Member& m, int32_t* cols)
{
    const int t = threadIdx.x & (WAVE - 1);
    const uint64_t mask = __ballot(m.is);
    if (m.is)
        cols[__popcll(mask & ((1ull << t) - 1))] = t * p.K + m.k;
    return __popcll(mask);
}

// What one wave wrote to its own LDS is there for its other lanes (the LDS
// instructions of a wave run in order; this only keeps the compiler from
// moving them).
__device__ inline void own_lds_written()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Coded blocks in a wave's own LDS, at a stride that spreads the reads over the
// banks: either AHEAD blocks of four columns or one block of sixteen.
constexpr int AHEAD = 2;
constexpr int FEW = 4;                    // columns of the fast path
constexpr int CODE_STRIDE = SCALE_BLOCK + 16;
struct Coded {
    uint8_t codes[16 * CODE_STRIDE];
    float scale[16];
};

// Codes four columns' block, rows row .. row+3 of `to`: 16 lanes share a
// column, eight elements each.
__device__ inline void encode8(Coded* to, int row, const float (&f)[8])
{
    const int l = threadIdx.x & 15;
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = fmaxf(top, fabsf(f[i]));
    top = max16(top);
    float inv, scale;
    block_scale(top, inv, scale);
    const v2u q{e4m3_pack4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                e4m3_pack4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)};
    const int at = row + (threadIdx.x >> 4 & 3);
    *(v2u*)(to->codes + at * CODE_STRIDE + l * 8) = q;
    if (l == 0)
        to->scale[at] = scale;
}

__device__ inline void unpack8(v4u v, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(v[i]);
        f[2 * i + 1] = bf16_hi(v[i]);
    }
}

// 32 codes of a lane's row (its 16-byte pieces g and g + 4) as fp16.
struct Half32 {
    v8h v[4];
};
__device__ inline Half32 convert32(v4u lo, v4u hi)
{
    return Half32{{e4m3_to_f16(lo.x, lo.y), e4m3_to_f16(lo.z, lo.w), e4m3_to_f16(hi.x, hi.y),
                   e4m3_to_f16(hi.z, hi.w)}};
}

__device__ inline Half32 coded_columns(const Coded* from, int r, int g)
{
    const uint8_t* row = from->codes + r * CODE_STRIDE + g * 16;
    return convert32(*(const v4u*)row, *(const v4u*)(row + 64));
}

// The block's products of 16 weight rows and 16 columns, in fp32 from zero.
__device__ inline v4f product(const Half32& a, const Half32& b)
{
    v4f t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        t = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[i], b.v[i], t, 0, 0, 0);
    return t;
}

__device__ inline v4u load16(const uint8_t* p) { return *(const v4u*)p; }

// A workgroup's waves share the blocks of a product.  Blocks go AHEAD at a
// time: the weights of the next ones are in flight while a wave works on the
// last.  Occupancy matters more than depth: four blocks ahead (two waves per
// SIMD instead of four) took 82 us for one token of a hidden-7168, 256-expert
// layer, two ahead 71.  Plain loads: with the nontemporal hint the two halves
// of a 128-byte line are fetched twice, 102 us against 82.
constexpr int GATE_WAVES = 4;
constexpr int DOWN_WAVES = 8;

// Lane (row r = l & 15, group g = l >> 4) of a 16 x 128 block of weights holds
// the 16-byte pieces g and g + 4 of row r; the columns' codes use the same
// order.

// h[t*K+k][f]: one workgroup per (distinct expert, 16 columns f); its waves
// share the blocks of H and add up through LDS.  NC: sets of 16 tokens.
template <int NC>
__global__ __launch_bounds__(GATE_WAVES* WAVE, NC == 1 ? 4 : 2) void few_gate_up_kernel(const FewTokens p, float* hbuf)
{
    extern __shared__ int32_t ids[];
    __shared__ uint32_t used[MAX_E_WORDS];
    __shared__ int32_t cols[MOE_TOKENS];
    __shared__ Coded coded[GATE_WAVES];
    __shared__ float part[GATE_WAVES][2][NC * 16][17];
    read_ids(p, ids, used);
    const int e = nth_expert(used, blockIdx.y);
    if (e < 0)
        return;
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int r = lane & 15, g = lane >> 4;
    const int KB = p.H / SCALE_BLOCK;
    const int f0 = blockIdx.x * 16;
    const uint8_t* gate = p.w13 + ((int64_t)e * 2 * p.F + f0 + r) * p.H + g * 16;
    const uint8_t* up = gate + (int64_t)p.F * p.H;
    const float* sg = p.s13 + ((int64_t)e * (2 * p.F / SCALE_BLOCK) + f0 / SCALE_BLOCK) * KB;
    const float* su = sg + (int64_t)(p.F / SCALE_BLOCK) * KB;
    const int k0 = KB * wave / GATE_WAVES, k1 = KB * (wave + 1) / GATE_WAVES;
    v4u w[AHEAD][4];
    auto fetch = [&](int kb, v4u(&to)[4]) {
        const int64_t o = (int64_t)min(kb, KB - 1) * SCALE_BLOCK;
        to[0] = load16(gate + o);
        to[1] = load16(gate + o + 64);
        to[2] = load16(up + o);
        to[3] = load16(up + o + 64);
    };
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
        fetch(k0 + u, w[u]);
    const Member me = member(p, ids, e);
    if (wave == 0)
        list_columns(p, me, cols);
    const int n = __popcll(__ballot(me.is));
    __syncthreads();
    v4f ag[NC], au[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        ag[c] = au[c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    auto columns = [&](const Half32& wg, const Half32& wu, int row, float s0, float s1, int c) {
        const Half32 q = coded_columns(&coded[wave], row, g);
        const float xs = coded[wave].scale[row];
        const v4f tg = product(wg, q), tu = product(wu, q);
        const float a0 = xs * s0, a1 = xs * s1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ag[c][i] = fmaf(tg[i], a0, ag[c][i]);
            au[c][i] = fmaf(tu[i], a1, au[c][i]);
        }
    };
    if (n <= FEW) {
        // at most four tokens (by far the most frequent): their rows come
        // ahead like the weights, and AHEAD blocks are coded at a time
        const uint16_t* xp = p.x + (int64_t)(cols[min(g, n - 1)] / p.K) * p.H + r * 8;
        v4u x[AHEAD];
        auto xrows = [&](int kb0) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                x[u] = *(const v4u*)(xp + min(kb0 + u, KB - 1) * SCALE_BLOCK);
        };
        xrows(k0);
        for (int kb0 = k0; kb0 < k1; kb0 += AHEAD) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                float f[8];
                unpack8(x[u], f);
                encode8(&coded[wave], u * FEW, f);
            }
            xrows(kb0 + AHEAD);
            own_lds_written();
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int kb = min(kb0 + u, KB - 1);
                const float live = kb0 + u < k1 ? 1.0f : 0.0f;   // a repeated block adds nothing
                const Half32 wg = convert32(w[u][0], w[u][1]), wu = convert32(w[u][2], w[u][3]);
                fetch(kb0 + u + AHEAD, w[u]);
                columns(wg, wu, u * FEW + (r & (FEW - 1)), sg[kb] * live, su[kb] * live, 0);
            }
            own_lds_written();
        }
    } else {
        for (int kb0 = k0; kb0 < k1; kb0 += AHEAD) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int kb = min(kb0 + u, KB - 1);
                const float live = kb0 + u < k1 ? 1.0f : 0.0f;
                const Half32 wg = convert32(w[u][0], w[u][1]), wu = convert32(w[u][2], w[u][3]);
                fetch(kb0 + u + AHEAD, w[u]);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    if (c * 16 >= n)
                        break;
                    const int nc = min(16, n - c * 16);
                    for (int q = 0; q < nc; q += FEW) {
                        float f[8];
                        unpack8(*(const v4u*)(p.x + (int64_t)(cols[min(c * 16 + q + g, n - 1)] / p.K) * p.H +
                                              kb * SCALE_BLOCK + r * 8),
                                f);
                        encode8(&coded[wave], q, f);
                    }
                    own_lds_written();
                    columns(wg, wu, r, sg[kb] * live, su[kb] * live, c);
                    own_lds_written();
                }
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
    __syncthreads();
    for (int v = threadIdx.x; v < n * 16; v += GATE_WAVES * WAVE) {
        const int col = v >> 4, f = v & 15;
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int q = 0; q < GATE_WAVES; ++q) {
            a += part[q][0][col][f];
            b += part[q][1][col][f];
        }
        hbuf[(int64_t)cols[col] * p.F + f0 + f] = a / (1.0f + __expf(-a)) * b;
    }
}

// out[t][n0 .. n0+15] of every token: the waves share the (expert, block of F)
// pairs in order; a wave adds an expert's finished part, times the router
// weight, to its own copy of the tile, and the copies are added in order.
template <int NC>
__global__ __launch_bounds__(DOWN_WAVES* WAVE, NC == 1 ? 4 : 2) void few_down_kernel(const FewTokens p, const float* hbuf)
{
    extern __shared__ int32_t ids[];
    __shared__ uint32_t used[MAX_E_WORDS];
    __shared__ int32_t cols[DOWN_WAVES][MOE_TOKENS];
    __shared__ float weight[DOWN_WAVES][MOE_TOKENS];
    __shared__ Coded coded[DOWN_WAVES];
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
        const int u0 = q / FB;
        const int kb0 = q - u0 * FB, kb1 = min(FB, kb0 + q1 - q);
        const int e = nth_expert(used, u0);
        const uint8_t* down = p.w2 + ((int64_t)e * p.H + n0 + r) * p.F + g * 16;
        const float* sd = p.s2 + ((int64_t)e * (p.H / SCALE_BLOCK) + n0 / SCALE_BLOCK) * FB;
        v4u w[AHEAD][2];
        auto fetch = [&](int kb, v4u(&to)[2]) {
            const int64_t o = (int64_t)min(kb, FB - 1) * SCALE_BLOCK;
            to[0] = load16(down + o);
            to[1] = load16(down + o + 64);
        };
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            fetch(kb0 + u, w[u]);
        const Member me = member(p, ids, e);
        const int n = list_columns(p, me, cols[wave]);
        if (me.is) {                            // the token's weight for this expert
            float mine = 0.0f;
            for (int k = 0; k < p.K; ++k)
                if (ids[lane * p.K + k] == e)
                    mine += p.w[lane * p.K + k];
            weight[wave][lane] = mine;
        }
        own_lds_written();
        v4f acc[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c)
            acc[c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        auto columns = [&](const Half32& wd, int row, float s0, int c) {
            const Half32 hq = coded_columns(&coded[wave], row, g);
            const float s = coded[wave].scale[row] * s0;
            const v4f t = product(wd, hq);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[c][i] = fmaf(t[i], s, acc[c][i]);
        };
        auto encode_h = [&](const v4f(&v)[2], int row) {
            const float f[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
            encode8(&coded[wave], row, f);
        };
        if (n <= FEW) {
            const float* hp = hbuf + (int64_t)cols[wave][min(g, n - 1)] * p.F + r * 8;
            v4f hv[AHEAD][2];
            auto hrows = [&](int k) {
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const v4f* h = (const v4f*)(hp + min(k + u, FB - 1) * SCALE_BLOCK);
                    hv[u][0] = h[0];
                    hv[u][1] = h[1];
                }
            };
            hrows(kb0);
            for (int k = kb0; k < kb1; k += AHEAD) {
#pragma unroll
                for (int u = 0; u < AHEAD; ++u)
                    encode_h(hv[u], u * FEW);
                hrows(k + AHEAD);
                own_lds_written();
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const float s0 = k + u < kb1 ? sd[min(k + u, FB - 1)] : 0.0f;
                    const Half32 wd = convert32(w[u][0], w[u][1]);
                    fetch(k + u + AHEAD, w[u]);
                    columns(wd, u * FEW + (r & (FEW - 1)), s0, 0);
                }
                own_lds_written();
            }
        } else {
            for (int k = kb0; k < kb1; k += AHEAD) {
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const int kb = min(k + u, FB - 1);
                    const float s0 = k + u < kb1 ? sd[kb] : 0.0f;
                    const Half32 wd = convert32(w[u][0], w[u][1]);
                    fetch(k + u + AHEAD, w[u]);
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        if (c * 16 >= n)
                            break;
                        const int nc = min(16, n - c * 16);
                        for (int i = 0; i < nc; i += FEW) {
                            const v4f* h = (const v4f*)(hbuf + (int64_t)cols[wave][min(c * 16 + i + g, n - 1)] * p.F +
                                                        kb * SCALE_BLOCK + r * 8);
                            const v4f v[2] = {h[0], h[1]};
                            encode_h(v, i);
                        }
                        own_lds_written();
                        columns(wd, r, s0, c);
                        own_lds_written();
                    }
                }
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (c * 16 + r < n) {
                const int t = cols[wave][c * 16 + r] / p.K;
                const float wt = weight[wave][t];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tile[wave][t][g * 4 + i] += wt * acc[c][i];
            }
        own_lds_written();
        q += kb1 - kb0;
    }
    __syncthreads();
    for (int v = threadIdx.x; v < p.T * 8; v += DOWN_WAVES * WAVE) {
        const int t = v >> 3, n = (v & 7) * 2;
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int q = 0; q < DOWN_WAVES; ++q) {
            a += tile[q][t][n];
            b += tile[q][t][n + 1];
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
