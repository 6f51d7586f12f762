// Per-token operators ahead of dispatch: residual addition with RMS norm (and
// the dispatch codec's e4m3 rows), and the choice of a token's experts.
#include "moe_ops.h"
#include "ops_common.h"

namespace moe {
namespace ops {
namespace {

// STREAM: the nontemporal hint, for rows that no cache will hold.
template <bool STREAM>
__device__ inline v4u load_row(const v4u* p)
{
    return STREAM ? __builtin_nontemporal_load(p) : *p;
}
template <bool STREAM>
__device__ inline void store_row(const v4u& v, v4u* p)
{
    if (STREAM)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}

// ---------------------------------------------------------------------------
// s = x + residual (fp32); y = s / sqrt(mean(s^2) + eps) * weight.
//
// One pass: a row is read once, stays in registers as fp32 (V vectors of 8
// elements per thread) through the sum of squares, and every output is
// written from there.  A row belongs to one or more waves, a short one to LANES
// lanes of a wave; the norm is of the fp32 sum,
// not of its bf16 rounding, and the codes are of the fp32 result, not of y's
// bf16 rounding, so each output is rounded once.
//
// Where mean(s^2) + eps is below 2^-100, squares may have left fp32's range
// (s below 2^-63 in a row with an eps as small): the sum is then that of (2^80
// s)^2, with 2^160 eps, and y = 2^80 s / its root.  A wave forms it where its
// own share of the sum is below 2^-80, which holds for every wave of such a
// row (65536 * 2^-100 at most); its largest square is then below 2^80, its
// smallest 2^-106 (bf16's smallest number is 2^-133).
// ---------------------------------------------------------------------------
struct NormArgs {
    int64_t rows;
    int hidden, vecs;         // vecs: 8-element vectors per row
    const uint16_t* x;
    const uint16_t* residual;
    const uint16_t* weight;
    float eps;
    uint16_t* residual_out;
    uint16_t* y;
    uint8_t* yq;
    float* ys;
};

// STREAM: 0 plain accesses, 1 the nontemporal hint for all rows but x, which the
// operator before has just written, 2 for x too.
template <int V, int STREAM, int LANES>
__global__ __launch_bounds__(1024) void add_rmsnorm_kernel(const NormArgs a, int waves_per_row)
{
    __shared__ float part[2][16];
    const int lane = threadIdx.x % LANES;
    const int wave = threadIdx.x / LANES;
    const int per_block = blockDim.x / LANES / waves_per_row;
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t row = block * per_block + wave / waves_per_row;
    const int t = (wave % waves_per_row) * LANES + lane;     // thread of the row
    const int nt = waves_per_row * LANES;
    const bool live = row < a.rows;
    const int64_t at = row * a.hidden;
    float s[V][8];
    float sum = 0.0f;
    v4u xv[V], rv[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int v = u * nt + t;
        xv[u] = rv[u] = v4u{0, 0, 0, 0};
        if (live && v < a.vecs) {
            xv[u] = load_row<STREAM == 2>((const v4u*)(a.x + at) + v);
            if (a.residual)
                rv[u] = load_row<(STREAM > 0)>((const v4u*)(a.residual + at) + v);
        }
    }
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            s[u][2 * c] = bf16_lo(xv[u][c]) + bf16_lo(rv[u][c]);
            s[u][2 * c + 1] = bf16_hi(xv[u][c]) + bf16_hi(rv[u][c]);
            sum = fmaf(s[u][2 * c], s[u][2 * c], sum);
            sum = fmaf(s[u][2 * c + 1], s[u][2 * c + 1], sum);
        }
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1)
        sum += __shfl_xor(sum, d, LANES);
    constexpr float UP = 0x1p80f;
    float small = 0.0f;                  // the sum of (UP s)^2, where sum is below 2^-80
    if (sum < 0x1p-80f) {
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                small = fmaf(s[u][c] * UP, s[u][c] * UP, small);
#pragma unroll
        for (int d = LANES / 2; d; d >>= 1)
            small += __shfl_xor(small, d, LANES);
    }
    if (LANES == WAVE && waves_per_row > 1) {
        if (lane == 0) {
            part[0][wave] = sum;
            part[1][wave] = small;
        }
        __syncthreads();
        sum = small = 0.0f;
        const int w0 = wave / waves_per_row * waves_per_row;
        for (int w = 0; w < waves_per_row; ++w) {
            sum += part[0][w0 + w];
            small += part[1][w0 + w];
        }
    }
    float mean = sum / (float)a.hidden + a.eps, up = 1.0f;
    if (mean < 0x1p-100f) {
        mean = small / (float)a.hidden + a.eps * UP * UP;
        up = UP;
    }
    const float r = 1.0f / sqrtf(mean);
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int v = u * nt + t;
        const bool mine = live && v < a.vecs;
        v4u wv{0, 0, 0, 0};
        if (mine) {
            wv = ((const v4u*)a.weight)[v];
            if (a.residual_out) {
                v4u o;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    o[c] = bf16_pack(s[u][2 * c], s[u][2 * c + 1]);
                store_row<true>(o, (v4u*)(a.residual_out + at) + v);      // not read soon
            }
        }
        if (up != 1.0f)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                s[u][c] *= up;
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            s[u][2 * c] = s[u][2 * c] * r * bf16_lo(wv[c]);        // |s r| is sqrt(hidden) at most
            s[u][2 * c + 1] = s[u][2 * c + 1] * r * bf16_hi(wv[c]);
            top = fmaxf(top, fmaxf(fabsf(s[u][2 * c]), fabsf(s[u][2 * c + 1])));
        }
        if (mine && a.y) {
            v4u o;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                o[c] = bf16_pack(s[u][2 * c], s[u][2 * c + 1]);
            store_row<(STREAM > 0)>(o, (v4u*)(a.y + at) + v);
        }
        if (a.yq) {
            // a block of 128 is 16 consecutive lanes
            top = max16(top);
            float inv, scale;
            block_scale(top, inv, scale);
            if (mine) {
                const v2u q{e4m3_pack4(s[u][0] * inv, s[u][1] * inv, s[u][2] * inv, s[u][3] * inv),
                            e4m3_pack4(s[u][4] * inv, s[u][5] * inv, s[u][6] * inv, s[u][7] * inv)};
                ((v2u*)(a.yq + at))[v] = q;
                if ((v & 15) == 0)
                    a.ys[row * (a.hidden / SCALE_BLOCK) + (v >> 4)] = scale;
            }
        }
    }
}

// What the lanes of a group trade when a reduction joins neighbours, then
// pairs, fours and so on: the other half's value (mirrored inside a row of 16,
// whose parts hold one value each by then).
template <int CTRL>
struct RowTrade {
    __device__ inline int operator()(int v) const { return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true); }
    __device__ inline float operator()(float v) const { return __int_as_float((*this)(__float_as_int(v))); }
};
template <int D>
struct WaveTrade {
    template <class T>
    __device__ inline T operator()(T v) const { return __shfl_xor(v, D, WAVE); }
};
template <int G, class Step>
__device__ inline void across(Step step)
{
    if constexpr (G > 1)
        step(RowTrade<0xB1>{});
    if constexpr (G > 2)
        step(RowTrade<0x4E>{});
    if constexpr (G > 4)
        step(RowTrade<0x141>{});
    if constexpr (G > 8)
        step(RowTrade<0x140>{});
    if constexpr (G > 16)
        step(WaveTrade<16>{});
    if constexpr (G > 32)
        step(WaveTrade<32>{});
}

// ---------------------------------------------------------------------------
// A token's K best experts and their softmax weights.  G lanes share a token,
// lane l of them holds experts l, l+G, ...; K times: the largest logit left
// (lowest expert among equals) is taken out.  NaN counts as -infinity.
//
// The chosen experts' exp(z - top) are as good as fp32 holds them.  The sum of
// all takes the plain base-2 exponential, whose error |z - top| 2^-24 counts
// there by its mean under the softmax: at most 5 * 2^-24 with 1024 experts,
// less than the additions' roundings.
// ---------------------------------------------------------------------------
template <int G, int V, bool BF16>
__global__ __launch_bounds__(256) void topk_route_kernel(int64_t tokens, int E, int K, const void* logits,
                                                         int renorm, int32_t* idx, float* w)
{
    constexpr int PER = 256 / G;
    const int l = threadIdx.x % G;
    const int64_t tok = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * PER + threadIdx.x / G;
    const int64_t row = (tok < tokens ? tok : tokens - 1) * E;
    float z[V];
    bool gone[V];                 // taken, or past the last expert
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * G + l;
        z[i] = -INFINITY;
        gone[i] = e >= E;
        if (e < E) {
            if (BF16)
                z[i] = __uint_as_float((uint32_t)((const uint16_t*)logits)[row + e] << 16);
            else
                z[i] = ((const float*)logits)[row + e];
            if (z[i] != z[i])
                z[i] = -INFINITY;
        }
        top = fmaxf(top, z[i]);
    }
    across<G>([&](auto trade) { top = fmaxf(top, trade(top)); });
    // p(z) = exp(z - top); infinite tops share the whole weight
    auto p = [&](float v, auto exp) {
        if (top == -INFINITY)
            return 0.0f;
        return v == top ? 1.0f : exp(v - top);
    };
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
        sum += i * G + l < E ? p(z[i], [](float d) { return __expf(d); }) : 0.0f;
    across<G>([&](auto trade) { sum += trade(sum); });
    float best_sum = 0.0f, mine = 0.0f;      // the sum of this lane's picks
    int mine_e = 0;
    for (int k = 0; k < K; ++k) {
        float bz = -INFINITY;
        int be = 1 << 30;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (!gone[i] && z[i] >= bz) {
                bz = z[i];
                be = i * G + l;
            }
        across<G>([&](auto trade) {
            const float oz = trade(bz);
            const int oe = trade(be);
            const bool better = oz > bz || (oz == bz && oe < be);
            bz = better ? oz : bz;
            be = better ? oe : be;
        });
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * G + l == be)
                gone[i] = true;
        const float v = p(bz, [](float d) { return exp_of(d); });
        // lane k % G keeps pick k and writes it when it must
        if (k % G == l) {
            best_sum += v;
            mine = v;
            mine_e = be;
        }
        if ((k % G == G - 1 || k == K - 1)) {
            const int k0 = k / G * G;
            if (tok < tokens && k0 + l <= k) {
                idx[tok * K + k0 + l] = mine_e;
                if (K > G)
                    w[tok * K + k0 + l] = mine;
            }
        }
    }
    across<G>([&](auto trade) { best_sum += trade(best_sum); });
    const float total = renorm ? best_sum : sum;
    const float scale = total > 0.0f ? 1.0f / total : 0.0f;
    if (tok < tokens)
        for (int k = l; k < K; k += G)
            w[tok * K + k] = (K > G ? w[tok * K + k] : mine) * scale;
}

// Floats as unsigned numbers in the same order; -0 as +0, NaN as -infinity.
// 0 is below all of them.
__device__ inline uint32_t ordered(float v)          // not for NaN and -0
{
    const uint32_t u = __float_as_uint(v);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ inline uint32_t order_of(float v) { return ordered(v == v ? v + 0.0f : -INFINITY); }
__device__ inline float value_of(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// Logits e .. e+3 of a row (-infinity past its end) as one load, whatever the
// row's alignment; WHOLE: E is a multiple of 4, else the row's last ones are
// loaded singly (that second path costs the whole rows 5-30%; 20000 tokens of
// 511 experts took 24 us with single loads, 21 with these).
template <bool BF16, bool WHOLE>
__device__ inline v4f four_logits(const void* logits, int64_t row, int e, int E)
{
    typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint32_t v2u_any __attribute__((ext_vector_type(2), aligned(2)));
    v4f v{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (e + (WHOLE ? 0 : 3) < E) {
        if (BF16) {
            const v2u b = *(const v2u_any*)((const uint16_t*)logits + row + e);
            v = v4f{bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y)};
        } else {
            v = *(const v4f_any*)((const float*)logits + row + e);
        }
    } else if (!WHOLE && e < E) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (e + c < E)
                v[c] = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)logits)[row + e + c] << 16)
                            : ((const float*)logits)[row + e + c];
    }
    return v;
}

// The same with a wave per token, for E <= 64 V: lane l holds experts
// l*V .. l*V+V-1, sorted once (largest first, stable).  A pick is then the
// largest of the lanes' heads, the lowest lane among equals (its experts are
// the lowest), and one shift of that lane's list; lists end in 0.  The logits
// are compared as ordered unsigned numbers, whose maximum is one instruction
// across lanes too.
template <int V, bool BF16, bool WHOLE>
__global__ __launch_bounds__(256) void topk_route_wave_kernel(int64_t tokens, int E, int K, const void* logits,
                                                              int renorm, int32_t* idx, float* w)
{
    const int lane = threadIdx.x & (WAVE - 1);
    const int64_t tok = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 + threadIdx.x / WAVE;
    if (tok >= tokens)
        return;
    float z[V];
    const int e0 = lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const v4f v = four_logits<BF16, WHOLE>(logits, tok * E, e0 + i, E);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            z[i + c] = v[c];
    }
    uint32_t key[V], best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        key[i] = e0 + i < E ? order_of(z[i]) : 0;
        best = max(best, key[i]);
    }
    const float top = value_of(wave_max(best));
    // p(z) = exp(z - top); infinite tops share the whole weight, and a token
    // with nothing but -infinity has none
    auto below = [&](float v) { return v == top ? 0.0f : v - top; };
    const bool none = top == -INFINITY;
    float sum = 0.0f;
    if (!renorm) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            sum += key[i] ? __expf(below(value_of(key[i]))) : 0.0f;
        sum = wave_sum(sum);
    }
    int at[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        at[i] = i;
#pragma unroll
    for (int n = V - 1; n > 0; --n)
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t a = key[i], b = key[i + 1];
            const int c = at[i], d = at[i + 1];
            key[i] = max(a, b);
            key[i + 1] = min(a, b);
            at[i] = a < b ? d : c;
            at[i + 1] = a < b ? c : d;
        }
    uint32_t order = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        order |= (uint32_t)at[i] << (4 * i);
    uint32_t mine = 0;
    int mine_e = 0;
    for (int k = 0; k < K; ++k) {
        const uint32_t pick = wave_max(key[0]);
        const int src = __builtin_ctzll(__ballot(key[0] == pick));
        const int e = src * V + (__builtin_amdgcn_readlane((int)order, src) & 15);
        mine = lane == k ? pick : mine;
        mine_e = lane == k ? e : mine_e;
        const uint32_t win = lane == src ? ~0u : 0u;     // a bit select per entry
#pragma unroll
        for (int i = 0; i + 1 < V; ++i)
            key[i] = (key[i + 1] & win) | (key[i] & ~win);
        key[V - 1] &= ~win;
        order >>= win & 4;
    }
    const float v = lane < K ? exp_of(below(value_of(mine))) : 0.0f;
    if (renorm)
        sum = wave_sum(v);
    if (lane < K) {
        idx[tok * K + lane] = mine_e;
        w[tok * K + lane] = none ? 0.0f : v / sum;
    }
}

// The same for up to 16 choices, four tokens per wave: a row of 16 lanes per
// token, LISTS sorted lists of four experts per lane, so that the rounds'
// instructions serve four tokens (a whole wave's maximum takes six steps and
// a scalar trip for one).  The vector unit bounds both.
template <int LISTS, bool BF16, bool WHOLE>
__global__ __launch_bounds__(256) void topk_route_rows_kernel(int64_t tokens, int E, int K, const void* logits,
                                                              int renorm, int32_t* idx, float* w)
{
    const int l = threadIdx.x & 15;
    const int64_t tok = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 16 + threadIdx.x / 16;
    const int64_t row = (tok < tokens ? tok : tokens - 1) * E;
    const int e0 = l * 4 * LISTS;                 // this lane's experts: e0 .. e0 + 4*LISTS - 1
    float z[LISTS][4];
#pragma unroll
    for (int j = 0; j < LISTS; ++j) {
        const v4f v = four_logits<BF16, WHOLE>(logits, row, e0 + 4 * j, E);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            z[j][c] = v[c] == v[c] ? v[c] + 0.0f : -INFINITY;
    }
    float top = z[0][0];
#pragma unroll
    for (int j = 0; j < LISTS; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            top = fmaxf(top, z[j][c]);
    across<16>([&](auto trade) { top = fmaxf(top, trade(top)); });
    // p(z) = exp(z - top); infinite tops share the whole weight (the minimum of
    // NaN and 0 is 0), and a token with nothing but -infinity has none
    auto below = [&](float v) { return fminf(v - top, 0.0f); };
    const bool none = top == -INFINITY;
    float sum = 0.0f;
    if (!renorm) {
#pragma unroll
        for (int j = 0; j < LISTS; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                sum += __expf(below(z[j][c]));
        across<16>([&](auto trade) { sum += trade(sum); });
    }
    uint32_t key[LISTS][4];
#pragma unroll
    for (int j = 0; j < LISTS; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            key[j][c] = ordered(z[j][c]) & (e0 + 4 * j + c < E ? ~0u : 0u);
    auto row_max = [](uint32_t v) {
        across<16>([&](auto trade) { v = max(v, (uint32_t)trade((int)v)); });
        return v;
    };
    uint32_t at[LISTS];                           // a list's experts, two bits each
#pragma unroll
    for (int j = 0; j < LISTS; ++j) {
        uint32_t i[4] = {0, 1, 2, 3};
#pragma unroll
        for (int n = 3; n > 0; --n)
#pragma unroll
            for (int c = 0; c < n; ++c) {
                const uint32_t a = key[j][c], b = key[j][c + 1], ia = i[c], ib = i[c + 1];
                key[j][c] = max(a, b);
                key[j][c + 1] = min(a, b);
                i[c] = a < b ? ib : ia;
                i[c + 1] = a < b ? ia : ib;
            }
        at[j] = i[0] | i[1] << 2 | i[2] << 4 | i[3] << 6;
    }
    const int lane = threadIdx.x & (WAVE - 1);
    const uint32_t before = (0xFFFFu << (lane & 16)) & ((1u << (lane & 31)) - 1);   // lanes of the row below this one
    int32_t* out = idx + tok * K;
    uint32_t mine = 0;
    for (int k = 0; k < K; ++k) {
        uint32_t head = key[0][0];
#pragma unroll
        for (int j = 1; j < LISTS; ++j)
            head = max(head, key[j][0]);
        const uint32_t pick = row_max(head);
        const uint64_t have = __ballot(head == pick);
        const uint32_t half = lane < 32 ? (uint32_t)have : (uint32_t)(have >> 32);
        bool win = head == pick && (half & before) == 0;
        const bool write = win && tok < tokens;
        int e = e0;
#pragma unroll
        for (int j = 0; j < LISTS; ++j) {
            const bool here = win && key[j][0] == pick;      // the first list that has it
            win = win && !here;
            e = here ? e0 + 4 * j + (int)(at[j] & 3) : e;
#pragma unroll
            for (int c = 0; c < 3; ++c)
                key[j][c] = here ? key[j][c + 1] : key[j][c];
            key[j][3] = here ? 0 : key[j][3];
            at[j] >>= here ? 2 : 0;
        }
        if (write)
            out[k] = e;
        mine = l == k ? pick : mine;
    }
    const float v = l < K ? exp_of(below(value_of(mine))) : 0.0f;
    if (renorm) {
        sum = v;
        across<16>([&](auto trade) { sum += trade(sum); });
    }
    if (l < K && tok < tokens)
        w[tok * K + l] = none ? 0.0f : v / sum;
}

// `blocks` workgroups as a grid whose dimensions times the threads stay below 2^32.
inline dim3 grid_of(int64_t blocks)
{
    constexpr int64_t ROW = 1 << 20;
    return dim3((uint32_t)(blocks < ROW ? blocks : ROW), (uint32_t)((blocks + ROW - 1) / ROW));
}

}  // namespace

template <int V, int STREAM, int LANES>
static hipError_t norm_lanes(const NormArgs& a, hipStream_t stream)
{
    constexpr int PER = 256 / LANES;
    add_rmsnorm_kernel<V, STREAM, LANES><<<grid_of((a.rows + PER - 1) / PER), dim3(256), 0, stream>>>(a, 1);
    return hipGetLastError();
}

// short rows: several to a workgroup of up to four waves
template <int V, int STREAM>
static hipError_t norm_waves(const NormArgs& a, int waves, hipStream_t stream)
{
    const int per = waves < 4 ? 4 / waves : 1;
    add_rmsnorm_kernel<V, STREAM, WAVE>
        <<<grid_of((a.rows + per - 1) / per), dim3(per * waves * WAVE), 0, stream>>>(a, waves);
    return hipGetLastError();
}

template <int STREAM>
static hipError_t norm(const NormArgs& a, hipStream_t stream)
{
    // Up to 512 elements, some lanes of a wave per row: 65536 rows of 32 with a
    // residual 7.5 us against 26 with a wave each, of 128 with codes 13.6 against
    // 36, of 384 23.8 against 38.
    if (a.vecs <= 4)
        return norm_lanes<1, STREAM, 4>(a, stream);
    if (a.vecs <= 16)
        return norm_lanes<1, STREAM, 16>(a, stream);
    if (a.vecs <= 64)
        return norm_lanes<4, STREAM, 16>(a, stream);
    const int waves = (a.vecs + 2 * WAVE - 1) / (2 * WAVE);     // at two vectors per thread
    return waves <= 16 ? norm_waves<2, STREAM>(a, waves, stream) : norm_waves<8, STREAM>(a, 16, stream);
}

hipError_t launch_add_rmsnorm(int64_t rows, int hidden, const uint16_t* x, const uint16_t* residual,
                              const uint16_t* weight, float eps, uint16_t* residual_out, uint16_t* y,
                              uint8_t* yq, float* ys, hipStream_t stream)
{
    if (rows == 0)
        return hipSuccess;
    const NormArgs a{rows, hidden, hidden / 8, x, residual, weight, eps, residual_out, y, yq, ys};
    // What no cache will hold is streamed.  Inputs beyond the 256 MB of the
    // memory-side cache, all of them: 65536 rows of 4096, 512 MB, take 171 us with
    // the hint, 180 without, 174 with x left out.  Beyond half of it, inputs and
    // outputs together, all but x: 4096 rows of 7168 with a residual and codes
    // (265 MB) take 45 us where each call has rows of its own and 46 where all
    // have the same ones; without the hint 52 and 42, with x too 46 and 48.
    const int64_t each = rows * hidden * 2;
    const int64_t in = each * (residual ? 2 : 1);
    const int64_t all = in + (residual_out ? each : 0) + (y ? each : 0) + (yq ? each / 2 : 0);
    if (in > (int64_t)256 << 20)
        return norm<2>(a, stream);
    return all > (int64_t)128 << 20 ? norm<1>(a, stream) : norm<0>(a, stream);
}

template <int G, int V>
static hipError_t route(int64_t tokens, int E, int K, const void* logits, int bf16, int renorm, int32_t* idx,
                        float* w, hipStream_t stream)
{
    const int64_t grid = (tokens + 256 / G - 1) / (256 / G);
    if (bf16)
        topk_route_kernel<G, V, true><<<grid_of(grid), dim3(256), 0, stream>>>(tokens, E, K, logits,
                                                                                     renorm, idx, w);
    else
        topk_route_kernel<G, V, false><<<grid_of(grid), dim3(256), 0, stream>>>(tokens, E, K, logits,
                                                                                      renorm, idx, w);
    return hipGetLastError();
}

template <int V>
static hipError_t route_wave(int64_t tokens, int E, int K, const void* logits, int bf16, int renorm,
                             int32_t* idx, float* w, hipStream_t stream)
{
    const dim3 grid = grid_of((tokens + 3) / 4), block(256);
    auto launch = [&](auto kernel) { kernel<<<grid, block, 0, stream>>>(tokens, E, K, logits, renorm, idx, w); };
    if (E % 4 == 0)
        launch(bf16 ? topk_route_wave_kernel<V, true, true> : topk_route_wave_kernel<V, false, true>);
    else
        launch(bf16 ? topk_route_wave_kernel<V, true, false> : topk_route_wave_kernel<V, false, false>);
    return hipGetLastError();
}

template <int LISTS>
static hipError_t route_rows(int64_t tokens, int E, int K, const void* logits, int bf16, int renorm,
                             int32_t* idx, float* w, hipStream_t stream)
{
    const dim3 grid = grid_of((tokens + 15) / 16), block(256);
    auto launch = [&](auto kernel) { kernel<<<grid, block, 0, stream>>>(tokens, E, K, logits, renorm, idx, w); };
    if (E % 4 == 0)
        launch(bf16 ? topk_route_rows_kernel<LISTS, true, true> : topk_route_rows_kernel<LISTS, false, true>);
    else
        launch(bf16 ? topk_route_rows_kernel<LISTS, true, false> : topk_route_rows_kernel<LISTS, false, false>);
    return hipGetLastError();
}

hipError_t launch_topk_route(int64_t tokens, int E, int K, const void* logits, int bf16, int renorm,
                             int32_t* idx, float* w, hipStream_t stream)
{
    if (tokens == 0)
        return hipSuccess;
    // Up to 16 experts, four lanes per token (131072 tokens, 16 experts, top 4 6.7
    // us against 13 with a row of 16 lanes and lists).  Up to 256 and 16 choices,
    // a row of 16 lanes (131072 tokens, top 8: 64 experts 17 against 24 with 8
    // lanes and no lists; 128 experts 26 against 56 with a wave per token; 256
    // experts 44-49 against 66, top 16 60 against 88; 300 tokens alike).  Beyond,
    // rows with eight lists would gain and lose (rows against wave, top 8 of
    // 50000 tokens: 384 experts 34 against 37, 431 45 against 40; of 3000: 384
    // experts 7.0 against 6.3; top 16 of 3000 9.6 against 6.7).
    if (E <= 16)
        return route<4, 4>(tokens, E, K, logits, bf16, renorm, idx, w, stream);
    if (K <= 16) {
        if (E <= 64)
            return route_rows<1>(tokens, E, K, logits, bf16, renorm, idx, w, stream);
        if (E <= 128)
            return route_rows<2>(tokens, E, K, logits, bf16, renorm, idx, w, stream);
        if (E <= 256)
            return route_rows<4>(tokens, E, K, logits, bf16, renorm, idx, w, stream);
    }
    if (E <= 64)
        return route<8, 8>(tokens, E, K, logits, bf16, renorm, idx, w, stream);
    if (E <= 256)
        return route_wave<4>(tokens, E, K, logits, bf16, renorm, idx, w, stream);
    if (E <= 512)
        return route_wave<8>(tokens, E, K, logits, bf16, renorm, idx, w, stream);
    return route<64, 16>(tokens, E, K, logits, bf16, renorm, idx, w, stream);
}

}  // namespace ops
}  // namespace moe
