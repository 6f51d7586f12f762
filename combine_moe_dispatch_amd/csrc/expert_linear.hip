// The bf16 product of rows grouped by expert (or of all rows with one weight),
// with bias, activation and residual, and its gradients:
//
//   forward       z[r][j]  = sum over i of x[r][i] w[e][j][i] + b[e][j],  y = act(z) + residual
//   grad_input    dx[r][i] = act'(z_before[r][i]) * sum over j of dz[r][j] w[e][j][i] + residual
//   grad_weight   dw[e][j][i] = sum over the expert's rows r of dz[r][j] x[r][i],  db[e][j] = sum of dz[r][j]
//
// All three are  out[u][v] = sum over t of U(u,t) V(v,t),  v the output's fast
// axis.  V takes the matrix instruction's row operand and U its column
// operand, so a lane holds four consecutive outputs of one output row.  An
// operand is contiguous in memory along t (x and w of the forward product, dz
// of grad_input) or along its own index (w of grad_input, both of grad_weight);
// the second kind lies in LDS as [t][index] and is read with the transposing
// LDS read.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "expert_tiles.h"
#include "moe_ep.h"
#include "moe_ops.h"
#include "ops_common.h"

namespace moe {
namespace ops {
namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lv4s;

enum class Kind { FORWARD, INPUT, WEIGHT };

constexpr int STEP = 64;              // summed indices per stage: 128 bytes of a contiguous operand

template <int BM_, int BN_, int WM_, int WN_, int S_>
struct Block {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_;
    static constexpr int WAVES = WM * WN;
    static constexpr int THREADS = WAVES * WAVE;
    static constexpr int TM = BM / WM, TN = BN / WN;
    static constexpr int MT = TM / 16, NT = TN / 16;
    static constexpr int V_BYTES = BN * STEP * 2, U_BYTES = BM * STEP * 2;
    static constexpr int STAGE = V_BYTES + U_BYTES;
    static constexpr bool DEEP = BM == 256;                 // S does not count there
    static constexpr int LDS = DEEP ? 3 * V_BYTES + 2 * U_BYTES : S * STAGE;
    // 1 KB loads of a stage, and how many of them each wave issues
    static constexpr int V_ALL = V_BYTES / 1024, U_ALL = U_BYTES / 1024;
    static constexpr int V_LOADS = V_ALL / WAVES, U_LOADS = (U_ALL + WAVES - 1) / WAVES;
    static constexpr int LOADS = V_LOADS + U_LOADS;
    static_assert(V_ALL % WAVES == 0 && U_ALL % 2 == 0 && WAVES % 2 == 0, "a wave's parts share the swizzle");
    static_assert(NT % 2 == 0, "the epilogue pairs subtiles");
};

// 16 bytes per lane from memory to LDS, 1 KB from `lds` on: at a uniform base
// and 32-bit offsets, or at 64-bit addresses.  The compiler does not see these
// as memory accesses: told of them, it would wait for all of them ahead of
// every transposing LDS read.  They are waited for by meet() alone, and stay
// between the two that enclose them (volatile statements keep their order).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"      // m0, a reserved register, is named as overwritten
__device__ inline void load_to_lds(const uint8_t* base, uint32_t offset, const uint8_t* lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base),
                 "s"((uint32_t)(uintptr_t)(lvoid*)lds)
                 : "m0");
}
__device__ inline void load_to_lds(const uint8_t* address, const uint8_t* lds)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(address),
                 "s"((uint32_t)(uintptr_t)(lvoid*)lds)
                 : "m0");
}

#pragma clang diagnostic pop

// Everything this wave loaded but its last N loads has arrived in LDS, its own
// LDS reads are done, and so it is with every wave of the workgroup.
template <int N>
__device__ inline void meet()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0), in a form that the compiler counts
    asm volatile("s_barrier" ::: "memory");
}

// What is loaded in place of indices behind the end of the sum.
__device__ const uint4 zeros = {0, 0, 0, 0};

// One operand of a tile: element (i, t) lies at base[i * ld + t] (CONTIG) or
// base[t * ld + i]; i <= last.
struct Side {
    const uint16_t* base;
    const uint16_t* upper;    // CONTIG, gated: where rows from half the tile on start
    int ld;
    int last;
};

// 16-byte piece c of row t of a transposed operand lies at place c ^ turn(t):
// the four rows of four that 16 lanes read at once, and the other four of a
// half wave, lie in different banks.
template <int PIECES>
__device__ inline int turn(int t)
{
    return ((t & 3) | (t >> 3 & 1) << 2) << 1 & (PIECES - 1);
}

// Loads of 1 KB that each wave issues for 64 summed indices of this many rows.
template <class C>
__host__ __device__ constexpr int loads_of(int rows)
{
    return (rows / 8 + C::WAVES - 1) / C::WAVES;
}

// Loads the operand's indices t0 .. t0+63 of the sum, of ROWS of its rows from
// `first` on, into LDS.  TAIL: only `left` of them lie before the sum's end.
// Addresses are a uniform base and 32-bit offsets in bytes, at most 256 rows of
// 65536 elements.  (from, to: some of the wave's loads only.)
template <class C, int ROWS, bool CONTIG, bool GATED, bool TAIL>
__device__ __forceinline__ void load_side(const Side& s, int first, int64_t t0, int left, uint8_t* lds, int wave,
                                          int lane, int from = 0, int to = loads_of<C>(ROWS))
{
    constexpr int ALL = ROWS / 8;
    if constexpr (CONTIG) {
        const uint32_t piece = (lane & 7) ^ swizzle(wave * 8 + (lane >> 3));
        const uint8_t* base = (const uint8_t*)(s.base + t0);
        const uint8_t* upper = (const uint8_t*)(s.upper + t0);
#pragma unroll
        for (int i = from; i < to; ++i) {
            const int part = (i * C::WAVES + wave) % ALL;
            const int row = first + part * 8 + (lane >> 3);
            const bool up = GATED && part * 8 >= ROWS / 2;
            const uint32_t at = (uint32_t)min(up ? row - ROWS / 2 : row, s.last) * (uint32_t)(s.ld * 2) + piece * 16;
            if constexpr (TAIL)
                load_to_lds((int)(piece * 8) >= left ? (const uint8_t*)&zeros : (up ? upper : base) + at, lds + part * 1024);
            else
                load_to_lds(up ? upper : base, at, lds + part * 1024);
        }
    } else {
        constexpr int PIECES = ROWS / 8;
        const uint8_t* base = (const uint8_t*)(s.base + t0 * s.ld);
#pragma unroll
        for (int i = from; i < to; ++i) {
            const int part = (i * C::WAVES + wave) % ALL;
            const int t = part * (WAVE / PIECES) + lane / PIECES;
            const int piece = min(first / 8 + ((lane % PIECES) ^ turn<PIECES>(t)), s.last >> 3);
            const uint32_t at = (uint32_t)t * (uint32_t)(s.ld * 2) + piece * 16;
            if constexpr (TAIL)
                load_to_lds(t >= left ? (const uint8_t*)&zeros : base + at, lds + part * 1024);
            else
                load_to_lds(base, at, lds + part * 1024);
        }
    }
}

// The operand's 16 rows from `row` on, summed indices 32*half .. +31, as the matrix instruction
// takes them: lane (r, g) holds row r, indices 8g .. 8g+7.
template <int ROWS, bool CONTIG>
__device__ __forceinline__ v8b read_side(const uint8_t* lds, int row, int half, int lane)
{
    const int r = lane & 15, g = lane >> 4;
    if constexpr (CONTIG) {
        const int at = row + r;
        return *(const v8b*)(lds + at * 128 + (((half * 4 + g) ^ swizzle(r)) << 4));
    } else {
        constexpr int PIECES = ROWS / 8;
        const int t = half * 32 + g * 8 + (r >> 2);
        const int piece = row / 8 + (r >> 1 & 1);
        const int at = t * ROWS * 2 + ((piece ^ turn<PIECES>(t)) << 4) + ((r & 1) << 3);
        const int at4 = (t + 4) * ROWS * 2 + ((piece ^ turn<PIECES>(t + 4)) << 4) + ((r & 1) << 3);
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lv4s*)(lds + at));
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lv4s*)(lds + at4));
        typedef short v8s __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(v8b, (v8s)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
}

// --- epilogues: eight consecutive outputs of a row ---------------------------------------------

__device__ inline void open8(const uint16_t* p, float (&f)[8])
{
    const v4u u = *(const v4u*)p;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        f[2 * c] = bf16_lo(u[c]);
        f[2 * c + 1] = bf16_hi(u[c]);
    }
}
__device__ inline void store8(uint16_t* p, const float (&f)[8])
{
    *(v4u*)p = v4u{bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3]), bf16_pack(f[4], f[5]), bf16_pack(f[6], f[7])};
}
__device__ inline void store8(float* p, const float (&f)[8])
{
    ((v4f*)p)[0] = v4f{f[0], f[1], f[2], f[3]};
    ((v4f*)p)[1] = v4f{f[4], f[5], f[6], f[7]};
}
__device__ inline void add8(const uint16_t* p, float (&f)[8])
{
    float r[8];
    open8(p, r);
#pragma unroll
    for (int c = 0; c < 8; ++c)
        f[c] += r[c];
}
__device__ inline void store_out(const Linear& p, int64_t at, const float (&f)[8])
{
    if (p.out_f32)
        store8((float*)p.out + at, f);
    else
        store8((uint16_t*)p.out + at, f);
}

constexpr float INV_SQRT_2PI = 0.39894228f;

__device__ inline float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + exp_of(-z)); }
__device__ inline float silu(float z) { return 0.25f * silu4(z); }
__device__ inline float silu_slope(float z)
{
    const float p = sigmoid(z);
    return p * fmaf(z, 1.0f - p, 1.0f);
}
// exp(-z^2 / 2): z^2 as a rounded square and what the rounding left; 0 from |z| = 16 on.
__device__ inline float bell(float z)
{
    const float a = fminf(fabsf(z), 16.0f);
    const float s = a * a;
    return exp_of(-0.5f * s) * fmaf(-0.5f, fmaf(a, a, -s), 1.0f);
}
// The normal distribution function, exact to a few places far below 0 too: its
// lower tail is e/2 q(|z|), e = bell(z), q(a) = exp(a^2/2) erfc(a/sqrt 2).  q is t
// times a polynomial in t = 1 / (1 + a/4), which takes a >= 0 to (0, 1] and q,
// about 0.8/a far out, to a smooth function; the polynomial is a minimax fit of
// degree 9 (relative, made by reweighted least squares), off by 2^-24.8; with
// fp32's roundings three of 2^-24.
__device__ inline float normal_cdf(float z, float e)
{
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.25f, 1.0f));
    float q = 0.03956406653719189f;
    q = fmaf(q, t, -0.16175482184497494f);
    q = fmaf(q, t, 0.19119449790180776f);
    q = fmaf(q, t, -0.06343532126457903f);
    q = fmaf(q, t, 0.12739834579149614f);
    q = fmaf(q, t, 0.11795027138357608f);
    q = fmaf(q, t, 0.16320622028890885f);
    q = fmaf(q, t, 0.1869327106141444f);
    q = fmaf(q, t, 0.19947286322022686f);
    q = fmaf(q, t, 0.1994711334462549f);
    const float tail = 0.5f * e * (q * t);
    return z < 0.0f ? tail : 1.0f - tail;
}

__device__ inline float activate(int act, float z)
{
    switch (act) {
    case MOE_ACT_RELU: return z <= 0.0f ? 0.0f : z;
    case MOE_ACT_GELU: return z * normal_cdf(z, bell(z));
    case MOE_ACT_SILU: return silu(z);
    default: return z;
    }
}
__device__ inline float slope(int act, float z)
{
    switch (act) {
    case MOE_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case MOE_ACT_GELU: {
        const float e = bell(z);
        return fmaf(z * INV_SQRT_2PI, e, normal_cdf(z, e));
    }
    case MOE_ACT_SILU: return silu_slope(z);
    default: return 1.0f;
    }
}

// z in fp32 to y; z, bias and residual as the call has them.
__device__ inline void finish_forward(const Linear& p, int e, int64_t row, int col, float (&v)[8])
{
    if (p.bias)
        add8(p.bias + (int64_t)e * p.n + col, v);
    if (p.z_out)
        store8(p.z_out + row * p.n + col, v);
    if (p.act != MOE_ACT_NONE)
#pragma unroll
        for (int c = 0; c < 8; ++c)
            v[c] = activate(p.act, v[c]);
    const int64_t at = row * p.n + col;
    if (p.residual)
        add8(p.residual + at, v);
    store_out(p, at, v);
}
__device__ inline void finish_gated(const Linear& p, int e, int64_t row, int col, float (&g)[8], float (&u)[8])
{
    const int f = p.n / 2;
    if (p.bias) {
        add8(p.bias + (int64_t)e * p.n + col, g);
        add8(p.bias + (int64_t)e * p.n + f + col, u);
    }
    if (p.z_out) {
        store8(p.z_out + row * p.n + col, g);
        store8(p.z_out + row * p.n + f + col, u);
    }
    float v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
        v[c] = silu(g[c]) * u[c];
    const int64_t at = row * f + col;
    if (p.residual)
        add8(p.residual + at, v);
    store_out(p, at, v);
}
// d of silu(gate) * up to the gradients of gate and up.
__device__ inline void gated_slopes(const float (&d)[8], float (&g)[8], float (&u)[8])
{
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const float z = g[c];
        g[c] = d[c] * u[c] * silu_slope(z);
        u[c] = d[c] * silu(z);
    }
}
__device__ inline void finish_input(const Linear& p, int64_t row, int col, float (&v)[8])
{
    if (p.act == MOE_ACT_SWIGLU) {
        const int64_t at = row * 2 * p.k + col;
        float g[8], u[8];
        open8(p.z_in + at, g);
        open8(p.z_in + at + p.k, u);
        gated_slopes(v, g, u);
        if (p.residual) {
            add8(p.residual + at, g);
            add8(p.residual + at + p.k, u);
        }
        store_out(p, at, g);
        store_out(p, at + p.k, u);
        return;
    }
    const int64_t at = row * p.k + col;
    if (p.act != MOE_ACT_NONE) {
        float z[8];
        open8(p.z_in + at, z);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            v[c] *= slope(p.act, z[c]);
    }
    if (p.residual)
        add8(p.residual + at, v);
    store_out(p, at, v);
}

// --- tiles -------------------------------------------------------------------------------------

// Tile t of T: consecutive workgroups go to the 8 XCDs in turn, each XCD takes
// one contiguous run of tiles.
__device__ inline bool tile_of_workgroup(int64_t tiles, int64_t& t)
{
    const int64_t per_xcd = (tiles + 7) / 8;
    const int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    t = (id & 7) * per_xcd + (id >> 3);
    return id >> 3 < per_xcd && t < tiles;
}

// Tile v of m_tiles x n_tiles, in groups of up to 8 row tiles, row tiles fastest inside a group.
__device__ inline void tile_in_group(int64_t v, int m_tiles, int n_tiles, int& m, int& n)
{
    constexpr int GROUP = 8;
    const int64_t per_group = (int64_t)GROUP * n_tiles;
    const int g = (int)(v / per_group);
    const int in = (int)(v - g * per_group);
    const int gm = min(GROUP, m_tiles - g * GROUP);
    m = g * GROUP + in % gm;
    n = in / gm;
}

template <int BM>
__device__ inline bool find_rows(const Linear& p, int n_tiles, Place& at)
{
    if (p.offsets)
        return p.E <= 4 * WAVE ? find_tile<BM, 4>(p.offsets, p.E, p.rows, n_tiles, at)
                               : find_tile<BM, 16>(p.offsets, p.E, p.rows, n_tiles, at);
    const int m_tiles = (int)((p.rows + BM - 1) / BM);
    int64_t t;
    if (!tile_of_workgroup((int64_t)m_tiles * n_tiles, t))
        return false;
    int m;
    tile_in_group(t, m_tiles, n_tiles, m, at.n_tile);
    at.e = 0;
    at.m0 = m * BM;
    at.rows = (int)min((int64_t)BM, p.rows - at.m0);
    return true;
}

// Rows of expert e, held to the tensors' room.
__device__ inline void expert_rows(const Linear& p, int e, int64_t& a, int64_t& b)
{
    a = 0;
    b = p.rows;
    if (p.offsets) {
        a = min(max((int64_t)p.offsets[e], (int64_t)0), p.rows);
        b = min(max((int64_t)p.offsets[e + 1], a), p.rows);
    }
}

// Hands a wave's sums to `finish`, eight consecutive outputs at a time; subtile
// (j, i) starts at LDS row vrow(j) of V and urow(i) of U.
template <class C, bool GATED, bool BIAS, int SUMS, class URow, class VRow, class Finish, class FinishBias>
__device__ __forceinline__ void hand_over(v4f (&acc)[C::NT][C::MT], v4f (&sums)[SUMS], URow urow, VRow vrow, int wn,
                                          int u_rows, int v_rows, int lane, Finish finish, FinishBias finish_bias)
{
    // Lane (r, g) holds column r of a subtile and rows 4g .. 4g+3; lanes of two
    // subtiles trade so that each holds eight consecutive outputs.
    const int r = lane & 15, g = lane >> 4;
    auto eight = [&](int j, int i, float (&v)[8]) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const auto two = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[j][i][c]),
                                                              __float_as_uint(acc[j + 1][i][c]), false, false);
            v[c] = __uint_as_float(two[0]);
            v[4 + c] = __uint_as_float(two[1]);
        }
    };
    constexpr int PAIRED = GATED ? C::NT / 2 : C::NT;
    static_assert(PAIRED % 2 == 0, "whole pairs of subtiles");
#pragma unroll
    for (int i = 0; i < C::MT; ++i) {
        const int u = urow(i) + r;
#pragma unroll
        for (int j = 0; j < PAIRED; j += 2) {
            const int v = vrow(j) + (g & 1) * 16 + (g >> 1) * 8;
            float a[8], b[8];
            eight(j, i, a);
            if constexpr (GATED)
                eight(j + C::NT / 2, i, b);
            if (u < u_rows && v < v_rows)
                finish(u, v, a, b);
        }
    }
    if constexpr (BIAS)
#pragma unroll
        for (int i = 0; i < SUMS; ++i) {
            const int u = urow(wn * SUMS + i) + r;
            if (wn * SUMS + i < C::MT && g == 0 && u < u_rows)
                finish_bias(u, sums[i][0]);
        }
}

// Sums U(u,t) V(v,t) over t in [t0, t1) for one tile and hands every eight
// consecutive outputs to `finish(u, v, out[, up])`.
template <class C, bool U_CONTIG, bool V_CONTIG, bool GATED, bool BIAS, class Finish, class FinishBias>
__device__ __forceinline__ void product_tile(const Side& us, const Side& vs, int64_t t0, int64_t t1, int u_rows,
                                             int v_rows, uint8_t* lds, Finish finish, FinishBias finish_bias)
{
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int wm = wave % C::WM, wn = wave / C::WM;
    const int steps = (int)((t1 - t0 + STEP - 1) / STEP);
    const int last_left = (int)(t1 - t0) - (steps - 1) * STEP;      // terms of the last stage
    auto issue = [&](int step, uint8_t* st, auto tail) {
        const int64_t t = t0 + (int64_t)step * STEP;
        load_side<C, C::BN, V_CONTIG, GATED, tail>(vs, 0, t, last_left, st, wave, lane);
        load_side<C, C::BM, U_CONTIG, false, tail>(us, 0, t, last_left, st + C::V_BYTES, wave, lane);
    };
    // LDS row of V's subtile j: gated tiles keep the gate's rows in their first half
    auto vrow = [&](int j) {
        if (GATED) {
            constexpr int HALF = C::NT / 2;
            return (j < HALF ? 0 : C::BN / 2) + wn * (C::TN / 2) + j % HALF * 16;
        }
        return wn * C::TN + j * 16;
    };
    const v4f zero{0.0f, 0.0f, 0.0f, 0.0f};
    v4f acc[C::NT][C::MT];
#pragma unroll
    for (int j = 0; j < C::NT; ++j)
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
            acc[j][i] = zero;
    // sums of U alone (the bias' gradient): the waves that share U's rows share its subtiles
    constexpr int SUMS = (C::MT + C::WN - 1) / C::WN;
    v4f sums[SUMS];
    v8b ones;
    if constexpr (BIAS) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            ones[c] = (__bf16)1.0f;
#pragma unroll
        for (int i = 0; i < SUMS; ++i)
            sums[i] = zero;
    }
#pragma unroll
    for (int s = 0; s < C::S; ++s)
        if (s < steps - 1)
            issue(s, lds + s * C::STAGE, std::false_type{});
        else if (s == steps - 1)
            issue(s, lds + s * C::STAGE, std::true_type{});
    // A stage is summed in two halves of 32.  Each half's operands are read
    // while the half before it is multiplied; in the middle of a stage all its
    // reads are done, its slot is free once every wave is there, and the next
    // stage has arrived.
    v8b vf[2][C::NT], uf[2][C::MT];
    auto read = [&](const uint8_t* st, int h) {
#pragma unroll
        for (int j = 0; j < C::NT; ++j)
            vf[h][j] = read_side<C::BN, V_CONTIG>(st, vrow(j), h, lane);
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
            uf[h][i] = read_side<C::BM, U_CONTIG>(st + C::V_BYTES, wm * C::TM + i * 16, h, lane);
    };
    auto multiply = [&](int h) {
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
#pragma unroll
            for (int j = 0; j < C::NT; ++j)
                acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[h][j], uf[h][i], acc[j][i], 0, 0, 0);
        if constexpr (BIAS)
#pragma unroll
            for (int i = 0; i < C::MT; ++i)
                if (i / SUMS == wn)
                    sums[i % SUMS] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, uf[h][i], sums[i % SUMS], 0, 0, 0);
        // a read beside every few products
        constexpr int READS = C::NT * (V_CONTIG ? 1 : 2) + C::MT * (U_CONTIG ? 1 : 2);
        constexpr int EACH = C::NT * C::MT / READS > 0 ? C::NT * C::MT / READS : 1;
#pragma unroll
        for (int q = 0; q < READS; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, EACH, 0);
        }
    };
    if (steps > 0) {
        if (steps >= C::S)
            meet<(C::S - 1) * C::LOADS>();
        else
            meet<0>();
        read(lds, 0);
    }
    int slot = 0;
    auto step_of = [&](int step, auto steady, auto tail) {
        uint8_t* st = lds + slot * C::STAGE;
        read(st, 1);
        multiply(0);
        meet<decltype(steady)::value ? (C::S - 2) * C::LOADS : 0>();
        if constexpr (decltype(steady)::value)
            issue(step + C::S, st, tail);
        slot = slot + 1 == C::S ? 0 : slot + 1;
        read(lds + slot * C::STAGE, 0);              // (past the last stage: stale, never used)
        multiply(1);
    };
    int step = 0;
    for (; step + C::S < steps - 1; ++step)
        step_of(step, std::true_type{}, std::false_type{});
    if (step + C::S < steps)
        step_of(step++, std::true_type{}, std::true_type{});
    for (; step < steps; ++step)
        step_of(step, std::false_type{}, std::false_type{});

    hand_over<C, GATED, BIAS>(acc, sums, [&](int i) { return wm * C::TM + i * 16; }, vrow, wn, u_rows, v_rows, lane,
                              finish, finish_bias);
}

// The same for the 256 x 256 tile, U in two halves of 128 rows, with V's
// stages in three slots of LDS and each half of U's in two: 160 KB.  A step is
// two phases, one for each half of U; a phase's operands are read while the
// phase before it is multiplied, and what has been read by every wave is
// loaded anew at once, so that a load has one and a half to two steps to
// arrive (with two slots for everything, one step).
template <class C, bool U_CONTIG, bool V_CONTIG, bool GATED, bool BIAS, class Finish, class FinishBias>
__device__ __forceinline__ void product_tile_deep(const Side& us, const Side& vs, int64_t t0, int64_t t1, int u_rows,
                                                  int v_rows, uint8_t* lds, Finish finish, FinishBias finish_bias)
{
    static_assert(C::BM == 256 && C::BN == 256 && C::WM == 2 && C::WN == 4, "eight waves of 128 x 64");
    constexpr int HALF = 128, HALF_BYTES = HALF * STEP * 2;
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int wm = wave % C::WM, wn = wave / C::WM;
    const int steps = (int)((t1 - t0 + STEP - 1) / STEP);
    const int last_left = (int)(t1 - t0) - (steps - 1) * STEP;
    uint8_t* const u_lds = lds + 3 * C::V_BYTES;
    auto v_slot = [&](int s) { return lds + s * C::V_BYTES; };
    auto u_slot = [&](int half, int s) { return u_lds + (half * 2 + s) * HALF_BYTES; };
    // Nothing is loaded behind the last stage, whose tail is zeros; `inner`: it is not the last.
    auto load_v = [&](int step, int slot, auto inner, int from, int to) {
        const int64_t t = t0 + (int64_t)step * STEP;
        if (inner || step < steps - 1)
            load_side<C, C::BN, V_CONTIG, GATED, false>(vs, 0, t, 0, v_slot(slot), wave, lane, from, to);
        else if (step == steps - 1)
            load_side<C, C::BN, V_CONTIG, GATED, true>(vs, 0, t, last_left, v_slot(slot), wave, lane, from, to);
    };
    auto load_u = [&](int half, int step, auto inner, int from, int to) {
        const int64_t t = t0 + (int64_t)step * STEP;
        uint8_t* const slot = u_slot(half, step & 1);
        if (inner || step < steps - 1)
            load_side<C, HALF, U_CONTIG, false, false>(us, half * HALF, t, 0, slot, wave, lane, from, to);
        else if (step == steps - 1)
            load_side<C, HALF, U_CONTIG, false, true>(us, half * HALF, t, last_left, slot, wave, lane, from, to);
    };
    auto vrow = [&](int j) {
        if (GATED) {
            constexpr int GH = C::NT / 2;
            return (j < GH ? 0 : C::BN / 2) + wn * (C::TN / 2) + j % GH * 16;
        }
        return wn * C::TN + j * 16;
    };
    constexpr int UT = C::MT / 2;                    // subtiles of a half
    const v4f zero{0.0f, 0.0f, 0.0f, 0.0f};
    v4f acc[C::NT][C::MT];
#pragma unroll
    for (int j = 0; j < C::NT; ++j)
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
            acc[j][i] = zero;
    constexpr int SUMS = C::MT / C::WN;
    v4f sums[SUMS];
    v8b ones;
    if constexpr (BIAS) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            ones[c] = (__bf16)1.0f;
#pragma unroll
        for (int i = 0; i < SUMS; ++i)
            sums[i] = zero;
    }
    v8b vf[2][C::NT], uf[2][2][UT];                  // V: [k half]; U: [row half][k half]
    auto read_v = [&](int slot, int h, int j) {
        vf[h][j] = read_side<C::BN, V_CONTIG>(v_slot(slot), vrow(j), h, lane);
    };
    auto read_u = [&](int half, int slot, int h, int i) {
        uf[half][h][i] = read_side<HALF, U_CONTIG>(u_slot(half, slot), wm * 64 + i * 16, h, lane);
    };
    // Four products, and the reads beside them, in this order.
    auto products = [&](int half, int h, int i) {
#pragma unroll
        for (int j = 0; j < C::NT; ++j)
            acc[j][half * UT + i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[h][j], uf[half][h][i],
                                                                           acc[j][half * UT + i], 0, 0, 0);
        if constexpr (BIAS)
            if ((half * UT + i) / SUMS == wn)
                sums[i % SUMS] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, uf[half][h][i], sums[i % SUMS], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    static_assert(C::NT == 4 && UT == 4, "the order of reads below");
    // A phase issues four loads, one beside every eight products: two of the half of U that the
    // phase before it was the last to read, and half of V's, whose slot was free before.
    constexpr int V_LOADS = loads_of<C>(C::BN), U_LOADS = loads_of<C>(HALF), PHASE = V_LOADS / 2 + U_LOADS;
    static_assert(V_LOADS == 4 && U_LOADS == 2, "four loads per phase");
    constexpr std::false_type any{};
    load_u(0, 0, any, 0, 2);
    load_v(0, 0, any, 0, 4);
    load_u(1, 0, any, 0, 2);
    load_v(1, 1, any, 0, 2);
    load_u(0, 1, any, 0, 2);
    load_v(1, 1, any, 2, 4);
    load_u(1, 1, any, 0, 2);
    load_v(2, 2, any, 0, 2);
    if (steps >= 3)
        meet<3 * PHASE>();
    else
        meet<0>();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        read_v(0, 0, q);
        read_u(0, 0, 0, q);
        read_u(0, 0, 1, q);
    }
    if (steps >= 3)
        meet<2 * PHASE>();
    else
        meet<0>();
    int now = 0, last = 2;                           // V's slots of this step and the one before it
    auto step_of = [&](int step, auto steady) {
        // every wave has read the first half of U and V's first indices of this step
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q < 2) {
                read_v(now, 1, 2 * q);
                read_v(now, 1, 2 * q + 1);
            } else if (q < 6) {
                read_u(1, step & 1, (q - 2) / 2, (q & 1) * 2);
                read_u(1, step & 1, (q - 2) / 2, (q & 1) * 2 + 1);
            }
            if (q == 0 || q == 2)
                load_u(0, step + 2, steady, q / 2, q / 2 + 1);
            if (q == 4 || q == 6)
                load_v(step + 2, last, steady, q / 2, q / 2 + 1);
            products(0, q / 4, q % 4);
        }
        meet<steady ? 2 * PHASE : 0>();
        // ... and V and the second half of U; what is read past the last stage is stale, and not used
        last = now;
        now = now == 2 ? 0 : now + 1;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q < 4) {
                read_u(0, (step + 1) & 1, q / 2, (q & 1) * 2);
                read_u(0, (step + 1) & 1, q / 2, (q & 1) * 2 + 1);
            } else if (q < 6) {
                read_v(now, 0, (q & 1) * 2);
                read_v(now, 0, (q & 1) * 2 + 1);
            }
            if (q == 0 || q == 2)
                load_u(1, step + 2, steady, q / 2, q / 2 + 1);
            if (q == 4 || q == 6)
                load_v(step + 3, last, steady, q / 2 - 2, q / 2 - 1);
            products(1, q / 4, q % 4);
        }
        meet<steady ? 2 * PHASE : 0>();
    };
    int step = 0;
    for (; step + 3 < steps - 1; ++step)
        step_of(step, std::true_type{});
    for (; step < steps; ++step)
        step_of(step, any);
    hand_over<C, GATED, BIAS>(acc, sums, [&](int i) { return i / UT * HALF + wm * 64 + i % UT * 16; }, vrow, wn, u_rows,
                              v_rows, lane, finish, finish_bias);
}

template <class C, bool U_CONTIG, bool V_CONTIG, bool GATED, bool BIAS, class Finish, class FinishBias>
__device__ __forceinline__ void run_tile(const Side& us, const Side& vs, int64_t t0, int64_t t1, int u_rows,
                                         int v_rows, uint8_t* lds, Finish finish, FinishBias finish_bias)
{
    if constexpr (C::DEEP)
        product_tile_deep<C, U_CONTIG, V_CONTIG, GATED, BIAS>(us, vs, t0, t1, u_rows, v_rows, lds, finish, finish_bias);
    else
        product_tile<C, U_CONTIG, V_CONTIG, GATED, BIAS>(us, vs, t0, t1, u_rows, v_rows, lds, finish, finish_bias);
}

// The part of [0, steps * STEP) that split `s` of `splits` sums.
__device__ inline void split_range(int64_t total, int splits, int s, int64_t& t0, int64_t& t1)
{
    const int64_t steps = (total + STEP - 1) / STEP, per = (steps + splits - 1) / splits;
    t0 = min(s * per * STEP, total);
    t1 = min(t0 + per * STEP, total);
}

// forward and grad_input: out rows are the token rows
template <Kind KIND, class C, bool GATED>
__global__ __launch_bounds__(C::THREADS) void linear_kernel(const Linear p, int n_tiles, int splits)
{
    extern __shared__ __align__(1024) uint8_t lds[];
    constexpr bool FWD = KIND == Kind::FORWARD;
    Place at;
    if (!find_rows<C::BM>(p, n_tiles, at))
        return;
    at.e = __builtin_amdgcn_readfirstlane(at.e);             // (uniform already, which the compiler cannot tell)
    at.m0 = __builtin_amdgcn_readfirstlane(at.m0);
    at.rows = __builtin_amdgcn_readfirstlane(at.rows);
    at.n_tile = __builtin_amdgcn_readfirstlane(at.n_tile);
    const int width = FWD ? p.n : p.k;                       // output columns
    const int f = GATED ? p.n / 2 : width;                   // columns that tiles divide
    const int v0 = at.n_tile * (GATED ? C::BN / 2 : C::BN);
    const int64_t total = FWD ? p.k : p.n;
    Side us, vs;
    us.ld = (int)total;
    us.base = (FWD ? p.x : p.dz) + (int64_t)at.m0 * total;
    us.upper = us.base;
    us.last = at.rows - 1;
    const uint16_t* w = p.w + (int64_t)at.e * p.n * p.k;
    vs.ld = p.k;
    vs.base = FWD ? w + (int64_t)v0 * p.k : w + v0;
    vs.upper = GATED ? vs.base + (int64_t)f * p.k : vs.base;
    vs.last = min(GATED ? C::BN / 2 : C::BN, f - v0) - 1;
    int64_t t0, t1;
    split_range(total, splits, blockIdx.z, t0, t1);
    float* part = (float*)p.workspace + (int64_t)blockIdx.z * p.rows * width;
    auto finish = [&](int u, int v, float(&a)[8], float(&b)[8]) {
        const int64_t row = at.m0 + u;
            const int col = v0 + v;
            if (splits > 1) {
                store8(part + row * width + col, a);
                if (GATED)
                    store8(part + row * width + f + col, b);
            } else if (GATED) {
                finish_gated(p, at.e, row, col, a, b);
            } else if (FWD) {
                finish_forward(p, at.e, row, col, a);
            } else {
                finish_input(p, row, col, a);
            }
        };
    run_tile<C, true, FWD, GATED, false>(us, vs, t0, t1, at.rows, vs.last + 1, lds, finish, [](int, float) {});
}

// grad_weight: out rows are an expert's weight rows
template <class C>
__global__ __launch_bounds__(C::THREADS) void linear_weight_kernel(const Linear p, int m_tiles, int n_tiles, int splits)
{
    extern __shared__ __align__(1024) uint8_t lds[];
    int64_t t;
    if (!tile_of_workgroup((int64_t)p.E * m_tiles * n_tiles, t))
        return;
    const int e = (int)(t / ((int64_t)m_tiles * n_tiles));
    int m, n;
    tile_in_group(t - (int64_t)e * m_tiles * n_tiles, m_tiles, n_tiles, m, n);
    int64_t a, b;
    expert_rows(p, e, a, b);
    a = __builtin_amdgcn_readfirstlane((int)a);              // (uniform already, which the compiler cannot tell)
    b = __builtin_amdgcn_readfirstlane((int)b);
    const int u0 = m * C::BM, v0 = n * C::BN;
    Side us, vs;
    us.ld = p.n;
    us.base = us.upper = p.dz + a * p.n + u0;
    us.last = min(C::BM, p.n - u0) - 1;
    vs.ld = p.k;
    vs.base = vs.upper = p.x + a * p.k + v0;
    vs.last = min(C::BN, p.k - v0) - 1;
    int64_t t0, t1;
    split_range(b - a, splits, blockIdx.z, t0, t1);
    const int64_t weights = (int64_t)p.E * p.n * p.k;
    float* part = (float*)p.workspace + (int64_t)blockIdx.z * weights;
    float* part_b = (float*)p.workspace + (int64_t)splits * weights + (int64_t)blockIdx.z * p.E * p.n;
    auto finish = [&](int u, int v, float(&o)[8], float(&)[8]) {
        const int64_t at = ((int64_t)e * p.n + u0 + u) * p.k + v0 + v;
        if (splits > 1)
            store8(part + at, o);
        else
            store_out(p, at, o);
    };
    auto finish_bias = [&](int u, float s) { (splits > 1 ? part_b : p.dbias)[(int64_t)e * p.n + u0 + u] = s; };
    if (p.dbias && n == 0)
        run_tile<C, false, false, false, true>(us, vs, t0, t1, us.last + 1, vs.last + 1, lds, finish, finish_bias);
    else
        run_tile<C, false, false, false, false>(us, vs, t0, t1, us.last + 1, vs.last + 1, lds, finish, finish_bias);
}

// --- joins of split sums -----------------------------------------------------------------------

__device__ inline void add_parts(const float* part, int64_t stride, int splits, float (&v)[8])
{
#pragma unroll
    for (int c = 0; c < 8; ++c)
        v[c] = 0.0f;
    for (int s = 0; s < splits; ++s, part += stride) {
        const v4f a = ((const v4f*)part)[0], b = ((const v4f*)part)[1];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[c] += a[c];
            v[4 + c] += b[c];
        }
    }
}

// The eight outputs of this thread, where threads go through rows of `width`.
__device__ inline void place_of_eight(int64_t rows, int width, int64_t& row, int& col)
{
    const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    const uint32_t per = width / 8;
    if (rows * per < (int64_t)1 << 31) {             // the whole launch alike: a division in 32 bits
        row = (uint32_t)i / per;
        col = (int)((uint32_t)i - (uint32_t)row * per) * 8;
    } else {
        row = i / per;
        col = (int)(i - row * per) * 8;
    }
}

// The expert of a row by bisection; rows behind the last expert's give false.
__device__ inline bool expert_of(const Linear& p, int64_t row, int& e)
{
    e = 0;
    if (!p.offsets)
        return true;
    int lo = 0, hi = p.E;                          // first e with offsets[e + 1] > row
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (p.offsets[mid + 1] > row)
            hi = mid;
        else
            lo = mid + 1;
    }
    e = lo;
    return lo < p.E;
}

template <Kind KIND, bool GATED>
__global__ __launch_bounds__(256) void join_rows_kernel(const Linear p, int splits)
{
    const int width = KIND == Kind::FORWARD ? p.n : p.k;
    const int f = GATED ? width / 2 : width;
    int64_t row;
    int col, e;
    place_of_eight(p.rows, f, row, col);
    if (row >= p.rows || !expert_of(p, row, e))
        return;
    const int64_t stride = p.rows * width;
    const float* part = (const float*)p.workspace + row * width + col;
    float a[8];
    add_parts(part, stride, splits, a);
    if constexpr (GATED) {
        float b[8];
        add_parts(part + f, stride, splits, b);
        finish_gated(p, e, row, col, a, b);
    } else if constexpr (KIND == Kind::FORWARD) {
        finish_forward(p, e, row, col, a);
    } else {
        finish_input(p, row, col, a);
    }
}

__global__ __launch_bounds__(256) void join_weight_kernel(const Linear p, int splits)
{
    const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    const int64_t weights = (int64_t)p.E * p.n * p.k, biases = (int64_t)p.E * p.n;
    float v[8];
    if (i * 8 < weights) {
        add_parts((const float*)p.workspace + i * 8, weights, splits, v);
        store_out(p, i * 8, v);
    }
    if (p.dbias && i * 8 < biases) {
        add_parts((const float*)p.workspace + splits * weights + i * 8, biases, splits, v);
        store8(p.dbias + i * 8, v);
    }
}

// dz = dy * act'(z), eight outputs per thread.  What is handed on is bf16, and
// sums over many rows of it follow, where a border rounded the other way counts
// more than all of fp32's roundings: so a product that fp32 (off by less than 8
// of its roundings) cannot tell from the middle between two bf16 numbers is
// formed again in 64 bits.  That is one in a thousand: 32768 x 4096, SWIGLU, 200 us
// against 196 without.
__device__ inline double slope64(int act, double z)
{
    if (act == MOE_ACT_GELU)
        return 0.5 * erfc(-0.70710678118654752440 * z) + z * exp(-0.5 * z * z) * 0.39894228040143267794;
    const double p = 1.0 / (1.0 + exp(-z));
    return p * (1.0 + z * (1.0 - p));
}
__device__ inline double silu64(double z) { return z / (1.0 + exp(-z)); }

// v, off by less than `err`, might round to bf16 as another number.
__device__ inline bool near_border(float v, float err)
{
    const float border = __uint_as_float((__float_as_uint(v) & 0xFFFF0000u) | 0x8000u);
    return fabsf(v - border) <= err;
}

__global__ __launch_bounds__(256) void activation_grad_kernel(const Linear p, const uint16_t* dy)
{
    const int f = p.act == MOE_ACT_SWIGLU ? p.n / 2 : p.n;
    int64_t row;
    int col;
    place_of_eight(p.rows, f, row, col);
    const int64_t rows = p.offsets ? min(p.rows, (int64_t)p.offsets[p.E]) : p.rows;
    if (row >= rows)
        return;
    constexpr float ERR = 0x1p-21f;
    float d[8], z[8], v[8];
    open8(dy + row * f + col, d);
    uint16_t* out = (uint16_t*)p.out + row * p.n + col;
    open8(p.z_in + row * p.n + col, z);
    if (p.act == MOE_ACT_SWIGLU) {
        float u[8], w[8];
        open8(p.z_in + row * p.n + f + col, u);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float g = d[c] * u[c];
            v[c] = g * silu_slope(z[c]);
            w[c] = d[c] * silu(z[c]);
            if (near_border(v[c], ERR * fabsf(g)))
                v[c] = (float)((double)d[c] * u[c] * slope64(MOE_ACT_SILU, z[c]));
            if (near_border(w[c], ERR * fabsf(w[c])))
                w[c] = (float)(d[c] * silu64(z[c]));
        }
        store8(out, v);
        store8(out + f, w);
        return;
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        v[c] = d[c] * slope(p.act, z[c]);
        if (p.act != MOE_ACT_RELU && near_border(v[c], ERR * fabsf(d[c])))
            v[c] = (float)(d[c] * slope64(p.act, z[c]));
    }
    store8(out, v);
}

// --- host --------------------------------------------------------------------------------------

template <class K>
hipError_t allow_lds(K kernel, std::atomic<uint64_t>& allowed)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(allowed.load(std::memory_order_relaxed) & bit) || !bit) {
        e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != hipSuccess)
            return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    return hipSuccess;
}

dim3 blocks_of(int64_t threads) { return grid_of((threads + 255) / 256); }

// Splits of a sum of `total` terms where a launch has `groups` workgroups.
int splits_of(int64_t groups, int64_t total)
{
    const int64_t steps = (total + STEP - 1) / STEP;
    if (groups > 128 || steps < 8)
        return 1;
    return (int)std::max<int64_t>(std::min<int64_t>({256 / groups, steps / 4, 32}), 1);
}

typedef Block<256, 256, 2, 4, 2> Rows256;
typedef Block<32, 256, 2, 4, 2> Rows32;
typedef Block<256, 256, 2, 4, 2> Weights256;

struct Shape {
    bool low;                 // the lower tile
    int n_tiles, splits;
};

Shape rows_shape(Kind kind, bool gated, int64_t rows, int E, int n, int k)
{
    Shape s;
    const int width = kind == Kind::FORWARD ? n : k;
    s.n_tiles = gated ? (width / 2 + 127) / 128 : (width + 255) / 256;
    s.low = rows / E <= 48;
    s.splits = splits_of(workgroups(rows, E, s.low ? Rows32::BM : Rows256::BM, s.n_tiles), kind == Kind::FORWARD ? k : n);
    return s;
}

int weight_splits(int64_t rows, int E, int n, int k)
{
    return splits_of((int64_t)E * ((n + 255) / 256) * ((k + 255) / 256), rows / E);
}

template <Kind KIND, bool GATED, class C>
hipError_t launch_rows(const Linear& p, const Shape& s, hipStream_t stream)
{
    static std::atomic<uint64_t> allowed{0};
    const hipError_t e = allow_lds(linear_kernel<KIND, C, GATED>, allowed);
    if (e != hipSuccess)
        return e;
    dim3 grid = grid_of(workgroups(p.rows, p.E, C::BM, s.n_tiles));
    grid.z = s.splits;
    linear_kernel<KIND, C, GATED><<<grid, dim3(C::THREADS), C::LDS, stream>>>(p, s.n_tiles, s.splits);
    return hipGetLastError();
}

template <Kind KIND, bool GATED>
hipError_t launch_rows(const Linear& p, hipStream_t stream)
{
    const Shape s = rows_shape(KIND, GATED, p.rows, p.E, p.n, p.k);
    const hipError_t e = s.low ? launch_rows<KIND, GATED, Rows32>(p, s, stream)
                               : launch_rows<KIND, GATED, Rows256>(p, s, stream);
    if (e != hipSuccess || s.splits == 1)
        return e;
    const int width = KIND == Kind::FORWARD ? p.n : p.k;
    join_rows_kernel<KIND, GATED><<<blocks_of(p.rows * ((GATED ? width / 2 : width) / 8)), dim3(256), 0, stream>>>(
        p, s.splits);
    return hipGetLastError();
}

}  // namespace

size_t linear_workspace(int64_t rows, int E, int n, int k)
{
    size_t most = 0;
    for (int gated = 0; gated < 2; ++gated) {
        const int s = rows_shape(Kind::FORWARD, gated, rows, E, n, k).splits;
        most = std::max(most, s > 1 ? (size_t)s * rows * n * 4 : 0);
    }
    const int si = rows_shape(Kind::INPUT, false, rows, E, n, k).splits;
    most = std::max(most, si > 1 ? (size_t)si * rows * k * 4 : 0);
    const int sw = weight_splits(rows, E, n, k);
    return std::max(most, sw > 1 ? (size_t)sw * E * n * (k + 1) * 4 : 0);
}

hipError_t launch_linear(const Linear& p, hipStream_t stream)
{
    return p.act == MOE_ACT_SWIGLU ? launch_rows<Kind::FORWARD, true>(p, stream)
                                   : launch_rows<Kind::FORWARD, false>(p, stream);
}

hipError_t launch_linear_grad_input(const Linear& p, hipStream_t stream)
{
    return launch_rows<Kind::INPUT, false>(p, stream);
}

hipError_t launch_linear_grad_weight(const Linear& p, hipStream_t stream)
{
    typedef Weights256 C;
    const int m_tiles = (p.n + C::BM - 1) / C::BM, n_tiles = (p.k + C::BN - 1) / C::BN;
    const int splits = weight_splits(p.rows, p.E, p.n, p.k);
    static std::atomic<uint64_t> allowed{0};
    const hipError_t e = allow_lds(linear_weight_kernel<C>, allowed);
    if (e != hipSuccess)
        return e;
    dim3 grid = grid_of(((int64_t)p.E * m_tiles * n_tiles + 7) / 8 * 8);
    grid.z = splits;
    linear_weight_kernel<C><<<grid, dim3(C::THREADS), C::LDS, stream>>>(p, m_tiles, n_tiles, splits);
    if (splits > 1)
        join_weight_kernel<<<blocks_of(((int64_t)p.E * p.n * p.k + 7) / 8), dim3(256), 0, stream>>>(p, splits);
    return hipGetLastError();
}

hipError_t launch_activation_grad(const Linear& p, const uint16_t* dy, hipStream_t stream)
{
    const int f = p.act == MOE_ACT_SWIGLU ? p.n / 2 : p.n;
    activation_grad_kernel<<<blocks_of(p.rows * (f / 8)), dim3(256), 0, stream>>>(p, dy);
    return hipGetLastError();
}

}  // namespace ops
}  // namespace moe
