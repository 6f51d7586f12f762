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
#include <cmath>
#include <type_traits>

#include "expert_tiles.h"
#include "moe_ep.h"
#include "moe_ops.h"
#include "ops_common.h"

namespace moe {
namespace ops {
namespace {

// The same number, which the compiler takes for a new one: what is formed from
// it is not formed ahead of a loop and held in registers that the loop needs.
__device__ inline int anew(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// The kernel's arguments, read again from where the launch left them (its first
// argument is a Linear): held through a main loop they would take the scalar
// registers that it needs.
__device__ inline const Linear& arguments()
{
    auto p = (const __attribute__((address_space(4))) Linear*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const Linear*)p;
}

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
    // first row of U's subtile i; the deep tile takes U in halves of 128 rows
    static __device__ inline int u_row_of(int i, int wm)
    {
        if constexpr (DEEP)
            return i / (MT / 2) * (BM / 2) + wm * (TM / 2) + i % (MT / 2) * 16;
        else
            return wm * TM + i * 16;
    }
};

// A buffer of memory as the buffer instructions address it: what lies outside
// [base, base + bytes) reads as zero.
typedef uint32_t Buffer __attribute__((ext_vector_type(4)));
__device__ inline Buffer buffer_of(const void* base, uint32_t bytes)
{
    constexpr uint32_t RAW32 = 0x00020000;               // 32-bit elements, no stride
    const uint64_t at = (uint64_t)base;
    // (uniform already, which the compiler cannot always tell)
    return Buffer{(uint32_t)__builtin_amdgcn_readfirstlane((int)at),
                  (uint32_t)__builtin_amdgcn_readfirstlane((int)(at >> 32)),
                  (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), RAW32};
}

// 16 bytes per lane from a buffer, at `offset` of the lane and `more` of all, to
// LDS, 1 KB from `lds` on.  The compiler does not see this as a memory access:
// told of it, it would wait for all such loads ahead of every transposing LDS
// read.  They are waited for by meet() alone, and stay between the two that
// enclose them (volatile statements keep their order).  The memory unit may read
// a scalar register five wait states after a vector instruction wrote it, as
// buffer_of's may just have done, and one after m0 was written; nothing holds it
// back, and the compiler counts wait states only for instructions it knows.  So
// they are here: one of the move, four of the s_nop (four more cost 1 to 1.5% of a
// large product: 16 experts, 32768 rows, 4096 x 7168 through SWIGLU 1572 and 1596 us).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"      // m0, a reserved register, is named as overwritten
__device__ inline void load_to_lds(Buffer b, uint32_t offset, uint32_t more, const uint8_t* lds)
{
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(offset), "s"(b),
                 "s"(more), "s"((uint32_t)(uintptr_t)(lvoid*)lds)
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

// One operand of a tile, from the tile's first index and the sum's first term
// on: element (i, t) lies at base[i * ld + t] (CONTIG) or base[t * ld + i].
struct Side {
    const uint16_t* base;
    const uint16_t* upper;    // CONTIG, gated: where rows from half the tile on start
    int ld;                   // elements
    int valid;                // indices i that exist (gated: of each half)
    int terms;                // t that exist
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

// Loads stage `step` of the operand's sum, ROWS of its rows from `first` on,
// into LDS: the wave's loads from .. to-1.  What does not exist is zero: rows
// lie outside the buffer, and so do a transposed operand's last terms; a
// contiguous one's (TAIL: the last stage) are sent there.  A lane's offset is
// the same in all loads of all stages, so that it takes one register.
template <class C, int ROWS, bool CONTIG, bool GATED, bool TAIL>
__device__ __forceinline__ void load_side(const Side& s, int first, int step, uint8_t* lds, int wave, int lane,
                                          int from = 0, int to = loads_of<C>(ROWS))
{
    constexpr int ALL = ROWS / 8;
    const int part0 = wave % ALL;                        // load i brings part i * WAVES + part0
    const uint32_t ld = (uint32_t)s.ld * 2;
    if constexpr (CONTIG) {
        constexpr int EACH = C::WAVES * 8;               // rows that the waves bring at a time
        constexpr int HALF = GATED ? ROWS / 2 : ROWS;
        static_assert(EACH >= ROWS || HALF % EACH == 0, "a load is of one half");
        const int piece = (lane & 7) ^ swizzle(part0 * 8 + (lane >> 3));
        uint32_t offset = (uint32_t)(part0 * 8 + (lane >> 3)) * ld + piece * 16;
        if (TAIL && piece * 8 >= s.terms - step * STEP)
            offset = 0x40000000;
        const uint32_t bytes = (uint32_t)(s.valid - 1) * ld + (uint32_t)s.terms * 2;
#pragma unroll
        for (int i = from; i < to; ++i) {
            const bool up = GATED && i * EACH >= HALF;
            load_to_lds(buffer_of(up ? s.upper : s.base, bytes), offset,
                        (uint32_t)(first + i * EACH - (up ? HALF : 0)) * ld + step * STEP * 2,
                        lds + (i * C::WAVES + part0) * 1024);
        }
    } else {
        constexpr int PIECES = ROWS / 8, TERMS = WAVE / PIECES;      // terms per load
        constexpr int EACH = C::WAVES * TERMS;
        static_assert(EACH >= STEP || EACH % 16 == 0, "one swizzle per lane");
        const int t = part0 * TERMS + lane / PIECES;
        const uint32_t offset = (uint32_t)t * ld + ((lane % PIECES) ^ turn<PIECES>(t)) * 16;
        const uint32_t terms = TAIL ? s.terms - step * STEP : STEP;
        const Buffer b = buffer_of(s.base + (int64_t)step * STEP * s.ld, (terms - 1) * ld + (uint32_t)s.valid * 2);
#pragma unroll
        for (int i = from; i < to; ++i)
            load_to_lds(b, offset, i * EACH * ld + first * 2, lds + (i * C::WAVES + part0) * 1024);
    }
}

// Reads an operand of a stage in LDS, as the matrix instruction takes it: lane
// (r, g) holds row r of 16, summed indices 32*half + 8g .. +7.  Where those of
// the wave's first subtile lie is held in registers (N subtiles of a transposed
// operand, whose places are an exclusive or apart); other rows, halves and slots
// are a constant away.
template <int ROWS, bool CONTIG, int N>
struct Reader {
    static constexpr int COUNT = CONTIG ? 2 : N;
    uint32_t at[COUNT];
    __device__ inline Reader(const uint8_t* lds, int row0, int lane)
    {
        const int r = lane & 15, g = lane >> 4;
        const uint32_t base = (uint32_t)(uintptr_t)(lvoid*)lds;
#pragma unroll
        for (int i = 0; i < COUNT; ++i)
            if constexpr (CONTIG) {
                at[i] = base + (row0 + r) * 128 + (((i * 4 + g) ^ swizzle(r)) << 4);
            } else {
                constexpr int PIECES = ROWS / 8;
                const int t = g * 8 + (r >> 2);
                at[i] = base + t * ROWS * 2 + (((row0 / 8 + 2 * i + (r >> 1 & 1)) ^ turn<PIECES>(t)) << 4) + ((r & 1) << 3);
            }
    }
    __device__ inline void move(uint32_t by)
    {
#pragma unroll
        for (int i = 0; i < COUNT; ++i)
            at[i] += by;
    }
    // The subtile `down` rows (CONTIG) below the first, or number i; `off` bytes further on.
    __device__ __forceinline__ v8b read(int half, int i, int down, int off) const
    {
        if constexpr (CONTIG) {
            typedef __attribute__((address_space(3))) const v8b lv8b;
            return *(lv8b*)(uintptr_t)(at[half] + down * 128 + off);
        } else {
            const uintptr_t p = at[i] + half * 32 * ROWS * 2 + off;      // (terms 4 apart share the turn)
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lv4s*)p);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lv4s*)(p + 4 * ROWS * 2));
            typedef short v8s __attribute__((ext_vector_type(8)));
            return __builtin_bit_cast(v8b, (v8s)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

// --- epilogues: eight consecutive outputs of a row ---------------------------------------------

__device__ inline void open8(const v4u& u, float (&f)[8])
{
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        f[2 * c] = bf16_lo(u[c]);
        f[2 * c + 1] = bf16_hi(u[c]);
    }
}
__device__ inline v4u load8(const uint16_t* p) { return *(const v4u*)p; }
// Results are stored past the caches where a wave's stores are whole lines, which
// all bf16 ones are: to the weights 256 experts of 128 rows, 2048 x 1024 370 us so and 455
// without, forward 295 and 319, 8192 x 8192 x 8192 775 and 787; nothing is lost where
// the next call reads them (4096 x 4096 after itself 204 and 206 us, 1024 rows of 1024
// alike).  Half lines are not: fp32 weights' gradients took 446 us so, 296 without.
__device__ inline void store_past(uint16_t* p, v4u u) { __builtin_nontemporal_store(u, (v4u*)p); }
__device__ inline void store8(uint16_t* p, const float (&f)[8])
{
    store_past(p, v4u{bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3]), bf16_pack(f[4], f[5]), bf16_pack(f[6], f[7])});
}
__device__ inline void store8(float* p, const float (&f)[8])
{
    ((v4f*)p)[0] = v4f{f[0], f[1], f[2], f[3]};
    ((v4f*)p)[1] = v4f{f[4], f[5], f[6], f[7]};
}
__device__ inline void add8(const v4u& u, float (&f)[8])
{
    float r[8];
    open8(u, r);
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

__device__ inline void activate8(int act, float (&z)[8])
{
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            z[c] = z[c] <= 0.0f ? 0.0f : z[c];
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            z[c] *= normal_cdf(z[c], bell(z[c]));
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            z[c] = silu(z[c]);
    }
}
// z to the activation's slopes there.
__device__ inline void slopes8(int act, float (&z)[8])
{
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            z[c] = z[c] > 0.0f ? 1.0f : 0.0f;
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float e = bell(z[c]);
            z[c] = fmaf(z[c] * INV_SQRT_2PI, e, normal_cdf(z[c], e));
        }
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            z[c] = silu_slope(z[c]);
    }
}

// What a call reads for eight outputs: bias, pre-activations, residual (with
// SWIGLU of both halves).
struct Extra {
    v4u z[2], residual[2];
};

template <Kind KIND, bool GATED>
struct Finish {
    static constexpr bool FWD = KIND == Kind::FORWARD;
    const Linear& p;
    __device__ inline explicit Finish(const Linear& p_) : p(p_) {}

    __device__ inline Extra fetch(int64_t row, int col) const
    {
        Extra e{};
        const bool two = !FWD && p.act == MOE_ACT_SWIGLU;
        const int width = FWD ? (GATED ? p.n / 2 : p.n) : two ? 2 * p.k : p.k;
        const int64_t at = row * width + col;
        if (!FWD && p.z_in) {
            e.z[0] = load8(p.z_in + at);
            if (two)
                e.z[1] = load8(p.z_in + at + p.k);
        }
        if (p.residual) {
            e.residual[0] = load8(p.residual + at);
            if (two)
                e.residual[1] = load8(p.residual + at + p.k);
        }
        return e;
    }
    __device__ inline void fetch_bias(int expert, int col, v4u (&bias)[2]) const
    {
        bias[0] = bias[1] = v4u{0, 0, 0, 0};
        if (FWD && p.bias) {
            bias[0] = load8(p.bias + (int64_t)expert * p.n + col);
            if (GATED)
                bias[1] = load8(p.bias + (int64_t)expert * p.n + p.n / 2 + col);
        }
    }
    // a: the sums (GATED: of the gate; b: of up)
    __device__ inline void operator()(int64_t row, int col, float (&a)[8], float (&b)[8], const Extra& e,
                                      const v4u (&bias)[2]) const
    {
        if constexpr (FWD) {
            if (p.bias) {
                add8(bias[0], a);
                if (GATED)
                    add8(bias[1], b);
            }
            if (p.z_out) {
                store8(p.z_out + row * p.n + col, a);
                if (GATED)
                    store8(p.z_out + row * p.n + p.n / 2 + col, b);
            }
            if constexpr (GATED) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    a[c] = silu(a[c]) * b[c];
            } else if (p.act != MOE_ACT_NONE) {
                activate8(p.act, a);
            }
            if (p.residual)
                add8(e.residual[0], a);
            store_out(p, row * (GATED ? p.n / 2 : p.n) + col, a);
        } else if (p.act == MOE_ACT_SWIGLU) {
            float g[8], u[8];
            open8(e.z[0], g);
            open8(e.z[1], u);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float z = g[c];
                g[c] = a[c] * u[c] * silu_slope(z);
                u[c] = a[c] * silu(z);
            }
            if (p.residual) {
                add8(e.residual[0], g);
                add8(e.residual[1], u);
            }
            const int64_t at = row * 2 * p.k + col;
            store_out(p, at, g);
            store_out(p, at + p.k, u);
        } else {
            if (p.act != MOE_ACT_NONE) {
                float z[8];
                open8(e.z[0], z);
                slopes8(p.act, z);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    a[c] *= z[c];
            }
            if (p.residual)
                add8(e.residual[0], a);
            store_out(p, row * p.k + col, a);
        }
    }
};

// --- tiles -------------------------------------------------------------------------------------

// Large tiles, which are bound by their products, go to the XCDs in short runs:
// to the weights 16 experts of 2048 rows, 4096 x 7168, 1824 -> 1629 us and 7168 x 2048
// 897 -> 834, forward 1592 -> 1538 and 905 -> 879.  Small ones, which are bound by
// the weights they stream, go in one run each: 64 experts of 31 rows, 4096 x 2048,
// 187 us so and 210 in short runs.
template <class C>
constexpr bool TURNS = C::BM >= 128;

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

template <int BM, bool TURNS>
__device__ inline bool find_rows(const Linear& p, int n_tiles, int64_t id, Place& at)
{
    if (p.offsets) {
        const int lane = anew(threadIdx.x & (WAVE - 1));
        const bool found = p.E <= 4 * WAVE ? find_tile<BM, 4, TURNS>(p.offsets, p.E, p.rows, n_tiles, at, id, lane)
                                           : find_tile<BM, 16, TURNS>(p.offsets, p.E, p.rows, n_tiles, at, id, lane);
        at.e = __builtin_amdgcn_readfirstlane(at.e);         // (uniform already, which the compiler cannot tell)
        at.m0 = __builtin_amdgcn_readfirstlane(at.m0);
        at.rows = __builtin_amdgcn_readfirstlane(at.rows);
        at.n_tile = __builtin_amdgcn_readfirstlane(at.n_tile);
        return found;
    }
    const int m_tiles = (int)((p.rows + BM - 1) / BM);
    int64_t t;
    if (!tile_of_id<TURNS>(id, (int64_t)m_tiles * n_tiles, t))
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

// One tile's product.
struct Work {
    Side us, vs;              // of as many terms
    __device__ inline int steps() const { return parts_of(us.terms, STEP); }
};

// LDS rows of V's subtiles: the wave's first, and how far below it subtile j is; gated tiles
// keep the gate's rows in their first half.
template <class C, bool GATED>
__device__ inline int v_row_of(int wn)
{
    return wn * (GATED ? C::TN / 2 : C::TN);
}
template <class C, bool GATED>
__device__ constexpr int v_down(int j)
{
    return GATED ? (j < C::NT / 2 ? 0 : C::BN / 2) + j % (C::NT / 2) * 16 : j * 16;
}

template <class C>
struct Sums {
    v4f acc[C::NT][C::MT];
    // Sums of U alone (the bias' gradient), by products with ones: the waves that share U's rows
    // share its subtiles, and one tile of those that share U's rows has them (`mine`: the subtiles
    // of this wave and tile).  A branch ahead of each, against a second main loop for such tiles,
    // keeps the registers that the loop has; pairs of terms added by the vector unit's dot product
    // instead took 1240 us where this takes 930 (32768 rows, 16 experts, 7168 x 2048; 880 without).
    static constexpr int ALONE = (C::MT + C::WN - 1) / C::WN;
    v4f alone[ALONE];
    uint32_t mine;
    __device__ inline void clear(uint32_t mine_)
    {
        const v4f zero{0.0f, 0.0f, 0.0f, 0.0f};
        mine = mine_;
#pragma unroll
        for (int i = 0; i < ALONE; ++i)
            alone[i] = zero;
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
#pragma unroll
            for (int j = 0; j < C::NT; ++j)
                acc[j][i] = zero;
    }
    static __device__ inline uint32_t of_wave(int wn) { return ((1u << ALONE) - 1) << (wn * ALONE); }
    template <bool BIAS>
    __device__ inline void add(int i, const v8b (&vf)[C::NT], v8b uf)
    {
#pragma unroll
        for (int j = 0; j < C::NT; ++j)
            acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[j], uf, acc[j][i], 0, 0, 0);
        if constexpr (BIAS)
            if (mine >> i & 1) {
                const int one = anew(0x3F803F80);        // two ones
                typedef int v4i __attribute__((ext_vector_type(4)));
                alone[i % ALONE] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(v8b, v4i{one, one, one, one}), uf, alone[i % ALONE], 0, 0, 0);
            }
    }
};

// Where nothing but a rounding is left to do: rounded sums through the wave's 4 KB of LDS, two parts
// of 16 rows of U by 64 of V at once.  Half the bytes of the fp32 way below and half its turns: 32768
// rows to 7168 columns by a sum of 256 184 us against 272, 8192 x 8192 x 8192 720 against 733.
template <class C, class Tiles>
__device__ __forceinline__ void hand_over_plain(const Sums<C>& sums, int u_rows, int v_rows, uint16_t* part, int wm, int wn,
                                                int lane, Tiles& tiles)
{
    constexpr int PARTS = C::MT > 1 ? 2 : 1;
    const int r = lane & 15, g = lane >> 4;
    // 16-byte piece q of row r lies at place q ^ r % 8
    auto place = [&](int row, int q) { return part + row * 64 + ((q ^ (row & 7)) << 3); };
#pragma unroll 1
    for (int i = 0; i < C::MT; i += PARTS) {
        // lane (r, g) holds row r of U and rows 4g .. 4g+3 of each subtile of V
#pragma unroll
        for (int s = 0; s < C::MT; ++s)
            if (s / PARTS * PARTS == i)
#pragma unroll
                for (int j = 0; j < C::NT; ++j) {
                    const v4f a = sums.acc[j][s];
                    *(v2u*)(place(s % PARTS * 16 + r, j * 2 + (g >> 1)) + ((g & 1) << 2)) =
                        v2u{bf16_pack(a[0], a[1]), bf16_pack(a[2], a[3])};
                }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int q = 0; q < 2 * PARTS; ++q) {
            const int row = q * 8 + (lane >> 3), c = lane & 7;
            const int u = C::u_row_of(i, wm) + row, v = wn * 64 + c * 8;
            const v4u o = *(const v4u*)place(row, c);
            if (u < u_rows && v < v_rows)
                tiles.finish_plain(u, v, o);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// The gated product's, without a residual, in bf16: bias and activation in the sums' own layout,
// rounded, and through the workgroup's LDS, 128 rows of U at a time: a wave has 32 columns of the
// gate and of up, which alone would be stored as half lines.  Against the way below, with half
// lines past the caches, and with them in the caches: 32768 rows, 8 experts, 2048 x 512 117 us, 123
// and 113, 256 experts, 2048 x 1024 292, 296 and 315, 16 experts, 7168 x 2048 885, 906 and 880.
template <class C, class Tiles>
__device__ __forceinline__ void hand_over_gated(const Sums<C>& sums, int u_rows, int f_rows, uint8_t* lds, int wave, int lane,
                                                Tiles& tiles)
{
    constexpr int F = C::BN / 2, SLICE = C::DEEP ? C::MT / 2 : C::MT, ROWS = SLICE * C::WM * 16;
    constexpr int PIECES = F / 8;                    // 16-byte pieces of a row of F columns
    static_assert(ROWS * F * 6 <= C::LDS, "gate, up and the product of a slice");
    const int wm = wave % C::WM, wn = wave / C::WM, r = lane & 15, g = lane >> 4;
    // 16-byte piece q of row u lies at place q ^ u % 8; the gate, up, then what they make
    auto place = [&](int of, int u, int q) { return (uint16_t*)lds + (of * ROWS + u) * F + ((q ^ (u & 7)) << 3); };
    float bias[C::NT][4];
#pragma unroll
    for (int j = 0; j < C::NT; ++j)
        tiles.fetch_bias4(wn * 32 + j % 2 * 16 + g * 4, j >= 2, f_rows, bias[j]);
    const bool keep = tiles.keeps_z();
#pragma unroll 1
    for (int i = 0; i < C::MT; ++i) {
        v4f a[C::NT];
#pragma unroll
        for (int s = 0; s < C::MT; ++s)
            if (s == i) {
#pragma unroll
                for (int j = 0; j < C::NT; ++j) {
                    a[j] = sums.acc[j][s];
                    asm volatile("" : "+v"(a[j]));   // (no instruction) merged, the copies would index the sums in memory
                }
            }
        const int u = C::u_row_of(i, wm) % ROWS + r;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                a[j][c] += bias[j][c];
                a[j + 2][c] += bias[j + 2][c];
                y[c] = silu(a[j][c]) * a[j + 2][c];
            }
            const int q = wn * 4 + j * 2 + (g >> 1), low = (g & 1) << 2;
            auto put = [&](int of, float p0, float p1, float p2, float p3) {
                *(v2u*)(place(of, u, q) + low) = v2u{bf16_pack(p0, p1), bf16_pack(p2, p3)};
            };
            if (keep) {
                put(0, a[j][0], a[j][1], a[j][2], a[j][3]);
                put(1, a[j + 2][0], a[j + 2][1], a[j + 2][2], a[j + 2][3]);
            }
            put(2, y[0], y[1], y[2], y[3]);
        }
        if ((i + 1) % SLICE)
            continue;
        meet<0>();
        const int u0 = i / SLICE * ROWS;
#pragma unroll 1
        for (int of = keep ? 0 : 2; of < 3; ++of)
#pragma unroll
            for (int t = 0; t < ROWS * PIECES / C::THREADS; ++t) {
                const int at = t * C::THREADS + wave * WAVE + lane, row = at / PIECES, q = at % PIECES;
                const v4u o = *(const v4u*)place(of, row, q);
                if (u0 + row < u_rows && q * 8 < f_rows)
                    tiles.finish_gated(of, u0 + row, q * 8, o);
            }
        meet<0>();
    }
}

// Hands a wave's sums to the tiles' finish, eight consecutive outputs at a time:
// 16 rows of U by the wave's 64 of V go through 4 KB of LDS of its own, so that
// its stores are whole lines (four lanes of 16 bytes from the sums' own layout
// are half lines), its code is that of one such part, and what the next part
// reads from memory is on its way meanwhile.
template <class C, bool GATED, class Tiles>
__device__ __forceinline__ void hand_over_rows(const Sums<C>& sums, int u_rows, int v_rows, float* part, int wm, int wn, int lane,
                                               Tiles& tiles)
{
    constexpr int PASSES = GATED ? 1 : 2;            // by 8 (GATED: 16) rows of U
    // 16-byte piece q of row r lies at place q ^ r: rows apart in the banks both ways
    auto place = [&](int row, int q) { return part + row * 64 + ((q ^ row) << 2); };
    const int row0 = GATED ? lane >> 2 : lane >> 3, col = GATED ? lane & 3 : lane & 7;
    const int v = (GATED ? wn * 32 : wn * 64) + col * 8;
    const bool live_v = v < v_rows;
    v4u bias[2];
    tiles.fetch_bias(live_v ? v : 0, bias);
    auto fetch = [&](int i, Extra (&e)[PASSES]) {
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
            const int u = C::u_row_of(i, wm) + q * 8 + row0;
            if (u < u_rows && live_v)
                e[q] = tiles.fetch(u, v);
        }
    };
    Extra now[PASSES], next[PASSES];
    fetch(0, next);
#pragma unroll 1
    for (int i = 0; i < C::MT; ++i) {
#pragma unroll
        for (int q = 0; q < PASSES; ++q)
            now[q] = next[q];
        if (i + 1 < C::MT)
            fetch(i + 1, next);
        // lane (r, g) holds row r of U and rows 4g .. 4g+3 of each subtile of V
#pragma unroll
        for (int s = 0; s < C::MT; ++s)
            if (s == i)
#pragma unroll
                for (int j = 0; j < C::NT; ++j)
                    *(v4f*)place(lane & 15, j * 4 + (lane >> 4)) = sums.acc[j][s];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
            const int row = q * 8 + row0, u = C::u_row_of(i, wm) + row;
            float a[8], b[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4f x = *(const v4f*)place(row, col * 2 + h);
                v4f y;
                if (GATED)
                    y = *(const v4f*)place(row, 8 + col * 2 + h);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    a[4 * h + c] = x[c];
                    if (GATED)
                        b[4 * h + c] = y[c];
                }
            }
            if (u < u_rows && live_v)
                tiles.finish(u, v, a, b, now[q], bias);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// fp32 outputs that nothing is done to, of the weights' gradient: four and four of a lane's lie 32
// apart, so that stores are whole lines.
template <class C, class Tiles>
__device__ __forceinline__ void hand_over_fp32(const Sums<C>& sums, int u_rows, int v_rows, float* part, int wm, int wn, int lane,
                                               Tiles& tiles)
{
    auto place = [&](int row, int q) { return part + row * 64 + ((q ^ row) << 2); };
    const int row0 = lane >> 3, col = lane & 7;
#pragma unroll 1
    for (int i = 0; i < C::MT; ++i) {
#pragma unroll
        for (int s = 0; s < C::MT; ++s)
            if (s == i)
#pragma unroll
                for (int j = 0; j < C::NT; ++j)
                    *(v4f*)place(lane & 15, j * 4 + (lane >> 4)) = sums.acc[j][s];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = q * 8 + row0, u = C::u_row_of(i, wm) + row;
                const v4f x = *(const v4f*)place(row, h * 8 + col);
                const int v = wn * 64 + h * 32 + col * 4;
                if (u < u_rows && v < v_rows)
                    tiles.finish4(u, v, x);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// A tile's sums to its outputs.
template <class C, bool GATED, bool BIAS, class Tiles>
__device__ __forceinline__ void hand_over(Sums<C>& sums, int u_rows, int v_rows, uint8_t* lds, int wave, int lane,
                                          Tiles& tiles)
{
    static_assert(C::NT == 4, "a wave has 64 rows of V");
    const int wm = wave % C::WM, wn = wave / C::WM;
    float* const part = (float*)(lds + wave * 4096);
    if constexpr (BIAS)
        if (sums.mine)
#pragma unroll
            for (int i = 0; i < Sums<C>::ALONE; ++i) {
                const int u = C::u_row_of(wn * Sums<C>::ALONE + i, wm) + lane;
                if (wn * Sums<C>::ALONE + i < C::MT && lane < 16 && u < u_rows)
                    tiles.finish_bias(u, sums.alone[i][0]);
            }
    if (!GATED && tiles.plain()) {
        hand_over_plain(sums, u_rows, v_rows, (uint16_t*)part, wm, wn, lane, tiles);
        return;
    }
    if constexpr (GATED)
        if (tiles.plain_gated()) {
            hand_over_gated(sums, u_rows, v_rows, lds, wave, lane, tiles);
            return;
        }
    if constexpr (Tiles::ROWS)
        hand_over_rows<C, GATED>(sums, u_rows, v_rows, part, wm, wn, lane, tiles);
    else
        hand_over_fp32(sums, u_rows, v_rows, part, wm, wn, lane, tiles);
}

// The product of one tile, with S stages of both operands in LDS: for tiles of which two workgroups
// fit a CU (128 x 256: one), whose loads, products and epilogues overlap.  Where weights bound them
// they arrive at 6.5 TB/s (64 experts, 256 rows, 4096 x 2048 166 us).
template <class C, bool U_CONTIG, bool V_CONTIG, bool GATED, bool BIAS>
__device__ __forceinline__ void sum_tile(const Work& w, uint8_t* lds, int wave, int lane, Sums<C>& sums)
{
    const int wm = wave % C::WM, wn = wave / C::WM;
    const int steps = w.steps();
    auto issue = [&](int step, uint8_t* st, auto tail) {
        load_side<C, C::BN, V_CONTIG, GATED, tail>(w.vs, 0, step, st, wave, lane);
        load_side<C, C::BM, U_CONTIG, false, tail>(w.us, 0, step, st + C::V_BYTES, wave, lane);
    };
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
    const Reader<C::BN, V_CONTIG, C::NT> v_reader(lds, v_row_of<C, GATED>(wn), lane);
    const Reader<C::BM, U_CONTIG, C::MT> u_reader(lds + C::V_BYTES, wm * C::TM, lane);
    auto read = [&](int slot, int h) {
#pragma unroll
        for (int j = 0; j < C::NT; ++j)
            vf[h][j] = v_reader.read(h, j, v_down<C, GATED>(j), slot * C::STAGE);
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
            uf[h][i] = u_reader.read(h, i, i * 16, slot * C::STAGE);
    };
    auto multiply = [&](int h) {
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
            sums.template add<BIAS>(i, vf[h], uf[h][i]);
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
        read(0, 0);
    }
    int slot = 0;
    auto step_of = [&](int step, auto steady, auto tail) {
        uint8_t* st = lds + slot * C::STAGE;
        read(slot, 1);
        multiply(0);
        meet<decltype(steady)::value ? (C::S - 2) * C::LOADS : 0>();
        if constexpr (decltype(steady)::value)
            issue(step + C::S, st, tail);
        slot = slot + 1 == C::S ? 0 : slot + 1;
        read(slot, 0);                               // (past the last stage: stale, never used)
        multiply(1);
    };
    int step = 0;
    for (; step + C::S < steps - 1; ++step)
        step_of(step, std::true_type{}, std::false_type{});
    if (step + C::S < steps)
        step_of(step++, std::true_type{}, std::true_type{});
    for (; step < steps; ++step)
        step_of(step, std::false_type{}, std::false_type{});
}

// The 256 x 256 tile: U in two halves of 128 rows, V's stages in three slots of
// LDS and each half of U's in two, 160 KB.  A step is two phases, one for each
// half of U; a phase's operands are read while the phase before it is
// multiplied, and what has been read by every wave is loaded anew at once, so
// that a load has one and a half to two steps to arrive (with two slots for
// everything, one step).  A phase issues four loads, one beside every eight
// products: two of the half of U that the phase before it was the last to read,
// and half of V's, whose slot was free before.  What bounds it is the matrix unit under
// the card's power limit: by the counters it is busy in 70 to 75% of the cycles, at a
// clock that falls to 1.6 to 1.8 GHz.  8192 x 8192 x 8192 takes 750 to 830 us forward
// (1320 to 1465 TFLOP/s; the library 670 to 770 us, by card and what ran before), 737 to
// 762 to the input (782 to 873) and 760 to 775 to the weights (902 to 985).  A tile costs about 8 us beside
// its steps of 1.4: finding it, the first loads and the epilogue, which nothing hides
// where one workgroup fills a CU.  Tried and slower or the same: 32 x 32 x 16 products
// (4%), a persistent workgroup that loads its next tile during the epilogue (forward
// 2%, to the weights 3%), wave priorities around the products.
template <class C, bool U_CONTIG, bool V_CONTIG, bool GATED>
struct DeepTile {
    static_assert(C::BM == 256 && C::BN == 256 && C::WM == 2 && C::WN == 4, "eight waves of 128 x 64");
    static constexpr int HALF = 128, HALF_BYTES = HALF * STEP * 2, UT = C::MT / 2;
    static constexpr int V_LOADS = loads_of<C>(C::BN), U_LOADS = loads_of<C>(HALF), PHASE = V_LOADS / 2 + U_LOADS;
    static_assert(V_LOADS == 4 && U_LOADS == 2 && C::NT == 4 && UT == 4, "the orders below");

    uint8_t* lds;
    int wave, lane, wm, wn;
    __device__ inline DeepTile(uint8_t* l, int wave_, int lane_)
        : lds(l), wave(wave_), lane(lane_), wm(wave_ % C::WM), wn(wave_ / C::WM)
    {
    }
    __device__ inline uint8_t* v_slot(int s) const { return lds + s * C::V_BYTES; }
    __device__ inline uint8_t* u_slot(int half, int step) const
    {
        return lds + 3 * C::V_BYTES + (half * 2 + (step & 1)) * HALF_BYTES;
    }
    // Nothing is loaded behind the last stage, whose tail is zeros; `inner`: it is not the last.
    template <class Inner>
    __device__ __forceinline__ void load_v(const Work& w, int steps, int step, int slot, Inner inner, int from, int to) const
    {
        if (inner || step < steps - 1)
            load_side<C, C::BN, V_CONTIG, GATED, false>(w.vs, 0, step, v_slot(slot), wave, lane, from, to);
        else if (step == steps - 1)
            load_side<C, C::BN, V_CONTIG, GATED, true>(w.vs, 0, step, v_slot(slot), wave, lane, from, to);
    }
    template <class Inner>
    __device__ __forceinline__ void load_u(const Work& w, int steps, int half, int step, Inner inner, int from, int to) const
    {
        uint8_t* const slot = u_slot(half, step);
        if (inner || step < steps - 1)
            load_side<C, HALF, U_CONTIG, false, false>(w.us, half * HALF, step, slot, wave, lane, from, to);
        else if (step == steps - 1)
            load_side<C, HALF, U_CONTIG, false, true>(w.us, half * HALF, step, slot, wave, lane, from, to);
    }
    // The first loads of a tile, in the order in which the phases issue theirs.
    __device__ __forceinline__ void start(const Work& w) const
    {
        constexpr std::false_type any{};
        const int steps = w.steps();
        load_u(w, steps, 0, 0, any, 0, 2);
        load_v(w, steps, 0, 0, any, 0, 4);
        load_u(w, steps, 1, 0, any, 0, 2);
        load_v(w, steps, 1, 1, any, 0, 2);
        load_u(w, steps, 0, 1, any, 0, 2);
        load_v(w, steps, 1, 1, any, 2, 4);
        load_u(w, steps, 1, 1, any, 0, 2);
        load_v(w, steps, 2, 2, any, 0, 2);
    }
    template <bool BIAS>
    __device__ __forceinline__ void sum(const Work& w, Sums<C>& sums) const
    {
        constexpr std::false_type any{};
        const int steps = w.steps();
        v8b vf[2][C::NT], uf[2][2][UT];              // V: [k half]; U: [row half][k half]
        Reader<C::BN, V_CONTIG, C::NT> v_reader(lds, v_row_of<C, GATED>(wn), lane);      // of this step's slot
        Reader<HALF, U_CONTIG, UT> u_reader(u_slot(0, 0), wm * 64, lane);
        auto read_v = [&](int h, int j) { vf[h][j] = v_reader.read(h, j, v_down<C, GATED>(j), 0); };
        auto read_u = [&](int half, int h, int i) {
            uf[half][h][i] = u_reader.read(h, i, i * 16, half * 2 * HALF_BYTES);
        };
        // Four products, behind the reads and loads before them.
        auto products = [&](int half, int h, int i) {
            sums.template add<BIAS>(half * UT + i, vf[h], uf[half][h][i]);
            __builtin_amdgcn_sched_barrier(0);
        };
        if (steps >= 3)
            meet<3 * PHASE>();
        else
            meet<0>();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            read_v(0, q);
            read_u(0, 0, q);
            read_u(0, 1, q);
        }
        if (steps >= 3)
            meet<2 * PHASE>();
        else
            meet<0>();
        int now = 0, last = 2;                       // V's slots of this step and the one before it
        auto step_of = [&](int step, auto steady) {
            // every wave has read the first half of U and V's first indices of this step
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (q < 2) {
                    read_v(1, 2 * q);
                    read_v(1, 2 * q + 1);
                } else if (q < 6) {
                    read_u(1, (q - 2) / 2, (q & 1) * 2);
                    read_u(1, (q - 2) / 2, (q & 1) * 2 + 1);
                }
                if (q == 0 || q == 2)
                    load_u(w, steps, 0, step + 2, steady, q / 2, q / 2 + 1);
                if (q == 4 || q == 6)
                    load_v(w, steps, step + 2, last, steady, q / 2, q / 2 + 1);
                products(0, q / 4, q % 4);
            }
            meet<steady ? 2 * PHASE : 0>();
            // ... and V and the second half of U; what is read past the last stage is stale, and not used
            last = now;
            now = now == 2 ? 0 : now + 1;
            v_reader.move(now ? C::V_BYTES : -2 * C::V_BYTES);
            u_reader.move(step & 1 ? -HALF_BYTES : HALF_BYTES);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (q < 4) {
                    read_u(0, q / 2, (q & 1) * 2);
                    read_u(0, q / 2, (q & 1) * 2 + 1);
                } else if (q < 6) {
                    read_v(0, (q & 1) * 2);
                    read_v(0, (q & 1) * 2 + 1);
                }
                if (q == 0 || q == 2)
                    load_u(w, steps, 1, step + 2, steady, q / 2, q / 2 + 1);
                if (q == 4 || q == 6)
                    load_v(w, steps, step + 3, last, steady, q / 2 - 2, q / 2 - 1);
                products(1, q / 4, q % 4);
            }
            meet<steady ? 2 * PHASE : 0>();
        };
        int step = 0;
        for (; step + 3 < steps - 1; ++step)
            step_of(step, std::true_type{});
        for (; step < steps; ++step)
            step_of(step, any);
    }
};

template <class C, bool U_CONTIG, bool V_CONTIG, bool GATED, bool BIAS, class Tiles>
__device__ __forceinline__ void sum_and_hand_over(uint8_t* lds, Tiles& tiles, const Work& w, int wave, int lane)
{
    Sums<C> sums;
    sums.clear(BIAS && tiles.with_bias() ? Sums<C>::of_wave(wave / C::WM) : 0);
    if constexpr (C::DEEP) {
        const DeepTile<C, U_CONTIG, V_CONTIG, GATED> tile(lds, wave, lane);
        tile.start(w);
        tile.template sum<BIAS>(w, sums);
    } else {
        sum_tile<C, U_CONTIG, V_CONTIG, GATED, BIAS>(w, lds, wave, lane, sums);
        meet<0>();                                   // the last reads, before LDS is written again
    }
    tiles.begin_finish();
    hand_over<C, GATED, BIAS>(sums, w.us.valid, w.vs.valid, lds, wave, anew(lane), tiles);
}

// A workgroup's tile: tiles.next() describes it (false: there is none), and its
// outputs go to tiles.finish().
template <class C, bool U_CONTIG, bool V_CONTIG, bool GATED, bool BIAS, class Tiles>
__device__ __forceinline__ void run_tile(uint8_t* lds, Tiles& tiles)
{
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    Work w;
    if (!tiles.next(workgroup_id(), w))
        return;
    if constexpr (C::DEEP) {
        // an expert's last rows, where half the tile is enough (us, without and with it, of the
        // gradient to the input: 16 experts, 32768 rows, 7168 x 2048 792, 771, of the product 64 experts,
        // 2048 x 4096 541, 528; nothing lost where all tiles are full)
        typedef Block<C::BM / 2, C::BN, C::WM, C::WN, 3> Low;
        static_assert(Low::LDS <= C::LDS && Low::THREADS == C::THREADS, "in the same launch");
        if (w.us.valid <= Low::BM) {
            sum_and_hand_over<Low, U_CONTIG, V_CONTIG, GATED, BIAS>(lds, tiles, w, wave, lane);
            return;
        }
    }
    sum_and_hand_over<C, U_CONTIG, V_CONTIG, GATED, BIAS>(lds, tiles, w, wave, lane);
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
struct RowTiles {
    static constexpr bool ROWS = true, FWD = KIND == Kind::FORWARD;
    int n_tiles, splits;
    Place at;
    Linear args;              // (read once: through the epilogue's loop they stay in scalar registers)

    // columns of an output row's sums, and those that tiles divide
    static __device__ inline int width(const Linear& p) { return FWD ? p.n : p.k; }
    static __device__ inline int f(const Linear& p) { return GATED ? p.n / 2 : width(p); }
    static __device__ inline int first_col(const Place& a) { return a.n_tile * (GATED ? C::BN / 2 : C::BN); }
    __device__ inline bool next(int64_t id, Work& w)
    {
        const Linear& p = arguments();
        if (!find_rows<C::BM, TURNS<C>>(p, n_tiles, id, at))
            return false;
        const int v0 = first_col(at);
        const int64_t total = FWD ? p.k : p.n;
        w.us.ld = (int)total;
        int64_t t0, t1;
        split_range(total, splits, blockIdx.z, t0, t1);
        w.us.base = w.us.upper = (FWD ? p.x : p.dz) + (int64_t)at.m0 * total + t0;
        w.us.valid = at.rows;
        const uint16_t* weights = p.w + (int64_t)at.e * p.n * p.k;
        w.vs.ld = p.k;
        w.vs.base = FWD ? weights + (int64_t)v0 * p.k + t0 : weights + t0 * p.k + v0;
        w.vs.upper = GATED ? w.vs.base + (int64_t)f(p) * p.k : w.vs.base;
        w.vs.valid = min(GATED ? C::BN / 2 : C::BN, f(p) - v0);
        w.us.terms = w.vs.terms = (int)(t1 - t0);
        return true;
    }
    __device__ inline void begin_finish() { args = arguments(); }
    __device__ inline bool with_bias() const { return false; }
    __device__ inline Extra fetch(int u, int v) const
    {
        return splits > 1 ? Extra{} : Finish<KIND, GATED>(args).fetch(at.m0 + u, first_col(at) + v);
    }
    __device__ inline void fetch_bias(int v, v4u (&bias)[2]) const
    {
        Finish<KIND, GATED>(args).fetch_bias(at.e, first_col(at) + v, bias);
    }
    __device__ inline void finish(int u, int v, float (&a)[8], float (&b)[8], const Extra& e, const v4u (&bias)[2]) const
    {
        const Linear& p = args;
        const int64_t row = at.m0 + u;
        const int col = first_col(at) + v;
        if (splits > 1) {
            float* part = (float*)p.workspace + ((int64_t)blockIdx.z * p.rows + row) * width(p) + col;
            store8(part, a);
            if (GATED)
                store8(part + f(p), b);
            return;
        }
        const Finish<KIND, GATED> whole(p);
        whole(row, col, a, b, e, bias);
    }
    __device__ inline void finish_bias(int, float) const {}
    __device__ inline bool plain() const
    {
        const Linear& p = args;
        return splits == 1 && !p.out_f32 && p.act == MOE_ACT_NONE && !p.residual && !(FWD && (p.bias || p.z_out));
    }
    __device__ inline bool plain_gated() const { return splits == 1 && !args.out_f32 && !args.residual; }
    __device__ inline bool keeps_z() const { return args.z_out; }
    // four of the gate's biases, or of up's
    __device__ inline void fetch_bias4(int v, bool up, int f_rows, float (&b)[4]) const
    {
        v2u u{0, 0};
        if (args.bias && v < f_rows)
            u = *(const v2u*)(args.bias + (int64_t)at.e * args.n + (up ? args.n / 2 : 0) + first_col(at) + v);
        b[0] = bf16_lo(u[0]);
        b[1] = bf16_hi(u[0]);
        b[2] = bf16_lo(u[1]);
        b[3] = bf16_hi(u[1]);
    }
    __device__ inline void finish_gated(int of, int u, int v, v4u o) const
    {
        const int64_t row = at.m0 + u;
        uint16_t* out = of == 2 ? (uint16_t*)args.out + row * (args.n / 2) : args.z_out + row * args.n + of * (args.n / 2);
        store_past(out + first_col(at) + v, o);
    }
    __device__ inline void finish_plain(int u, int v, v4u o) const
    {
        store_past((uint16_t*)args.out + (int64_t)(at.m0 + u) * width(args) + first_col(at) + v, o);
    }
};

template <Kind KIND, class C, bool GATED>
__global__ __launch_bounds__(C::THREADS) void linear_kernel(const Linear p, int n_tiles, int splits)
{
    extern __shared__ __align__(1024) uint8_t lds[];
    RowTiles<KIND, C, GATED> tiles{n_tiles, splits};
    run_tile<C, true, KIND == Kind::FORWARD, GATED, false>(lds, tiles);
}

// grad_weight: out rows are an expert's weight rows
template <class C>
struct WeightTiles {
    static constexpr bool ROWS = false;
    int m_tiles, n_tiles, splits;
    struct Spot {
        int e, m, n;
    } at;
    const Linear* args;

    __device__ inline bool next(int64_t id, Work& w)
    {
        const Linear& p = arguments();
        int64_t t;
        if (!tile_of_id<TURNS<C>>(id, (int64_t)p.E * m_tiles * n_tiles, t))
            return false;
        const int per = m_tiles * n_tiles;                   // 2^20 at most (32 x 128 tiles of 65536 x 65536)
        at.e = (int)(t / per);
        tile_in_group(t - (int64_t)at.e * per, m_tiles, n_tiles, at.m, at.n);
        int64_t a, b;
        expert_rows(p, at.e, a, b);
        a = __builtin_amdgcn_readfirstlane((int)a);          // (uniform already, which the compiler cannot tell)
        b = __builtin_amdgcn_readfirstlane((int)b);
        const int u0 = at.m * C::BM, v0 = at.n * C::BN;
        int64_t t0, t1;
        split_range(b - a, splits, blockIdx.z, t0, t1);
        w.us.ld = p.n;
        w.us.base = w.us.upper = p.dz + (a + t0) * p.n + u0;
        w.us.valid = min(C::BM, p.n - u0);
        w.vs.ld = p.k;
        w.vs.base = w.vs.upper = p.x + (a + t0) * p.k + v0;
        w.vs.valid = min(C::BN, p.k - v0);
        w.us.terms = w.vs.terms = (int)(t1 - t0);
        return true;
    }
    __device__ inline void begin_finish() { args = &arguments(); }
    __device__ inline bool with_bias() const { return at.n == 0; }
    __device__ inline int64_t out_at(const Linear& p, int u, int v) const
    {
        return ((int64_t)at.e * p.n + at.m * C::BM + u) * p.k + at.n * C::BN + v;
    }
    __device__ inline bool plain() const { return splits == 1 && !args->out_f32; }
    __device__ inline void finish_plain(int u, int v, v4u o) const
    {
        const Linear& p = *args;
        store_past((uint16_t*)p.out + out_at(p, u, v), o);
    }
    __device__ inline void finish4(int u, int v, v4f o) const
    {
        const Linear& p = *args;
        const int64_t i = out_at(p, u, v);
        if (splits > 1)
            *(v4f*)((float*)p.workspace + (int64_t)blockIdx.z * p.E * p.n * p.k + i) = o;
        else
            __builtin_nontemporal_store(o, (v4f*)((float*)p.out + i));
    }
    __device__ inline void finish_bias(int u, float s) const
    {
        const Linear& p = *args;
        const int64_t biases = (int64_t)p.E * p.n;
        float* out = p.dbias;
        if (splits > 1)
            out = (float*)p.workspace + splits * biases * p.k + blockIdx.z * biases;
        out[(int64_t)at.e * p.n + at.m * C::BM + u] = s;
    }
};

template <class C, bool BIAS>
__global__ __launch_bounds__(C::THREADS) void linear_weight_kernel(const Linear p, int m_tiles, int n_tiles, int splits)
{
    extern __shared__ __align__(1024) uint8_t lds[];
    WeightTiles<C> tiles{m_tiles, n_tiles, splits};
    run_tile<C, false, false, false, BIAS>(lds, tiles);
}

// grad_weight where an expert has a few rows: the weights' gradient is then what
// costs, written once.  A lane has eight columns of x of FEW_ROWS rows in
// registers, a wave goes through 8 weight rows at a time, whose dz are uniform;
// a workgroup has 512 columns by 64 weight rows.  Against the 256 x 256 tile,
// whose one step costs less than finding it, its first loads and its outputs, 64
// experts, 4096 x 2048 (1.07 GB): 184 us against 230 with 1 row each, 181 against
// 237 with 4, 197 against 241 with 6, 227 against 241 with 8, where the vector
// unit's multiply-adds are what bounds it (8 ragged rows each of 8 experts of 4096
// x 4096 63 to 72 against 61 to 64); of small gradients the latencies (16 experts of
// 6 rows, 1000 x 384 14 us against 8).  The choice is by the mean, since the host
// does not know the rows: an expert that holds many of them goes through its rows in
// the few workgroups of its own weights.  448 rows of 64 experts, 4096 x 2048, 202 us
// with 7 rows each, 436 with 385 of them on one; 512 x 2048 34 and, all on one, 323;
// 7168 rows of 1024 experts, 512 x 512, 116 and, all on one, 6900.
constexpr int FEW_ROWS = 8, FEW_COLS = 512, FEW_N = 64;
constexpr int FEW_MEAN = 7;                      // rows per expert
constexpr int64_t FEW_LEAST = 1 << 24;           // weights

__global__ __launch_bounds__(256) void linear_weight_few_kernel(const Linear p, int n_chunks, int k_chunks)
{
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    int64_t id = workgroup_id();
    const int kc = (int)(id % k_chunks);
    id /= k_chunks;
    const int e = (int)(id / n_chunks), nc = (int)(id % n_chunks);
    if (e >= p.E)
        return;
    int64_t a, b;
    expert_rows(p, e, a, b);
    const int col = kc * FEW_COLS + lane * 8;
    const bool live = col < p.k;
    constexpr int EACH = FEW_N / 4;                  // weight rows per wave
#pragma unroll 1
    for (int n0 = nc * FEW_N + wave * EACH; n0 < min(nc * FEW_N + (wave + 1) * EACH, p.n); n0 += 8) {
        float acc[8][8] = {}, alone = 0.0f;
#pragma unroll 1
        for (int64_t r0 = a; r0 < b; r0 += FEW_ROWS) {
            v4u x[FEW_ROWS];
#pragma unroll
            for (int r = 0; r < FEW_ROWS; ++r)
                x[r] = live && r0 + r < b ? load8(p.x + (r0 + r) * p.k + col) : v4u{0, 0, 0, 0};
#pragma unroll
            for (int r = 0; r < FEW_ROWS; ++r)
                if (r0 + r < b) {
                    float d[8], v[8];
                    open8(load8(p.dz + (r0 + r) * p.n + n0), d);
                    open8(x[r], v);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            acc[j][c] = fmaf(d[j], v[c], acc[j][c]);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        alone += lane == j ? d[j] : 0.0f;
                }
        }
        const int64_t at = (int64_t)e * p.n + n0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (live)
                store_out(p, (at + j) * p.k + col, acc[j]);
        if (p.dbias && kc == 0 && lane < 8)
            p.dbias[at + lane] = alone;
    }
}

// --- joins of split sums -----------------------------------------------------------------------

// The sum of eight neighbours over the splits, in their order, four splits in flight: a launch of
// its own, mostly latency (128 x 256 in eight splits 4.1 us behind a product of 7.8).
__device__ inline void add_parts(const float* part, int64_t stride, int splits, float (&v)[8])
{
    constexpr int AHEAD = 4;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        v[c] = 0.0f;
    for (int s = 0; s < splits; s += AHEAD) {
        v4f a[AHEAD][2];
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            const v4f* at = (const v4f*)(part + min(s + q, splits - 1) * stride);
            a[q][0] = at[0];
            a[q][1] = at[1];
        }
#pragma unroll
        for (int q = 0; q < AHEAD; ++q)
            if (s + q < splits)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    v[c] += a[q][c / 4][c % 4];
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
    const Finish<KIND, GATED> finish(p);
    const Extra extra = finish.fetch(row, col);
    v4u bias[2];
    finish.fetch_bias(e, col, bias);
    const int64_t stride = p.rows * width;
    const float* part = (const float*)p.workspace + row * width + col;
    float a[8], b[8];
    add_parts(part, stride, splits, a);
    if (GATED)
        add_parts(part + f, stride, splits, b);
    finish(row, col, a, b, extra, bias);
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
// sums over many rows of it follow, in which a value next to a border that is
// rounded the other way counts more than all of their own roundings (one in
// 50000 values, 2^-8 of itself).  So the slopes are the formulas' elementary
// operations in fp32 in the order written here, each rounded once and none fused:
// whoever forms them so gets the same bf16 numbers.  Not so GELU's below -2:
// there 1 + erf has lost what it is off by, 2^-24 of 1, which is 13 of 2^-24 of the
// slope at -2, 3% at -6, and the lower tail is formed as in the products'
// epilogues.  So each slope is off by a few roundings of 2^-24 of its two parts.
// The vector unit bounds them: 32768 x 4096 GELU 212 us (190 without the tail), SILU
// 154, SWIGLU 118, 3.8 to 5.7 TB/s.
__device__ inline float logistic_by_steps(float z)
{
#pragma clang fp contract(off)
    return 1.0f / (1.0f + expf(-z));
}
// (d * p) * (1 + z * (1 - p))
__device__ inline float silu_grad_by_steps(float d, float z, float p)
{
#pragma clang fp contract(off)
    return d * p * (1.0f + z * (1.0f - p));
}
__device__ inline float gelu_grad_by_steps(float d, float z)
{
#pragma clang fp contract(off)
    const float e = expf(-0.5f * z * z);             // (z is bf16: its square is exact)
    float cdf = 0.5f * (1.0f + erff(z * 0.70710678118654752f));
    if (z < -2.0f)
        cdf = normal_cdf(z, e);
    return d * (cdf + z * e * 0.39894228040143268f);
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
    float d[8], z[8], v[8];
    open8(load8(dy + row * f + col), d);
    uint16_t* out = (uint16_t*)p.out + row * p.n + col;
    open8(load8(p.z_in + row * p.n + col), z);
    if (p.act == MOE_ACT_SWIGLU) {
        float u[8], w[8];
        open8(load8(p.z_in + row * p.n + f + col), u);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float s = logistic_by_steps(z[c]);
            v[c] = silu_grad_by_steps(d[c] * u[c], z[c], s);
            w[c] = d[c] * z[c] * s;
        }
        store8(out, v);
        store8(out + f, w);
        return;
    }
    if (p.act == MOE_ACT_RELU) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            v[c] = z[c] > 0.0f ? d[c] : 0.0f;
    } else if (p.act == MOE_ACT_GELU) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            v[c] = gelu_grad_by_steps(d[c], z[c]);
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            v[c] = silu_grad_by_steps(d[c], z[c], logistic_by_steps(z[c]));
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

// The tiles of a launch, from high to low.
enum class Form { T256, T128W, T128, T64, T32W, T32, FEW };

template <Form F>
struct Tile;
template <>
struct Tile<Form::T256> : Block<256, 256, 2, 4, 2> {};
template <>
struct Tile<Form::T128W> : Block<128, 256, 2, 4, 3> {};
template <>
struct Tile<Form::T128> : Block<128, 128, 2, 2, 2> {};
template <>
struct Tile<Form::T64> : Block<64, 128, 2, 2, 3> {};
template <>
struct Tile<Form::T32W> : Block<32, 256, 2, 4, 2> {};
template <>
struct Tile<Form::T32> : Block<32, 128, 2, 2, 4> {};

template <class F>
auto with_tile(Form form, F f)
{
    switch (form) {
    case Form::T256: return f(Tile<Form::T256>{});
    case Form::T128W: return f(Tile<Form::T128W>{});
    case Form::T128: return f(Tile<Form::T128>{});
    case Form::T64: return f(Tile<Form::T64>{});
    case Form::T32W: return f(Tile<Form::T32W>{});
    default: return f(Tile<Form::T32>{});
    }
}

struct Plan {
    Form form;
    int m_tiles, n_tiles;     // m_tiles: of grad_weight
    int64_t groups;
    int splits;
};

void set_tiles(Plan& s, Form form, Kind kind, bool gated, int64_t rows, int E, int n, int k)
{
    s.form = form;
    with_tile(form, [&](auto c) {
        typedef decltype(c) C;
        const int width = kind == Kind::FORWARD ? n : k, bn = gated ? C::BN / 2 : C::BN;
        s.n_tiles = ((gated ? width / 2 : width) + bn - 1) / bn;
        s.m_tiles = (n + C::BM - 1) / C::BM;
        s.groups = kind == Kind::WEIGHT ? ((int64_t)E * s.m_tiles * s.n_tiles + 7) / 8 * 8
                                        : workgroups(rows, E, C::BM, s.n_tiles);
    });
}

// The tile and the number of splits that an estimate of the launch's time finds
// best: rounds of workgroups, each of its steps and of what a tile costs beside
// them (finding it, its first loads, its outputs); a join where sums are split
// (a second launch, the partial sums written and read); never less than the
// bytes take.  Steps and tiles (us, all workgroups of a CU together; other by a
// factor to the weights) are fitted to 120 measured shapes of all three
// products, from 1 to 32768 rows, 1 to 256 experts and 8 to 7168 columns, every
// tile and split of each (the choice was 1.7% above the best of them in the
// mean, 17% at most).  Both sides of some choices, us:
//  - 256 x 256 against 128 x 256 and 128 x 128: 4096 x 4096 x 4096 105, 143,
//    166; 16 experts, 32768 rows, 4096 x 2048 489, 540, 618; 64 experts of about
//    128 rows, 2048 x 2048 154, 135, 144 (64 x 128: 155);
//  - 64 x 128 against 128 x 128: one expert, 1000 rows, 4096 x 4096 43.8
//    against 45.9 (256 x 256 in four splits 54.5); 64 experts of about 64 rows 121
//    against 134;
//  - 32 x 128 against 32 x 256: 64 experts, 16 rows, 4096 x 2048 37.4 against 36.4,
//    one expert, 1000 rows, 512 x 512 7.4 against 8.1; against 64 x 128: 8 experts of
//    about 37 rows, 1000 x 384, to the input 8.7 against 10.4;
//  - 128 x 128 against 256 x 256 to the weights: 8 experts of about 250 rows, 4096 x
//    2048 57 against 64;
//  - splits: 128 rows, 256 x 7168 in 1, 4, 8, 16 splits 20, 13.6, 11.6, 11.7; 64
//    rows, 4096 x 4096 in 1, 2, 4, 8 24, 14.5, 13.1, 14.9.
// Eight splits at most leave CUs idle where a small gradient to the weights sums
// many rows: 64 x 64 of 32768 rows 27 us, of 131072 89, for 8 and 34 MB.
struct Cost {
    Form form;
    int bm, bn, per_cu;
    float step, tile;
    float last;               // tiles that an expert has beyond its rows' share
};
constexpr Cost COSTS[] = {
    {Form::T256, 256, 256, 1, 1.29f, 9.5f, 0.27f}, {Form::T128W, 128, 256, 1, 0.89f, 4.2f, 0.54f},
    {Form::T128, 128, 128, 2, 1.03f, 3.4f, 0.54f}, {Form::T64, 64, 128, 2, 0.59f, 3.4f, 0.54f},
    {Form::T32W, 32, 256, 2, 1.22f, 1.7f, 0.54f},  {Form::T32, 32, 128, 2, 0.49f, 2.2f, 0.54f},
};

// f32: of the weights' gradient, whose tiles cost more in fp32, the more the smaller they are (256
// experts of 128 rows, 2048 x 1024: 256 x 256 529 us, 128 x 256 572, 128 x 128 676; in bf16, 64 rows, 1024 x 1024: 139,
// 156 and 140).
Plan plan_of(Kind kind, bool gated, int64_t rows, int E, int n, int k, bool f32 = false)
{
    const bool weight = kind == Kind::WEIGHT;
    if (weight && rows <= (int64_t)FEW_MEAN * E && k >= FEW_COLS / 2 && (int64_t)E * n * k >= FEW_LEAST) {
        Plan few{};
        few.form = Form::FEW;
        few.m_tiles = (n + FEW_N - 1) / FEW_N;
        few.n_tiles = (k + FEW_COLS - 1) / FEW_COLS;
        few.groups = (int64_t)E * few.m_tiles * few.n_tiles;
        few.splits = 1;
        return few;
    }
    const int width = kind == Kind::FORWARD ? n : k;
    const float used = (float)std::max<int64_t>(std::min<int64_t>(rows, E), 1);
    const int64_t total = kind == Kind::FORWARD ? k : kind == Kind::INPUT ? n : rows / E;
    const int steps = (int)std::max<int64_t>((total + STEP - 1) / STEP, 1);
    const float outputs = weight ? (float)E * n * k : (float)rows * width;
    const float bytes = 2.0f * ((weight ? (f32 ? 2.0f : 1.0f) * E : used) * n * k + (float)rows * n + (float)rows * k);
    float best = 0.0f;
    const Cost* form = nullptr;
    int best_splits = 1;
    for (const Cost& c : COSTS) {
        const float across = (float)((width + c.bn - 1) / c.bn);
        float tiles;
        if (weight)
            tiles = (float)E * ((n + c.bm - 1) / c.bm) * ((k + c.bn - 1) / c.bn);
        else if (E == 1)
            tiles = (float)((rows + c.bm - 1) / c.bm) * across;
        else                                             // an expert's last tile is half full, or a half one
            tiles = std::max(used, (float)rows / c.bm + c.last * used) * across;
        for (int splits = 1; splits <= 8 && (splits == 1 || steps >= 2 * splits); splits *= 2) {
            const float load = tiles * splits / (256.0f * c.per_cu);
            const bool counted = (weight || E == 1) && load <= 4.0f;
            const float rounds =
                std::max(1.0f, counted ? std::ceil(load) : load <= 3.0f ? std::ceil(1.05f * load) : load + 0.5f);
            const float step = (load <= 0.5f ? 0.66f : 1.0f) * (weight ? 0.82f : 1.0f) * c.step;
            float tile = (weight ? 1.17f : 1.0f) * c.tile;
            if (f32 && splits == 1)
                tile += (c.bm == 256 ? 1.0e-4f : 1.5e-4f) * c.per_cu * c.bm * c.bn;
            float us = rounds * ((steps + splits - 1) / splits * step + tile);
            if (splits > 1)
                us += 4.5f + splits * outputs * 1.2e-6f;                     // 8 bytes at 6.75 TB/s
            us = std::max(us, bytes / 5.6e6f) + 0.03f * us;
            if (!form || us < best) {
                best = us;
                form = &c;
                best_splits = splits;
            }
        }
    }
    Plan s{};
    set_tiles(s, form->form, kind, gated, rows, E, n, k);
    s.splits = best_splits;
    return s;
}

// Fp32 partial sums of a call whose sums are split.
size_t parts(const Plan& s, int64_t outputs) { return s.splits > 1 ? (size_t)s.splits * outputs * 4 : 0; }

template <Kind KIND, bool GATED, class C>
hipError_t launch_rows(const Linear& p, const Plan& s, hipStream_t stream)
{
    static std::atomic<uint64_t> allowed{0};
    const hipError_t e = allow_lds(linear_kernel<KIND, C, GATED>, allowed);
    if (e != hipSuccess)
        return e;
    dim3 grid = grid_of(s.groups);
    grid.z = s.splits;
    linear_kernel<KIND, C, GATED><<<grid, dim3(C::THREADS), C::LDS, stream>>>(p, s.n_tiles, s.splits);
    return hipGetLastError();
}

template <Kind KIND, bool GATED>
hipError_t launch_rows(const Linear& p, hipStream_t stream)
{
    const Plan s = plan_of(KIND, GATED, p.rows, p.E, p.n, p.k);
    const hipError_t e =
        with_tile(s.form, [&](auto c) { return launch_rows<KIND, GATED, decltype(c)>(p, s, stream); });
    if (e != hipSuccess || s.splits == 1)
        return e;
    const int width = KIND == Kind::FORWARD ? p.n : p.k;
    join_rows_kernel<KIND, GATED><<<blocks_of(p.rows * ((GATED ? width / 2 : width) / 8)), dim3(256), 0, stream>>>(
        p, s.splits);
    return hipGetLastError();
}

template <class C, bool BIAS>
hipError_t launch_weight(const Linear& p, const Plan& s, hipStream_t stream)
{
    static std::atomic<uint64_t> allowed{0};
    const hipError_t e = allow_lds(linear_weight_kernel<C, BIAS>, allowed);
    if (e != hipSuccess)
        return e;
    dim3 grid = grid_of(s.groups);
    grid.z = s.splits;
    linear_weight_kernel<C, BIAS><<<grid, dim3(C::THREADS), C::LDS, stream>>>(p, s.m_tiles, s.n_tiles, s.splits);
    return hipGetLastError();
}

}  // namespace

const char* linear_form(int kind, bool gated, int64_t rows, int E, int n, int k, int* splits)
{
    const Plan s = plan_of((Kind)std::min(kind, 2), gated, rows, E, n, k, kind == 3);
    *splits = s.splits;
    static const char* const names[] = {"256 x 256", "128 x 256", "128 x 128", "64 x 128", "32 x 256", "32 x 128", "few rows"};
    return names[(int)s.form];
}

size_t linear_workspace(int64_t rows, int E, int n, int k)
{
    const int64_t weights = (int64_t)E * n * (k + 1);
    size_t most = std::max(parts(plan_of(Kind::WEIGHT, false, rows, E, n, k), weights),
                           parts(plan_of(Kind::WEIGHT, false, rows, E, n, k, true), weights));
    most = std::max(most, parts(plan_of(Kind::INPUT, false, rows, E, n, k), rows * k));
    most = std::max(most, parts(plan_of(Kind::FORWARD, false, rows, E, n, k), rows * n));
    if (n % 16 == 0)
        most = std::max(most, parts(plan_of(Kind::FORWARD, true, rows, E, n, k), rows * n));
    return most;
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
    const Plan s = plan_of(Kind::WEIGHT, false, p.rows, p.E, p.n, p.k, p.out_f32);
    if (s.form == Form::FEW) {
        linear_weight_few_kernel<<<grid_of(s.groups), dim3(256), 0, stream>>>(p, s.m_tiles, s.n_tiles);
        return hipGetLastError();
    }
    const hipError_t e = with_tile(s.form, [&](auto c) {
        return p.dbias ? launch_weight<decltype(c), true>(p, s, stream) : launch_weight<decltype(c), false>(p, s, stream);
    });
    if (e != hipSuccess || s.splits == 1)
        return e;
    join_weight_kernel<<<blocks_of(((int64_t)p.E * p.n * p.k + 7) / 8), dim3(256), 0, stream>>>(p, s.splits);
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
