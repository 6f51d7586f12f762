// A whole expert layer for a few tokens.
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
// matrix instruction's registers, 16 rows by 128 bytes per instruction, the
// tokens of an expert are its columns, 16 at a time.
//
// Few tokens per expert: two kernels; every wave codes its columns on the way
// in, which costs the vector unit less than the wait for the weights and saves
// two launches.  More: x and h are coded once, by launches of their own, the
// first of which also works out who needs which expert, and the products read
// the codes.  Where the output is too narrow to occupy the chip, the experts of
// the down product are split over workgroups, whose fp32 parts one more launch
// adds in order.
//
// Who needs an expert is worked out from topk_idx alone: lane t of a wave looks
// through token t's K ids (at most 64 tokens).  A token that names an expert
// twice is one column with the sum of its weights.
#include <algorithm>

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

// Coded blocks in a wave's own LDS, AHEAD blocks of FEW columns, at a stride
// that spreads the reads over the banks.
constexpr int AHEAD = 2;
constexpr int FEW = 4;                    // columns that a product kernel codes at a time
constexpr int DIRECT_TOKENS = 16;         // most tokens that the product kernels code themselves
constexpr int CODE_STRIDE = SCALE_BLOCK + 16;
struct Coded {
    uint8_t codes[AHEAD * FEW * CODE_STRIDE];
    float scale[AHEAD * FEW];
};

// Codes a block that 16 lanes share, eight elements each.
__device__ inline v2u encode8(const float (&f)[8], float& scale)
{
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = fmaxf(top, fabsf(f[i]));
    top = max16(top);
    float inv;
    block_scale(top, inv, scale);
    return v2u{e4m3_pack4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
               e4m3_pack4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)};
}

// The same to rows row .. row+3 of `to`.
__device__ inline void encode8(Coded* to, int row, const float (&f)[8])
{
    const int l = threadIdx.x & 15;
    float scale;
    const v2u q = encode8(f, scale);
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

// Operand layout.  A load instruction should take whole 128-byte lines, eight
// lanes each, but the matrix instruction gives a row only four lanes.  So a
// weight load brings 8 rows of 128 codes, the lanes l and l ^ 1 (l & 15 = 2a,
// 2a + 1) holding the pieces 2g and 2g + 1 of row a (16 codes each, g = l >> 4),
// and the instruction sees 16 rows: row a's even pieces and its odd ones.  It
// runs once with the columns' even pieces and once with the odd; of the first
// the even rows count, of the second the odd, and a lane that holds rows 4g ..
// 4g+3 of the results holds both halves of two weight rows.  Half the products
// are for nothing, but the matrix unit has time: the kernels wait for memory.

// 16 weight codes of a lane, and 32 codes of a column (pieces 2g and 2g + 1), as
// fp16.
struct Half16 {
    v8h v[2];
};
struct Half32 {
    Half16 even, odd;
};
struct Rows16 {                           // two loads of 8 weight rows
    Half16 a[2];
};
__device__ inline Half16 convert16(v4u raw)
{
    return Half16{{e4m3_to_f16(raw.x, raw.y), e4m3_to_f16(raw.z, raw.w)}};
}

__device__ inline Rows16 convert_rows(const v4u (&raw)[2]) { return Rows16{{convert16(raw[0]), convert16(raw[1])}}; }

__device__ inline Half32 coded_columns(const Coded* from, int r, int g)
{
    const v4u* at = (const v4u*)(from->codes + r * CODE_STRIDE + g * 32);
    return Half32{convert16(at[0]), convert16(at[1])};
}

__device__ inline v4f product(const Half16& a, const Half16& b)
{
    const v4f zero{0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(
        a.v[1], b.v[1], __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[0], b.v[0], zero, 0, 0, 0), 0, 0, 0);
}

// The block's products of 16 weight rows (two loads of 8) and 16 columns, in
// fp32 from zero: of column l & 15, the rows out_row(g, 0 .. 3).
__device__ inline v4f product(const Rows16& rows, const Half32& b)
{
    v4f t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const v4f even = product(rows.a[i], b.even), odd = product(rows.a[i], b.odd);
        t[2 * i] = even[0] + odd[1];
        t[2 * i + 1] = even[2] + odd[3];
    }
    return t;
}
__device__ inline int out_row(int g, int i) { return (i >> 1) * 8 + 2 * g + (i & 1); }

// Where in its 8 rows of `stride` bytes a lane's weight piece lies.
__device__ inline uint32_t piece_of(int stride)
{
    const int l = threadIdx.x & (WAVE - 1);
    return ((l & 15) >> 1) * stride + ((l >> 4) * 2 + (l & 1)) * 16;
}

__device__ inline v4u load16(const uint8_t* p) { return *(const v4u*)p; }

// A workgroup's waves share the blocks of a product.  Blocks go AHEAD at a
// time: the weights of the next ones are in flight while a wave works on the
// last.  Occupancy matters more than depth: four blocks ahead (two waves per
// SIMD instead of four) took 82 us for one token of a hidden-7168, 256-expert
// layer, two ahead 71.  Whole lines per load against 64-byte halves (a row's
// pieces g, then g + 4): that layer 68 us against 73, 32 tokens of it 1187
// against 1255, 64 tokens of 8 experts, hidden 4096 68 against 79.  Plain loads:
// the nontemporal hint gains up to 3% on those that come from HBM (32 tokens
// 1174) and costs up to 20% where the weights stay in the memory-side cache or
// are read again for more columns (64 tokens of 8 experts 82).
constexpr int GATE_WAVES = 4;
constexpr int DOWN_WAVES = 8;

// Weight rows of 16 columns f of an expert's gate and up products.
struct GateUpRows {
    const uint8_t *gate, *up;
    const float *sg, *su;
    int64_t next8;
    uint32_t piece;
    int KB;
    __device__ inline GateUpRows(const FewTokens& p, int e, int f0)
    {
        KB = p.H / SCALE_BLOCK;
        next8 = (int64_t)8 * p.H;
        piece = piece_of(p.H);
        gate = p.w13 + ((int64_t)e * 2 * p.F + f0) * p.H;
        up = gate + (int64_t)p.F * p.H;
        sg = p.s13 + ((int64_t)e * (2 * p.F / SCALE_BLOCK) + f0 / SCALE_BLOCK) * KB;
        su = sg + (int64_t)(p.F / SCALE_BLOCK) * KB;
    }
    __device__ inline void fetch(int kb, v4u (&to)[2][2]) const
    {
        const int64_t o = (int64_t)min(kb, KB - 1) * SCALE_BLOCK;
        to[0][0] = load16(gate + o + piece);
        to[0][1] = load16(gate + o + next8 + piece);
        to[1][0] = load16(up + o + piece);
        to[1][1] = load16(up + o + next8 + piece);
    }
};

struct DownRows {
    const uint8_t* down;
    const float* sd;
    int64_t next8;
    uint32_t piece;
    int FB;
    __device__ inline DownRows(const FewTokens& p, int e, int n0)
    {
        FB = p.F / SCALE_BLOCK;
        next8 = (int64_t)8 * p.F;
        piece = piece_of(p.F);
        down = p.w2 + ((int64_t)e * p.H + n0) * p.F;
        sd = p.s2 + ((int64_t)e * (p.H / SCALE_BLOCK) + n0 / SCALE_BLOCK) * FB;
    }
    __device__ inline void fetch(int kb, v4u (&to)[2]) const
    {
        const int64_t o = (int64_t)min(kb, FB - 1) * SCALE_BLOCK;
        to[0] = load16(down + o + piece);
        to[1] = load16(down + o + next8 + piece);
    }
};

// acc + t * s, or acc alone for a block that is read only to keep the loop
// whole (whatever its numbers are).
__device__ inline void add_block(v4f& acc, const v4f& t, float s, bool live)
{
    s = live ? s : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        acc[i] = fmaf(live ? t[i] : 0.0f, s, acc[i]);
}

// Lane t: the router weight of token t for expert e.
__device__ inline float weight_of(const FewTokens& p, const int32_t* ids, int e)
{
    const int t = threadIdx.x & (WAVE - 1);
    float w = 0.0f;
    for (int k = 0; k < p.K; ++k)
        if (ids[t * p.K + k] == e)
            w += p.w[t * p.K + k];
    return w;
}

// h[t*K+k][f] of up to DIRECT_TOKENS tokens, FEW at a time: one workgroup per (distinct expert, 16
// columns f); its waves share the blocks of H and add up through LDS.
__global__ __launch_bounds__(GATE_WAVES* WAVE, 4) void few_gate_up_kernel(const FewTokens p, float* hbuf)
{
    extern __shared__ int32_t ids[];
    __shared__ uint32_t used[MAX_E_WORDS];
    __shared__ int32_t cols[DIRECT_TOKENS];
    __shared__ Coded coded[GATE_WAVES];
    __shared__ float part[GATE_WAVES][2][FEW][17];
    read_ids(p, ids, used);
    const int e = nth_expert(used, blockIdx.y);
    if (e < 0)
        return;
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int r = lane & 15, g = lane >> 4;
    const int f0 = blockIdx.x * 16;
    const GateUpRows rows(p, e, f0);
    const int KB = rows.KB;
    const int k0 = KB * wave / GATE_WAVES, k1 = KB * (wave + 1) / GATE_WAVES;
    v4u w[AHEAD][2][2];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
        rows.fetch(k0 + u, w[u]);
    const Member me = member(p, ids, e);
    if (wave == 0)
        list_columns(p, me, cols);
    const int n = __popcll(__ballot(me.is));
    __syncthreads();
    for (int c0 = 0; c0 < n; c0 += FEW) {
        // the tokens' rows come ahead like the weights; AHEAD blocks are coded at a time
        const uint16_t* xp = p.x + (int64_t)(cols[min(c0 + g, n - 1)] / p.K) * p.H + r * 8;
        v4u x[AHEAD];
        auto xrows = [&](int kb0) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                x[u] = *(const v4u*)(xp + min(kb0 + u, KB - 1) * SCALE_BLOCK);
        };
        v4f ag{0.0f, 0.0f, 0.0f, 0.0f}, au = ag;
        xrows(k0);
        if (c0 > 0)
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                rows.fetch(k0 + u, w[u]);
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
                const int kb = min(kb0 + u, KB - 1), row = u * FEW + (r & (FEW - 1));
                const bool live = kb0 + u < k1;
                const Rows16 wg = convert_rows(w[u][0]), wu = convert_rows(w[u][1]);
                rows.fetch(kb0 + u + AHEAD, w[u]);
                const Half32 q = coded_columns(&coded[wave], row, g);
                const float xs = coded[wave].scale[row];
                add_block(ag, product(wg, q), xs * rows.sg[kb], live);
                add_block(au, product(wu, q), xs * rows.su[kb], live);
            }
            own_lds_written();
        }
        // lane (r, g) has rows out_row(g, 0 .. 3) of column r
        if (r < FEW)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                part[wave][0][r][out_row(g, i)] = ag[i];
                part[wave][1][r][out_row(g, i)] = au[i];
            }
        __syncthreads();
        for (int v = threadIdx.x; v < min(n - c0, FEW) * 16; v += GATE_WAVES * WAVE) {
            const int col = v >> 4, f = v & 15;
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int q = 0; q < GATE_WAVES; ++q) {
                a += part[q][0][col][f];
                b += part[q][1][col][f];
            }
            hbuf[(int64_t)cols[c0 + col] * p.F + f0 + f] = silu4(a) * (0.25f * b);
        }
        __syncthreads();
    }
}

// The tile [T][16] of the output that a workgroup's waves have summed in copies
// of their own, added in order: the result, or with several shares this one's
// part of it, [share][T][H] in fp32.
template <bool SPLIT, int TOKENS>
__device__ inline void join_tile(const FewTokens& p, const float (&tile)[DOWN_WAVES][TOKENS][17], int n0, float* parts)
{
    __syncthreads();
    for (int v = threadIdx.x; v < p.T * 8; v += DOWN_WAVES * WAVE) {
        const int t = v >> 3, n = (v & 7) * 2;
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int q = 0; q < DOWN_WAVES; ++q) {
            a += tile[q][t][n];
            b += tile[q][t][n + 1];
        }
        const int64_t o = (int64_t)t * p.H + n0 + n;
        if (SPLIT)
            *(float2*)(parts + (int64_t)blockIdx.y * p.T * p.H + o) = float2{a, b};
        else
            *(uint32_t*)(p.out + o) = bf16_pack(a, b);
    }
}

// The (expert, block of F) pairs of this wave, in order, of those that the
// shares' waves divide among them.
template <bool SPLIT>
__device__ inline int share_start(int pairs, int wave)
{
    const int at = SPLIT ? blockIdx.y * DOWN_WAVES + wave : wave;
    return (int)((int64_t)pairs * at / (SPLIT ? (int)gridDim.y * DOWN_WAVES : DOWN_WAVES));
}

// out[t][n0 .. n0+15] of up to DIRECT_TOKENS tokens: the waves of the workgroups
// (n0, share) divide the (expert, block of F) pairs in order; a wave adds an expert's finished part, times the router
// weight, to its own copy of the tile.
template <bool SPLIT>
__global__ __launch_bounds__(DOWN_WAVES* WAVE, 4) void few_down_kernel(const FewTokens p, const float* hbuf,
                                                                       float* parts)
{
    extern __shared__ int32_t ids[];
    __shared__ uint32_t used[MAX_E_WORDS];
    __shared__ int32_t cols[DOWN_WAVES][DIRECT_TOKENS];
    __shared__ float weight[DOWN_WAVES][DIRECT_TOKENS];
    __shared__ Coded coded[DOWN_WAVES];
    __shared__ float tile[DOWN_WAVES][DIRECT_TOKENS][17];
    for (int i = threadIdx.x; i < DOWN_WAVES * DIRECT_TOKENS * 17; i += DOWN_WAVES * WAVE)
        (&tile[0][0][0])[i] = 0.0f;
    read_ids(p, ids, used);
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int r = lane & 15, g = lane >> 4;
    const int FB = p.F / SCALE_BLOCK;
    const int n0 = blockIdx.x * 16;
    const int pairs = count_experts(used) * FB;
    const int q0 = share_start<SPLIT>(pairs, wave), q1 = share_start<SPLIT>(pairs, wave + 1);
    for (int q = q0; q < q1;) {
        const int u0 = q / FB;
        const int kb0 = q - u0 * FB, kb1 = min(FB, kb0 + q1 - q);
        const int e = nth_expert(used, u0);
        const DownRows rows(p, e, n0);
        v4u w[AHEAD][2];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            rows.fetch(kb0 + u, w[u]);
        const Member me = member(p, ids, e);
        const int n = list_columns(p, me, cols[wave]);
        if (me.is)
            weight[wave][lane] = weight_of(p, ids, e);
        own_lds_written();
        for (int c0 = 0; c0 < n; c0 += FEW) {
            const float* hp = hbuf + (int64_t)cols[wave][min(c0 + g, n - 1)] * p.F + r * 8;
            v4f hv[AHEAD][2];
            auto hrows = [&](int k) {
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const v4f* h = (const v4f*)(hp + min(k + u, FB - 1) * SCALE_BLOCK);
                    hv[u][0] = h[0];
                    hv[u][1] = h[1];
                }
            };
            v4f acc{0.0f, 0.0f, 0.0f, 0.0f};
            hrows(kb0);
            if (c0 > 0)
#pragma unroll
                for (int u = 0; u < AHEAD; ++u)
                    rows.fetch(kb0 + u, w[u]);
            for (int k = kb0; k < kb1; k += AHEAD) {
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const float f[8] = {hv[u][0].x, hv[u][0].y, hv[u][0].z, hv[u][0].w,
                                        hv[u][1].x, hv[u][1].y, hv[u][1].z, hv[u][1].w};
                    encode8(&coded[wave], u * FEW, f);
                }
                hrows(k + AHEAD);
                own_lds_written();
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const int row = u * FEW + (r & (FEW - 1));
                    const float s = coded[wave].scale[row] * rows.sd[min(k + u, FB - 1)];
                    const Rows16 wd = convert_rows(w[u]);
                    rows.fetch(k + u + AHEAD, w[u]);
                    add_block(acc, product(wd, coded_columns(&coded[wave], row, g)), s, k + u < kb1);
                }
                own_lds_written();
            }
            if (r < FEW && c0 + r < n) {
                const int t = cols[wave][c0 + r] / p.K;
                const float wt = weight[wave][t];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tile[wave][t][out_row(g, i)] += wt * acc[i];
            }
        }
        own_lds_written();
        q += kb1 - kb0;
    }
    join_tile<SPLIT>(p, tile, n0, parts);
}

// ---- more tokens: codes made once ----

__device__ inline void read8(const uint16_t* from, float (&f)[8]) { unpack8(*(const v4u*)from, f); }
__device__ inline void read8(const float* from, float (&f)[8])
{
    const v4f a = *(const v4f*)from, b = *(const v4f*)(from + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = a[i];
        f[4 + i] = b[i];
    }
}

constexpr int CODE_THREADS = 256;
template <class V>
__device__ inline void code_blocks(const V* from, int64_t block, int64_t blocks, uint8_t* codes, float* scales)
{
    const int64_t b = block * (CODE_THREADS / 16) + threadIdx.x / 16;
    if (b >= blocks)
        return;
    const int64_t at = b * SCALE_BLOCK + (threadIdx.x & 15) * 8;
    float f[8], scale;
    read8(from + at, f);
    *(v2u*)(codes + at) = encode8(f, scale);
    if ((threadIdx.x & 15) == 0)
        scales[b] = scale;
}

// Who needs which expert, worked out once: the distinct experts' number, and of
// the u-th its id, its columns' number, their items t*K+k and router weights
// (MOE_TOKENS places each).  Where every workgroup worked it out, 39 tokens, 130
// experts, top 5, hidden 384, f 2432 took 140 us against 131.
struct Plan {
    int32_t *count, *expert, *columns, *items;
    float* weights;
};

// Codes x, and in the workgroups past those plans an expert per wave.
__global__ __launch_bounds__(CODE_THREADS) void code_and_plan_kernel(const FewTokens p, int64_t blocks, int coders,
                                                                     uint8_t* codes, float* scales, const Plan plan)
{
    extern __shared__ int32_t ids[];
    __shared__ uint32_t used[MAX_E_WORDS];
    if ((int)blockIdx.x < coders) {
        code_blocks(p.x, blockIdx.x, blocks, codes, scales);
        return;
    }
    read_ids(p, ids, used);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int u = (blockIdx.x - coders) * (CODE_THREADS / WAVE) + wave;
    if (u == 0)
        *plan.count = count_experts(used);
    const int e = nth_expert(used, u);
    if (e < 0)
        return;
    const Member me = member(p, ids, e);
    const int t = threadIdx.x & (WAVE - 1);
    const uint64_t mask = __ballot(me.is);
    if (me.is) {
        const int at = u * MOE_TOKENS + __popcll(mask & ((1ull << t) - 1));
        plan.items[at] = t * p.K + me.k;
        plan.weights[at] = weight_of(p, ids, e);
    }
    if (t == 0) {
        plan.expert[u] = e;
        plan.columns[u] = __popcll(mask);
    }
}

__global__ __launch_bounds__(CODE_THREADS) void code_kernel(const float* from, int64_t blocks, uint8_t* codes,
                                                            float* scales)
{
    code_blocks(from, blockIdx.x, blocks, codes, scales);
}

// Blocks of 16 coded rows as the product's columns, AHEAD at a time.
struct CodedRows {
    const uint8_t* codes;
    const float* scales;
    int blocks;
    v4u q[AHEAD][2];
    float s[AHEAD];
    __device__ inline CodedRows(const uint8_t* code_rows, const float* scale_rows, int64_t row, int blocks_)
        : codes(code_rows + row * blocks_ * SCALE_BLOCK + ((threadIdx.x & (WAVE - 1)) >> 4) * 32),
          scales(scale_rows + row * blocks_), blocks(blocks_)
    {
    }
    __device__ inline void fetch(int u, int kb)
    {
        kb = min(kb, blocks - 1);
        q[u][0] = load16(codes + kb * SCALE_BLOCK);
        q[u][1] = load16(codes + kb * SCALE_BLOCK + 16);
        s[u] = scales[kb];
    }
    __device__ inline Half32 columns(int u) const { return Half32{convert16(q[u][0]), convert16(q[u][1])}; }
};

// h as above, 16 columns at a time (an expert with more reads its weights
// again, from the caches: 32 at a time took 1475 us against 1258 for 32 tokens
// of the 256-expert layer, and 77 against 83 for 64 tokens of one with 8
// experts).  Three waves per SIMD: four leave too few registers (1367 against
// 1187 for the 32 tokens).
__global__ __launch_bounds__(GATE_WAVES* WAVE, 3) void coded_gate_up_kernel(const FewTokens p, const Plan plan,
                                                                             const uint8_t* xq, const float* xs,
                                                                             float* hbuf)
{
    __shared__ float part[GATE_WAVES][2][16][17];
    if ((int)blockIdx.y >= *plan.count)
        return;
    const int e = plan.expert[blockIdx.y], n = plan.columns[blockIdx.y];
    const int32_t* cols = plan.items + blockIdx.y * MOE_TOKENS;
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int r = lane & 15, g = lane >> 4;
    const int f0 = blockIdx.x * 16;
    const GateUpRows rows(p, e, f0);
    const int KB = rows.KB;
    const int k0 = KB * wave / GATE_WAVES, k1 = KB * (wave + 1) / GATE_WAVES;
    v4u w[AHEAD][2][2];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
        rows.fetch(k0 + u, w[u]);
    for (int c0 = 0; c0 < n; c0 += 16) {
        CodedRows x(xq, xs, cols[min(c0 + r, n - 1)] / p.K, KB);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            x.fetch(u, k0 + u);
            if (c0 > 0)
                rows.fetch(k0 + u, w[u]);
        }
        v4f ag{0.0f, 0.0f, 0.0f, 0.0f}, au = ag;
        for (int kb0 = k0; kb0 < k1; kb0 += AHEAD)
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int kb = min(kb0 + u, KB - 1);
                const bool live = kb0 + u < k1;
                const Rows16 wg = convert_rows(w[u][0]), wu = convert_rows(w[u][1]);
                rows.fetch(kb0 + u + AHEAD, w[u]);
                const Half32 q = x.columns(u);
                add_block(ag, product(wg, q), x.s[u] * rows.sg[kb], live);
                add_block(au, product(wu, q), x.s[u] * rows.su[kb], live);
                x.fetch(u, kb0 + u + AHEAD);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            part[wave][0][r][out_row(g, i)] = ag[i];
            part[wave][1][r][out_row(g, i)] = au[i];
        }
        __syncthreads();
        for (int v = threadIdx.x; v < min(n - c0, 16) * 16; v += GATE_WAVES * WAVE) {
            const int col = v >> 4, f = v & 15;
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int q = 0; q < GATE_WAVES; ++q) {
                a += part[q][0][col][f];
                b += part[q][1][col][f];
            }
            hbuf[(int64_t)cols[c0 + col] * p.F + f0 + f] = silu4(a) * (0.25f * b);
        }
        __syncthreads();
    }
}

// The down product as above.
template <bool SPLIT>
__global__ __launch_bounds__(DOWN_WAVES* WAVE, 4) void coded_down_kernel(const FewTokens p, const Plan plan,
                                                                          const uint8_t* hq, const float* hs,
                                                                          float* parts)
{
    __shared__ float tile[DOWN_WAVES][MOE_TOKENS][17];
    for (int i = threadIdx.x; i < DOWN_WAVES * MOE_TOKENS * 17; i += DOWN_WAVES * WAVE)
        (&tile[0][0][0])[i] = 0.0f;
    __syncthreads();
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int r = lane & 15, g = lane >> 4;
    const int FB = p.F / SCALE_BLOCK;
    const int n0 = blockIdx.x * 16;
    const int pairs = *plan.count * FB;
    const int q0 = share_start<SPLIT>(pairs, wave), q1 = share_start<SPLIT>(pairs, wave + 1);
    for (int q = q0; q < q1;) {
        const int u0 = q / FB;
        const int kb0 = q - u0 * FB, kb1 = min(FB, kb0 + q1 - q);
        const int e = plan.expert[u0], n = plan.columns[u0];
        const int32_t* cols = plan.items + u0 * MOE_TOKENS;
        const float* weight = plan.weights + u0 * MOE_TOKENS;
        const DownRows rows(p, e, n0);
        v4u w[AHEAD][2];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            rows.fetch(kb0 + u, w[u]);
        for (int c0 = 0; c0 < n; c0 += 16) {
            CodedRows h(hq, hs, cols[min(c0 + r, n - 1)], FB);
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                h.fetch(u, kb0 + u);
                if (c0 > 0)
                    rows.fetch(kb0 + u, w[u]);
            }
            v4f acc{0.0f, 0.0f, 0.0f, 0.0f};
            for (int k = kb0; k < kb1; k += AHEAD)
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const float sd = rows.sd[min(k + u, FB - 1)];
                    const Rows16 wd = convert_rows(w[u]);
                    rows.fetch(k + u + AHEAD, w[u]);
                    add_block(acc, product(wd, h.columns(u)), h.s[u] * sd, k + u < kb1);
                    h.fetch(u, k + u + AHEAD);
                }
            if (c0 + r < n) {
                const int t = cols[c0 + r] / p.K;
                const float wt = weight[c0 + r];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tile[wave][t][out_row(g, i)] += wt * acc[i];
            }
        }
        own_lds_written();
        q += kb1 - kb0;
    }
    join_tile<SPLIT>(p, tile, n0, parts);
}

__global__ __launch_bounds__(CODE_THREADS) void add_parts_kernel(const float* parts, int shares, int64_t elements,
                                                                 uint16_t* out)
{
    const int64_t at = ((int64_t)blockIdx.x * CODE_THREADS + threadIdx.x) * 4;
    if (at >= elements)
        return;
    v4f sum{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < shares; ++s) {
        const v4f v = *(const v4f*)(parts + s * elements + at);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sum[i] += v[i];
    }
    *(v2u*)(out + at) = v2u{bf16_pack(sum[0], sum[1]), bf16_pack(sum[2], sum[3])};
}

// Whether the product kernels code their columns themselves.  That saves two
// launches, some 4 us, and costs by the columns: an expert with more than FEW
// reads its weights again, and each pass keeps more of the vector unit.  So up
// to FEW tokens; and up to DIRECT_TOKENS where experts have 2.5 columns at most
// on average and either few weights are read (256 MB) or columns are few (1/3).
// Measured (us, direct against coded):
//  - 5 tokens, 160 experts, top 3, hidden 768, f 384 18.1 against 22.3; 16
//    tokens, top 1 of 200, hidden 1024, f 512 16.4 against 21.3; 13 tokens, top
//    2 of 117, hidden 6400, f 256 33.6 against 38.5;
//  - hidden 4096, f 2048 from here on, 8 experts, top 2: 8 tokens 40 against 46,
//    10 (2.5 columns) 40 against 45, 12 46.5 against 45.5, 16 58 against 48.5; 8
//    tokens, top 4 59 against 49; 16 experts, top 4: 12 tokens 100 against 93;
//  - 64 experts, top 4: 6 tokens (0.4 columns) 114 against 114, 8 139 against 135,
//    12 177 against 170, 16 188 against 180; 16 experts, top 4 (400 MB): 8 tokens
//    86 against 81;
//  - hidden 7168, 256 experts, top 8: 8 tokens (0.25) 445 against 450, 16 (0.5)
//    816 against 817;
//  - beyond 16 tokens: 29 tokens, 5 experts, top 5, hidden 1024, f 1536 62 against
//    38, 32 tokens, 8 experts, top 2, hidden 4096 99 against 51, 64 tokens of the
//    256-expert layer 1751 against 1675.
inline bool direct(const FewTokens& p)
{
    const int columns = p.T * p.K;
    const int64_t bytes = (int64_t)std::min(columns, p.E) * 3 * p.F * p.H;
    return p.T <= FEW ||
           (p.T <= DIRECT_TOKENS && 2 * columns <= 5 * p.E && (bytes <= (int64_t)256 << 20 || 3 * columns <= p.E));
}

// Shares of the down product: 512 workgroups, two per CU, as long as each wave
// has some eight blocks to its share; none where that is two shares or less.  61 tokens, 177 experts, hidden 384 (24
// workgroups without): 152 -> 74 us; 10 tokens, top 6 of 187, hidden 384, f 2432
// 151 -> 87.  Hidden 4096 gains nothing from a second share (8 tokens, 8 experts
// 42 against 46, 32 tokens 55 against 59); hidden 2048 (26 tokens, 79 experts)
// takes 241 with two, 249 with three, 233 with four.
inline int down_shares(int T, int K, int H, int F)
{
    const int wide = H / 16;
    const int blocks = (int)std::min<int64_t>((int64_t)T * K * (F / SCALE_BLOCK) / (8 * DOWN_WAVES), 16);
    return wide > 200 ? 1 : std::max(1, std::min(512 / wide, blocks));
}

// The workspace: h in fp32, and where x and h may be coded once their codes,
// scales and the parts.
struct Workspace {
    size_t h = 0, xq = 0, hq = 0, parts = 0, xs = 0, hs = 0, count = 0, expert = 0, columns = 0, items = 0,
           weights = 0, bytes = 0;
    Workspace(int T, int K, int H, int F)
    {
        const size_t x = (size_t)T * H, products = (size_t)T * K * F;
        const int shares = down_shares(T, K, H, F);
        auto take = [&](size_t n) {
            const size_t at = bytes;
            bytes += (n + 15) / 16 * 16;
            return at;
        };
        h = take(products * 4);
        parts = take(shares > 1 ? shares * x * 4 : 0);
        if (T <= FEW)
            return;
        xq = take(x);
        hq = take(products);
        xs = take(x / SCALE_BLOCK * 4);
        hs = take(products / SCALE_BLOCK * 4);
        const size_t experts = std::min(T * K, MAX_E_WORDS * 32);
        count = take(4);
        expert = take(experts * 4);
        columns = take(experts * 4);
        items = take(experts * MOE_TOKENS * 4);
        weights = take(experts * MOE_TOKENS * 4);
    }
};

inline dim3 grid_of(int64_t n, int per) { return dim3((uint32_t)((n + per - 1) / per)); }

// The workspace's places, and how the layer is divided among launches.
struct Launches {
    const FewTokens& p;
    hipStream_t stream;
    Workspace at;
    uint8_t* ws;
    float *h, *parts;
    int experts, shares;
    uint32_t ids;
    Launches(const FewTokens& p_, hipStream_t stream_)
        : p(p_), stream(stream_), at(p.T, p.K, p.H, p.F), ws((uint8_t*)p.workspace), h((float*)(ws + at.h)),
          parts((float*)(ws + at.parts)), experts(std::min(p.T * p.K, p.E)),       // distinct ones, at most
          shares(down_shares(p.T, p.K, p.H, p.F)), ids((uint32_t)(p.T * p.K) * 4)
    {
    }
    hipError_t direct() const
    {
        few_gate_up_kernel<<<dim3(p.F / 16, experts), dim3(GATE_WAVES * WAVE), ids, stream>>>(p, h);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        const dim3 grid(p.H / 16, shares), block(DOWN_WAVES * WAVE);
        if (shares > 1)
            few_down_kernel<true><<<grid, block, ids, stream>>>(p, h, parts);
        else
            few_down_kernel<false><<<grid, block, ids, stream>>>(p, h, parts);
        return hipGetLastError();
    }
    hipError_t coded() const
    {
        uint8_t *xq = ws + at.xq, *hq = ws + at.hq;
        float *xs = (float*)(ws + at.xs), *hs = (float*)(ws + at.hs);
        const Plan plan{(int32_t*)(ws + at.count), (int32_t*)(ws + at.expert), (int32_t*)(ws + at.columns),
                        (int32_t*)(ws + at.items), (float*)(ws + at.weights)};
        const int64_t xb = (int64_t)p.T * p.H / SCALE_BLOCK, hb = (int64_t)p.T * p.K * p.F / SCALE_BLOCK;
        const int coders = (int)grid_of(xb, CODE_THREADS / 16).x;
        const int planners = (int)grid_of(experts, CODE_THREADS / WAVE).x;
        code_and_plan_kernel<<<dim3(coders + planners), dim3(CODE_THREADS), ids, stream>>>(p, xb, coders, xq, xs, plan);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        coded_gate_up_kernel<<<dim3(p.F / 16, experts), dim3(GATE_WAVES * WAVE), 0, stream>>>(p, plan, xq, xs, h);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        code_kernel<<<grid_of(hb, CODE_THREADS / 16), dim3(CODE_THREADS), 0, stream>>>(h, hb, hq, hs);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        const dim3 grid(p.H / 16, shares), block(DOWN_WAVES * WAVE);
        if (shares > 1)
            coded_down_kernel<true><<<grid, block, 0, stream>>>(p, plan, hq, hs, parts);
        else
            coded_down_kernel<false><<<grid, block, 0, stream>>>(p, plan, hq, hs, parts);
        return hipGetLastError();
    }
    hipError_t add_parts() const
    {
        if (shares == 1)
            return hipSuccess;
        const int64_t x = (int64_t)p.T * p.H;
        add_parts_kernel<<<grid_of(x, CODE_THREADS * 4), dim3(CODE_THREADS), 0, stream>>>(parts, shares, x, p.out);
        return hipGetLastError();
    }
};

}  // namespace

size_t few_token_workspace(int T, int K, int H, int F)
{
    return Workspace(T, K, H, F).bytes;
}

const char* few_token_form(const FewTokens& p)
{
    const bool split = down_shares(p.T, p.K, p.H, p.F) > 1;
    return direct(p) ? split ? "direct split" : "direct" : split ? "coded split" : "coded";
}

hipError_t launch_few_token_layer(const FewTokens& p, hipStream_t stream)
{
    if (p.T == 0)
        return hipSuccess;
    const Launches layer(p, stream);
    const hipError_t e = direct(p) ? layer.direct() : layer.coded();
    return e == hipSuccess ? layer.add_parts() : e;
}

}  // namespace ops
}  // namespace moe
