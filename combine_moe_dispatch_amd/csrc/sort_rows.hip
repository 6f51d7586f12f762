// Tokens sorted by expert and back: the plan (a stable counting sort of the
// (token, k) pairs by expert), the copy of the tokens' rows into that order,
// the weighted sum of the experts' rows back to the tokens, and its gradient.
#include <algorithm>

#include "moe_kernels.h"
#include "moe_ops.h"
#include "ops_common.h"

namespace moe {
namespace ops {
namespace {

// ---------------------------------------------------------------------------
// The plan.  Pair p = t*K + k of expert e gets row
//   slot[p] = (pairs of experts below e) + (pairs before p of expert e).
// A workgroup has a contiguous range of pairs, each of its waves a contiguous
// part of that, so the ranks need only counts in order: per wave in LDS, per
// workgroup in the workspace (a launch before this one, none where one
// workgroup has all pairs).  Inside 64 pairs the rank is the number of lower
// lanes with the same expert, found bit by bit of its id.  Latencies bound it:
// 131072 pairs, 256 experts take 4.8 us to count and 7.7 to place, 1 token's 8
// pairs 3.2 in one workgroup.
// ---------------------------------------------------------------------------
constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_ALONE = 8192;            // pairs up to which one workgroup has all
constexpr int PLAN_RANGE = 2048;            // pairs of a workgroup beyond, at least
constexpr int PLAN_GROUPS = 128;            // workgroups, at most

struct Plan {
    int64_t pairs;
    int E, groups, bits;
    int64_t range;            // pairs per workgroup, a multiple of its threads
    const int32_t* idx;
    int32_t* counts;          // [groups][E], null with one workgroup
    int32_t* offsets;
    int32_t* slot;
    int32_t* source;
};

__global__ __launch_bounds__(PLAN_THREADS) void count_pairs_kernel(const Plan p)
{
    __shared__ int count[MAX_EXPERTS];
    for (int e = threadIdx.x; e < p.E; e += PLAN_THREADS)
        count[e] = 0;
    __syncthreads();
    const int64_t end = min(p.range * (blockIdx.x + 1), p.pairs);
    for (int64_t i = p.range * blockIdx.x + threadIdx.x; i < end; i += PLAN_THREADS) {
        const int e = p.idx[i];
        if ((uint32_t)e < (uint32_t)p.E)
            atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += PLAN_THREADS)
        p.counts[(int64_t)blockIdx.x * p.E + e] = count[e];
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void sort_plan_kernel(const Plan p)
{
    constexpr int WAVES = THREADS / WAVE;
    extern __shared__ int hist[];                  // [WAVES][E], then all[E + 1], then below[E]
    int* const all = hist + WAVES * p.E;
    int* const below = all + p.E + 1;              // pairs of the workgroups before this one
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    int* const mine = hist + wave * p.E;
    for (int e = threadIdx.x; e < (WAVES + 2) * p.E + 1; e += THREADS)
        hist[e] = 0;
    __syncthreads();
    if (p.counts) {
        // all threads share the [groups][E] counts: so many rows of them at a time
        const int rows = max(THREADS / p.E, 1), e0 = threadIdx.x % p.E, g0 = threadIdx.x / p.E;
        for (int e = e0; e < p.E && g0 < rows; e += THREADS) {
            int before = 0, total = 0;
#pragma unroll 8
            for (int g = g0; g < p.groups; g += rows) {
                const int c = p.counts[g * p.E + e];
                before += g < (int)blockIdx.x ? c : 0;
                total += c;
            }
            atomicAdd(&below[e], before);
            atomicAdd(&all[e], total);
        }
    }
    const int64_t part = p.range / WAVES;          // a multiple of 64
    const int64_t begin = p.range * blockIdx.x + part * wave;
    const int64_t end = min(begin + part, p.pairs);
    for (int64_t i = begin + lane; i < end; i += WAVE) {
        const int e = p.idx[i];
        if ((uint32_t)e < (uint32_t)p.E)
            atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    // each wave's pairs start behind those of the waves and workgroups before it
    for (int e = threadIdx.x; e < p.E; e += THREADS) {
        int before = below[e];
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const int c = hist[w * p.E + e];
            hist[w * p.E + e] = before;
            before += c;
        }
        if (!p.counts)
            all[e] = before;
    }
    __syncthreads();
    if (wave == 0) {
        const int per = (p.E + WAVE - 1) / WAVE;
        const int e0 = min(lane * per, p.E), e1 = min(e0 + per, p.E);
        int sum = 0;
        for (int e = e0; e < e1; ++e)
            sum += all[e];
        const int upto = wave_scan(sum);
        int at = upto - sum;
        for (int e = e0; e < e1; ++e) {
            const int c = all[e];
            all[e] = at;
            at += c;
        }
        if (lane == WAVE - 1)
            all[p.E] = upto;
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= p.E; e += THREADS)
            p.offsets[e] = all[e];
    for (int64_t i0 = begin; i0 < end; i0 += WAVE) {
        const int64_t i = i0 + lane;
        const int e = i < end ? p.idx[i] : -1;
        const bool valid = (uint32_t)e < (uint32_t)p.E;
        uint64_t same = __ballot(valid);
        for (int b = 0; b < p.bits; ++b) {
            const bool one = e >> b & 1;
            const uint64_t m = __ballot(one);
            same &= one ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int row = 0;
        if (valid && rank == 0)
            row = all[e] + atomicAdd(&mine[e], __popcll(same));
        row = __shfl(row, valid ? __ffsll((unsigned long long)same) - 1 : lane, WAVE) + rank;
        if (i < end)
            p.slot[i] = valid ? row : -1;
        if (valid && p.source)
            p.source[row] = (int)i;
    }
}

// ---------------------------------------------------------------------------
// Rows.  A token's row is V vectors of 16 bytes; LANES lanes of a wave (all 64
// of them, in chunks, where V >= 64) hold one vector each.
// ---------------------------------------------------------------------------
struct Rows {
    int64_t tokens, rows;
    int K, vecs, chunks;      // chunks of LANES vectors per token
    int extra;                // 4-byte words per row of the scales
    const void* x;
    const float* xs;
    const int32_t* slot;
    const float* w;
    void* out;
    float* outs;
    const void* dout;
    void* dy;
    float* dw;
};

// Task of these lanes: a chunk of a token.
template <int LANES>
__device__ inline int64_t task_of()
{
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    int64_t t = block * (blockDim.x / LANES) + threadIdx.x / LANES;
    if (LANES == WAVE)
        t = (int64_t)__builtin_amdgcn_readfirstlane((int)(t >> 32)) << 32 |
            (uint32_t)__builtin_amdgcn_readfirstlane((int)t);
    return t;
}

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

// sorted[slot[t][k]] = x[t]: read once, written K times, bound by the memory behind the caches, and
// there by writes that jump from row to row: 16384 tokens of 7168 to 8 experts each 402 us, 5.3
// TB/s, 4096 of 4096 to 6 39 us, 6.0 (a copy 6.6).  No better: a hint on the reads too (409, 46 us),
// slots read eight at a time (422, 46), larger workgroups, neighbouring rows on one XCD.
template <int LANES, bool STREAM>
__global__ __launch_bounds__(256) void sort_rows_kernel(const Rows r)
{
    const int64_t task = task_of<LANES>();
    const int64_t t = task / r.chunks;
    if (t >= r.tokens)
        return;
    const int v = (int)(task - t * r.chunks) * LANES + threadIdx.x % LANES;
    const bool live = v < r.vecs;
    const v4u x = ((const v4u*)r.x)[t * r.vecs + (live ? v : 0)];
    const float s = v < r.extra ? r.xs[t * r.extra + v] : 0.0f;
    for (int k = 0; k < r.K; ++k) {
        const int64_t row = r.slot[t * r.K + k];
        if ((uint64_t)row >= (uint64_t)r.rows)
            continue;
        if (live)
            store_row<STREAM>(x, (v4u*)r.out + row * r.vecs + v);
        if (v < r.extra)
            r.outs[row * r.extra + v] = s;
    }
}

// The elements of a vector as fp32, and back, rounded once.
template <bool F32>
struct Vec {
    static constexpr int N = F32 ? 4 : 8;
    static __device__ inline void open(const v4u& u, float (&f)[N])
    {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if constexpr (F32) {
                f[c] = __uint_as_float(u[c]);
            } else {
                f[2 * c] = bf16_lo(u[c]);
                f[2 * c + 1] = bf16_hi(u[c]);
            }
    }
    static __device__ inline v4u close(const float (&f)[N])
    {
        v4u u;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if constexpr (F32)
                u[c] = __float_as_uint(f[c]);
            else
                u[c] = bf16_pack(f[2 * c], f[2 * c + 1]);
        return u;
    }
};

constexpr int AHEAD = 8;      // rows of a token in flight

// out[t] = sum over k, ascending, of w[t][k] * y[slot[t][k]]: an fp32 chain of
// multiply-adds from +0, as moe_combine_recv forms it, rounded once.  Bound by reads of rows that
// lie apart: 16384 tokens of 7168, 8 rows each, 364 us, 5.8 TB/s; with AHEAD loads in flight per lane
// against one after the other 415.
template <int LANES, bool F32, bool STREAM>
__global__ __launch_bounds__(256) void unsort_rows_kernel(const Rows r)
{
    typedef Vec<F32> V;
    const int64_t task = task_of<LANES>();
    const int64_t t = task / r.chunks;
    if (t >= r.tokens)
        return;
    const int v = (int)(task - t * r.chunks) * LANES + threadIdx.x % LANES;
    if (v >= r.vecs)
        return;
    const v4u* y = (const v4u*)r.x + v;
    float acc[V::N] = {};
    for (int k0 = 0; k0 < r.K; k0 += AHEAD) {
        v4u u[AHEAD];
        float w[AHEAD];
        bool has[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int64_t at = t * r.K + min(k0 + a, r.K - 1);
            const int64_t row = r.slot[at];
            has[a] = k0 + a < r.K && (uint64_t)row < (uint64_t)r.rows;
            w[a] = r.w ? r.w[at] : 1.0f;
            if (has[a])
                u[a] = load_row<STREAM>(y + row * r.vecs);
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
            if (has[a]) {
                float f[V::N];
                V::open(u[a], f);
#pragma unroll
                for (int c = 0; c < V::N; ++c)
                    acc[c] = fmaf(w[a], f[c], acc[c]);
            }
    }
    store_row<STREAM>(V::close(acc), (v4u*)r.out + t * r.vecs + v);
}

// dy[slot[t][k]] = w[t][k] * dout[t];  dw[t][k] = dout[t] . y[slot[t][k]].
// A token's row lies in the registers of `waves` waves (U vectors per lane)
// while its K rows go by, GRAD_AHEAD of them in flight; a dot product is summed
// per lane, over the lanes, then over the waves in their order.  Rows are read and written once:
// 16384 tokens of 7168, 8 rows each, 793 us, 5.0 TB/s, where a copy reaches 6.6: as for the sort,
// what is written jumps from row to row.  Rows of more than 32 wave-wide vectors (fp32 from 8200 on, bf16
// from 16392) take U = 16, whose registers spill (184 bytes of scratch per lane, bf16 656): 8192
// tokens of fp32, 4 rows each, 426 us of 8192 and 671 of 8200 (5.7, 3.6 TB/s); 4096 of bf16 213 us of
// 16384 and 1082 of 16392 (5.7, 1.1 TB/s).
constexpr int GRAD_AHEAD = 4;

template <int LANES, int U, bool F32, bool STREAM>
__global__ __launch_bounds__(1024) void unsort_rows_grad_kernel(const Rows r, int waves)
{
    typedef Vec<F32> V;
    constexpr int AT_ONCE = U > 4 ? 1 : GRAD_AHEAD;
    __shared__ float part[MAX_TOPK][16];
    const int lane = threadIdx.x % LANES;
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int wave = LANES == WAVE ? __builtin_amdgcn_readfirstlane(threadIdx.x / LANES) : 0;
    const int64_t t = LANES == WAVE ? block : block * (blockDim.x / LANES) + threadIdx.x / LANES;
    if (t >= r.tokens)
        return;
    auto vec = [&](int u) { return (u * waves + wave) * LANES + lane; };
    float d[U][V::N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        v4u raw{0, 0, 0, 0};
        if (vec(u) < r.vecs)
            raw = ((const v4u*)r.dout)[t * r.vecs + vec(u)];
        V::open(raw, d[u]);
    }
    for (int k0 = 0; k0 < r.K; k0 += AT_ONCE) {
        v4u raw[AT_ONCE][U];
        int64_t row[AT_ONCE];
        bool has[AT_ONCE];
        float w[AT_ONCE], dot[AT_ONCE];
#pragma unroll
        for (int a = 0; a < AT_ONCE; ++a) {
            const int64_t at = t * r.K + min(k0 + a, r.K - 1);
            row[a] = r.slot[at];
            has[a] = k0 + a < r.K && (uint64_t)row[a] < (uint64_t)r.rows;
            w[a] = r.w ? r.w[at] : 1.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw[a][u] = v4u{0, 0, 0, 0};
                if (r.dw && has[a] && vec(u) < r.vecs)
                    raw[a][u] = load_row<STREAM>((const v4u*)r.x + row[a] * r.vecs + vec(u));
            }
        }
#pragma unroll
        for (int a = 0; a < AT_ONCE; ++a) {
            if (r.dy && has[a])
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float g[V::N];
#pragma unroll
                    for (int c = 0; c < V::N; ++c)
                        g[c] = w[a] * d[u][c];
                    if (vec(u) < r.vecs)
                        store_row<STREAM>(V::close(g), (v4u*)r.dy + row[a] * r.vecs + vec(u));
                }
            dot[a] = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[V::N];
                V::open(raw[a][u], f);
#pragma unroll
                for (int c = 0; c < V::N; ++c)
                    dot[a] = has[a] ? fmaf(d[u][c], f[c], dot[a]) : 0.0f;
            }
        }
        if (r.dw) {
#pragma unroll
            for (int s = LANES / 2; s; s >>= 1)
#pragma unroll
                for (int a = 0; a < AT_ONCE; ++a)
                    dot[a] += __shfl_xor(dot[a], s, LANES);
#pragma unroll
            for (int a = 0; a < AT_ONCE; ++a)
                if (lane == 0 && k0 + a < r.K) {
                    if (LANES < WAVE || waves == 1)
                        r.dw[t * r.K + k0 + a] = dot[a];
                    else
                        part[k0 + a][wave] = dot[a];
                }
        }
    }
    if (LANES == WAVE && waves > 1 && r.dw) {
        __syncthreads();
        if ((int)threadIdx.x < r.K) {
            float sum = 0.0f;
            for (int w = 0; w < waves; ++w)
                sum += part[threadIdx.x][w];
            r.dw[t * r.K + threadIdx.x] = sum;
        }
    }
}

dim3 grid_of(int64_t blocks)
{
    constexpr int64_t ROW = 1 << 20;              // a grid dimension times the threads stays below 2^32
    return dim3((uint32_t)std::min(blocks, ROW), (uint32_t)((blocks + ROW - 1) / ROW));
}

int lanes_for(int vecs)
{
    int lanes = 1;
    while (lanes < vecs && lanes < WAVE)
        lanes *= 2;
    return lanes;
}

// Calls f with the number of lanes per row as a constant.
template <class F>
void with_lanes(int vecs, F f)
{
    switch (lanes_for(vecs)) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    case 32: return f(std::integral_constant<int, 32>{});
    default: return f(std::integral_constant<int, 64>{});
    }
}

Rows rows_of(const SortRows& p, int elem_bytes)
{
    Rows r{};
    r.tokens = p.tokens;
    r.rows = p.rows;
    r.K = p.K;
    r.vecs = (int)((int64_t)p.hidden * elem_bytes / 16);
    r.chunks = (r.vecs + WAVE - 1) / WAVE;
    r.x = p.x;
    r.xs = p.xs;
    r.slot = p.slot;
    r.w = p.w;
    r.out = p.out;
    r.outs = p.outs;
    r.dout = p.dout;
    r.dy = p.dy;
    r.dw = p.dw;
    return r;
}

int plan_groups(int64_t pairs)
{
    return pairs <= PLAN_ALONE ? 1 : (int)std::min<int64_t>((pairs + PLAN_RANGE - 1) / PLAN_RANGE, PLAN_GROUPS);
}

}  // namespace

size_t sort_workspace(int64_t pairs, int E)
{
    const int groups = plan_groups(pairs);
    return groups > 1 ? (size_t)groups * E * sizeof(int32_t) : 0;
}

hipError_t launch_sort_plan(int64_t pairs, int E, const int32_t* idx, int32_t* offsets, int32_t* slot,
                            int32_t* source, void* workspace, hipStream_t stream)
{
    Plan p{};
    p.pairs = pairs;
    p.E = E;
    p.groups = plan_groups(pairs);
    while ((1 << p.bits) < E)
        ++p.bits;
    p.idx = idx;
    p.offsets = offsets;
    p.slot = slot;
    p.source = source;
    const int64_t share = (pairs + p.groups - 1) / p.groups;
    p.range = std::max<int64_t>((share + PLAN_THREADS - 1) / PLAN_THREADS, 1) * PLAN_THREADS;
    if (p.groups > 1) {
        p.counts = (int32_t*)workspace;
        count_pairs_kernel<<<dim3(p.groups), dim3(PLAN_THREADS), 0, stream>>>(p);
    }
    auto launch = [&](auto threads) {                  // at most 41 KB of counts
        const int bytes = ((threads / WAVE + 2) * E + 1) * 4;
        sort_plan_kernel<threads><<<dim3(p.groups), dim3(threads), bytes, stream>>>(p);
    };
    if (E <= MAX_EXPERTS / 2)
        launch(std::integral_constant<int, PLAN_THREADS>{});
    else
        launch(std::integral_constant<int, PLAN_THREADS / 2>{});
    return hipGetLastError();
}

// The nontemporal hint (us with it, without, on rows that no cache holds yet):
// sort 131072 rows of 7168 401, 405, 24576 of 4096 39, 47, 8192 of 4096 14.2, 15.3;
// unsort 364, 415, 41, 49, 14.2, 17.9; its gradient 793, 798, 81, 90, 28, 31.  Unsort
// reads for the last time; what the other two write is the next operator's
// input, so they take it only from a size on that the 256 MB cache would not keep
// (sort 16384 rows of 4096 again and again 25.5, 23.1).  Not for rows that do not
// fill a wave, whose lines would be written in parts: sort 400000 rows of 200
// 56, 33.
constexpr int64_t WRITTEN_PAST = 128 << 20, READ_PAST = 32 << 20;

// Calls f with the hint as a constant, for the rows of `lanes` lanes.
template <class L, class F>
static void with_hint(L lanes, const Rows& r, int64_t from, F f)
{
    if constexpr (lanes == WAVE)
        if (r.rows * r.vecs * 16 >= from)
            return f(std::true_type{});
    f(std::false_type{});
}

hipError_t launch_sort_rows(const SortRows& p, int elem_bytes, hipStream_t stream)
{
    Rows r = rows_of(p, elem_bytes);
    r.extra = p.xs ? p.hidden / SCALE_BLOCK : 0;
    with_lanes(r.vecs, [&](auto lanes) {
        const int64_t blocks = (r.tokens * r.chunks + 256 / lanes - 1) / (256 / lanes);
        with_hint(lanes, r, WRITTEN_PAST, [&](auto hint) {
            sort_rows_kernel<lanes, hint><<<grid_of(blocks), dim3(256), 0, stream>>>(r);
        });
    });
    return hipGetLastError();
}

hipError_t launch_unsort_rows(const SortRows& p, bool f32, hipStream_t stream)
{
    const Rows r = rows_of(p, f32 ? 4 : 2);
    with_lanes(r.vecs, [&](auto lanes) {
        const int64_t blocks = (r.tokens * r.chunks + 256 / lanes - 1) / (256 / lanes);
        with_hint(lanes, r, READ_PAST, [&](auto hint) {
            if (f32)
                unsort_rows_kernel<lanes, true, hint><<<grid_of(blocks), dim3(256), 0, stream>>>(r);
            else
                unsort_rows_kernel<lanes, false, hint><<<grid_of(blocks), dim3(256), 0, stream>>>(r);
        });
    });
    return hipGetLastError();
}

template <int LANES, int U>
static void launch_grad(const Rows& r, bool f32, int waves, hipStream_t stream)
{
    const int threads = LANES == WAVE ? waves * WAVE : 256;
    const int64_t per = LANES == WAVE ? 1 : 256 / LANES;
    const dim3 grid = grid_of((r.tokens + per - 1) / per);
    with_hint(std::integral_constant<int, LANES>{}, r, WRITTEN_PAST, [&](auto hint) {
        if (f32)
            unsort_rows_grad_kernel<LANES, U, true, hint><<<grid, dim3(threads), 0, stream>>>(r, waves);
        else
            unsort_rows_grad_kernel<LANES, U, false, hint><<<grid, dim3(threads), 0, stream>>>(r, waves);
    });
}

hipError_t launch_unsort_rows_grad(const SortRows& p, bool f32, hipStream_t stream)
{
    const Rows r = rows_of(p, f32 ? 4 : 2);
    with_lanes(r.vecs, [&](auto lanes) {
        if constexpr (lanes < WAVE) {
            launch_grad<lanes, 1>(r, f32, 1, stream);
        } else {
            const int units = (r.vecs + WAVE - 1) / WAVE;      // wave-wide vectors of a row: up to 256
            if (units <= 1)
                launch_grad<WAVE, 1>(r, f32, 1, stream);
            else if (units <= 32)
                launch_grad<WAVE, 2>(r, f32, (units + 1) / 2, stream);
            else
                launch_grad<WAVE, 16>(r, f32, (units + 15) / 16, stream);
        }
    });
    return hipGetLastError();
}

}  // namespace ops
}  // namespace moe
