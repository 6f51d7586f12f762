// What the products of rows grouped by expert share: loads from memory to LDS,
// the LDS layout of 128-byte rows, and the division of ragged experts' rows
// into tiles.
#pragma once

#include <algorithm>

#include "ops_common.h"

namespace moe {
namespace ops {

typedef const __attribute__((address_space(1))) void gvoid;
typedef __attribute__((address_space(3))) void lvoid;

// STREAM: the nontemporal hint, for bytes that no other workgroup will read.
template <bool STREAM>
__device__ inline void load_lds16(const uint8_t* g, uint8_t* l)
{
    __builtin_amdgcn_global_load_lds((gvoid*)g, (lvoid*)l, 16, 0, STREAM ? 2 : 0);
}

__device__ inline void load_lds4(const float* g, uint8_t* l)
{
    __builtin_amdgcn_global_load_lds((gvoid*)g, (lvoid*)l, 4, 0, 0);
}

// Everything this wave loaded but its last n loads has arrived in LDS, its own
// LDS reads are done, and so it is with every wave of the workgroup.
template <int N>
__device__ inline void wait_loads_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16-byte piece c of row r lies at place c ^ swizzle(r) of the row's 128
// bytes, so that the 16 rows a fragment reads at once spread over the banks.
__device__ inline int swizzle(int r) { return (r >> 1) & 7; }

// How many parts of `size` (the last one smaller) n >= 0 indices have.  An expert
// may have nearly 2^31 rows: what is added to them passes that.
__host__ __device__ constexpr int parts_of(int n, int size)
{
    return (int)(((uint32_t)n + (uint32_t)(size - 1)) / (uint32_t)size);
}
static_assert(parts_of(0, 64) == 0 && parts_of(1, 64) == 1 && parts_of(64, 64) == 1 && parts_of(65, 64) == 2 &&
                  parts_of(INT32_MAX, 64) == 1 << 25 && parts_of(INT32_MAX, 256) == 1 << 23,
              "up to the most rows");

struct Place {
    int e, m0, rows;          // expert, first row of the tile, rows of the tile (> 0)
    int n_tile;
};

// Workgroups of a launch are numbered over both grid dimensions.
__device__ inline int64_t workgroup_id() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// The tile of workgroup `id` of a launch.  Consecutive workgroups go to the 8
// XCDs in turn: each XCD takes one contiguous run of tiles, so that the tiles
// sharing weights share its L2.  TURNS: runs of 32 tiles in turn, as many as run on
// an XCD at once, so that the XCDs work near each other and share the cache behind
// their L2 too; what is left of a whole round of 256 in one run each.
template <bool TURNS>
__device__ inline bool tile_of_id(int64_t id, int64_t tiles, int64_t& t)
{
    int64_t first = 0;
    if (TURNS) {
        first = tiles & ~(int64_t)255;
        if (id < first) {
            t = (id & ~(int64_t)255) + ((id & 7) << 5) + (id >> 3 & 31);
            return true;
        }
        id -= first;
    }
    const int64_t per_xcd = (tiles - first + 7) / 8;
    const int64_t at = id >> 3;
    t = first + (id & 7) * per_xcd + at;
    return at < per_xcd && t < tiles;
}

// Tile t of the launch: experts in order, each expert's tiles in groups of up
// to 8 row tiles, row tiles fastest inside a group.  Every wave finds it for
// itself: lane l holds experts [l*per, (l+1)*per), PER >= per of them in
// registers, so that one trip to memory is enough.
template <int BM, int PER, bool TURNS = false>
__device__ inline bool find_tile(const int32_t* __restrict__ offsets, int E, int64_t rows_max, int n_tiles,
                                 Place& out, int64_t id = workgroup_id(), int lane = threadIdx.x & (WAVE - 1))
{
    const int per = (E + WAVE - 1) / WAVE;
    const int rmax = (int)rows_max;
    int o[PER + 1];
#pragma unroll
    for (int i = 0; i <= PER; ++i)
        o[i] = offsets[min(lane * per + min(i, per), E)];
    int mine = 0;
#pragma unroll
    for (int i = 0; i <= PER; ++i) {
        o[i] = min(max(o[i], 0), rmax);
        if (i > 0)
            mine += parts_of(max(o[i] - o[i - 1], 0), BM);
    }
    const int upto = wave_scan(mine);
    const int64_t tiles = (int64_t)__builtin_amdgcn_readlane(upto, WAVE - 1) * n_tiles;
    int64_t t;
    if (!tile_of_id<TURNS>(id, tiles, t))
        return false;
    // the lane whose experts hold the tile, and there the expert
    const int src = __popcll(__ballot((int64_t)upto * n_tiles <= t));
    int64_t u = t - (int64_t)(upto - mine) * n_tiles;
    int e = lane * per, a = o[0], b = o[1], m_tiles = parts_of(max(b - a, 0), BM);
#pragma unroll
    for (int i = 1; i < PER; ++i)
        if (u >= (int64_t)m_tiles * n_tiles) {
            u -= (int64_t)m_tiles * n_tiles;
            e = lane * per + i;
            a = o[i];
            b = o[i + 1];
            m_tiles = parts_of(max(b - a, 0), BM);
        }
    out.e = __builtin_amdgcn_readlane(e, src);
    a = __builtin_amdgcn_readlane(a, src);
    b = __builtin_amdgcn_readlane(b, src);
    m_tiles = parts_of(max(b - a, 0), BM);
    const int64_t v = (int64_t)__builtin_amdgcn_readlane((int)(u >> 32), src) << 32 |
                      (uint32_t)__builtin_amdgcn_readlane((int)u, src);
    // (ascending offsets always pass; others, whose tiles may be beyond counting,
    // stay inside the rows)
    if (b <= a || v < 0 || v >= (int64_t)m_tiles * n_tiles)
        return false;
    constexpr int GROUP = 8;
    const int64_t per_group = (int64_t)GROUP * n_tiles;
    const int g = (int)(v / per_group);
    const int in = (int)(v - g * per_group);
    const int gm = min(GROUP, m_tiles - g * GROUP);
    out.m0 = a + (g * GROUP + in % gm) * BM;
    out.rows = min(BM, b - out.m0);
    out.n_tile = in / gm;
    return true;
}

// Workgroups of a launch that covers every way the rows can fall to the
// experts, for tiles of BM rows: sum of ceil(rows_e / BM) over the experts
// that can have rows, at most, times the tiles of columns; a multiple of 8.
inline int64_t workgroups(int64_t rows, int E, int bm, int n_tiles)
{
    const int64_t used = std::min<int64_t>(rows, E);
    return (((rows - used) / bm + used) * n_tiles + 7) / 8 * 8;
}

inline dim3 grid_of(int64_t blocks)
{
    constexpr int64_t ROW = 1 << 20;              // a grid dimension times the threads stays below 2^32
    return dim3((uint32_t)std::min(blocks, ROW), (uint32_t)((blocks + ROW - 1) / ROW));
}

}  // namespace ops
}  // namespace moe
