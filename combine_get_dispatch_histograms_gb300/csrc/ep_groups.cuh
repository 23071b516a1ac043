// ep_groups.cuh -- groups of rows cut into tiles: what the products' kernels share.
#pragma once
#include "ep_tcgen05.cuh"

namespace ep {

constexpr int kMaxGroups = 4096;
constexpr int kMaxTiles = 1 << 25;      // 32 groups' tiles, and a block's next tile, stay within 31 bits; no memory holds more
constexpr int kChunkRows = 2048;       // rows that share a pass over the weight's tiles

// The groups of a launch: rows as ep_row_groups says, columns in n_tiles tiles.
struct TileArgs {
    int G, n_tiles;
    int most;           // tiles of groups that share no row, at most
    const int32_t *counts, *offsets, *bases;
    int per_base;
    int64_t group_stride, rows;
};

struct GemmTile {
    int g, n;   // group, column tile
    int row0;   // first row
    int rows;   // 1 .. rows of a tile; 0: no tile is left
};

__device__ __forceinline__ int64_t group_first(const TileArgs& a, int g) {
    int64_t r = a.offsets ? (int64_t)a.offsets[g] : (int64_t)g * a.group_stride;
    if (a.bases) r += a.bases[g / a.per_base];
    return r;
}
// Rows of group g inside the arrays: what lies past their end is cut off and flagged.
__device__ __forceinline__ int group_rows(const TileArgs& a, int g, bool* cut) {
    int64_t n = a.counts ? (int64_t)a.counts[g] : a.group_stride;
    const int64_t f = group_first(a, g);
    if (n <= 0) return 0;
    if (!a.offsets && n > a.group_stride) {  // more than its region holds
        *cut = true;
        n = a.group_stride;
    }
    if (f < 0 || f >= a.rows) {
        *cut = true;
        return 0;
    }
    if (f + n > a.rows) {
        *cut = true;
        n = a.rows - f;
    }
    return (int)n;
}

// Position in a ring of barriers, by the number of steps taken: the slot's
// barrier and the parity of its next phase.  kSize is a power of two.
template <int kSize>
struct RingPos {
    uint32_t n = 0;
    __device__ __forceinline__ int slot() const { return n & (kSize - 1); }
    __device__ __forceinline__ uint32_t phase() const { return n / kSize & 1; }
    __device__ __forceinline__ uint32_t bar(uint32_t first) const { return first + slot() * 8; }
};
// One warp walks the groups for tile t, t + units, ...: 32 groups at a time,
// each lane one group's tiles.  Groups in order; inside a group, chunks of
// kChunkRows rows, column tiles inside a chunk, row tiles innermost, so that
// what runs at the same time shares a chunk of rows and few weight tiles.
template <int kTileM>
struct TileWalk {
    static constexpr int kChunkM = kChunkRows / kTileM;
    int g0 = -32, start = 0, sum = 0;  // batch of groups, its first tile, its tiles
    int inc, tiles, rows, first;       // this lane's group: tiles up to and with it, tiles, rows, first row
    bool cut = false;

    // false: no tile t.  A group has at most kMaxTiles tiles, and t is no larger, so that no sum passes 31 bits.
    __device__ __forceinline__ bool find(const TileArgs& a, int t, int lane, GemmTile* out) {
        while (t >= start + sum) {
            start += sum;
            g0 += 32;
            if (g0 >= a.G) {
                sum = 0;
                g0 = a.G;
                return false;
            }
            const int g = g0 + lane;
            rows = g < a.G ? group_rows(a, g, &cut) : 0;
            first = rows ? (int)group_first(a, g) : 0;
            tiles = (rows + kTileM - 1) / kTileM * a.n_tiles;
            inc = tiles;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            sum = __shfl_sync(0xffffffffu, inc, 31);
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, t < start + inc)) - 1;
        const int n = __shfl_sync(0xffffffffu, rows, src);
        int r = t - start - __shfl_sync(0xffffffffu, inc - tiles, src);
        const int mt = (n + kTileM - 1) / kTileM, chunk = r / (kChunkM * a.n_tiles);
        r -= chunk * kChunkM * a.n_tiles;
        const int m0 = chunk * kChunkM, mc = min(kChunkM, mt - m0), m = m0 + r % mc;
        out->g = g0 + src;
        out->n = r / mc;
        out->row0 = __shfl_sync(0xffffffffu, first, src) + m * kTileM;
        out->rows = min(kTileM, n - m * kTileM);
        return true;
    }
};

// Tiles of a launch, at most: a group's last tile may be partial, and a group
// with a tile has a row.
inline int64_t most_tiles(const TileArgs& a, int tile_rows) {
    const int64_t most = (a.rows + (int64_t)a.G * (tile_rows - 1)) / tile_rows;
    return (most < a.rows ? most : a.rows) * a.n_tiles;
}

}  // namespace ep
