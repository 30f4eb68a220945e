// expert_rows.cuh -- which rows of the receive buffer a CTA of the experts'
// products takes, and the gate of a pair.  P: the parameters of a product (E in
// w.E, mode, capacity, counts, offsets, R, err_flags).
#pragma once
#include "block_device.cuh"

namespace ep {

// x times its sigmoid, by exp(-|x|): that never overflows, so a large negative
// x leaves what exp(x) leaves of it.  expf is good to two units in the last
// place; the fast form's error grows with |x|.
__device__ __forceinline__ float silu(float x) {
    const float e = expf(-fabsf(x));
    return x * __fdividef(x < 0.f ? e : 1.f, 1.f + e);
}

struct RowTile {
    int e;          // expert, -1: none
    int rows;       // rows of the tile
    int64_t first;  // its first row
};

// Rows of expert e that lie inside the buffer; a claim beyond it gives none.
template <typename P>
__device__ __forceinline__ int expert_rows(const P& p, int e, int64_t* first, bool* bad) {
    int64_t a, n;
    if (p.mode != 0) {
        a = (int64_t)e * p.capacity;
        n = min(p.counts[e], p.capacity);
    } else if (p.offsets != nullptr) {
        a = p.offsets[e];
        n = p.offsets[e + 1] - a;
    } else {
        a = 0;
        n = p.R;
    }
    *first = a;
    *bad = n > 0 && (a < 0 || a + n > p.R);
    return *bad || n < 0 ? 0 : (int)n;
}

// tile_rows is a power of two
__device__ __forceinline__ int tiles_of(int rows, int tile_rows) {
    return (rows >> (31 - __clz(tile_rows))) + ((rows & (tile_rows - 1)) != 0);
}

constexpr int kMaxTiles = (1 << 26) - 1;     // 32 lanes' worth of them fit 31 bits
constexpr int kScan = 8;    // experts whose rows a lane looks up at a time: their loads are in flight together

// Tile `at` in the order of experts and of rows within an expert.  One warp;
// lane l counts the tiles of experts [l * per, (l + 1) * per).
template <typename P>
__device__ __forceinline__ RowTile find_tile(const P& p, int at, int tile_rows, int grid_tiles) {
    const int lane = threadIdx.x & 31;
    const int per = (p.w.E + 31) / 32;
    const int e0 = min(lane * per, p.w.E), e1 = min(e0 + per, p.w.E);
    // bad offsets may claim every row many times: a lane's sum is cut off where no good layout comes to
    int mine = 0;
    bool any_bad = false;
    int64_t first[kScan];
    int n[kScan];
    auto look_up = [&](int from) {
        bool bad[kScan];
#pragma unroll
        for (int j = 0; j < kScan; ++j) {
            n[j] = 0;
            bad[j] = false;
            if (from + j < e1) n[j] = expert_rows(p, from + j, &first[j], &bad[j]);
        }
#pragma unroll
        for (int j = 0; j < kScan; ++j) any_bad |= bad[j];
    };
    for (int from = e0; from < e1; from += kScan) {
        look_up(from);
#pragma unroll
        for (int j = 0; j < kScan; ++j) mine = min(mine + tiles_of(n[j], tile_rows), kMaxTiles);
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
    }
    const int total = __shfl_sync(0xffffffffu, upto, 31);
    if (at == 0 && p.err_flags != nullptr) {
        if (any_bad) atomicOr(p.err_flags, kErrBadSlot);
        if (total > grid_tiles && lane == 0) atomicOr(p.err_flags, kErrCapacity);
    }
    RowTile r{-1, 0, 0};
    if (at >= total) return r;
    const int owner = __ffs(__ballot_sync(0xffffffffu, upto > at)) - 1;
    if (lane == owner) {
        int left = at - (upto - mine);
        for (int from = e0; from < e1 && r.e < 0; from += kScan) {
            if (per > kScan) look_up(from);       // else n still holds them all
#pragma unroll
            for (int j = 0; j < kScan; ++j) {
                const int tiles = tiles_of(n[j], tile_rows);
                if (r.e < 0 && left >= 0 && left < tiles)
                    r = RowTile{from + j, min(n[j] - left * tile_rows, tile_rows), first[j] + (int64_t)left * tile_rows};
                left -= tiles;
            }
        }
    }
    r.e = __shfl_sync(0xffffffffu, r.e, owner);
    r.rows = __shfl_sync(0xffffffffu, r.rows, owner);
    r.first = __shfl_sync(0xffffffffu, r.first, owner);
    return r;
}

// The same for a single matrix: every thread looks for itself.
template <typename P>
__device__ __forceinline__ RowTile tile_of_one(const P& p, int at, int tile_rows, int grid_tiles) {
    int64_t first;
    bool bad;
    const int n = expert_rows(p, 0, &first, &bad), tiles = tiles_of(n, tile_rows);
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.err_flags != nullptr) {
        if (bad) atomicOr(p.err_flags, kErrBadSlot);
        if (tiles > grid_tiles) atomicOr(p.err_flags, kErrCapacity);
    }
    if (at >= tiles) return RowTile{-1, 0, 0};
    return RowTile{0, min(n - at * tile_rows, tile_rows), first + (int64_t)at * tile_rows};
}

}  // namespace ep
