// i8_tiles.h -- how the 8-bit products cut experts' rows into tiles, as plain
// host/device functions, so that the arithmetic is checked on the CPU at the
// largest buffers (R up to 2^31 - 1).
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define EP_HOST_DEVICE_INLINE __host__ __device__ __forceinline__
#else
#define EP_HOST_DEVICE_INLINE inline
#endif

namespace ep {

// Sums of tiles stop here.  A good layout, of less than 2^31 rows and up to 1024
// experts, makes fewer; bad offsets may claim rows many times.
constexpr int kMostTiles = (1 << 26) + 1024;

EP_HOST_DEVICE_INLINE int add_tiles(int a, int b) { return a + b < kMostTiles ? a + b : kMostTiles; }

// Tiles of up to `tile` rows that n rows (0..2^31 - 1) need.  The sum is beyond what a signed 32-bit number holds.
EP_HOST_DEVICE_INLINE int tiles_needed(int n, int tile) { return (int)(((uint32_t)n + (uint32_t)tile - 1) / (uint32_t)tile); }

// Tiles of n rows (n > 0): as few as hold them, each of about as many rows, in 16s (which
// is never more than `tile`, a multiple of 16, while n rows need them all).
EP_HOST_DEVICE_INLINE int tile_rows_of(int n, int tile) {
    return (tiles_needed(n, tiles_needed(n, tile)) + 15) & ~15;          // as many tiles, of how many rows each
}

}  // namespace ep
