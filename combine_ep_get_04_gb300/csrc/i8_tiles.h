// i8_tiles.h -- how the 8-bit products cut experts' rows into tiles, as plain
// host/device functions, so that the arithmetic is checked on the CPU at the
// largest buffers (R up to 2^31 - 1).
#pragma once

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

// Tiles of up to `tile` rows that n rows need.
EP_HOST_DEVICE_INLINE int tiles_needed(int n, int tile) { return n / tile + (n % tile != 0); }

// Tiles of n rows (n > 0): as few as hold them, each of about as many rows, in 16s (which
// is never more than `tile`, a multiple of 16, while n rows need them all).
EP_HOST_DEVICE_INLINE int tile_rows_of(int n, int tile) {
    const int tiles = tiles_needed(n, tile);
    return (n / tiles + (n % tiles != 0) + 15) & ~15;
}

}  // namespace ep
