// Host-side check of how the 8-bit products cut rows into tiles (i8_tiles.h), up
// to the largest buffer: the tiles of an expert cover its rows once, none is
// larger than the kernel's, sums of tiles of every good layout are exact, and
// those of bad ones stop at kMostTiles.  Prints one line; exit code 0 when all pass.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <vector>

#include "i8_tiles.h"

using namespace ep;

static long cases = 0;

static bool cut(int64_t n, int tile) {
    ++cases;
    const int64_t tiles = (n + tile - 1) / tile;
    const int64_t size = tile_rows_of((int)n, tile);
    // the last tile begins before the end, all of them reach it
    const bool good = tiles_needed((int)n, tile) == tiles && size > 0 && size <= tile && size % 16 == 0 && (tiles - 1) * size < n && tiles * size >= n;
    if (!good) std::printf("n=%lld tile=%d: %d tiles of %lld rows\n", (long long)n, tile, tiles_needed((int)n, tile), (long long)size);
    return good;
}

static bool sum(const std::vector<int64_t>& rows, int tile) {
    ++cases;
    int64_t exact = 0;
    int got = 0;
    for (int64_t n : rows) {
        exact += (n + tile - 1) / tile;
        got = add_tiles(got, tiles_needed((int)n, tile));
    }
    const int64_t want = exact < kMostTiles ? exact : kMostTiles;
    if (got != want) std::printf("%zu experts, tile=%d: %d tiles, not %lld\n", rows.size(), tile, got, (long long)want);
    return got == want;
}

int main() {
    bool good = true;
    for (int tile : {32, 64, 128, 160}) {
        for (int n = 1; n <= 5000; ++n) good &= cut(n, tile);
        for (int64_t at : {(int64_t)1 << 16, (int64_t)1 << 24, (int64_t)1 << 30, (int64_t)INT_MAX - 400})
            for (int64_t n = at - 400; n <= at + 400; ++n) good &= cut(n, tile);
        for (int E : {1, 2, 31, 300, 1024}) {
            // all rows with one expert; one row each and the rest with the last; bad: all rows with every expert
            good &= sum({INT_MAX}, tile);
            std::vector<int64_t> few(E, 1), bad(E, INT_MAX);
            few.back() = INT_MAX - (E - 1);
            good &= sum(few, tile) && sum(bad, tile);
        }
    }
    // what a good layout makes at most is below the limit: rows that leave 31 over with every expert
    const int64_t E = 1024, most = ((int64_t)INT_MAX + 31 * E) / 32;
    good &= most < kMostTiles;
    if (!good) return 1;
    std::printf("i8 tiles ok: %ld cases\n", cases);
    return 0;
}
