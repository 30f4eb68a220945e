// Host-side check of the tokens that a CTA's warps take (route_runs.h): replays
// every warp's walk over single runs, also at the end of the largest batches,
// as the kernels make it (the next token is fetched before the present one is
// worked on), and checks that each token of the run is fetched and worked on
// exactly once and no other is.  Also that runs cover the tokens and that a
// grid holds their number.  Prints one line; exit code 0 when all cases pass.
#include <climits>
#include <cstdio>
#include <vector>

#include "route_runs.h"

using namespace ep;

static bool walk(int begin, int end, int warps) {
    std::vector<int> fetched(end - begin), worked(end - begin);
    bool good = true;
    auto mark = [&](std::vector<int>& seen, uint32_t t) {
        if (t < (uint32_t)begin || t >= (uint32_t)end)
            good = false;
        else
            ++seen[t - (uint32_t)begin];
    };
    for (int w = 0; w < warps; ++w) {
        auto fetch = [&](uint32_t t) {
            if (!in_run(t, end)) return;
            mark(fetched, t);
        };
        fetch(first_token(begin, w));
        int steps = 0;
        for (uint32_t t = first_token(begin, w); in_run(t, end); t = next_token(t, warps)) {
            fetch(next_token(t, warps));
            mark(worked, t);
            if (++steps > end - begin) return false;
        }
    }
    for (int n : fetched) good &= n == 1;
    for (int n : worked) good &= n == 1;
    return good;
}

int main() {
    long cases = 0;
    for (int warps : {4, 8, 16})
        for (int tokens = 0; tokens <= 300; ++tokens)
            for (int64_t end : {(int64_t)tokens, (int64_t)tokens + 1, (int64_t)tokens + 12345, (int64_t)INT_MAX - 20, (int64_t)INT_MAX - 1,
                                (int64_t)INT_MAX}) {
                ++cases;
                if (!walk((int)(end - tokens), (int)end, warps)) {
                    std::printf("warps=%d tokens=%d end=%lld: not every token once\n", warps, tokens, (long long)end);
                    return 1;
                }
            }
    for (int T : {0, 1, 15, 16, 17, 4864, 4865, 9728, 9729, 77824, 77825, INT_MAX - 4864, INT_MAX - 4863, INT_MAX - 1, INT_MAX})
        for (int S : {1, 65535}) {
            ++cases;
            const int chunk = run_tokens(T);
            const int64_t runs = num_runs(T, chunk, S);
            const int want = T > 15 * 4864 ? 256 : T <= 4864 ? 16 : (T - 1) / 4864 * 16 + 16;
            if (chunk != want || runs - (S - 1) != ((int64_t)T + chunk - 1) / chunk || runs > INT_MAX) {
                std::printf("T=%d S=%d: chunk=%d runs=%lld\n", T, S, chunk, (long long)runs);
                return 1;
            }
        }
    std::printf("route runs ok: %ld cases\n", cases);
    return 0;
}
