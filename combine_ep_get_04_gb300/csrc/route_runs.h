// route_runs.h -- which tokens a CTA and each of its warps take, as plain
// host/device functions, so that the arithmetic is checked on the CPU at the
// largest batches (T up to 2^31 - 1).
#pragma once

#include <algorithm>
#include <cstdint>

#if defined(__CUDACC__)
#define EP_HOST_DEVICE_INLINE __host__ __device__ __forceinline__
#else
#define EP_HOST_DEVICE_INLINE inline
#endif

namespace ep {

constexpr int kRunWarps = 16;          // of a CTA that sums its run

// Tokens of a run: one for each warp until there are two CTAs for every SM,
// then more, so that the per-run sums stay small beside the logits (forward pass
// of 32,768 tokens, 256 experts 32.1 us; with runs of up to 64 tokens 36.3).
inline int run_tokens(int T) { return kRunWarps * std::min((T - 1) / (kRunWarps * 304) + 1, 16); }

// Runs of T tokens in S sequences: they end at multiples of `chunk` tokens and
// at the ends of sequences.
inline int64_t num_runs(int T, int chunk, int S) { return ((int64_t)T + chunk - 1) / chunk + S - 1; }

// Warp w of a run [begin, end) takes token begin + w and then every warps-th.
// The numbers it compares with the end go up to `warps` past it, beyond what a
// signed 32-bit number holds.
EP_HOST_DEVICE_INLINE uint32_t first_token(int begin, int w) { return (uint32_t)begin + (uint32_t)w; }
EP_HOST_DEVICE_INLINE uint32_t next_token(uint32_t t, int warps) { return t + (uint32_t)warps; }
EP_HOST_DEVICE_INLINE bool in_run(uint32_t t, int end) { return t < (uint32_t)end; }

}  // namespace ep
