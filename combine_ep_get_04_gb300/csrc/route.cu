// route.cu -- the choice of experts from router logits, per-expert counts,
// the balance and z losses, and the gradient of all of it.
//
// One warp per token, the token's logits in registers, as wide loads bring them:
// a lane's NPL values are vectors of neighbours, up to 16 bytes, 32 vectors
// apart, and a group of experts is in most cases a few lanes' vectors.  The choice compares 32-bit keys whose unsigned order is
// that of the floats, so a maximum over the warp is one redux.sync.  What is
// summed over tokens (probabilities, copies, squared log normalisers) is
// summed per run of tokens of one sequence by one CTA and then over the runs in
// their order, so the losses do not depend on which CTA runs first.
#include <algorithm>
#include <cstring>
#include <cuda_bf16.h>

#include "block_device.cuh"
#include "block_kernels.h"
#include "route_runs.h"

namespace ep {
namespace {

constexpr int kMaxRouteWarps = 16;
constexpr int kChoiceTokens = 8;       // most tokens of its warps
constexpr int kBackwardWarps = 8;
constexpr int kBackwardTokens = 4;     // most tokens of a warp in the backward pass
constexpr int kSumWarps = 32;
constexpr int kSumRuns = 8;
constexpr int kSumCluster = 8;         // most CTAs of a sequence
constexpr uint32_t kAll = 0xffffffffu;

// Unsigned order of the key = order of the float; -0 counts as 0, NaN comes
// below everything, and keys up to kUnchoosable (-inf) are never chosen.
constexpr uint32_t kUnchoosable = 0x007fffffu;

__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));
    const uint32_t key = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return x != x ? 0u : key;
}

// Run `c` holds tokens [begin, end) of sequence s: runs end at multiples of
// `chunk` tokens and at the ends of sequences, and run floor(t / chunk) + s
// holds token t of sequence s, so that the runs of a sequence are consecutive.
struct Run {
    int s, begin, end;
};

__device__ __forceinline__ int seq_begin(const RouteParams& p, int s) {
    if (p.seq_offsets == nullptr) return s == 0 ? 0 : p.T;
    return min(max(p.seq_offsets[s], 0), p.T);
}

__device__ __forceinline__ Run find_run(const RouteParams& p, int c) {
    if (p.seq_offsets == nullptr) {
        const int64_t first = (int64_t)c * p.chunk;
        return Run{0, (int)min(first, (int64_t)p.T), (int)min(first + p.chunk, (int64_t)p.T)};
    }
    int lo = 0, hi = p.S - 1;
    {
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_begin(p, mid) / p.chunk + mid <= c)
                lo = mid;
            else
                hi = mid - 1;
        }
    }
    const int64_t first = (int64_t)(c - lo) * p.chunk;
    return Run{lo, (int)min(max(first, (int64_t)seq_begin(p, lo)), (int64_t)p.T),
               (int)min(first + p.chunk, (int64_t)seq_begin(p, lo + 1))};
}

template <bool F32>
__device__ __forceinline__ float load_logit(const void* base, int64_t at) {
    if (F32) return static_cast<const float*>(base)[at];
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(base)[at] << 16);
}

// Values of one wide access: 16 bytes of them, or all that a lane has.
__host__ __device__ constexpr int wide_values(int npl, bool f32) { return f32 ? (npl < 4 ? npl : 4) : (npl < 8 ? npl : 8); }

// Where value i of a lane lies behind its first, value lane * V of the row.
template <int V>
__device__ __forceinline__ constexpr int value_at(int i) { return i / V * 32 * V + i % V; }

template <int WORDS> struct Wide;
template <> struct Wide<1> { using T = uint32_t; };
template <> struct Wide<2> { using T = uint2; };
template <> struct Wide<4> { using T = uint4; };

// A lane's NPL logits as they lie in memory, -inf beyond the row.  `row` is the
// place of the lane's first, `left` the values from there to the row's end.
template <int NPL, bool F32>
struct RawLogits {
    static constexpr int V = wide_values(NPL, F32), kWords = F32 ? V : V / 2;
    uint32_t w[F32 ? NPL : NPL / 2];

    __device__ __forceinline__ void load(const unsigned char* row, int left, bool wide) {
#pragma unroll
        for (int v = 0; v < NPL / V; ++v) {
            const int first = v * 32 * V;
            if (wide) {
                const bool in = first < left;
                typename Wide<kWords>::T x{};
                if (in) x = *reinterpret_cast<const typename Wide<kWords>::T*>(row + first * (F32 ? 4 : 2));
                uint32_t words[kWords];
                memcpy(words, &x, sizeof(x));
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[v * kWords + i] = in ? words[i] : F32 ? 0xff800000u : 0xff80ff80u;
            } else {
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    const int at = first + (F32 ? i : 2 * i);
                    if (F32) {
                        w[v * kWords + i] = at < left ? reinterpret_cast<const uint32_t*>(row)[at] : 0xff800000u;
                    } else {
                        const uint16_t* from = reinterpret_cast<const uint16_t*>(row);
                        const uint32_t lo = at < left ? from[at] : 0xff80u, hi = at + 1 < left ? from[at + 1] : 0xff80u;
                        w[v * kWords + i] = lo | hi << 16;
                    }
                }
            }
        }
    }
    __device__ __forceinline__ float get(int i) const {
        return F32 ? __uint_as_float(w[i]) : __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

// Writes a lane's NPL values.
template <int NPL, bool F32>
__device__ __forceinline__ void store_values(unsigned char* row, int left, bool wide, const float (&d)[NPL]) {
    constexpr int V = wide_values(NPL, F32), kWords = F32 ? V : V / 2;
#pragma unroll
    for (int v = 0; v < NPL / V; ++v) {
        const int first = v * 32 * V;
        if (wide) {
            uint32_t w[kWords];
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const int at = v * V + (F32 ? i : 2 * i);
                w[i] = F32 ? __float_as_uint(d[at]) : pack_bf16x2(d[at], d[F32 ? at : at + 1]);
            }
            typename Wide<kWords>::T x;
            memcpy(&x, w, sizeof(x));
            if (first < left) *reinterpret_cast<typename Wide<kWords>::T*>(row + first * (F32 ? 4 : 2)) = x;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (first + i >= left) continue;
                if (F32)
                    reinterpret_cast<float*>(row)[first + i] = d[v * V + i];
                else
                    reinterpret_cast<__nv_bfloat16*>(row)[first + i] = __float2bfloat16_rn(d[v * V + i]);
            }
        }
    }
}

// A lane's NPL words of a row in shared memory, V neighbours each.
template <int NPL, int V>
__device__ __forceinline__ void load_shared(const uint32_t* row, uint32_t (&x)[NPL]) {
    constexpr int kWords = V < 4 ? V : 4;
#pragma unroll
    for (int i = 0; i < NPL; i += kWords) {
        const auto w = *reinterpret_cast<const typename Wide<kWords>::T*>(row + value_at<V>(i));
        memcpy(x + i, &w, sizeof(w));
    }
}

template <int NPL, int V>
__device__ __forceinline__ void store_shared(uint32_t* row, const float (&x)[NPL]) {
    constexpr int kWords = V < 4 ? V : 4;
#pragma unroll
    for (int i = 0; i < NPL; i += kWords) {
        typename Wide<kWords>::T w;
        memcpy(&w, x + i, sizeof(w));
        *reinterpret_cast<typename Wide<kWords>::T*>(row + value_at<V>(i)) = w;
    }
}

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Sorts N (a power of two) values, largest first: Batcher's odd-even merge
// sort (K. E. Batcher, "Sorting networks and their applications", 1968).
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&v)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t hi = max(v[i + j], v[i + j + k]), lo = min(v[i + j], v[i + j + k]);
                        v[i + j] = hi;
                        v[i + j + k] = lo;
                    }
}

// The groups a token may choose from, as a mask.  A group is `lanes` lanes'
// vectors, a power of two, or of any size (lanes = 0).  `best` is a row of 32
// words of shared memory.
template <int NPL, int V>
__device__ __forceinline__ uint32_t choose_groups(const RouteParams& p, int lanes, const uint32_t (&key)[NPL], uint32_t* best) {
    const int lane = threadIdx.x & 31;
    uint32_t mine = 0;             // the largest key of group `lane`
    if (lanes > 0) {
        const int shift = __ffs(lanes) - 1, from = lane << shift;       // the group's first vector
#pragma unroll
        for (int v = 0; v < NPL / V; ++v) {
            uint32_t m = key[v * V];
#pragma unroll
            for (int i = 1; i < V; ++i) m = max(m, key[v * V + i]);
            for (int d = 1; d < lanes; d <<= 1) m = max(m, __shfl_xor_sync(kAll, m, d));
            m = __shfl_sync(kAll, m, from);
            mine = from >> 5 == v ? m : mine;
        }
    } else {
        best[lane] = 0;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane * V + value_at<V>(i);
            if (e < p.E) atomicMax(&best[e / p.per_group], key[i]);
        }
        __syncwarp();
        mine = best[lane];
        __syncwarp();
    }
    mine = lane < p.groups ? mine : 0u;
    // a group stays if fewer than topk_groups come before it
    int before = 0;
#pragma unroll 8
    for (int g = 0; g < p.groups; ++g) before += __shfl_sync(kAll, mine, g) + (g < lane ? 1u : 0u) > mine ? 1 : 0;
    return __ballot_sync(kAll, mine > kUnchoosable && before < p.topk_groups);
}

// The choice by whole keys, for tokens whose best keys agree in their upper 22
// bits: every round looks for the next pair (key, index) in memory.  Returns
// lane j's expert, or -1.
template <bool F32>
__device__ __noinline__ int choose_exactly(const RouteParams& p, uint32_t t, uint32_t keep) {
    const int lane = threadIdx.x & 31;
    uint32_t last = kAll;
    int last_e = -1, chosen = -1;
    for (int j = 0; j < p.k; ++j) {
        uint32_t top = 0;
        int top_e = 0;
        for (int e = lane; e < p.E; e += 32) {
            if (!(keep >> (e / p.per_group) & 1u)) continue;
            const float x = load_logit<F32>(p.logits, t * p.ld + e);
            const uint32_t key = order_key(p.select_bias != nullptr ? __fadd_rn(x, p.select_bias[e]) : x);
            if ((key < last || (key == last && e > last_e)) && key > top) {
                top = key;
                top_e = e;
            }
        }
        const uint32_t best = __reduce_max_sync(kAll, top);
        if (best <= kUnchoosable) break;
        last = best;
        last_e = (int)__reduce_min_sync(kAll, top == best ? (uint32_t)top_e : kAll);
        if (lane == j) chosen = last_e;
    }
    return chosen;
}

// Puts candidates (lane j: the expert `e` of place j by its word, -1 beyond the
// last) into the order of their whole keys: one look at each key, and every
// lane counts the candidates before its own.  Returns lane j's expert.
template <bool F32>
__device__ __forceinline__ int reorder(const RouteParams& p, uint32_t t, int e, int count) {
    const int lane = threadIdx.x & 31;
    uint32_t key = 0;
    if (e >= 0) {
        const float x = load_logit<F32>(p.logits, t * p.ld + e);
        key = order_key(p.select_bias != nullptr ? __fadd_rn(x, p.select_bias[e]) : x);
    }
    int before = 0;
    for (int j = 0; j < count; ++j) {
        const uint32_t k = __shfl_sync(kAll, key, j);
        const int o = __shfl_sync(kAll, e, j);
        before += k > key || (k == key && o < e) ? 1 : 0;
    }
    if (e < 0) before = 32;
    int chosen = -1;
    for (int j = 0; j < min(count, p.k); ++j) {
        const int from = __ffs(__ballot_sync(kAll, before == j)) - 1;
        const int o = __shfl_sync(kAll, e, from);
        if (lane == j) chosen = o;
    }
    return chosen;
}

// The choice, and for training what the losses need.
//
// A lane sorts its experts by words that hold the upper 22 bits of the key and
// the index below them (lower indices larger), two instructions a comparison;
// then a round is one redux.sync over the lanes' first words, and the lane it
// came from moves on to its next.  Where neighbours among the best agree in
// their 22 bits (one token in fifty of normal logits in fp32, none in bf16,
// whose keys have 16 bits) the rounds go on to the end of that stretch, and the
// candidates are put into the order of their whole keys.
//
// Bound by instruction issue (60 % of the slots, some 560 instructions a token of
// 128 experts in groups) and by a token's chain of reductions, not by memory:
// choice alone, 256 fp32 logits: 128 tokens 2.9 us, 4,096 4.7, 32,768 22.0 (1.5
// TB/s of logits); 16,384 tokens of 128 bf16 logits in 8 groups 13.5.  One warp a
// token rather than a thread or half a warp: the reductions are single
// instructions, and a small batch spreads over the SMs.  64 registers: with 40,
// for three CTAs of 16 warps an SM, the sort spills (choice of 128 bf16 logits
// 15.2 against 13.5 us, with the losses 27.7 against 20.5).
template <int NPL, bool F32>
__global__ void __launch_bounds__(kMaxRouteWarps * 32, NPL <= 8 ? 2 : 1) route_kernel(const __grid_constant__ RouteParams p) {
    constexpr int V = wide_values(NPL, F32), kRow = NPL * 32;      // kRow: words of a row of shared memory
    extern __shared__ __align__(16) uint32_t smem[];   // rows: copies, selection bias, group bits, and a warp's probabilities each
    __shared__ uint32_t group_best[kMaxRouteWarps][32];
    __shared__ float warp_z[kMaxRouteWarps];
    __shared__ int warp_live[kMaxRouteWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int e0 = lane * V, left = p.E - e0;
    uint32_t *hist = smem, *bias = smem + kRow, *group_bit = smem + 2 * kRow, *prob = smem + 3 * kRow;
    const bool sums = p.losses != nullptr, has_bias = p.select_bias != nullptr, exact = !F32 && !has_bias;
    // lanes of a group, if it is whole vectors, a power of two of them, and no more than a warp has lanes
    const int vectors = p.per_group / V;
    const int group_lanes = p.per_group % V == 0 && (vectors & (vectors - 1)) == 0 && vectors <= 32 ? vectors : 0;
    for (int e = threadIdx.x; e < kRow; e += blockDim.x) {
        if (sums) hist[e] = 0;
        if (p.groups > 1 && group_lanes == 0) group_bit[e] = e < p.E ? 1u << (e / p.per_group) : 0u;
    }
    pdl_launch_dependents();
    pdl_wait();
    if (has_bias)
        for (int e = threadIdx.x; e < kRow; e += blockDim.x) bias[e] = e < p.E ? __float_as_uint(p.select_bias[e]) : 0u;
    if (sums && blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;      // of the kernel after this one
    const Run run = find_run(p, blockIdx.x);
    __syncthreads();
    constexpr int kSize = F32 ? 4 : 2;
    const unsigned char* row = static_cast<const unsigned char*>(p.logits) + ((int64_t)first_token(run.begin, warp) * p.ld + e0) * kSize;
    RawLogits<NPL, F32> next;
    bool next_mask = true;
    auto fetch = [&](uint32_t t) {      // a token's logits are on their way while the one before it is worked on
        if (!in_run(t, run.end)) return;
        next.load(row, left, p.wide != 0);
        next_mask = p.token_mask == nullptr || p.token_mask[t] != 0;
        row += warps * p.ld * kSize;
    };
    float psum[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) psum[i] = 0.f;
    float z = 0.f;
    int n_live = 0;
    fetch(first_token(run.begin, warp));
    for (uint32_t t = first_token(run.begin, warp); in_run(t, run.end); t = next_token(t, warps)) {
        float l[NPL], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            l[i] = next.get(i);
            top = fmaxf(top, l[i]);
        }
        const bool mask = next_mask;
        fetch(next_token(t, warps));
        const int64_t at = (int64_t)t * p.k;
        top = warp_max(top);
        if (!mask || !(top > -INFINITY)) {
            if (lane < p.k) {
                p.topk_idx[at + lane] = -1;
                p.topk_w[at + lane] = 0.f;
            }
            if (p.lse != nullptr && lane == 0) p.lse[t] = -INFINITY;
            continue;
        }
        uint32_t word[NPL];
        if (has_bias) {
            uint32_t b[NPL];
            load_shared<NPL, V>(bias + e0, b);
#pragma unroll
            for (int i = 0; i < NPL; ++i) word[i] = order_key(__fadd_rn(l[i], __uint_as_float(b[i])));
        } else {
#pragma unroll
            for (int i = 0; i < NPL; ++i) word[i] = order_key(l[i]);
        }
        uint32_t keep = kAll;
        if (p.groups > 1) {
            keep = choose_groups<NPL, V>(p, group_lanes, word, group_best[warp]);
            if (group_lanes > 0) {
                const int shift = __ffs(group_lanes) - 1;
#pragma unroll
                for (int v = 0; v < NPL / V; ++v) {
                    const bool kept = keep >> ((v * 32 + lane) >> shift) & 1u;
#pragma unroll
                    for (int i = 0; i < V; ++i) word[v * V + i] = kept ? word[v * V + i] : 0u;
                }
            } else {
                uint32_t bit[NPL];
                load_shared<NPL, V>(group_bit + e0, bit);
#pragma unroll
                for (int i = 0; i < NPL; ++i) word[i] = (keep & bit[i]) != 0 ? word[i] : 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            word[i] = word[i] > kUnchoosable ? (word[i] & ~1023u) | (uint32_t)(1023 - e0 - value_at<V>(i)) : 0u;
        sort_down<NPL>(word);
        uint32_t mine = 0, last = 0;
        auto pop = [&](uint32_t best) {
            const bool own = word[0] == best;
#pragma unroll
            for (int i = 0; i + 1 < NPL; ++i) word[i] = own ? word[i + 1] : word[i];
            word[NPL - 1] = own ? 0u : word[NPL - 1];
        };
        int count = p.k;
#pragma unroll 4
        for (int j = 0; j < p.k; ++j) {
            last = __reduce_max_sync(kAll, word[0]);     // 0 once nothing is left
            mine = lane == j ? last : mine;
            pop(last);
        }
        if (!exact) {
            for (; count < 32; ++count) {
                const uint32_t next_best = __reduce_max_sync(kAll, word[0]);
                if (next_best == 0 || (next_best ^ last) >= 1024u) break;
                last = next_best;
                mine = lane == count ? next_best : mine;
                pop(next_best);
            }
        }
        int chosen = mine != 0 ? 1023 - (int)(mine & 1023u) : -1;
        if (!exact) {
            const uint32_t before = __shfl_up_sync(kAll, mine, 1);
            const bool close = __any_sync(kAll, lane > 0 && mine != 0 && (mine ^ before) < 1024u);
            if (count == 32 && last != 0 && (__reduce_max_sync(kAll, word[0]) ^ last) < 1024u)
                chosen = choose_exactly<F32>(p, t, keep);       // the stretch goes on
            else if (close)
                chosen = reorder<F32>(p, t, chosen, count);
        }
        const float logit = chosen >= 0 ? load_logit<F32>(p.logits, t * p.ld + chosen) : -INFINITY;
        float lse = 0.f;
        if (sums || p.full_softmax || p.lse != nullptr) {
            // expf, not the fast form, whose error grows with the argument (up to 55 units of 2^-24 measured down to -80): 0 to 3 % of the pass
            float ex[NPL], s = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                ex[i] = expf(l[i] - top);
                s += ex[i];
            }
            s = warp_sum(s);
            lse = top + logf(s);
            if (sums) {
                const float r = 1.f / s;
#pragma unroll
                for (int i = 0; i < NPL; ++i) psum[i] = fmaf(ex[i], r, psum[i]);
                z = fmaf(lse, lse, z);
                ++n_live;
            }
            if (p.lse != nullptr && lane == 0) p.lse[t] = lse;
        }
        float w;
        if (p.full_softmax) {
            w = chosen >= 0 ? expf(logit - lse) : 0.f;
        } else {
            const float m = warp_max(logit);
            w = chosen >= 0 ? expf(logit - m) : 0.f;
            const float s = warp_sum(w);
            w = chosen >= 0 ? w / s : 0.f;
        }
        if (lane < p.k) {
            p.topk_idx[at + lane] = chosen;
            p.topk_w[at + lane] = w;
        }
        if (sums && chosen >= 0) atomicAdd(&hist[chosen], 1u);
    }
    if (!sums) return;
    store_shared<NPL, V>(prob + warp * kRow + e0, psum);
    if (lane == 0) {
        warp_z[warp] = z;
        warp_live[warp] = n_live;
    }
    __syncthreads();
    const int64_t part = (int64_t)blockIdx.x * p.E;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        float s = 0.f;
        for (int w = 0; w < warps; ++w) s += __uint_as_float(prob[w * kRow + e]);
        p.part_prob[part + e] = s;
        p.part_count[part + e] = (int32_t)hist[e];
    }
    if (threadIdx.x == 0) {
        float s = 0.f;
        int n = 0;
        for (int w = 0; w < warps; ++w) {
            s += warp_z[w];
            n += warp_live[w];
        }
        p.part_z[blockIdx.x] = s;
        p.part_live[blockIdx.x] = n;
    }
}

// Adds the runs of sequence blockIdx.y for 32 experts: each warp every
// kSumWarps-th run, then the warps' sums in their order.  The losses need all
// CTAs: those of a single sequence are a cluster if they may be one, and the
// first is handed the others' shares; else the shares go to the workspace and
// the CTA that finishes last adds them up.  (Forward pass of 4,096 tokens, 256
// experts, one sequence: 10.0 us with the cluster, 11.4 without; a cluster for
// each of 3 to 16 sequences costs 0.3 to 0.5 us more than it saves.)  Bound by
// latency: about 3 us from the first kernel's end, of which the runs' loads, all
// of a warp in flight at once, are one round trip.
__host__ __device__ inline bool joins_in_cluster(int S, int E) { return S == 1 && E > 32 && E <= 32 * kSumCluster; }

__global__ void __launch_bounds__(kSumWarps * 32) route_sums_kernel(const __grid_constant__ RouteParams p) {
    __shared__ float fpart[kSumWarps][32];
    __shared__ int ipart[kSumWarps][32];
    __shared__ float share[kSumCluster];
    __shared__ float z_sum;
    __shared__ int live;
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool cluster = joins_in_cluster(p.S, p.E);
    if (cluster) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    pdl_launch_dependents();
    pdl_wait();
    const int s = blockIdx.y, e = blockIdx.x * 32 + lane;
    const int begin = seq_begin(p, s), end = seq_begin(p, s + 1);
    if (threadIdx.x == 0 && blockIdx.x == 0 && p.seq_offsets != nullptr && p.err_flags != nullptr) {
        const int a = p.seq_offsets[s], b = p.seq_offsets[s + 1];
        if (a > b || (s == 0 && a != 0) || (s == p.S - 1 && b != p.T)) atomicOr(p.err_flags, kErrBadSeq);
    }
    const int first = begin / p.chunk + s, runs = end > begin ? (end - 1) / p.chunk + s + 1 - first : 0;
    float prob = 0.f;
    int count = 0;
    if (e < p.E) {
        // kSumRuns at a time, whose loads are in flight together
        const int64_t step = (int64_t)kSumWarps * p.E;
        const float* fp = p.part_prob + (int64_t)(first + warp) * p.E + e;
        const int32_t* ip = p.part_count + (int64_t)(first + warp) * p.E + e;
        for (int r = warp; r < runs; r += kSumRuns * kSumWarps, fp += kSumRuns * step, ip += kSumRuns * step) {
            float f[kSumRuns];
            int n[kSumRuns];
#pragma unroll
            for (int j = 0; j < kSumRuns; ++j) {
                const bool in = r + j * kSumWarps < runs;
                f[j] = in ? fp[j * step] : 0.f;
                n[j] = in ? ip[j * step] : 0;
            }
#pragma unroll
            for (int j = 0; j < kSumRuns; ++j) {
                prob += f[j];
                count += n[j];
            }
        }
    }
    fpart[warp][lane] = prob;
    ipart[warp][lane] = count;
    __syncthreads();
    float loss = 0.f;
    if (warp == 0) {
        prob = 0.f;
        count = 0;
#pragma unroll
        for (int w = 0; w < kSumWarps; ++w) {
            prob += fpart[w][lane];
            count += ipart[w][lane];
        }
        if (e < p.E) {
            p.prob_sums[(int64_t)s * p.E + e] = prob;
            p.counts[(int64_t)s * p.E + e] = count;
        }
        loss = warp_sum((float)count * prob);
        if (!cluster && lane == 0) p.part_loss[(int64_t)s * gridDim.x + blockIdx.x] = loss;
    }
    if (warp == 1 && blockIdx.x == 0) {
        float z = 0.f;
        int n = 0;
        for (int r = lane; r < runs; r += 32) {
            z += p.part_z[first + r];
            n += p.part_live[first + r];
        }
        z = warp_sum(z);
        n = (int)__reduce_add_sync(kAll, (unsigned)n);
        if (lane == 0) {
            z_sum = z;
            live = n;
            p.seq_tokens[s] = n;
            if (!cluster) p.seq_z[s] = z;
        }
    }
    __syncwarp();
    float balance = 0.f, z = 0.f;
    int tokens = 0, seqs = 0;
    if (cluster) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");      // all have started
        if (threadIdx.x == 0) {
            uint32_t to;
            asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_addr(&share[blockIdx.x])));
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(loss) : "memory");
        }
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (blockIdx.x != 0 || warp != 0) return;
        if (live > 0) {
            for (unsigned b = 0; b < gridDim.x; ++b) balance += share[b];
            balance *= (float)p.E / ((float)p.k * (float)live * (float)live);
            z = z_sum;
            tokens = live;
            seqs = 1;
        }
    } else {
        __syncthreads();
        if (threadIdx.x == 0) {
            // released: what the CTA's threads wrote before the barrier goes before the ticket; acquired: the others' sums
            uint32_t ticket;
            asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(ticket) : "l"(p.ticket) : "memory");
            last = ticket == gridDim.x * gridDim.y - 1;
        }
        __syncthreads();
        if (!last || warp != 0) return;
        for (int q = lane; q < p.S; q += 32) {
            const int n = __ldcg(&p.seq_tokens[q]);
            if (n == 0) continue;
            float sum = 0.f;
            for (unsigned b = 0; b < gridDim.x; ++b) sum += __ldcg(&p.part_loss[(int64_t)q * gridDim.x + b]);
            balance += sum * ((float)p.E / ((float)p.k * (float)n * (float)n));
            z += __ldcg(&p.seq_z[q]);
            tokens += n;
            ++seqs;
        }
        balance = warp_sum(balance);
        z = warp_sum(z);
        tokens = (int)__reduce_add_sync(kAll, (unsigned)tokens);
        seqs = (int)__reduce_add_sync(kAll, (unsigned)seqs);
    }
    if (lane == 0) {
        p.losses[0] = seqs > 0 ? p.balance_coef * balance / (float)seqs : 0.f;
        p.losses[1] = tokens > 0 ? p.z_coef * z / (float)tokens : 0.f;
        p.seq_tokens[p.S] = tokens;
        p.seq_tokens[p.S + 1] = seqs;
    }
}

// Gradient, one warp per token: the probabilities are recomputed from the
// logits and lse; what the chosen experts add is scattered through a row of
// shared memory, which stays zero between tokens.  32,768 tokens of 256 fp32
// logits 14.9 us, 4.7 TB/s; 4,096 tokens 3.3 us, latency.
template <int NPL, bool F32>
__global__ void __launch_bounds__(kBackwardWarps * 32) route_backward_kernel(const __grid_constant__ RouteParams p) {
    constexpr int V = wide_values(NPL, F32), kRow = NPL * 32;
    __shared__ __align__(16) uint32_t extra_all[kBackwardWarps * kRow];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e0 = lane * V, left = p.E - e0;
    uint32_t* extra = extra_all + warp * kRow;
#pragma unroll
    for (int i = 0; i < NPL; ++i) extra[i * 32 + lane] = 0;
    __syncwarp();
    pdl_launch_dependents();
    pdl_wait();
    const Run run = find_run(p, blockIdx.x);
    constexpr int kSize = F32 ? 4 : 2;
    const unsigned char* row = static_cast<const unsigned char*>(p.logits) + ((int64_t)first_token(run.begin, warp) * p.ld + e0) * kSize;
    unsigned char* d_row = static_cast<unsigned char*>(p.d_logits) + ((int64_t)first_token(run.begin, warp) * p.E + e0) * kSize;
    RawLogits<NPL, F32> next;
    float next_lse = 0.f, next_w = 0.f, next_dw = 0.f;
    int next_chosen = -1;
    auto fetch = [&](uint32_t t) {      // a token's values are on their way while the one before it is worked on
        if (!in_run(t, run.end)) return;
        next_lse = p.lse[t];
        next.load(row, left, p.wide != 0);
        row += kBackwardWarps * p.ld * kSize;
        if (lane < p.k && p.d_topk_w != nullptr) {
            const int64_t at = (int64_t)t * p.k + lane;
            next_chosen = p.topk_idx[at];
            next_w = p.topk_w[at];
            next_dw = p.d_topk_w[at];
        }
    };
    fetch(first_token(run.begin, warp));
    const int n_s = p.seq_tokens[run.s], n = p.seq_tokens[p.S], seqs = p.seq_tokens[p.S + 1];
    float d_balance = 0.f, d_z = 0.f;
    if (p.d_losses != nullptr && n_s > 0) {
        d_balance = p.d_losses[0] * p.balance_coef / (float)seqs * ((float)p.E / ((float)p.k * (float)n_s * (float)n_s));
        d_z = p.d_losses[1] * 2.f * p.z_coef / (float)n;
    }
    float g[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        g[i] = value_at<V>(i) < left ? d_balance * (float)p.counts[(int64_t)run.s * p.E + e0 + value_at<V>(i)] : 0.f;
    for (uint32_t t = first_token(run.begin, warp); in_run(t, run.end); t = next_token(t, kBackwardWarps)) {
        float l[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) l[i] = next.get(i);
        const float lse = next_lse;
        const int chosen = next_chosen >= 0 && next_chosen < p.E ? next_chosen : -1;
        const float w = chosen >= 0 ? next_w : 0.f;
        float dw = chosen >= 0 ? next_dw : 0.f;
        fetch(next_token(t, kBackwardWarps));
        float d[NPL];
        if (lse == -INFINITY) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) d[i] = 0.f;
        } else {
            if (!p.full_softmax) dw = w * (dw - warp_sum(w * dw));
            if (chosen >= 0) extra[chosen] = __float_as_uint(dw);
            __syncwarp();
            float pr[NPL], dot = 0.f;
            uint32_t ex[NPL];
            load_shared<NPL, V>(extra + e0, ex);
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                pr[i] = expf(l[i] - lse);
                d[i] = __uint_as_float(ex[i]);
                dot = fmaf(pr[i], p.full_softmax ? g[i] + d[i] : g[i], dot);
            }
            dot = warp_sum(dot) - d_z * lse;
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                d[i] = p.full_softmax ? pr[i] * (g[i] + d[i] - dot) : fmaf(pr[i], g[i] - dot, d[i]);
            __syncwarp();
            if (chosen >= 0) extra[chosen] = 0;
            __syncwarp();
        }
        store_values<NPL, F32>(d_row, left, p.wide != 0, d);
        d_row += (int64_t)kBackwardWarps * p.E * kSize;
    }
}

// Experts of a lane.
int lane_values(int E) { return E <= 64 ? 2 : E <= 128 ? 4 : E <= 256 ? 8 : E <= 512 ? 16 : 32; }

// Can the rows be read, or written, by wide accesses?
bool wide_rows(const RouteParams& p, const void* base, int64_t ld) {
    const int values = wide_values(lane_values(p.E), p.f32 != 0), bytes = values * (p.f32 ? 4 : 2);
    return p.E % values == 0 && ld % values == 0 && reinterpret_cast<uintptr_t>(base) % bytes == 0;
}

template <int NPL, bool F32>
cudaError_t launch_choice(const RouteParams& p, dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(route_kernel<NPL, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(true, route_kernel<NPL, F32>, grid, block, smem, stream, p);
}

template <bool F32>
cudaError_t launch_forward(const RouteParams& p, dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
    if (p.E <= 64) return launch_choice<2, F32>(p, grid, block, smem, stream);
    if (p.E <= 128) return launch_choice<4, F32>(p, grid, block, smem, stream);
    if (p.E <= 256) return launch_choice<8, F32>(p, grid, block, smem, stream);
    if (p.E <= 512) return launch_choice<16, F32>(p, grid, block, smem, stream);
    return launch_choice<32, F32>(p, grid, block, smem, stream);
}

template <bool F32>
cudaError_t launch_gradient(const RouteParams& p, dim3 grid, cudaStream_t stream) {
    const dim3 block(kBackwardWarps * 32);
    if (p.E <= 64) return launch_kernel(true, route_backward_kernel<2, F32>, grid, block, 0, stream, p);
    if (p.E <= 128) return launch_kernel(true, route_backward_kernel<4, F32>, grid, block, 0, stream, p);
    if (p.E <= 256) return launch_kernel(true, route_backward_kernel<8, F32>, grid, block, 0, stream, p);
    if (p.E <= 512) return launch_kernel(true, route_backward_kernel<16, F32>, grid, block, 0, stream, p);
    return launch_kernel(true, route_backward_kernel<32, F32>, grid, block, 0, stream, p);
}

}  // namespace

size_t route_workspace(RouteParams* p, void* base) {
    const size_t runs = (size_t)std::max<int64_t>(num_runs(p->T, run_tokens(p->T), p->S), 1);
    const size_t blocks = (size_t)(p->E + 31) / 32;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        unsigned char* q = base != nullptr ? static_cast<unsigned char*>(base) + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return q;
    };
    p->part_prob = reinterpret_cast<float*>(take(runs * p->E * 4));
    p->part_count = reinterpret_cast<int32_t*>(take(runs * p->E * 4));
    p->part_z = reinterpret_cast<float*>(take(runs * 4));
    p->part_live = reinterpret_cast<int32_t*>(take(runs * 4));
    p->part_loss = reinterpret_cast<float*>(take((size_t)p->S * blocks * 4));
    p->seq_z = reinterpret_cast<float*>(take((size_t)p->S * 4));
    p->ticket = reinterpret_cast<uint32_t*>(take(4));
    return at;
}

cudaError_t launch_route(const RouteParams& in, int num_sms, cudaStream_t stream) {
    RouteParams p = in;
    const bool sums = p.losses != nullptr;
    p.per_group = p.E / p.groups;
    if (!sums) {
        p.seq_offsets = nullptr;
        p.S = 1;
    }
    // of a CTA that only chooses (32,768 tokens: 256 experts 23.7 us with 4, 22.0 with 8; 512 experts in groups 20.3 and 22.0)
    const int choice_warps = p.E <= 256 ? 8 : 4;
    const int warps = sums ? kRunWarps : choice_warps;
    // one token a warp until there are 8 CTAs for every SM (32,768 tokens of 256 fp32 logits: 25.3 us one by one, 22.0 so)
    p.chunk = sums ? run_tokens(p.T) : choice_warps * std::min(std::max(p.T / (choice_warps * 8 * num_sms), 1), kChoiceTokens);
    const dim3 grid((unsigned)std::max<int64_t>(num_runs(p.T, p.chunk, p.S), 1)), block(warps * 32);
    const size_t smem = (size_t)(3 + (sums ? kRunWarps : 0)) * lane_values(p.E) * 32 * 4;
    p.wide = wide_rows(p, p.logits, p.ld);
    cudaError_t e = p.f32 ? launch_forward<true>(p, grid, block, smem, stream) : launch_forward<false>(p, grid, block, smem, stream);
    if (e != cudaSuccess || !sums) return e;
    const int ctas = (p.E + 31) / 32;
    return launch_clusters(true, joins_in_cluster(p.S, p.E) ? ctas : 1, route_sums_kernel, dim3(ctas, p.S), dim3(kSumWarps * 32), 0,
                           stream, p);
}

cudaError_t launch_route_backward(const RouteParams& in, int num_sms, cudaStream_t stream) {
    RouteParams p = in;
    // A wave of CTAs, as the registers hold them, up to 4 tokens a warp: a token's loads come behind the work on the one
    // before (us with 1, 2, 3 and 4: 4,096 tokens of 256 fp32 logits 3.3, 4.4, 5.4, 6.1; 32,768 19.8, 16.1, 15.6, 14.9;
    // 16,384 of 128 bf16 6.6, 5.5, 5.2, 6.3; 8,192 of 512 fp32 11.8, 9.5, 10.5, 8.2).
    const int wave = kBackwardWarps * num_sms * (p.E <= 128 ? 6 : p.E <= 256 ? 4 : p.E <= 512 ? 2 : 1);
    p.chunk = kBackwardWarps * std::min((p.T - 1) / wave + 1, kBackwardTokens);
    const dim3 grid((unsigned)num_runs(p.T, p.chunk, p.S));
    p.wide = wide_rows(p, p.logits, p.ld) && wide_rows(p, p.d_logits, p.E);
    return p.f32 ? launch_gradient<true>(p, grid, stream) : launch_gradient<false>(p, grid, stream);
}

}  // namespace ep
