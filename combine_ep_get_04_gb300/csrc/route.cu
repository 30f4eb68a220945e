// route.cu -- the choice of experts from router logits, per-expert counts,
// the balance and z losses, and the gradient of all of it.
//
// One warp per token, the token's logits in registers (lane l holds experts
// l, l + 32, ...).  The choice compares 32-bit keys whose unsigned order is
// that of the floats, so a maximum over the warp is one redux.sync.  What is
// summed over tokens (probabilities, copies, squared log normalisers) is
// summed per run of tokens of one sequence by one CTA and then over the runs in
// their order, so the losses do not depend on which CTA runs first.
#include <algorithm>
#include <cuda_bf16.h>

#include "ep_device.cuh"
#include "ep_kernels.h"

namespace ep {
namespace {

constexpr int kMaxRouteWarps = 16;
constexpr int kRunWarps = 16;          // of a CTA that sums its run
constexpr int kChoiceWarps = 4;        // of a CTA that only chooses: more of them, on more SMs
constexpr int kChoiceTokens = 8;       // most tokens of its warps
constexpr int kBackwardWarps = 8;
constexpr int kBackwardTokens = 2;     // a warp's, in the backward pass: the second's loads overlap the first
constexpr int kSumWarps = 32;
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

// The largest of each group's keys -> the groups a token may choose from, as
// a mask.  `best` is a row of 32 words of shared memory.
template <int NPL>
__device__ __forceinline__ uint32_t choose_groups(const RouteParams& p, int per, const uint32_t (&key)[NPL], uint32_t* best) {
    const int lane = threadIdx.x & 31;
    if ((per & (per - 1)) == 0) {
        // a power of two: maxima over the lanes of a group, or over a lane's values and the warp
        const int shift = 31 - __clz(per);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            uint32_t m = key[i];
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1)
                if (d < per) m = max(m, __shfl_xor_sync(kAll, m, d));
            const int e = i * 32 + lane;
            if (e < p.E && (lane & (per - 1)) == 0) {
                if (per <= 32 || (i * 32 & (per - 1)) == 0)
                    best[e >> shift] = m;
                else
                    best[e >> shift] = max(best[e >> shift], m);      // the same lane, 0, writes all parts of a group
            }
        }
    } else {
        best[lane] = 0;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (i * 32 + lane < p.E) atomicMax(&best[(i * 32 + lane) / per], key[i]);
    }
    __syncwarp();
    // a group stays if fewer than topk_groups come before it
    const uint32_t mine = lane < p.groups ? best[lane] : 0u;
    int before = 0;
#pragma unroll 4
    for (int g = 0; g < p.groups; ++g) {
        const uint32_t other = best[g];
        before += other > mine || (other == mine && g < lane) ? 1 : 0;
    }
    const uint32_t keep = __ballot_sync(kAll, mine > kUnchoosable && before < p.topk_groups);
    __syncwarp();
    return keep;
}

// The choice by whole keys, for tokens whose best keys agree in their upper 22
// bits: every round looks for the next pair (key, index) in memory.  Returns
// lane j's expert, or -1.
template <bool F32>
__device__ __noinline__ int choose_exactly(const RouteParams& p, int t, int per, uint32_t keep) {
    const int lane = threadIdx.x & 31;
    uint32_t last = kAll;
    int last_e = -1, chosen = -1;
    for (int j = 0; j < p.k; ++j) {
        uint32_t top = 0;
        int top_e = 0;
        for (int e = lane; e < p.E; e += 32) {
            if (p.groups > 1 && !(keep >> (e / per) & 1u)) continue;
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
__device__ __forceinline__ int reorder(const RouteParams& p, int t, int e, int count) {
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
template <int NPL, bool F32>
__global__ void __launch_bounds__(kMaxRouteWarps * 32, NPL <= 8 ? 2 : 1) route_kernel(const __grid_constant__ RouteParams p) {
    extern __shared__ unsigned char smem[];   // [E] copies, [E] group bits, then [warps][E] probabilities
    __shared__ uint32_t group_best[kMaxRouteWarps][32];
    __shared__ float warp_z[kMaxRouteWarps];
    __shared__ int warp_live[kMaxRouteWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int32_t* hist = reinterpret_cast<int32_t*>(smem);
    uint32_t* group_bit = reinterpret_cast<uint32_t*>(smem) + p.E;
    float* prob = reinterpret_cast<float*>(smem) + 2 * p.E;
    const bool sums = p.losses != nullptr, exact = !F32 && p.select_bias == nullptr;
    const int per = p.per_group;
    if (sums)
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
    if (p.groups > 1)
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) group_bit[e] = 1u << (e / per);
    pdl_launch_dependents();
    pdl_wait();
    if (sums && blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
    const Run run = find_run(p, blockIdx.x);
    __syncthreads();
    float psum[NPL], next[NPL];
    bool next_mask = true;
    auto fetch = [&](int t) {      // a token's logits are on their way while the one before it is worked on
        if (t >= run.end) return;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 32 + lane;
            next[i] = e < p.E ? load_logit<F32>(p.logits, t * p.ld + e) : -INFINITY;
        }
        next_mask = p.token_mask == nullptr || p.token_mask[t] != 0;
    };
#pragma unroll
    for (int i = 0; i < NPL; ++i) psum[i] = 0.f;
    float z = 0.f;
    int n_live = 0;
    fetch(run.begin + warp);
    for (int t = run.begin + warp; t < run.end; t += warps) {
        float l[NPL], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            l[i] = next[i];
            top = fmaxf(top, l[i]);
        }
        const bool mask = next_mask;
        fetch(t + warps);
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
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 32 + lane;
            word[i] = order_key(p.select_bias != nullptr && e < p.E ? __fadd_rn(l[i], p.select_bias[e]) : l[i]);
        }
        uint32_t keep = kAll;
        if (p.groups > 1) keep = choose_groups<NPL>(p, per, word, group_best[warp]);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 32 + lane;
            const bool may = word[i] > kUnchoosable && (p.groups == 1 || (e < p.E && (keep & group_bit[e]) != 0));
            word[i] = may ? (word[i] & ~1023u) | (1023u - e) : 0u;
        }
        sort_down<NPL>(word);
        uint32_t mine = 0, last = 0;
        bool close = false;
        auto pop = [&](uint32_t best) {
            const bool own = word[0] == best;
#pragma unroll
            for (int i = 0; i + 1 < NPL; ++i) word[i] = own ? word[i + 1] : word[i];
            word[NPL - 1] = own ? 0u : word[NPL - 1];
        };
        int count = p.k;
#pragma unroll 4
        for (int j = 0; j < p.k; ++j) {
            const uint32_t best = __reduce_max_sync(kAll, word[0]);     // 0 once nothing is left
            close |= best != 0 && (best ^ last) < 1024u;
            last = best;
            mine = lane == j ? best : mine;
            pop(best);
        }
        if (!exact) {
            for (; count < 32; ++count) {
                const uint32_t next_best = __reduce_max_sync(kAll, word[0]);
                if (next_best == 0 || (next_best ^ last) >= 1024u) break;
                close = true;
                last = next_best;
                mine = lane == count ? next_best : mine;
                pop(next_best);
            }
        }
        int chosen = mine != 0 ? 1023 - (int)(mine & 1023u) : -1;
        if (!exact && count == 32 && last != 0 && (__reduce_max_sync(kAll, word[0]) ^ last) < 1024u)
            chosen = choose_exactly<F32>(p, t, per, keep);       // the stretch goes on
        else if (!exact && close)
            chosen = reorder<F32>(p, t, chosen, count);
        else if (lane >= p.k)
            chosen = -1;
        const float logit = chosen >= 0 ? load_logit<F32>(p.logits, t * p.ld + chosen) : -INFINITY;
        float lse = 0.f;
        if (sums || p.full_softmax || p.lse != nullptr) {
            float ex[NPL], s = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                ex[i] = __expf(l[i] - top);
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
        if (sums && chosen >= 0) atomicAdd(&hist[chosen], 1);
    }
    if (!sums) return;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        if (i * 32 + lane < p.E) prob[warp * p.E + i * 32 + lane] = psum[i];
    if (lane == 0) {
        warp_z[warp] = z;
        warp_live[warp] = n_live;
    }
    __syncthreads();
    const int64_t row = (int64_t)blockIdx.x * p.E;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        float s = 0.f;
        for (int w = 0; w < warps; ++w) s += prob[w * p.E + e];
        p.part_prob[row + e] = s;
        p.part_count[row + e] = hist[e];
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
// kSumWarps-th run, then the warps' sums in their order.  The CTA that finishes
// last adds up the losses.
__global__ void __launch_bounds__(kSumWarps * 32) route_sums_kernel(RouteParams p) {
    __shared__ float fpart[kSumWarps][32];
    __shared__ int ipart[kSumWarps][32];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
        const float* fp = p.part_prob + (int64_t)first * p.E + e;
        const int32_t* ip = p.part_count + (int64_t)first * p.E + e;
#pragma unroll 8
        for (int r = warp; r < runs; r += kSumWarps) {
            prob += fp[(int64_t)r * p.E];
            count += ip[(int64_t)r * p.E];
        }
    }
    fpart[warp][lane] = prob;
    ipart[warp][lane] = count;
    __syncthreads();
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
        const float loss = warp_sum((float)count * prob);
        if (lane == 0) p.part_loss[(int64_t)s * gridDim.x + blockIdx.x] = loss;
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
            p.seq_z[s] = z;
            p.seq_tokens[s] = n;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();       // what the CTA's threads wrote before the barrier goes before the ticket
        last = atomicAdd(p.ticket, 1u) == gridDim.x * gridDim.y - 1;
        __threadfence();
    }
    __syncthreads();
    if (!last || warp != 0) return;
    float balance = 0.f, z = 0.f;
    int tokens = 0, seqs = 0;
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
    if (lane == 0) {
        p.losses[0] = seqs > 0 ? p.balance_coef * balance / (float)seqs : 0.f;
        p.losses[1] = tokens > 0 ? p.z_coef * z / (float)tokens : 0.f;
        p.seq_tokens[p.S] = tokens;
        p.seq_tokens[p.S + 1] = seqs;
    }
}

// Gradient, one warp per token: the probabilities are recomputed from the
// logits and lse; what the chosen experts add is scattered through a row of
// shared memory, which stays zero between tokens.
template <int NPL, bool F32>
__global__ void __launch_bounds__(kBackwardWarps * 32) route_backward_kernel(RouteParams p) {
    extern __shared__ float extra_all[];      // [warps][E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* extra = extra_all + warp * p.E;
    for (int e = lane; e < p.E; e += 32) extra[e] = 0.f;
    __syncwarp();
    pdl_launch_dependents();
    pdl_wait();
    const Run run = find_run(p, blockIdx.x);
    float next[NPL], next_lse = 0.f, next_w = 0.f, next_dw = 0.f;
    int next_chosen = -1;
    auto fetch = [&](int t) {      // a token's values are on their way while the one before it is worked on
        if (t >= run.end) return;
        next_lse = p.lse[t];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 32 + lane;
            next[i] = e < p.E ? load_logit<F32>(p.logits, t * p.ld + e) : -INFINITY;
        }
        if (lane < p.k && p.d_topk_w != nullptr) {
            const int64_t at = (int64_t)t * p.k + lane;
            next_chosen = p.topk_idx[at];
            next_w = p.topk_w[at];
            next_dw = p.d_topk_w[at];
        }
    };
    fetch(run.begin + warp);
    const int n_s = p.seq_tokens[run.s], n = p.seq_tokens[p.S], seqs = p.seq_tokens[p.S + 1];
    float d_balance = 0.f, d_z = 0.f;
    if (p.d_losses != nullptr && n_s > 0) {
        d_balance = p.d_losses[0] * p.balance_coef / (float)seqs * ((float)p.E / ((float)p.k * (float)n_s * (float)n_s));
        d_z = p.d_losses[1] * 2.f * p.z_coef / (float)n;
    }
    float g[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 32 + lane;
        g[i] = e < p.E ? d_balance * (float)p.counts[(int64_t)run.s * p.E + e] : 0.f;
    }
    for (int t = run.begin + warp; t < run.end; t += kBackwardWarps) {
        float l[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) l[i] = next[i];
        const float lse = next_lse;
        const int chosen = next_chosen >= 0 && next_chosen < p.E ? next_chosen : -1;
        const float w = chosen >= 0 ? next_w : 0.f;
        float dw = chosen >= 0 ? next_dw : 0.f;
        fetch(t + kBackwardWarps);
        float d[NPL];
        if (lse == -INFINITY) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) d[i] = 0.f;
        } else {
            if (!p.full_softmax) dw = w * (dw - warp_sum(w * dw));
            if (chosen >= 0) extra[chosen] = dw;
            __syncwarp();
            float pr[NPL], dot = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const int e = i * 32 + lane;
                pr[i] = __expf(l[i] - lse);
                d[i] = e < p.E ? extra[e] : 0.f;
                dot = fmaf(pr[i], p.full_softmax ? g[i] + d[i] : g[i], dot);
            }
            dot = warp_sum(dot) - d_z * lse;
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                d[i] = p.full_softmax ? pr[i] * (g[i] + d[i] - dot) : fmaf(pr[i], g[i] - dot, d[i]);
            __syncwarp();
            if (chosen >= 0) extra[chosen] = 0.f;
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 32 + lane;
            if (e >= p.E) continue;
            if (F32)
                static_cast<float*>(p.d_logits)[(int64_t)t * p.E + e] = d[i];
            else
                static_cast<__nv_bfloat16*>(p.d_logits)[(int64_t)t * p.E + e] = __float2bfloat16_rn(d[i]);
        }
    }
}

// Tokens of a run: one for each warp until there are two CTAs for every SM,
// then more, so that the per-run sums stay small beside the logits.
int run_tokens(int T) {
    const int per = (T + kRunWarps * 304 - 1) / (kRunWarps * 304);
    return kRunWarps * std::min(std::max(per, 1), 16);
}

int64_t num_runs(int T, int chunk, int S) { return ((int64_t)T + chunk - 1) / chunk + S - 1; }

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
cudaError_t launch_gradient(const RouteParams& p, dim3 grid, size_t smem, cudaStream_t stream) {
    const dim3 block(kBackwardWarps * 32);
    if (p.E <= 64) return launch_kernel(true, route_backward_kernel<2, F32>, grid, block, smem, stream, p);
    if (p.E <= 128) return launch_kernel(true, route_backward_kernel<4, F32>, grid, block, smem, stream, p);
    if (p.E <= 256) return launch_kernel(true, route_backward_kernel<8, F32>, grid, block, smem, stream, p);
    if (p.E <= 512) return launch_kernel(true, route_backward_kernel<16, F32>, grid, block, smem, stream, p);
    return launch_kernel(true, route_backward_kernel<32, F32>, grid, block, smem, stream, p);
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
    const int warps = sums ? kRunWarps : kChoiceWarps;
    // one token a warp until there are 8 CTAs for every SM
    p.chunk = sums ? run_tokens(p.T) : kChoiceWarps * std::min(std::max(p.T / (kChoiceWarps * 8 * num_sms), 1), kChoiceTokens);
    const dim3 grid((unsigned)std::max<int64_t>(num_runs(p.T, p.chunk, p.S), 1)), block(warps * 32);
    const size_t smem = (size_t)(2 + (sums ? kRunWarps : 0)) * p.E * 4;
    cudaError_t e = p.f32 ? launch_forward<true>(p, grid, block, smem, stream) : launch_forward<false>(p, grid, block, smem, stream);
    if (e != cudaSuccess || !sums) return e;
    return launch_kernel(true, route_sums_kernel, dim3((p.E + 31) / 32, p.S), dim3(kSumWarps * 32), 0, stream, p);
}

cudaError_t launch_route_backward(const RouteParams& in, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    RouteParams p = in;
    p.chunk = kBackwardWarps * kBackwardTokens;
    const dim3 grid((unsigned)num_runs(p.T, p.chunk, p.S));
    const size_t smem = (size_t)kBackwardWarps * p.E * 4;
    return p.f32 ? launch_gradient<true>(p, grid, smem, stream) : launch_gradient<false>(p, grid, smem, stream);
}

}  // namespace ep
