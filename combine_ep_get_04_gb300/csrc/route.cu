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

constexpr int kRouteWarps = 8;
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
    int lo = 0, hi = p.S - 1;
    if (p.seq_offsets != nullptr) {
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

template <int NPL, bool F32>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteParams p) {
    extern __shared__ unsigned char smem[];   // [E] copies, then [warps][E] probabilities
    __shared__ uint32_t group_best[kRouteWarps][32];
    __shared__ float warp_z[kRouteWarps];
    __shared__ int warp_live[kRouteWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t* hist = reinterpret_cast<int32_t*>(smem);
    float* prob = reinterpret_cast<float*>(smem) + p.E;
    const bool sums = p.losses != nullptr;
    const int per = p.E / p.groups;
    if (sums)
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
    pdl_launch_dependents();
    pdl_wait();
    if (sums && blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
    const Run run = find_run(p, blockIdx.x);
    if (sums) __syncthreads();
    float psum[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) psum[i] = 0.f;
    float z = 0.f;
    int n_live = 0;
    for (int t = run.begin + warp; t < run.end; t += kRouteWarps) {
        float l[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 32 + lane;
            l[i] = e < p.E ? load_logit<F32>(p.logits, t * p.ld + e) : -INFINITY;
        }
        bool some = false;
#pragma unroll
        for (int i = 0; i < NPL; ++i) some |= l[i] > -INFINITY;
        const bool live = (p.token_mask == nullptr || p.token_mask[t] != 0) && __any_sync(kAll, some);
        const int64_t at = (int64_t)t * p.k;
        if (!live) {
            if (lane < p.k) {
                p.topk_idx[at + lane] = -1;
                p.topk_w[at + lane] = 0.f;
            }
            if (p.lse != nullptr && lane == 0) p.lse[t] = -INFINITY;
            continue;
        }
        uint32_t key[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 32 + lane;
            key[i] = order_key(e < p.E && p.select_bias != nullptr ? __fadd_rn(l[i], p.select_bias[e]) : l[i]);
        }
        if (p.groups > 1) {
            uint32_t* best = group_best[warp];
            best[lane] = 0;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (i * 32 + lane < p.E) atomicMax(&best[(i * 32 + lane) / per], key[i]);
            __syncwarp();
            uint32_t mine = lane < p.groups ? best[lane] : 0u;
            uint32_t keep = 0;
            for (int r = 0; r < p.topk_groups; ++r) {
                const uint32_t top = __reduce_max_sync(kAll, mine);
                if (top <= kUnchoosable) break;
                const int g = __ffs(__ballot_sync(kAll, mine == top)) - 1;
                keep |= 1u << g;
                if (lane == g) mine = 0;
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const int e = i * 32 + lane;
                if (e < p.E && !(keep >> (e / per) & 1u)) key[i] = 0;
            }
        }
        // lane j ends up with the expert of place j and its logit
        int chosen = -1;
        float logit = -INFINITY;
        for (int j = 0; j < p.k; ++j) {
            uint32_t top = 0;
            int at_i = 0;
            float top_l = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (key[i] > top) {
                    top = key[i];
                    at_i = i;
                    top_l = l[i];
                }
            const uint32_t best = __reduce_max_sync(kAll, top);
            if (best <= kUnchoosable) break;
            const int e = (int)__reduce_min_sync(kAll, top == best ? (uint32_t)(at_i * 32 + lane) : kAll);
            const float x = __shfl_sync(kAll, top_l, e & 31);
            if (lane == j) {
                chosen = e;
                logit = x;
            }
            if (lane == (e & 31)) {
#pragma unroll
                for (int i = 0; i < NPL; ++i)
                    if (i == e >> 5) key[i] = 0;
            }
        }
        float lse = 0.f;
        if (sums || p.full_softmax || p.lse != nullptr) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < NPL; ++i) m = fmaxf(m, l[i]);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, d));
            float ex[NPL], s = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                ex[i] = __expf(l[i] - m);
                s += ex[i];
            }
            s = warp_sum(s);
            lse = m + logf(s);
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
            float m = logit;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, d));
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
#pragma unroll
        for (int w = 0; w < kRouteWarps; ++w) s += prob[w * p.E + e];
        p.part_prob[row + e] = s;
        p.part_count[row + e] = hist[e];
    }
    if (threadIdx.x == 0) {
        float s = 0.f;
        int n = 0;
        for (int w = 0; w < kRouteWarps; ++w) {
            s += warp_z[w];
            n += warp_live[w];
        }
        p.part_z[blockIdx.x] = s;
        p.part_live[blockIdx.x] = n;
    }
}

// Adds the runs of sequence blockIdx.y for 32 experts; the CTA that finishes
// last adds up the losses.
__global__ void __launch_bounds__(256) route_sums_kernel(RouteParams p) {
    __shared__ float fpart[8][32];
    __shared__ int ipart[8][32];
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
    if (e < p.E)
        for (int r = warp; r < runs; r += 8) {
            prob += p.part_prob[(int64_t)(first + r) * p.E + e];
            count += p.part_count[(int64_t)(first + r) * p.E + e];
        }
    fpart[warp][lane] = prob;
    ipart[warp][lane] = count;
    __syncthreads();
    if (warp == 0) {
        prob = 0.f;
        count = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
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
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(p.ticket, 1u) == gridDim.x * gridDim.y - 1;
    __syncthreads();
    if (!last || warp != 0) return;
    __threadfence();
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
__global__ void __launch_bounds__(kRouteWarps * 32) route_backward_kernel(RouteParams p) {
    extern __shared__ float extra_all[];      // [warps][E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* extra = extra_all + warp * p.E;
    for (int e = lane; e < p.E; e += 32) extra[e] = 0.f;
    __syncwarp();
    pdl_launch_dependents();
    pdl_wait();
    const Run run = find_run(p, blockIdx.x);
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
    for (int t = run.begin + warp; t < run.end; t += kRouteWarps) {
        const float lse = p.lse[t];
        const bool live = lse != -INFINITY;
        float d[NPL];
        if (!live) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) d[i] = 0.f;
        } else {
            int chosen = -1;
            float w = 0.f, dw = 0.f;
            if (lane < p.k && p.d_topk_w != nullptr) {
                const int64_t at = (int64_t)t * p.k + lane;
                chosen = p.topk_idx[at];
                if (chosen < 0 || chosen >= p.E) chosen = -1;
                if (chosen >= 0) {
                    w = p.topk_w[at];
                    dw = p.d_topk_w[at];
                }
            }
            if (!p.full_softmax) dw = w * (dw - warp_sum(w * dw));
            if (chosen >= 0) extra[chosen] = dw;
            __syncwarp();
            float pr[NPL], dot = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const int e = i * 32 + lane;
                pr[i] = e < p.E ? __expf(load_logit<F32>(p.logits, t * p.ld + e) - lse) : 0.f;
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

// Tokens a CTA takes: one for each warp until there are four CTAs for every
// SM, then more, so that the per-run sums stay small beside the logits.
int run_tokens(int T) {
    const int per = T / (kRouteWarps * 608);
    return kRouteWarps * std::min(std::max(per, 1), 16);
}

int64_t num_runs(int T, int chunk, int S) { return ((int64_t)T + chunk - 1) / chunk + S - 1; }

template <bool F32>
cudaError_t launch_forward(const RouteParams& p, dim3 grid, size_t smem, cudaStream_t stream) {
    const dim3 block(kRouteWarps * 32);
    if (p.E <= 64) return launch_kernel(true, route_kernel<2, F32>, grid, block, smem, stream, p);
    if (p.E <= 128) return launch_kernel(true, route_kernel<4, F32>, grid, block, smem, stream, p);
    if (p.E <= 256) return launch_kernel(true, route_kernel<8, F32>, grid, block, smem, stream, p);
    if (p.E <= 512) return launch_kernel(true, route_kernel<16, F32>, grid, block, smem, stream, p);
    return launch_kernel(true, route_kernel<32, F32>, grid, block, smem, stream, p);
}

template <bool F32>
cudaError_t launch_gradient(const RouteParams& p, dim3 grid, size_t smem, cudaStream_t stream) {
    const dim3 block(kRouteWarps * 32);
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
    (void)num_sms;
    RouteParams p = in;
    const bool sums = p.losses != nullptr;
    if (!sums) {
        p.seq_offsets = nullptr;
        p.S = 1;
    }
    p.chunk = run_tokens(p.T);
    const dim3 grid((unsigned)std::max<int64_t>(num_runs(p.T, p.chunk, p.S), 1));
    const size_t smem = sums ? (size_t)(1 + kRouteWarps) * p.E * 4 : 0;
    cudaError_t e = p.f32 ? launch_forward<true>(p, grid, smem, stream) : launch_forward<false>(p, grid, smem, stream);
    if (e != cudaSuccess || !sums) return e;
    return launch_kernel(true, route_sums_kernel, dim3((p.E + 31) / 32, p.S), dim3(256), 0, stream, p);
}

cudaError_t launch_route_backward(const RouteParams& in, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    RouteParams p = in;
    p.chunk = run_tokens(p.T);
    const dim3 grid((unsigned)num_runs(p.T, p.chunk, p.S));
    const size_t smem = (size_t)kRouteWarps * p.E * 4;
    return p.f32 ? launch_gradient<true>(p, grid, smem, stream) : launch_gradient<false>(p, grid, smem, stream);
}

}  // namespace ep
