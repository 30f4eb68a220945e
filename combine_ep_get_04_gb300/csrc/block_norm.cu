// block_norm.cu -- the end of one block and the start of the next:
//   u = y * r1 * w_post,  h_out = res_scale * h + gate * u,  n = h_out * r2 * w_pre
// with r = 1 / sqrt(mean square + eps), and its gradients.  One pass over the
// rows in each direction; every value in between stays in registers, so the
// kernels read and write each tensor once and are bound by HBM.
#include <algorithm>

#include "ep_device.cuh"
#include "ep_kernels.h"

namespace ep {
namespace {

constexpr int kGateChannel = 1;
constexpr int kGateToken = 2;
constexpr int kVec = 8;   // channels a thread handles at once: 16 bytes of bf16

struct Vec8 {
    float v[kVec];
};

__device__ __forceinline__ Vec8 load_bf16(const void* base, int64_t at) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(base) + at * 2);
    return Vec8{{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y), bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w),
                 bf16_hi(w.w)}};
}

__device__ __forceinline__ Vec8 load_f32(const void* base, int64_t at) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

__device__ __forceinline__ void store_bf16(void* base, int64_t at, const Vec8& x) {
    uint4 w;
    w.x = pack_bf16x2(x.v[0], x.v[1]);
    w.y = pack_bf16x2(x.v[2], x.v[3]);
    w.z = pack_bf16x2(x.v[4], x.v[5]);
    w.w = pack_bf16x2(x.v[6], x.v[7]);
    *reinterpret_cast<uint4*>(static_cast<unsigned char*>(base) + at * 2) = w;
}

__device__ __forceinline__ void store_f32(void* base, int64_t at, const Vec8& x) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
    p[1] = make_float4(x.v[4], x.v[5], x.v[6], x.v[7]);
}

template <bool F32>
__device__ __forceinline__ Vec8 load_stream(const void* base, int64_t at) {
    return F32 ? load_f32(base, at) : load_bf16(base, at);
}

template <bool F32>
__device__ __forceinline__ void store_stream(void* base, int64_t at, const Vec8& x) {
    if (F32)
        store_f32(base, at, x);
    else
        store_bf16(base, at, x);
}

__device__ __forceinline__ Vec8 zeros() { return Vec8{{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}}; }
__device__ __forceinline__ Vec8 ones() { return Vec8{{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}}; }

// Sum over the `warps` warps of one row.  `red` holds one float for each warp
// of the CTA; every thread of the CTA takes part.  One barrier: a caller that
// sums twice uses two arrays in turn.
__device__ __forceinline__ float row_sum(float x, float* red, int warps) {
    x = warp_sum(x);
    if (warps == 1) return x;
    const int warp = threadIdx.x >> 5, first = warp - warp % warps;
    if ((threadIdx.x & 31) == 0) red[warp] = x;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += red[first + i];
    return s;
}

// Threads of a row hold NV vectors of 8 channels each, `lanes` threads apart.
struct RowShape {
    int warps;   // warps a row
    int rows;    // rows a CTA works on at once
};

RowShape row_shape(int H, int nv, int least_warps) {
    const int vecs = H / kVec;
    RowShape r;
    r.warps = (vecs + nv * 32 - 1) / (nv * 32);
    r.rows = std::max(1, least_warps / r.warps);
    return r;
}

// Forward.  A row's h and y stay in registers between its two norms: the mean
// square of y, then that of h_out, one barrier each (none where a row fits a
// warp).
template <int NV, bool F32>
__global__ void __launch_bounds__(1024) norm_kernel(NormParams p, RowShape shape) {
    __shared__ float red1[32], red2[32];
    pdl_launch_dependents();
    pdl_wait();
    const int lanes = shape.warps * 32;
    const int sub = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int64_t t = (int64_t)blockIdx.x * shape.rows + sub;
    const bool live = t < p.T;
    const int vecs = p.H / kVec;
    Vec8 h[NV], y[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lane + i * lanes;
        const bool in = live && v < vecs;
        h[i] = in ? load_stream<F32>(p.h, t * p.ld_h + v * kVec) : zeros();
        y[i] = in && p.y != nullptr ? load_bf16(p.y, t * p.ld_y + v * kVec) : zeros();
    }
    const float scale = p.res_scale != nullptr ? *p.res_scale : 1.f;
    const float token_gate = p.gate_kind == kGateToken && live ? p.gate[t] : 1.f;
    float r1 = 1.f;
    if (p.w_post != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int c = 0; c < kVec; ++c) ss = fmaf(y[i].v[c], y[i].v[c], ss);
        r1 = rsqrtf(row_sum(ss, red1, shape.warps) / (float)p.H + p.eps);
        if (live && lane == 0 && p.rstd != nullptr) p.rstd[t] = r1;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lane + i * lanes;
        if (!live || v >= vecs) continue;
        const Vec8 w = p.w_post != nullptr ? load_f32(p.w_post, v * kVec) : ones();
        const Vec8 g = p.gate_kind == kGateChannel ? load_f32(p.gate, v * kVec) : ones();
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            const float u = y[i].v[c] * r1 * w.v[c];
            h[i].v[c] = fmaf(scale, h[i].v[c], token_gate * g.v[c] * u);
            ss = fmaf(h[i].v[c], h[i].v[c], ss);
        }
        if (p.h_out != nullptr) store_stream<F32>(p.h_out, t * p.H + v * kVec, h[i]);
    }
    if (p.w_pre == nullptr) return;
    const float r2 = rsqrtf(row_sum(ss, red2, shape.warps) / (float)p.H + p.eps);
    if (live && lane == 0 && p.rstd != nullptr) p.rstd[p.T + t] = r2;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lane + i * lanes;
        if (!live || v >= vecs) continue;
        const Vec8 w = load_f32(p.w_pre, v * kVec);
        Vec8 n;
#pragma unroll
        for (int c = 0; c < kVec; ++c) n.v[c] = h[i].v[c] * r2 * w.v[c];
        store_bf16(p.n, t * p.H + v * kVec, n);
    }
}

// ---------------------------------------------------------------- backward
//
// A row needs one reduction only: with e = d_h_out + r2 t (t = d_n w_pre) and
// u = yn w_post, the gradient is d = e - hn * (r2 m2), m2 = mean(t hn), so that
// the second norm's mean(g d u) = (sum g u e - r2 m2 sum g u hn) / H follows from
// sums that are known before m2 is.
//
// A CTA owns up to kCols columns, one vector of 8 to a thread, and keeps their
// weights and their sums over rows (d_w_post, d_w_pre, a channel gate's
// gradient) in registers for all its rows; wider rows are shared by a cluster
// of CTAs.  A producer warp keeps a ring of row stages filled by bulk copies.
// Consumer warps put their share of a row's three sums into every CTA of the
// cluster (pass 1) and take up the row again `lag` rows later (pass 2), when the
// sums have long arrived, so that no warp stands still at a row's end.  The CTAs'
// sums over rows go to the workspace once, and norm_columns_kernel adds them in
// CTA order, so that nothing depends on the order in which CTAs run.

constexpr int kCols = 4096;
constexpr int kMaxStages = 6;
constexpr int kSlots = 8;          // rows whose sums may be on their way; a writer is less than 6 rows ahead of a reader
constexpr int kMaxWarps = kCols / kVec / 32;

struct BackwardShape {
    int cluster;    // CTAs a row is shared by
    int cols;       // columns of a CTA (the last may have fewer)
    int warps;      // consumer warps
    int stages;
    int lag;
    int clusters;   // clusters of the grid
    int per_sm;     // CTAs an SM holds
};

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t in_cta(uint32_t smem, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
    return a;
}

// mbar_wait whose phase may be completed by other CTAs of the cluster.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (done) return true;
        if (global_timer_ns() - t0 > kWaitLimitNs) return false;
    }
}

template <bool F32>
__global__ void __launch_bounds__(kMaxWarps * 32 + 32) norm_backward_kernel(NormParams p, BackwardShape s) {
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], summed[kSlots];
    __shared__ float3 sums[kSlots][8 * kMaxWarps];
    __shared__ float scale_part[kMaxWarps];
    constexpr int kStream = F32 ? 4 : 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % s.cluster, group = blockIdx.x / s.cluster;
    const int col0 = rank * s.cols, cols = min(s.cols, p.H - col0);
    // a stage: h, d_h_out (stream type), y, d_n (bf16)
    const int at_dh = s.cols * kStream, at_y = at_dh * 2, at_dn = at_y + s.cols * 2, stage_bytes = at_dn + s.cols * 2;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < s.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], s.warps);
        }
        for (int i = 0; i < kSlots; ++i) mbar_init(&summed[i], s.warps * s.cluster);
        fence_mbar_init();
    }
    __syncthreads();
    if (s.cluster > 1) cluster_barrier();
    pdl_wait();
    const int rows = group < p.T ? (p.T - 1 - group) / s.clusters + 1 : 0;
    bool good = true;
    if (warp == s.warps) {
        // producer
        int filled = 0;
        for (; filled < rows; ++filled) {
            const int st = filled % s.stages, round = filled / s.stages;
            if (round > 0 && !__all_sync(0xffffffffu, mbar_wait(&empty[st], (round - 1) & 1))) {
                good = false;
                break;
            }
            if (lane == 0) {
                const int64_t t = group + (int64_t)filled * s.clusters;
                unsigned char* to = ring + st * stage_bytes;
                const int wide = cols * kStream, narrow = cols * 2;
                mbar_arrive_expect_tx(&full[st], wide + (p.d_h_out != nullptr ? wide : 0) + (p.y != nullptr ? narrow : 0) +
                                                     (p.d_n != nullptr ? narrow : 0));
                bulk_load(to, static_cast<const unsigned char*>(p.h) + (t * p.ld_h + col0) * kStream, wide, &full[st]);
                if (p.y != nullptr)
                    bulk_load(to + at_y, static_cast<const unsigned char*>(p.y) + (t * p.ld_y + col0) * 2, narrow, &full[st]);
                if (p.d_n != nullptr)
                    bulk_load(to + at_dn, static_cast<const unsigned char*>(p.d_n) + (t * p.H + col0) * 2, narrow, &full[st]);
                if (p.d_h_out != nullptr)
                    bulk_load(to + at_dh, static_cast<const unsigned char*>(p.d_h_out) + (t * p.H + col0) * kStream, wide, &full[st]);
            }
            __syncwarp();
        }
        // no copy may be in flight when the CTA ends, whatever its consumers did
        for (int i = max(0, filled - s.stages); i < filled; ++i) mbar_wait(&full[i % s.stages], (i / s.stages) & 1);
    } else {
        const int v = warp * 32 + lane;
        const bool in = v * kVec < cols;
        const int c0 = in ? v * kVec : 0;                  // column within the CTA
        const float inv_h = 1.f / (float)p.H;
        const float scale = p.res_scale != nullptr ? *p.res_scale : 1.f;
        const Vec8 w = in && p.w_post != nullptr ? load_f32(p.w_post, col0 + c0) : ones();
        const Vec8 g = in && p.gate_kind == kGateChannel ? load_f32(p.gate, col0 + c0) : ones();
        const Vec8 q = in && p.w_pre != nullptr ? load_f32(p.w_pre, col0 + c0) : zeros();
        Vec8 s_post = zeros(), s_gate = zeros(), s_pre = zeros();
        float s_scale = 0.f;
        for (int i = 0; i < rows + s.lag; ++i) {
            if (i < rows) {
                // pass 1: the row's three sums
                const int st = i % s.stages;
                const int64_t t = group + (int64_t)i * s.clusters;
                const float r1 = p.w_post != nullptr ? p.rstd[t] : 1.f;
                const float r2 = p.w_pre != nullptr ? p.rstd[p.T + t] : 0.f;
                const float token_gate = p.gate_kind == kGateToken ? p.gate[t] : 1.f;
                if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (i / s.stages) & 1))) good = false;
                float sum0 = 0.f, sum1 = 0.f, sum2 = 0.f;
                if (in && good) {
                    const unsigned char* from = ring + st * stage_bytes;
                    const Vec8 h = load_stream<F32>(from, c0), dh = p.d_h_out != nullptr ? load_stream<F32>(from + at_dh, c0) : zeros();
                    const Vec8 y = p.y != nullptr ? load_bf16(from + at_y, c0) : zeros();
                    const Vec8 dn = p.d_n != nullptr ? load_bf16(from + at_dn, c0) : zeros();
#pragma unroll
                    for (int c = 0; c < kVec; ++c) {
                        const float gu = g.v[c] * (y.v[c] * r1 * w.v[c]);
                        const float hn = r2 * fmaf(scale, h.v[c], token_gate * gu);
                        const float tt = dn.v[c] * q.v[c];
                        const float e = fmaf(r2, tt, dh.v[c]);
                        s_pre.v[c] = fmaf(dn.v[c], hn, s_pre.v[c]);
                        sum0 = fmaf(tt, hn, sum0);
                        sum1 = fmaf(gu, e, sum1);
                        sum2 = fmaf(gu, hn, sum2);
                    }
                }
                sum0 = warp_sum(sum0);
                sum1 = warp_sum(sum1);
                sum2 = warp_sum(sum2);
                if (lane < s.cluster) {
                    const uint32_t to = in_cta(smem_addr(&sums[i % kSlots][rank * s.warps + warp]), lane);
                    asm volatile("st.shared::cluster.f32 [%0], %1;\n\tst.shared::cluster.f32 [%0+4], %2;\n\tst.shared::cluster.f32 [%0+8], %3;"
                                 ::"r"(to), "f"(sum0), "f"(sum1), "f"(sum2) : "memory");
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                                 ::"r"(in_cta(smem_addr(&summed[i % kSlots]), lane)) : "memory");
                }
            }
            if (i >= s.lag) {
                // pass 2: the gradients of the row `lag` rows back
                const int j = i - s.lag, st = j % s.stages;
                const int64_t t = group + (int64_t)j * s.clusters;
                const float r1 = p.w_post != nullptr ? p.rstd[t] : 1.f;
                const float r2 = p.w_pre != nullptr ? p.rstd[p.T + t] : 0.f;
                const float token_gate = p.gate_kind == kGateToken ? p.gate[t] : 1.f;
                if (!__all_sync(0xffffffffu, mbar_wait_cluster(&summed[j % kSlots], (j / kSlots) & 1))) good = false;
                float sum0 = 0.f, sum1 = 0.f, sum2 = 0.f;
                for (int k = lane; k < s.warps * s.cluster; k += 32) {
                    const float3 x = sums[j % kSlots][k];
                    sum0 += x.x;
                    sum1 += x.y;
                    sum2 += x.z;
                }
                sum0 = warp_sum(sum0);
                const float m2 = r2 * (sum0 * inv_h);
                const float gu_d = warp_sum(sum1) - m2 * warp_sum(sum2);          // sum of g u d (without a token's gate)
                const float m1 = p.w_post != nullptr ? token_gate * gu_d * inv_h : 0.f;
                if (p.gate_kind == kGateToken && rank == 0 && threadIdx.x == 0) p.d_gate[t] = gu_d;
                if (in && good) {
                    const unsigned char* from = ring + st * stage_bytes;
                    const Vec8 h = load_stream<F32>(from, c0), dh = p.d_h_out != nullptr ? load_stream<F32>(from + at_dh, c0) : zeros();
                    const Vec8 y = p.y != nullptr ? load_bf16(from + at_y, c0) : zeros();
                    const Vec8 dn = p.d_n != nullptr ? load_bf16(from + at_dn, c0) : zeros();
                    Vec8 d_h, d_y;
#pragma unroll
                    for (int c = 0; c < kVec; ++c) {
                        const float yn = y.v[c] * r1, u = yn * w.v[c];
                        const float hn = r2 * fmaf(scale, h.v[c], token_gate * (g.v[c] * u));
                        const float d = fmaf(-hn, m2, fmaf(r2, dn.v[c] * q.v[c], dh.v[c]));
                        const float du = token_gate * (g.v[c] * d);
                        s_scale = fmaf(d, h.v[c], s_scale);
                        s_gate.v[c] = fmaf(d, u, s_gate.v[c]);
                        s_post.v[c] = fmaf(du, yn, s_post.v[c]);
                        d_h.v[c] = scale * d;
                        d_y.v[c] = r1 * fmaf(-yn, m1, du * w.v[c]);
                    }
                    store_stream<F32>(p.d_h, t * p.H + col0 + c0, d_h);
                    if (p.d_y != nullptr) store_bf16(p.d_y, t * p.H + col0 + c0, d_y);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
            }
            if (!good) break;
        }
        if (!in) s_scale = 0.f;
        s_scale = warp_sum(s_scale);
        if (lane == 0) scale_part[warp] = s_scale;
        if (in) {
            float* out = p.partial + (int64_t)group * 3 * p.H + col0 + c0;
            store_f32(out, 0, s_post);
            store_f32(out, p.H, s_gate);
            store_f32(out, 2 * (int64_t)p.H, s_pre);
        }
    }
    if (!good && lane == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrTimeout);
    __syncthreads();
    if (threadIdx.x == 0) {
        float sum = 0.f;
        for (int i = 0; i < s.warps; ++i) sum += scale_part[i];
        p.partial[(int64_t)s.clusters * 3 * p.H + blockIdx.x] = sum;
    }
    if (s.cluster > 1) cluster_barrier();      // no CTA ends while another may still write to it
}

// Adds `groups` rows of column sums and `ctas` sums for d_res_scale.  A CTA takes 32 columns; its 8 warps add
// every eighth row, then the eight sums are added in order.
__global__ void __launch_bounds__(256) norm_columns_kernel(NormParams p, int groups, int ctas) {
    __shared__ float part[8][32];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t width = 3 * (int64_t)p.H;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < width)
        for (int r = warp; r < groups; r += 8) s += p.partial[r * width + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < width) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[i][lane];
        const int which = (int)(c / p.H), at = (int)(c % p.H);
        float* out = which == 0 ? p.d_w_post : which == 1 ? (p.gate_kind == kGateChannel ? p.d_gate : nullptr) : p.d_w_pre;
        if (out != nullptr) out[at] = s;
    }
    if (blockIdx.x == 0 && warp == 1 && p.d_res_scale != nullptr) {
        s = 0.f;
        for (int r = lane; r < ctas; r += 32) s += p.partial[groups * width + r];
        s = warp_sum(s);
        if (lane == 0) *p.d_res_scale = s;
    }
}

constexpr int kMaxSms = 192;                      // the workspace has room for this many
constexpr size_t kRingBytes = 200 * 1024;         // shared memory of an SM that the rings may take

// clusters: at most this many, 0 for the workspace's bound.
BackwardShape backward_shape(int T, int H, int f32, int num_sms) {
    BackwardShape s{};
    s.cluster = H <= kCols ? 1 : H <= 2 * kCols ? 2 : 4;
    s.cols = ((H / kVec + s.cluster - 1) / s.cluster) * kVec;
    s.warps = (s.cols / kVec + 31) / 32;
    // narrow rows: as many CTAs on an SM as keep 16 consumer warps
    s.per_sm = std::max(1, std::min(4, 16 / s.warps));
    const size_t stage = (size_t)s.cols * (f32 ? 12 : 8);
    s.stages = (int)std::min<size_t>(kMaxStages, kRingBytes / s.per_sm / stage);
    // a cluster's sums take longer to arrive
    s.lag = std::min(s.cluster > 1 ? 2 : 1, s.stages - 2);
    s.clusters = std::min(T, std::min(num_sms, kMaxSms) * s.per_sm / s.cluster);
    return s;
}

}  // namespace

size_t norm_workspace_bytes(int T, int H) {
    const BackwardShape s = backward_shape(T, H, 0, kMaxSms);
    return ((size_t)s.clusters * (3 * (size_t)H + s.cluster) * sizeof(float) + 15) / 16 * 16;
}

cudaError_t launch_block_norm(const NormParams& p, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    const RowShape s = row_shape(p.H, 2, 4);
    const dim3 grid((unsigned)(((int64_t)p.T + s.rows - 1) / s.rows)), block(s.warps * 32 * s.rows);
    return p.f32 ? launch_kernel(true, norm_kernel<2, true>, grid, block, 0, stream, p, s)
                 : launch_kernel(true, norm_kernel<2, false>, grid, block, 0, stream, p, s);
}

cudaError_t launch_block_norm_backward(const NormParams& p, int num_sms, cudaStream_t stream) {
    const BackwardShape s = backward_shape(p.T, p.H, p.f32, num_sms);
    if (s.clusters > 0) {
        auto kern = p.f32 ? norm_backward_kernel<true> : norm_backward_kernel<false>;
        const size_t smem = (size_t)s.stages * s.cols * (p.f32 ? 12 : 8);
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
        if (e != cudaSuccess) return e;
        e = launch_clusters(true, s.cluster, kern, dim3(s.clusters * s.cluster), dim3(s.warps * 32 + 32), smem, stream, p, s);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((3 * (int64_t)p.H + 31) / 32));
    return launch_kernel(true, norm_columns_kernel, grid, dim3(256), 0, stream, p, s.clusters, s.clusters * s.cluster);
}

}  // namespace ep
