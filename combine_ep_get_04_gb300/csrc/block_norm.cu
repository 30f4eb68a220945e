// block_norm.cu -- the end of one block and the start of the next:
//   u = y * r1 * w_post,  h_out = res_scale * h + gate * u,  n = h_out * r2 * w_pre
// with r = 1 / sqrt(mean square + eps), and its gradients.  One pass over the
// rows in each direction; every value in between stays in registers, so the
// kernels read and write each tensor once and are bound by HBM.
#include <algorithm>

#include "block_device.cuh"
#include "block_kernels.h"

namespace ep {
namespace {

constexpr int kGateChannel = 1;
constexpr int kGateToken = 2;
constexpr int kVec = 8;   // channels a thread handles at once: 16 bytes of bf16
constexpr int kMaxStages = 8;

// Eight fp32 values as four pairs (f32x2), which halves the instructions a row costs.
struct Vec8 {
    uint64_t v[4];
};

__device__ __forceinline__ float total(uint64_t p) {
    const float2 x = halves(p);
    return x.x + x.y;
}

__device__ __forceinline__ Vec8 bf16_vec(uint4 w) {
    return Vec8{{pair(bf16_lo(w.x), bf16_hi(w.x)), pair(bf16_lo(w.y), bf16_hi(w.y)), pair(bf16_lo(w.z), bf16_hi(w.z)),
                 pair(bf16_lo(w.w), bf16_hi(w.w))}};
}

__device__ __forceinline__ Vec8 f32_vec(float4 a, float4 b) { return Vec8{{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}}; }

__device__ __forceinline__ Vec8 load_bf16(const void* base, int64_t at) {
    return bf16_vec(*reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(base) + at * 2));
}

__device__ __forceinline__ Vec8 load_f32(const void* base, int64_t at) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    return f32_vec(p[0], p[1]);
}

__device__ __forceinline__ void store_bf16(void* base, int64_t at, const Vec8& x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = halves(x.v[i]);
        w[i] = pack_bf16x2(f.x, f.y);
    }
    *reinterpret_cast<uint4*>(static_cast<unsigned char*>(base) + at * 2) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_f32(void* base, int64_t at, const Vec8& x) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    const float2 a = halves(x.v[0]), b = halves(x.v[1]), c = halves(x.v[2]), d = halves(x.v[3]);
    p[0] = make_float4(a.x, a.y, b.x, b.y);
    p[1] = make_float4(c.x, c.y, d.x, d.y);
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

__device__ __forceinline__ Vec8 all(float x) { return Vec8{{both(x), both(x), both(x), both(x)}}; }

// Sum over the warps of a CTA.  `red` holds one float for each warp; one
// barrier: a caller that sums again uses another array until the next.
__device__ __forceinline__ float cta_sum(float x, float* red, int warps) {
    x = warp_sum(x);
    if (warps == 1) return x;
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    return warp_sum(lane < warps ? red[lane] : 0.f);
}

// ----------------------------------------------------------------- forward
//
// A CTA takes a row at a time, NV vectors of 8 channels to a thread, rows a
// grid apart, and holds the weights of its channels in registers for all its
// rows (NV = 1).  The next row's h and y are on their way while a row is worked
// on; in between the row stays in registers: the mean square of y, then that of
// h_out, one barrier each (none where a row fits a warp).
//
// FULL: y, both norms and h_out are there, which saves the tests for them.
//
// Two to 32 CTAs an SM hide the barriers up to 4,096 channels: T=16384 H=4096 bf16
// 86 us, 6.2 TB/s, 92 % of the measured copy rate; T=9000 H=1672 fp32 34 us, 78 %;
// a decode batch of 128 rows of 7168 is latency, 3.3 us.
template <int NV, bool F32, bool FULL>
__global__ void __launch_bounds__(1024) norm_kernel(NormParams p) {
    __shared__ float red[4][32];
    const int lanes = blockDim.x, warps = lanes >> 5, vecs = p.H / kVec;
    const bool has_y = FULL || p.y != nullptr, has_post = FULL || p.w_post != nullptr, has_pre = FULL || p.w_pre != nullptr;
    const float inv_h = 1.f / (float)p.H;
    pdl_launch_dependents();
    pdl_wait();
    const float scale = p.res_scale != nullptr ? *p.res_scale : 1.f;
    bool in[NV];
    int at[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * lanes;
        in[i] = v < vecs;
        at[i] = v * kVec;
    }
    Vec8 w[NV], g[NV], q[NV];
    auto load_weights = [&](int i) {
        w[i] = in[i] && has_post ? load_f32(p.w_post, at[i]) : all(1.f);
        g[i] = in[i] && p.gate_kind == kGateChannel ? load_f32(p.gate, at[i]) : all(1.f);
        q[i] = in[i] && has_pre ? load_f32(p.w_pre, at[i]) : all(0.f);
    };
    constexpr int kRaw = F32 ? 2 : 1;
    uint4 next_h[NV][kRaw], next_y[NV];
    float next_gate = 1.f;
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int r = 0; r < kRaw; ++r) next_h[i][r] = make_uint4(0, 0, 0, 0);
            next_y[i] = make_uint4(0, 0, 0, 0);
            if (in[i] && t < p.T) {
                const uint4* h = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.h) + (t * p.ld_h + at[i]) * (F32 ? 4 : 2));
#pragma unroll
                for (int r = 0; r < kRaw; ++r) next_h[i][r] = h[r];
                if (has_y) next_y[i] = *reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.y) + (t * p.ld_y + at[i]) * 2);
            }
        }
        if (p.gate_kind == kGateToken && t < p.T) next_gate = p.gate[t];
    };
    if (NV == 1) load_weights(0);
    fetch(blockIdx.x);
    int flip = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, flip ^= 2) {
        Vec8 h[NV], y[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint4 a = next_h[i][0], b = next_h[i][kRaw - 1];
            h[i] = F32 ? f32_vec(make_float4(__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w)),
                                 make_float4(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)))
                       : bf16_vec(a);
            y[i] = bf16_vec(next_y[i]);
        }
        const float gate = next_gate;
        fetch(t + gridDim.x);
        float r1 = 1.f;
        if (has_post) {
            uint64_t ss = both(0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) ss = fma2(y[i].v[c], y[i].v[c], ss);
            r1 = rsqrtf(fmaf(cta_sum(total(ss), red[flip], warps), inv_h, p.eps));
            if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[t] = r1;
        }
        uint64_t ss = both(0.f);
        const uint64_t r1_gate = both(r1 * gate), a2 = both(scale);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (NV > 1) load_weights(i);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint64_t gu = mul2(g[i].v[c], mul2(mul2(y[i].v[c], r1_gate), w[i].v[c]));
                h[i].v[c] = fma2(a2, h[i].v[c], gu);
                ss = fma2(h[i].v[c], h[i].v[c], ss);
            }
            if (in[i] && (FULL || p.h_out != nullptr)) store_stream<F32>(p.h_out, t * p.H + at[i], h[i]);
        }
        if (!has_pre) continue;
        const float r2 = rsqrtf(fmaf(cta_sum(total(ss), red[flip + 1], warps), inv_h, p.eps));
        if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[p.T + t] = r2;
        const uint64_t r2_2 = both(r2);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Vec8 n;
#pragma unroll
            for (int c = 0; c < 4; ++c) n.v[c] = mul2(mul2(h[i].v[c], r2_2), q[i].v[c]);
            if (in[i]) store_bf16(p.n, t * p.H + at[i], n);
        }
    }
}

// The barrier of a turn, which the producer warp joins.
__device__ __forceinline__ void rows_barrier(int warps) { asm volatile("bar.sync 1, %0;" ::"r"(warps * 32) : "memory"); }

// Sums of two values over a CTA: lanes 0 to 15 deal with the first, the others
// with the second.  `red` has two rows of 32.
__device__ __forceinline__ float2 cta_sum2(float a, float b, float (*red)[32], int warps) {
    const int lane = threadIdx.x & 31;
    const bool high = lane & 16;
    float x = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 16);
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    {
        if ((lane & 15) == 0) red[lane >> 4][threadIdx.x >> 5] = x;
        rows_barrier(warps + 1);
        const int w = lane & 15;
        x = (w < warps ? red[lane >> 4][w] : 0.f) + (w + 16 < warps ? red[lane >> 4][w + 16] : 0.f);
#pragma unroll
        for (int d = 8; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    }
    const float other = __shfl_xor_sync(0xffffffffu, x, 16);
    return high ? make_float2(other, x) : make_float2(x, other);
}

// Waits for a row's copies, at most kWaitLimitNs.  A wait that runs out sets
// *lost, with which the others end too.
__device__ __forceinline__ void wait_row(uint64_t* bar, uint32_t parity, volatile int* lost) {
    if (mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*lost != 0) return;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *lost = 1;
            return;
        }
    }
}

// Many wide rows.  As above, with two differences.  A row is taken up in two
// turns, so that its two sums come with those of its neighbours: turn i has the
// mean square of row i's y and, with that of row i - 1 known, row i - 1's h_out
// and its mean square, both joined behind one barrier.  And rows come by bulk
// copies into a ring of stages in shared memory; a producer warp joins the
// barrier and fills the stage that it sets free.
//
// T=16384 H=4096 fp32 128 us, 6.3 TB/s, 92 % of the measured copy rate; T=4096 H=7168
// fp32 59.5 us, 87 %, bf16 41.7 us, 83 %.  (Rows copied by each thread for itself, without
// a producer, took 150, 78 and 42 us: a 16-byte copy of fp32 fetches half a sector.  The
// ring filled by a consumer thread took 144, 60 and 46 us: all others wait for it.)
template <bool F32, bool FULL>
__global__ void __launch_bounds__(1024) norm_rows_kernel(NormParams p, int stages) {
    extern __shared__ __align__(128) unsigned char ring[];       // [stages][h, y]
    __shared__ uint64_t full[kMaxStages];
    __shared__ float red[2][2][32];
    __shared__ int lost;                                         // a copy did not come in time
    constexpr int kStream = F32 ? 4 : 2;
    const int warps = (blockDim.x >> 5) - 1, at_y = p.H * kStream, stage_bytes = p.H * (kStream + 2);
    const bool has_y = FULL || p.y != nullptr, has_post = FULL || p.w_post != nullptr, has_pre = FULL || p.w_pre != nullptr;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
        lost = 0;
    }
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();
    const int rows = blockIdx.x < p.T ? (p.T - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    if (threadIdx.x >> 5 == warps) {
        // producer: fills the ring, then the stage of row i - 1 behind the barrier of turn i
        const int lane = threadIdx.x & 31;
        const unsigned char* h = static_cast<const unsigned char*>(p.h) + (int64_t)blockIdx.x * p.ld_h * kStream;
        const unsigned char* y = static_cast<const unsigned char*>(p.y) + (int64_t)blockIdx.x * p.ld_y * 2;
        volatile int* const missing = &lost;
        int filled = 0;
        auto fetch = [&](int st) {
            ++filled;
            if (lane == 0) {
                unsigned char* to = ring + st * stage_bytes;
                mbar_arrive_expect_tx(&full[st], has_y ? stage_bytes : at_y);
                bulk_load(to, h, at_y, &full[st]);
                if (has_y) bulk_load(to + at_y, y, p.H * 2, &full[st]);
            }
            h += gridDim.x * p.ld_h * kStream;
            y += gridDim.x * p.ld_y * 2;
        };
        for (int i = 0; i < min(stages, rows); ++i) fetch(i);
        int st = 0;
        for (int i = 0; i <= rows; ++i) {
            __syncwarp();
            rows_barrier(warps + 1);
            if (i == 0) continue;
            // all consumers have seen row i - 1 come, or one of them has set `lost`
            if (i - 1 + stages < rows && *missing == 0) fetch(st);
            if (++st == stages) st = 0;
        }
        __syncwarp();
        rows_barrier(warps + 1);
        if (*missing != 0) {
            // no copy may be in flight when the CTA ends; and the loss is seen in what is written
            for (int i = max(0, filled - stages); i < filled; ++i) mbar_wait(&full[i % stages], (i / stages) & 1);
            for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
                for (int at = lane * kVec; at < p.H; at += 32 * kVec) {
                    if (p.h_out != nullptr) store_stream<F32>(p.h_out, t * p.H + at, all(NAN));
                    if (has_pre) store_bf16(p.n, t * p.H + at, all(NAN));
                }
                if (lane == 0 && p.rstd != nullptr) {
                    if (has_post) p.rstd[t] = NAN;
                    if (has_pre) p.rstd[p.T + t] = NAN;
                }
            }
        }
        return;
    }
    const float inv_h = 1.f / (float)p.H;
    const float scale = p.res_scale != nullptr ? *p.res_scale : 1.f;
    const bool in = threadIdx.x < p.H / kVec;
    const int at = in ? threadIdx.x * kVec : 0;
    const Vec8 q = in && has_pre ? load_f32(p.w_pre, at) : all(0.f);
    Vec8 w = in && has_post ? load_f32(p.w_post, at) : all(1.f);
    if (in && p.gate_kind == kGateChannel) {
        const Vec8 g = load_f32(p.gate, at);
#pragma unroll
        for (int c = 0; c < 4; ++c) w.v[c] = mul2(w.v[c], g.v[c]);
    }
    unsigned char* h_to = static_cast<unsigned char*>(p.h_out) + (int64_t)blockIdx.x * p.H * kStream;
    unsigned char* n_to = static_cast<unsigned char*>(p.n) + (int64_t)blockIdx.x * p.H * 2;
    int64_t t = blockIdx.x;                       // row of turn i
    float r1 = 1.f, gate = 1.f, next_gate = 1.f;
    int st = 0, before = 0;                       // stages of rows i and i - 1
    uint32_t parity = 0;
    for (int i = 0; i <= rows; ++i) {
        if (p.gate_kind == kGateToken && i < rows) next_gate = p.gate[t];
        Vec8 h;
        uint64_t ss2 = both(0.f), ss1 = ss2;
        if (i > 0) {
            const uint64_t r1_gate = both(r1 * gate), a2 = both(scale);
            const unsigned char* row = ring + before * stage_bytes;
            const Vec8 y = in && has_y ? load_bf16(row + at_y, at) : all(0.f);
            h = in ? load_stream<F32>(row, at) : all(0.f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                h.v[c] = fma2(a2, h.v[c], mul2(mul2(y.v[c], r1_gate), w.v[c]));
                ss2 = fma2(h.v[c], h.v[c], ss2);
            }
            if (in && (FULL || p.h_out != nullptr)) store_stream<F32>(h_to, at, h);
            h_to += (int64_t)gridDim.x * p.H * kStream;
        }
        if (i < rows) {
            wait_row(&full[st], parity, &lost);
            const Vec8 y = in && has_y ? load_bf16(ring + st * stage_bytes + at_y, at) : all(0.f);
#pragma unroll
            for (int c = 0; c < 4; ++c) ss1 = fma2(y.v[c], y.v[c], ss1);
        }
        const float2 sums = cta_sum2(total(ss1), total(ss2), red[i & 1], warps);
        if (i > 0 && has_pre) {
            const float r2 = rsqrtf(fmaf(sums.y, inv_h, p.eps));
            if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[p.T + t - gridDim.x] = r2;
            const uint64_t r2_2 = both(r2);
            Vec8 n;
#pragma unroll
            for (int c = 0; c < 4; ++c) n.v[c] = mul2(mul2(h.v[c], r2_2), q.v[c]);
            if (in) store_bf16(n_to, at, n);
            n_to += (int64_t)gridDim.x * p.H * 2;
        }
        if (has_post) {
            r1 = rsqrtf(fmaf(sums.x, inv_h, p.eps));
            if (threadIdx.x == 0 && p.rstd != nullptr && i < rows) p.rstd[t] = r1;
        }
        gate = next_gate;
        t += gridDim.x;
        before = st;
        if (++st == stages) {
            st = 0;
            parity ^= 1;
        }
    }
    rows_barrier(warps + 1);
}

// ---------------------------------------------------------------- backward
//
// A row needs one reduction only: with e = d_h_out + r2 t (t = d_n w_pre) and
// v = y w_post (times a channel's gate), the gradient is d = e - hn * (r2 m2),
// m2 = mean(t hn), so that the second norm's mean follows from sums that are
// known before m2 is: sum(v d) = sum(v e) - r2 m2 sum(v hn).
//
// Over rows there are two sums to a column: d_n hn, which is d_w_pre, and
// r1 d y (times a token's gate), which times the gate is d_w_post and times
// w_post the gradient of a channel's gate.
//
// A CTA owns up to kCols columns, one vector of 8 to a thread, and keeps their
// weights and their sums over rows in registers for all its rows; wider rows are shared by a cluster
// of CTAs.  A producer warp keeps a ring of row stages filled by bulk copies.
// Consumer warps leave their share of a row's three sums to another warp, which
// adds them and joins them with those of the cluster's other CTAs (pass 1), and
// take up the row again `lag` rows later (pass 2), when the sums are there, so
// that none stands still at a row's end.  The CTAs' sums over rows go to the
// workspace once, and norm_columns_kernel adds them in CTA order, so that nothing depends on the order in which CTAs run.
//
// T=16384 H=4096 fp32 188 us, 6.4 TB/s, 95 % of the measured copy rate; T=4096 H=7168
// fp32 83 us, 93 %; bf16 66 us, 5.3 TB/s: at two bytes a value the instructions of the
// two passes (58 % of the issue slots with 16 warps an SM) weigh as much as the bytes.

constexpr int kCols = 4096;
constexpr int kMaxCluster = 4;
constexpr int kSlots = 8;          // rows whose sums may be on their way; a writer is less than 6 rows ahead of a reader
constexpr int kMaxWarps = kCols / kVec / 32;
constexpr int kColumnWarps = 16;

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

// A sum on its way between CTAs: the value and, in the same 64-bit word, which
// row it is of, so that no fence has to order the two.  (An arrival on the
// receiver's barrier with release semantics waits until the SM's stores have
// drained, and with the gradients streaming out that took longer than a row.)
__device__ __forceinline__ void post(uint32_t to, float value, uint32_t row) {
    const uint64_t word = (uint64_t)row << 32 | __float_as_uint(value);
    asm volatile("st.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(to), "l"(word) : "memory");
}

// Waits, at most kWaitLimitNs, for the word of `row` and returns its value.
__device__ __forceinline__ bool collect(const uint64_t* from, uint32_t row, float* value) {
    uint64_t t0 = 0;
    for (;;) {
        uint64_t word;
        asm volatile("ld.relaxed.cluster.shared::cta.b64 %0, [%1];" : "=l"(word) : "r"(smem_addr(from)) : "memory");
        if ((uint32_t)(word >> 32) == row) {
            *value = __uint_as_float((uint32_t)word);
            return true;
        }
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) return false;
    }
}

// What a row's threads all need; gate is the token's.
struct __align__(16) RowValues {
    float r2, r2_scale, r2_r1_gate, r1_gate;
    float r1, gate, unused[2];
};

// Sums of three values over a warp in six shuffles: lane 0 ends up with the
// first, lane 16 with the second, lane 8 with the third.
__device__ __forceinline__ float warp_sum3(float x0, float x1, float x2) {
    const int lane = threadIdx.x & 31;
    const bool high = lane & 16, third = lane & 8;
    float y = (high ? x1 : x0) + __shfl_xor_sync(0xffffffffu, high ? x0 : x1, 16);
    x2 += __shfl_xor_sync(0xffffffffu, x2, 16);
    y = (third ? x2 : y) + __shfl_xor_sync(0xffffffffu, third ? y : x2, 8);
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1) y += __shfl_xor_sync(0xffffffffu, y, d);
    return y;
}

// FULL: y, d_n and d_h_out are there, which saves the tests for them.
// WARPS: most warps of a CTA; up to 16 a thread has 128 registers, which is what it needs, with 18 it has 96.
template <bool F32, bool FULL, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) norm_backward_kernel(NormParams p, BackwardShape s) {
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], added[kSlots], summed[kSlots];
    __shared__ float warp_sums[kSlots][3][kMaxWarps];
    __shared__ float4 sums[kSlots];
    __shared__ uint64_t posted[kSlots][kMaxCluster][4];       // the three sums of each CTA of the cluster
    __shared__ RowValues row_values[kMaxStages];
    __shared__ float scale_part[kMaxWarps];
    constexpr int kStream = F32 ? 4 : 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % s.cluster, group = blockIdx.x / s.cluster;
    const int col0 = rank * s.cols, cols = min(s.cols, p.H - col0);
    const bool has_y = FULL || p.y != nullptr, has_dn = FULL || p.d_n != nullptr, has_dh = FULL || p.d_h_out != nullptr;
    // a stage: h, d_h_out (stream type), y, d_n (bf16)
    const int at_dh = s.cols * kStream, at_y = at_dh * 2, at_dn = at_y + s.cols * 2, stage_bytes = at_dn + s.cols * 2;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < s.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], s.warps);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&added[i], s.warps);
            mbar_init(&summed[i], 1);
        }
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < kSlots * kMaxCluster * 4; i += blockDim.x) (&posted[0][0][0])[i] = 0;
    __syncthreads();
    if (s.cluster > 1) cluster_barrier();
    pdl_wait();
    const int rows = group < p.T ? (p.T - 1 - group) / s.clusters + 1 : 0;
    const float scale = p.res_scale != nullptr ? *p.res_scale : 1.f;
    bool good = true;
    if (warp == s.warps) {
        // producer
        int filled = 0, st = 0;
        uint32_t parity = 1;                      // of the stage's previous use
        // the next row's values are on their way while a stage is waited for
        float r1 = 1.f, r2 = 0.f, gate = 1.f;
        auto look_up = [&](int i) {
            const int64_t t = group + (int64_t)i * s.clusters;
            if (lane == 1 && i < rows) {
                if (p.w_post != nullptr) r1 = p.rstd[t];
                if (p.w_pre != nullptr) r2 = p.rstd[p.T + t];
                if (p.gate_kind == kGateToken) gate = p.gate[t];
            }
        };
        look_up(0);
        for (; filled < rows; ++filled) {
            if (filled >= s.stages && !__all_sync(0xffffffffu, mbar_wait(&empty[st], parity))) {
                good = false;
                break;
            }
            const int64_t t = group + (int64_t)filled * s.clusters;
            if (lane == 0) {
                unsigned char* to = ring + st * stage_bytes;
                const int wide = cols * kStream, narrow = cols * 2;
                mbar_expect_tx(&full[st], wide + (has_dh ? wide : 0) + (has_y ? narrow : 0) + (has_dn ? narrow : 0));
                bulk_load(to, static_cast<const unsigned char*>(p.h) + (t * p.ld_h + col0) * kStream, wide, &full[st]);
                if (has_y) bulk_load(to + at_y, static_cast<const unsigned char*>(p.y) + (t * p.ld_y + col0) * 2, narrow, &full[st]);
                if (has_dn) bulk_load(to + at_dn, static_cast<const unsigned char*>(p.d_n) + (t * p.H + col0) * 2, narrow, &full[st]);
                if (has_dh)
                    bulk_load(to + at_dh, static_cast<const unsigned char*>(p.d_h_out) + (t * p.H + col0) * kStream, wide, &full[st]);
            }
            if (lane == 1) row_values[st] = RowValues{r2, r2 * scale, r2 * r1 * gate, r1 * gate, r1, gate, {0.f, 0.f}};
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);          // after the row's values are written
            look_up(filled + 1);
            if (++st == s.stages) {
                st = 0;
                parity ^= 1;
            }
        }
        // no copy may be in flight when the CTA ends, whatever its consumers did
        for (int i = max(0, filled - s.stages); i < filled; ++i) mbar_wait(&full[i % s.stages], (i / s.stages) & 1);
    } else if (warp == s.warps + 1) {
        // adds the warps' sums of each row
        uint32_t parity = 0;
        auto add = [&](int slot, float (&x)[3]) {
            good = __all_sync(0xffffffffu, mbar_wait(&added[slot], parity));
            if (slot == kSlots - 1) parity ^= 1;
#pragma unroll
            for (int k = 0; k < 3; ++k) x[k] = warp_sum(lane < s.warps ? warp_sums[slot][k][lane] : 0.f);
            return good;
        };
        if (s.cluster == 1) {
            for (int i = 0; i < rows; ++i) {
                const int slot = i % kSlots;
                float x[3];
                if (!add(slot, x)) break;
                if (lane == 0) {
                    sums[slot] = make_float4(x[0], x[1], x[2], 0.f);
                    mbar_arrive(&summed[slot]);
                }
            }
        } else {
            // posts them to every CTA and joins those of the row before, which have arrived by now: lane 4 r + k deals
            // with sum k of CTA r
            const int r = lane >> 2, k = lane & 3;
            const bool part = r < s.cluster && k < 3;
            const uint32_t to = in_cta(smem_addr(&posted[0][rank][k]), part ? r : 0);
            for (int i = 0; i <= rows; ++i) {
                const int slot = i % kSlots;
                if (i < rows) {
                    float x[3];
                    if (!add(slot, x)) break;
                    if (part) post(to + slot * (uint32_t)sizeof(posted[0]), k == 0 ? x[0] : k == 1 ? x[1] : x[2], (uint32_t)i + 1);
                }
                if (i > 0) {
                    const int before = (i - 1) % kSlots;
                    float x = 0.f;
                    good = __all_sync(0xffffffffu, !part || collect(&posted[before][r][k], (uint32_t)i, &x));
                    if (!good) break;
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    if (lane < 3) (&sums[before].x)[lane] = x;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&summed[before]);
                }
            }
        }
        __syncwarp();
    } else {
        const int v = warp * 32 + lane;
        const bool in = v * kVec < cols;                   // the others go through it with weights of 0 and store nothing
        const int c0 = in ? v * kVec : 0;                  // column within the CTA
        const float inv_h = 1.f / (float)p.H;
        const Vec8 q = in && p.w_pre != nullptr ? load_f32(p.w_pre, col0 + c0) : all(0.f);
        Vec8 wg = all(in ? 1.f : 0.f);
        if (in && p.w_post != nullptr) wg = load_f32(p.w_post, col0 + c0);
        if (in && p.gate_kind == kGateChannel) {
            const Vec8 g = load_f32(p.gate, col0 + c0);
#pragma unroll
            for (int c = 0; c < 4; ++c) wg.v[c] = mul2(wg.v[c], g.v[c]);
        }
        Vec8 s_dy = all(0.f), s_pre = all(0.f);
        uint64_t s_scale = both(0.f);
        const unsigned char* first = ring + c0 * 2;        // the thread's place in a bf16 row
        auto take = [&](int at, Vec8& h, Vec8& dh, Vec8& y, Vec8& dn) {
            const unsigned char* from = first + at;
            const unsigned char* wide = from + (F32 ? c0 * 2 : 0);
            h = load_stream<F32>(wide, 0);
            dh = has_dh ? load_stream<F32>(wide + at_dh, 0) : all(0.f);
            y = has_y ? load_bf16(from + at_y, 0) : all(0.f);
            dn = has_dn ? load_bf16(from + at_dn, 0) : all(0.f);
        };
        int st1 = 0, st2 = 0, at1 = 0, at2 = 0;
        uint32_t full_parity = 0, summed_parity = 0;
        const int64_t stride = (int64_t)s.clusters * p.H;
        unsigned char* d_h_row = static_cast<unsigned char*>(p.d_h) + ((int64_t)group * p.H + col0 + c0) * kStream;
        unsigned char* d_y_row = has_y ? static_cast<unsigned char*>(p.d_y) + ((int64_t)group * p.H + col0 + c0) * 2 : nullptr;
        float* d_gate = p.gate_kind == kGateToken && rank == 0 && threadIdx.x == 0 ? p.d_gate + group : nullptr;
        for (int i = 0; i < rows + s.lag; ++i) {
            if (i < rows) {
                // pass 1: the row's three sums
                good = __all_sync(0xffffffffu, mbar_wait(&full[st1], full_parity));
                if (!good) break;
                uint64_t sum0 = both(0.f), sum1 = sum0, sum2 = sum0;
                {
                    const RowValues& rv = row_values[st1];
                    const uint64_t r2 = both(rv.r2), r2_scale = both(rv.r2_scale), r2_r1_gate = both(rv.r2_r1_gate);
                    Vec8 h, dh, y, dn;
                    take(at1, h, dh, y, dn);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint64_t v = mul2(y.v[c], wg.v[c]);
                        const uint64_t hn = fma2(r2_r1_gate, v, mul2(r2_scale, h.v[c]));
                        const uint64_t t = mul2(dn.v[c], q.v[c]);
                        const uint64_t e = fma2(r2, t, dh.v[c]);
                        s_pre.v[c] = fma2(dn.v[c], hn, s_pre.v[c]);
                        sum0 = fma2(t, hn, sum0);
                        sum1 = fma2(v, e, sum1);
                        sum2 = fma2(v, hn, sum2);
                    }
                }
                const float x = warp_sum3(total(sum0), total(sum1), total(sum2));
                const int slot = i % kSlots;
                if ((lane & 7) == 0 && lane != 24) warp_sums[slot][lane == 0 ? 0 : lane == 16 ? 1 : 2][warp] = x;
                __syncwarp();
                if (lane == 0) mbar_arrive(&added[slot]);
                at1 += stage_bytes;
                if (++st1 == s.stages) {
                    st1 = at1 = 0;
                    full_parity ^= 1;
                }
            }
            if (i >= s.lag) {
                // pass 2: the gradients of the row `lag` rows back
                const int slot = (i - s.lag) % kSlots;
                good = __all_sync(0xffffffffu, mbar_wait(&summed[slot], summed_parity));
                if (!good) break;
                if (slot == kSlots - 1) summed_parity ^= 1;
                const float4 x = sums[slot];
                const RowValues& rv = row_values[st2];
                const float m2 = rv.r2 * (x.x * inv_h);
                const float u_d = rv.r1 * (x.y - m2 * x.z);          // sum of g u d (without a token's gate)
                const float m1 = p.w_post != nullptr ? rv.gate * u_d * inv_h : 0.f;
                if (d_gate != nullptr) {
                    *d_gate = u_d;
                    d_gate += s.clusters;
                }
                const uint64_t r2 = both(rv.r2), r2_scale = both(rv.r2_scale), r2_r1_gate = both(rv.r2_r1_gate);
                const uint64_t r1_gate = both(rv.r1_gate), a2 = both(scale), minus_m2 = both(-m2), back = both(-rv.r1 * rv.r1 * m1);
                Vec8 h, dh, y, dn, d_h, d_y;
                take(at2, h, dh, y, dn);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint64_t hn = fma2(r2_r1_gate, mul2(y.v[c], wg.v[c]), mul2(r2_scale, h.v[c]));
                    const uint64_t e = fma2(r2, mul2(dn.v[c], q.v[c]), dh.v[c]);
                    const uint64_t d = fma2(minus_m2, hn, e), rd = mul2(r1_gate, d);
                    s_scale = fma2(d, h.v[c], s_scale);
                    s_dy.v[c] = fma2(rd, y.v[c], s_dy.v[c]);
                    d_h.v[c] = mul2(a2, d);
                    d_y.v[c] = fma2(wg.v[c], rd, mul2(back, y.v[c]));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st2]);
                if (in) {
                    store_stream<F32>(d_h_row, 0, d_h);
                    if (has_y) store_bf16(d_y_row, 0, d_y);
                }
                d_h_row += stride * kStream;
                if (has_y) d_y_row += stride * 2;
                at2 += stage_bytes;
                if (++st2 == s.stages) st2 = at2 = 0;
            }
        }
        const float sum = warp_sum(in ? total(s_scale) : 0.f);
        if (lane == 0) scale_part[warp] = sum;
        if (in) {
            float* out = p.partial + (int64_t)group * 2 * p.H + col0 + c0;
            store_f32(out, 0, s_dy);
            store_f32(out, p.H, s_pre);
        }
    }
    if (!good && lane == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrTimeout);
    __syncthreads();
    if (threadIdx.x == 0) {
        float sum = 0.f;
        for (int i = 0; i < s.warps; ++i) sum += scale_part[i];
        p.partial[(int64_t)s.clusters * 2 * p.H + blockIdx.x] = sum;
    }
    if (s.cluster > 1) cluster_barrier();      // no CTA ends while another may still write to it
}

// Adds `groups` rows of column sums and `ctas` sums for d_res_scale.  A CTA takes 32 columns; each warp adds every
// kColumnWarps-th row, then the warps' sums are added in order.  4.4 MB at T=4096 H=7168, 6.5 us by itself from a cold
// cache: latency.
__global__ void __launch_bounds__(kColumnWarps * 32) norm_columns_kernel(NormParams p, int groups, int ctas) {
    __shared__ float part[kColumnWarps][32];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t width = 2 * (int64_t)p.H;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < width)
#pragma unroll 4
        for (int r = warp; r < groups; r += kColumnWarps) s += p.partial[r * width + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < width) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < kColumnWarps; ++i) s += part[i][lane];
        if (c >= p.H) {
            if (p.d_w_pre != nullptr) p.d_w_pre[c - p.H] = s;
        } else {
            const bool channel = p.gate_kind == kGateChannel;
            if (p.d_w_post != nullptr) p.d_w_post[c] = channel ? s * p.gate[c] : s;
            if (channel) p.d_gate[c] = p.w_post != nullptr ? s * p.w_post[c] : s;
        }
    }
    if (blockIdx.x == 0 && warp == 1 && p.d_res_scale != nullptr) {
        s = 0.f;
        for (int r = lane; r < ctas; r += 32) s += p.partial[groups * width + r];
        s = warp_sum(s);
        if (lane == 0) *p.d_res_scale = s;
    }
}

constexpr int kMaxSms = 192;                      // the workspace has room for this many
constexpr size_t kRingBytes = 216 * 1024;         // shared memory of an SM that the rings may take
constexpr size_t kSmBytes = 228 * 1024;           // all of it,
constexpr size_t kBesideRing = 4608;              // and what a CTA of the backward pass takes beside its ring: 3328 of its own, 1 KB reserved

BackwardShape backward_shape(int T, int H, int f32, int num_sms) {
    BackwardShape s{};
    s.cluster = H <= kCols ? 1 : H <= 2 * kCols ? 2 : 4;
    s.cols = ((H / kVec + s.cluster - 1) / s.cluster) * kVec;
    s.warps = (s.cols / kVec + 31) / 32;
    // narrow rows: as many CTAs on an SM as make 16 consumer warps and as its registers hold, 96 a thread, five warps to each
    // quarter of the SM (T=8192 H=256 bf16 21 us, with one CTA an SM 48; T=9000 H=1672 fp32 47 and 53)
    s.per_sm = std::max(1, std::min({6, 16 / s.warps, 20 / (s.warps + 2)}));
    const size_t stage = (size_t)s.cols * (f32 ? 12 : 8);
    // no more stages than leave room for per_sm CTAs, or the grid runs a second, half-empty wave
    s.stages = (int)std::min<size_t>(kMaxStages, std::min(kRingBytes / s.per_sm, kSmBytes / s.per_sm - kBesideRing) / stage);
    // one CTA an SM has nothing else to do until a row's sums are there (T=4096 H=7168 bf16, 7 stages: 91 us with a lag of
    // 1, 67 with 2, 66 with 3; fp32, 5 stages: 95, 83 and 88)
    s.lag = std::min(s.per_sm > 1 ? 1 : s.stages >= 7 ? 3 : 2, s.stages - 2);
    s.clusters = std::min(T, std::min(num_sms, kMaxSms) * s.per_sm / s.cluster);
    return s;
}

size_t ring_bytes(const BackwardShape& s, int f32) { return (size_t)s.stages * s.cols * (f32 ? 12 : 8); }

using BackwardKernel = void (*)(NormParams, BackwardShape);

BackwardKernel backward_kernel(const BackwardShape& s, int f32, bool full) {
    if (s.warps + 2 <= 16 && s.per_sm == 1)
        return f32 ? (full ? norm_backward_kernel<true, true, 16> : norm_backward_kernel<true, false, 16>)
                   : (full ? norm_backward_kernel<false, true, 16> : norm_backward_kernel<false, false, 16>);
    return f32 ? (full ? norm_backward_kernel<true, true, 18> : norm_backward_kernel<true, false, 18>)
               : (full ? norm_backward_kernel<false, true, 18> : norm_backward_kernel<false, false, 18>);
}

size_t workspace_bytes(int T, int H) {
    const BackwardShape s = backward_shape(T, H, 0, kMaxSms);
    return ((size_t)s.clusters * (2 * (size_t)H + s.cluster) * sizeof(float) + 15) / 16 * 16;
}

template <bool F32>
cudaError_t launch_rows(const NormParams& p, int num_sms, cudaStream_t stream) {
    const int warps = (p.H / kVec + 31) / 32;
    const dim3 grid((unsigned)std::min(p.T, num_sms)), block(warps * 32 + 32);
    const bool full = p.y != nullptr && p.w_post != nullptr && p.w_pre != nullptr && p.h_out != nullptr;
    const size_t row = (size_t)p.H * (F32 ? 6 : 4);
    const int stages = (int)std::min<size_t>(kMaxStages, kRingBytes / row);
    auto kern = full ? norm_rows_kernel<F32, true> : norm_rows_kernel<F32, false>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
    if (e != cudaSuccess) return e;
    return launch_kernel(false, kern, grid, block, stages * row, stream, p, stages);
}

template <int NV, bool F32>
cudaError_t launch_forward(const NormParams& p, int num_sms, cudaStream_t stream) {
    const int warps = (p.H / kVec + 32 * NV - 1) / (32 * NV);
    // 32 warps on an SM, whole rows
    const dim3 grid((unsigned)std::min<int64_t>(p.T, (int64_t)num_sms * (32 / warps))), block(warps * 32);
    const bool full = p.y != nullptr && p.w_post != nullptr && p.w_pre != nullptr && p.h_out != nullptr;
    // started early, many rows' CTAs take the SMs from the kernel before (forward and backward of T=16384 H=4096 f32: 351
    // against 323 us); a decode batch's, a row to an SM, gain the launch gap
    const bool early = p.T <= num_sms;
    return full ? launch_kernel(early, norm_kernel<NV, F32, true>, grid, block, 0, stream, p)
                : launch_kernel(early, norm_kernel<NV, F32, false>, grid, block, 0, stream, p);
}

}  // namespace

size_t norm_workspace_bytes(int T, int H) { return workspace_bytes(T, H); }

cudaError_t launch_block_norm(const NormParams& p, int num_sms, cudaStream_t stream) {
    // Wide rows, where the other form has one CTA on an SM, and many of them (us, other form | this one: T=16384 H=4096 f32
    // 135 | 128; T=8192 H=5120 bf16 65 | 58, f32 99 | 80; T=4096 H=7168 bf16 42.7 | 41.7, f32 66.5 | 59.5; T=2560 H=7168
    // bf16 28.5 | 29.4; T=700 10.5 | 12.7; T=16384 H=4096 bf16 86 | 98).  H > 7936 leaves no warp for the producer.
    if (p.T >= 20 * num_sms && p.H >= (p.f32 ? 4096 : 4104) && p.H <= 31 * 32 * kVec)
        return p.f32 ? launch_rows<true>(p, num_sms, stream) : launch_rows<false>(p, num_sms, stream);
    if (p.H <= 32 * 32 * kVec) return p.f32 ? launch_forward<1, true>(p, num_sms, stream) : launch_forward<1, false>(p, num_sms, stream);
    return p.f32 ? launch_forward<2, true>(p, num_sms, stream) : launch_forward<2, false>(p, num_sms, stream);
}

cudaError_t launch_block_norm_backward(const NormParams& p, int num_sms, cudaStream_t stream) {
    const BackwardShape s = backward_shape(p.T, p.H, p.f32, num_sms);
    if (s.clusters > 0) {
        const BackwardKernel kern = backward_kernel(s, p.f32, p.y != nullptr && p.d_n != nullptr && p.d_h_out != nullptr);
        const size_t smem = ring_bytes(s, p.f32);
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
        if (e != cudaSuccess) return e;
        e = launch_clusters(true, s.cluster, kern, dim3(s.clusters * s.cluster), dim3(s.warps * 32 + 64), smem, stream, p, s);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((2 * (int64_t)p.H + 31) / 32));
    return launch_kernel(true, norm_columns_kernel, grid, dim3(kColumnWarps * 32), 0, stream, p, s.clusters, s.clusters * s.cluster);
}

}  // namespace ep
