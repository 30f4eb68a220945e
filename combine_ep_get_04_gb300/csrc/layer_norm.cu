// layer_norm.cu -- the residual sum of a block's output after dropout, and the
// layer norm before the next block:
//   h_out = h + (kept ? y * scale : 0)
//   n     = (h_out - mean) * r * w + b,   r = 1 / sqrt(variance + eps)
// and its gradients.  One pass over the rows in each direction; each tensor is
// read and written once, so the kernels are bound by HBM.
#include <algorithm>

#include "block_kernels.h"
#include "dropout.cuh"

namespace ep {
namespace {

constexpr int kMaxStages = 8;
constexpr int kSlots = 4;                         // rows whose sums may be on their way
constexpr int kMaxWarps = 16;                     // consumer warps of a CTA
constexpr int kMaxSms = 192;                      // the workspace has room for this many
constexpr size_t kRingBytes = 212 * 1024;         // shared memory of an SM that the rings may take
constexpr int kColumnWarps = 16;

// A thread has NV vectors of 8 channels, `lanes` vectors apart.
struct RowShape {
    int nv, warps, per_sm, stages, ctas;
};

RowShape row_shape(int T, int H, size_t row_bytes, int num_sms) {
    RowShape s{};
    s.nv = H <= 4096 ? 1 : H <= 8192 ? 2 : 4;
    s.warps = (H / kVec + 32 * s.nv - 1) / (32 * s.nv);
    s.per_sm = s.nv > 1 ? 1 : std::max(1, std::min(8, 20 / (s.warps + 1)));      // 96 registers a thread: 20 warps
    s.ctas = (int)std::min<int64_t>(T, (int64_t)std::min(num_sms, kMaxSms) * s.per_sm);
    s.stages = (int)std::max<size_t>(1, std::min<size_t>(kMaxStages, (kRingBytes / s.per_sm - 2048) / row_bytes));
    return s;
}

// The rows of a CTA are a grid apart.
__device__ __forceinline__ int rows_of_cta(int T) { return (int)blockIdx.x < T ? (T - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0; }

// Sums of two values over a warp, in six shuffles, to all its lanes.
__device__ __forceinline__ float2 warp_sum2(float a, float b) {
    const bool high = threadIdx.x & 16;
    float x = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 16);
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    const float other = __shfl_xor_sync(0xffffffffu, x, 16);
    return high ? make_float2(other, x) : make_float2(x, other);
}

// Of four values, in eight.
__device__ __forceinline__ float4 warp_sum4(float a, float b, float c, float d) {
    const bool high = threadIdx.x & 16, second = threadIdx.x & 8;
    const float x = (high ? b : a) + __shfl_xor_sync(0xffffffffu, high ? a : b, 16);
    const float y = (high ? d : c) + __shfl_xor_sync(0xffffffffu, high ? c : d, 16);
    float z = (second ? y : x) + __shfl_xor_sync(0xffffffffu, second ? x : y, 8);
#pragma unroll
    for (int i = 4; i >= 1; i >>= 1) z += __shfl_xor_sync(0xffffffffu, z, i);
    return make_float4(__shfl_sync(0xffffffffu, z, 0), __shfl_sync(0xffffffffu, z, 16), __shfl_sync(0xffffffffu, z, 8), __shfl_sync(0xffffffffu, z, 24));
}

// Channels of a row that belong to warp w.
template <int NV>
__device__ __forceinline__ int warp_channels(int w, int warps, int vecs) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) n += max(0, min(32, vecs - (i * warps + w) * 32));
    return n * kVec;
}

__device__ __forceinline__ Vec8 round_bf16(const Vec8& x) {
    Vec8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = halves(x.v[i]);
        const uint32_t w = pack_bf16x2(f.x, f.y);
        r.v[i] = pair(bf16_lo(w), bf16_hi(w));
    }
    return r;
}

// ----------------------------------------------------------------- forward
//
// A producer warp keeps a ring of rows (h, y) filled by bulk copies.  A row is
// taken up in two turns.  Turn i sums row i, writes its h_out and leaves each
// warp's sum and squared deviations from the warp's own mean; beside that row
// i - 1, whose warps' values are all there by now, is normed from registers, so
// that no warp stands still at a row's end.  The warps' moments join by
//   M2 = sum over warps of M2_w + n_w (mean_w - mean)^2,
// which never subtracts large squares from each other.
//
// T=16384 H=4096 fp32 with dropout 132 us, 6.1 TB/s, 91 % of the measured copy rate;
// T=4096 H=7168 bf16 40.5 us, 5.8 TB/s, with dropout 56 us, 4.2 TB/s: 310 instructions
// a vector of a warp, twenty of them the generator's wide products, with 14 warps to
// hide each other's waits.  (The two rows' sums each in chains of their own: 63 us;
// twice the warps with half the registers 60, spilled ones among them; keys of the
// rounds in shared memory 61.)
template <int NV, bool F32, bool DROP, int THREADS>
__global__ void __launch_bounds__(THREADS) layer_norm_kernel(LayerNormParams p, int warps, int stages) {
    extern __shared__ __align__(128) unsigned char ring[];       // [stages][h, y]
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], summed[kSlots];
    __shared__ float2 moments[kSlots][kMaxWarps];
    constexpr int kStream = F32 ? 4 : 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool has_y = DROP || p.y != nullptr;
    const int at_y = p.H * kStream, stage_bytes = at_y + (has_y ? p.H * 2 : 0);
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], warps);
        }
        for (int i = 0; i < kSlots; ++i) mbar_init(&summed[i], warps);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    const int rows = rows_of_cta(p.T);
    bool good = true;
    if (warp == warps) {
        const unsigned char* h = static_cast<const unsigned char*>(p.h) + (int64_t)blockIdx.x * p.ld_h * kStream;
        const unsigned char* y = static_cast<const unsigned char*>(p.y) + (int64_t)blockIdx.x * p.ld_y * 2;
        int filled = 0, st = 0;
        uint32_t parity = 1;                      // of the stage's previous use
        for (; filled < rows; ++filled) {
            if (filled >= stages && !__all_sync(0xffffffffu, mbar_wait(&empty[st], parity))) {
                good = false;
                break;
            }
            if (lane == 0) {
                unsigned char* to = ring + st * stage_bytes;
                mbar_arrive_expect_tx(&full[st], stage_bytes);
                bulk_load(to, h, at_y, &full[st]);
                if (has_y) bulk_load(to + at_y, y, p.H * 2, &full[st]);
            }
            __syncwarp();
            h += gridDim.x * p.ld_h * kStream;
            y += gridDim.x * p.ld_y * 2;
            if (++st == stages) {
                st = 0;
                parity ^= 1;
            }
        }
        // no copy may be in flight when the CTA ends, whatever its consumers did
        for (int i = max(0, filled - stages); i < filled; ++i) mbar_wait(&full[i % stages], (i / stages) & 1);
    } else {
        const int lanes = warps * 32, vecs = p.H / kVec;
        bool in[NV] = {};
        int at[NV] = {};
        Vec8 w[NV], b[NV];
        auto load_weights = [&](int i) {
            w[i] = in[i] && p.w != nullptr ? load_f32(p.w, at[i]) : all(1.f);
            b[i] = in[i] && p.b != nullptr ? load_f32(p.b, at[i]) : all(0.f);
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * lanes;
            in[i] = v < vecs;
            at[i] = in[i] ? v * kVec : 0;
            if (NV <= 2) load_weights(i);
        }
        const int mine = warp_channels<NV>(warp, warps, vecs), theirs = lane < warps ? warp_channels<NV>(lane, warps, vecs) : 0;
        const float inv_mine = mine > 0 ? 1.f / (float)mine : 0.f, n_theirs = (float)theirs, inv_theirs = theirs > 0 ? 1.f / n_theirs : 0.f;
        const float inv_h = 1.f / (float)p.H;
        Counters ctr{};
        if (DROP) ctr = counters(p.drop);
        Vec8 z[NV];
        int st = 0;
        uint32_t parity = 0, summed_parity = 0;
        int64_t t = blockIdx.x;
        for (int i = 0; i <= rows; ++i, t += gridDim.x) {
            Vec8 before[NV];
#pragma unroll
            for (int k = 0; k < NV; ++k) before[k] = z[k];
            uint64_t sum = both(0.f);
            if (i < rows) {
                good = __all_sync(0xffffffffu, mbar_wait(&full[st], parity));
                if (!good) break;
                const unsigned char* row = ring + st * stage_bytes;
                Vec8 y[NV];
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    z[k] = in[k] ? load_stream<F32>(row, at[k]) : all(0.f);
                    y[k] = in[k] && has_y ? load_bf16(row + at_y, at[k]) : all(0.f);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
                if (++st == stages) {
                    st = 0;
                    parity ^= 1;
                }
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    if (DROP) apply(y[k], random_bits((uint64_t)t * vecs + threadIdx.x + k * lanes, ctr), p.drop);
                    if (has_y) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) z[k].v[c] = add2(z[k].v[c], y[k].v[c]);
                        if (!F32) z[k] = round_bf16(z[k]);
                        if (in[k]) store_stream<F32>(p.h_out, t * p.H + at[k], z[k]);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) sum = add2(sum, z[k].v[c]);
                }
            }
            // row i's first sum with row i - 1's last join, whose chains of shuffles are then one
            float2 m = make_float2(0.f, 0.f);
            if (i > 0) {
                const int slot = (i - 1) % kSlots;
                good = __all_sync(0xffffffffu, mbar_wait(&summed[slot], summed_parity));
                if (!good) break;
                if (slot == kSlots - 1) summed_parity ^= 1;
                if (lane < warps) m = moments[slot][lane];
            }
            const float2 first = warp_sum2(total(sum), m.x);
            const float mean = first.y * inv_h, off = fmaf(-n_theirs, mean, m.x);
            const uint64_t from_own = both(-first.x * inv_mine);
            uint64_t squares = both(0.f);
            if (i < rows)
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (in[k])
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint64_t d = add2(z[k].v[c], from_own);
                            squares = fma2(d, d, squares);
                        }
            const float2 second = warp_sum2(total(squares), fmaf(off * off, inv_theirs, m.y));
            if (i < rows && lane == 0) {
                moments[i % kSlots][warp] = make_float2(first.x, second.x);
                mbar_arrive(&summed[i % kSlots]);
            }
            if (i > 0) {
                const float r = rsqrtf(fmaf(second.y, inv_h, p.eps));
                const int64_t from = t - gridDim.x;
                if (threadIdx.x == 0 && p.stats != nullptr) {
                    p.stats[from] = mean;
                    p.stats[p.T + from] = r;
                }
                const uint64_t less = both(-mean), r2 = both(r);
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    if (NV > 2) load_weights(k);
                    Vec8 n;
#pragma unroll
                    for (int c = 0; c < 4; ++c) n.v[c] = fma2(mul2(add2(before[k].v[c], less), r2), w[k].v[c], b[k].v[c]);
                    if (in[k]) store_bf16(p.n, from * p.H + at[k], n);
                }
            }
        }
    }
    if (!good && lane == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrTimeout);
}

// ---------------------------------------------------------------- backward
//
// With xn = (h_out - mean) r and t = d_n w:
//   d   = d_h_out + r (t - mean(t) - xn mean(t xn)),   d_h = d,   d_y = d as dropout takes it
//   d_w = sum over rows of d_n xn,   d_b = sum over rows of d_n
// Turn i leaves each warp's two sums of row i; then row i - lag, whose sums are
// all there by now, is read from the ring once more and finished.  A thread
// keeps its channels' weights and their sums over rows in registers for all the
// rows of its CTA; the CTAs' sums go to the workspace once and
// layer_norm_columns_kernel adds them in CTA order, so that nothing depends on
// the order in which CTAs run.
//
// T=16384 H=4096 fp32 with dropout 174 us, 6.2 TB/s, 92 %; T=4096 H=7168 bf16 57 us,
// 5.1 TB/s: as above.
template <int NV, bool F32, bool DROP, int THREADS>
__global__ void __launch_bounds__(THREADS) layer_norm_backward_kernel(LayerNormParams p, int warps, int stages) {
    extern __shared__ __align__(128) unsigned char ring[];       // [stages][h_out, d_h_out, d_n]
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], summed[kSlots];
    __shared__ float2 sums[kSlots][kMaxWarps];
    __shared__ float2 row_stats[kMaxStages];
    constexpr int kStream = F32 ? 4 : 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool has_dh = p.d_h_out != nullptr;
    const int wide = p.H * kStream, narrow = p.H * 2, at_dn = 2 * wide, stage_bytes = at_dn + narrow;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], warps);
        }
        for (int i = 0; i < kSlots; ++i) mbar_init(&summed[i], warps);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    const int rows = rows_of_cta(p.T);
    const int lag = stages > 1 ? 1 : 0;
    bool good = true;
    if (warp == warps) {
        int filled = 0, st = 0;
        uint32_t parity = 1;
        // the next row's statistics are on their way while a stage is waited for
        float mean = 0.f, r = 0.f;
        auto look_up = [&](int i) {
            const int64_t t = blockIdx.x + (int64_t)i * gridDim.x;
            if (lane == 0 && i < rows) {
                mean = p.stats[t];
                r = p.stats[p.T + t];
            }
        };
        look_up(0);
        for (; filled < rows; ++filled) {
            if (filled >= stages && !__all_sync(0xffffffffu, mbar_wait(&empty[st], parity))) {
                good = false;
                break;
            }
            const int64_t t = blockIdx.x + (int64_t)filled * gridDim.x;
            if (lane == 0) {
                unsigned char* to = ring + st * stage_bytes;
                mbar_expect_tx(&full[st], wide + (has_dh ? wide : 0) + narrow);
                bulk_load(to, static_cast<const unsigned char*>(p.h) + t * p.ld_h * kStream, wide, &full[st]);
                if (has_dh) bulk_load(to + wide, static_cast<const unsigned char*>(p.d_h_out) + t * wide, wide, &full[st]);
                bulk_load(to + at_dn, static_cast<const unsigned char*>(p.d_n) + t * narrow, narrow, &full[st]);
                row_stats[st] = make_float2(mean, r);
                mbar_arrive(&full[st]);           // after the row's statistics are written
            }
            __syncwarp();
            look_up(filled + 1);
            if (++st == stages) {
                st = 0;
                parity ^= 1;
            }
        }
        for (int i = max(0, filled - stages); i < filled; ++i) mbar_wait(&full[i % stages], (i / stages) & 1);
    } else {
        const int lanes = warps * 32, vecs = p.H / kVec;
        bool in[NV] = {};
        int at[NV] = {};
        Vec8 w[NV], s_w[NV], s_b[NV];
        auto load_weights = [&](int k) { w[k] = !in[k] ? all(0.f) : p.w != nullptr ? load_f32(p.w, at[k]) : all(1.f); };
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = threadIdx.x + k * lanes;
            in[k] = v < vecs;                     // the others go through it with weights of 0 and store nothing
            at[k] = in[k] ? v * kVec : 0;
            s_w[k] = s_b[k] = all(0.f);
            if (NV <= 2) load_weights(k);
        }
        const float inv_h = 1.f / (float)p.H;
        Counters ctr{};
        if (DROP) ctr = counters(p.drop);
        int st1 = 0, st2 = 0;
        uint32_t full_parity = 0, summed_parity = 0;
        for (int i = 0; i < rows + lag; ++i) {
            uint64_t sum0 = both(0.f), sum1 = sum0;
            if (i < rows) {
                good = __all_sync(0xffffffffu, mbar_wait(&full[st1], full_parity));
                if (!good) break;
                const unsigned char* row = ring + st1 * stage_bytes;
                const float2 rs = row_stats[st1];
                const uint64_t less = both(-rs.x), r = both(rs.y);
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    if (NV > 2) load_weights(k);
                    // 0 where a thread has no channels: a weight of 0 alone would make NaN of an infinity
                    const Vec8 x = load_stream<F32>(row, at[k]), dn = in[k] ? load_bf16(row + at_dn, at[k]) : all(0.f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint64_t xn = mul2(add2(x.v[c], less), r), t = mul2(dn.v[c], w[k].v[c]);
                        s_w[k].v[c] = fma2(dn.v[c], xn, s_w[k].v[c]);
                        s_b[k].v[c] = add2(dn.v[c], s_b[k].v[c]);
                        sum0 = add2(t, sum0);
                        sum1 = fma2(t, xn, sum1);
                    }
                }
                if (++st1 == stages) {
                    st1 = 0;
                    full_parity ^= 1;
                }
            }
            // the sums of a row and of the one `lag` before, whose warps' sums are there by now, in one chain of shuffles
            auto leave = [&](float a, float b) {
                if (lane == 0) {
                    sums[i % kSlots][warp] = make_float2(a, b);
                    mbar_arrive(&summed[i % kSlots]);
                }
            };
            auto others = [&]() {
                const int slot = (i - lag) % kSlots;
                good = __all_sync(0xffffffffu, mbar_wait(&summed[slot], summed_parity));
                if (slot == kSlots - 1) summed_parity ^= 1;
                return good && lane < warps ? sums[slot][lane] : make_float2(0.f, 0.f);
            };
            float2 s;
            if (lag == 0) {
                const float2 own = warp_sum2(total(sum0), total(sum1));
                leave(own.x, own.y);
                const float2 part = others();
                if (!good) break;
                s = warp_sum2(part.x, part.y);
            } else {
                float2 part = make_float2(0.f, 0.f);
                if (i > 0) {
                    part = others();
                    if (!good) break;
                }
                const float4 four = warp_sum4(total(sum0), total(sum1), part.x, part.y);
                if (i < rows) leave(four.x, four.y);
                s = make_float2(four.z, four.w);
            }
            if (i >= lag) {
                const float m1 = s.x * inv_h, m2 = s.y * inv_h;
                const unsigned char* row = ring + st2 * stage_bytes;
                const float2 rs = row_stats[st2];
                const uint64_t less = both(-rs.x), r = both(rs.y), minus_m1 = both(-m1), minus_m2 = both(-m2);
                const int64_t t_row = blockIdx.x + (int64_t)(i - lag) * gridDim.x;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    if (NV > 2) load_weights(k);
                    const Vec8 x = load_stream<F32>(row, at[k]), dn = load_bf16(row + at_dn, at[k]);
                    const Vec8 dh = has_dh ? load_stream<F32>(row + wide, at[k]) : all(0.f);
                    Vec8 d;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint64_t xn = mul2(add2(x.v[c], less), r), t = mul2(dn.v[c], w[k].v[c]);
                        d.v[c] = fma2(r, fma2(minus_m2, xn, add2(t, minus_m1)), dh.v[c]);
                    }
                    if (in[k]) {
                        store_stream<F32>(p.d_h, t_row * p.H + at[k], d);
                        if (DROP) apply(d, random_bits((uint64_t)t_row * vecs + threadIdx.x + k * lanes, ctr), p.drop);
                        if (p.d_y != nullptr) store_bf16(p.d_y, t_row * p.H + at[k], d);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st2]);
                if (++st2 == stages) st2 = 0;
            }
        }
        float* out = p.partial + (int64_t)blockIdx.x * 2 * p.H;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (in[k]) {
                store_f32(out, at[k], s_w[k]);
                store_f32(out, p.H + at[k], s_b[k]);
            }
    }
    if (!good && lane == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrTimeout);
}

// ------------------------------------------------------------- narrow rows
//
// A warp takes a row by itself: no barrier, no join, and as many rows on their
// way as an SM has warps.  NV vectors of 8 channels a lane; rows are dealt to the
// CTAs first, then to their warps.  As far as the registers hold a row (backward,
// the two sums over rows too).  T=65536, us, in brackets by the ring:
//
//                    bf16                     fp32
//   forward          no dropout   dropout     no dropout   dropout
//   H=256            30  (59)     31  (70)    37  (59)     37  (69)
//   H=512            49  (78)     54  (92)    64  (85)     65  (91)
//   H=1024           92 (151)    102 (140)   123 (131)    125 (138)
//   backward with the column sums
//   H=256            44  (85)     51  (90)    55  (67)     57  (89)
//   H=512            72  (83)    102 (136)    89  (85)    103 (140)
//
// H=1024 backward by a warp: 262 and 348 us bf16, 330 and 348 fp32, its sums spilled;
// by the ring 115 and 153, 174 and 242.

constexpr int kNarrow = 1024, kNarrowBackward = 512;

// Warps of a CTA, one CTA an SM, as many as the registers hold.
constexpr int narrow_warps(int nv, bool backward) { return backward ? nv == 1 ? 24 : 16 : nv == 1 ? 32 : nv == 2 ? 24 : 16; }

template <int NV, bool F32>
__device__ __forceinline__ void load_row(Vec8 (&x)[NV], const unsigned char* row, int vecs, int lane) {
#pragma unroll
    for (int k = 0; k < NV; ++k) x[k] = lane + 32 * k < vecs ? load_stream<F32>(row, (lane + 32 * k) * kVec) : all(0.f);
}

template <int NV, bool F32, bool DROP>
__global__ void __launch_bounds__(narrow_warps(NV, false) * 32) layer_norm_narrow_kernel(LayerNormParams p) {
    constexpr int kStream = F32 ? 4 : 2;
    const int lane = threadIdx.x & 31, vecs = p.H / kVec;
    const bool has_y = DROP || p.y != nullptr;
    const float inv_h = 1.f / (float)p.H;
    pdl_launch_dependents();
    pdl_wait();
    Counters ctr{};
    if (DROP) ctr = counters(p.drop);
    const int64_t apart = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t t = blockIdx.x + (int64_t)gridDim.x * (threadIdx.x >> 5); t < p.T; t += apart) {
        Vec8 z[NV], y[NV];
        load_row<NV, F32>(z, static_cast<const unsigned char*>(p.h) + t * p.ld_h * kStream, vecs, lane);
        if (has_y) load_row<NV, false>(y, static_cast<const unsigned char*>(p.y) + t * p.ld_y * 2, vecs, lane);
        uint64_t sum = both(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = lane + 32 * k;
            if (DROP) apply(y[k], random_bits((uint64_t)t * vecs + v, ctr), p.drop);
            if (has_y) {
#pragma unroll
                for (int c = 0; c < 4; ++c) z[k].v[c] = add2(z[k].v[c], y[k].v[c]);
                if (!F32) z[k] = round_bf16(z[k]);
                if (v < vecs) store_stream<F32>(p.h_out, t * p.H + v * kVec, z[k]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) sum = add2(sum, z[k].v[c]);
        }
        const float mean = warp_sum(total(sum)) * inv_h;
        const uint64_t less = both(-mean);
        uint64_t squares = both(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const bool in = lane + 32 * k < vecs;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                z[k].v[c] = in ? add2(z[k].v[c], less) : both(0.f);
                squares = fma2(z[k].v[c], z[k].v[c], squares);
            }
        }
        const float r = rsqrtf(fmaf(warp_sum(total(squares)), inv_h, p.eps));
        if (lane == 0 && p.stats != nullptr) {
            p.stats[t] = mean;
            p.stats[p.T + t] = r;
        }
        const uint64_t r2 = both(r);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = (lane + 32 * k) * kVec;
            if (at >= p.H) continue;
            const Vec8 w = p.w != nullptr ? load_f32(p.w, at) : all(1.f), b = p.b != nullptr ? load_f32(p.b, at) : all(0.f);
            Vec8 n;
#pragma unroll
            for (int c = 0; c < 4; ++c) n.v[c] = fma2(mul2(z[k].v[c], r2), w.v[c], b.v[c]);
            store_bf16(p.n, t * p.H + at, n);
        }
    }
}

template <int NV, bool F32, bool DROP>
__global__ void __launch_bounds__(narrow_warps(NV, true) * 32) layer_norm_narrow_backward_kernel(LayerNormParams p) {
    extern __shared__ __align__(128) unsigned char ring[];       // [warps][2 H] column sums
    constexpr int kStream = F32 ? 4 : 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, vecs = p.H / kVec;
    const float inv_h = 1.f / (float)p.H;
    pdl_launch_dependents();
    pdl_wait();
    Counters ctr{};
    if (DROP) ctr = counters(p.drop);
    Vec8 s_w[NV], s_b[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) s_w[k] = s_b[k] = all(0.f);
    const int64_t apart = (int64_t)gridDim.x * warps;
    for (int64_t t = blockIdx.x + (int64_t)gridDim.x * warp; t < p.T; t += apart) {
        Vec8 x[NV], dn[NV], dh[NV];
        load_row<NV, F32>(x, static_cast<const unsigned char*>(p.h) + t * p.ld_h * kStream, vecs, lane);
        load_row<NV, false>(dn, static_cast<const unsigned char*>(p.d_n) + t * p.H * 2, vecs, lane);
        if (p.d_h_out != nullptr) {
            load_row<NV, F32>(dh, static_cast<const unsigned char*>(p.d_h_out) + t * p.H * kStream, vecs, lane);
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) dh[k] = all(0.f);
        }
        const uint64_t less = both(-p.stats[t]), r = both(p.stats[p.T + t]);
        uint64_t sum0 = both(0.f), sum1 = sum0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = (lane + 32 * k) * kVec;
            const Vec8 w = at >= p.H ? all(0.f) : p.w != nullptr ? load_f32(p.w, at) : all(1.f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[k].v[c] = mul2(add2(x[k].v[c], less), r);
                s_w[k].v[c] = fma2(dn[k].v[c], x[k].v[c], s_w[k].v[c]);
                s_b[k].v[c] = add2(dn[k].v[c], s_b[k].v[c]);
                dn[k].v[c] = mul2(dn[k].v[c], w.v[c]);
                sum0 = add2(dn[k].v[c], sum0);
                sum1 = fma2(dn[k].v[c], x[k].v[c], sum1);
            }
        }
        const float2 s = warp_sum2(total(sum0), total(sum1));
        const uint64_t minus_m1 = both(-s.x * inv_h), minus_m2 = both(-s.y * inv_h);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = lane + 32 * k;
            if (v >= vecs) continue;
            Vec8 d;
#pragma unroll
            for (int c = 0; c < 4; ++c) d.v[c] = fma2(r, fma2(minus_m2, x[k].v[c], add2(dn[k].v[c], minus_m1)), dh[k].v[c]);
            store_stream<F32>(p.d_h, t * p.H + v * kVec, d);
            if (DROP) apply(d, random_bits((uint64_t)t * vecs + v, ctr), p.drop);
            if (p.d_y != nullptr) store_bf16(p.d_y, t * p.H + v * kVec, d);
        }
    }
    // the warps' sums over rows, in their order
    float* parts = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int at = (lane + 32 * k) * kVec;
        if (at >= p.H) continue;
        store_f32(parts + (int64_t)warp * 2 * p.H, at, s_w[k]);
        store_f32(parts + (int64_t)warp * 2 * p.H, p.H + at, s_b[k]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.H; c += blockDim.x) {
        float sum = 0.f;
        for (int i = 0; i < warps; ++i) sum += parts[i * 2 * p.H + c];
        p.partial[(int64_t)blockIdx.x * 2 * p.H + c] = sum;
    }
}

// Adds `groups` rows of column sums.  A CTA takes 32 columns; each warp adds
// every kColumnWarps-th row, then the warps' sums are added in order.
__global__ void __launch_bounds__(kColumnWarps * 32) layer_norm_columns_kernel(LayerNormParams p, int groups) {
    __shared__ float part[kColumnWarps][32];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t width = 2 * (int64_t)p.H;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < width)
#pragma unroll 8
        for (int r = warp; r < groups; r += kColumnWarps) s += p.partial[r * width + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < width) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < kColumnWarps; ++i) s += part[i][lane];
        if (c < p.H) {
            if (p.d_w != nullptr) p.d_w[c] = s;
        } else if (p.d_b != nullptr) {
            p.d_b[c - p.H] = s;
        }
    }
}

using Kernel = void (*)(LayerNormParams, int, int);
using Kernel1 = void (*)(LayerNormParams);

// 16 warps with the producer's have 128 registers a thread, 17 have 96.
template <int NV, bool F32, bool DROP>
Kernel kernel_of(bool backward, int warps) {
    if constexpr (NV > 1)
        if (warps < 16) return backward ? layer_norm_backward_kernel<NV, F32, DROP, 512> : layer_norm_kernel<NV, F32, DROP, 512>;
    return backward ? layer_norm_backward_kernel<NV, F32, DROP, 544> : layer_norm_kernel<NV, F32, DROP, 544>;
}

template <bool F32, bool DROP>
Kernel kernel_of(bool backward, int nv, int warps) {
    return nv == 1 ? kernel_of<1, F32, DROP>(backward, warps) : nv == 2 ? kernel_of<2, F32, DROP>(backward, warps) : kernel_of<4, F32, DROP>(backward, warps);
}

cudaError_t launch_rows(const LayerNormParams& p, const RowShape& s, bool backward, size_t row_bytes, cudaStream_t stream) {
    const bool drop = p.drop.rng != nullptr;
    const Kernel kern = p.f32 ? (drop ? kernel_of<true, true>(backward, s.nv, s.warps) : kernel_of<true, false>(backward, s.nv, s.warps))
                              : (drop ? kernel_of<false, true>(backward, s.nv, s.warps) : kernel_of<false, false>(backward, s.nv, s.warps));
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
    if (e != cudaSuccess) return e;
    return launch_kernel(true, kern, dim3(s.ctas), dim3(s.warps * 32 + 32), s.stages * row_bytes, stream, p, s.warps, s.stages);
}

template <bool F32, bool DROP>
Kernel1 narrow_kernel(bool backward, int nv) {
    if (backward) return nv == 1 ? layer_norm_narrow_backward_kernel<1, F32, DROP> : layer_norm_narrow_backward_kernel<2, F32, DROP>;
    return nv == 1 ? layer_norm_narrow_kernel<1, F32, DROP> : nv == 2 ? layer_norm_narrow_kernel<2, F32, DROP> : layer_norm_narrow_kernel<4, F32, DROP>;
}

// *ctas: of the grid.
cudaError_t launch_narrow(const LayerNormParams& p, int num_sms, bool backward, int* ctas, cudaStream_t stream) {
    const int nv = p.H <= 256 ? 1 : p.H <= 512 ? 2 : 4, ctas_now = std::min(p.T, std::min(num_sms, kMaxSms));
    // no more warps than rows
    const int warps = std::min(narrow_warps(nv, backward), (p.T - 1) / ctas_now + 1);
    const bool drop = p.drop.rng != nullptr;
    const Kernel1 kern = p.f32 ? (drop ? narrow_kernel<true, true>(backward, nv) : narrow_kernel<true, false>(backward, nv))
                               : (drop ? narrow_kernel<false, true>(backward, nv) : narrow_kernel<false, false>(backward, nv));
    const size_t smem = backward ? (size_t)warps * 2 * p.H * sizeof(float) : 0;
    if (backward) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, narrow_warps(nv, true) * 2 * 256 * nv * (int)sizeof(float));
        if (e != cudaSuccess) return e;
    }
    *ctas = ctas_now;
    return launch_kernel(true, kern, dim3(ctas_now), dim3(warps * 32), smem, stream, p);
}

}  // namespace

size_t layer_norm_workspace_bytes(int T, int H) { return (size_t)row_shape(T, H, 1, kMaxSms).ctas * 2 * H * sizeof(float); }

cudaError_t launch_layer_norm(const LayerNormParams& p, int num_sms, cudaStream_t stream) {
    int ctas;
    if (p.H <= kNarrow) return launch_narrow(p, num_sms, false, &ctas, stream);
    const size_t row = (size_t)p.H * ((p.f32 ? 4 : 2) + (p.y != nullptr ? 2 : 0));
    return launch_rows(p, row_shape(p.T, p.H, row, num_sms), false, row, stream);
}

cudaError_t launch_layer_norm_backward(const LayerNormParams& p, int num_sms, cudaStream_t stream) {
    int ctas = 0;
    if (p.T > 0) {
        cudaError_t e;
        if (p.H <= kNarrowBackward) {
            e = launch_narrow(p, num_sms, true, &ctas, stream);
        } else {
            const size_t row = (size_t)p.H * (p.f32 ? 10 : 6);
            const RowShape s = row_shape(p.T, p.H, row, num_sms);
            ctas = s.ctas;
            e = launch_rows(p, s, true, row, stream);
        }
        if (e != cudaSuccess) return e;
    }
    if (p.d_w == nullptr && p.d_b == nullptr) return cudaSuccess;
    return launch_kernel(true, layer_norm_columns_kernel, dim3((unsigned)((2 * (int64_t)p.H + 31) / 32)), dim3(kColumnWarps * 32), 0, stream, p, ctas);
}

}  // namespace ep
