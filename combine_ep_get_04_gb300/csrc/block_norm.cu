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

// Backward.  Each CTA walks rows a grid apart and keeps its sums over rows
// (d_w_post, d_w_pre, a channel gate's gradient) in registers, in fp32; they
// go to the workspace once, and norm_columns_kernel adds the CTAs' sums in
// CTA order, so that nothing depends on the order in which CTAs run.
template <int NV, bool F32, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_backward_kernel(NormParams p, RowShape shape) {
    __shared__ float red1[32], red2[32], red3[32];
    extern __shared__ float col[];   // [3][H] when a CTA works on several rows at once
    pdl_launch_dependents();
    pdl_wait();
    const int lanes = shape.warps * 32;
    const int sub = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int vecs = p.H / kVec;
    const float inv_h = 1.f / (float)p.H;
    const float scale = p.res_scale != nullptr ? *p.res_scale : 1.f;
    Vec8 s_post[NV], s_gate[NV], s_pre[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) s_post[i] = s_gate[i] = s_pre[i] = zeros();
    float s_scale = 0.f;
    for (int64_t t0 = (int64_t)blockIdx.x * shape.rows; t0 < p.T; t0 += (int64_t)gridDim.x * shape.rows) {
        const int64_t t = t0 + sub;
        const bool live = t < p.T;
        const float r1 = live && p.w_post != nullptr ? p.rstd[t] : 1.f;
        const float r2 = live && p.w_pre != nullptr ? p.rstd[p.T + t] : 0.f;
        const float token_gate = live && p.gate_kind == kGateToken ? p.gate[t] : 1.f;
        Vec8 h[NV], y[NV], dn[NV], dh[NV];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * lanes;
            const bool in = live && v < vecs;
            h[i] = in ? load_stream<F32>(p.h, t * p.ld_h + v * kVec) : zeros();
            y[i] = in && p.y != nullptr ? load_bf16(p.y, t * p.ld_y + v * kVec) : zeros();
            dn[i] = in && p.d_n != nullptr ? load_bf16(p.d_n, t * p.H + v * kVec) : zeros();
            dh[i] = in && p.d_h_out != nullptr ? load_stream<F32>(p.d_h_out, t * p.H + v * kVec) : zeros();
        }
        // hn takes the place of nothing: it is kept beside h, whose gradient needs both
        Vec8 hn[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * lanes;
            const bool in = live && v < vecs;
            const Vec8 w = in && p.w_post != nullptr ? load_f32(p.w_post, v * kVec) : ones();
            const Vec8 g = in && p.gate_kind == kGateChannel ? load_f32(p.gate, v * kVec) : ones();
            const Vec8 q = in && p.w_pre != nullptr ? load_f32(p.w_pre, v * kVec) : zeros();
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                y[i].v[c] *= r1;
                const float u = y[i].v[c] * w.v[c];
                hn[i].v[c] = r2 * fmaf(scale, h[i].v[c], token_gate * g.v[c] * u);
                s_pre[i].v[c] = fmaf(dn[i].v[c], hn[i].v[c], s_pre[i].v[c]);
                dn[i].v[c] *= q.v[c];
                dot = fmaf(dn[i].v[c], hn[i].v[c], dot);
            }
        }
        const float m2 = p.w_pre != nullptr ? row_sum(dot, red1, shape.warps) * inv_h : 0.f;
        float dot_y = 0.f, dot_g = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * lanes;
            const bool in = live && v < vecs;
            const Vec8 w = in && p.w_post != nullptr ? load_f32(p.w_post, v * kVec) : ones();
            const Vec8 g = in && p.gate_kind == kGateChannel ? load_f32(p.gate, v * kVec) : ones();
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
                const float d = fmaf(r2, dn[i].v[c] - hn[i].v[c] * m2, dh[i].v[c]);
                s_scale = fmaf(d, h[i].v[c], s_scale);
                const float u = y[i].v[c] * w.v[c];
                s_gate[i].v[c] = fmaf(d, u, s_gate[i].v[c]);
                dot_g = fmaf(d, u, dot_g);
                h[i].v[c] = scale * d;
                const float du = token_gate * g.v[c] * d;
                s_post[i].v[c] = fmaf(du, y[i].v[c], s_post[i].v[c]);
                dn[i].v[c] = du * w.v[c];
                dot_y = fmaf(dn[i].v[c], y[i].v[c], dot_y);
            }
            if (in) store_stream<F32>(p.d_h, t * p.H + v * kVec, h[i]);
        }
        const float m1 = p.w_post != nullptr ? row_sum(dot_y, red2, shape.warps) * inv_h : 0.f;
        if (p.gate_kind == kGateToken) {
            const float sum = row_sum(dot_g, red3, shape.warps);
            if (live && lane == 0) p.d_gate[t] = sum;
        }
        if (p.d_y != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = lane + i * lanes;
                if (!live || v >= vecs) continue;
                Vec8 d;
#pragma unroll
                for (int c = 0; c < kVec; ++c) d.v[c] = r1 * (dn[i].v[c] - y[i].v[c] * m1);
                store_bf16(p.d_y, t * p.H + v * kVec, d);
            }
        }
        // the next row's sums reuse the arrays that this row's last readers may still read
        if (shape.warps > 1) __syncthreads();
    }
    // the CTA's sums: rows worked on side by side are added in their order
    float* out = p.partial + (int64_t)blockIdx.x * 3 * p.H;
    for (int r = 0; r < shape.rows; ++r) {
        if (sub == r) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = lane + i * lanes;
                if (v >= vecs) continue;
                float* to[3] = {col + v * kVec, col + p.H + v * kVec, col + 2 * p.H + v * kVec};
                const Vec8* from[3] = {&s_post[i], &s_gate[i], &s_pre[i]};
#pragma unroll
                for (int a = 0; a < 3; ++a) {
                    if (shape.rows == 1) {
                        store_f32(out, (int64_t)a * p.H + v * kVec, *from[a]);
                        continue;
                    }
#pragma unroll
                    for (int c = 0; c < kVec; ++c) to[a][c] = (r == 0 ? 0.f : to[a][c]) + from[a]->v[c];
                }
            }
        }
        if (shape.rows > 1) __syncthreads();
    }
    if (shape.rows > 1)
        for (int i = threadIdx.x; i < 3 * p.H; i += blockDim.x) out[i] = col[i];
    if (p.d_res_scale != nullptr) {
        s_scale = warp_sum(s_scale);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red1[threadIdx.x >> 5] = s_scale;
        __syncthreads();
        if (threadIdx.x == 0) {
            float s = 0.f;
            for (int i = 0; i < (int)blockDim.x / 32; ++i) s += red1[i];
            p.partial[(int64_t)gridDim.x * 3 * p.H + blockIdx.x] = s;
        }
    }
}

// Adds `ctas` rows of column sums.  A CTA takes 32 columns; its 8 warps add
// every eighth row, then the eight sums are added in order.
__global__ void __launch_bounds__(256) norm_columns_kernel(NormParams p, int ctas) {
    __shared__ float part[8][32];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t width = 3 * (int64_t)p.H;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < width)
        for (int r = warp; r < ctas; r += 8) s += p.partial[r * width + c];
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
        for (int r = lane; r < ctas; r += 32) s += p.partial[ctas * width + r];
        s = warp_sum(s);
        if (lane == 0) *p.d_res_scale = s;
    }
}

// One CTA on each SM; never more than the workspace has room for.
constexpr int kMaxBackwardCtas = 192;

int backward_ctas(int T, int rows, int num_sms) {
    return (int)std::min<int64_t>(((int64_t)T + rows - 1) / rows, std::min(num_sms, kMaxBackwardCtas));
}

}  // namespace

size_t norm_workspace_bytes(int T, int H) {
    const RowShape s = row_shape(H, 2, 8);
    const size_t ctas = (size_t)backward_ctas(T, s.rows, kMaxBackwardCtas);
    return (ctas * (3 * (size_t)H + 1) * sizeof(float) + 15) / 16 * 16;
}

cudaError_t launch_block_norm(const NormParams& p, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    const RowShape s = row_shape(p.H, 2, 4);
    const dim3 grid((unsigned)(((int64_t)p.T + s.rows - 1) / s.rows)), block(s.warps * 32 * s.rows);
    return p.f32 ? launch_kernel(true, norm_kernel<2, true>, grid, block, 0, stream, p, s)
                 : launch_kernel(true, norm_kernel<2, false>, grid, block, 0, stream, p, s);
}

cudaError_t launch_block_norm_backward(const NormParams& p, int num_sms, cudaStream_t stream) {
    const RowShape s = row_shape(p.H, 2, 8);
    const int ctas = backward_ctas(p.T, s.rows, num_sms);
    if (ctas > 0) {
        const size_t smem = s.rows > 1 ? 3 * (size_t)p.H * sizeof(float) : 0;
        const dim3 grid(ctas), block(s.warps * 32 * s.rows);
        cudaError_t e;
        if (block.x <= 512)
            e = p.f32 ? launch_kernel(true, norm_backward_kernel<2, true, 512>, grid, block, smem, stream, p, s)
                      : launch_kernel(true, norm_backward_kernel<2, false, 512>, grid, block, smem, stream, p, s);
        else
            e = p.f32 ? launch_kernel(true, norm_backward_kernel<2, true, 1024>, grid, block, smem, stream, p, s)
                      : launch_kernel(true, norm_backward_kernel<2, false, 1024>, grid, block, smem, stream, p, s);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((3 * (int64_t)p.H + 31) / 32));
    return launch_kernel(true, norm_columns_kernel, grid, dim3(256), 0, stream, p, ctas);
}

}  // namespace ep
