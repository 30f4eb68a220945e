// dropout.cu -- dropout from counters, with a mask that is never stored:
//   y = residual + (kept ? x * scale : 0)
// The gradient is the same call on the gradient of y.
#include <algorithm>

#include "block_kernels.h"
#include "dropout.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;     // vectors of a thread whose loads are in flight together

// Rows of `width` elements.  WIDE: whole vectors at 16-byte boundaries; else a
// vector's elements one by one, those past the row's end left out.
template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kThreads) dropout_kernel(DropoutParams p, int64_t rows, int64_t width) {
    constexpr int kSize = F32 ? 4 : 2;
    pdl_launch_dependents();
    pdl_wait();
    const Counters c = counters(p.drop);
    const int64_t vecs = (width + kVec - 1) / kVec;
    const int64_t v0 = (int64_t)blockIdx.x * blockDim.x * kUnroll + threadIdx.x;
    for (int64_t r = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; r < rows; r += (int64_t)gridDim.y * blockDim.y) {
        const unsigned char* x = static_cast<const unsigned char*>(p.x) + r * p.ld_x * kSize;
        const unsigned char* res = static_cast<const unsigned char*>(p.residual) + r * p.ld_res * kSize;
        unsigned char* y = static_cast<unsigned char*>(p.y) + r * p.ld_y * kSize;
        Vec8 a[kUnroll], b[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t v = v0 + u * blockDim.x, at = v * kVec;
            a[u] = b[u] = all(0.f);
            if (v >= vecs) continue;
            if (WIDE) {
                a[u] = load_stream<F32>(x, at);
                if (p.residual != nullptr) b[u] = load_stream<F32>(res, at);
            } else {
                float f[kVec], g[kVec];
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const bool in = at + i < width;
                    f[i] = in ? load_one<F32>(x, at + i) : 0.f;
                    g[i] = in && p.residual != nullptr ? load_one<F32>(res, at + i) : 0.f;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[u].v[i] = pair(f[2 * i], f[2 * i + 1]);
                    b[u].v[i] = pair(g[2 * i], g[2 * i + 1]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t v = v0 + u * blockDim.x, at = v * kVec;
            if (v >= vecs) continue;
            apply(a[u], random_bits(r * vecs + v, c), p.drop);
            if (p.residual != nullptr)
#pragma unroll
                for (int i = 0; i < 4; ++i) a[u].v[i] = add2(a[u].v[i], b[u].v[i]);
            if (WIDE) {
                store_stream<F32>(y, at, a[u]);
            } else {
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float2 f = halves(a[u].v[i / 2]);
                    if (at + i < width) store_one<F32>(y, at + i, i & 1 ? f.y : f.x);
                }
            }
        }
    }
}

template <bool F32>
cudaError_t launch(const DropoutParams& p, cudaStream_t stream) {
    constexpr int kSize = F32 ? 4 : 2;
    auto wide = [&](const void* at, int64_t ld) { return at == nullptr || ((reinterpret_cast<uintptr_t>(at) & 15u) == 0 && (p.T == 1 || ld * kSize % 16 == 0)); };
    const bool whole = p.H % kVec == 0;
    const bool dense = p.ld_x == p.H && p.ld_y == p.H && (p.residual == nullptr || p.ld_res == p.H);
    int64_t rows = p.T, width = p.H;
    // vectors do not cross rows, so dense rows are one
    if (whole && dense) {
        rows = 1;
        width *= p.T;
    }
    const int64_t vecs = (width + kVec - 1) / kVec;
    int bx = 32;
    while (bx < kThreads && bx * kUnroll < vecs) bx *= 2;
    const dim3 block(bx, kThreads / bx);
    const int64_t gx = (vecs + (int64_t)bx * kUnroll - 1) / ((int64_t)bx * kUnroll);
    const dim3 grid((unsigned)gx, (unsigned)std::min<int64_t>((rows + block.y - 1) / block.y, 65535));
    auto kern = whole && wide(p.x, p.ld_x) && wide(p.y, p.ld_y) && wide(p.residual, p.ld_res) ? dropout_kernel<F32, true> : dropout_kernel<F32, false>;
    return launch_kernel(true, kern, grid, block, 0, stream, p, rows, width);
}

}  // namespace

cudaError_t launch_dropout(const DropoutParams& p, cudaStream_t stream) { return p.f32 ? launch<true>(p, stream) : launch<false>(p, stream); }

}  // namespace ep
