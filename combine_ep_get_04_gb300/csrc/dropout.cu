// dropout.cu -- dropout from counters, with a mask that is never stored:
//   y = residual + (kept ? x * scale : 0)
// The gradient is the same call on the gradient of y.
#include <algorithm>

#include "block_kernels.h"
#include "dropout.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;

// CTAs of an SM, by the registers that a form needs: what hides the memory's
// latency is warps (T=16384 H=4096 bf16, forward and gradient: two vectors a thread
// and 4 CTAs 120 us, one and 7 CTAs 95; fp32 with a residual 5 CTAs 200, 7 208).
constexpr int ctas(bool f32, bool residual) { return residual ? f32 ? 5 : 6 : 7; }

// Rows of `width` elements, a grid apart; within a row a thread's vectors are a
// grid apart too.  Whole vectors at 16-byte boundaries.
//
// T=16384 H=4096 bf16 47 us, 5.7 TB/s, 85 % of the measured copy rate: the
// generator's products and some 120 instructions a vector; fp32 100 us with a residual, HBM.
template <bool F32, bool RESIDUAL>
__global__ void __launch_bounds__(kThreads, ctas(F32, RESIDUAL)) dropout_kernel(DropoutParams p, int64_t rows, int64_t width) {
    constexpr int kSize = F32 ? 4 : 2;
    pdl_launch_dependents();
    pdl_wait();
    const bool drop = p.drop.rng != nullptr;
    Counters c{};
    if (drop) c = counters(p.drop);
    const int64_t vecs = width / kVec, apart = (int64_t)gridDim.x * blockDim.x;
    for (int64_t r = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; r < rows; r += (int64_t)gridDim.y * blockDim.y) {
        const unsigned char* x = static_cast<const unsigned char*>(p.x) + r * p.ld_x * kSize;
        const unsigned char* res = static_cast<const unsigned char*>(p.residual) + r * p.ld_res * kSize;
        unsigned char* y = static_cast<unsigned char*>(p.y) + r * p.ld_y * kSize;
        for (int64_t v = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; v < vecs; v += apart) {
            Vec8 a = load_stream<F32>(x, v * kVec), b;
            if (RESIDUAL) b = load_stream<F32>(res, v * kVec);
            if (drop) apply(a, random_bits(r * vecs + v, c), p.drop);
            if (RESIDUAL)
#pragma unroll
                for (int i = 0; i < 4; ++i) a.v[i] = add2(a.v[i], b.v[i]);
            store_stream<F32>(y, v * kVec, a);
        }
    }
}

// Rows of any width and place: a warp takes 256 neighbours of a row, its lanes
// those 32 apart, so that its accesses are of neighbours, and hands each lane what
// another found out about its eight.
template <bool F32, bool RESIDUAL>
__global__ void __launch_bounds__(kThreads, 4) dropout_any_kernel(DropoutParams p, int64_t rows, int64_t width) {
    constexpr int kSize = F32 ? 4 : 2;
    pdl_launch_dependents();
    pdl_wait();
    const bool drop = p.drop.rng != nullptr;
    Counters c{};
    if (drop) c = counters(p.drop);
    const float scale = drop ? p.drop.scale : 1.f;
    const int lane = threadIdx.x & 31;
    const int64_t vecs = (width + kVec - 1) / kVec, apart = (int64_t)gridDim.x * blockDim.x;
    for (int64_t r = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; r < rows; r += (int64_t)gridDim.y * blockDim.y) {
        const unsigned char* x = static_cast<const unsigned char*>(p.x) + r * p.ld_x * kSize;
        const unsigned char* res = static_cast<const unsigned char*>(p.residual) + r * p.ld_res * kSize;
        unsigned char* y = static_cast<unsigned char*>(p.y) + r * p.ld_y * kSize;
        for (int64_t v = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; v - lane < vecs; v += apart) {
            const int64_t first = (v - lane) * kVec + lane;
            float a[kVec], b[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const bool in = first + 32 * j < width;
                a[j] = in ? load_one<F32>(x, first + 32 * j) : 0.f;
                b[j] = RESIDUAL && in ? load_one<F32>(res, first + 32 * j) : 0.f;
            }
            uint32_t stays = 0xff;                 // bit i: element i of the lane's eight
            if (drop) {
                const uint4 bits = random_bits(r * vecs + v, c);
                const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
                stays = 0;
#pragma unroll
                for (int i = 0; i < kVec; ++i) stays |= (uint32_t)((i & 1 ? w[i / 2] : w[i / 2] << 16) > p.drop.most) << i;
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const uint32_t eight = __shfl_sync(0xffffffffu, stays, 4 * j + (lane >> 3));
                float f = eight >> (lane & 7) & 1 ? __fmul_rn(a[j], scale) : 0.f;
                if (RESIDUAL) f = __fadd_rn(f, b[j]);
                if (first + 32 * j < width) store_one<F32>(y, first + 32 * j, f);
            }
        }
    }
}

template <bool F32, bool RESIDUAL>
cudaError_t launch(const DropoutParams& p, int num_sms, cudaStream_t stream) {
    constexpr int kSize = F32 ? 4 : 2;
    auto wide = [&](const void* at, int64_t ld) { return at == nullptr || ((reinterpret_cast<uintptr_t>(at) & 15u) == 0 && (p.T == 1 || ld * kSize % 16 == 0)); };
    const bool whole = p.H % kVec == 0;
    const bool dense = p.ld_x == p.H && p.ld_y == p.H && (!RESIDUAL || p.ld_res == p.H);
    int64_t rows = p.T, width = p.H;
    // vectors do not cross rows, so dense rows are one
    if (whole && dense) {
        rows = 1;
        width *= p.T;
    }
    const int64_t vecs = (width + kVec - 1) / kVec, most = (int64_t)num_sms * 28;
    int bx = 32;
    while (bx < kThreads && bx < vecs) bx *= 2;
    const dim3 block(bx, kThreads / bx);
    const int64_t gx = std::min((vecs + bx - 1) / bx, most), gy = std::min((rows + block.y - 1) / block.y, std::max<int64_t>(1, most / gx));
    auto kern = whole && wide(p.x, p.ld_x) && wide(p.y, p.ld_y) && wide(p.residual, p.ld_res) ? dropout_kernel<F32, RESIDUAL>
                                                                                           : dropout_any_kernel<F32, RESIDUAL>;
    return launch_kernel(true, kern, dim3((unsigned)gx, (unsigned)gy), block, 0, stream, p, rows, width);
}

template <bool F32>
cudaError_t launch(const DropoutParams& p, int num_sms, cudaStream_t stream) {
    return p.residual != nullptr ? launch<F32, true>(p, num_sms, stream) : launch<F32, false>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_dropout(const DropoutParams& p, int num_sms, cudaStream_t stream) {
    return p.f32 ? launch<true>(p, num_sms, stream) : launch<false>(p, num_sms, stream);
}

}  // namespace ep
