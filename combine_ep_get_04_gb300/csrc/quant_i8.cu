// quant_i8.cu -- rows of the receive buffer to 8-bit integers with a scale each:
//   scale = amax / 127,  q = round(127 x / amax)
// 127 x of a bf16 x is exact in fp32 (15 bits), and a quotient of the two that is
// not a half itself lies further from one than fp32 rounds it, so the codes are
// those of the real numbers, halves to even.  The quotient is made from one
// reciprocal a row (Markstein's correction, as in quotient_rn), with amax brought
// into [2^-64, 2^64] first, where no step that matters under- or overflows.
#include <algorithm>

#include "block_device.cuh"
#include "block_kernels.h"

namespace ep {
namespace {

constexpr int kMaxThreads = 512;

// Rows of a CTA: those of one expert (capacity mode, blockIdx.y), or all rows
// in use.  A thread has NV vectors of 8 channels.  One pass: the row stays in
// registers between its largest magnitude and its codes.
//
// 32768 packed rows of 2048 32.7 us, 6.2 TB/s, 92 % of the measured copy rate; 1024
// rows of 7168 in a capacity buffer of 256 x 128 6.8 us, where the CTAs of experts
// with few rows find nothing to do.
template <int NV>
__global__ void __launch_bounds__(kMaxThreads) quant_i8_kernel(QuantParams p) {
    __shared__ float red[2][kMaxThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    int64_t first = 0, rows = p.R;
    if (p.mode != 0) {
        first = (int64_t)blockIdx.y * p.capacity;
        rows = min(p.counts[blockIdx.y], p.capacity);
    } else if (p.offsets != nullptr) {
        rows = p.offsets[p.E];
        if (rows > p.R) {
            if (blockIdx.x == 0 && threadIdx.x == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrBadSlot);
            rows = p.R;
        }
    }
    const int warps = blockDim.x >> 5, vecs = p.K / kVec;
    int flip = 0;
    for (int64_t i = blockIdx.x; i < rows; i += gridDim.x, flip ^= 1) {
        const int64_t r = first + i;
        const unsigned char* x = static_cast<const unsigned char*>(p.x) + r * p.ld * 2;
        uint4 raw[NV];
        uint32_t top = 0;          // largest magnitude: bits of non-negative bf16 values compare as the values do
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            raw[k] = v < vecs ? *reinterpret_cast<const uint4*>(x + (int64_t)v * kVec * 2) : make_uint4(0, 0, 0, 0);
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[k].x & 0x7fff7fffu, raw[k].y & 0x7fff7fffu), __vmaxu2(raw[k].z & 0x7fff7fffu, raw[k].w & 0x7fff7fffu)));
        }
        top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) red[flip][threadIdx.x >> 5] = __uint_as_float(top << 16);
            __syncthreads();
            top = (threadIdx.x & 31) < warps ? __float_as_uint(red[flip][threadIdx.x & 31]) >> 16 : 0;
            top = __reduce_max_sync(0xffffffffu, top);
        }
        // a row that holds an infinity or a NaN has no scale: NaN, with codes of 0
        const bool fine = top < 0x7f80u;
        const float amax = __uint_as_float(top << 16);
        const float unit = amax >= 0x1p64f ? 0x1p-100f : amax < 0x1p-64f ? 0x1p100f : 1.f;
        const float d = top != 0 ? amax * unit : 1.f, rd = __frcp_rn(d), unit127 = 127.f * unit;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v >= vecs) continue;
            const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
            uint32_t q[2] = {0, 0};
            if (fine) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float t = (j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1])) * unit127;
                    const float q0 = t * rd;
                    const float c = __fmaf_rn(__fmaf_rn(-q0, d, t), rd, q0);
                    // beside 1.5 * 2^23 a number has no places after the point: the sum's low byte is the rounded code
                    q[j >> 2] |= (__float_as_uint(__fadd_rn(c, 0x1.8p23f)) & 0xffu) << (8 * (j & 3));
                }
            }
            *reinterpret_cast<uint2*>(p.q + r * p.K + (int64_t)v * kVec) = make_uint2(q[0], q[1]);
        }
        if (threadIdx.x == 0) p.scales[r] = fine ? __fdiv_rn(amax, 127.f) : NAN;
    }
}

}  // namespace

cudaError_t launch_quant_i8(const QuantParams& p, int num_sms, cudaStream_t stream) {
    const int vecs = p.K / kVec, nv = vecs <= 128 ? 1 : 4;
    const int threads = (vecs + 32 * nv - 1) / (32 * nv) * 32;
    const int64_t most = (int64_t)num_sms * (2048 / threads) * 2;          // two waves
    dim3 grid((unsigned)std::min(p.R, most));
    if (p.mode != 0) grid = dim3((unsigned)std::min<int64_t>(p.capacity, std::max<int64_t>(8, most / p.E)), (unsigned)p.E);
    return launch_kernel(true, nv == 1 ? quant_i8_kernel<1> : quant_i8_kernel<4>, grid, dim3(threads), 0, stream, p);
}

}  // namespace ep
