// block_device.cuh -- device helpers of the kernels at the ends of a block.
#pragma once
#include "ep_device.cuh"

namespace ep {

constexpr uint32_t kErrBadSeq = 16u;

// ----------------------------------------------------------------- warps

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// ------------------------------------------------------------------ f32x2
//
// Two fp32 values in one 64-bit register; products and sums take both at once,
// each rounded as by itself.

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }

__device__ __forceinline__ float2 halves(uint64_t p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

}  // namespace ep
