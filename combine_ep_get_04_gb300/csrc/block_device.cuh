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

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// --------------------------------------------------------------- vectors

constexpr int kVec = 8;   // channels a thread handles at once: 16 bytes of bf16

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

// A single element of a stream.
template <bool F32>
__device__ __forceinline__ float load_one(const void* base, int64_t at) {
    return F32 ? static_cast<const float*>(base)[at] : bf16_lo(static_cast<const uint16_t*>(base)[at]);
}

template <bool F32>
__device__ __forceinline__ void store_one(void* base, int64_t at, float x) {
    if (F32)
        static_cast<float*>(base)[at] = x;
    else
        static_cast<uint16_t*>(base)[at] = (uint16_t)pack_bf16x2(x, 0.f);
}

}  // namespace ep
