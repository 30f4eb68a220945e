// dropout.cuh -- the random numbers of dropout, made where they are used.
#pragma once
#include "block_device.cuh"
#include "block_kernels.h"

namespace ep {

// A dropout's counters: its step (with the site) and its seed as the key.
struct Counters {
    uint32_t step0, step1, key0, key1;
};

__device__ __forceinline__ Counters counters(const Dropout& d) {
    const uint64_t seed = (uint64_t)d.rng[0], step = (uint64_t)d.rng[1] + d.site;
    return Counters{(uint32_t)step, (uint32_t)(step >> 32), (uint32_t)seed, (uint32_t)(seed >> 32)};
}

// 128 random bits for eight neighbouring elements: Philox4x32 with ten rounds
// (J. K. Salmon, M. A. Moraes, R. O. Dror and D. E. Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC11), counter = (block of eight, step), key =
// seed.  A round is two 32 x 32 -> 64-bit products, of which an SM makes about
// 28 a clock: eight 16-bit numbers a counter cost 2.5 products each, a bf16 read
// and written at the copy rate leaves room for 4.8.
__device__ __forceinline__ uint4 random_bits(uint64_t block, const Counters& c) {
    uint32_t x0 = (uint32_t)block, x1 = (uint32_t)(block >> 32), x2 = c.step0, x3 = c.step1, k0 = c.key0, k1 = c.key1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)0xD2511F53u * x0, b = (uint64_t)0xCD9E8D57u * x2;
        x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
        x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
        x1 = (uint32_t)b;
        x3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
}

// x times the scale where it stays, and 0, whatever x is, where it does not.
// One rounding each.
__device__ __forceinline__ void apply(Vec8& x, uint4 bits, const Dropout& d) {
    const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = halves(mul2(x.v[i], both(d.scale)));
        x.v[i] = pair((w[i] & 0xffffu) >= d.limit ? v.x : 0.f, (w[i] >> 16) >= d.limit ? v.y : 0.f);
    }
}

}  // namespace ep
