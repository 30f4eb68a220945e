// dropout.cuh -- the random numbers of dropout, made where they are used.
#pragma once
#include "block_device.cuh"
#include "block_kernels.h"

namespace ep {

constexpr int kRounds = 10;

// What all counters of a dropout have in common: the step (with the site), and
// the rounds' keys, which follow from the seed.
struct Counters {
    uint32_t step0, step1;
    uint2 keys[kRounds];
};

__device__ __forceinline__ Counters counters(const Dropout& d) {
    const uint64_t seed = (uint64_t)d.rng[0], step = (uint64_t)d.rng[1] + d.site;
    Counters c;
    c.step0 = (uint32_t)step;
    c.step1 = (uint32_t)(step >> 32);
#pragma unroll
    for (int i = 0; i < kRounds; ++i) c.keys[i] = make_uint2((uint32_t)seed + i * 0x9E3779B9u, (uint32_t)(seed >> 32) + i * 0xBB67AE85u);
    return c;
}

// 128 random bits for eight neighbouring elements: Philox4x32 with ten rounds
// (J. K. Salmon, M. A. Moraes, R. O. Dror and D. E. Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC11), counter = (block of eight, step), key =
// seed.  Its twenty 32 x 32 -> 64-bit products take 80 cycles a warp of a quarter
// of an SM (measured); a bf16 vector read and written at the copy rate leaves 177.
__device__ __forceinline__ uint4 random_bits(uint64_t block, const Counters& c) {
    uint32_t x0 = (uint32_t)block, x1 = (uint32_t)(block >> 32), x2 = c.step0, x3 = c.step1;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const uint64_t a = (uint64_t)0xD2511F53u * x0, b = (uint64_t)0xCD9E8D57u * x2;
        x0 = (uint32_t)(b >> 32) ^ x1 ^ c.keys[i].x;
        x2 = (uint32_t)(a >> 32) ^ x3 ^ c.keys[i].y;
        x1 = (uint32_t)b;
        x3 = (uint32_t)a;
    }
    return make_uint4(x0, x1, x2, x3);
}

// x times the scale where it stays, and 0, whatever x is, where it does not.
// One rounding each.  Sixteen bits stay when they, with zeros or anything behind
// them, are above limit * 65536 - 1.
__device__ __forceinline__ void apply(Vec8& x, uint4 bits, const Dropout& d) {
    const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = halves(mul2(x.v[i], both(d.scale)));
        x.v[i] = pair(w[i] << 16 > d.most ? v.x : 0.f, w[i] > d.most ? v.y : 0.f);
    }
}

}  // namespace ep
