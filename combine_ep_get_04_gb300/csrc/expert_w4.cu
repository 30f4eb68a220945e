// expert_w4.cu -- the experts' products over the receive buffer with 4-bit
// weights and group scales:
//   y[r, n] = sum_k x[r, k] * (code[e, n, k] - 8) * scale[e, n, k / group]
//
// A decode batch gives an expert a handful of rows, so the bytes of the weights
// decide the time.  They are laid out once so that a CTA's stream of them is
// contiguous and every thread finds its matrix-instruction operands in one
// 16-byte word: tiles of 16 weight rows x 128 input channels, 1024 bytes of
// codes and then the tile's scales, eight tiles side by side for each step
// along K.  A producer warp keeps a ring of such steps (and the matching
// 128-channel pieces of the token rows) filled with bulk copies; four consumer
// warps, two tiles each, widen the codes to bf16 (f16 beside fp8 rows: either
// holds code - 8 and f16 every e4m3 value exactly) and multiply with
// mma.m16n8k16, the weights as the 16-row side and 8 tokens as the other.  A
// group's products are summed unscaled in fp32 and enter the accumulator
// through one fused multiply-add with the group's scale.
#include <algorithm>
#include <atomic>
#include <cuda.h>
#include <type_traits>

#include "block_device.cuh"
#include "block_kernels.h"

namespace ep {
namespace {

constexpr int kTileRows = 16;      // weight rows of one tile (the matrix instruction's)
constexpr int kTileK = 128;        // input channels of one tile
constexpr int kTiles = 8;          // tiles of one step
constexpr int kCodeBytes = kTileRows * kTileK / 2;
constexpr int kStep = 2;           // tiles along K of one stage of the ring
constexpr int kRing = 2;           // stages

// OWN: tiles of a consumer warp.  Two share the rows' operands; one, with twice
// the warps, takes half the time for a step where an SM has few warps.
__host__ __device__ constexpr int consumer_warps(int own) { return kTiles / own; }
__host__ __device__ constexpr int block_threads(int own) { return (consumer_warps(own) + 1) * 32; }

__host__ __device__ constexpr int tile_bytes(int group) { return kCodeBytes + kTileK / group * 32; }

// Tiles along the output: a paired tile is 8 gate rows and the 8 up rows of
// the same channels, so that one thread ends up with both products.
__host__ __device__ inline int row_tiles(const W4Shape& w) { return w.paired ? (w.N + 7) / 8 : (w.N + 15) / 16; }
__host__ __device__ inline int row_blocks(const W4Shape& w) { return (row_tiles(w) + kTiles - 1) / kTiles; }
__host__ __device__ inline int k_blocks(const W4Shape& w) { return (w.K + kTileK - 1) / kTileK; }

// Token rows in a stage.  A few rows come by one bulk copy each, every row's
// piece 64 bytes (32 for fp8) longer than it is; more rows come as boxes of 32
// channels, [channels / 32][rows][32 channels], by tensor copies, whose number
// does not grow with the rows.  Either way the eight rows that a warp reads at
// once fall into different banks.
__host__ __device__ constexpr bool x_boxes(int nt) { return nt > 2; }
__host__ __device__ constexpr int x_row(int nt, bool fp8) {       // from one row to the next
    return x_boxes(nt) ? (fp8 ? 32 : 64) : fp8 ? kStep * kTileK + 32 : kStep * kTileK * 2 + 64;
}
__host__ __device__ constexpr int x_chunk(int nt, bool fp8) {     // from 32 channels to the next
    return x_boxes(nt) ? 8 * nt * x_row(nt, fp8) : fp8 ? 32 : 64;
}
__host__ __device__ constexpr int x_bytes(int nt, bool fp8) {
    return x_boxes(nt) ? kStep * kTileK / 32 * x_chunk(nt, fp8) : 8 * nt * x_row(nt, fp8);
}
__host__ __device__ constexpr int weight_bytes(int group) { return kTiles * tile_bytes(group); }
__host__ __device__ constexpr int stage_bytes(int group, int nt, bool fp8) { return kStep * weight_bytes(group) + x_bytes(nt, fp8); }

// One word of codes: 8 input channels of one weight row, channel 2j in bits
// 4j and channel 2j + 1 in bits 16 + 4j, so that a shift by 4j and a mask
// leave a pair of neighbours in the two halves of a register.
__global__ void __launch_bounds__(256) w4_pack_kernel(W4Shape w, const uint8_t* codes, const uint16_t* scales, unsigned char* packed) {
    const int64_t tile = blockIdx.x;           // [E][row block][k block][kTiles]
    const int nk = k_blocks(w), nb = row_blocks(w);
    const int rt = (int)(tile % kTiles), kb = (int)(tile / kTiles % nk);
    const int64_t blk = tile / kTiles / nk;
    const int rb = (int)(blk % nb), e = (int)(blk / nb);
    const int groups = (w.K + w.group - 1) / w.group, rows = w.paired ? 2 * w.N : w.N;
    unsigned char* out = packed + tile * tile_bytes(w.group);
    auto source_row = [&](int r) {             // weight row of row r of the tile; -1: padding
        const int at = rb * kTiles + rt;
        const int row = w.paired ? at * 8 + (r & 7) : at * 16 + r;
        return row >= w.N ? -1 : w.paired && r >= 8 ? w.N + row : row;
    };
    {
        const int half = threadIdx.x >> 7, lane = threadIdx.x >> 2 & 31, i = threadIdx.x & 3;
        const int row = source_row(half * 8 + (lane >> 2)), k = kb * kTileK + 32 * i + 8 * (lane & 3);
        uint32_t word = 0x88888888u;           // code 8: zero
        if (row >= 0 && k < w.K) {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + (((int64_t)e * rows + row) * w.K + k) / 2);
            word = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) word |= (c >> (8 * j) & 0xfu) << (4 * j) | (c >> (8 * j + 4) & 0xfu) << (16 + 4 * j);
        }
        *reinterpret_cast<uint32_t*>(out + half * 512 + lane * 16 + i * 4) = word;
    }
    const int per = kTileK / w.group;
    if (threadIdx.x < 16 * per) {
        const int r = threadIdx.x & 15, g = threadIdx.x >> 4;
        const int row = source_row(r), at = kb * per + g;
        const uint16_t s = row >= 0 && at < groups ? scales[((int64_t)e * rows + row) * groups + at] : (uint16_t)0;
        *reinterpret_cast<uint16_t*>(out + kCodeBytes + g * 32 + (r & 7) * 4 + (r >> 3) * 2) = s;
    }
}

// D = A B + C for one 16 x 8 x 16 step, fp32 accumulators.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1, float c2,
                                         float c3) {
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// A code masked out of its half of a word, in bits 0-3 or 4-7, is a tiny
// number as it stands: subnormals and the first binade above them are one
// linear range, so as f16 it is code * 2^-24 or code * 2^-20, as bf16 code *
// 2^-133 or code * 2^-129.  One shift and four masks leave the four pairs of
// a word: 0 and 2 the low, 1 and 3 the high kind.
__device__ __forceinline__ void unpack(uint32_t word, uint32_t (&pair)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) pair[j] = (j < 2 ? word : word >> 8) & (j & 1 ? 0x00f000f0u : 0x000f000fu);
}

// One fused multiply-add brings the pairs up to (code - 8) * 2^-6 in bf16 or
// (code - 8) * 2^-9 in f16.  Exact.  (Pairs that enter the products as they are,
// with one more product for the offset, are not an alternative: the matrix
// instruction lines products up by their exponents, a subnormal's as 2^-14
// whatever its value, and cuts off what lies too far below the largest.  A
// channel at e4m3's 448 under a zero weight cost 3 to 13 % of a result of its
// smallest values.  256 experts, 4 fp8 rows each, gate and up, by groups of 32, 64
// and 128: 717, 645 and 609 us so, 671, 637 and 619 with the multiply-adds.)
template <bool F16>
__device__ __forceinline__ void widen(uint32_t (&pair)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (F16)       // by 2^15 or 2^11, less 8 * 2^-9
            asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(pair[j]) : "r"(j & 1 ? 0x68006800u : 0x78007800u), "r"(0xa400a400u));
        else           // by 2^127 or 2^123, less 8 * 2^-6
            asm("fma.rn.bf16x2 %0, %0, %1, %2;" : "+r"(pair[j]) : "r"(j & 1 ? 0x7d007d00u : 0x7f007f00u), "r"(0xbe00be00u));
    }
}

// What the codes are divided by.
template <bool FP8>
constexpr float kUnit = FP8 ? 512.f : 64.f;

// Four e4m3 codes -> two pairs of f16, exact.
__device__ __forceinline__ void f16x2_of_e4m3x4(uint32_t codes, uint32_t* lo, uint32_t* hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(*lo), "=r"(*hi) : "r"(codes));
}

// Transposes an 8 x 8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void clear(float (&v)[4]) { v[0] = v[1] = v[2] = v[3] = 0.f; }

// x times its sigmoid, by exp(-|x|): that never overflows, so a large negative
// x leaves what exp(x) leaves of it.  expf is good to two units in the last
// place; the fast form's error grows with |x|.
__device__ __forceinline__ float silu(float x) {
    const float e = expf(-fabsf(x));
    return x * __fdividef(x < 0.f ? e : 1.f, 1.f + e);
}

struct RowTile {
    int e;          // expert, -1: none
    int rows;       // rows of the tile
    int64_t first;  // its first row
};

// Rows of expert e that lie inside the buffer; a claim beyond it gives none.
__device__ __forceinline__ int expert_rows(const W4Params& p, int e, int64_t* first, bool* bad) {
    int64_t a, n;
    if (p.mode != 0) {
        a = (int64_t)e * p.capacity;
        n = min(p.counts[e], p.capacity);
    } else if (p.offsets != nullptr) {
        a = p.offsets[e];
        n = p.offsets[e + 1] - a;
    } else {
        a = 0;
        n = p.R;
    }
    *first = a;
    *bad = n > 0 && (a < 0 || a + n > p.R);
    return *bad || n < 0 ? 0 : (int)n;
}

// tile_rows is a power of two
__device__ __forceinline__ int tiles_of(int rows, int tile_rows) {
    return (rows >> (31 - __clz(tile_rows))) + ((rows & (tile_rows - 1)) != 0);
}

constexpr int kMaxTiles = (1 << 26) - 1;     // 32 lanes' worth of them fit 31 bits
constexpr int kScan = 8;    // experts whose rows a lane looks up at a time: their loads are in flight together

// Tile `at` in the order of experts and of rows within an expert.  One warp;
// lane l counts the tiles of experts [l * per, (l + 1) * per).
__device__ __forceinline__ RowTile find_tile(const W4Params& p, int at, int tile_rows, int grid_tiles) {
    const int lane = threadIdx.x & 31;
    const int per = (p.w.E + 31) / 32;
    const int e0 = min(lane * per, p.w.E), e1 = min(e0 + per, p.w.E);
    // bad offsets may claim every row many times: a lane's sum is cut off where no good layout comes to
    int mine = 0;
    bool any_bad = false;
    int64_t first[kScan];
    int n[kScan];
    auto look_up = [&](int from) {
        bool bad[kScan];
#pragma unroll
        for (int j = 0; j < kScan; ++j) {
            n[j] = 0;
            bad[j] = false;
            if (from + j < e1) n[j] = expert_rows(p, from + j, &first[j], &bad[j]);
        }
#pragma unroll
        for (int j = 0; j < kScan; ++j) any_bad |= bad[j];
    };
    for (int from = e0; from < e1; from += kScan) {
        look_up(from);
#pragma unroll
        for (int j = 0; j < kScan; ++j) mine = min(mine + tiles_of(n[j], tile_rows), kMaxTiles);
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
    }
    const int total = __shfl_sync(0xffffffffu, upto, 31);
    if (at == 0 && p.err_flags != nullptr) {
        if (any_bad) atomicOr(p.err_flags, kErrBadSlot);
        if (total > grid_tiles && lane == 0) atomicOr(p.err_flags, kErrCapacity);
    }
    RowTile r{-1, 0, 0};
    if (at >= total) return r;
    const int owner = __ffs(__ballot_sync(0xffffffffu, upto > at)) - 1;
    if (lane == owner) {
        int left = at - (upto - mine);
        for (int from = e0; from < e1 && r.e < 0; from += kScan) {
            if (per > kScan) look_up(from);       // else n still holds them all
#pragma unroll
            for (int j = 0; j < kScan; ++j) {
                const int tiles = tiles_of(n[j], tile_rows);
                if (r.e < 0 && left >= 0 && left < tiles)
                    r = RowTile{from + j, min(n[j] - left * tile_rows, tile_rows), first[j] + (int64_t)left * tile_rows};
                left -= tiles;
            }
        }
    }
    r.e = __shfl_sync(0xffffffffu, r.e, owner);
    r.rows = __shfl_sync(0xffffffffu, r.rows, owner);
    r.first = __shfl_sync(0xffffffffu, r.first, owner);
    return r;
}

// The same for a single matrix: every thread looks for itself.
__device__ __forceinline__ RowTile tile_of_one(const W4Params& p, int at, int tile_rows, int grid_tiles) {
    int64_t first;
    bool bad;
    const int n = expert_rows(p, 0, &first, &bad), tiles = tiles_of(n, tile_rows);
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.err_flags != nullptr) {
        if (bad) atomicOr(p.err_flags, kErrBadSlot);
        if (tiles > grid_tiles) atomicOr(p.err_flags, kErrCapacity);
    }
    if (at >= tiles) return RowTile{-1, 0, 0};
    return RowTile{0, min(n - at * tile_rows, tile_rows), first + (int64_t)at * tile_rows};
}

// Starts bringing `bytes` (a multiple of 16) at a 16-byte boundary into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Writes to the same place in another CTA's shared memory.
__device__ __forceinline__ void cluster_store(const float4* p, uint32_t rank, const float (&v)[4]) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}

// A box of 32 channels x 8 NT rows, completion counted in bytes on `bar`.
__device__ __forceinline__ void box_load(void* dst, const CUtensorMap* map, int channel, int row, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                     smem_addr(dst)),
                 "l"(map), "r"(channel), "r"(row), "r"(smem_addr(bar))
                 : "memory");
}

// One tile step along K (128 channels) of a consumer warp: adds scale * code
// sums to the accumulators, in units of 1 / kUnit.  wt: the warp's tiles, xr:
// the lane's place in the first token row, xs: the rows' scales (fp8).
template <int NT, int OWN, int NL, int G, bool FP8>
__device__ __forceinline__ void tile_step(float (&acc)[OWN][NT][4], const unsigned char* wt, const unsigned char* xr, const float* xs) {
    constexpr int kTile = 8 * x_row(NT, FP8), kChunk = x_chunk(NT, FP8);
    const int lane = threadIdx.x & 31, g = lane >> 2;
    uint32_t w[OWN][2][4];                // [tile][row g, row g + 8][32 channels each]
#pragma unroll
    for (int u = 0; u < OWN; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 v = *reinterpret_cast<const uint4*>(wt + u * tile_bytes(G) + h * 512 + lane * 16);
            w[u][h][0] = v.x;
            w[u][h][1] = v.y;
            w[u][h][2] = v.z;
            w[u][h][3] = v.w;
        }
    float part[OWN][NL][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool first = i * 32 % G == 0;
        // operands of the low and the high pairs: channels 0 1 4 5 and 2 3 6 7 of the lane's eight
        uint32_t a[OWN][2][4];
#pragma unroll
        for (int u = 0; u < OWN; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t pair[4];
                unpack(w[u][h][i], pair);
                widen<FP8>(pair);
#pragma unroll
                for (int j = 0; j < 4; ++j) a[u][j & 1][(j >> 1) * 2 + h] = pair[j];
            }
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            uint32_t b[4];
            if (FP8) {
                const uint2 v = *reinterpret_cast<const uint2*>(xr + n * kTile + i * kChunk);
                f16x2_of_e4m3x4(v.x, &b[0], &b[1]);
                f16x2_of_e4m3x4(v.y, &b[2], &b[3]);
            } else {
                const uint4 v = *reinterpret_cast<const uint4*>(xr + n * kTile + i * kChunk);
                b[0] = v.x;
                b[1] = v.y;
                b[2] = v.z;
                b[3] = v.w;
            }
            auto multiply = [&](float (&d)[4], const uint32_t (&low)[4], const uint32_t (&high)[4]) {
                if (first)
                    mma16816<FP8>(d, low, b[0], b[2], 0.f, 0.f, 0.f, 0.f);
                else
                    mma16816<FP8>(d, low, b[0], b[2], d[0], d[1], d[2], d[3]);
                mma16816<FP8>(d, high, b[1], b[3], d[0], d[1], d[2], d[3]);
            };
#pragma unroll
            for (int u = 0; u < OWN; ++u) multiply(part[u][n], a[u][0], a[u][1]);
        }
        if ((i + 1) * 32 % G == 0) {
#pragma unroll
            for (int u = 0; u < OWN; ++u) {
                const uint32_t sc = *reinterpret_cast<const uint32_t*>(wt + u * tile_bytes(G) + kCodeBytes + i * 32 / G * 32 + g * 4);
                const uint64_t s0 = both(bf16_lo(sc)), s1 = both(bf16_hi(sc));
#pragma unroll
                for (int n = 0; n < NL; ++n) {
                    float (&v)[4] = acc[u][n];
                    const float (&d)[4] = part[u][n];
                    const uint64_t d0 = pair(d[0], d[1]), d1 = pair(d[2], d[3]);
                    uint64_t t0 = s0, t1 = s1;
                    if (FP8) {
                        const float2 q = *reinterpret_cast<const float2*>(xs + n * 8);
                        t0 = mul2(s0, pair(q.x, q.y));
                        t1 = mul2(s1, pair(q.x, q.y));
                    }
                    const float2 v0 = halves(fma2(d0, t0, pair(v[0], v[1]))), v1 = halves(fma2(d1, t1, pair(v[2], v[3])));
                    v[0] = v0.x;
                    v[1] = v0.y;
                    v[2] = v1.x;
                    v[3] = v1.y;
                }
            }
        }
    }
}

// A consumer warp's walk along K: `blocks` tile steps, kStep to a stage of the
// ring from stage s on, NL x 8 tokens.  False if a wait timed out.
template <int NT, int OWN, int NL, int G, bool FP8>
__device__ __forceinline__ bool consume(float (&acc)[OWN][NT][4], const unsigned char* smem, const float* xs, uint64_t* full,
                                        uint64_t* empty, int blocks, int& s, uint32_t& parity) {
    constexpr int kStage = stage_bytes(G, NT, FP8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const unsigned char* own = smem + warp * OWN * tile_bytes(G);
    const unsigned char* rows = smem + kStep * weight_bytes(G) + g * x_row(NT, FP8) + (FP8 ? 8 : 16) * t;
    xs += 2 * t;
    for (int left = blocks; left > 0; left -= kStep) {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[s], parity))) return false;
        const unsigned char* wt = own + s * kStage;
        const unsigned char* xr = rows + s * kStage;
        // not unrolled: a short product runs this code from a cold instruction cache
#pragma unroll 1
        for (int q = min(left, kStep); q > 0; --q) {
            tile_step<NT, OWN, NL, G, FP8>(acc, wt, xr, xs);
            wt += weight_bytes(G);
            xr += kTileK / 32 * x_chunk(NT, FP8);
            if (FP8) xs += 8 * NT;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        if (++s == kRing) {
            s = 0;
            parity ^= 1;
        }
    }
    return true;
}

// One CTA: `units` row blocks (128 weight rows each) of one tile of up to 8 NT
// token rows, over one of `splits` shares of K.  The ring runs on from one row
// block to the next.  The shares of a product form a cluster (of one row block
// each) and add their accumulators through distributed shared memory in the
// order of the shares.
//
// Up to 8 rows an expert the weights' bytes decide: 256 experts with 4 rows each,
// gate and up (7168 -> 2 x 2048, fp8 rows) 618 us, down (2048 -> 7168, bf16 rows)
// 326 us, 6.2 and 6.1 TB/s, 91 and 90 % of the measured copy rate.  With more
// rows the matrix instructions and the widening do: 220 to 285 TFLOP/s from 16 to
// 32 rows.  One row through one matrix of 4096 x 7168 is latency: 6.9 us against
// 2.2 for its bytes.
template <int NT, int OWN, int G, bool FP8>
__global__ void __launch_bounds__(block_threads(OWN), NT <= 2 ? 4 : OWN == 1 ? 2 : 3) expert_w4_kernel(W4Params p, const __grid_constant__ CUtensorMap rows_map, int splits, int units,
                                                                                    int grid_tiles) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[kRing], empty[kRing];
    __shared__ RowTile shared_tile;
    constexpr int kWarps = consumer_warps(OWN), kThreads = block_threads(OWN);
    constexpr int kWeights = weight_bytes(G);
    constexpr int kRows = 8 * NT;
    constexpr int kStage = stage_bytes(G, NT, FP8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x % splits;
    const int blocks = row_blocks(p.w), nk = k_blocks(p.w), parts_of = (blocks + units - 1) / units;
    const int rb0 = blockIdx.x / splits % parts_of * units, rb1 = min(rb0 + units, blocks), at = blockIdx.x / splits / parts_of;
    const int kb0 = (int)((int64_t)nk * split / splits), kb1 = (int)((int64_t)nk * (split + 1) / splits);
    const unsigned char* weights = static_cast<const unsigned char*>(p.packed) + ((int64_t)rb0 * nk + kb0) * kWeights;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        // a single matrix: its first steps are known before the rows are
        if (p.w.E == 1) prefetch_l2(weights, (uint32_t)min(kb1 - kb0, kRing * kStep) * kWeights);
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        fence_mbar_init();
    }
    pdl_wait();
    // a single matrix: the producer starts on its first stages while the rows are looked up
    int primed = 0;
    RowTile tile;
    if (p.w.E == 1) {
        __syncthreads();
        if (warp == kWarps) {
            for (; primed < kRing && kb0 + primed * kStep < kb1; ++primed)
                if (lane == 0) {
                    const uint32_t bytes = kWeights * min(kStep, kb1 - kb0 - primed * kStep);
                    mbar_expect_tx(&full[primed], bytes);
                    bulk_load(smem + primed * kStage, weights + (int64_t)primed * kStep * kWeights, bytes, &full[primed]);
                }
        }
        tile = tile_of_one(p, at, kRows, grid_tiles);
    } else {
        if (warp == 0) {
            const RowTile r = find_tile(p, at, kRows, grid_tiles);
            if (lane == 0) shared_tile = r;
        }
        __syncthreads();
        tile = shared_tile;
    }
    if (splits > 1) cluster_arrive();
    if (tile.e < 0) {                    // the same in all CTAs of a cluster
        if (warp == kWarps)
            for (int s = 0; s < primed; ++s) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
                mbar_wait(&full[s], 0);
            }
        __syncwarp();
        if (splits > 1) cluster_wait();
        return;
    }
    weights += (int64_t)tile.e * blocks * nk * kWeights;
    float* xs = reinterpret_cast<float*>(smem + kRing * kStage);          // [k block][kRows] (fp8)
    float4* parts = reinterpret_cast<float4*>(smem + kRing * kStage + (FP8 ? (int64_t)nk * kRows * 4 : 0));   // [kTiles][NT][32]
    if (FP8) {
        for (int i = threadIdx.x; i < (kb1 - kb0) * kRows; i += kThreads) {
            const int kb = kb0 + i / kRows, r = i % kRows;
            float s = 0.f;
            if (r < tile.rows) {
                const int64_t from = (tile.first + r) * nk + kb;
                if (p.ue8m0) {
                    const uint32_t e = static_cast<const uint8_t*>(p.x_scales)[from];
                    s = __uint_as_float(e == 0 ? 0x00400000u : e << 23);      // 0 is 2^-127, a subnormal
                } else {
                    s = static_cast<const float*>(p.x_scales)[from];
                }
            }
            xs[i] = s;
        }
        __syncthreads();
    }
    if (warp == kWarps) {
        // producer
        constexpr int kSize = FP8 ? 1 : 2;
        const int64_t row_bytes = (int64_t)p.w.K * kSize;
        const unsigned char* x = static_cast<const unsigned char*>(p.x) + tile.first * row_bytes;
        bool good = true;
        int filled = 0;
        for (int rb = rb0; rb < rb1 && good; ++rb) {
            const unsigned char* weight = weights + (int64_t)(rb - rb0) * nk * kWeights;
            for (int kb = kb0; kb < kb1; kb += kStep, ++filled) {
                const int s = filled % kRing, round = filled / kRing;
                if (round > 0 && !__all_sync(0xffffffffu, mbar_wait(&empty[s], (round - 1) & 1))) {
                    good = false;
                    break;
                }
                unsigned char* st = smem + s * kStage;
                unsigned char* xt = st + kStep * kWeights;
                const int blocks_here = min(kStep, kb1 - kb);
                const uint32_t wanted = blocks_here * kTileK * kSize;
                const uint32_t piece = min((uint32_t)(p.w.K - kb * kTileK) * kSize, wanted);
                if (x_boxes(NT)) {
                    // rows past the buffer and channels past the rows' end arrive as zeros
                    if (lane == 0) {
                        constexpr int kBox = x_chunk(NT, FP8);
                        const int boxes = blocks_here * (kTileK / 32);
                        mbar_arrive_expect_tx(&full[s], (filled < primed ? 0 : kWeights * blocks_here) + boxes * kBox);
                        if (filled >= primed) bulk_load(st, weight, kWeights * blocks_here, &full[s]);
                        for (int i = 0; i < boxes; ++i)
                            box_load(xt + i * kBox, &rows_map, kb * kTileK + i * 32, (int)tile.first, &full[s]);
                    }
                } else {
                    constexpr int kRow = x_row(NT, FP8);
                    if (piece < wanted) {
                        // a short last step: zeros stand in for the channels past the end
                        const uint32_t words = (wanted - piece) / 16;
                        for (uint32_t i = lane; i < words * tile.rows; i += 32)
                            *reinterpret_cast<uint4*>(xt + i / words * kRow + piece + i % words * 16) = make_uint4(0, 0, 0, 0);
                        // the next row block's copies write the same bytes: plain stores go before them
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&full[s], (filled < primed ? 0 : kWeights * blocks_here) + piece * tile.rows);
                        if (filled >= primed) bulk_load(st, weight, kWeights * blocks_here, &full[s]);
                        const unsigned char* from = x + (int64_t)kb * kTileK * kSize;
                        for (int r = 0; r < tile.rows; ++r, xt += kRow, from += row_bytes) bulk_load(xt, from, piece, &full[s]);
                    }
                }
                __syncwarp();
                weight += kStep * kWeights;
            }
        }
        if (!good && lane == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrTimeout);
        // no copy may be in flight when the CTA ends, whatever its consumers did
        for (int i = max(0, filled - kRing); i < filled; ++i) mbar_wait(&full[i % kRing], (i / kRing) & 1);
        __syncwarp();
        if (splits > 1) {
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
        return;
    }
    bool good = true;
    int stage = 0;
    uint32_t parity = 0;
    for (int rb = rb0; rb < rb1 && good; ++rb) {
        float acc[OWN][NT][4];
#pragma unroll
        for (int u = 0; u < OWN; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n) clear(acc[u][n]);
        // a form for each number of 8-token columns in use
        auto walk = [&](auto columns) {
            constexpr int NL = decltype(columns)::value < NT ? decltype(columns)::value : NT;
            good = consume<NT, OWN, NL, G, FP8>(acc, smem, xs, full, empty, kb1 - kb0, stage, parity);
#pragma unroll
            for (int u = 0; u < OWN; ++u)
#pragma unroll
                for (int n = 0; n < NL; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[u][n][c] *= kUnit<FP8>;      // a power of two
        };
        if (NT == 1 || (NT == 2 && tile.rows <= 8))
            walk(std::integral_constant<int, 1>{});
        else if (NT == 2 || tile.rows <= 16)
            walk(std::integral_constant<int, 2>{});
        else if (tile.rows <= 24)
            walk(std::integral_constant<int, 3>{});
        else
            walk(std::integral_constant<int, 4>{});
        if (!good && lane == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrTimeout);
        if (splits > 1) {
            // share i adds up the tiles i, i + splits, ...: the others send it theirs
            const int owned = kTiles / splits;
            cluster_wait();                    // all CTAs of the cluster have started
#pragma unroll
            for (int u = 0; u < OWN; ++u) {
                const int own = warp * OWN + u;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    cluster_store(parts + ((split * owned + own / splits) * NT + n) * 32 + lane, (uint32_t)(own % splits), acc[u][n]);
            }
            __syncwarp();
            cluster_arrive();
            cluster_wait();
#pragma unroll
            for (int u = 0; u < OWN; ++u) {
                const int own = warp * OWN + u;
                if (own % splits != split) continue;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    clear(acc[u][n]);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        if (r >= splits) break;
                        const float4 v = parts[((r * owned + own / splits) * NT + n) * 32 + lane];
                        acc[u][n][0] += v.x;
                        acc[u][n][1] += v.y;
                        acc[u][n][2] += v.z;
                        acc[u][n][3] += v.w;
                    }
                }
            }
        }
        if (!good) break;
        // 8 channels x 8 tokens at a time: rounded, transposed, 4 bytes a lane
        const int g = lane >> 2, t = lane & 3;
        uint16_t* y = static_cast<uint16_t*>(p.y) + tile.first * p.w.N;
#pragma unroll
        for (int u = 0; u < OWN; ++u) {
            const int own = warp * OWN + u, tile_at = rb * kTiles + own;
            if (own % splits != split) continue;          // another share writes it
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int row = n * 8 + g;
                const float (&v)[4] = acc[u][n];
                if (p.w.paired) {
                    const uint32_t o = transpose8x8(pack_bf16x2(silu(v[0]) * v[2], silu(v[1]) * v[3]));
                    if (row < tile.rows && tile_at * 8 < p.w.N)
                        *reinterpret_cast<uint32_t*>(y + (int64_t)row * p.w.N + tile_at * 8 + 2 * t) = o;
                } else {
                    const uint32_t o0 = transpose8x8(pack_bf16x2(v[0], v[1])), o1 = transpose8x8(pack_bf16x2(v[2], v[3]));
                    uint16_t* to = y + (int64_t)row * p.w.N + tile_at * 16 + 2 * t;
                    if (row < tile.rows && tile_at * 16 < p.w.N) *reinterpret_cast<uint32_t*>(to) = o0;
                    if (row < tile.rows && tile_at * 16 + 8 < p.w.N) *reinterpret_cast<uint32_t*>(to + 8) = o1;
                }
            }
        }
    }
}

size_t w4_smem(const W4Shape& w, int nt, bool fp8, int splits) {
    return kRing * (size_t)stage_bytes(w.group, nt, fp8) + (fp8 ? (size_t)k_blocks(w) * 8 * nt * 4 : 0) + (splits > 1 ? (size_t)kTiles * nt * 32 * 16 : 0);
}

constexpr size_t kMaxSmem = 227 * 1024 - 1024;
constexpr size_t kSmSmem = 228 * 1024;

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Describes x [R, K] for copies of 32 channels x `rows` rows.
cudaError_t describe_rows(const W4Params& p, int rows, CUtensorMap* map) {
    static const EncodeFn encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeFn>(f) : nullptr;
    }();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t size = p.fp8 ? 1 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)p.w.K, (cuuint64_t)p.R}, strides[1] = {(cuuint64_t)p.w.K * size};
    const cuuint32_t box[2] = {32, (cuuint32_t)rows}, steps[2] = {1, 1};
    const CUresult r = encode(map, p.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                              const_cast<void*>(p.x), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Shared memory that a CTA asks for beyond its own needs, so that clusters are
// spread over all SMs: the scheduler fills an SM before it takes the next, and
// with room for four CTAs on each a few clusters would sit on half of them (one
// row, 7168 -> 2 x 2048: 9.1 us so, 6.8 spread out).  At most as many CTAs to an
// SM as leave a place for every cluster: a second wave would cost far more.
template <int NT, int OWN, int G, bool FP8>
size_t spread_clusters(size_t smem, int splits, int64_t ctas, dim3 block) {
    constexpr int kMost = 3;
    static std::atomic<int> places[4][kMost];            // + 1, of clusters of 2, 4 and 8; 0: not asked yet
    const int which = splits == 2 ? 1 : splits == 4 ? 2 : 3;
    for (int per_sm = 1; per_sm <= kMost; ++per_sm) {
        const size_t spread = (size_t)kSmSmem / (per_sm + 1);        // one more does not fit
        if (spread > kMaxSmem || spread < smem) continue;
        std::atomic<int>& known = places[which][per_sm - 1];
        int n = known.load(std::memory_order_relaxed);
        if (n == 0) {
            cudaLaunchConfig_t cfg{};
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = (unsigned)splits;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.gridDim = dim3((unsigned)splits);
            cfg.blockDim = block;
            cfg.dynamicSmemBytes = spread;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, expert_w4_kernel<NT, OWN, G, FP8>, &cfg) != cudaSuccess) {
                (void)cudaGetLastError();
                return smem;
            }
            known.store(++n, std::memory_order_relaxed);
        }
        if ((int64_t)(n - 1) * splits >= ctas) return spread;
    }
    return smem;
}

template <int NT, int OWN, int G, bool FP8>
cudaError_t launch_form(const W4Params& p, int splits, int units, int64_t tiles, cudaStream_t stream) {
    auto kern = expert_w4_kernel<NT, OWN, G, FP8>;
    const dim3 grid((unsigned)(tiles * ((row_blocks(p.w) + units - 1) / units) * splits)), block(block_threads(OWN));
    // the same value whatever a call needs: another thread may be between this and its launch
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
    size_t smem = w4_smem(p.w, NT, FP8, splits);
    if (splits > 1) smem = spread_clusters<NT, OWN, G, FP8>(smem, splits, grid.x, block);
    CUtensorMap map{};
    if (x_boxes(NT)) {
        e = describe_rows(p, 8 * NT, &map);
        if (e != cudaSuccess) return e;
    }
    return launch_clusters(true, splits, kern, grid, block, smem, stream, p, map, splits, units, (int)tiles);
}

template <int NT, int OWN, bool FP8>
cudaError_t launch_group(const W4Params& p, int splits, int units, int64_t tiles, cudaStream_t stream) {
    if (p.w.group == 32) return launch_form<NT, OWN, 32, FP8>(p, splits, units, tiles, stream);
    if (p.w.group == 64) return launch_form<NT, OWN, 64, FP8>(p, splits, units, tiles, stream);
    return launch_form<NT, OWN, 128, FP8>(p, splits, units, tiles, stream);
}

template <int NT>
cudaError_t launch_rows(const W4Params& p, int num_sms, cudaStream_t stream) {
    // every row in a tile of its expert: full tiles, and a last one for each expert in use
    const int64_t tiles = std::min<int64_t>(p.w.E, p.max_rows) + p.max_rows / (8 * NT);
    // tiles there will be: one for each expert in use, or full ones
    const int64_t products = std::max<int64_t>(std::min<int64_t>(p.w.E, p.max_rows), p.max_rows / (8 * NT)) * row_blocks(p.w);
    // few products: share K among the CTAs of a cluster until there are two CTAs for every SM (one with wide tiles, whose
    // sums are larger): one row of 4096 x 7168 11.7 us without, 9.6 with one CTA an SM, 6.9 with two; 16 experts with 32 rows
    // of 1024 -> 2 x 1000 16.0 with one, 24.2 with two
    int splits = 1;
    while (splits < 8 && products * splits < (NT <= 2 ? 2 : 1) * num_sms && k_blocks(p.w) >= 4 * splits) splits *= 2;
    // many short ones: several to a CTA, for at least 64 steps of K, as long as 16 CTAs for every SM remain (256 experts,
    // down, 2048 -> 7168: 361 us one by one, 326 four to a CTA)
    int units = 1;
    while (units * k_blocks(p.w) < 64 && products >= 32 * (int64_t)num_sms * units) units *= 2;
    // few CTAs of wide tiles: one tile a warp (16 rows of 4096 x 4096 8.4 us with two, 7.1 with one; 40 of 4096 -> 2 x 1024 9.8
    // and 8.8; 16 experts with 32 rows of 1024 -> 2 x 1000 16.0 and 19.0, 64 with 16 of 7168 -> 2 x 2048 242 and 291)
    if (NT > 2 && tiles * row_blocks(p.w) * splits <= 2 * num_sms) {
        constexpr int OWN = NT > 2 ? 1 : 2;
        return p.fp8 ? launch_group<NT, OWN, true>(p, splits, units, tiles, stream)
                     : launch_group<NT, OWN, false>(p, splits, units, tiles, stream);
    }
    return p.fp8 ? launch_group<NT, 2, true>(p, splits, units, tiles, stream) : launch_group<NT, 2, false>(p, splits, units, tiles, stream);
}

// Tokens of a tile, in columns of 8: enough for about twice an expert's share of the rows, up to 32 (16 rows an expert, gate
// and up: 282 us with 16 to a tile, 242 with 32; one row of 4096 x 7168: 11.9 with 16, 6.9 with 8).
int token_columns(const W4Shape& w, int64_t max_rows) {
    return max_rows <= 8 ? 1 : max_rows / std::min<int64_t>(w.E, max_rows) <= 8 ? 2 : 4;
}

}  // namespace

size_t w4_bytes(const W4Shape& w) {
    return (size_t)w.E * row_blocks(w) * k_blocks(w) * kTiles * tile_bytes(w.group);
}

bool w4_packs(const W4Shape& w) { return (int64_t)w.E * row_blocks(w) * k_blocks(w) * kTiles <= INT32_MAX; }

bool w4_fits(const W4Shape& w, int64_t max_rows, int fp8) {
    // shared memory of the call's form, sharing K; CTAs of the narrowest
    return w4_smem(w, token_columns(w, max_rows), fp8 != 0, 8) <= kMaxSmem &&
           (std::min<int64_t>(w.E, max_rows) + max_rows / 8) * row_blocks(w) * 8 <= INT32_MAX && max_rows <= (int64_t)1 << 29;
}

cudaError_t launch_w4_pack(const W4Shape& w, const uint8_t* codes, const void* scales, void* packed, cudaStream_t stream) {
    const int64_t tiles = (int64_t)w.E * row_blocks(w) * k_blocks(w) * kTiles;
    return launch_kernel(false, w4_pack_kernel, dim3((unsigned)tiles), dim3(256), 0, stream, w, codes,
                         static_cast<const uint16_t*>(scales), static_cast<unsigned char*>(packed));
}

cudaError_t launch_expert_w4(const W4Params& p, int num_sms, cudaStream_t stream) {
    if (p.max_rows == 0) return cudaSuccess;
    const int nt = token_columns(p.w, p.max_rows);
    return nt == 1 ? launch_rows<1>(p, num_sms, stream) : nt == 2 ? launch_rows<2>(p, num_sms, stream) : launch_rows<4>(p, num_sms, stream);
}

}  // namespace ep
