// expert_i8.cu -- the experts' products over the receive buffer in 8-bit integers:
//   y[r, n] = x_scale[r] * w_scale[e, n] * sum_k x[r, k] * w[e, n, k]
//
// This part multiplies 8-bit integers at 151 TOP/s (mma.sync, measured), f16 at
// thirteen times that, so the codes go through the tensor cores as f16, which
// holds them exactly: a product of two has 15 bits and sums stay exact below 2^24.
// A block of 128 weight rows is the M side of tcgen05.mma, up to 128 token rows the
// N side, 64 input channels a step.  A producer warp keeps a ring of weight codes
// filled by bulk copies; four warps widen them into tensor memory, a row to a
// thread, which is the instruction's A operand; four more load token codes and
// widen them into shared memory (B); one thread issues the products.
#include <algorithm>

#include "block_kernels.h"
#include "expert_rows.cuh"

namespace ep {
namespace {

constexpr int kRows = 128;         // weight rows of a block
constexpr int kStep = 64;          // input channels of a step
constexpr int kStepBytes = kRows * kStep;
constexpr int kOps = 4;            // steps whose operands are widened ahead
constexpr int kThreads = 320;      // four warps of weights, four of tokens, the producer, the issuer
constexpr int kAColumns = kStep / 2;              // tensor memory columns of a step's A operand
constexpr uint32_t kColumns = 256;                // tensor memory columns of a CTA: two on an SM

__host__ __device__ inline int k_steps(const I8Shape& w) { return (w.K + kStep - 1) / kStep; }
// A paired block is 64 gate rows and the 64 up rows of the same channels.
__host__ __device__ inline int block_channels(const I8Shape& w) { return w.paired ? kRows / 2 : kRows; }
__host__ __device__ inline int row_blocks(const I8Shape& w) { return (w.N + block_channels(w) - 1) / block_channels(w); }
__host__ __device__ inline int64_t scales_at(const I8Shape& w) { return (int64_t)w.E * row_blocks(w) * k_steps(w) * kStepBytes; }

// Output channel of row r of block b, and whether it is an up row: every warp's 32
// rows are 16 gate rows and their 16 up rows.
__host__ __device__ inline int channel_of(const I8Shape& w, int b, int r, bool* up) {
    *up = w.paired && (r & 16);
    return w.paired ? b * 64 + (r >> 5) * 16 + (r & 15) : b * kRows + r;
}

// The order in which a step's 64 channels enter the products.  A thread that
// widens 16 neighbouring channels of a token writes two runs of 8; runs
// 16-channel groups apart are neighbours, so that eight lanes' writes fall into
// different banks: run h * 4 + c holds channels 16 c + 8 h and up.
__host__ __device__ constexpr int run_channel(int run) { return (run & 3) * 16 + (run >> 2) * 8; }

// Packed: steps [E][row block][step][two runs][row][16 bytes], codes plus 128;
// then the scales [E][row block][row].
__global__ void __launch_bounds__(256) i8_pack_kernel(I8Shape w, const int8_t* codes, const float* scales, unsigned char* packed) {
    const int64_t step = blockIdx.x;
    const int nk = k_steps(w), nb = row_blocks(w), rows = w.paired ? 2 * w.N : w.N;
    const int kt = (int)(step % nk), b = (int)(step / nk % nb), e = (int)(step / nk / nb);
    for (int i = threadIdx.x; i < kStepBytes / 8; i += blockDim.x) {
        const int r = i / 2 % kRows, run = i / 2 / kRows * 2 + i % 2, k = kt * kStep + run_channel(run);
        bool up;
        const int c = channel_of(w, b, r, &up);
        uint2 v = make_uint2(0x80808080u, 0x80808080u);
        if (c < w.N && k < w.K) {
            v = *reinterpret_cast<const uint2*>(codes + ((int64_t)e * rows + (up ? w.N : 0) + c) * w.K + k);
            v.x ^= 0x80808080u;
            v.y ^= 0x80808080u;
        }
        reinterpret_cast<uint2*>(packed + step * kStepBytes)[i] = v;
    }
    if (kt == 0 && threadIdx.x < kRows) {
        bool up;
        const int c = channel_of(w, b, threadIdx.x, &up);
        reinterpret_cast<float*>(packed + scales_at(w))[((int64_t)e * nb + b) * kRows + threadIdx.x] =
            c < w.N ? scales[(int64_t)e * rows + (up ? w.N : 0) + c] : 0.f;
    }
}

// ------------------------------------------------------------ tensor cores

__device__ __forceinline__ void tmem_alloc(uint32_t* at, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}

__device__ __forceinline__ void tcgen05_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrives on `bar` once every product issued so far by this thread is done.
__device__ __forceinline__ void tcgen05_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// D[128, n] (+)= A[128, 16] B[n, 16]^T, f16 operands, fp32 sums; A and D in tensor memory.
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
        : "memory");
}

// 32 columns of a warp's 32 rows of tensor memory, one row to a lane.
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
        "%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
        "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
        "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
          "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at)
        : "memory");
}

// Four codes plus 128 -> two pairs of f16: a byte below 0x64 is 1024 + byte, and
// 1152 less is the code.  Exact.
__device__ __forceinline__ void widen(uint32_t biased, uint32_t* lo, uint32_t* hi) {
    const uint32_t a = __byte_perm(biased, 0x64646464u, 0x4140), b = __byte_perm(biased, 0x64646464u, 0x4342);
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(*lo) : "r"(a), "r"(0xe480e480u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(*hi) : "r"(b), "r"(0xe480e480u));
}

// ------------------------------------------------------------------ kernel

// A step's B operand: runs of 8 channels of NT rows, 16 bytes a row, runs
// (NT + 2) * 16 bytes apart (the 32 bytes more keep neighbouring runs' rows in
// different banks).
template <int NT>
constexpr int kRunBytes = (NT + 2) * 16;
template <int NT>
constexpr int kBBytes = kStep / 8 * kRunBytes<NT>;
template <int NT, int RING>
constexpr int kSmemBytes = RING * kStepBytes + kOps * kBBytes<NT>;

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t in_cta(uint32_t smem, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
    return a;
}

// One CTA: a block of 128 weight rows with one tile of up to NT token rows, over
// one of `splits` shares of K.  The shares of a product form a cluster; each
// owns a part of the tile's token rows, whose sums the others push to it.
template <int NT, int RING>
__global__ void __launch_bounds__(kThreads, 2) expert_i8_kernel(I8Params p, int splits, int grid_tiles) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t ring_full[RING], ring_empty[RING], op_full[kOps], op_empty[kOps], done;
    __shared__ uint32_t tmem_at;
    __shared__ RowTile shared_tile;
    __shared__ float row_scale[NT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x % splits, nb = row_blocks(p.w), nk = k_steps(p.w);
    const int b = blockIdx.x / splits % nb, at = blockIdx.x / splits / nb;
    const int k0 = (int)((int64_t)nk * split / splits), k1 = (int)((int64_t)nk * (split + 1) / splits);
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(&ring_full[i], 1);
            mbar_init(&ring_empty[i], 4);
        }
        for (int i = 0; i < kOps; ++i) {
            mbar_init(&op_full[i], 8);
            mbar_init(&op_empty[i], 1);
        }
        mbar_init(&done, 1);
        fence_mbar_init();
    }
    // a share may push to another once that runs
    if (splits > 1) {
        __syncwarp();
        cluster_barrier();
    }
    pdl_wait();
    // not before the wait: a CTA that holds tensor memory must not wait for one that may need it
    if (warp == 9) tmem_alloc(&tmem_at, kColumns);
    if (warp == 0) {
        const RowTile r = p.w.E == 1 ? tile_of_one(p, at, NT, grid_tiles) : find_tile(p, at, NT, grid_tiles);
        if (lane == 0) shared_tile = r;
    }
    tcgen05_before();
    __syncthreads();
    tcgen05_after();
    const RowTile tile = shared_tile;
    const uint32_t tmem = tmem_at;
    if (tile.e >= 0) {
        const int rows = tile.rows, cols = (rows + 15) & ~15;      // the products' N: a multiple of 16
        unsigned char* ring = smem;
        unsigned char* ops = smem + RING * kStepBytes;
        const uint32_t a_at = tmem + NT;                           // past the sums' columns
        bool good = true;
        if (warp == 8) {
            const unsigned char* weights = static_cast<const unsigned char*>(p.packed) + (((int64_t)tile.e * nb + b) * nk + k0) * kStepBytes;
            int filled = 0;
            for (; filled < k1 - k0; ++filled) {
                const int s = filled % RING;
                if (filled >= RING && !__all_sync(0xffffffffu, mbar_wait(&ring_empty[s], (filled / RING - 1) & 1))) {
                    good = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&ring_full[s], kStepBytes);
                    bulk_load(ring + s * kStepBytes, weights + (int64_t)filled * kStepBytes, kStepBytes, &ring_full[s]);
                }
                __syncwarp();
            }
            // no copy may be in flight when the CTA ends, whatever its consumers did
            for (int i = max(0, filled - RING); i < filled; ++i) mbar_wait(&ring_full[i % RING], (i / RING) & 1);
        } else if (warp == 9) {
            const uint32_t kind = 1u << 4 | (uint32_t)(cols / 8) << 17 | (kRows / 16) << 24;      // fp32 sums, f16 operands, N, M
            // runs of 8 channels kRunBytes apart, 8 rows 128 bytes apart, no swizzle
            const uint64_t desc = (uint64_t)(kRunBytes<NT> / 16) << 16 | (uint64_t)(128 / 16) << 32 | (uint64_t)1 << 46;
            for (int i = 0; i < k1 - k0; ++i) {
                const int s = i % kOps;
                if (!__all_sync(0xffffffffu, mbar_wait(&op_full[s], (i / kOps) & 1))) {
                    good = false;
                    break;
                }
                tcgen05_after();
                if (lane == 0) {
                    const uint32_t from = smem_addr(ops + s * kBBytes<NT>);
#pragma unroll
                    for (int j = 0; j < kStep / 16; ++j)
                        mma_f16(tmem, a_at + s * kAColumns + j * 8, desc | ((from + j * 2 * kRunBytes<NT>) >> 4 & 0x3fff), kind, i > 0 || j > 0);
                    tcgen05_commit(&op_empty[s]);
                }
                __syncwarp();
            }
            if (lane == 0) tcgen05_commit(&done);
            __syncwarp();
            good = __all_sync(0xffffffffu, mbar_wait(&done, 0)) && good;
        } else if (warp >= 4) {
            // tokens: a thread has 16 channels of every 32nd row
            const int t = threadIdx.x - 128, c = t & 3, n0 = t >> 2;
            const int8_t* x = p.x + tile.first * p.w.K + c * 16;
            for (int n = t; n < NT; n += 128) row_scale[n] = n < rows ? p.x_scales[tile.first + n] : 0.f;
            uint4 raw[NT / 32];
            auto fetch = [&](int step) {
                const int k = (k0 + step) * kStep;
#pragma unroll
                for (int j = 0; j < NT / 32; ++j) {
                    raw[j] = make_uint4(0, 0, 0, 0);               // channels past the end
                    const int n = n0 + 32 * j;
                    if (n < rows && step < k1 - k0 && k + c * 16 < p.w.K) raw[j] = *reinterpret_cast<const uint4*>(x + (int64_t)n * p.w.K + k);
                }
            };
            fetch(0);
            for (int i = 0; i < k1 - k0; ++i) {
                const int s = i % kOps;
                if (i >= kOps && !__all_sync(0xffffffffu, mbar_wait(&op_empty[s], (i / kOps - 1) & 1))) {
                    good = false;
                    break;
                }
                unsigned char* to = ops + s * kBBytes<NT> + c * kRunBytes<NT>;
#pragma unroll
                for (int j = 0; j < NT / 32; ++j) {
                    const int n = n0 + 32 * j;
                    if (n < rows) {
                        uint4 lo, hi;
                        widen(raw[j].x ^ 0x80808080u, &lo.x, &lo.y);
                        widen(raw[j].y ^ 0x80808080u, &lo.z, &lo.w);
                        widen(raw[j].z ^ 0x80808080u, &hi.x, &hi.y);
                        widen(raw[j].w ^ 0x80808080u, &hi.z, &hi.w);
                        *reinterpret_cast<uint4*>(to + n * 16) = lo;
                        *reinterpret_cast<uint4*>(to + 4 * kRunBytes<NT> + n * 16) = hi;
                    }
                }
                fetch(i + 1);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&op_full[s]);
            }
        } else {
            // weights: a thread has one row
            for (int i = 0; i < k1 - k0; ++i) {
                const int s = i % kOps, r = i % RING;
                if (!__all_sync(0xffffffffu, mbar_wait(&ring_full[r], (i / RING) & 1))) {
                    good = false;
                    break;
                }
                uint32_t v[32];
                const unsigned char* from = ring + r * kStepBytes + threadIdx.x * 16;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 raw = *reinterpret_cast<const uint4*>(from + q * kRows * 16);
                    widen(raw.x, &v[q * 8], &v[q * 8 + 1]);
                    widen(raw.y, &v[q * 8 + 2], &v[q * 8 + 3]);
                    widen(raw.z, &v[q * 8 + 4], &v[q * 8 + 5]);
                    widen(raw.w, &v[q * 8 + 6], &v[q * 8 + 7]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ring_empty[r]);
                if (i >= kOps && !__all_sync(0xffffffffu, mbar_wait(&op_empty[s], (i / kOps - 1) & 1))) {
                    good = false;
                    break;
                }
                tcgen05_after();
                tmem_store32(a_at + s * kAColumns + ((uint32_t)warp * 32 << 16), v);
                tmem_store_wait();
                tcgen05_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&op_full[s]);
            }
            good = __all_sync(0xffffffffu, mbar_wait(&done, 0)) && good;
            tcgen05_after();
        }
        __syncwarp();
        good = __syncthreads_and(good);
        if (!good && threadIdx.x == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrTimeout);
        // epilogue: a thread has one weight row, 16 tokens at a time
        const int own = (rows + splits - 1) / splits;              // token rows that a share of K owns
        float* parts = reinterpret_cast<float*>(ops + kOps * kBBytes<NT>);       // [share][own][weight row]
        if (splits > 1) {
            if (warp < 4 && good) {
                for (int n0 = 0; n0 < rows; n0 += 16) {
                    uint32_t v[16];
                    tmem_load16(tmem + n0 + ((uint32_t)warp * 32 << 16), v);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (n0 + j < rows) {
                            const int owner = (n0 + j) / own;
                            const uint32_t to = in_cta(smem_addr(parts + ((int64_t)split * own + n0 + j - owner * own) * kRows + threadIdx.x), owner);
                            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to), "r"(v[j]) : "memory");
                        }
                }
            }
            __syncwarp();
            cluster_barrier();
        }
        if (warp < 4 && good) {
            bool up;
            const int c = channel_of(p.w, b, threadIdx.x, &up);
            const float scale = reinterpret_cast<const float*>(static_cast<const unsigned char*>(p.packed) + scales_at(p.w))[((int64_t)tile.e * nb + b) * kRows + threadIdx.x];
            uint16_t* y = static_cast<uint16_t*>(p.y) + tile.first * p.w.N + c;
            auto finish = [&](int n, float sum) {
                float f = sum * scale * row_scale[n];
                if (p.w.paired) f = silu(f) * __shfl_xor_sync(0xffffffffu, f, 16);
                if (c < p.w.N && !up) y[(int64_t)n * p.w.N] = (uint16_t)pack_bf16x2(f, 0.f);
            };
            if (splits > 1) {
                for (int n = split * own; n < min(rows, (split + 1) * own); ++n) {
                    float sum = 0.f;
                    for (int q = 0; q < splits; ++q) sum += parts[((int64_t)q * own + n - split * own) * kRows + threadIdx.x];
                    finish(n, sum);
                }
            } else {
                for (int n0 = 0; n0 < rows; n0 += 16) {
                    uint32_t v[16];
                    tmem_load16(tmem + n0 + ((uint32_t)warp * 32 << 16), v);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (n0 + j < rows) finish(n0 + j, __uint_as_float(v[j]));
                }
            }
            tcgen05_before();
        }
    }
    __syncthreads();
    if (warp == 9) {
        tcgen05_after();
        tmem_free(tmem, kColumns);
    }
}

// Tiles of up to `tile` rows that max_rows rows of E experts make at most.
int64_t most_tiles(int E, int64_t max_rows, int tile) {
    const int64_t used = std::min<int64_t>(E, max_rows);
    return used + (max_rows - used) / tile;
}

template <int NT, int RING>
cudaError_t launch(const I8Params& p, int num_sms, cudaStream_t stream) {
    const int64_t tiles = most_tiles(p.w.E, p.max_rows, NT), products = tiles * row_blocks(p.w);
    int splits = 1;
    while (splits < 8 && products * splits * 2 <= 2 * num_sms && k_steps(p.w) >= splits * 4) splits *= 2;
    const size_t smem = kSmemBytes<NT, RING> + (splits > 1 ? (size_t)(NT + splits) * kRows * 4 : 0);
    auto kern = expert_i8_kernel<NT, RING>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<NT, RING> + (NT + 8) * kRows * 4);
    if (e != cudaSuccess) return e;
    return launch_clusters(true, splits, kern, dim3((unsigned)(products * splits)), dim3(kThreads), smem, stream, p, splits, (int)tiles);
}

}  // namespace

size_t i8_bytes(const I8Shape& w) { return (size_t)scales_at(w) + (size_t)w.E * row_blocks(w) * kRows * sizeof(float); }

bool i8_packs(const I8Shape& w) { return (int64_t)w.E * row_blocks(w) * k_steps(w) <= INT32_MAX; }

bool i8_fits(const I8Shape& w, int64_t max_rows) { return most_tiles(w.E, max_rows, 32) * row_blocks(w) <= INT32_MAX / 8; }

cudaError_t launch_i8_pack(const I8Shape& w, const int8_t* codes, const float* scales, void* packed, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)w.E * row_blocks(w) * k_steps(w)));
    return launch_kernel(false, i8_pack_kernel, grid, dim3(256), 0, stream, w, codes, scales, static_cast<unsigned char*>(packed));
}

cudaError_t launch_expert_i8(const I8Params& p, int num_sms, cudaStream_t stream) {
    return p.max_rows <= (int64_t)24 * p.w.E ? launch<32, 10>(p, num_sms, stream) : launch<128, 5>(p, num_sms, stream);
}

}  // namespace ep
