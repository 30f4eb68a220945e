// expert_i8.cu -- the experts' products over the receive buffer in 8-bit integers:
//   y[r, n] = x_scale[r] * w_scale[e, n] * sum_k x[r, k] * w[e, n, k]
//
// This part multiplies 8-bit integers at 151 TOP/s (mma.sync, measured), f16 at
// thirteen times that, so the codes go through the tensor cores as f16, which
// holds them exactly: a product of two has 15 bits and sums stay exact below 2^24.
// Two blocks of 128 weight rows are the M side of tcgen05.mma, up to 128 token rows
// the N side of both, 128 input channels a step.  One CTA an SM takes item after
// item (two blocks with one tile of token rows).  A warp finds the items; a
// producer warp keeps a ring of weight codes filled by bulk copies; eight warps
// widen them into tensor memory, a row to a thread, which is the instruction's A
// operand; eight more load token codes and widen them into shared memory (B), and
// write the sums out; one thread issues the products.
#include <algorithm>

#include "ep.h"

#include "block_kernels.h"
#include "expert_rows.cuh"

namespace ep {
namespace {

constexpr int kRows = 128;         // weight rows of a block
constexpr int kTokens = 128;       // most token rows of a tile
constexpr int kStep = 128;         // input channels of a step
constexpr int kStepBytes = kRows * kStep;
constexpr int kMaxRing = 6;        // steps of weight codes
constexpr int kA = 2;              // steps whose weights are widened ahead
constexpr int kB = 3;              // steps whose tokens are
constexpr int kSteps = 6;          // barriers of steps under way: a multiple of both
constexpr int kItems = 4;          // items found ahead
constexpr int kAhead = 2;          // steps whose token codes are on their way
// warps: 8 of weights, 8 of tokens, the producer, the issuer, the one that finds items
constexpr int kProducer = 16, kIssuer = 17, kFinder = 18;
constexpr int kThreads = 19 * 32;
constexpr int kItemReaders = 18;
constexpr uint32_t kColumns = 512;                // tensor memory: the two blocks' sums, then kA x 2 A operands
constexpr int kAColumns = kStep / 2;

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

// The order in which a step's 128 channels enter the products.  A thread that
// widens 16 neighbouring channels of a token writes two runs of 8; runs
// 16-channel groups apart are neighbours, so that eight lanes' writes fall into
// different banks: run h * 8 + c holds channels 16 c + 8 h and up.
__host__ __device__ constexpr int run_channel(int run) { return (run & 7) * 16 + (run >> 3) * 8; }

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

// One thread of a whole warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Four codes plus 128 -> two pairs of f16: a byte below 0x64 is 1024 + byte, and
// 1152 less is the code.  Exact.
__device__ __forceinline__ void widen(uint32_t biased, uint32_t* lo, uint32_t* hi) {
    const uint32_t a = __byte_perm(biased, 0x64646464u, 0x4140), b = __byte_perm(biased, 0x64646464u, 0x4342);
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(*lo) : "r"(a), "r"(0xe480e480u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(*hi) : "r"(b), "r"(0xe480e480u));
}

// ------------------------------------------------------------------ kernel

// A step's B operand: runs of 8 channels of up to tile_rows rows, 16 bytes a row;
// 16 bytes more keep the runs that eight lanes write at once in different banks.
// What shared memory is left holds the ring of weight codes.
constexpr int kRuns = kStep / 8;
constexpr int kSmemBytes = 208 * 1024;

__host__ __device__ constexpr int run_bytes(int tile_rows) { return (tile_rows + 1) * 16; }
__host__ __device__ constexpr int ring_steps(int tile_rows) {
    const int fit = (kSmemBytes - kB * kRuns * run_bytes(tile_rows)) / (2 * kStepBytes);
    return fit < kMaxRing ? fit : kMaxRing;
}
static_assert(ring_steps(kTokens) >= 3, "the widest tile leaves too little for the ring");

// Waits for a phase, at most kWaitLimitNs and a few tries.  A try suspends the
// thread for a while by itself, which leaves the issue slots to others; the clock
// is looked at once in 64 of them.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t tries = 1;; ++tries) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (done) return true;
        if (tries % 64 == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitLimitNs) return false;
        }
    }
}

// A place in a ring and the parity of its phase.
struct Place {
    int at = 0;
    uint32_t parity = 0;

    __device__ __forceinline__ void next(int size) {
        if (++at == size) {
            at = 0;
            parity ^= 1;
        }
    }
};

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t in_cta(uint32_t smem, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
    return a;
}

// Two blocks of weight rows (one where `two` is not set) with a tile of token rows.
struct Item {
    int e;            // expert, -1: no more
    int rows;
    int first;        // the tile's first row
    int b;            // the first block
    int two;
};

// Tiles of n rows: as few as hold them, each of about as many rows, in 16s (which
// is never more than `tile` while n rows need them all).
__device__ __forceinline__ int tile_rows_of(int n, int tile) {
    const int tiles = (n + tile - 1) / tile;
    return ((n + tiles - 1) / tiles + 15) & ~15;
}

// The sums of a weight row to a lane, scaled, paired and stored.
struct Writer {
    uint16_t* y;             // at the lane's channel of the tile's first row (the upper lanes' of a pair: of the second)
    const float* row_scale;  // of the tile's first row
    float scale;
    int N, rows;
    bool paired, stores;

    __device__ __forceinline__ Writer(const I8Params& p, const Item& it, int b, int row) {
        bool up;
        const int c = channel_of(p.w, b, row, &up);
        scale = reinterpret_cast<const float*>(static_cast<const unsigned char*>(p.packed) + scales_at(p.w))[((int64_t)it.e * row_blocks(p.w) + b) * kRows + row];
        N = p.w.N;
        paired = p.w.paired;
        y = static_cast<uint16_t*>(p.y) + (int64_t)it.first * N + c + (paired && (threadIdx.x & 16) ? N : 0);
        row_scale = p.x_scales + it.first;
        rows = it.rows;
        stores = c < N;
    }

    // Token rows n and n + 1.  xs(r): the scale of row r (r = n or n + 1 in a lane).  Of a pair, the lower
    // lanes have the gates and finish row n, the upper ones have the ups and finish row n + 1.
    template <typename Scale>
    __device__ __forceinline__ void put(int n, float s0, float s1, Scale xs) const {
        const bool upper = threadIdx.x & 16;
        const float a = s0 * scale, b = s1 * scale;
        uint16_t* to = y + (int64_t)n * N;
        if (paired) {
            const float other = __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
            const int r = n + upper;
            const float f = xs(r), gate = (upper ? other : a) * f, up = (upper ? b : other) * f;
            const uint16_t out = (uint16_t)pack_bf16x2(silu(gate) * up, 0.f);
            if (stores && r < rows) *to = out;
        } else {
            const float f0 = xs(n), f1 = xs(n + 1);
            if (stores && n < rows) *to = (uint16_t)pack_bf16x2(a * f0, 0.f);
            if (stores && n + 1 < rows) to[N] = (uint16_t)pack_bf16x2(b * f1, 0.f);
        }
    }
};

// items: a grid of clusters of `splits` CTAs takes them a grid apart; with more
// than one share of K (which a launch of few products has) a cluster takes one.
__global__ void __launch_bounds__(kThreads, 1) expert_i8_kernel(I8Params p, int splits, int tile_rows) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t ring_full[kMaxRing], ring_empty[kMaxRing], op_full[kSteps], op_done[kSteps], item_full[kItems], item_empty[kItems];
    __shared__ uint64_t done, drained;
    __shared__ uint32_t tmem_at;
    __shared__ Item items[kItems];
    __shared__ int table_first[EP_MAX_EXPERTS], table_rows[EP_MAX_EXPERTS], table_upto[EP_MAX_EXPERTS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x % splits, cluster = blockIdx.x / splits, clusters = gridDim.x / splits;
    const int nb = row_blocks(p.w), nk = k_steps(p.w);
    const int k0 = (int)((int64_t)nk * split / splits), steps = (int)((int64_t)nk * (split + 1) / splits) - k0;
    const int ring = ring_steps(tile_rows), run = run_bytes(tile_rows), b_bytes = kRuns * run;
    unsigned char* ops = smem + ring * 2 * kStepBytes;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < ring; ++i) {
            mbar_init(&ring_full[i], 1);
            mbar_init(&ring_empty[i], 8);
        }
        for (int i = 0; i < kSteps; ++i) {
            mbar_init(&op_full[i], 16);
            mbar_init(&op_done[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], kItemReaders);
        }
        mbar_init(&done, 1);
        mbar_init(&drained, 8);
        fence_mbar_init();
    }
    pdl_wait();
    // not before the wait: a CTA that holds tensor memory must not wait for one that may need it
    if (warp == kIssuer) tmem_alloc(&tmem_at, kColumns);
    for (int e = threadIdx.x; e < p.w.E; e += kThreads) {
        int64_t first;
        bool bad;
        table_rows[e] = expert_rows(p, e, &first, &bad);
        table_first[e] = (int)first;
        if (bad && blockIdx.x == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrBadSlot);
    }
    tcgen05_before();
    __syncthreads();
    tcgen05_after();
    const uint32_t tmem = tmem_at, a_at = tmem + 2 * kTokens;
    bool good = true;
    auto await = [&](uint64_t* bar, uint32_t parity) {
        good = __all_sync(0xffffffffu, wait_phase(bar, parity));
        return good;
    };
    auto next_item = [&](int j, Item* it) {
        const int slot = j % kItems;
        if (!await(&item_full[slot], (j / kItems) & 1)) return false;
        *it = items[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[slot]);
        return it->e >= 0;
    };
    Item it;
    if (warp == kFinder) {
        // tiles up to and with each expert: lane l adds up those of experts [l * per, (l + 1) * per)
        const int per = (p.w.E + 31) / 32, e0 = min(lane * per, p.w.E), e1 = min(e0 + per, p.w.E);
        int mine = 0;
        for (int e = e0; e < e1; ++e) {
            mine = min(mine + (table_rows[e] + tile_rows - 1) / tile_rows, 1 << 25);      // bad offsets may claim rows many times
            table_upto[e] = mine;
        }
        int before = 0, total = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, total, d);
            if (lane >= d) total += v;
        }
        before = total - mine;
        total = __shfl_sync(0xffffffffu, total, 31);
        for (int e = e0; e < e1; ++e) table_upto[e] += before;
        __syncwarp();
        const int pairs = (nb + 1) / 2;
        const int64_t all_items = (int64_t)total * pairs, most = splits > 1 ? min(all_items, (int64_t)clusters) : all_items;
        if (most < all_items && blockIdx.x == 0 && lane == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrCapacity);
        for (int j = 0;; ++j) {
            const int slot = j % kItems;
            const int64_t at = cluster + (int64_t)j * clusters;
            if (j >= kItems && !await(&item_empty[slot], (j / kItems - 1) & 1)) break;
            it.e = -1;
            if (at < most) {
                const int tile = (int)(at / pairs);
                int lo = 0, hi = p.w.E - 1;                    // the first expert with upto > tile
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (table_upto[mid] > tile)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                const int n = table_rows[lo], size = tile_rows_of(n, tile_rows), from = (tile - (lo > 0 ? table_upto[lo - 1] : 0)) * size;
                it.e = lo;
                it.rows = min(size, n - from);
                it.first = table_first[lo] + from;
                it.b = (int)(at - (int64_t)tile * pairs) * 2;
                it.two = it.b + 1 < nb;
            }
            if (lane == 0) {
                items[slot] = it;
                mbar_arrive(&item_full[slot]);
            }
            __syncwarp();
            if (it.e < 0) break;
        }
    } else if (warp == kProducer) {
        int64_t filled = 0;
        Place r{0, 1};                           // the parity of the place's previous use
        for (int j = 0; next_item(j, &it); ++j) {
            const unsigned char* weights = static_cast<const unsigned char*>(p.packed) + (((int64_t)it.e * nb + it.b) * nk + k0) * kStepBytes;
            for (int i = 0; i < steps; ++i, ++filled, weights += kStepBytes, r.next(ring)) {
                if (filled >= ring && !await(&ring_empty[r.at], r.parity)) break;
                if (lane == 0) {
                    unsigned char* to = smem + r.at * 2 * kStepBytes;
                    mbar_arrive_expect_tx(&ring_full[r.at], it.two ? 2 * kStepBytes : kStepBytes);
                    bulk_load(to, weights, kStepBytes, &ring_full[r.at]);
                    if (it.two) bulk_load(to + kStepBytes, weights + (int64_t)nk * kStepBytes, kStepBytes, &ring_full[r.at]);
                }
                __syncwarp();
            }
            if (!good) break;
        }
        // no copy may be in flight when the CTA ends, whatever its consumers did
        for (int64_t i = max((int64_t)0, filled - ring); i < filled; ++i) wait_phase(&ring_full[i % ring], (i / ring) & 1);
    } else if (warp == kIssuer) {
        // one thread from here to its end: the products' operands then stay in uniform registers
        if (elect_one()) {
            // runs of 8 channels `run` bytes apart, 8 rows 128 bytes apart, no swizzle
            const uint32_t run16 = run / 16;
            const uint64_t desc = (uint64_t)run16 << 16 | (uint64_t)(128 / 16) << 32 | (uint64_t)1 << 46;
            const uint64_t first_b = desc | (smem_addr(ops) >> 4 & 0x3fff);          // in a cluster, addresses have a rank above
            int committed = 0;
            Place g, a, b;
            for (int j = 0;; ++j) {
                const int slot = j % kItems;
                good = wait_phase(&item_full[slot], (j / kItems) & 1);
                if (!good) break;
                const int e = items[slot].e, rows = items[slot].rows, two = items[slot].two;
                mbar_arrive(&item_empty[slot]);
                if (e < 0) break;
                const uint32_t cols = (rows + 15) & ~15;           // the products' N: a multiple of 16
                const uint32_t kind = 1u << 4 | (cols / 8) << 17 | (uint32_t)(kRows / 16) << 24;      // fp32 sums, f16 operands, N, M
                if (j > 0) good = wait_phase(&drained, (j - 1) & 1);
                for (int i = 0; i < steps && good; ++i, g.next(kSteps), a.next(kA), b.next(kB)) {
                    good = wait_phase(&op_full[g.at], g.parity);
                    if (!good) break;
                    tcgen05_after();
                    const uint32_t from_a = a_at + a.at * 2 * kAColumns;
                    const uint64_t from_b = first_b + (uint32_t)(b.at * kRuns) * run16;
#pragma unroll
                    for (int k = 0; k < kStep / 16; ++k) mma_f16(tmem, from_a + k * 8, from_b + k * 2 * run16, kind, i > 0 || k > 0);
                    if (two)
#pragma unroll
                        for (int k = 0; k < kStep / 16; ++k)
                            mma_f16(tmem + kTokens, from_a + kAColumns + k * 8, from_b + k * 2 * run16, kind, i > 0 || k > 0);
                    tcgen05_commit(&op_done[g.at]);
                }
                tcgen05_commit(&done);
                ++committed;
                if (!good) break;
            }
            // every product is over before tensor memory is given back
            if (committed > 0) good = wait_phase(&done, (committed - 1) & 1) && good;
        }
        __syncwarp();
        good = __all_sync(0xffffffffu, good);
    } else if (warp >= 8) {
        // tokens: a thread has 16 channels of every 32nd row
        const int t = threadIdx.x - 256, c = t & 7, n0 = t >> 3, half = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
        uint4 raw[kAhead][kTokens / 32];
        int j = 0, made = 0;                     // made: steps, up to kB
        Place g, b, before;                      // this step's barrier and room; the barrier of the room's last step
        Item last{};
        auto write_out = [&](int item) {
            if (!await(&done, item & 1)) return;
            tcgen05_after();
            if (half == 0 || last.two) {
                const Writer w(p, last, last.b + half, row);
                for (int n = 0; n < last.rows; n += 16) {
                    uint32_t v[16];
                    const float mine = (lane & 15) + n < last.rows ? w.row_scale[n + (lane & 15)] : 0.f;
                    tmem_load16(tmem + half * kTokens + n + lanes, v);
#pragma unroll
                    for (int i = 0; i < 16; i += 2)
                        w.put(n + i, __uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                              [&](int r) { return __shfl_sync(0xffffffffu, mine, r - n); });
                }
            }
            tcgen05_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&drained);
        };
        for (; next_item(j, &it); ++j) {
            const int8_t* x = p.x + (int64_t)it.first * p.w.K + (int64_t)k0 * kStep + c * 16;
            const int left = p.w.K - k0 * kStep - c * 16;          // channels from the thread's on
            auto fetch = [&](uint4 (&r)[kTokens / 32], int step) {
                const bool in = step < steps && step * kStep < left;
#pragma unroll
                for (int i = 0; i < kTokens / 32; ++i) {
                    const int n = n0 + 32 * i;
                    r[i] = make_uint4(0, 0, 0, 0);                 // channels past the end
                    if (n < it.rows && in) r[i] = *reinterpret_cast<const uint4*>(x + (uint32_t)n * (uint32_t)p.w.K + (uint32_t)(step * kStep));
                }
            };
#pragma unroll
            for (int u = 0; u < kAhead; ++u) fetch(raw[u], u);
            for (int base = 0; base < steps && good; base += kAhead) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int i = base + u;
                    if (i >= steps || !good) break;
                    // the next item's first steps are made while the products of this one end; then its sums are written out
                    if (i == kB - 1 && j > 0 && splits == 1) {
                        write_out(j - 1);
                        if (!good) break;
                    }
                    if (made < kB) {
                        ++made;
                    } else {
                        if (!await(&op_done[before.at], before.parity)) break;
                        before.next(kSteps);
                    }
                    unsigned char* to = ops + b.at * b_bytes + c * run;
#pragma unroll
                    for (int m = 0; m < kTokens / 32; ++m) {
                        const int n = n0 + 32 * m;
                        if (n < it.rows) {
                            uint4 lo, hi;
                            widen(raw[u][m].x ^ 0x80808080u, &lo.x, &lo.y);
                            widen(raw[u][m].y ^ 0x80808080u, &lo.z, &lo.w);
                            widen(raw[u][m].z ^ 0x80808080u, &hi.x, &hi.y);
                            widen(raw[u][m].w ^ 0x80808080u, &hi.z, &hi.w);
                            *reinterpret_cast<uint4*>(to + n * 16) = lo;
                            *reinterpret_cast<uint4*>(to + 8 * run + n * 16) = hi;
                        }
                    }
                    fetch(raw[u], i + kAhead);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&op_full[g.at]);
                    g.next(kSteps);
                    b.next(kB);
                }
            }
            if (!good) break;
            if (j > 0 && splits == 1 && steps < kB) write_out(j - 1);
            if (!good) break;
            last = it;
        }
        if (good && j > 0 && splits == 1) write_out(j - 1);
        it = last;
        if (j == 0) it.e = -1;
    } else {
        // weights: a thread has one row of one block
        const int half = warp >> 2;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
        int made = 0;
        Place g, a, r, before;
        for (int j = 0; next_item(j, &it); ++j) {
            const bool here = half == 0 || it.two;
            for (int i = 0; i < steps; ++i) {
                if (!await(&ring_full[r.at], r.parity)) break;
                uint32_t v[2][32];
                if (here) {
                    const unsigned char* from = smem + (r.at * 2 + half) * kStepBytes + (threadIdx.x & 127) * 16;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const uint4 raw = *reinterpret_cast<const uint4*>(from + q * kRows * 16);
                        uint32_t* to = &v[q >> 2][(q & 3) * 8];
                        widen(raw.x, to, to + 1);
                        widen(raw.y, to + 2, to + 3);
                        widen(raw.z, to + 4, to + 5);
                        widen(raw.w, to + 6, to + 7);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ring_empty[r.at]);
                if (made < kA) {
                    ++made;
                } else {
                    if (!await(&op_done[before.at], before.parity)) break;
                    before.next(kSteps);
                }
                if (here) {
                    tcgen05_after();
                    const uint32_t to = a_at + (a.at * 2 + half) * kAColumns + lanes;
                    tmem_store32(to, v[0]);
                    tmem_store32(to + 32, v[1]);
                    tmem_store_wait();
                    tcgen05_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&op_full[g.at]);
                g.next(kSteps);
                a.next(kA);
                r.next(ring);
            }
            if (!good) break;
        }
    }
    __syncwarp();
    if (!good && lane == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrTimeout);
    good = __syncthreads_and(good);
    if (splits > 1) {
        // the shares' sums: each CTA owns some of the tile's token rows, whose sums the others push to it
        cluster_barrier();                       // the rings are free
        float* parts = reinterpret_cast<float*>(smem);         // [share][own][block][weight row]
        const int half = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
        const bool writes = warp >= 8 && warp < 16 && it.e >= 0 && (half == 0 || it.two);
        const int own = (it.rows + splits - 1) / splits;
        if (writes && good) {
            tcgen05_after();
            for (int n = 0; n < it.rows; n += 16) {
                uint32_t v[16];
                tmem_load16(tmem + half * kTokens + n + ((uint32_t)(warp & 3) * 32 << 16), v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (n + i < it.rows) {
                        const int owner = (n + i) / own;
                        const uint32_t to = in_cta(smem_addr(parts + ((split * own + n + i - owner * own) * 2 + half) * kRows + row), owner);
                        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to), "r"(v[i]) : "memory");
                    }
            }
            tcgen05_before();
        }
        __syncwarp();
        cluster_barrier();
        if (writes && good) {
            Writer w(p, it, it.b + half, row);
            const int to = min(it.rows, (split + 1) * own);
            w.rows = to;                         // the rows after them are another's
            for (int n = split * own; n < to; n += 2) {
                float sum[2] = {0.f, 0.f};
                for (int q = 0; q < splits; ++q)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (n + i < to) sum[i] += parts[((q * own + n + i - split * own) * 2 + half) * kRows + row];
                w.put(n, sum[0], sum[1], [&](int r) { return r < to ? w.row_scale[r] : 0.f; });
            }
        }
    }
    __syncthreads();
    if (warp == kIssuer) {
        tcgen05_after();
        tmem_free(tmem, kColumns);
    }
}

// Tiles of up to `tile` rows that max_rows rows of E experts make at most.
int64_t most_tiles(int E, int64_t max_rows, int tile) {
    const int64_t used = std::min<int64_t>(E, max_rows);
    return used + (max_rows - used) / tile;
}

}  // namespace

size_t i8_bytes(const I8Shape& w) { return (size_t)scales_at(w) + (size_t)w.E * row_blocks(w) * kRows * sizeof(float); }

bool i8_packs(const I8Shape& w) { return (int64_t)w.E * row_blocks(w) * k_steps(w) <= INT32_MAX; }

bool i8_fits(const I8Shape& w, int64_t max_rows) { return most_tiles(w.E, max_rows, 16) * row_blocks(w) <= INT32_MAX / 8; }

cudaError_t launch_i8_pack(const I8Shape& w, const int8_t* codes, const float* scales, void* packed, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)w.E * row_blocks(w) * k_steps(w)));
    return launch_kernel(false, i8_pack_kernel, grid, dim3(256), 0, stream, w, codes, scales, static_cast<unsigned char*>(packed));
}

cudaError_t launch_expert_i8(const I8Params& p, int num_sms, cudaStream_t stream) {
    const int pairs = (row_blocks(p.w) + 1) / 2;
    // Tiles of twice the mean: the smaller the tile, the longer the ring.
    int tile = kTokens, splits = 1;
    while (tile > 32 && p.max_rows * 4 <= (int64_t)p.w.E * tile) tile /= 2;
    while (tile > 32 && most_tiles(p.w.E, p.max_rows, tile) * pairs * 2 <= num_sms) tile /= 2;
    const int64_t most = most_tiles(p.w.E, p.max_rows, tile) * pairs;
    while (splits < 8 && most * splits * 2 <= num_sms && k_steps(p.w) >= splits * 4) splits *= 2;
    const cudaError_t e = cudaFuncSetAttribute(expert_i8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    const unsigned clusters = (unsigned)std::min<int64_t>(most, num_sms / splits);
    return launch_clusters(true, splits, expert_i8_kernel, dim3(clusters * splits), dim3(kThreads), kSmemBytes, stream, p, splits, tile);
}

}  // namespace ep
