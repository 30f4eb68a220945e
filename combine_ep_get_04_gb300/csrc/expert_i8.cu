// expert_i8.cu -- the experts' products over the receive buffer in 8-bit integers:
//   y[r, n] = x_scale[r] * w_scale[e, n] * sum_k x[r, k] * w[e, n, k]
//
// This part multiplies 8-bit integers at 151 TOP/s (mma.sync, measured), f16 at
// thirteen times that, so the codes go through the tensor cores as f16, which
// holds them exactly: a product of two has 15 bits and sums stay exact below 2^24.
// Two blocks of 128 weight rows are the M side of tcgen05.mma, up to 160 token rows
// the N side of both, 128 input channels a step.  One CTA an SM takes item after
// item (two blocks with one tile of token rows).  A warp finds the items; a
// producer warp keeps a ring of weight codes filled by bulk copies; eight warps
// widen them into tensor memory, a row to a thread, which is the instruction's A
// operand; eight more load token codes, several steps ahead, and widen them into
// shared memory (B), and write the sums out; one thread issues the products.
//
// That chain of roles costs some 7 us before the first sum is out, so a batch of little
// work goes another way (expert_i8_few_kernel).
#include <algorithm>

#include "ep.h"

#include "block_kernels.h"
#include "expert_rows.cuh"
#include "i8_tiles.h"
#include "per_device.h"

namespace ep {
namespace {

constexpr int kRows = 128;         // weight rows of a block
constexpr int kTokens = 160;       // most token rows of a tile
constexpr int kStep = 128;         // input channels of a step
constexpr int kStepBytes = kRows * kStep;
constexpr int kMaxRing = 12;       // units of weight codes: a step of one block each
constexpr int kMaxA = 6;           // units that are widened ahead
constexpr int kB = 3;              // steps whose tokens are
constexpr int kItems = 4;          // items found ahead
constexpr int kWeightWarps = 8, kTokenWarps = 8;
constexpr int kProducer = kWeightWarps + kTokenWarps, kIssuer = kProducer + 1, kFinder = kProducer + 2;
constexpr int kThreads = (kFinder + 1) * 32;
constexpr int kItemReaders = kFinder;
constexpr uint32_t kColumns = 512;                // tensor memory: the two blocks' sums, a tile's columns each, then A operands
constexpr int kAColumns = kStep / 2;

__host__ __device__ constexpr int a_places(int tile_rows) {
    const int fit = ((int)kColumns - 2 * tile_rows) / kAColumns;
    return fit < kMaxA ? fit : kMaxA;
}
static_assert(a_places(kTokens) >= 3, "the widest tile leaves too little for the A operands");

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
constexpr int kControlBytes = 13 * 1024;         // barriers, items and the table of experts
constexpr int kSmemBytes = 212 * 1024;           // the rest

__host__ __device__ constexpr int run_bytes(int tile_rows) { return (tile_rows + 1) * 16; }
__host__ __device__ constexpr int ring_units(int tile_rows) {
    const int fit = (kSmemBytes - kB * kRuns * run_bytes(tile_rows)) / kStepBytes;
    return fit < kMaxRing ? fit : kMaxRing;
}
// A group that waits for unit u to arrive has seen unit u - 2 - a_places multiplied, so the place's last unit has arrived.
constexpr bool ring_is_ahead(int tile_rows) { return ring_units(tile_rows) >= a_places(tile_rows) + 2; }
static_assert(ring_is_ahead(kTokens) && ring_is_ahead(128) && ring_is_ahead(64) && ring_is_ahead(32), "a place of the ring could be waited for a round early");

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

// The sums of a weight row to a lane, scaled, paired and stored.
struct Writer {
    uint16_t* y;             // at the lane's channel of the tile's first row (the upper lanes' of a pair: of the second)
    float scale;
    int64_t N;
    int rows;
    bool paired, stores;

    __device__ __forceinline__ Writer(const I8Params& p, const Item& it, int b, int row) {
        bool up;
        const int c = channel_of(p.w, b, row, &up);
        scale = reinterpret_cast<const float*>(static_cast<const unsigned char*>(p.packed) + scales_at(p.w))[((int64_t)it.e * row_blocks(p.w) + b) * kRows + row];
        N = p.w.N;
        paired = p.w.paired;
        y = static_cast<uint16_t*>(p.y) + (int64_t)it.first * N + c + (paired && (threadIdx.x & 16) ? N : 0);
        rows = it.rows;
        stores = c < N;
    }

    // Token rows n and n + 1 to `to` (y of row n).  xs(r): the scale of row r (r = n or n + 1 in a lane).  Of a pair, the
    // lower lanes have the gates and finish row n, the upper ones have the ups and finish row n + 1.
    template <typename Scale>
    __device__ __forceinline__ void put(int n, uint16_t* to, float s0, float s1, Scale xs) const {
        const bool upper = threadIdx.x & 16;
        const float a = s0 * scale, b = s1 * scale;
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

// What the warps share beside the rings, at the start of shared memory.
struct Control {
    uint64_t ring_full[kMaxRing], ring_empty[kMaxRing], a_full[kMaxA], a_done[kMaxA], b_full[kB], b_done[kB];
    uint64_t item_full[kItems], item_empty[kItems], done, drained;
    Item items[kItems];
    uint32_t tmem;
    int first[EP_MAX_EXPERTS], rows[EP_MAX_EXPERTS], upto[EP_MAX_EXPERTS];       // of each expert; tiles up to and with it
};

static_assert(kMostTiles >= (1 << 26) + EP_MAX_EXPERTS, "a good layout of tiles of 32 rows would be cut off");
static_assert(sizeof(Control) <= kControlBytes, "the shared state has outgrown its room");

extern __shared__ __align__(128) unsigned char smem[];

__device__ __forceinline__ Control& control() { return *reinterpret_cast<Control*>(smem); }
__device__ __forceinline__ unsigned char* ring_base() { return smem + kControlBytes; }

__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_suspended(bar, parity)); }

// Item j of the CTA, for a whole warp.  False if a wait ran out.
__device__ __forceinline__ bool next_item(int j, Item* it) {
    Control& c = control();
    const int slot = j % kItems;
    if (!await(&c.item_full[slot], (j / kItems) & 1)) return false;
    *it = c.items[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&c.item_empty[slot]);
    return true;
}

// The roles.  Each is a function of its own, so that what one keeps in registers
// costs the others none: with all of shared memory in use there is next to no L1,
// and a value that is spilled comes back from L2.  A role returns false if a wait
// ran out.

// Finds the items: item j of cluster c is number c + j * clusters in the order of
// experts, tiles and blocks.
__device__ __noinline__ bool find_items(int E, int nb, int width, int tile_rows, int cluster, int clusters, bool one, uint32_t* err_flags) {
    Control& c = control();
    const int lane = threadIdx.x & 31;
    // lane l adds up the tiles of experts [l * per, (l + 1) * per)
    const int per = (E + 31) / 32, e0 = min(lane * per, E), e1 = min(e0 + per, E);
    int mine = 0;
    for (int e = e0; e < e1; ++e) {
        mine = add_tiles(mine, tiles_needed(c.rows[e], tile_rows));
        c.upto[e] = mine;
    }
    int total = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, total, d);
        if (lane >= d) total = add_tiles(total, v);
    }
    int before = __shfl_up_sync(0xffffffffu, total, 1);
    if (lane == 0) before = 0;
    total = __shfl_sync(0xffffffffu, total, 31);
    for (int e = e0; e < e1; ++e) c.upto[e] = add_tiles(c.upto[e], before);
    __syncwarp();
    const int across = (nb + width - 1) / width;       // items of a tile
    const int64_t all = (int64_t)total * across, most = one ? min(all, (int64_t)clusters) : all;
    if ((most < all || total == kMostTiles) && cluster == 0 && lane == 0 && err_flags != nullptr) atomicOr(err_flags, kErrCapacity);
    for (int j = 0;; ++j) {
        const int slot = j % kItems;
        const int64_t at = cluster + (int64_t)j * clusters;
        if (j >= kItems && !await(&c.item_empty[slot], (j / kItems - 1) & 1)) return false;
        Item it{-1, 0, 0, 0, 0};
        if (at < most) {
            const int tile = (int)(at / across);
            int lo = 0, hi = E - 1;                    // the first expert with upto > tile
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (c.upto[mid] > tile)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            const int n = c.rows[lo], size = tile_rows_of(n, tile_rows), from = (tile - (lo > 0 ? c.upto[lo - 1] : 0)) * size;
            const int b = (int)(at - (int64_t)tile * across) * width;
            it = Item{lo, min(size, n - from), c.first[lo] + from, b, width > 1 && b + 1 < nb};
        }
        if (lane == 0) {
            c.items[slot] = it;
            mbar_arrive(&c.item_full[slot]);
        }
        __syncwarp();
        if (it.e < 0) return true;
    }
}

// Keeps the ring of codes filled, in the order of the products: a step's first block, its second, the next step.
__device__ __noinline__ bool produce(const unsigned char* packed, int nb, int nk, int k0, int steps, int ring) {
    Control& c = control();
    const int lane = threadIdx.x & 31;
    int64_t filled = 0;
    bool good = true;
    Item it;
    Place r{0, 1};                           // the parity of the place's previous use
    for (int j = 0; good; ++j) {
        good = next_item(j, &it);
        if (!good || it.e < 0) break;
        const unsigned char* weights = packed + (((int64_t)it.e * nb + it.b) * nk + k0) * kStepBytes;
        const int blocks = it.two ? 2 : 1;
        for (int i = 0; i < steps && good; ++i, weights += kStepBytes) {
            for (int h = 0; h < blocks; ++h, ++filled, r.next(ring)) {
                if (filled >= ring) good = await(&c.ring_empty[r.at], r.parity);
                if (!good) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&c.ring_full[r.at], kStepBytes);
                    bulk_load(ring_base() + r.at * kStepBytes, weights + (int64_t)(h * nk) * kStepBytes, kStepBytes, &c.ring_full[r.at]);
                }
                __syncwarp();
            }
        }
    }
    // no copy may be in flight when the CTA ends, whatever its consumers did
    for (int64_t i = max((int64_t)0, filled - ring); i < filled; ++i) mbar_wait_suspended(&c.ring_full[i % ring], (i / ring) & 1);
    return good;
}

// Issues the products.  One thread: their operands then stay in uniform registers.
__device__ __noinline__ bool issue(uint32_t tmem, int steps, int tile_rows, int ring) {
    Control& c = control();
    const int places = a_places(tile_rows);
    const uint32_t a_at = tmem + 2 * tile_rows, run16 = run_bytes(tile_rows) / 16;
    // runs of 8 channels run16 * 16 bytes apart, 8 rows 128 bytes apart, no swizzle
    const uint64_t desc = (uint64_t)run16 << 16 | (uint64_t)(128 / 16) << 32 | (uint64_t)1 << 46;
    const unsigned char* ops = ring_base() + ring * kStepBytes;
    const uint64_t first_b = desc | (smem_addr(ops) >> 4 & 0x3fff);          // in a cluster, addresses have a rank above
    int committed = 0;
    bool good = true;
    Place a, b;
    for (int j = 0; good; ++j) {
        const int slot = j % kItems;
        good = mbar_wait_suspended(&c.item_full[slot], (j / kItems) & 1);
        if (!good) break;
        const int e = c.items[slot].e, rows = c.items[slot].rows, two = c.items[slot].two;
        mbar_arrive(&c.item_empty[slot]);
        if (e < 0) break;
        const uint32_t cols = (rows + 15) & ~15;           // the products' N: a multiple of 16
        const uint32_t kind = 1u << 4 | (cols / 8) << 17 | (uint32_t)(kRows / 16) << 24;      // fp32 sums, f16 operands, N, M
        if (j > 0) good = mbar_wait_suspended(&c.drained, (j - 1) & 1);
        for (int i = 0; i < steps && good; ++i, b.next(kB)) {
            const uint64_t from_b = first_b + (uint32_t)(b.at * kRuns) * run16;
            good = mbar_wait_suspended(&c.b_full[b.at], b.parity);
            for (int h = 0; h <= two && good; ++h, a.next(places)) {
                const uint32_t from_a = a_at + a.at * kAColumns, to = tmem + h * tile_rows;
                good = mbar_wait_suspended(&c.a_full[a.at], a.parity);
                if (!good) break;
                tcgen05_after();
#pragma unroll
                for (int k = 0; k < kStep / 16; ++k) mma_f16(to, from_a + k * 8, from_b + k * 2 * run16, kind, i > 0 || k > 0);
                tcgen05_commit(&c.a_done[a.at]);
            }
            if (good) tcgen05_commit(&c.b_done[b.at]);
        }
        tcgen05_commit(&c.done);
        ++committed;
    }
    // every product is over before tensor memory is given back
    if (committed > 0) good = mbar_wait_suspended(&c.done, (committed - 1) & 1) && good;
    return good;
}

// An item's sums, out of tensor memory: a row of a block to a lane.
__device__ __noinline__ bool write_sums(const I8Params& p, int j, uint32_t tmem, int tile_rows) {
    Control& c = control();
    const int lane = threadIdx.x & 31, half = (threadIdx.x >> 7) & 1, row = threadIdx.x & 127;
    const Item it = c.items[j % kItems];
    const bool here = half == 0 || it.two;
    const Writer w(p, it, it.b + (here ? half : 0), row);
    float xs[kTokens / 32];
#pragma unroll
    for (int k = 0; k < kTokens / 32; ++k) xs[k] = lane + 32 * k < it.rows ? p.x_scales[it.first + lane + 32 * k] : 0.f;
    if (!await(&c.done, j & 1)) return false;
    tcgen05_after();
    if (here) {
        uint16_t* y = w.y;
        // not unrolled further: addresses made ahead would not fit the registers
#pragma unroll 1
        for (int n = 0; n < it.rows; n += 16) {
            uint32_t v[16];
            tmem_load16(tmem + half * tile_rows + ((uint32_t)(row >> 5) * 32 << 16) + n, v);
            float mine = xs[0];
#pragma unroll
            for (int k = 1; k < kTokens / 32; ++k) mine = n >= 32 * k ? xs[k] : mine;
#pragma unroll
            for (int i = 0; i < 16; i += 2, y += 2 * w.N)
                w.put(n + i, y, __uint_as_float(v[i]), __uint_as_float(v[i + 1]), [&](int r) { return __shfl_sync(0xffffffffu, mine, r); });
        }
    }
    tcgen05_before();
    __syncwarp();
    if (lane == 0) {
        mbar_arrive(&c.drained);
        mbar_arrive(&c.item_empty[j % kItems]);
    }
    return true;
}

__device__ __forceinline__ void store_shared(uint32_t to, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Tokens: a thread has 16 channels of every 32nd row, of up to 32 CHUNKS, and loads
// them AHEAD steps ahead: with HBM busy an L2 hit takes some 1700 cycles, longer
// than a step (256 experts, 4 rows each, one step ahead 1378 us, two 1131).  Each
// tile has chunks of its own: with those of the next wider one, 64 rows an expert
// take 342 us instead of 334 and 32 rows 311 instead of 305 (64 experts, rows on average).
template <int CHUNKS, int AHEAD>
__device__ __noinline__ bool widen_tokens(const I8Params& p, uint32_t tmem, int k0, int steps, int tile_rows, int ring, bool writes) {
    static_assert(AHEAD <= kB, "steps that are made before an item's sums are written find rooms");
    Control& c = control();
    const int K = p.w.K, run = run_bytes(tile_rows);
    const int t = threadIdx.x - kWeightWarps * 32, n0 = t >> 3;
    const uint32_t ops = smem_addr(ring_base()) + ring * kStepBytes + (t & 7) * run + n0 * 16;
    const int8_t* const first_x = p.x + (int64_t)k0 * kStep + (t & 7) * 16 + (int64_t)n0 * K;
    const int left = K - k0 * kStep - (t & 7) * 16;            // channels from the thread's on
    bool full = false;                       // whether all rooms have been used
    Place b;                                 // this step's room
    uint4 raw[AHEAD][CHUNKS];
    for (int j = 0;; ++j) {
        const int slot = j % kItems;
        if (!await(&c.item_full[slot], (j / kItems) & 1)) return false;
        const int count = c.items[slot].e >= 0 ? steps : 0;    // the end comes as an item without steps
        const int rows = c.items[slot].rows - n0;              // from the thread's first on
        const int8_t* x = first_x + (int64_t)c.items[slot].first * K;
        __syncwarp();
        if (!writes && (threadIdx.x & 31) == 0) mbar_arrive(&c.item_empty[slot]);
        auto fetch = [&](uint4 (&r)[CHUNKS], int step) {
            const bool in = step < count && step * kStep < left;
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                r[i] = make_uint4(0, 0, 0, 0);                 // channels past the end
                if (32 * i < rows && in) r[i] = *reinterpret_cast<const uint4*>(x + (uint32_t)(32 * i) * (uint32_t)K + (uint32_t)(step * kStep));
            }
        };
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) fetch(raw[u], u);
        for (int base = 0;; base += AHEAD) {
            if (CHUNKS == 1 && writes && j > 0 && base == min(AHEAD, (count + AHEAD - 1) / AHEAD * AHEAD))
                if (!write_sums(p, j - 1, tmem, tile_rows)) return false;
            if (base >= count) break;
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int i = base + u;
                if (i >= count) break;
                if (full && !await(&c.b_done[b.at], b.parity ^ 1)) return false;
                const uint32_t to = ops + b.at * kRuns * run;
#pragma unroll
                for (int m = 0; m < CHUNKS; ++m) {
                    if (32 * m < rows) {
                        uint4 lo, hi;
                        widen(raw[u][m].x ^ 0x80808080u, &lo.x, &lo.y);
                        widen(raw[u][m].y ^ 0x80808080u, &lo.z, &lo.w);
                        widen(raw[u][m].z ^ 0x80808080u, &hi.x, &hi.y);
                        widen(raw[u][m].w ^ 0x80808080u, &hi.z, &hi.w);
                        store_shared(to + 32 * m * 16, lo.x, lo.y, lo.z, lo.w);
                        store_shared(to + 8 * run + 32 * m * 16, hi.x, hi.y, hi.z, hi.w);
                    }
                }
                fetch(raw[u], i + AHEAD);
                fence_proxy_async_smem();
                __syncwarp();
                if ((threadIdx.x & 31) == 0) mbar_arrive(&c.b_full[b.at]);
                b.next(kB);
                full = full || b.at == 0;
            }
        }
        if (count == 0) return true;
    }
}

// Weights: two groups of warps take the units in turn, a row to a thread: what a
// unit costs a group is mostly waiting, for barriers, shared memory and tensor
// memory in turn.
//
// Who writes the sums out (`writes`; where K is shared, join_shares does) gives an
// item's place back when that is done: these warps for wide tiles, where the tokens'
// have the most to do and no registers left, else the tokens' (256 experts, 4 rows
// each, 2048 -> 7168: 532 us so, 568 by these).
__device__ __noinline__ bool widen_weights(const I8Params& p, uint32_t tmem, int steps, int tile_rows, int ring, bool writes) {
    Control& c = control();
    const int places = a_places(tile_rows);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp >> 2;
    const uint32_t to = tmem + 2 * tile_rows + ((uint32_t)(warp & 3) * 32 << 16);
    const unsigned char* from = ring_base() + (threadIdx.x & 127) * 16;
    int next = group;                        // the group's next unit, from the item's first on
    bool full = false;                       // whether all of its A operands' places have been used
    Place a, r;                              // the unit's A operand, its place in the ring
    if (group == 1) {
        a.next(places);
        r.next(ring);
    }
    for (int j = 0;; ++j) {
        const int slot = j % kItems;
        if (!await(&c.item_full[slot], (j / kItems) & 1)) return false;
        const int count = c.items[slot].e >= 0 ? steps * (c.items[slot].two ? 2 : 1) : 0;        // the end comes as an item without units
        __syncwarp();
        if (!writes && lane == 0) mbar_arrive(&c.item_empty[slot]);
        bool waiting = writes && j > 0;      // the sums of the item before
        for (;; next += 2) {
            // an item's first units are made while the products of the one before end; then the sums of that are written out
            if (waiting && (next >= places || next >= count)) {
                if (!write_sums(p, j - 1, tmem, tile_rows)) return false;
                waiting = false;
            }
            if (next >= count) break;
            if (!await(&c.ring_full[r.at], r.parity)) return false;
            uint32_t v[2][32];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint4 raw = *reinterpret_cast<const uint4*>(from + r.at * kStepBytes + q * kRows * 16);
                uint32_t* w = &v[q >> 2][(q & 3) * 8];
                widen(raw.x, w, w + 1);
                widen(raw.y, w + 2, w + 3);
                widen(raw.z, w + 4, w + 5);
                widen(raw.w, w + 6, w + 7);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.ring_empty[r.at]);
            if (full && !await(&c.a_done[a.at], a.parity ^ 1)) return false;
            tcgen05_after();
            tmem_store32(to + a.at * kAColumns, v[0]);
            tmem_store32(to + a.at * kAColumns + 32, v[1]);
            tmem_store_wait();
            tcgen05_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.a_full[a.at]);
            // two units on
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                r.next(ring);
                a.next(places);
                full = full || a.at == 0;
            }
        }
        if (count == 0) return true;
        next -= count;
    }
}

// The sums of an item whose K a cluster shares: each CTA owns some of the tile's
// token rows, whose sums the others push to it.  All threads of the cluster; it.e
// is -1 where there is none.
__device__ __noinline__ void join_shares(const I8Params& params, const Item it, uint32_t tmem, int tile_rows, int split, int splits, bool good) {
    cluster_barrier();                       // the rings are free
    const I8Params p = params;
    float* parts = reinterpret_cast<float*>(ring_base());          // [share][own][block][weight row]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
    const bool writes = good && warp >= kWeightWarps && warp < kProducer && it.e >= 0 && (half == 0 || it.two);
    const int own = (it.rows + splits - 1) / splits;
    if (writes) {
        tcgen05_after();
        for (int n = 0; n < it.rows; n += 16) {
            uint32_t v[16];
            tmem_load16(tmem + half * tile_rows + n + ((uint32_t)(warp & 3) * 32 << 16), v);
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
    if (writes) {
        Writer w(p, it, it.b + half, row);
        w.rows = min(it.rows, (split + 1) * own);              // the rows after them are another's
        for (int n = split * own; n < w.rows; n += 2) {
            float sum[2] = {0.f, 0.f};
            for (int q = 0; q < splits; ++q)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (n + i < w.rows) sum[i] += parts[((q * own + n + i - split * own) * 2 + half) * kRows + row];
            w.put(n, w.y + (int64_t)n * w.N, sum[0], sum[1], [&](int r) { return r < w.rows ? p.x_scales[it.first + r] : 0.f; });
        }
    }
}

// A grid of clusters of `splits` CTAs takes the items, of `width` blocks, a grid
// apart; with more than one share of K (which a launch of few products has) a
// cluster takes one.
//
// Up to some 32 rows an expert the weights' bytes decide: 256 experts with 4 rows
// each, gate and up (7168 -> 2 x 2048) 1026 us, down (2048 -> 7168) 532 us, 7.2 and
// 7.0 TB/s of weights.  With 128 rows each gate and up take 1640 us, 1173 TFLOP/s, down
// 976 us, 985 TFLOP/s; with 128 on average, as routers deal them, 1832 and 1057 us; and
// one matrix with 19456 rows 802 us, 1424 TFLOP/s: every step passes codes and operands
// through shared memory two or three times (of tiles of 160 rows 256 cycles for the
// weights' copies, 256 for their loads, 320 for the tokens' stores, 640 for the
// products' reads and as many as 160 for the tokens' way in), and the rest is waiting
// of the roles for one another; without the tokens' loads 1832 and 802 would be 1635 and
// 740 us, without the weights' 1734 and 753.
//
// Tiles of up to 160 rows leave tensor memory for three A operands of one block.  An
// expert with more rows needs a second tile, which reads and widens all its weights
// again: of 256 with 128 rows on average 46 to 54, of tiles of 128 rows many more
// (operands of both blocks 1990 us on the same part, of one block 1952).  Measured and
// not kept, at 128 rows on average and by tiles of 128:
// steps of 64 channels 2797 us; token codes by tensor copies of 8 rows 2532, of 32
// rows 2082 (one more pass through shared memory); sixteen warps for the weights
// 2095; one lane of a warp waiting for the others 3093; of 160: tokens fetched into L2
// three steps earlier 1970.
__global__ void __launch_bounds__(kThreads, 1) expert_i8_kernel(const __grid_constant__ I8Params p, int splits, int width, int tile_rows) {
    Control& c = control();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x % splits, cluster = blockIdx.x / splits, nb = row_blocks(p.w), nk = k_steps(p.w);
    const int ring = ring_units(tile_rows);
    const int k0 = (int)((int64_t)nk * split / splits), steps = (int)((int64_t)nk * (split + 1) / splits) - k0;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxRing; ++i) {
            mbar_init(&c.ring_full[i], 1);
            mbar_init(&c.ring_empty[i], kWeightWarps / 2);
        }
        for (int i = 0; i < kMaxA; ++i) {
            mbar_init(&c.a_full[i], kWeightWarps / 2);
            mbar_init(&c.a_done[i], 1);
        }
        for (int i = 0; i < kB; ++i) {
            mbar_init(&c.b_full[i], kTokenWarps);
            mbar_init(&c.b_done[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&c.item_full[i], 1);
            mbar_init(&c.item_empty[i], kItemReaders);
        }
        mbar_init(&c.done, 1);
        mbar_init(&c.drained, kWeightWarps);
        fence_mbar_init();
    }
    // a share may push to another once that runs
    if (splits > 1) {
        __syncwarp();
        cluster_barrier();
    }
    pdl_wait();
    // not before the wait: a CTA that holds tensor memory must not wait for one that may need it
    if (warp == kIssuer) tmem_alloc(&c.tmem, kColumns);
    for (int e = threadIdx.x; e < p.w.E; e += kThreads) {
        int64_t first;
        bool bad;
        c.rows[e] = expert_rows(p, e, &first, &bad);
        c.first[e] = (int)first;
        if (bad && blockIdx.x == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrBadSlot);
    }
    tcgen05_before();
    __syncthreads();
    tcgen05_after();
    bool good = true;
    if (warp == kFinder) {
        good = find_items(p.w.E, nb, width, tile_rows, cluster, gridDim.x / splits, splits > 1, p.err_flags);
    } else if (warp == kProducer) {
        good = produce(static_cast<const unsigned char*>(p.packed), nb, nk, k0, steps, ring);
    } else if (warp == kIssuer) {
        if (elect_one()) good = issue(c.tmem, steps, tile_rows, ring);
    } else if (warp >= kWeightWarps) {
        good = tile_rows <= 32    ? widen_tokens<1, 2>(p, c.tmem, k0, steps, tile_rows, ring, splits == 1)
               : tile_rows <= 64  ? widen_tokens<2, 3>(p, c.tmem, k0, steps, tile_rows, ring, false)
               : tile_rows <= 128 ? widen_tokens<4, 3>(p, c.tmem, k0, steps, tile_rows, ring, false)
                                  : widen_tokens<kTokens / 32, 3>(p, c.tmem, k0, steps, tile_rows, ring, false);
    } else {
        const bool writes = splits == 1 && tile_rows > 32;
        good = widen_weights(p, c.tmem, steps, tile_rows, ring, writes);
    }
    __syncwarp();
    good = __all_sync(0xffffffffu, good);
    if (!good && lane == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrTimeout);
    good = __syncthreads_and(good);
    // the one item's slot is not used again
    if (splits > 1) join_shares(p, c.items[0], c.tmem, tile_rows, split, splits, good);
    __syncthreads();
    if (warp == kIssuer) {
        tcgen05_after();
        tmem_free(c.tmem, kColumns);
    }
}

// ------------------------------------------------------------ little work
//
// No stages, no tensor memory, nothing to wait for but the weights.  A CTA has 16
// weight rows (of a pair 8 gate rows and their up rows) and up to 8 token rows; its
// warps take the steps of K in turn, straight from memory into the operands of
// mma.m16n8k32 in 8-bit integers, whose rate is enough for eight tokens.  The packed
// order suits it as it is: a thread's 16 bytes of a row are four products' operands,
// and the tokens' side of the four is 32 channels in a row.  Codes are stored plus
// 128; a token's sum of codes, times 128, comes off at the end.  Whole numbers of 32
// bits throughout, so the sums are exact and their order does not matter.
//
// Bound by the latency of memory, a warp's 2 KB a step: 16 warps with a step on its way
// while there are two CTAs an SM at most, else 8 warps with two (three would leave room
// for two CTAs instead of three: one row, 7168 -> 18432, 29.6 us against 25.5).  One
// row, 7168 -> 4096: 7.5 us, 3.9 TB/s (8 warps 9.7 us); 1024 -> 1024: 2.5 us.

constexpr int kFewRows = 8;               // token rows of a tile
constexpr int kMaxFewK = 65536;           // 255 * 128 * K fits 31 bits

__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool PAIRED, int kWarps, int kAhead>
__global__ void __launch_bounds__(kWarps * 32) expert_i8_few_kernel(I8Params p, int grid_tiles) {
    constexpr int kSecond = PAIRED ? 16 : 8;                           // from a thread's first weight row to its other
    __shared__ int sums[kWarps][16][kFewRows], token_sums[kWarps][kFewRows];
    __shared__ RowTile shared_tile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nb = row_blocks(p.w), nk = k_steps(p.w), b = blockIdx.x / 8, group = blockIdx.x % 8;
    const int row0 = PAIRED ? group / 2 * 32 + group % 2 * 8 : group * 16;
    pdl_launch_dependents();
    pdl_wait();
    RowTile tile;
    if (p.w.E == 1) {
        tile = tile_of_one(p, blockIdx.y, kFewRows, grid_tiles);
    } else {
        if (warp == 0) {
            const RowTile r = find_tile(p, blockIdx.y, kFewRows, grid_tiles);
            if (lane == 0) shared_tile = r;
        }
        __syncthreads();
        tile = shared_tile;
    }
    if (tile.e < 0) return;
    const unsigned char* packed = static_cast<const unsigned char*>(p.packed);
    const unsigned char* weights = packed + ((int64_t)tile.e * nb + b) * nk * kStepBytes + (t * kRows + row0 + g) * 16;
    const int8_t* x = p.x + (tile.first + g) * p.w.K + 32 * t;
    uint4 a[kAhead][4], q[kAhead][2];
    auto fetch = [&](int s, uint4 (&a)[4], uint4 (&q)[2]) {
        q[0] = q[1] = make_uint4(0, 0, 0, 0);
        if (s >= nk) return;
#pragma unroll
        for (int i = 0; i < 4; ++i)            // both rows, then the same four units of 16 bytes further
            a[i] = *reinterpret_cast<const uint4*>(weights + (int64_t)s * kStepBytes + ((i >> 1) * 4 * kRows + (i & 1) * kSecond) * 16);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (g < tile.rows && s * kStep + 32 * t + 16 * h < p.w.K) q[h] = *reinterpret_cast<const uint4*>(x + s * kStep + 16 * h);
    };
    int acc[4] = {}, token = 0;
    auto multiply = [&](const uint4 (&a)[4], const uint4 (&q)[2]) {
        const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) token = __dp4a((int)w[i], 0x01010101, token);
        mma_u8s8(acc, a[0].x, a[1].x, a[2].x, a[3].x, w[0], w[2]);
        mma_u8s8(acc, a[0].y, a[1].y, a[2].y, a[3].y, w[1], w[3]);
        mma_u8s8(acc, a[0].z, a[1].z, a[2].z, a[3].z, w[4], w[6]);
        mma_u8s8(acc, a[0].w, a[1].w, a[2].w, a[3].w, w[5], w[7]);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(warp + i * kWarps, a[i], q[i]);
    for (int s = warp; s < nk; s += kAhead * kWarps) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (s + i * kWarps >= nk) break;
            multiply(a[i], q[i]);
            fetch(s + (kAhead + i) * kWarps, a[i], q[i]);
        }
    }
    token += __shfl_xor_sync(0xffffffffu, token, 1);
    token += __shfl_xor_sync(0xffffffffu, token, 2);
    if (t == 0) token_sums[warp][g] = token;
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][g + (i >> 1) * 8][2 * t + (i & 1)] = acc[i];
    __syncthreads();
    // a channel to a thread
    constexpr int kChannels = PAIRED ? 8 : 16;
    const int row = threadIdx.x % kChannels, n = threadIdx.x / kChannels, c = b * (PAIRED ? kRows / 2 : kRows) + group * kChannels + row;
    if (n >= tile.rows || c >= p.w.N) return;
    int less = 0, first = 0, second = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        less += token_sums[w][n];
        first += sums[w][row][n];
        if (PAIRED) second += sums[w][row + 8][n];
    }
    const float* scales = reinterpret_cast<const float*>(packed + scales_at(p.w)) + ((int64_t)tile.e * nb + b) * kRows + row0 + row;
    const float xs = p.x_scales[tile.first + n];
    float f = (float)(first - 128 * less) * scales[0] * xs;
    if (PAIRED) f = silu(f) * ((float)(second - 128 * less) * scales[16] * xs);
    static_cast<uint16_t*>(p.y)[(tile.first + n) * p.w.N + c] = (uint16_t)pack_bf16x2(f, 0.f);
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

namespace {

// Clusters of 2, 4 or 8 CTAs that the current device runs at the same time.
int clusters_at_once(int splits) {
    static PerDevice<3> known;
    int device = -1;
    if (cudaGetDevice(&device) != cudaSuccess) device = -1;
    return known.get(device, splits == 2 ? 0 : splits == 4 ? 1 : 2, 1, [&](int* got) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(splits);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kControlBytes + kSmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)splits;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(got, expert_i8_kernel, &cfg) == cudaSuccess) return true;
        (void)cudaGetLastError();
        return false;
    });
}

}  // namespace

cudaError_t launch_expert_i8(const I8Params& p, int num_sms, cudaStream_t stream) {
    // Small CTAs where an SM gets 8 of them at most and, if they read weights more than once, 300 steps: one row of 7168 ->
    // 4096 in 7.5 us against the tiles' 13.3, 4 experts' pairs of 7168 -> 2048 (1024 CTAs) in 26.5 against 29.5, 32 rows of
    // 1024 -> 1024 in 2.8 against 10.7, of 7168 -> 1024 (118 steps) in 7.9 against 12.9; but 64 rows of 7168 -> 2048 (424
    // steps) in 21.3 against 16.6, 8 experts of 2048 -> 7168 (3584 CTAs) in 36.7 against 30.1.
    const int64_t few_tiles = most_tiles(p.w.E, p.max_rows, kFewRows), few_ctas = few_tiles * row_blocks(p.w) * 8;
    const bool once = few_tiles == std::min<int64_t>(p.w.E, p.max_rows);
    if (few_ctas <= 8 * num_sms && (once || few_ctas * k_steps(p.w) <= 300 * num_sms) && p.w.K <= kMaxFewK) {
        const bool wide = few_ctas <= 2 * num_sms;
        const auto kernel = p.w.paired ? (wide ? expert_i8_few_kernel<true, 16, 1> : expert_i8_few_kernel<true, 8, 2>)
                                       : (wide ? expert_i8_few_kernel<false, 16, 1> : expert_i8_few_kernel<false, 8, 2>);
        return launch_kernel(true, kernel, dim3((unsigned)(few_ctas / few_tiles), (unsigned)few_tiles), dim3(wide ? 512 : 256), 0, stream, p, (int)few_tiles);
    }
    const cudaError_t e = cudaFuncSetAttribute(expert_i8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kControlBytes + kSmemBytes);
    if (e != cudaSuccess) return e;
    // Tiles of twice the mean rows, as far as they go (64 rows an expert in tiles of 160 348 us, of 128 336): the smaller the
    // tile, the longer the ring.  Then as many items as there are SMs: by single blocks, by smaller tiles, by shares of K, of
    // which a cluster that did not run at once would double the time (one row, 7168 -> 4096, by this kernel: 16 clusters of
    // 8 23 us, of 4 16.5).
    const int nb = row_blocks(p.w);
    int tile = kTokens, width = 2, splits = 1;
    auto smaller = [](int tile) { return tile > 128 ? 128 : tile / 2; };
    while (tile > 32 && p.max_rows * (tile > 128 ? 2 : 4) <= (int64_t)p.w.E * tile) tile = smaller(tile);
    auto items = [&]() { return most_tiles(p.w.E, p.max_rows, tile) * ((nb + width - 1) / width); };
    if (items() * 2 <= num_sms) width = 1;
    while (tile > 32 && items() * 2 <= num_sms) tile = smaller(tile);
    while (splits < 8 && items() * splits * 2 <= num_sms && k_steps(p.w) >= splits * 4 && items() <= clusters_at_once(splits * 2)) splits *= 2;
    const unsigned clusters = (unsigned)std::min<int64_t>(items(), num_sms / splits);
    return launch_clusters(true, splits, expert_i8_kernel, dim3(clusters * splits), dim3(kThreads), kControlBytes + kSmemBytes, stream, p, splits, width,
                           tile);
}

}  // namespace ep
