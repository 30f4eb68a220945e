// expert_i8.cu -- the experts' products over the receive buffer in 8-bit integers:
//   y[r, n] = x_scale[r] * w_scale[e, n] * sum_k x[r, k] * w[e, n, k]
#include <algorithm>

#include "block_kernels.h"
#include "dropout.cuh"

namespace ep {
namespace {

constexpr int kRows = 128;         // weight rows of a block
constexpr int kChannels = 128;     // input channels of a tile
constexpr int kTileBytes = kRows * kChannels;

__host__ __device__ inline int k_tiles(const I8Shape& w) { return (w.K + kChannels - 1) / kChannels; }
// A paired block is 64 gate rows and the 64 up rows of the same channels.
__host__ __device__ inline int block_channels(const I8Shape& w) { return w.paired ? kRows / 2 : kRows; }
__host__ __device__ inline int row_blocks(const I8Shape& w) { return (w.N + block_channels(w) - 1) / block_channels(w); }
__host__ __device__ inline int64_t scales_at(const I8Shape& w) { return (int64_t)w.E * row_blocks(w) * k_tiles(w) * kTileBytes; }

// Output channel of row r of block b, and whether it is an up row: every warp's 32
// rows are 16 gate rows and their 16 up rows.
__host__ __device__ inline int channel_of(const I8Shape& w, int b, int r, bool* up) {
    *up = w.paired && (r & 16);
    return w.paired ? b * 64 + (r >> 5) * 16 + (r & 15) : b * kRows + r;
}

// Packed: tiles [E][row block][k tile][16 channels each][row][16 bytes], codes plus
// 128; then the scales [E][row block][row].
__global__ void __launch_bounds__(256) i8_pack_kernel(I8Shape w, const int8_t* codes, const float* scales, unsigned char* packed) {
    const int64_t tile = blockIdx.x;
    const int nk = k_tiles(w), nb = row_blocks(w), rows = w.paired ? 2 * w.N : w.N;
    const int kt = (int)(tile % nk), b = (int)(tile / nk % nb), e = (int)(tile / nk / nb);
    for (int i = threadIdx.x; i < kTileBytes / 16; i += blockDim.x) {
        const int r = i % kRows, k = kt * kChannels + i / kRows * 16;
        bool up;
        const int c = channel_of(w, b, r, &up);
        uint4 v = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
        if (c < w.N && k < w.K) {
            v = *reinterpret_cast<const uint4*>(codes + ((int64_t)e * rows + (up ? w.N : 0) + c) * w.K + k);
            v.x ^= 0x80808080u;
            v.y ^= 0x80808080u;
            v.z ^= 0x80808080u;
            v.w ^= 0x80808080u;
        }
        reinterpret_cast<uint4*>(packed + tile * kTileBytes)[i] = v;
    }
    if (kt == 0 && threadIdx.x < kRows) {
        bool up;
        const int c = channel_of(w, b, threadIdx.x, &up);
        reinterpret_cast<float*>(packed + scales_at(w))[((int64_t)e * nb + b) * kRows + threadIdx.x] =
            c < w.N ? scales[(int64_t)e * rows + (up ? w.N : 0) + c] : 0.f;
    }
}

__device__ __forceinline__ float silu(float x) {
    const float e = expf(-fabsf(x));
    return x * __fdividef(x < 0.f ? e : 1.f, 1.f + e);
}

// The simplest form: a thread has one weight row and up to 8 token rows.
__global__ void __launch_bounds__(kRows) expert_i8_kernel(I8Params p) {
    const int b = blockIdx.x, e = blockIdx.y, nk = k_tiles(p.w), nb = row_blocks(p.w);
    pdl_launch_dependents();
    pdl_wait();
    int64_t first = 0, rows = p.R;
    if (p.mode != 0) {
        first = (int64_t)e * p.capacity;
        rows = min(p.counts[e], p.capacity);
    } else if (p.offsets != nullptr) {
        first = p.offsets[e];
        rows = p.offsets[e + 1] - first;
    }
    if (rows > 0 && (first < 0 || first + rows > p.R)) {
        if (threadIdx.x == 0 && b == 0 && p.err_flags != nullptr) atomicOr(p.err_flags, kErrBadSlot);
        return;
    }
    const unsigned char* packed = static_cast<const unsigned char*>(p.packed);
    const uint4* wt = reinterpret_cast<const uint4*>(packed + ((int64_t)e * nb + b) * nk * kTileBytes) + threadIdx.x;
    const float ws = reinterpret_cast<const float*>(packed + scales_at(p.w))[((int64_t)e * nb + b) * kRows + threadIdx.x];
    bool up;
    const int c = channel_of(p.w, b, threadIdx.x, &up);
    for (int64_t r0 = 0; r0 < rows; r0 += 8) {
        const int n = (int)min((int64_t)8, rows - r0);
        const int8_t* x = p.x + (first + r0) * p.w.K;
        int acc[8] = {};
        for (int k = 0; k < p.w.K; k += 16) {
            uint4 v = wt[k / 16 * kRows];
            v.x ^= 0x80808080u;
            v.y ^= 0x80808080u;
            v.z ^= 0x80808080u;
            v.w ^= 0x80808080u;
            for (int j = 0; j < n; ++j) {
                const uint4 q = *reinterpret_cast<const uint4*>(x + (int64_t)j * p.w.K + k);
                acc[j] = __dp4a((int)v.x, (int)q.x, __dp4a((int)v.y, (int)q.y, __dp4a((int)v.z, (int)q.z, __dp4a((int)v.w, (int)q.w, acc[j]))));
            }
        }
        for (int j = 0; j < 8; ++j) {
            float f = j < n ? (float)acc[j] * ws * p.x_scales[first + r0 + j] : 0.f;
            if (p.w.paired) f = silu(f) * __shfl_xor_sync(0xffffffffu, f, 16);
            if (j < n && c < p.w.N && !up) static_cast<uint16_t*>(p.y)[(first + r0 + j) * p.w.N + c] = (uint16_t)pack_bf16x2(f, 0.f);
        }
    }
}

}  // namespace

size_t i8_bytes(const I8Shape& w) { return (size_t)scales_at(w) + (size_t)w.E * row_blocks(w) * kRows * sizeof(float); }

bool i8_packs(const I8Shape& w) { return (int64_t)w.E * row_blocks(w) * k_tiles(w) <= INT32_MAX; }

bool i8_fits(const I8Shape&, int64_t) { return true; }

cudaError_t launch_i8_pack(const I8Shape& w, const int8_t* codes, const float* scales, void* packed, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)w.E * row_blocks(w) * k_tiles(w)));
    return launch_kernel(false, i8_pack_kernel, grid, dim3(256), 0, stream, w, codes, scales, static_cast<unsigned char*>(packed));
}

cudaError_t launch_expert_i8(const I8Params& p, int, cudaStream_t stream) {
    return launch_kernel(false, expert_i8_kernel, dim3(row_blocks(p.w), p.w.E), dim3(kRows), 0, stream, p);
}

}  // namespace ep
