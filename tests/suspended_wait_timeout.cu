// The bounded wait of the 8-bit products' warps (mbar_wait_suspended in
// ep_device.cuh), made to run out on the GPU without a fault: the warps of a CTA
// wait for a phase that nothing completes, give up, flag it and return, as the
// products' roles do.  Then a phase is completed by a bulk copy and by an arrival
// (both must be seen, no flag), and a plain kernel runs on the same context.
// Prints one line; exit code 0 once all ran.
#include <cstdint>
#include <cstdio>

#include "ep_device.cuh"

using namespace ep;

constexpr int kWarps = 4;

__global__ void never(uint32_t* flags, unsigned long long* waited_ns) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);          // nothing arrives
        fence_mbar_init();
    }
    __syncthreads();
    const uint64_t t0 = global_timer_ns();
    const bool good = __all_sync(0xffffffffu, mbar_wait_suspended(&bar, 0));
    if ((threadIdx.x & 31) == 0) {
        waited_ns[threadIdx.x >> 5] = global_timer_ns() - t0;
        if (!good) atomicOr(flags, kErrTimeout);
    }
    __syncthreads();
}

__global__ void completed(const uint4* src, uint32_t* flags, uint4* out) {
    __shared__ __align__(128) uint4 buf[8];
    __shared__ uint64_t copied, arrived;
    if (threadIdx.x == 0) {
        mbar_init(&copied, 1);
        mbar_init(&arrived, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&copied, sizeof(buf));
        bulk_load(buf, src, sizeof(buf), &copied);
    }
    __syncthreads();
    bool good = mbar_wait_suspended(&copied, 0);
    if (threadIdx.x == 0) mbar_arrive(&arrived);
    good = mbar_wait_suspended(&arrived, 0) && good;
    if (!good) atomicOr(flags, kErrTimeout);
    if (good && threadIdx.x == 0) out[0] = buf[7];
}

__global__ void plain(int* v) { v[threadIdx.x] = (int)threadIdx.x * 3; }

int main() {
    uint32_t* flags = nullptr;
    unsigned long long* waited = nullptr;
    uint4 *src = nullptr, *out = nullptr;
    int* v = nullptr;
    if (cudaMalloc(&flags, 8) || cudaMalloc(&waited, kWarps * 8) || cudaMalloc(&src, 8 * sizeof(uint4)) || cudaMalloc(&out, sizeof(uint4)) ||
        cudaMalloc(&v, 32 * sizeof(int)))
        return 2;
    uint4 h_src[8];
    for (int i = 0; i < 8; ++i) h_src[i] = make_uint4(i, i + 1, i + 2, i + 3);
    cudaMemcpy(src, h_src, sizeof(h_src), cudaMemcpyHostToDevice);

    cudaMemset(flags, 0, 8);
    never<<<1, kWarps * 32>>>(flags, waited);
    const cudaError_t e1 = cudaDeviceSynchronize();
    uint32_t f1 = 0;
    unsigned long long ns[kWarps] = {}, least = ~0ull, most = 0;
    cudaMemcpy(&f1, flags, 4, cudaMemcpyDeviceToHost);
    cudaMemcpy(ns, waited, sizeof(ns), cudaMemcpyDeviceToHost);
    for (unsigned long long n : ns) {
        least = n < least ? n : least;
        most = n > most ? n : most;
    }

    cudaMemset(flags, 0, 8);
    completed<<<1, kWarps * 32>>>(src, flags, out);
    const cudaError_t e2 = cudaDeviceSynchronize();
    uint32_t f2 = 0;
    uint4 got{};
    cudaMemcpy(&f2, flags, 4, cudaMemcpyDeviceToHost);
    cudaMemcpy(&got, out, sizeof(got), cudaMemcpyDeviceToHost);

    plain<<<1, 32>>>(v);
    const cudaError_t e3 = cudaDeviceSynchronize();
    int hv[32] = {};
    cudaMemcpy(hv, v, sizeof(hv), cudaMemcpyDeviceToHost);

    printf("timeout_flag=%u timeout_bit=%u least_ms=%.1f most_ms=%.1f err1=%s completed_flag=%u completed_ok=%d err2=%s plain_ok=%d err3=%s\n", f1,
           (unsigned)kErrTimeout, least / 1e6, most / 1e6, cudaGetErrorName(e1), f2, got.x == 7 && got.w == 10, cudaGetErrorName(e2), hv[31] == 93,
           cudaGetErrorName(e3));
    return 0;
}
