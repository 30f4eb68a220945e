// The wait for a row of the block norm's ring (wait_row in block_norm.cu), made
// to run out on the GPU without a fault: three warps wait for barriers armed for
// bytes that no copy delivers, the second from half a second after the first,
// the third after the first has ended.  The first runs its limit and marks the
// loss, the others end with it.  A fourth barrier completes and is not marked.
// Prints one line; exit code 0 once it ran.
#include <cstdio>

#include "block_norm.cu"

__global__ void waits(unsigned long long* ns, int* marks) {
    __shared__ uint64_t bars[4];
    __shared__ int lost, lost_not;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) ep::mbar_init(&bars[i], 1);
        ep::fence_mbar_init();
        for (int i = 0; i < 3; ++i) ep::mbar_arrive_expect_tx(&bars[i], 16);       // no copy will bring these bytes
        ep::mbar_arrive(&bars[3]);
        lost = lost_not = 0;
    }
    __syncthreads();
    const uint64_t t0 = ep::global_timer_ns();
    if (warp == 1)
        while (ep::global_timer_ns() - t0 < 500000000ull) {}
    if (warp == 2)
        while (ep::global_timer_ns() - t0 < 1200000000ull) {}
    const uint64_t t1 = ep::global_timer_ns();
    if (warp < 3)
        ep::wait_row(&bars[warp], 0, &lost);
    else
        ep::wait_row(&bars[3], 0, &lost_not);
    if ((threadIdx.x & 31) == 0) ns[warp] = ep::global_timer_ns() - t1;
    __syncthreads();
    if (threadIdx.x == 0) {
        marks[0] = lost;
        marks[1] = lost_not;
    }
}

int main() {
    unsigned long long* ns = nullptr;
    int* marks = nullptr;
    if (cudaMalloc(&ns, 4 * 8) || cudaMalloc(&marks, 8)) return 2;
    waits<<<1, 128>>>(ns, marks);
    const cudaError_t e = cudaDeviceSynchronize();
    unsigned long long h[4] = {};
    int m[2] = {};
    cudaMemcpy(h, ns, sizeof(h), cudaMemcpyDeviceToHost);
    cudaMemcpy(m, marks, sizeof(m), cudaMemcpyDeviceToHost);
    std::printf("err=%s lost=%d lost_not=%d first_ms=%.1f second_ms=%.1f third_ms=%.1f there_ms=%.1f\n", cudaGetErrorName(e), m[0], m[1],
                h[0] / 1e6, h[1] / 1e6, h[2] / 1e6, h[3] / 1e6);
    return 0;
}
