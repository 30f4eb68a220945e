// The launch of the block norm's backward pass for every width and type: as many
// CTAs as it plans for an SM (per_sm) are held by one, registers and shared
// memory counted, and the ring has the stages that its lag needs.  Launches
// nothing.  Prints one line; exit code 0 when every width passes.
#include <cstdio>

#include "block_norm.cu"

int main() {
    int dev = 0, num_sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 2;
    int bad = 0, shapes = 0;
    for (int f32 = 0; f32 < 2; ++f32)
        for (int H = 8; H <= 16384; H += 8) {
            const ep::BackwardShape s = ep::backward_shape(1 << 20, H, f32, num_sms);
            for (int full = 0; full < 2; ++full) {
                const ep::BackwardKernel kern = ep::backward_kernel(s, f32, full != 0);
                if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ep::kRingBytes) != cudaSuccess) return 2;
                int held = 0;
                if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&held, kern, s.warps * 32 + 64, ep::ring_bytes(s, f32)) != cudaSuccess) return 2;
                ++shapes;
                if (held < s.per_sm || s.lag < 1 || s.stages < s.lag + 2 || s.clusters * s.cluster > num_sms * s.per_sm) {
                    if (bad++ < 20)
                        std::printf("H=%d f32=%d full=%d: %d CTAs an SM planned, %d held, %d stages, lag %d\n", H, f32, full, s.per_sm, held,
                                    s.stages, s.lag);
                }
            }
        }
    std::printf("%d of %d shapes hold fewer CTAs than planned\n", bad, shapes);
    return bad != 0;
}
