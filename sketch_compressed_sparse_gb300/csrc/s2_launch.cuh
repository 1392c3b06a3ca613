// Launches whose start-up overlaps the end of the kernel before them in the stream.
//
// Back to back, such a kernel starts about 2 us earlier where the one before it was of
// this kind too: 8192 x 4096 bfloat16 packed in 17.6 us instead of 19.3 and unpacked in
// 17.0 instead of 18.5, a 33278 x 512 weight packed in 19.7 instead of 22.4,
// 24 x 267735 x 1024 multiplied in 50.0 instead of 52.8; in a CUDA graph one
// token's packing and product by 4096 x 4096 6.3 us instead of 7.0.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace s2 {

// Called by every thread before its first access to global memory: returns when
// the kernels before this one in the stream have ended and their writes are
// visible. (Every thread: this kernel must not end before they do.) From then on
// the next launch of this kind may put its blocks where there is room; they wait
// at the same place. Letting them start before this wait gained nothing more.
// Loads after it are plain ones: a load declared read-only might be moved up.
__device__ __forceinline__ void stream_order() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// kernel<<<grid, threads, smem, s>>>(args...) in clusters of `cluster` blocks
// (0: as the kernel is declared), started early; the kernel calls stream_order().
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), uint32_t grid, uint32_t threads, size_t smem, uint32_t cluster,
                         cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace s2
