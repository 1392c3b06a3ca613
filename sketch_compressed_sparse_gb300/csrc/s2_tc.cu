// Host side of the tensor-core kernels: tensor maps, and the device word in
// which waits that ran out are counted.
#include "s2_internal.h"
#include "s2_tc.cuh"

#include <mutex>

namespace s2 {
namespace {

__device__ uint32_t g_wait_faults;

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's entry point, through the runtime: libs2 links no driver library.
EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

}  // namespace

namespace tc {

cudaError_t make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t cols, uint64_t rows,
                     uint64_t stride, uint32_t box_cols, uint32_t box_rows, bool swizzle) {
    const EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {stride};
    const cuuint32_t box[2] = {box_cols, box_rows}, one[2] = {1, 1};
    const CUresult r = fn(map, type, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t wait_fault_word(uint32_t** word) {
    static uint32_t* cache[64];
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!cache[dev]) {
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_wait_faults);
        if (e != cudaSuccess) return e;
        cache[dev] = static_cast<uint32_t*>(p);
    }
    *word = cache[dev];
    return cudaSuccess;
}

cudaError_t allow_smem(const void* fn, size_t smem) {
    struct Entry {
        int dev;
        const void* fn;
    };
    static std::mutex mu;
    static Entry table[256];
    static int used = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
        if (table[i].dev == dev && table[i].fn == fn) return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && used < 256) table[used++] = {dev, fn};
    return e;
}

cudaError_t max_pairs(const void* fn, int threads, size_t smem, int* pairs) {
    struct Entry {
        int dev;
        const void* fn;
        int pairs;
    };
    static std::mutex mu;
    static Entry table[64];
    static int used = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
        if (table[i].dev == dev && table[i].fn == fn) {
            *pairs = table[i].pairs;
            return cudaSuccess;
        }
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    if (used < 64) table[used++] = {dev, fn, n};
    *pairs = n;
    return cudaSuccess;
}

}  // namespace tc

cudaError_t read_wait_faults(uint32_t* count) {
    uint32_t* word = nullptr;
    cudaError_t e = tc::wait_fault_word(&word);
    // the copy alone would not wait for streams that do not synchronise with the default one
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    return e == cudaSuccess ? cudaMemcpy(count, word, sizeof(*count), cudaMemcpyDeviceToHost) : e;
}

}  // namespace s2
