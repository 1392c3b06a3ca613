// A row of logits shared by the blocks of a cluster, for the operators that go
// over whole rows of a vocabulary (s2_distill, s2_sample).
//
// The row is cut into groups of eight elements whose addresses are multiples of
// eight elements, so that every group but the first and the last of a row is
// read in 16-byte accesses whatever the row's own alignment (rows of an odd
// length start anywhere). Block `rank` of C owns the groups [NG*rank/C,
// NG*(rank+1)/C). Elements outside the row read as -infinity.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

namespace s2 {
namespace rows {

constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;
constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRowSmem = 204 * 1024;  // beside up to 22 KB of a kernel's own

__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xff800000u); }

struct Part {
    uint32_t off;    // elements between the address of group 0 and the row's first
    uint32_t first;  // first group of this block
    uint32_t count;  // groups of this block
    __device__ __forceinline__ uint32_t groups(uint32_t V) const { return (uint32_t)(((uint64_t)V + off + 7) / 8); }
};
// Element i of the row lies in group (i + off) / 8, at place (i + off) % 8.
template <typename T>
__device__ __forceinline__ Part part_of(const T* row, uint32_t V, uint32_t rank, uint32_t blocks) {
    Part p;
    p.off = (uint32_t)(reinterpret_cast<uintptr_t>(row) / sizeof(T)) % 8;
    const uint64_t n = p.groups(V);
    p.first = (uint32_t)(n * rank / blocks);
    p.count = (uint32_t)(n * (rank + 1) / blocks) - p.first;
    return p;
}
// All eight elements of group g belong to the row.
__device__ __forceinline__ bool inner(const Part& p, uint32_t g, uint32_t V) {
    return (g > 0 || p.off == 0) && (uint64_t)g * 8 + 8 <= (uint64_t)V + p.off;
}
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Group g of the row from global memory, in the type's own bits: two or four words per eight elements.
template <typename T>
struct Raw {
    uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ float element(const Raw<T>& r, int j) {
    if constexpr (sizeof(T) == 4) {
        const uint4 a = r.w[j / 4];
        return __uint_as_float(j % 4 == 0 ? a.x : j % 4 == 1 ? a.y : j % 4 == 2 ? a.z : a.w);
    } else {
        const uint32_t w = j / 2 == 0 ? r.w[0].x : j / 2 == 1 ? r.w[0].y : j / 2 == 2 ? r.w[0].z : r.w[0].w;
        return __uint_as_float(j % 2 ? w & 0xffff0000u : w << 16);
    }
}
template <typename T>
__device__ __forceinline__ Raw<T> edge_group(const T* row, const Part& p, uint32_t g, uint32_t V) {
    uint32_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t i = (int64_t)g * 8 + j - p.off;
        const bool there = i >= 0 && i < (int64_t)V;
        if constexpr (sizeof(T) == 4) e[j] = there ? __float_as_uint(row[i]) : 0xff800000u;
        else e[j] = there ? row[i] : 0xff80u;
    }
    Raw<T> r;
    if constexpr (sizeof(T) == 4) {
        r.w[0] = make_uint4(e[0], e[1], e[2], e[3]);
        r.w[1] = make_uint4(e[4], e[5], e[6], e[7]);
    } else {
        r.w[0] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    }
    return r;
}
template <typename T>
__device__ __forceinline__ Raw<T> load_group(const T* row, const Part& p, uint32_t g, uint32_t V) {
    if (!inner(p, g, V)) return edge_group(row, p, g, V);
    Raw<T> r;
    const uint4* q = reinterpret_cast<const uint4*>(row + ((int64_t)g * 8 - p.off));
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h) r.w[h] = q[h];
    return r;
}

// ---- a block's groups in shared memory -------------------------------------------
// Half h of local group l lies at (h * room + l) * 16: neighbouring lanes read
// neighbouring 16 bytes.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Starts this thread's copies: groups threadIdx.x, threadIdx.x + kRowThreads, ...
template <typename T>
__device__ __forceinline__ void stage(uint4* room, uint32_t size, const T* row, const Part& p, uint32_t V) {
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(room);
    for (uint32_t l = threadIdx.x; l < p.count; l += kRowThreads) {
        const uint32_t g = p.first + l;
        if (inner(p, g, V)) {
            const T* q = row + ((int64_t)g * 8 - p.off);
#pragma unroll
            for (int h = 0; h < (int)sizeof(T) / 2; ++h) copy16(base + (h * size + l) * 16, q + h * 16 / sizeof(T));
        } else {
            const Raw<T> r = edge_group(row, p, g, V);
#pragma unroll
            for (int h = 0; h < (int)sizeof(T) / 2; ++h) room[h * size + l] = r.w[h];
        }
    }
}
template <typename T>
__device__ __forceinline__ Raw<T> staged(const uint4* room, uint32_t size, uint32_t l) {
    Raw<T> r;
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h) r.w[h] = room[h * size + l];
    return r;
}
// Element at place j of local group l.
template <typename T>
__device__ __forceinline__ float staged_at(const uint4* room, uint32_t size, uint32_t l, uint32_t j) {
    if constexpr (sizeof(T) == 4) return reinterpret_cast<const float*>(room + (j / 4 * size + l))[j % 4];
    else return to_float(reinterpret_cast<const uint16_t*>(room + l)[j]);
}

// ---- reductions --------------------------------------------------------------------
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
// The same bits in every lane: each step adds the same two numbers in both.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Address of what lies at `p` in block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float peer_float(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t peer_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t peer_u64(uint32_t a) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}

// Clusters of `blocks` blocks of kernel `fn` that the device holds at once, 0 if
// none (cached); also lets the kernel use kRowSmem bytes of dynamic shared memory.
inline cudaError_t resident_clusters(const void* fn, uint32_t blocks, size_t smem, int* clusters) {
    struct Entry {
        int dev;
        const void* fn;
        uint32_t blocks;
        size_t smem;
        int clusters;
    };
    static std::mutex mu;
    static Entry table[256];
    static int used = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
        if (table[i].dev == dev && table[i].fn == fn && table[i].blocks == blocks && table[i].smem == smem) {
            *clusters = table[i].clusters;
            return cudaSuccess;
        }
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
        cudaGetLastError();  // a failed query is not a launch error
        n = 0;
    }
    if (used < 256) table[used++] = {dev, fn, blocks, smem, n};
    *clusters = n;
    return cudaSuccess;
}

}  // namespace rows
}  // namespace s2
