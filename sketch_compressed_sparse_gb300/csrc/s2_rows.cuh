// A row of logits shared by the blocks of a cluster, for the operators that go
// over whole rows of a vocabulary (s2_distill, s2_sample).
//
// The row is cut into groups of eight elements whose addresses are multiples of
// eight elements, so that every group but the first and the last of a row is
// read in 16-byte accesses whatever the row's own alignment (rows of an odd
// length start anywhere). Block `rank` of C, a power of two, owns the
// groups [NG*rank/C, NG*(rank+1)/C). Elements outside the row read as -infinity.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "s2_remember.h"

namespace s2 {
namespace rows {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRowSmem = 208 * 1024;  // beside up to 18 KB of a kernel's own

__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xff800000u); }

template <typename T>
struct Part {
    const T* base;   // address of this block's first group
    uint32_t off;    // elements between the address of the row's group 0 and its first element
    uint32_t first;  // this block's first group
    uint32_t count;  // its groups
    uint32_t lo, n;  // its groups lo..lo+n-1 lie in the row as a whole
    __device__ __forceinline__ bool inner(uint32_t l) const { return l - lo < n; }
    __device__ __forceinline__ uint64_t groups(uint32_t V) const { return ((uint64_t)V + off + 7) / 8; }
    // index in the row of element j of local group l (beyond the row's ends: below 0 or not below V)
    __device__ __forceinline__ int64_t index(uint32_t l, int j) const { return (int64_t)(first + l) * 8 + j - off; }
    // the row's element i lies in this block
    __device__ __forceinline__ bool holds(uint32_t i, uint32_t V) const {
        return i < V && (uint32_t)(((uint64_t)i + off) / 8) - first < count;
    }
};
// The groups of block `rank` of 2^log2_blocks.
template <typename T>
__device__ __forceinline__ Part<T> part_of(const T* row, uint32_t V, uint32_t rank, uint32_t log2_blocks) {
    Part<T> p;
    p.off = (uint32_t)(reinterpret_cast<uintptr_t>(row) / sizeof(T)) % 8;
    const uint64_t end = (uint64_t)V + p.off, n = (end + 7) / 8;
    p.first = (uint32_t)(n * rank >> log2_blocks);
    p.count = (uint32_t)(n * (rank + 1) >> log2_blocks) - p.first;
    p.base = row + ((int64_t)p.first * 8 - p.off);
    const uint32_t whole = (uint32_t)(end / 8);  // groups before this one end in the row
    p.lo = p.first == 0 && p.off && p.count ? 1 : 0;
    const uint32_t last = whole < p.first + p.count ? whole : p.first + p.count;
    p.n = last > p.first + p.lo ? last - p.first - p.lo : 0;
    return p;
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
// A group at one of the row's ends.
template <typename T>
__device__ __noinline__ Raw<T> edge_group(const Part<T> p, uint32_t l, uint32_t V) {
    uint32_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t i = p.index(l, j);
        const bool there = i >= 0 && i < (int64_t)V;
        if constexpr (sizeof(T) == 4) e[j] = there ? __float_as_uint(p.base[l * 8 + j]) : 0xff800000u;
        else e[j] = there ? p.base[l * 8 + j] : 0xff80u;
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
__device__ __forceinline__ Raw<T> load_inner(const Part<T>& p, uint32_t l) {
    Raw<T> r;
    const uint4* q = reinterpret_cast<const uint4*>(p.base + (uint64_t)l * 8);
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h) r.w[h] = q[h];
    return r;
}
template <typename T>
__device__ __forceinline__ Raw<T> load_group(const Part<T>& p, uint32_t l, uint32_t V) {
    return p.inner(l) ? load_inner(p, l) : edge_group(p, l, V);
}

// ---- a block's groups in shared memory -------------------------------------------
// Half h of local group l lies at (h * room + l) * 16: neighbouring lanes read
// neighbouring 16 bytes.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Starts the copy of local group l, one in the midst of the row, to its place, which only this thread reads.
template <typename T>
__device__ __forceinline__ void stage_inner(uint4* room, uint32_t size, const Part<T>& p, uint32_t l) {
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(room + l);
    const T* q = p.base + (uint64_t)l * 8;
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h) copy16(dst + h * size * 16, q + h * 16 / sizeof(T));
}
// Any group.
template <typename T>
__device__ __forceinline__ void stage_group(uint4* room, uint32_t size, const Part<T>& p, uint32_t l, uint32_t V) {
    if (p.inner(l)) {
        stage_inner(room, size, p, l);
    } else {
        const Raw<T> r = edge_group(p, l, V);
#pragma unroll
        for (int h = 0; h < (int)sizeof(T) / 2; ++h) room[h * size + l] = r.w[h];
    }
}
template <typename T>
__device__ __forceinline__ Raw<T> staged(const uint4* room, uint32_t size, uint32_t l) {
    Raw<T> r;
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h) r.w[h] = room[h * size + l];
    return r;
}
// ---- two floats in one instruction ----------------------------------------------
struct Two {
    uint64_t b;
};
__device__ __forceinline__ Two two(float x, float y) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.b) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 apart(Two a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.b));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(a.b), "l"(b.b), "l"(c.b));
    return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}
// Elements 2j and 2j + 1 of a group.
template <typename T>
__device__ __forceinline__ Two element2(const Raw<T>& r, int j) {
    return two(element(r, 2 * j), element(r, 2 * j + 1));
}
// The largest of a group, NaN aside.
__device__ __forceinline__ float group_max(const Raw<float>& r) {
    return fmaxf(fmaxf(fmaxf(element(r, 0), element(r, 1)), fmaxf(element(r, 2), element(r, 3))),
                 fmaxf(fmaxf(element(r, 4), element(r, 5)), fmaxf(element(r, 6), element(r, 7))));
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float group_max(const Raw<uint16_t>& r) {
    const uint32_t m = max_bf16x2(max_bf16x2(r.w[0].x, r.w[0].y), max_bf16x2(r.w[0].z, r.w[0].w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

// ---- reductions --------------------------------------------------------------------
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
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
// Sum of the words at `p` in the blocks of the cluster (sixteen at most): the
// loads do not wait for one another.
__device__ __forceinline__ uint64_t sum_of_blocks(const void* p, uint32_t blocks) {
    uint64_t sum = 0;
#pragma unroll
    for (uint32_t half = 0; half < 16; half += 8) {
        if (half && blocks <= 8) break;
        uint64_t v[8];
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r) v[r] = half + r < blocks ? peer_u64(peer(p, half + r)) : 0;
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r) sum += v[r];
    }
    return sum;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}

// Shared memory for a slice, in few different sizes: what follows keeps an answer for each.
inline uint64_t smem_of(uint64_t bytes) { return (bytes + 2047) / 2048 * 2048; }

// A question of resident_clusters.
struct Residency {
    const void* fn;
    uint64_t smem;
    uint32_t blocks;
    int dev, threads;
    bool operator==(const Residency& o) const {
        return fn == o.fn && smem == o.smem && blocks == o.blocks && dev == o.dev && threads == o.threads;
    }
    uint64_t hash() const {
        return spread(spread(reinterpret_cast<uintptr_t>(fn) + smem) + (uint64_t)blocks * 4096 * 256 + (uint64_t)threads * 256 + (uint64_t)dev);
    }
};

// Clusters of `blocks` blocks of kernel `fn` that the device holds at once, 0 if
// none (kept); also lets the kernel use kRowSmem bytes of dynamic shared memory.
inline cudaError_t resident_clusters(const void* fn, int threads, uint32_t blocks, size_t smem, int* clusters) {
    static std::mutex mu;
    static Remembered<Residency, int, 512> kept;
    Residency q{fn, smem, blocks, 0, threads};
    cudaError_t e = cudaGetDevice(&q.dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (kept.find(q, clusters)) return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3((unsigned)threads);
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
    kept.put(q, n);
    *clusters = n;
    return cudaSuccess;
}

}  // namespace rows
}  // namespace s2
