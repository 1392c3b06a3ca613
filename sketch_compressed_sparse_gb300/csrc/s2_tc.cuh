// Blackwell tensor-core building blocks (sm_103a): barriers in shared memory
// with bounded waits, tiled copies (TMA), tensor memory and tcgen05 products.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace s2 {
namespace tc {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

// True in one lane of a converged warp. The warps that issue copies and
// products stay converged and issue under this predicate: their loop counters
// and addresses are then uniform, which those instructions' operands have to be.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{.reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p;}" : "=r"(p));
    return p != 0;
}

// ---- mbarriers ---------------------------------------------------------------
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_fence_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{.reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p;}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// Every wait is bounded. One that runs out (kWaitNs after it began to be slow)
// sets the block's `dead` word, which ends the other waits of the block, and
// counts in *faults; the block then finishes its copies in flight, frees its
// tensor memory and returns. The call's outputs are not valid then.
constexpr uint64_t kWaitNs = 4000000000ull;

struct Wait {
    volatile uint32_t* dead;  // shared memory
    uint32_t* faults;         // device memory
};

static __device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, const Wait w) {
    uint64_t t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 256; ++i)
            if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;
        if (t0 == 0) t0 = now_ns();
        const bool late = now_ns() - t0 > kWaitNs;
        if (late && threadIdx.x % 32 == 0) {
            *w.dead = 1;
            atomicAdd(w.faults, 1u);
        }
        if (__any_sync(0xffffffffu, late || *w.dead)) return false;
    }
}
// Whole warp, converged; the answer is the same in every lane. (Kept small
// where it is inlined: the warps of a block run many different loops, and their
// instructions have to stay in the cache.)
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const Wait& w) {
    return __all_sync(0xffffffffu, bar_try(bar, parity)) || bar_wait_slow(bar, parity, w);
}
// For the copies in flight of a block that gave up: no `dead` word ends it.
static __device__ __noinline__ void bar_drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = now_ns();
    while (!bar_try(bar, parity) && now_ns() - t0 < kWaitNs) {
    }
}

// Position in a ring of N slots and the parity of the phase that its next use completes.
template <int N>
struct Slot {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) {
            at = 0;
            phase ^= 1;
        }
    }
};

// ---- TMA ---------------------------------------------------------------------
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tensor memory -----------------------------------------------------------
// Whole warp; `slot` in shared memory receives the address.
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 or 32 neighbouring columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
// Waits for the loads in flight, one of which fills r: r is not touched before.
// (A wait that does not name the registers would not keep their uses behind it.)
__device__ __forceinline__ void wait_ld16(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// ---- products ----------------------------------------------------------------
// Descriptor of an operand tile in shared memory under the 128-byte swizzle.
// lead, stride: the strides in bytes between repeats of the 128-byte row
// (only for operands whose rows run along M or N) and between groups of eight rows.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// Arrives at `bar` once the products issued by this thread so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 8-bit operands with a scale byte for each row and 32 elements of K.
__device__ __forceinline__ void mma_mx8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        bool add) {
    asm volatile(
        "{.reg .pred p; setp.ne.u32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add)
        : "memory");
}
// bfloat16 operands.
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{.reg .pred p; setp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

// ---- pairs of blocks (a cluster of two on one tile) -----------------------------
__device__ __forceinline__ void tmem_alloc_pair(uint32_t slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
// Arrives at `bar` of both blocks once the products issued by this thread so far are done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{.reg .pred p; setp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_mx8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, bool add) {
    asm volatile(
        "{.reg .pred p; setp.ne.u32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add)
        : "memory");
}
// Address, in the cluster's window, of what lies at `addr` in the pair's first block.
__device__ __forceinline__ uint32_t in_first(uint32_t addr) {
    uint32_t p;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(p) : "r"(addr));
    return p;
}
// Copy into this block's memory that reports to a barrier of the pair's first block (its cluster address).
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// Arrives at the barrier that lies at `bar` in the first block of the pair.
__device__ __forceinline__ void bar_arrive_first(uint32_t bar) {
    asm volatile(
        "{.reg .b32 p; mapa.shared::cluster.u32 p, %0, 0;\n"
        "mbarrier.arrive.shared::cluster.b64 _, [p];}" ::"r"(bar)
        : "memory");
}

// ---- clusters ----------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The sum, in the order of the ranks, of the four floats at `addr` of blocks
// 0..blocks-1 (at most 8). All loads are on their way before the first addition.
__device__ __forceinline__ float4 sum_of_peers(uint32_t addr, uint32_t blocks) {
    float4 v[8];
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r) {
        v[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < blocks) {
            uint32_t p;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(addr), "r"(r));
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                         : "r"(p)
                         : "memory");
        }
    }
    float4 s = v[0];
#pragma unroll
    for (uint32_t r = 1; r < 8; ++r) {
        s.x += v[r].x;
        s.y += v[r].y;
        s.z += v[r].z;
        s.w += v[r].w;
    }
    return s;
}

// ---- host: tensor maps -------------------------------------------------------
// Two-dimensional map of `rows` rows of `cols` elements, `stride` bytes apart,
// copied in boxes of box_rows x box_cols under the 128-byte swizzle; what lies
// outside reads as zero. Base 16-byte aligned, stride a multiple of 16.
// (swizzle = false: rows of the box lie one after the other.)
cudaError_t make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t cols, uint64_t rows,
                     uint64_t stride, uint32_t box_cols, uint32_t box_rows, bool swizzle = true);

// Lets kernel `fn` use `smem` bytes of dynamic shared memory (set once per device).
cudaError_t allow_smem(const void* fn, size_t smem);

// Pairs of blocks of kernel `fn` that the device holds at once (cached); also
// lets the kernel use `smem` bytes of dynamic shared memory.
cudaError_t max_pairs(const void* fn, int threads, size_t smem, int* pairs);

// Device word that counts waits that ran out.
cudaError_t wait_fault_word(uint32_t** word);

}  // namespace tc
}  // namespace s2
