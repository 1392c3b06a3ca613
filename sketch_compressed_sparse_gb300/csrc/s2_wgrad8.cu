// dW[n][k] (+)= sum_t dY[t][n] * X[t][k] with dY in bfloat16 and X an 8-bit
// packed activation.
//
// A code times its power-of-two scale has four significant bits, so it is
// exact in bfloat16: the 8-bit rows are widened on the way into shared memory
// and the product is a bfloat16 one on the tensor cores with float32 sums, at
// half the activation's bytes. Both operands are read as they lie, rows along
// the outputs' axes (tokens are the summed axis), so nothing is transposed.
//
// Features of X are the accumulator's lanes and outputs its columns:
// neighbouring lanes hold neighbouring k, so stores run along dW's rows
// whatever its alignment. A block of 128 features shares one scale per token.
// dY comes by tiled copies where its rows start on 16 bytes. Else (an odd
// vocabulary) the rows t = r mod 8 are one matrix whose rows all miss 16 bytes
// by the same amount; each r is copied from the 16-byte boundary before (the
// piece that holds the row's first element) and its warp shifts the rows into
// place.
//
// Measured: 200 tokens, 512 x 512 4.4 us in a CUDA graph; 8192 tokens, 4096 x 4096
// into bfloat16 196 us in a long loop (1.40 PFLOP/s, 0.73 of a cuBLAS product at
// its burst rate) and 177 us for ten in a row; 2048 tokens, 267735 x 1024, odd
// rows, into float32 1.03 ms (1.09 PFLOP/s).
#include "s2_chunks.h"
#include "s2_internal.h"
#include "s2_launch.cuh"
#include "s2_tc.cuh"

namespace s2 {
namespace {

using namespace tc;

constexpr int kBT = 64;                    // tokens per stage
constexpr int kBF = 128;                   // features per tile
constexpr uint32_t kGroupBytes = kBT * 128;  // 64 outputs or features by kBT tokens
constexpr uint32_t kABytes = 2 * kGroupBytes;
// The tensor cores add to their float32 sums with truncation. Normal inputs,
// relative error of one sum: 6.4e-7 at 2048 tokens, 3.7e-6 at 8192, 4.8e-5 at
// 65536 (a float32 matrix product: 1.5e-7, 3.6e-7, 1.5e-6); 2.4e-6 and 9.5e-6 at
// the first two with heavy-tailed gradients. So a float32 result is taken in
// chunks of at most kChunk stages that are added up with rounding: 1.9e-7 up to
// 8192 tokens, 2.6e-7 at 65536, 4.0e-7 at 262144 (the additions' own roundings
// grow with the root of their number); heavy-tailed 8e-7 at 2048.
// The sum stays in tensor memory, in the accumulator of the tile's first chunk;
// later chunks use the other one, and the products wait only while it is added
// (additions in L2 or through registers took twice as long in all).
constexpr uint32_t kChunk = 11;
// A bfloat16 result is rounded by up to 2^-8 of itself, 1.7e-3 in the mean square,
// so its chunks are longer: 2048 tokens lose 6e-7 to 2.4e-6, at most a 700th of
// that, whatever the number of chunks. (One chunk went on growing with the tokens,
// always towards zero; 8192 x 4096 x 4096, ten in a row: one chunk 172 us, chunks of
// 32 stages 177, of 11 198.)
constexpr uint32_t kChunk16 = 32;
constexpr int kLoaders = 8;                // warps that shift a misaligned dY into place

struct Args {
    const uint16_t* dy;
    uint64_t lddy;
    const uint8_t* x;
    uint64_t ldx;
    const uint8_t* xs;
    void* dw;
    uint64_t lddw;
    uint32_t T, N, K, nblk;
    uint32_t tiles_k, tiles_n;
    uint32_t split;
    uint32_t nt;  // outputs per tile, a multiple of 32
    int dtype;
    uint32_t* faults;
};

// The scale 2^(b - 127) as a bfloat16, twice in a word (the byte 0 is a
// subnormal number, 255 stands for NaN).
__device__ __forceinline__ uint32_t factor_of(uint32_t b) {
    const uint32_t f = b == 0 ? 0x0040u : b == 255 ? 0x7fffu : b << 7;
    return f | f << 16;
}

// Sixteen codes times their scale to bfloat16, in order. Every step is exact
// (a code has four significant bits; scales from 2^-117 on keep it normal), and
// NaN stays NaN. Arithmetic on the bits with a check for NaN instead of the
// conversions measured 211 us for 198 us (8192 tokens, 4096 x 4096).
__device__ __forceinline__ void widen16(const uint4& c, uint32_t factor, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[2];
        asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
            : "=r"(h[0]), "=r"(h[1])
            : "r"(w[i]));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float l, u;
            uint32_t p;
            asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(l), "=f"(u) : "r"(h[j]));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p) : "f"(u), "f"(l));
            asm("mul.bf16x2 %0, %1, %2;" : "=r"(o[2 * i + j]) : "r"(p), "r"(factor));
        }
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ void st_shared(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Makes this thread's shared-memory stores visible to the tensor cores.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) {
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(*p) : "f"(v));  // the one rounding to 16 bits: dW's own type
}
__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Sixteen sums of a feature to the outputs from p on, `step` apart, of which
// the first `count` exist.
template <typename T>
__device__ __forceinline__ void store16(T* p, uint64_t step, int count, const uint32_t* r) {
    if (count >= 16) {
#pragma unroll
        for (int j = 0; j < 16; ++j, p += step) put(p, __uint_as_float(r[j]));
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j, p += step)
            if (j < count) put(p, __uint_as_float(r[j]));
    }
}
template <typename T>
__device__ __forceinline__ void load16(const T* p, uint64_t step, int count, T* v) {
    if (count >= 16) {
#pragma unroll
        for (int j = 0; j < 16; ++j, p += step) v[j] = *p;
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j, p += step) v[j] = j < count ? *p : T(0);
    }
}

// A tile's sums to dW; the next ones leave tensor memory while sixteen are stored
// (12 tokens, 12000 x 2944 into bfloat16 28 us; loading and storing in turn 31).
template <typename T>
__device__ __forceinline__ void store_tile(T* p, uint64_t step, int count, uint32_t nt, uint32_t sum) {
    uint32_t r[16], next[16];
    tmem_ld16(sum, r);
    wait_ld16(r);
#pragma unroll 1
    for (uint32_t c = 0; c < nt; c += 32, count -= 32) {  // (nt is a multiple of 32)
        tmem_ld16(sum + c + 16, next);
        store16(p, step, count, r);
        p += 16 * step;
        wait_ld16(next);
        if (c + 32 < nt) tmem_ld16(sum + c + 32, r);
        store16(p, step, count - 16, next);
        p += 16 * step;
        wait_ld16(r);
    }
}

// dW += a tile's sums. A thread's sixteen old values are loaded together, and
// before the stores of the sixteen before: one by one, 12000 x 2944 of them
// took 843 us, so 77 (12 tokens, float32; 3.7 TB/s). Adding in memory took 56,
// but turns subnormal numbers into zeros. A kernel of its own (ADD): in one with
// the plain stores the old values cost those registers, 33 -> 45 us.
template <typename T>
__device__ __forceinline__ void add_tile(T* p, uint64_t step, int count, uint32_t nt, uint32_t sum) {
    T old[16];
    load16(p, step, count, old);
#pragma unroll 1
    for (uint32_t c = 0; c < nt; c += 16, p += 16 * step, count -= 16) {
        uint32_t r[16];
        tmem_ld16(sum + c, r);
        wait_ld16(r);
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(value(old[j]) + __uint_as_float(r[j]));
        if (c + 16 < nt) load16(p + 16 * step, step, count - 16, old);
        store16(p, step, count, r);
    }
}

// Sixteen bytes from byte `shift` (even, below 16) of a and b on: whole words
// by the (warp-uniform) branch, half a word by the funnel.
template <int WORDS>
__device__ __forceinline__ uint4 from_word(const uint4& a, const uint4& b, uint32_t bits) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint4 o;
    o.x = __funnelshift_r(w[WORDS], w[WORDS + 1], bits);
    o.y = __funnelshift_r(w[WORDS + 1], w[WORDS + 2], bits);
    o.z = __funnelshift_r(w[WORDS + 2], w[WORDS + 3], bits);
    o.w = __funnelshift_r(w[WORDS + 3], w[(WORDS + 4) % 8], bits);
    return o;
}

// A tile is 128 features by 128 outputs on one SM, or twice that each way on a
// pair of SMs (CTAS = 2): each block widens its own 128 features and fetches
// 128 of the outputs, and the pair's product reads both blocks' shared memory,
// so it does four times the products of one block's on twice the loads.
//
// What bounds it is the traffic of shared memory. A stage of 256 outputs, 512
// clocks of products, moves in units of 128 bytes: products' reads 256, dY 128
// (misaligned: copy 136, load 160, store 128), X copy 64, load 64, store 128:
// 640 aligned and 936 misaligned, where 754 and 1045 clocks were measured.
// Widened X in tensor memory instead took 256 of that away, but left room for
// 192 outputs only, and the copies from L2 (24 KB for 384 clocks of products)
// bound it then: 216 us for 191 at 8192 x 4096 x 4096.
//
// The loops of the block's roles are kept small on purpose: with a copy of the
// shift for each misalignment the instruction cache missed and the misaligned
// form took 2.3 times as long.
constexpr int kHalfN = 128;            // outputs that a block fetches
constexpr uint32_t kXRaw = kBT * kBF;  // 8-bit part of a stage
constexpr uint32_t kBBytes = kHalfN / 64 * kGroupBytes;
constexpr uint32_t kRowRaw = (kHalfN + 8) * 2;     // a misaligned row's piece: 8 elements more
constexpr uint32_t kYRaw = kBT * kRowRaw;

struct YMaps {
    CUtensorMap m[8];  // aligned rows: m[0]; else the rows t = r mod 8 for each r
};

// Four rings in shared memory: 8-bit rows of X, widened X (A), dY in place (B)
// and, for misaligned rows, dY as it lies. B and the raw rows are the deeper
// ones: they wait for HBM, A only for the arithmetic.
template <bool ALIGNED, int CTAS>
struct Form {
    // Teams of four warps widen X, a stage each in turn. A has a slot per team
    // and the raw rows of X kXs, so that a team meets every use of its own
    // slots and can tell their phases by one bit.
    static constexpr int kTeams = ALIGNED ? 4 : 3, kXs = ALIGNED ? 1 : 2;
    static constexpr int kA = kTeams, kX = kXs * kTeams, kB = ALIGNED ? 7 : 3, kY = ALIGNED ? 0 : 4;
    static constexpr uint32_t kBAt = kA * kABytes, kXAt = kBAt + kB * kBBytes, kYAt = kXAt + kX * kXRaw;
    static constexpr size_t kSmem = kYAt + kY * kYRaw + 1024;
    static constexpr int kAcc = 2;
    static constexpr uint32_t kTileN = CTAS * kHalfN, kCols = kAcc * kTileN;
    static constexpr int kWideners = 4 * kTeams;
    static constexpr int kWarps = 4 + kWideners + 2 + (ALIGNED ? 0 : kLoaders);
    static constexpr int kBars = 2 * kX + 2 * kA + 3 * kB + 2 * kY + 2 * kAcc + 1;
    static_assert(kYRaw % 1024 == 0, "rings start on the swizzle's period");
    static_assert(kB >= kA, "a stage's B outlives its A");
    static_assert(kSmem <= 226 * 1024, "shared memory");
    static_assert((size_t)kTileN * kBF * 4 <= kSmem - 1024 || CTAS == 2, "a partial tile fits where the rings were");
};

// Arrives at a barrier of the block that issues the products.
template <int CTAS>
__device__ __forceinline__ void arrive_issuer(uint32_t bar) {
    if constexpr (CTAS == 2) bar_arrive_first(bar);
    else bar_arrive(bar);
}
template <int CTAS>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (CTAS == 2) mma_commit_pair(bar);
    else mma_commit(bar);
}

__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// Shifts one warp's rows of every stage into place: row q of residue r goes to
// row 8r + (q ^ r % 2) of the operand (the tokens of a stage may lie in any
// order as long as both operands agree), which keeps this warp's and the
// wideners' stores free of bank conflicts.
template <int CTAS>
__device__ __forceinline__ void realign(uint32_t stages, uint32_t y0, uint32_t b0, uint32_t yfull, uint32_t yempty,
                                        uint32_t bfull, uint32_t bempty, const Wait& wt, uint32_t r, uint32_t lane,
                                        uint32_t shift) {
    using P = Form<false, CTAS>;
    const uint32_t q = lane % 8, c0 = lane / 8 * 4, row = q ^ (r % 2), bits = shift % 4 * 8;
    Slot<P::kY> ys;
    Slot<P::kB> bs;
    for (uint32_t it = 0; it < stages; ++it) {
        if (!bar_wait(yfull + 8 * ys.at, ys.phase, wt)) return;
        const uint32_t src = y0 + ys.at * kYRaw + (r * 8 + q) * kRowRaw + c0 * 16;
        uint4 v[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) v[i] = ld_shared(src + 16 * i);
        uint4 o[4];
        switch (shift / 4) {
            case 0:
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = from_word<0>(v[i], v[i + 1], bits);
                break;
            case 1:
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = from_word<1>(v[i], v[i + 1], bits);
                break;
            case 2:
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = from_word<2>(v[i], v[i + 1], bits);
                break;
            default:
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = from_word<3>(v[i], v[i + 1], bits);
        }
        if (!bar_wait(bempty + 8 * bs.at, bs.phase ^ 1, wt)) return;
        const uint32_t dst = b0 + bs.at * kBBytes + (r * 8 + row) * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = c0 + i;
            st_shared(dst + c / 8 * kGroupBytes + ((c % 8) ^ row) * 16, o[i]);
        }
        // The raw slot is released only here: the stores above have the loaded
        // values, and the fence orders the loads before the next copy into the
        // slot. (An arrival right after the loads were issued let that copy
        // overtake them.)
        fence_async();
        __syncwarp();
        if (lane == 0) {
            bar_arrive(yempty + 8 * ys.at);
            arrive_issuer<CTAS>(bfull + 8 * bs.at);
        }
        ys.next();
        bs.next();
    }
}

template <bool ALIGNED, int CTAS, bool ADD>
__global__ void __launch_bounds__(Form<ALIGNED, CTAS>::kWarps * 32, 1)
    wgrad8_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ YMaps ymaps, const Args a) {
    using P = Form<ALIGNED, CTAS>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[P::kBars];
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t dead;

    const uint32_t a0 = (smem_u32(raw) + 1023u) & ~1023u, b0 = a0 + P::kBAt, x0 = a0 + P::kXAt, y0 = a0 + P::kYAt;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // the block's place in its pair, and (CTAS = 1) its part of the tokens
    const uint32_t rank = CTAS == 2 ? cluster_rank() : 0, part = CTAS == 1 && a.split > 1 ? cluster_rank() : 0;
    const uint32_t xfull = smem_u32(bars), xempty = xfull + 8 * P::kX;
    const uint32_t afull = xempty + 8 * P::kX, aempty = afull + 8 * P::kA;       // the first block's afull counts
    const uint32_t bfull = aempty + 8 * P::kA, bempty = bfull + 8 * P::kB;       // both; the same for bfull
    const uint32_t copied = bempty + 8 * P::kB;                                  // this block's B, by tiled copy
    const uint32_t yfull = copied + 8 * P::kB, yempty = yfull + 8 * P::kY;
    const uint32_t acc_full = yempty + 8 * P::kY, acc_empty = acc_full + 8 * P::kAcc, drain = acc_empty + 8 * P::kAcc;

    if (threadIdx.x == 0) {
        for (int s = 0; s < P::kX; ++s) {
            bar_init(xfull + 8 * s, 1);
            bar_init(xempty + 8 * s, 4);
        }
        for (int s = 0; s < P::kA; ++s) {
            bar_init(afull + 8 * s, CTAS * 4);
            bar_init(aempty + 8 * s, 1);
        }
        for (int s = 0; s < P::kB; ++s) {
            bar_init(bfull + 8 * s, CTAS * kLoaders);
            bar_init(bempty + 8 * s, 1);
            bar_init(copied + 8 * s, 1);
        }
        for (int s = 0; s < P::kY; ++s) {
            bar_init(yfull + 8 * s, 1);
            bar_init(yempty + 8 * s, kLoaders);
        }
        for (int s = 0; s < P::kAcc; ++s) {
            bar_init(acc_full + 8 * s, 1);
            bar_init(acc_empty + 8 * s, CTAS * 4);
        }
        bar_init(drain, 1);
        dead = 0;
        bar_fence_init();
    }
    constexpr int kCopier = 4 + P::kWideners, kIssuer = kCopier + 1;
    if (warp == kIssuer) {
        if constexpr (CTAS == 2) tmem_alloc_pair(smem_u32(&tmem_slot), P::kCols);
        else tmem_alloc(smem_u32(&tmem_slot), P::kCols);
    }
    fence_before();
    if constexpr (CTAS == 2) cluster_sync();
    else __syncthreads();
    fence_after();
    stream_order();
    const uint32_t tmem = tmem_slot;
    const Wait wt{&dead, a.faults};
    const uint32_t group = CTAS == 2 ? 2 : a.split;  // blocks that work on one tile
    const uint32_t first = blockIdx.x / group, step = gridDim.x / group, tiles = a.tiles_k * a.tiles_n;
    const uint32_t all_tb = (a.T + kBT - 1) / kBT, tb0 = (uint32_t)((uint64_t)all_tb * part / a.split);
    const uint32_t tblocks = (uint32_t)((uint64_t)all_tb * (part + 1) / a.split) - tb0;
    const uint32_t mine = first < tiles ? (tiles - first - 1) / step + 1 : 0, stages = mine * tblocks;
    const uint32_t chunks = chunk_count(tblocks, a.dtype == 0 ? kChunk : kChunk16);

    if (warp == kCopier) {
        const bool leader = elect();
        Slot<P::kX> xs;
        Slot<ALIGNED ? P::kB : P::kY> ys;
        uint32_t nx = 0, ny = 0;  // copies issued
        bool ok = true;
        for (uint32_t tile = first; ok && tile < tiles; tile += step) {
            const int k0 = (int)((tile % a.tiles_k * CTAS + rank) * kBF);
            const int n0 = (int)(tile / a.tiles_k * a.nt + rank * (a.nt / CTAS));
            for (uint32_t tb = 0; tb < tblocks; ++tb) {
                if (!(ok = bar_wait(xempty + 8 * xs.at, xs.phase ^ 1, wt))) break;
                if (leader) {
                    bar_expect(xfull + 8 * xs.at, kXRaw);
                    tma_2d(x0 + xs.at * kXRaw, &xmap, xfull + 8 * xs.at, k0, (int)((tb0 + tb) * kBT));
                }
                xs.next();
                ++nx;
                if (!(ok = bar_wait((ALIGNED ? bempty : yempty) + 8 * ys.at, ys.phase ^ 1, wt))) break;
                if (leader) {
                    if (ALIGNED) {
                        bar_expect(copied + 8 * ys.at, kBBytes);
#pragma unroll
                        for (int c = 0; c < kHalfN / 64; ++c)
                            tma_2d(b0 + ys.at * kBBytes + c * kGroupBytes, &ymaps.m[0], copied + 8 * ys.at, n0 + 64 * c,
                                   (int)((tb0 + tb) * kBT));
                    } else {
                        bar_expect(yfull + 8 * ys.at, kYRaw);
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            tma_2d(y0 + ys.at * kYRaw + r * 8 * kRowRaw, &ymaps.m[r], yfull + 8 * ys.at, n0,
                                   (int)((tb0 + tb) * kBT / 8) + (r < (int)a.T ? 0 : 8));
                    }
                }
                ys.next();
                ++ny;
            }
        }
        // nothing of this block's may still be on its way when it ends
        if (dead && leader) {
            constexpr uint32_t kYs = ALIGNED ? P::kB : P::kY;
            for (uint32_t j = nx > (uint32_t)P::kX ? nx - P::kX : 0; j < nx; ++j)
                bar_drain(xfull + 8 * (j % P::kX), (j / P::kX) & 1);
            for (uint32_t j = ny > kYs ? ny - kYs : 0; j < ny; ++j)
                bar_drain((ALIGNED ? copied : yfull) + 8 * (j % kYs), (j / kYs) & 1);
        }
    } else if (warp == kIssuer) {
        if (rank == 0) {
            const bool leader = elect();  // the thread that issues the products also commits them
            // D float32, A and B bfloat16, both with rows along M and N
            const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | 1u << 15 | 1u << 16 | (a.nt / 8) << 17 |
                                   (uint32_t)(CTAS * kBF / 16) << 24;
            Slot<P::kA> as;
            Slot<P::kB> bs;
            uint32_t acc = 0, uses[P::kAcc] = {};  // how often each accumulator was taken
            bool ok = true;
            for (uint32_t tile = first; ok && tile < tiles; tile += step, acc ^= 1) {
                for (uint32_t c = 0, tb = 0; ok && c < chunks; ++c) {
                    const uint32_t at = c ? acc ^ 1 : acc, from = tb, end = chunk_end(tblocks, chunks, c);
                    if (!(ok = bar_wait(acc_empty + 8 * at, (uses[at]++ & 1) ^ 1, wt))) break;
                    fence_after();
                    for (; tb < end; ++tb) {
                        if (!ALIGNED && !(ok = bar_wait(bfull + 8 * bs.at, bs.phase, wt))) break;
                        if (!(ok = bar_wait(afull + 8 * as.at, as.phase, wt))) break;
                        fence_after();
                        const uint64_t ad = smem_desc(a0 + as.at * kABytes, kGroupBytes, 1024);
                        const uint64_t bd = smem_desc(b0 + bs.at * kBBytes, kGroupBytes, 1024);
                        if (leader) {
#pragma unroll
                            for (int j = 0; j < kBT / 16; ++j) {  // 16 tokens: two groups of eight rows
                                const uint32_t d = tmem + at * P::kTileN;
                                if constexpr (CTAS == 2) mma_bf16_pair(d, ad + 128 * j, bd + 128 * j, idesc, tb > from || j > 0);
                                else mma_bf16(d, ad + 128 * j, bd + 128 * j, idesc, tb > from || j > 0);
                            }
                            commit<CTAS>(aempty + 8 * as.at);
                            commit<CTAS>(bempty + 8 * bs.at);
                        }
                        as.next();
                        bs.next();
                    }
                    if (ok && leader) commit<CTAS>(acc_full + 8 * at);
                }
            }
            if (dead && leader) {
                commit<CTAS>(drain);
                bar_drain(drain, 0);
            }
        }
    } else if (warp > kIssuer) {
        const uint32_t r = warp - kIssuer - 1;
        realign<CTAS>(stages, y0, b0, yfull, yempty, bfull, bempty, wt, r, lane,
                (uint32_t)((reinterpret_cast<uintptr_t>(a.dy) + (uint64_t)r * a.lddy * 2) % 16));
    } else if (warp >= 4) {
        // Widen X: a warp takes sixteen tokens, eight tokens by 64 features at a
        // step, four lanes a token. Neighbouring tokens take the halves of the
        // features in opposite order, so that the pieces of eight neighbouring
        // lanes lie in different banks on both sides. The teams take the stages
        // in turn: a stage's chain of waits, loads and fences is several times
        // as long as its product.
        const uint32_t team = (warp - 4) / 4, w = warp % 4, piece = lane % 4, odd = lane / 4 % 2, sub = lane / 8 * 2 + odd;
        const uint32_t src0 = x0 + team * kXRaw + (w * 16 + sub) * 128 + ((odd * 4 + piece) ^ sub) * 16;
        const uint32_t dst = a0 + team * kABytes + odd * kGroupBytes;
        uint32_t to[2];  // token's row in the operand, and its first piece; the other is 16 bytes up or down
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t row = ALIGNED ? w * 16 + i * 8 + sub : sub * 8 + ((w * 2 + i) ^ odd);
            to[i] = dst + row * 128 + ((2 * piece) ^ (row % 8)) * 16;
        }
        bool ok = true;
        // scale bytes are fetched one turn ahead
        uint32_t ahead = first, ahead_tb = team, kb = first % a.tiles_k * CTAS + rank;
        auto next_scales = [&](uint32_t* b) {
            while (ahead_tb >= tblocks && ahead < tiles) {
                ahead_tb -= tblocks;
                ahead += step;
                kb = ahead % a.tiles_k * CTAS + rank;
            }
            b[0] = b[1] = 127;
            if (ahead < tiles && kb < a.nblk) {
                const uint32_t t = (tb0 + ahead_tb) * kBT + w * 16 + sub;
                const uint8_t* p = a.xs + (uint64_t)t * a.nblk + kb;
                if (t < a.T) b[0] = *p;
                if (t + 8 < a.T) b[1] = p[8 * a.nblk];
            }
            ahead_tb += P::kTeams;
        };
        uint32_t now[2], then[2], phase = 0;
        next_scales(then);
        Slot<P::kXs> xs;
        Slot<P::kB> bs;
        for (uint32_t i = 0; i < team; ++i) bs.next();
        for (uint32_t it = team; ok && it < stages; it += P::kTeams, phase ^= 1) {
            now[0] = then[0];
            now[1] = then[1];
            next_scales(then);
            const uint32_t x = team + xs.at * P::kTeams, src = src0 + xs.at * P::kTeams * kXRaw;
            if (!(ok = bar_wait(xfull + 8 * x, xs.phase, wt))) break;
            uint4 c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = ld_shared((src ^ (i % 2 * 64)) + i / 2 * 1024);
            xs.next();
            // all the arithmetic before the wait: only the stores lie between a
            // slot's release and its next product
            uint4 lo[4], up[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) widen16(c[i], factor_of(now[i / 2]), lo[i], up[i]);
            if (!(ok = bar_wait(aempty + 8 * team, phase ^ 1, wt))) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t at = to[i / 2] + (i % 2 ? (odd ? -kGroupBytes : kGroupBytes) : 0);
                st_shared(at, lo[i]);
                st_shared(at ^ 16, up[i]);
            }
            fence_async();
            // this arrival also tells the first block that this block's B has come
            if (ALIGNED && !(ok = bar_wait(copied + 8 * bs.at, bs.phase, wt))) break;
            __syncwarp();
            if (lane == 0) {
                bar_arrive(xempty + 8 * x);  // as in realign(): not before the loaded values are stored
                arrive_issuer<CTAS>(afull + 8 * team);
            }
#pragma unroll
            for (int i = 0; i < P::kTeams; ++i) bs.next();
        }
    } else {
        uint32_t acc = 0, uses[P::kAcc] = {};
        bool ok = true;
        const uint32_t mine0 = tmem + ((uint32_t)warp << 21);
        for (uint32_t tile = first; ok && tile < tiles; tile += step, acc ^= 1) {
            const uint32_t sum = mine0 + acc * P::kTileN, other = mine0 + (acc ^ 1) * P::kTileN;
            if (ADD && (CTAS == 2 || a.split == 1)) {
                // the old values on their way to L2 while the products run (8192 x 8192, 12 tokens: 199 -> 131 us)
                const uint32_t pk = (tile % a.tiles_k * CTAS + rank) * kBF + warp * 32, pn = tile / a.tiles_k * a.nt;
                for (uint32_t c = lane; pk < a.K && c < a.nt && pn + c < a.N; c += 32)
                    prefetch_l2(static_cast<const uint8_t*>(a.dw) + ((uint64_t)(pn + c) * a.lddw + pk) * (a.dtype == 0 ? 4 : 2));
            }
            if (!(ok = bar_wait(acc_full + 8 * acc, uses[acc]++ & 1, wt))) break;
            for (uint32_t i = 1; i < chunks; ++i) {
                if (!(ok = bar_wait(acc_full + 8 * (acc ^ 1), uses[acc ^ 1]++ & 1, wt))) break;
                fence_after();
#pragma unroll 1
                for (uint32_t c = 0; c < a.nt; c += 16) {
                    uint32_t r[16], v[16];
                    tmem_ld16(sum + c, r);
                    tmem_ld16(other + c, v);
                    wait_ld16(r);
                    wait_ld16(v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(v[j]));
                    tmem_st16(sum + c, r);
                }
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_issuer<CTAS>(acc_empty + 8 * (acc ^ 1));
                wait_st();
            }
            if (!ok) break;
            fence_after();
            const uint32_t k = (tile % a.tiles_k * CTAS + rank) * kBF + warp * 32 + lane, n0 = tile / a.tiles_k * a.nt;
            const uint64_t at = (uint64_t)n0 * a.lddw + k;
            const int rows = n0 < a.N ? (int)min(a.N - n0, a.nt) : 0;
            if (ADD && (CTAS == 2 || a.split == 1)) {
                // (features past the end add nothing, but read their part of the accumulator with the others)
                const int count = k < a.K ? rows : 0;
                if (a.dtype == 0) add_tile(static_cast<float*>(a.dw) + at, a.lddw, count, a.nt, sum);
                else add_tile(static_cast<uint16_t*>(a.dw) + at, a.lddw, count, a.nt, sum);
            } else if (CTAS == 1 && a.split > 1) {
                // this block's part of the sums, where the rings were
                float* part_sums = reinterpret_cast<float*>(raw + (a0 - smem_u32(raw)));
#pragma unroll 1
                for (uint32_t c = 0; c < a.nt; c += 16) {
                    uint32_t r[16];
                    tmem_ld16(sum + c, r);
                    wait_ld16(r);
#pragma unroll
                    for (int j = 0; j < 16; ++j) part_sums[(c + j) * kBF + warp * 32 + lane] = __uint_as_float(r[j]);
                }
            } else {
                const int count = k < a.K ? rows : 0;
                if (a.dtype == 0) store_tile(static_cast<float*>(a.dw) + at, a.lddw, count, a.nt, sum);
                else store_tile(static_cast<uint16_t*>(a.dw) + at, a.lddw, count, a.nt, sum);
            }
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_issuer<CTAS>(acc_empty + 8 * acc);
        }
    }

    __syncwarp();
    if (CTAS == 1 && a.split > 1) {
        // one tile per cluster: each block adds the parts of its own columns,
        // in the order of the parts, so the sums do not depend on timing
        cluster_sync();
        const uint32_t k = first % a.tiles_k * kBF + lane * 4, n0 = first / a.tiles_k * a.nt;
        const uint32_t c0 = a.nt * part / a.split, c1 = a.nt * (part + 1) / a.split;
        if (!dead) {
            for (uint32_t c = c0 + warp; c < c1 && n0 + c < a.N; c += P::kWarps) {  // a warp per output, four features a lane
                const float4 v = sum_of_peers(a0 + (c * kBF + lane * 4) * 4, a.split);
                float e[4] = {v.x, v.y, v.z, v.w};
                float* p = static_cast<float*>(a.dw) + (uint64_t)(n0 + c) * a.lddw + k;
                uint16_t* q = static_cast<uint16_t*>(a.dw) + (uint64_t)(n0 + c) * a.lddw + k;
                if (ADD) {
                    float old[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) old[j] = k + j >= a.K ? 0.0f : a.dtype == 0 ? p[j] : value(q[j]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[j] += old[j];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (k + j < a.K && a.dtype == 0) put(p + j, e[j]);
                    if (k + j < a.K && a.dtype != 0) put(q + j, e[j]);
                }
            }
        }
    }
    fence_before();
    // the others' products, arrivals and loads reach into this block
    if (group > 1) cluster_sync();
    else __syncthreads();
    if (warp == kIssuer) {
        if constexpr (CTAS == 2) tmem_free_pair(tmem, P::kCols);
        else tmem_free(tmem, P::kCols);
    }
}

// Estimated times in nanoseconds, fitted to 1 to 8192 tokens and layers of 512
// to 4096 (most within 10 %): what a launch and a tile's first and last steps
// take, a stage (64 tokens; widening X does not get shorter with the tile), the
// stores of a tile, and adding up the parts of a tile whose tokens are split.
// The rounds of tiles overlap their stores with the next round's products. At
// 4096 x 4096 tiles of 224 outputs fill 4 rounds of pairs where 256 fill 3.4.
struct Plan {
    uint32_t nt, split;
    int ctas;
    uint64_t ns;
};

inline uint64_t rounds_ns(uint64_t rounds, uint64_t stages_ns, uint64_t store_ns) {
    return (rounds - 1) * (stages_ns > store_ns ? stages_ns : store_ns) + stages_ns + store_ns;
}

Plan choose(uint32_t T, uint32_t N, uint32_t K, bool aligned, int sms, int pairs) {
    Plan best{32, 1, 1, ~0ull};
    const uint64_t stages = (T + kBT - 1) / kBT, shift = aligned ? 0 : 190;
    const uint64_t tk = (K + kBF - 1) / kBF, pk = (K + 2 * kBF - 1) / (2 * kBF);
    for (uint32_t nt = 32; nt <= 128; nt *= 2) {
        const uint64_t tiles = tk * ((N + nt - 1) / nt);
        for (uint32_t split = 1; split <= 8 && split <= stages; split *= 2) {
            // clusters of four and eight do not fill every SM
            if (split > 1 && tiles * split > (uint64_t)(split == 2 ? sms : split == 4 ? sms - 8 : sms - 32)) break;
            const uint64_t rounds = split > 1 ? 1 : (tiles + sms - 1) / sms, tb = (stages + split - 1) / split;
            const uint64_t ns = 3600 + rounds_ns(rounds, tb * (260 + nt / 2 + shift), 300 + 9 * nt) + (split > 1 ? 600 + 7 * nt : 0);
            if (ns < best.ns) best = {nt, split, 1, ns};
        }
    }
    for (uint32_t nt = 256; nt >= 160; nt -= 32) {
        const uint64_t rounds = (pk * ((N + nt - 1) / nt) + pairs - 1) / pairs;
        const uint64_t ns = 5200 + rounds_ns(rounds, stages * (200 + nt * 2 / 3 + shift), 300 + 9 * nt);
        if (ns < best.ns) best = {nt, 1, 2, ns};
    }
    return best;
}

template <bool ALIGNED, int CTAS>
cudaError_t launch(const Wgrad8Args& m, Args a, int sms, cudaStream_t s) {
    using P = Form<ALIGNED, CTAS>;
    CUtensorMap xmap;
    YMaps ymaps{};
    cudaError_t e = make_map(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, m.x, m.K, m.T, m.ldx, kBF, kBT);
    if (e != cudaSuccess) return e;
    if (ALIGNED) {
        e = make_map(&ymaps.m[0], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, m.dy, m.N, m.T, m.lddy * 2, 64, kBT);
        if (e != cudaSuccess) return e;
    } else {
        for (uint32_t r = 0; r < 8; ++r) {
            // row r rounded down to 16 bytes and every eighth row from there:
            // the same shift in all of them. A residue without rows (T < 8) gets
            // the first row's map and is read past its end, which gives zeros.
            const uint32_t row0 = r < m.T ? r : 0;
            const uintptr_t row = reinterpret_cast<uintptr_t>(m.dy) + (uint64_t)row0 * m.lddy * 2;
            const uint32_t shift = row % 16;
            e = make_map(&ymaps.m[r], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, reinterpret_cast<const void*>(row - shift),
                         m.N + shift / 2, (m.T - row0 + 7) / 8, m.lddy * 16, kHalfN + 8, kBT / 8, false);
            if (e != cudaSuccess) return e;
        }
    }
    a.tiles_k = (m.K + CTAS * kBF - 1) / (CTAS * kBF);
    const auto kernel = m.accumulate ? wgrad8_kernel<ALIGNED, CTAS, true> : wgrad8_kernel<ALIGNED, CTAS, false>;
    int groups = sms;
    if (CTAS == 2) e = max_pairs(reinterpret_cast<const void*>(kernel), P::kWarps * 32, P::kSmem, &groups);
    else e = allow_smem(reinterpret_cast<const void*>(kernel), P::kSmem);
    if (e != cudaSuccess) return e;
    a.tiles_n = (m.N + a.nt - 1) / a.nt;
    const uint64_t tiles = (uint64_t)a.tiles_k * a.tiles_n;
    const uint32_t size = CTAS == 2 ? 2 : a.split;
    const uint32_t grid = size * (uint32_t)(a.split > 1 || tiles < (uint64_t)groups ? tiles : groups);
    return launch_early(kernel, grid, P::kWarps * 32, P::kSmem, size > 1 ? size : 0, s, xmap, ymaps, a);
}

}  // namespace

cudaError_t launch_wgrad8(const Wgrad8Args& m, cudaStream_t s) {
    DeviceInfo di{};
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    Args a{};
    a.dy = static_cast<const uint16_t*>(m.dy);
    a.lddy = m.lddy;
    a.x = m.x;
    a.ldx = m.ldx;
    a.xs = m.xs;
    a.dw = m.dw;
    a.lddw = m.lddw;
    a.T = m.T;
    a.N = m.N;
    a.K = m.K;
    a.nblk = (m.K + kBF - 1) / kBF;
    a.dtype = m.dtype;
    e = tc::wait_fault_word(&a.faults);
    if (e != cudaSuccess) return e;
    const bool tma = reinterpret_cast<uintptr_t>(m.dy) % 16 == 0 && m.lddy % 8 == 0;
    int pairs = 0;
    using P = Form<true, 2>;
    e = tc::max_pairs(reinterpret_cast<const void*>(wgrad8_kernel<true, 2, false>), P::kWarps * 32, P::kSmem, &pairs);
    if (e != cudaSuccess) return e;
    const Plan plan = choose(m.T, m.N, m.K, tma, di.sms, pairs);
    a.nt = plan.nt;
    a.split = plan.split;
    if (plan.ctas == 2) return tma ? launch<true, 2>(m, a, di.sms, s) : launch<false, 2>(m, a, di.sms, s);
    return tma ? launch<true, 1>(m, a, di.sms, s) : launch<false, 1>(m, a, di.sms, s);
}

}  // namespace s2
