// Y[m][n] = sum_k X[m][k] * W[n][k] for two 4-bit packed matrices (MXFP4).
//
// The tensor cores multiply e2m1 codes 64 k at a time, scaled by a byte for each
// 32 of them, into one float32 accumulator in tensor memory. The scale bytes are
// stored in the order that tensor memory wants (512 bytes for 128 rows by 128
// columns: 32 lanes of four words), so they travel as the codes do: a tiled copy
// brings a stage's codes and scales to shared memory, and the warp that issues
// the products first issues copies of the scales from there to tensor memory.
// No thread touches an operand.
//
// A tile is 128 features (rows of W, the accumulator's lanes) by NT tokens (rows
// of X, its columns), as in the 8-bit product: neighbouring lanes store
// neighbouring elements of Y's rows.
//
// Measured in CUDA graphs: one token by 4096 x 4096 4.2 us (a launch, the
// pipeline's fill and 8.9 MB from L2); 24 tokens by 267735 x 1024 into float32
// 29.2 us, 5.9 TB/s of its 171 MB (0.88 of a copy's rate), 64 into bfloat16 29.3;
// 8192 x 4096 x 4096 44 us (6.2 PFLOP/s), 4096 x 4096 x 16384 87 us (6.4), bound by
// shared memory: for a product of 64 k an SM reads 10 KB of it and copies write 7.7
// KB, 139 clocks at 128 bytes a clock, where the tensor cores would take 101; 2048 x
// 267735 x 1024 into bfloat16 385 us, which its stores take (2 bytes of 548 million
// elements in rows that start on odd addresses, three sectors to a request).
#include "s2_internal.h"
#include "s2_launch.cuh"
#include "s2_product.cuh"
#include "s2_tc.cuh"

namespace s2 {
namespace {

using namespace tc;

constexpr int kBK = 128;                 // bytes of a row per stage
constexpr int kBKe = 2 * kBK;            // elements of K
constexpr int kBF = 128;                 // features per tile
constexpr int kWarps = 6;                // 0-3 store, 4 copies, 5 products
constexpr uint32_t kABytes = kBF * kBK;  // W part of a stage
constexpr uint32_t kSBytes = 1024;       // scales of 128 rows and a stage's K: two tiles of 512
constexpr uint32_t kSWords = kSBytes / 4;

// The tensor cores cut off what they add to a float32 sum, so a long sum drifts
// towards zero, by as much for each addition, of 64 k here. As in the 8-bit
// product a float32 result is taken in chunks of 128 additions that are added
// with rounding, and a bfloat16 result where there are more than 2048.
constexpr uint32_t kChunk = 32;
constexpr uint32_t kLong16 = 512;

struct Args {
    void* y;
    uint64_t ldy;
    uint32_t M, N, nblk;  // nblk: stages of K
    int dtype;
    uint32_t tiles_f, tiles_t;
    uint32_t nt;            // tokens per tile of the pair form, 128 or 192
    uint32_t tokens_inner;  // tiles of one feature range are neighbours in the order
    uint32_t split;         // blocks (one cluster) per tile, each with a part of K
    uint32_t* faults;
};

// Scales [32 lanes][four words] at a descriptor to four columns of tensor memory, for each quarter of its lanes.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (8ull << 16) | (8ull << 32) | (1ull << 46);  // groups of eight lanes: 128 bytes
}
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void scales_to_tmem_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// 4-bit operands with a scale byte for each row and 32 elements of K, 64 elements.
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, bool add) {
    asm volatile(
        "{.reg .pred p; setp.ne.u32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_mx4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, bool add) {
    asm volatile(
        "{.reg .pred p; setp.ne.u32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add)
        : "memory");
}
// D float32, A and B e2m1, both along K, UE8M0 scales, n columns, m lanes.
__device__ __forceinline__ uint32_t instruction(uint32_t m, uint32_t n) {
    return 1u << 7 | 1u << 10 | (n / 8) << 17 | 1u << 23 | (m / 128) << 27;
}
// The pair of scale bytes of a word (0: the first two, 2: the last two) that a product takes.
__device__ __forceinline__ uint32_t scale_pair(uint32_t i) { return i << 4 | i << 29; }

template <int NT, bool CHUNKS>
struct Shape {
    static constexpr uint32_t kBBytes = NT * kBK;
    static constexpr uint32_t kScaleAt = kABytes + kBBytes;
    static constexpr uint32_t kStage = kScaleAt + 2 * kSBytes;
    static constexpr int kStages = (int)(200 * 1024 / kStage) < 10 ? (int)(200 * 1024 / kStage) : 10;
    static constexpr int kAcc = 2;          // accumulators in tensor memory
    static constexpr int kScaleCols = 16;   // of a stage: two groups of 128 k, four columns of W and four of X each
    static constexpr uint32_t kScaleCol = kAcc * NT;
    static constexpr uint32_t kSumAt = kScaleCol + kStages * kScaleCols;
    static constexpr uint32_t kUsed = kSumAt + (CHUNKS ? NT : 0);
    static constexpr uint32_t kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
    static_assert(kUsed <= 512, "tensor memory");
    static_assert(kStage % 1024 == 0, "stages start on the swizzle's period");
    static_assert((size_t)NT * kBF * 4 <= (size_t)kStages * kStage, "a partial tile fits where the stages were");
};

template <int NT, bool CHUNKS>
__global__ void __launch_bounds__(kWarps * 32, 1)
    matmul4_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                   const __grid_constant__ CUtensorMap wsmap, const __grid_constant__ CUtensorMap xsmap, const Args a) {
    using S = Shape<NT, CHUNKS>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * S::kStages + 2 * S::kAcc + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t dead;

    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages;
    const uint32_t acc_full = empty + 8 * S::kStages, acc_empty = acc_full + 8 * S::kAcc, drain = acc_empty + 8 * S::kAcc;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            bar_init(full + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < S::kAcc; ++s) {
            bar_init(acc_full + 8 * s, 1);
            bar_init(acc_empty + 8 * s, 4);
        }
        bar_init(drain, 1);
        dead = 0;
        bar_fence_init();
    }
    if (warp == 5) tmem_alloc(smem_u32(&tmem_slot), S::kCols);
    if (threadIdx.x == 4 * 32) {
        tma_prefetch(&wmap);
        tma_prefetch(&xmap);
        tma_prefetch(&wsmap);
        tma_prefetch(&xsmap);
    }
    fence_before();
    __syncthreads();
    fence_after();
    stream_order();
    const uint32_t tmem = tmem_slot;
    const Wait wt{&dead, a.faults};

    const uint32_t rank = a.split > 1 ? cluster_rank() : 0;
    const uint32_t first = blockIdx.x / a.split, step = gridDim.x / a.split, tiles = a.tiles_f * a.tiles_t;
    const uint32_t kb0 = (uint32_t)((uint64_t)a.nblk * rank / a.split);
    const uint32_t kb1 = (uint32_t)((uint64_t)a.nblk * (rank + 1) / a.split);
    // (tiles of fewer than 128 tokens stand alone: a row of them begins at token 0)
    auto place = [&](uint32_t tile, uint32_t& f0, uint32_t& t0) {
        const uint32_t inner = a.tokens_inner ? a.tiles_t : a.tiles_f, o = tile / inner, i = tile - o * inner;
        f0 = (a.tokens_inner ? o : i) * kBF;
        t0 = (a.tokens_inner ? i : o) * NT;
    };

    if (warp == 4) {
        const bool leader = elect();
        Slot<S::kStages> s;
        uint32_t issued = 0;
        bool ok = true;
        for (uint32_t tile = first; ok && tile < tiles; tile += step) {
            uint32_t f0, t0;
            place(tile, f0, t0);
            for (uint32_t kb = kb0; kb < kb1; ++kb) {
                if (!(ok = bar_wait(empty + 8 * s.at, s.phase ^ 1, wt))) break;
                const uint32_t dst = base + s.at * S::kStage, f = full + 8 * s.at;
                if (leader) {
                    bar_expect(f, S::kStage);
                    tma_2d(dst, &wmap, f, (int)(kb * kBK), (int)f0);
                    tma_2d(dst + kABytes, &xmap, f, (int)(kb * kBK), (int)t0);
                    tma_2d(dst + S::kScaleAt, &wsmap, f, (int)(kb * kSWords), (int)(f0 / 128));
                    tma_2d(dst + S::kScaleAt + kSBytes, &xsmap, f, (int)(kb * kSWords), (int)(t0 / 128));
                }
                s.next();
                ++issued;
            }
        }
        // nothing of this block's may still be on its way when it ends
        if (dead)
            for (uint32_t j = issued > (uint32_t)S::kStages ? issued - S::kStages : 0; j < issued; ++j)
                bar_drain(full + 8 * (j % S::kStages), (j / S::kStages) & 1);
    } else if (warp == 5) {
        const bool leader = elect();  // the thread that issues the products also commits them
        const uint32_t idesc = instruction(kBF, NT);
        Slot<S::kStages> s;
        Slot<S::kAcc> acc;
        bool ok = true;
        for (uint32_t tile = first; ok && tile < tiles; tile += step) {
            for (uint32_t from = kb0, end; ok && from < kb1; from = end) {
                if (!(ok = bar_wait(acc_empty + 8 * acc.at, acc.phase ^ 1, wt))) break;
                fence_after();
                const uint32_t d = tmem + acc.at * NT;
                end = CHUNKS && kb1 - from > kChunk ? from + kChunk : kb1;
                for (uint32_t kb = from; kb < end; ++kb) {
                    if (!(ok = bar_wait(full + 8 * s.at, s.phase, wt))) break;
                    fence_after();
                    const uint32_t at = base + s.at * S::kStage;
                    const uint64_t ad = smem_desc(at, 16, 1024), bd = smem_desc(at + kABytes, 16, 1024);
                    const uint64_t wsd = scale_desc(at + S::kScaleAt), xsd = scale_desc(at + S::kScaleAt + kSBytes);
                    // a stage's scales have columns of their own, which are free again when its memory is
                    const uint32_t sf = tmem + S::kScaleCol + s.at * S::kScaleCols;
                    if (leader) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            scales_to_tmem(sf + 8 * g, wsd + 32 * g);  // 512 bytes on
                            scales_to_tmem(sf + 8 * g + 4, xsd + 32 * g);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)  // 32 bytes of K each
                            mma_mx4(d, ad + 2 * j, bd + 2 * j, idesc | scale_pair(j % 2 * 2), sf + j / 2 * 8, sf + j / 2 * 8 + 4,
                                    kb > from || j > 0);
                        mma_commit(empty + 8 * s.at);
                    }
                    s.next();
                }
                if (ok && leader) mma_commit(acc_full + 8 * acc.at);
                acc.next();
            }
        }
        if (dead && leader) {  // products in flight still read this block's memory
            mma_commit(drain);
            bar_drain(drain, 0);
        }
    } else {
        Slot<S::kAcc> acc;
        uint32_t kb = kb0;  // where the chunk begins
        const uint32_t mine = tmem + ((uint32_t)warp << 21);
        for (uint32_t tile = first; tile < tiles;) {
            if (!bar_wait(acc_full + 8 * acc.at, acc.phase, wt)) break;
            fence_after();
            uint32_t f0, t0;
            place(tile, f0, t0);
            const uint32_t f = f0 + warp * 32 + lane;
            const bool more = CHUNKS && kb1 - kb > kChunk;
#pragma unroll 1
            for (int c = 0; c < NT; c += 16) {
                uint32_t r[16];
                load_sums16(mine + acc.at * NT + c, mine + S::kSumAt + c, CHUNKS && kb > kb0, r);
                if (more) {
                    tmem_st16(mine + S::kSumAt + c, r);
                    wait_st();
                } else if (a.split > 1) {
                    // this block's part of the sums, where the stages were
                    float* part = reinterpret_cast<float*>(raw + (base - smem_u32(raw)));
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c + j) * kBF + warp * 32 + lane] = __uint_as_float(r[j]);
                } else if (f < a.N) {
                    store16(a, t0 + c, f, r);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(acc_empty + 8 * acc.at);
            acc.next();
            kb += kChunk;
            if (!more) {
                tile += step;
                kb = kb0;
            }
        }
    }

    __syncwarp();
    if (a.split > 1) {
        // One tile per cluster: every block adds the parts of its own columns
        // in the order of the ranks, so the sums do not depend on timing.
        cluster_sync();
        uint32_t f0, t0;
        place(first, f0, t0);
        const uint32_t c0 = NT * rank / a.split, c1 = NT * (rank + 1) / a.split, q = lane * 4;
        if (!dead) {
            for (uint32_t c = c0 + warp; c < c1 && t0 + c < a.M; c += kWarps) {  // a warp per token, four features a lane
                const float4 v = sum_of_peers(base + (c * kBF + q) * 4, a.split);
                const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (f0 + q + j < a.N) store(a, t0 + c, f0 + q + j, e[j]);
            }
        }
        cluster_sync();
    }
    fence_before();
    __syncthreads();
    if (warp == 5) tmem_free(tmem, S::kCols);
}

// Bytes of a row, rows of scale tiles, 32-bit words in such a row, bytes.
inline uint64_t row_bytes(uint32_t K) { return ((uint64_t)K + 1) / 2; }
inline uint64_t tiles128(uint32_t n) { return ((uint64_t)n + 127) / 128; }

// Map of a packed matrix's scales: two tiles of K by `tiles` of rows; what lies outside reads as 0, which is not NaN.
inline cudaError_t scale_map(CUtensorMap* map, const uint8_t* scales, uint32_t rows, uint32_t K, uint32_t tiles) {
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, scales, tiles128(K) * 128, tiles128(rows), tiles128(K) * 512, kSWords, tiles, false);
}

template <int NT, bool CHUNKS>
cudaError_t launch(const Matmul4Args& m, Args a, cudaStream_t s) {
    using S = Shape<NT, CHUNKS>;
    DeviceInfo di{};
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    CUtensorMap wmap, xmap, wsmap, xsmap;
    e = make_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, m.w, row_bytes(m.K), m.N, m.ldw, kBK, kBF);
    if (e != cudaSuccess) return e;
    e = make_map(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, m.x, row_bytes(m.K), m.M, m.ldx, kBK, NT);
    if (e != cudaSuccess) return e;
    e = scale_map(&wsmap, m.ws, m.N, m.K, 1);
    if (e != cudaSuccess) return e;
    e = scale_map(&xsmap, m.xs, m.M, m.K, 1);
    if (e != cudaSuccess) return e;
    a.tiles_f = (m.N + kBF - 1) / kBF;
    a.tiles_t = (m.M + NT - 1) / NT;
    const uint64_t tiles = (uint64_t)a.tiles_f * a.tiles_t;
    // the operand with the fewer bytes is the one that tiles in a row re-read
    a.tokens_inner = m.M <= m.N;
    auto kernel = matmul4_kernel<NT, CHUNKS>;
    e = allow_smem(reinterpret_cast<const void*>(kernel), S::kSmem);
    if (e != cudaSuccess) return e;
    const uint32_t grid = (uint32_t)(a.split > 1 ? tiles * a.split : tiles < (uint64_t)di.sms ? tiles : di.sms);
    return launch_early(kernel, grid, kWarps * 32, S::kSmem, a.split > 1 ? a.split : 0, s, wmap, xmap, wsmap, xsmap, a);
}

// ---- a pair of blocks per tile ---------------------------------------------------

// A tile is 256 features by 192 or 128 tokens on two SMs: each block holds 128 of
// the features, half of the tokens' codes, and the scales of its features and of
// all the tokens. Tiles begin on 64 tokens: the scales of 192 tokens lie in six of
// the eight columns that two rows of scale tiles fill, the first or the last six.
template <bool CHUNKS>
struct Pair {
    static constexpr int kMaxNT = CHUNKS ? 128 : 192;    // the sum of chunks takes as many columns again
    static constexpr uint32_t kHalf = kMaxNT / 2 * kBK;  // X part of a stage
    static constexpr uint32_t kRowTiles = CHUNKS ? 1 : 2;
    static constexpr uint32_t kScaleAt = kABytes + kHalf;
    static constexpr uint32_t kStage = kScaleAt + (1 + kRowTiles) * kSBytes;
    static constexpr int kStages = CHUNKS ? 7 : 5;
    static constexpr int kAcc = 2;
    static constexpr int kGroupCols = 4 + 4 * kRowTiles;  // columns of 128 k: of W, then of X
    static constexpr int kScaleCols = 2 * kGroupCols;
    static constexpr uint32_t kScaleCol = kAcc * kMaxNT;
    static constexpr uint32_t kSumAt = kScaleCol + kStages * kScaleCols;
    static constexpr uint32_t kCols = 512;
    static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
    static_assert(kSumAt + (CHUNKS ? kMaxNT : 0) <= kCols, "tensor memory");
    static_assert(kSmem <= 227 * 1024 - 1024, "shared memory");
    static_assert(kStage % 1024 == 0 && kHalf % 1024 == 0, "stages start on the swizzle's period");
};

template <bool CHUNKS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWarps * 32, 1)
    matmul4_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                        const __grid_constant__ CUtensorMap wsmap, const __grid_constant__ CUtensorMap xsmap, const Args a) {
    using S = Pair<CHUNKS>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * S::kStages + 2 * S::kAcc + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t dead;

    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    // full and acc_empty of the first block count both blocks
    const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages;
    const uint32_t acc_full = empty + 8 * S::kStages, acc_empty = acc_full + 8 * S::kAcc, drain = acc_empty + 8 * S::kAcc;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            bar_init(full + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < S::kAcc; ++s) {
            bar_init(acc_full + 8 * s, 1);
            bar_init(acc_empty + 8 * s, 8);
        }
        bar_init(drain, 1);
        dead = 0;
        bar_fence_init();
    }
    if (warp == 5) tmem_alloc_pair(smem_u32(&tmem_slot), S::kCols);
    fence_before();
    cluster_sync();
    fence_after();
    stream_order();
    const uint32_t tmem = tmem_slot;
    const Wait wt{&dead, a.faults};
    const uint32_t first = blockIdx.x / 2, step = gridDim.x / 2, tiles = a.tiles_f * a.tiles_t;
    auto place = [&](uint32_t tile, uint32_t& f0, uint32_t& t0) {
        const uint32_t inner = a.tokens_inner ? a.tiles_t : a.tiles_f, o = tile / inner, i = tile - o * inner;
        f0 = (a.tokens_inner ? o : i) * (2 * kBF) + rank * kBF;
        t0 = (a.tokens_inner ? i : o) * a.nt;
    };

    if (warp == 4) {
        const bool leader = elect();
        const uint32_t bytes = 2 * (kABytes + a.nt / 2 * kBK + (1 + S::kRowTiles) * kSBytes), full0 = in_first(full);
        Slot<S::kStages> s;
        uint32_t issued = 0;
        bool ok = true;
        for (uint32_t tile = first; ok && tile < tiles; tile += step) {
            uint32_t f0, t0;
            place(tile, f0, t0);
            const int x_row = (int)(t0 + rank * (a.nt / 2));
            for (uint32_t kb = 0; kb < a.nblk; ++kb) {
                if (!(ok = bar_wait(empty + 8 * s.at, s.phase ^ 1, wt))) break;
                const uint32_t dst = base + s.at * S::kStage, f = full0 + 8 * s.at;
                if (leader) {
                    if (rank == 0) bar_expect(full + 8 * s.at, bytes);
                    tma_2d_pair(dst, &wmap, f, (int)(kb * kBK), (int)f0);
                    tma_2d_pair(dst + kABytes, &xmap, f, (int)(kb * kBK), x_row);
                    tma_2d_pair(dst + S::kScaleAt, &wsmap, f, (int)(kb * kSWords), (int)(f0 / 128));
                    tma_2d_pair(dst + S::kScaleAt + kSBytes, &xsmap, f, (int)(kb * kSWords), (int)(t0 / 128));
                }
                s.next();
                ++issued;
            }
        }
        // nothing of the pair's may still be on its way when it ends
        if (dead && leader && rank == 0)
            for (uint32_t j = issued > (uint32_t)S::kStages ? issued - S::kStages : 0; j < issued; ++j)
                bar_drain(full + 8 * (j % S::kStages), (j / S::kStages) & 1);
    } else if (warp == 5) {
        if (rank == 0) {
            const bool leader = elect();  // the thread that issues the products also commits them
            const uint32_t idesc = instruction(2 * kBF, a.nt);
            Slot<S::kStages> s;
            Slot<S::kAcc> acc;
            bool ok = true;
            for (uint32_t tile = first; ok && tile < tiles; tile += step) {
                uint32_t f0, t0;
                place(tile, f0, t0);
                const uint32_t x_col = 4 + t0 % 128 / 32;  // where the tile's tokens begin
                for (uint32_t from = 0, end; ok && from < a.nblk; from = end) {
                    if (!(ok = bar_wait(acc_empty + 8 * acc.at, acc.phase ^ 1, wt))) break;
                    fence_after();
                    const uint32_t d = tmem + acc.at * S::kMaxNT;
                    end = CHUNKS && a.nblk - from > kChunk ? from + kChunk : a.nblk;
                    for (uint32_t kb = from; kb < end; ++kb) {
                        if (!(ok = bar_wait(full + 8 * s.at, s.phase, wt))) break;
                        fence_after();
                        const uint32_t at = base + s.at * S::kStage;
                        const uint64_t ad = smem_desc(at, 16, 1024), bd = smem_desc(at + kABytes, 16, 1024);
                        const uint64_t sd = scale_desc(at + S::kScaleAt);
                        const uint32_t sf = tmem + S::kScaleCol + s.at * S::kScaleCols;
                        if (leader) {
#pragma unroll
                            for (int g = 0; g < 2; ++g)
#pragma unroll
                                for (uint32_t q = 0; q < 1 + S::kRowTiles; ++q)  // W's, then X's rows of tiles
                                    scales_to_tmem_pair(sf + g * S::kGroupCols + 4 * q, sd + 64 * q + 32 * g);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma_mx4_pair(d, ad + 2 * j, bd + 2 * j, idesc | scale_pair(j % 2 * 2), sf + j / 2 * S::kGroupCols,
                                             sf + j / 2 * S::kGroupCols + x_col, kb > from || j > 0);
                            mma_commit_pair(empty + 8 * s.at);
                        }
                        s.next();
                    }
                    if (ok && leader) mma_commit_pair(acc_full + 8 * acc.at);
                    acc.next();
                }
            }
            if (dead && leader) {
                mma_commit_pair(drain);
                bar_drain(drain, 0);
            }
        }
    } else {
        Slot<S::kAcc> acc;
        uint32_t kb = 0;  // where the chunk begins
        const uint32_t mine = tmem + ((uint32_t)warp << 21);
        for (uint32_t tile = first; tile < tiles;) {
            if (!bar_wait(acc_full + 8 * acc.at, acc.phase, wt)) break;
            fence_after();
            uint32_t f0, t0;
            place(tile, f0, t0);
            const uint32_t f = f0 + warp * 32 + lane;
            const bool more = CHUNKS && a.nblk - kb > kChunk;
#pragma unroll 1
            for (uint32_t c = 0; c < a.nt; c += 16) {
                uint32_t r[16];
                load_sums16(mine + acc.at * S::kMaxNT + c, mine + S::kSumAt + c, CHUNKS && kb > 0, r);
                if (more) {
                    tmem_st16(mine + S::kSumAt + c, r);
                    wait_st();
                } else if (f < a.N) {
                    store16(a, t0 + c, f, r);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_first(acc_empty + 8 * acc.at);
            acc.next();
            kb += kChunk;
            if (!more) {
                tile += step;
                kb = 0;
            }
        }
    }

    __syncwarp();
    fence_before();
    cluster_sync();  // the other block's products, copies and arrivals reach into this one
    if (warp == 5) tmem_free_pair(tmem, S::kCols);
}

// Estimated times in nanoseconds, fitted to products of 1 to 8192 tokens by 512 to
// 267735 features and 512 to 16384 of K: what a launch and a tile's first and last
// steps take, a stage (256 of K), the stores of a tile, and adding up the parts of a
// tile that is split. The rounds of tiles overlap their stores with the next
// round's products. (One token by 4096 x 4096: whole 5.8 us, in two parts 4.8, in
// four 4.1. 256 x 4096 x 4096: single blocks 7.4, pairs of 128 tokens 6.6, of 192
// 9.0; 8192 x 4096 x 4096: 60.9, 55.2 and 44.3 us.)
struct Plan {
    int nt;  // tokens per tile
    int split;
    bool pair;
    uint64_t ns;
};

inline uint64_t rounds_ns(uint64_t rounds, uint64_t stages_ns, uint64_t store_ns) {
    return (rounds - 1) * (stages_ns > store_ns ? stages_ns : store_ns) + stages_ns + store_ns;
}

Plan choose(uint32_t M, uint32_t N, uint32_t nblk, int pair_nt, int sms, int pairs) {
    const uint64_t tf = ((uint64_t)N + kBF - 1) / kBF;
    const int nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    const uint64_t tiles = tf * (((uint64_t)M + nt - 1) / nt);
    Plan best{nt, 1, false, ~0ull};
    for (int split = 1; split <= 8 && (uint32_t)split <= nblk; split *= 2) {
        // clusters of four and eight do not fill every SM
        if (split > 1 && tiles * split > (uint64_t)(split == 2 ? sms : split == 4 ? sms - 8 : sms - 32)) break;
        const uint64_t rounds = split > 1 ? 1 : (tiles + sms - 1) / sms, kb = (nblk + split - 1) / split;
        const uint64_t ns = 2900 + rounds_ns(rounds, kb * (200 + nt * 7 / 10), 300 + 9 * nt) + (split > 1 ? 600 + 7 * nt : 0);
        if (ns < best.ns) best = {nt, split, false, ns};
    }
    if (M <= 64) return best;  // pairs' tiles are at least 128 tokens wide
    const uint64_t pf = ((uint64_t)N + 2 * kBF - 1) / (2 * kBF);
    for (int nt = pair_nt; nt >= 128; nt -= 64) {
        const uint64_t rounds = (pf * (((uint64_t)M + nt - 1) / nt) + pairs - 1) / pairs;
        const uint64_t ns = 2900 + rounds_ns(rounds, (uint64_t)nblk * (90 + nt * 7 / 8), 9 * nt);
        if (ns < best.ns) best = {nt, 1, true, ns};
    }
    return best;
}

template <bool CHUNKS>
cudaError_t launch_pair(const Matmul4Args& m, Args a, int pairs, cudaStream_t s) {
    using S = Pair<CHUNKS>;
    a.tiles_f = (m.N + 2 * kBF - 1) / (2 * kBF);
    a.tiles_t = (m.M + a.nt - 1) / a.nt;
    const uint64_t tiles = (uint64_t)a.tiles_f * a.tiles_t;
    a.tokens_inner = m.M <= m.N;
    CUtensorMap wmap, xmap, wsmap, xsmap;
    cudaError_t e = make_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, m.w, row_bytes(m.K), m.N, m.ldw, kBK, kBF);
    if (e != cudaSuccess) return e;
    e = make_map(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, m.x, row_bytes(m.K), m.M, m.ldx, kBK, a.nt / 2);
    if (e != cudaSuccess) return e;
    e = scale_map(&wsmap, m.ws, m.N, m.K, 1);
    if (e != cudaSuccess) return e;
    e = scale_map(&xsmap, m.xs, m.M, m.K, S::kRowTiles);
    if (e != cudaSuccess) return e;
    const uint32_t grid = 2 * (uint32_t)(tiles < (uint64_t)pairs ? tiles : pairs);
    return launch_early(matmul4_pair_kernel<CHUNKS>, grid, kWarps * 32, S::kSmem, 0, s, wmap, xmap, wsmap, xsmap, a);
}

template <bool CHUNKS>
cudaError_t plan_and_launch(const Matmul4Args& m, Args a, int sms, cudaStream_t s) {
    int pairs = 0;
    const cudaError_t e = max_pairs(reinterpret_cast<const void*>(matmul4_pair_kernel<CHUNKS>), kWarps * 32, Pair<CHUNKS>::kSmem, &pairs);
    if (e != cudaSuccess) return e;
    const Plan plan = choose(m.M, m.N, a.nblk, Pair<CHUNKS>::kMaxNT, sms, pairs);
    a.split = (uint32_t)plan.split;
    a.nt = (uint32_t)plan.nt;
    if (plan.pair) return launch_pair<CHUNKS>(m, a, pairs, s);
    switch (plan.nt) {
        case 16: return launch<16, CHUNKS>(m, a, s);
        case 32: return launch<32, CHUNKS>(m, a, s);
        case 64: return launch<64, CHUNKS>(m, a, s);
    }
    return launch<128, CHUNKS>(m, a, s);
}

}  // namespace

cudaError_t launch_matmul4(const Matmul4Args& m, cudaStream_t s) {
    Args a{};
    a.y = m.y;
    a.ldy = m.ldy;
    a.M = m.M;
    a.N = m.N;
    a.nblk = (uint32_t)(((uint64_t)m.K + kBKe - 1) / kBKe);
    a.dtype = m.dtype;
    cudaError_t e = wait_fault_word(&a.faults);
    if (e != cudaSuccess) return e;
    DeviceInfo di{};
    e = device_info(&di);
    if (e != cudaSuccess) return e;
    if (a.nblk > (m.dtype == 0 ? kChunk : kLong16)) return plan_and_launch<true>(m, a, di.sms, s);
    return plan_and_launch<false>(m, a, di.sms, s);
}

}  // namespace s2
