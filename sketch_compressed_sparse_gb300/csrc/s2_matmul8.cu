// Y[m][n] = sum_k X[m][k] * W[n][k] for two 8-bit packed matrices.
//
// The scales are powers of two, one byte each, which is what the tensor cores'
// block scaling takes: every product of 32 k is scaled by both bytes and added
// to one float32 accumulator in tensor memory, so a tile needs no pass over
// its sums between the blocks of K. The hardware takes a byte for each 32
// elements; a block of 128 gives the same byte to four products.
//
// A tile is 128 features (rows of W, the accumulator's lanes) by NT tokens
// (rows of X, its columns): neighbouring lanes hold neighbouring features, so
// stores to Y run along its rows whatever its alignment, and few tokens cost a
// small NT instead of an idle part of the tile.
//
// Measured: one token by 4096 x 4096 5.1 us in a CUDA graph (a launch, the
// pipeline's fill and 16.8 MB that come from L2); 24 tokens by 267735 x 1024
// into float32 50.0 us, 0.88 of a copy's rate for its 300 MB; 500 x 2000 x 1024
// 4.8 us; 8192 x 4096 x 4096 95 us in a long loop (2.9 PFLOP/s, power-capped)
// and 80 us for ten in a row (3.4); 2048 x 267735 x 1024 into bfloat16 540 us.
#include "s2_internal.h"
#include "s2_launch.cuh"
#include "s2_product.cuh"
#include "s2_tc.cuh"

namespace s2 {
namespace {

using namespace tc;

constexpr int kBK = 128;                 // bytes (= elements) of K per stage
constexpr int kBF = 128;                 // features per tile
constexpr int kGroup = 4;                // K blocks whose scale bytes share a 32-bit word
constexpr int kWarps = 10;               // 0-3 store, 4-7 scales, 8 copies, 9 products
constexpr uint32_t kABytes = kBF * kBK;  // W part of a stage

// The tensor cores cut off what they add to a float32 sum, so a long sum drifts
// towards zero. Normal inputs, relative error of one sum: 2.2e-7 at K = 4096,
// 1.2e-6 at 16384, 7.7e-6 at 65536, 1.9e-5 at 131072 (a float32 product of the
// unpacked values: 8e-8, 1.9e-7, 4.9e-7, 7.9e-7); twice that where a few
// channels are far larger. A float32 result is therefore taken in chunks of 32
// blocks of K that are added with rounding: 2.2e-7 at 16384, 2.3e-7 at 65536 (the
// additions' own roundings grow with the root of their number: 3.1e-7 at K = 2^22,
// in eight parts). The sum of chunks stays in tensor memory beside the two
// accumulators. That leaves a pair 160 tokens a tile where it has 224:
// 2048 x 1024 x 267735 505 -> 513 us, 8192 x 4096 x 16384 336 -> 369 us. Adding
// to Y in global memory kept the 224 and took 592 and 367.
constexpr uint32_t kChunk = 32;
// A bfloat16 result is rounded by up to 2^-8 of itself, 1.7e-3 in the mean square.
// Up to this many blocks of K it is taken in one chunk, which loses 7.7e-6 to
// 1.6e-5, a 100th of that, and keeps the 224 tokens (8192 x 4096 x 8192 150 us, in
// chunks 180; 2048 x 8192 x 28672 352 and 426). Beyond, the loss would go on growing
// with K, always towards zero (4e-5 at 267735), and chunks are taken: 2048 x 4096 x
// 66048 367 -> 374 us, 8192 x 4096 x 66048 1.28 -> 1.55 ms.
constexpr uint32_t kLong16 = 512;
static_assert(kChunk % kGroup == 0, "chunks end between two scale words");

struct Args {
    const uint8_t *xs, *ws;
    void* y;
    uint64_t ldy;
    uint32_t M, N, nblk, w_shift;
    int dtype;
    uint32_t tiles_f, tiles_t;
    uint32_t nt;            // tokens per tile of the pair form, a multiple of 32
    uint32_t tokens_inner;  // tiles of one feature range are neighbours in the order
    uint32_t split;         // blocks (one cluster) per tile, each with a part of K
    uint32_t* faults;
};

template <int NT, bool CHUNKS>
struct Shape {
    static constexpr uint32_t kStage = kABytes + NT * kBK;
    static constexpr int kStages = (int)(200 * 1024 / kStage) < 10 ? (int)(200 * 1024 / kStage) : 10;
    static constexpr int kAcc = 2;                          // accumulators in tensor memory
    static constexpr int kScaleB = (NT + 127) / 128 * 4;    // columns of X's scales, in fours
    static constexpr int kScaleCols = 4 + kScaleB;          // columns of one group's scales
    static constexpr int kRing = 2;                         // groups of scales in tensor memory
    static constexpr uint32_t kSumAt = kAcc * NT + kRing * kScaleCols;
    static constexpr uint32_t kUsed = kSumAt + (CHUNKS ? NT : 0);
    static constexpr uint32_t kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
    static_assert(kUsed <= 512, "tensor memory");
    static_assert((size_t)NT * kBF * 4 <= (size_t)kStages * kStage, "a partial tile fits where the stages were");
};

// The scale bytes of K blocks kb..kb+3 of one row as a word; blocks past the
// end repeat 1.0, which no product uses. Words: rows of bytes start on four
// bytes and their number is a multiple of four.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* s, uint32_t kb, uint32_t nblk, bool words) {
    if (words) return *reinterpret_cast<const uint32_t*>(s + kb);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) w |= (kb + i < nblk ? (uint32_t)s[kb + i] : 127u) << (8 * i);
    return w;
}
__device__ __forceinline__ bool in_words(const uint8_t* s, uint32_t nblk) {
    return nblk % kGroup == 0 && reinterpret_cast<uintptr_t>(s) % kGroup == 0;
}

template <int NT, bool CHUNKS>
__global__ void __launch_bounds__(kWarps * 32, 1)
    matmul8_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, const Args a) {
    using S = Shape<NT, CHUNKS>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * S::kStages + 2 * S::kRing + 2 * S::kAcc + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t dead;

    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S::kStages + s); };
    auto sf_full = [&](int s) { return bar0 + 8u * (2 * S::kStages + s); };
    auto sf_empty = [&](int s) { return bar0 + 8u * (2 * S::kStages + S::kRing + s); };
    auto acc_full = [&](int s) { return bar0 + 8u * (2 * S::kStages + 2 * S::kRing + s); };
    auto acc_empty = [&](int s) { return bar0 + 8u * (2 * S::kStages + 2 * S::kRing + S::kAcc + s); };
    const uint32_t drain = bar0 + 8u * (2 * S::kStages + 2 * S::kRing + 2 * S::kAcc);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        for (int s = 0; s < S::kRing; ++s) {
            bar_init(sf_full(s), 4);
            bar_init(sf_empty(s), 1);
        }
        for (int s = 0; s < S::kAcc; ++s) {
            bar_init(acc_full(s), 1);
            bar_init(acc_empty(s), 4);
        }
        bar_init(drain, 1);
        dead = 0;
        bar_fence_init();
    }
    if (warp == 9) tmem_alloc(smem_u32(&tmem_slot), S::kCols);
    if (threadIdx.x == 8 * 32) {
        tma_prefetch(&wmap);
        tma_prefetch(&xmap);
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
    auto place = [&](uint32_t tile, uint32_t& f0, uint32_t& t0) {
        const uint32_t inner = a.tokens_inner ? a.tiles_t : a.tiles_f, o = tile / inner, i = tile - o * inner;
        f0 = (a.tokens_inner ? o : i) * kBF;
        t0 = (a.tokens_inner ? i : o) * NT;
    };

    if (warp == 8) {
        {
            const bool leader = elect();
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t tile = first; ok && tile < tiles; tile += step) {
                uint32_t f0, t0;
                place(tile, f0, t0);
                for (uint32_t kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % S::kStages;
                    if (!(ok = bar_wait(empty(s), ((it / S::kStages) & 1) ^ 1, wt))) break;
                    const uint32_t dst = base + s * S::kStage;
                    if (leader) {
                        bar_expect(full(s), S::kStage);
                        tma_2d(dst, &wmap, full(s), (int)(kb * kBK), (int)f0);
                        tma_2d(dst + kABytes, &xmap, full(s), (int)(kb * kBK), (int)t0);
                    }
                }
            }
            // nothing of this block's may still be on its way when it ends
            if (dead)
                for (uint32_t j = it > (uint32_t)S::kStages ? it - S::kStages : 0; j < it; ++j)
                    bar_drain(full(j % S::kStages), (j / S::kStages) & 1);
        }
    } else if (warp == 9) {
        {
            const bool leader = elect();  // the thread that issues the products also commits them
            // D float32, A and B e4m3, both along K, UE8M0 scales, N = NT, M = 128
            const uint32_t idesc = (uint32_t)(NT / 8) << 17 | 1u << 23 | (uint32_t)(kBF / 16) << 24;
            uint32_t it = 0, grp = 0, n = 0;
            bool ok = true;
            for (uint32_t tile = first; ok && tile < tiles; tile += step) {
                for (uint32_t from = kb0, end; ok && from < kb1; from = end, ++n) {
                    const int buf = n % S::kAcc;
                    if (!(ok = bar_wait(acc_empty(buf), ((n / S::kAcc) & 1) ^ 1, wt))) break;
                    fence_after();
                    const uint32_t d = tmem + buf * NT;
                    end = CHUNKS && kb1 - from > kChunk ? from + kChunk : kb1;
                    for (uint32_t kb = from; kb < end; ++kb, ++it) {
                        const uint32_t i = (kb - from) % kGroup;
                        const uint32_t sf = tmem + S::kAcc * NT + (grp % S::kRing) * S::kScaleCols;
                        if (i == 0 && !(ok = bar_wait(sf_full(grp % S::kRing), (grp / S::kRing) & 1, wt))) break;
                        const int s = it % S::kStages;
                        if (!(ok = bar_wait(full(s), (it / S::kStages) & 1, wt))) break;
                        fence_after();
                        const uint64_t ad = smem_desc(base + s * S::kStage, 16, 1024);
                        const uint64_t bd = smem_desc(base + s * S::kStage + kABytes, 16, 1024);
                        const uint32_t id = idesc | i << 4 | i << 29;
                        const bool last = i == kGroup - 1 || kb + 1 == end;
                        if (leader) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)  // 32 bytes of K each
                                mma_mx8(d, ad + 2 * j, bd + 2 * j, id, sf, sf + 4, kb > from || j > 0);
                            mma_commit(empty(s));
                            if (last) mma_commit(sf_empty(grp % S::kRing));
                        }
                        if (last) ++grp;
                    }
                    if (ok && leader) mma_commit(acc_full(buf));
                }
            }
            if (dead && leader) {  // products in flight still read this block's memory
                mma_commit(drain);
                bar_drain(drain, 0);
            }
        }
    } else if (warp >= 4) {
        // Each of the four warps writes the same words to its own 32 lanes:
        // word c of lane l holds the bytes of row 32c + l.
        uint32_t grp = 0;
        bool ok = true;
        const uint32_t quarter = (uint32_t)(warp % 4) << 21;  // lane 32 * (warp % 4)
        // (a block's part of K may begin between two words)
        const bool w_words = in_words(a.ws, a.nblk) && kb0 % kGroup == 0, x_words = in_words(a.xs, a.nblk) && kb0 % kGroup == 0;
        for (uint32_t tile = first; ok && tile < tiles; tile += step) {
            uint32_t f0, t0;
            place(tile, f0, t0);
            for (uint32_t kb = kb0; kb < kb1; kb += kGroup, ++grp) {
                uint32_t wa[4], wb[S::kScaleB];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t f = f0 + 32 * c + lane;
                    wa[c] = f < a.N ? scale_word(a.ws + (uint64_t)(f >> a.w_shift) * a.nblk, kb, a.nblk, w_words) : 0x7f7f7f7fu;
                }
#pragma unroll
                for (int c = 0; c < S::kScaleB; ++c) {
                    const uint32_t t = t0 + 32 * c + lane;
                    wb[c] = 32 * c < NT && t < a.M ? scale_word(a.xs + (uint64_t)t * a.nblk, kb, a.nblk, x_words) : 0x7f7f7f7fu;
                }
                if (!(ok = bar_wait(sf_empty(grp % S::kRing), ((grp / S::kRing) & 1) ^ 1, wt))) break;
                fence_after();
                const uint32_t sf = tmem + quarter + S::kAcc * NT + (grp % S::kRing) * S::kScaleCols;
                tmem_st4(sf, wa[0], wa[1], wa[2], wa[3]);
#pragma unroll
                for (int c = 0; c < S::kScaleB; c += 4) tmem_st4(sf + 4 + c, wb[c], wb[c + 1], wb[c + 2], wb[c + 3]);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(sf_full(grp % S::kRing));
            }
        }
    } else {
        uint32_t n = 0, kb = kb0;  // kb: where the chunk begins
        const uint32_t mine = tmem + ((uint32_t)warp << 21);
        for (uint32_t tile = first; tile < tiles; ++n) {
            const int buf = n % S::kAcc;
            if (!bar_wait(acc_full(buf), (n / S::kAcc) & 1, wt)) break;
            fence_after();
            uint32_t f0, t0;
            place(tile, f0, t0);
            const uint32_t f = f0 + warp * 32 + lane;
            const bool more = CHUNKS && kb1 - kb > kChunk;
#pragma unroll 1
            for (int c = 0; c < NT; c += 16) {
                uint32_t r[16];
                load_sums16(mine + buf * NT + c, mine + S::kSumAt + c, CHUNKS && kb > kb0, r);
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
            if (lane == 0) bar_arrive(acc_empty(buf));
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
    if (warp == 9) tmem_free(tmem, S::kCols);
}

template <int NT, bool CHUNKS>
cudaError_t launch(const Matmul8Args& m, Args a, cudaStream_t s) {
    using S = Shape<NT, CHUNKS>;
    DeviceInfo di{};
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    CUtensorMap wmap, xmap;
    e = make_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, m.w, m.K, m.N, m.ldw, kBK, kBF);
    if (e != cudaSuccess) return e;
    e = make_map(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, m.x, m.K, m.M, m.ldx, kBK, NT);
    if (e != cudaSuccess) return e;
    a.tiles_f = (m.N + kBF - 1) / kBF;
    a.tiles_t = (m.M + NT - 1) / NT;
    const uint64_t tiles = (uint64_t)a.tiles_f * a.tiles_t;
    // the operand with the fewer bytes is the one that tiles in a row re-read
    a.tokens_inner = m.M <= m.N;
    auto kernel = matmul8_kernel<NT, CHUNKS>;
    e = allow_smem(reinterpret_cast<const void*>(kernel), S::kSmem);
    if (e != cudaSuccess) return e;
    const uint32_t grid = (uint32_t)(a.split > 1 ? tiles * a.split : tiles < (uint64_t)di.sms ? tiles : di.sms);
    return launch_early(kernel, grid, kWarps * 32, S::kSmem, a.split > 1 ? a.split : 0, s, wmap, xmap, a);
}

// ---- a pair of blocks per tile ---------------------------------------------------

// A tile is 256 features by up to 224 tokens on two SMs. Each block holds 128
// of the features and half of the tokens' codes; the pair's product reads both,
// so a block fetches 30 KB per 128 of K where a block by itself would fetch
// 44 KB for the same rate (8192 x 4096 x 4096: 134 us with single blocks, 98 with
// pairs). Two accumulators of 224 columns leave 64 columns of tensor memory for
// the scales (256 would leave none).
//
// A stage of 128 of K takes 550 to 610 clocks for 448 of products (tensor pipe
// active 0.80 of the time). It did not get shorter with a copying warp for each
// operand, with scale words fetched a group ahead, with twice the storing
// warps, nor with clusters of two pairs that share the tokens' copies (23 KB a
// block and stage). With K = 1024 the stores bind: 2048 x 267735 takes, ten in a
// row, 453 us into bfloat16 and 533 us into twice the bytes in as many requests,
// 371 us without stores (540 into bfloat16 in a long loop, at a lower clock); at
// K = 128 the stores alone take 393. Turning bfloat16 through
// shared memory for longer requests, or for whole 32-byte sectors where rows
// start on odd addresses, took more time than it saved.
template <bool CHUNKS>
struct Pair {
    static constexpr int kMaxNT = CHUNKS ? 160 : 224;    // the sum of chunks takes as many columns again
    static constexpr uint32_t kHalf = kMaxNT / 2 * kBK;  // X part of a stage
    static constexpr uint32_t kStage = kABytes + kHalf;
    static constexpr int kStages = CHUNKS ? 8 : 7;
    static constexpr int kAcc = 2;
    static constexpr int kScaleCols = 12;  // 4 of W, 8 of X
    static constexpr int kRing = CHUNKS ? 2 : 4;
    static constexpr uint32_t kSumAt = kAcc * kMaxNT;
    static constexpr uint32_t kScaleAt = kSumAt + (CHUNKS ? kMaxNT : 0);
    static constexpr uint32_t kCols = 512;
    static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
    static_assert(kScaleAt + kRing * kScaleCols <= kCols, "tensor memory");
    static_assert(kSmem <= 227 * 1024 - 1024, "shared memory");
    static_assert(kHalf % 1024 == 0, "stages start on the swizzle's period");
};

template <bool CHUNKS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWarps * 32, 1)
    matmul8_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, const Args a) {
    using S = Pair<CHUNKS>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * S::kStages + 2 * S::kRing + 2 * S::kAcc + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t dead;

    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    // full, sf_full and acc_empty of the first block count both blocks
    const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages;
    const uint32_t sf_full = empty + 8 * S::kStages, sf_empty = sf_full + 8 * S::kRing;
    const uint32_t acc_full = sf_empty + 8 * S::kRing, acc_empty = acc_full + 8 * S::kAcc, drain = acc_empty + 8 * S::kAcc;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            bar_init(full + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < S::kRing; ++s) {
            bar_init(sf_full + 8 * s, 8);
            bar_init(sf_empty + 8 * s, 1);
        }
        for (int s = 0; s < S::kAcc; ++s) {
            bar_init(acc_full + 8 * s, 1);
            bar_init(acc_empty + 8 * s, 8);
        }
        bar_init(drain, 1);
        dead = 0;
        bar_fence_init();
    }
    if (warp == 9) tmem_alloc_pair(smem_u32(&tmem_slot), S::kCols);
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

    if (warp == 8) {
        const bool leader = elect();
        const uint32_t bytes = 2 * (kABytes + a.nt / 2 * kBK), full0 = in_first(full);
        Slot<S::kStages> s;
        uint32_t issued = 0;
        bool ok = true;
        for (uint32_t tile = first; ok && tile < tiles; tile += step) {
            uint32_t f0, t0;
            place(tile, f0, t0);
            const int x_row = (int)(t0 + rank * (a.nt / 2));
            for (uint32_t kb = 0; kb < a.nblk; ++kb) {
                if (!(ok = bar_wait(empty + 8 * s.at, s.phase ^ 1, wt))) break;
                const uint32_t dst = base + s.at * S::kStage;
                if (leader) {
                    if (rank == 0) bar_expect(full + 8 * s.at, bytes);
                    tma_2d_pair(dst, &wmap, full0 + 8 * s.at, (int)(kb * kBK), (int)f0);
                    tma_2d_pair(dst + kABytes, &xmap, full0 + 8 * s.at, (int)(kb * kBK), x_row);
                }
                s.next();
                ++issued;
            }
        }
        // nothing of the pair's may still be on its way when it ends
        if (dead && leader && rank == 0)
            for (uint32_t j = issued > (uint32_t)S::kStages ? issued - S::kStages : 0; j < issued; ++j)
                bar_drain(full + 8 * (j % S::kStages), (j / S::kStages) & 1);
    } else if (warp == 9) {
        if (rank == 0) {
            const bool leader = elect();  // the thread that issues the products also commits them
            // D float32, A and B e4m3, both along K, UE8M0 scales, N = nt, M = 256
            const uint32_t idesc = (a.nt / 8) << 17 | 1u << 23 | (uint32_t)(2 * kBF / 16) << 24;
            Slot<S::kStages> s;
            Slot<S::kRing> g;
            Slot<S::kAcc> acc;
            bool ok = true;
            for (uint32_t tile = first; ok && tile < tiles; tile += step) {
                for (uint32_t from = 0, end; ok && from < a.nblk; from = end) {
                    if (!(ok = bar_wait(acc_empty + 8 * acc.at, acc.phase ^ 1, wt))) break;
                    fence_after();
                    const uint32_t d = tmem + acc.at * S::kMaxNT;
                    end = CHUNKS && a.nblk - from > kChunk ? from + kChunk : a.nblk;
                    for (uint32_t kb = from; kb < end; ++kb) {
                        const uint32_t i = kb % kGroup;
                        if (i == 0 && !(ok = bar_wait(sf_full + 8 * g.at, g.phase, wt))) break;
                        if (!(ok = bar_wait(full + 8 * s.at, s.phase, wt))) break;
                        fence_after();
                        const uint64_t ad = smem_desc(base + s.at * S::kStage, 16, 1024);
                        const uint64_t bd = smem_desc(base + s.at * S::kStage + kABytes, 16, 1024);
                        const uint32_t id = idesc | i << 4 | i << 29, sf = tmem + S::kScaleAt + g.at * S::kScaleCols;
                        const bool last = i == kGroup - 1 || kb + 1 == end;
                        if (leader) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma_mx8_pair(d, ad + 2 * j, bd + 2 * j, id, sf, sf + 4, kb > from || j > 0);
                            mma_commit_pair(empty + 8 * s.at);
                            if (last) mma_commit_pair(sf_empty + 8 * g.at);
                        }
                        if (last) g.next();
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
    } else if (warp >= 4) {
        // As above; each block holds the scales of its own features and of all the tile's tokens.
        Slot<S::kRing> g;
        bool ok = true;
        const uint32_t quarter = (uint32_t)(warp % 4) << 21;
        const bool w_words = in_words(a.ws, a.nblk), x_words = in_words(a.xs, a.nblk);
        for (uint32_t tile = first; ok && tile < tiles; tile += step) {
            uint32_t f0, t0;
            place(tile, f0, t0);
            for (uint32_t kb = 0; kb < a.nblk; kb += kGroup) {
                uint32_t wa[4], wb[8];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t f = f0 + 32 * c + lane;
                    wa[c] = f < a.N ? scale_word(a.ws + (uint64_t)(f >> a.w_shift) * a.nblk, kb, a.nblk, w_words) : 0x7f7f7f7fu;
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint32_t t = t0 + 32 * c + lane;
                    wb[c] = 32 * c < a.nt && t < a.M ? scale_word(a.xs + (uint64_t)t * a.nblk, kb, a.nblk, x_words) : 0x7f7f7f7fu;
                }
                if (!(ok = bar_wait(sf_empty + 8 * g.at, g.phase ^ 1, wt))) break;
                fence_after();
                const uint32_t sf = tmem + quarter + S::kScaleAt + g.at * S::kScaleCols;
                tmem_st4(sf, wa[0], wa[1], wa[2], wa[3]);
                tmem_st4(sf + 4, wb[0], wb[1], wb[2], wb[3]);
                tmem_st4(sf + 8, wb[4], wb[5], wb[6], wb[7]);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_first(sf_full + 8 * g.at);
                g.next();
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
    if (warp == 9) tmem_free_pair(tmem, S::kCols);
}

// Estimated times in nanoseconds, fitted to products of 1 to 2048 tokens by 500
// to 4096 features and 512 to 4096 of K (most within 10 %): what a launch and a
// tile's first and last steps take, a stage (128 of K), the stores of a tile,
// and adding up the parts of a tile that is split. The rounds of tiles overlap
// their stores with the next round's products.
struct Plan {
    int nt;  // tokens per tile
    int split;
    bool pair;
    uint64_t ns;
};

inline uint64_t rounds_ns(uint64_t rounds, uint64_t stages_ns, uint64_t store_ns) {
    return (rounds - 1) * (stages_ns > store_ns ? stages_ns : store_ns) + stages_ns + store_ns;
}

Plan choose(uint32_t M, uint32_t N, uint32_t nblk, bool chunks, int sms, int pairs) {
    Plan best{16, 1, false, ~0ull};
    const uint64_t tf = (N + kBF - 1) / kBF;
    for (int nt : {16, 32, 64, 128, 224}) {
        if ((nt > 16 && (uint32_t)nt >= 2 * M) || (chunks && nt > 128)) break;
        const uint64_t tiles = tf * ((M + nt - 1) / nt);
        for (int split = 1; split <= 8 && (uint32_t)split <= nblk; split *= 2) {
            // clusters of four and eight do not fill every SM
            if (split > 1 && tiles * split > (uint64_t)(split == 2 ? sms : split == 4 ? sms - 8 : sms - 32)) break;
            const uint64_t rounds = split > 1 ? 1 : (tiles + sms - 1) / sms, kb = (nblk + split - 1) / split;
            const uint64_t ns = 2900 + rounds_ns(rounds, kb * (200 + nt * 7 / 10), 300 + 9 * nt) + (split > 1 ? 600 + 7 * nt : 0);
            if (ns < best.ns) best = {nt, split, false, ns};
        }
    }
    if (M <= 64) return best;  // pairs' tiles are at least 160 tokens wide
    const uint64_t pf = (N + 2 * kBF - 1) / (2 * kBF);
    for (int nt = chunks ? Pair<true>::kMaxNT : Pair<false>::kMaxNT; nt >= 160; nt -= 32) {
        const uint64_t rounds = (pf * ((M + nt - 1) / nt) + pairs - 1) / pairs;
        const uint64_t ns = 4500 + rounds_ns(rounds, (uint64_t)nblk * (60 + nt), 9 * nt);
        if (ns < best.ns) best = {nt, 1, true, ns};
    }
    return best;
}

template <bool CHUNKS>
cudaError_t launch_pair(const Matmul8Args& m, Args a, int pairs, cudaStream_t s) {
    a.tiles_f = (m.N + 2 * kBF - 1) / (2 * kBF);
    a.tiles_t = (m.M + a.nt - 1) / a.nt;
    const uint64_t tiles = (uint64_t)a.tiles_f * a.tiles_t;
    a.tokens_inner = m.M <= m.N;
    CUtensorMap wmap, xmap;
    cudaError_t e = make_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, m.w, m.K, m.N, m.ldw, kBK, kBF);
    if (e != cudaSuccess) return e;
    e = make_map(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, m.x, m.K, m.M, m.ldx, kBK, a.nt / 2);
    if (e != cudaSuccess) return e;
    const uint32_t grid = 2 * (uint32_t)(tiles < (uint64_t)pairs ? tiles : pairs);
    return launch_early(matmul8_pair_kernel<CHUNKS>, grid, kWarps * 32, Pair<CHUNKS>::kSmem, 0, s, wmap, xmap, a);
}

template <bool CHUNKS>
cudaError_t plan_and_launch(const Matmul8Args& m, Args a, int sms, cudaStream_t s) {
    int pairs = 0;
    const cudaError_t e = max_pairs(reinterpret_cast<const void*>(matmul8_pair_kernel<CHUNKS>), kWarps * 32, Pair<CHUNKS>::kSmem, &pairs);
    if (e != cudaSuccess) return e;
    const Plan plan = choose(m.M, m.N, a.nblk, CHUNKS, sms, pairs);
    a.split = (uint32_t)plan.split;
    a.nt = (uint32_t)plan.nt;
    if (plan.pair) return launch_pair<CHUNKS>(m, a, pairs, s);
    switch (plan.nt) {
        case 16: return launch<16, CHUNKS>(m, a, s);
        case 32: return launch<32, CHUNKS>(m, a, s);
        case 64: return launch<64, CHUNKS>(m, a, s);
        case 128: return launch<128, CHUNKS>(m, a, s);
    }
    if constexpr (CHUNKS) return cudaErrorInvalidValue;  // (not chosen: no room for the sum of chunks)
    else return launch<224, false>(m, a, s);
}

}  // namespace

cudaError_t launch_matmul8(const Matmul8Args& m, cudaStream_t s) {
    Args a{};
    a.xs = m.xs;
    a.ws = m.ws;
    a.y = m.y;
    a.ldy = m.ldy;
    a.M = m.M;
    a.N = m.N;
    a.nblk = (m.K + kBK - 1) / kBK;
    a.w_shift = m.w_shift;
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
