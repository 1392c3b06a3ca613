// dW[n][k] (+)= sum_t dY[t][n] * X[t][k] with dY in bfloat16 and X an 8-bit
// packed activation.
//
// A code times its power-of-two scale has four significant bits, so it is
// exact in bfloat16: the 8-bit rows are widened on the way into shared memory
// and the product is a bfloat16 one on the tensor cores with float32 sums, at
// half the activation's bytes. Both operands are read as they lie, rows along
// the outputs' axes (tokens are the summed axis), so nothing is transposed.
//
// A tile is 128 features of X (the accumulator's lanes) by NT outputs
// (columns): neighbouring lanes hold neighbouring k, so stores run along dW's
// rows whatever its alignment. A block of 128 features shares one scale per
// token. dY comes by tiled copies where its rows start on 16 bytes; else
// (an odd vocabulary) eight warps fetch it, each the rows t = w mod 8, whose
// misalignment is the same for the whole call, so that a row is shifted into
// place by a constant amount.
#include "s2_internal.h"
#include "s2_tc.cuh"

namespace s2 {
namespace {

using namespace tc;

constexpr int kBT = 64;                    // tokens per stage
constexpr int kBF = 128;                   // features per tile
constexpr uint32_t kGroupBytes = kBT * 128;  // 64 outputs or features by kBT tokens
constexpr uint32_t kABytes = 2 * kGroupBytes;
constexpr int kLoaders = 8;                // warps that fetch a misaligned dY

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
    int dtype, accumulate;
    uint32_t* faults;
};

template <int NT, bool TMA>
struct Shape {
    static constexpr uint32_t kStage = kABytes + NT / 64 * kGroupBytes;
    static constexpr int kStages = (int)(200 * 1024 / kStage) < 8 ? (int)(200 * 1024 / kStage) : 8;
    static constexpr int kAcc = 2;
    static constexpr uint32_t kCols = kAcc * NT;  // a power of two
    static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
    static constexpr int kWarps = TMA ? 10 : 10 + kLoaders;
    static_assert((size_t)NT * kBF * 4 <= (size_t)kStages * kStage, "a partial tile fits where the stages were");
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four codes times 2^e to four bfloat16, exactly (NaN stays NaN).
__device__ __forceinline__ uint2 widen4(uint32_t codes, float scale) {
    uint32_t h[2];
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
        : "=r"(h[0]), "=r"(h[1])
        : "r"(codes));
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float lo, hi;
        asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
            : "=f"(lo), "=f"(hi)
            : "r"(h[i]));
        o[i] = bf16x2(lo * scale, hi * scale);
    }
    return make_uint2(o[0], o[1]);
}

__device__ __forceinline__ void st_shared(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Makes this thread's shared-memory stores visible to the tensor cores.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void store(const Args& a, uint32_t n, uint32_t k, float v) {
    const uint64_t at = (uint64_t)n * a.lddw + k;
    if (a.dtype == 0) {
        float* p = static_cast<float*>(a.dw) + at;
        *p = a.accumulate ? *p + v : v;
    } else {
        uint16_t* p = static_cast<uint16_t*>(a.dw) + at;
        if (a.accumulate) v += __uint_as_float((uint32_t)*p << 16);
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(*p) : "f"(v));  // the one rounding to 16 bits: dW's own type
    }
}

// Eight elements of dY from p on, which lies `shift` bytes past a 16-byte
// boundary; `lo` and `hi` bound the array. Sixteen aligned bytes that the
// array does not hold whole are read element by element.
__device__ __forceinline__ uint4 load_piece(const uint8_t* q, const uint8_t* lo, const uint8_t* hi) {
    if (q >= lo && q + 16 <= hi) return ld_stream_u4(q);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint8_t* e = q + 2 * i;
        if (e >= lo && e + 2 <= hi) w[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(e) << (16 * (i % 2));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int SHIFT>
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    constexpr int k = SHIFT / 4, r = SHIFT % 4 * 8;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = r ? __funnelshift_r(w[i + k], w[(i + k + 1) % 8], r) : w[i + k];
    return make_uint4(o[0], o[1], o[2], o[3]);
}

struct Ring {
    uint32_t base, bar0, first, step, tiles;
    uint32_t tb0, tb1;  // this block's token blocks
};

// One loader warp's rows of every tile: t = w mod 8, SHIFT bytes past a boundary.
template <int NT, int SHIFT>
__device__ __forceinline__ void load_rows(const Args& a, const Ring& g, const Wait& wt, uint32_t w, uint32_t lane) {
    using S = Shape<NT, false>;
    constexpr int kChunks = NT / 8;               // 16-byte pieces of a row
    constexpr int kRows = 32 / kChunks;           // rows of one load
    constexpr int kLoads = kBT / 8 / kRows;       // loads per stage
    const uint8_t* lo = reinterpret_cast<const uint8_t*>(a.dy);
    const uint8_t* hi = lo + ((uint64_t)(a.T - 1) * a.lddy + a.N) * 2;
    const uint32_t piece = lane % kChunks, sub = lane / kChunks;
    uint32_t it = 0;
    for (uint32_t tile = g.first; tile < g.tiles; tile += g.step) {
        const uint32_t n = tile / a.tiles_k * NT + piece * 8;
        for (uint32_t tb = g.tb0; tb < g.tb1; ++tb, ++it) {
            uint4 v[kLoads];
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const uint32_t t = tb * kBT + w + 8 * (j * kRows + sub);
                v[j] = make_uint4(0, 0, 0, 0);
                if (t < a.T && n < a.N) {
                    const uint8_t* q = lo + ((uint64_t)t * a.lddy + n) * 2 - SHIFT;
                    const uint4 b0 = load_piece(q, lo, hi);
                    v[j] = SHIFT ? shifted<SHIFT>(b0, load_piece(q + 16, lo, hi)) : b0;
                }
            }
            const int s = it % S::kStages;
            if (!__all_sync(kFull, bar_wait(g.bar0 + 8u * (S::kStages + s), ((it / S::kStages) & 1) ^ 1, wt))) return;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const uint32_t t = w + 8 * (j * kRows + sub);  // t % 8 == w
                st_shared(g.base + s * S::kStage + kABytes + piece / 8 * kGroupBytes + t * 128 + ((piece % 8) ^ w) * 16, v[j]);
            }
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(g.bar0 + 8u * s);
        }
    }
}

template <int NT, bool TMA>
__global__ void __launch_bounds__(Shape<NT, TMA>::kWarps * 32, 1)
    wgrad8_kernel(const __grid_constant__ CUtensorMap ymap, const Args a) {
    using S = Shape<NT, TMA>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[3 * S::kStages + 2 * S::kAcc + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t dead;

    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S::kStages + s); };
    auto acc_full = [&](int s) { return bar0 + 8u * (2 * S::kStages + s); };
    auto acc_empty = [&](int s) { return bar0 + 8u * (2 * S::kStages + S::kAcc + s); };
    const uint32_t drain = bar0 + 8u * (2 * S::kStages + 2 * S::kAcc);
    auto copied = [&](int s) { return drain + 8u * (1 + s); };  // dY's part of a stage, by tiled copy

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            bar_init(full(s), TMA ? 4 : 4 + kLoaders);
            bar_init(empty(s), 1);
            bar_init(copied(s), 1);
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
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;
    const Wait wt{&dead, a.faults};

    const uint32_t rank = a.split > 1 ? cluster_rank() : 0;
    const uint32_t tblocks = (a.T + kBT - 1) / kBT;
    Ring g;
    g.base = base;
    g.bar0 = bar0;
    g.first = blockIdx.x / a.split;
    g.step = gridDim.x / a.split;
    g.tiles = a.tiles_k * a.tiles_n;
    g.tb0 = (uint32_t)((uint64_t)tblocks * rank / a.split);
    g.tb1 = (uint32_t)((uint64_t)tblocks * (rank + 1) / a.split);

    if (warp == 8) {
        if (TMA && lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t tile = g.first; ok && tile < g.tiles; tile += g.step) {
                const uint32_t n0 = tile / a.tiles_k * NT;
                for (uint32_t tb = g.tb0; tb < g.tb1; ++tb, ++it) {
                    const int s = it % S::kStages;
                    if (!(ok = bar_wait(empty(s), ((it / S::kStages) & 1) ^ 1, wt))) break;
                    bar_expect(copied(s), NT / 64 * kGroupBytes);
#pragma unroll
                    for (int c = 0; c < NT / 64; ++c)
                        tma_2d(base + s * S::kStage + kABytes + c * kGroupBytes, &ymap, copied(s), (int)(n0 + 64 * c),
                               (int)(tb * kBT));
                }
            }
            // nothing of this block's may still be on its way when it ends
            if (dead)
                for (uint32_t j = it > (uint32_t)S::kStages ? it - S::kStages : 0; j < it; ++j)
                    bar_drain(copied(j % S::kStages), (j / S::kStages) & 1);
        }
    } else if (warp == 9) {
        if (lane == 0) {
            // D float32, A and B bfloat16, both with rows along M and N
            const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | 1u << 15 | 1u << 16 | (uint32_t)(NT / 8) << 17 |
                                   (uint32_t)(kBF / 16) << 24;
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (uint32_t tile = g.first; ok && tile < g.tiles; tile += g.step, ++n) {
                const int buf = n % S::kAcc;
                if (!(ok = bar_wait(acc_empty(buf), ((n / S::kAcc) & 1) ^ 1, wt))) break;
                fence_after();
                for (uint32_t tb = g.tb0; tb < g.tb1; ++tb, ++it) {
                    const int s = it % S::kStages;
                    if (!(ok = bar_wait(full(s), (it / S::kStages) & 1, wt))) break;
                    if (TMA && !(ok = bar_wait(copied(s), (it / S::kStages) & 1, wt))) break;
                    fence_after();
                    const uint64_t ad = smem_desc(base + s * S::kStage, kGroupBytes, 1024);
                    const uint64_t bd = smem_desc(base + s * S::kStage + kABytes, kGroupBytes, 1024);
#pragma unroll
                    for (int j = 0; j < kBT / 16; ++j)  // 16 tokens: two groups of eight rows
                        mma_bf16(tmem + buf * NT, ad + 128 * j, bd + 128 * j, idesc, tb > g.tb0 || j > 0);
                    mma_commit(empty(s));
                }
                if (ok) mma_commit(acc_full(buf));
            }
            if (dead) {
                mma_commit(drain);
                bar_drain(drain, 0);
            }
        }
    } else if (warp >= 10) {
        // the same shift for every row t = w mod 8 and every tile: 8 rows and 8 outputs are multiples of 16 bytes
        const uint32_t w = warp - 10;
        switch ((reinterpret_cast<uintptr_t>(a.dy) + (uint64_t)w * a.lddy * 2) % 16 / 2) {
            case 0: load_rows<NT, 0>(a, g, wt, w, lane); break;
            case 1: load_rows<NT, 2>(a, g, wt, w, lane); break;
            case 2: load_rows<NT, 4>(a, g, wt, w, lane); break;
            case 3: load_rows<NT, 6>(a, g, wt, w, lane); break;
            case 4: load_rows<NT, 8>(a, g, wt, w, lane); break;
            case 5: load_rows<NT, 10>(a, g, wt, w, lane); break;
            case 6: load_rows<NT, 12>(a, g, wt, w, lane); break;
            default: load_rows<NT, 14>(a, g, wt, w, lane); break;
        }
    } else if (warp >= 4) {
        // widen X: a warp takes eight tokens by 64 features at a time, four lanes a token
        constexpr int kPieces = 4;
        const uint32_t w = warp - 4, tsub = lane / 4, piece = lane % 4;
        uint32_t it = 0;
        bool ok = true;
        for (uint32_t tile = g.first; ok && tile < g.tiles; tile += g.step) {
            const uint32_t kb = tile % a.tiles_k;
            for (uint32_t tb = g.tb0; tb < g.tb1; ++tb, ++it) {
                uint4 c[kPieces];
                float sc[kPieces];
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const uint32_t t = tb * kBT + (w * 2 + i / 2) * 8 + tsub, k = kb * kBF + (i % 2) * 64 + piece * 16;
                    c[i] = make_uint4(0, 0, 0, 0);
                    sc[i] = 0.0f;
                    if (t < a.T) {
                        const uint8_t* p = a.x + (uint64_t)t * a.ldx + k;
                        const uint32_t b = __ldg(a.xs + (uint64_t)t * a.nblk + kb);
                        sc[i] = __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fffffffu : b << 23);
                        if (k + 16 <= a.K) {
                            c[i] = __ldg(reinterpret_cast<const uint4*>(p));
                        } else {
                            uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (k + j < a.K) v[j / 4] |= (uint32_t)p[j] << (8 * (j % 4));
                            c[i] = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                }
                const int s = it % S::kStages;
                if (!(ok = __all_sync(kFull, bar_wait(empty(s), ((it / S::kStages) & 1) ^ 1, wt)))) break;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const uint32_t row = (w * 2 + i / 2) * 8 + tsub;  // row % 8 == tsub
                    const uint32_t at = base + s * S::kStage + (i % 2) * kGroupBytes + row * 128;
                    const uint2 p0 = widen4(c[i].x, sc[i]), p1 = widen4(c[i].y, sc[i]);
                    const uint2 p2 = widen4(c[i].z, sc[i]), p3 = widen4(c[i].w, sc[i]);
                    st_shared(at + ((2 * piece) ^ tsub) * 16, make_uint4(p0.x, p0.y, p1.x, p1.y));
                    st_shared(at + ((2 * piece + 1) ^ tsub) * 16, make_uint4(p2.x, p2.y, p3.x, p3.y));
                }
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(full(s));
            }
        }
    } else {
        uint32_t n = 0;
        for (uint32_t tile = g.first; tile < g.tiles; tile += g.step, ++n) {
            const int buf = n % S::kAcc;
            if (!__all_sync(kFull, bar_wait(acc_full(buf), (n / S::kAcc) & 1, wt))) break;
            fence_after();
            const uint32_t k = tile % a.tiles_k * kBF + warp * 32 + lane, n0 = tile / a.tiles_k * NT;
#pragma unroll 1
            for (int c = 0; c < NT; c += 16) {
                uint32_t r[16];
                tmem_ld16(tmem + ((uint32_t)warp << 21) + buf * NT + c, r);
                wait_ld();
                if (a.split > 1) {
                    float* part = reinterpret_cast<float*>(raw + (base - smem_u32(raw)));
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c + j) * kBF + warp * 32 + lane] = __uint_as_float(r[j]);
                } else if (k < a.K) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (n0 + c + j < a.N) store(a, n0 + c + j, k, __uint_as_float(r[j]));
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(acc_empty(buf));
        }
    }

    __syncwarp();
    if (a.split > 1) {
        // one tile per cluster: parts are added in the order of the ranks
        cluster_sync();
        const uint32_t k = g.first % a.tiles_k * kBF + threadIdx.x % kBF, n0 = g.first / a.tiles_k * NT;
        const uint32_t c0 = NT * rank / a.split, c1 = NT * (rank + 1) / a.split;
        if (!dead && threadIdx.x < 2 * kBF) {
            for (uint32_t c = c0 + threadIdx.x / kBF; c < c1 && n0 + c < a.N; c += 2) {
                float v = 0.0f;
                for (uint32_t r = 0; r < a.split; ++r) v += ld_peer(base + (c * kBF + threadIdx.x % kBF) * 4, r);
                if (k < a.K) store(a, n0 + c, k, v);
            }
        }
        cluster_sync();
    }
    fence_before();
    __syncthreads();
    if (warp == 9) tmem_free(tmem, S::kCols);
}

template <int NT, bool TMA>
cudaError_t launch(const Wgrad8Args& m, Args a, int sms, cudaStream_t s) {
    using S = Shape<NT, TMA>;
    CUtensorMap ymap{};
    if (TMA) {
        const cudaError_t e = make_map(&ymap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, m.dy, m.N, m.T, m.lddy * 2, 64, kBT);
        if (e != cudaSuccess) return e;
    }
    a.tiles_n = (m.N + NT - 1) / NT;
    const uint64_t tiles = (uint64_t)a.tiles_k * a.tiles_n;
    if (tiles > 0x7fffffffull) return cudaErrorInvalidValue;
    const uint32_t tblocks = (m.T + kBT - 1) / kBT;
    a.split = 1;
    while (a.split < 8 && tiles * a.split * 2 <= (uint64_t)sms && a.split * 2 <= tblocks) a.split *= 2;
    auto kernel = wgrad8_kernel<NT, TMA>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.split > 1 ? tiles * a.split : tiles < (uint64_t)sms ? tiles : sms));
    cfg.blockDim = dim3(S::kWarps * 32);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, ymap, a);
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
    a.nblk = a.tiles_k = (m.K + kBF - 1) / kBF;
    a.dtype = m.dtype;
    a.accumulate = m.accumulate;
    e = tc::wait_fault_word(&a.faults);
    if (e != cudaSuccess) return e;
    const bool tma = reinterpret_cast<uintptr_t>(m.dy) % 16 == 0 && m.lddy % 8 == 0;
    const bool wide = (uint64_t)a.tiles_k * ((m.N + 255) / 256) >= (uint64_t)di.sms;
    if (tma) return wide ? launch<256, true>(m, a, di.sms, s) : launch<64, true>(m, a, di.sms, s);
    return wide ? launch<256, false>(m, a, di.sms, s) : launch<64, false>(m, a, di.sms, s);
}

}  // namespace s2
