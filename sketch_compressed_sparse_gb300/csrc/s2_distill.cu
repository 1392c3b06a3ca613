// The loss of a softmax layer against a teacher's top logits, and its gradient.
//
// With q = softmax(t / T) over the teacher's entries, p = softmax(z / T) and
// r = softmax(z) over a row of V logits, y its target:
//   loss = soft * sum_k q_k (log q_k - log p_{i_k}) - hard * log r_y
//   dz_i = soft / T * (p_i - sum over k with i_k = i of q_k) + hard * (r_i - [i = y])
// Only two sums over the row are needed for all of it, of exp((z - max) / T) and
// of exp(z - max), so the row is read once: its cluster of blocks keeps it in
// shared memory while the sums are joined, and writes the gradient from there.
// The few entries of the teacher and the target are put right afterwards, one
// by one: the dense part is the same for every element.
//
// Bound by HBM: a logit is read once, its gradient written once.
#include <cfloat>
#include <type_traits>

#include "s2_internal.h"
#include "s2_launch.cuh"
#include "s2_rows.cuh"

namespace s2 {
namespace {

using namespace rows;

constexpr float kLog2e = 1.44269504088896340736f;

// What a block knows of its part of a row.
struct Record {
    float max;         // of its logits (lowest finite number where it has none)
    float soft, hard;  // sums of exp((z - max) / T), exp(z - max)
    float cross;       // sum of q (log q - (z - max) / T) over the teacher's entries here
    float mass;        // sum of their q
    float target;      // the target's logit
    uint32_t has;      // 1: the target is here
};

struct Sums {
    float max, a, b;    // logits
    float tmax, tsum;   // teacher's entries
};

// Joins the sums of the lanes of a warp.
template <bool TWO>
__device__ __forceinline__ void join(Sums& s, float c, float ct) {
    const float m = warp_max(s.max), tm = warp_max(s.tmax);
    s.a = warp_sum(s.a * ex2((s.max - m) * c));
    if (TWO) s.b = warp_sum(s.b * ex2((s.max - m) * kLog2e));
    s.tsum = warp_sum(s.tsum * ex2((s.tmax - tm) * ct));
    s.max = m;
    s.tmax = tm;
}

__device__ __forceinline__ uint32_t bf16_bits(float v) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
    return h;
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)bf16_bits(v); }
__device__ __forceinline__ void put8(float* p, const float* v) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void put8(uint16_t* p, const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A gradient's eight elements of group g. wide: dz is aligned as the logits are.
template <typename TO>
__device__ __forceinline__ void store_group(TO* dz, const Part& p, uint32_t g, uint32_t V, bool wide, const float* v) {
    if (wide && inner(p, g, V)) {
        put8(dz + ((int64_t)g * 8 - p.off), v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t i = (int64_t)g * 8 + j - p.off;
        if (i >= 0 && i < (int64_t)V) put(dz + i, v[j]);
    }
}

// TO: the gradient's type, void for the loss alone. TWO: both sums are needed
// and differ. STAGED: the block's part of a row fits in shared memory (`room`
// groups); else it is read again from global memory.
template <typename TI, typename TO, bool TWO, bool STAGED>
__global__ void __launch_bounds__(kRowThreads, 2) distill_kernel(const DistillArgs a, uint32_t room) {
    constexpr bool kGrad = !std::is_same<TO, void>::value;
    extern __shared__ uint4 slice[];
    __shared__ Sums warp_sums[kRowWarps];
    __shared__ float2 warp_cross[kRowWarps];
    __shared__ Record records[2];
    stream_order();
    const uint32_t blocks = cluster_size(), rank = cluster_rank();
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const float c = a.use_soft ? a.ct : kLog2e;  // of the first sum
    uint32_t turn = 0;
    for (uint64_t row = blockIdx.x / blocks; row < a.T; row += gridDim.x / blocks, turn ^= 1) {
        const TI* z = static_cast<const TI*>(a.z) + row * a.ld;
        const Part p = part_of(z, a.V, rank, blocks);
        const float weight = a.row_weight ? a.row_weight[row] : 1.0f;
        const int32_t* idx = a.idx + row * a.K;
        const float* t = a.t + row * a.K;
        const uint32_t y = a.use_hard ? (uint32_t)a.targets[row] : 0xffffffffu;
        const bool hard = y < a.V;
        const bool alive = weight != 0.0f;
        if (STAGED && alive) stage(slice, room, z, p, a.V);

        Sums s{-FLT_MAX, 0.0f, 0.0f, -FLT_MAX, 0.0f};
        if (alive && a.use_soft) {
            for (uint32_t k = threadIdx.x; k < a.K; k += kRowThreads) {
                if ((uint32_t)idx[k] >= a.V) continue;
                const float v = t[k], m = fmaxf(s.tmax, v);
                s.tsum = s.tsum * ex2((s.tmax - m) * a.ct) + ex2((v - m) * a.ct);
                s.tmax = m;
            }
        }
        if (STAGED) copies_done();  // a thread's own groups; the others' behind the next barrier
        if (alive) {
#pragma unroll 2
            for (uint32_t l = threadIdx.x; l < p.count; l += kRowThreads) {
                const Raw<TI> r = STAGED ? staged<TI>(slice, room, l) : load_group(z, p, p.first + l, a.V);
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = element(r, j);
                const float m = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
                if (m > s.max) {
                    s.a *= ex2((s.max - m) * c);
                    if (TWO) s.b *= ex2((s.max - m) * kLog2e);
                    s.max = m;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = v[j] - s.max;
                    s.a += ex2(d * c);
                    if (TWO) s.b += ex2(d * kLog2e);
                }
            }
        }
        join<TWO>(s, c, a.ct);
        if (lane == 0) warp_sums[warp] = s;
        __syncthreads();
        s = warp_sums[lane % kRowWarps];
        if (lane >= kRowWarps) s.a = s.b = s.tsum = 0.0f;
        join<TWO>(s, c, a.ct);  // of the block, in every warp
        const bool soft = alive && a.use_soft && !(s.tsum == 0.0f);

        // this block's entries: log q = (t - tmax) / T - log(tsum)
        const float inv_tsum = 1.0f / s.tsum, log_tsum = logf(s.tsum);
        auto logit = [&](uint32_t i) {
            const uint64_t j = (uint64_t)i + p.off;
            return STAGED ? staged_at<TI>(slice, room, (uint32_t)(j / 8) - p.first, (uint32_t)(j % 8)) : to_float(z[i]);
        };
        auto mine = [&](uint32_t i) { return i < a.V && (uint32_t)(((uint64_t)i + p.off) / 8) - p.first < p.count; };
        auto prob = [&](uint32_t k) { return ex2((t[k] - s.tmax) * a.ct) * inv_tsum; };
        float cross = 0.0f, mass = 0.0f;
        if (soft) {
            for (uint32_t k = threadIdx.x; k < a.K; k += kRowThreads) {
                const uint32_t i = (uint32_t)idx[k];
                if (!mine(i)) continue;
                const float q = prob(k);
                if (q == 0.0f) continue;
                cross += q * ((t[k] - s.tmax) * a.inv_t - log_tsum - (logit(i) - s.max) * a.inv_t);
                mass += q;
            }
            cross = warp_sum(cross);
            mass = warp_sum(mass);
        }
        if (lane == 0) warp_cross[warp] = make_float2(cross, mass);
        __syncthreads();
        if (warp == 0) {
            const float2 w = lane < kRowWarps ? warp_cross[lane] : make_float2(0.0f, 0.0f);
            const float cs = warp_sum(w.x), ms = warp_sum(w.y);
            if (lane == 0) {
                const bool has = alive && hard && mine(y);
                records[turn] = {s.max, s.a, TWO ? s.b : s.a, cs, ms, has ? logit(y) : 0.0f, has};
            }
        }
        cluster_barrier();
        // of the row, in every warp: a lane reads a block's record
        Record r{-FLT_MAX, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0};
        if (lane < blocks) {
            const uint32_t at = peer(&records[turn], lane);
            r = {peer_float(at), peer_float(at + 4), peer_float(at + 8), peer_float(at + 12), peer_float(at + 16), peer_float(at + 20), peer_u32(at + 24)};
        }
        const float max = warp_max(r.max);
        const float sa = warp_sum(r.soft * ex2((r.max - max) * c));
        const float sb = TWO ? warp_sum(r.hard * ex2((r.max - max) * kLog2e)) : sa;
        if (rank == 0 && warp == 0) {
            // (a row of nothing has probability 0 everywhere: its loss is infinite already)
            const double log_a = sa == 0.0f ? 0.0 : (double)logf(sa), log_b = sb == 0.0f ? 0.0 : (double)logf(sb);
            double sum = 0.0;
            if (soft) sum += (double)a.soft * ((double)r.cross + (r.mass == 0.0f ? 0.0 : (double)r.mass * (((double)max - r.max) * a.inv_t + log_a)));
            if (r.has) sum += (double)a.hard * ((double)max - r.target + log_b);
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            if (lane == 0) a.loss[row] = alive && (soft || hard) ? (float)(sum * weight) : 0.0f;
        }
        if constexpr (kGrad) {
            TO* dz = static_cast<TO*>(a.dz) + row * a.ldd;
            const float g = weight * a.scale;
            const float gq = soft ? g * a.soft * a.inv_t : 0.0f, gy = alive && hard ? g * a.hard : 0.0f;
            float ca = sa == 0.0f ? 0.0f : gq / sa, cb = sb == 0.0f ? 0.0f : gy / sb;
            if (!TWO) ca += cb;
            const bool some = alive && (soft || hard);
            auto dense = [&](float v) {
                const float d = v - max;
                const float e = ca * ex2(d * c);
                return TWO ? e + cb * ex2(d * kLog2e) : e;
            };
#pragma unroll 2
            for (uint32_t l = threadIdx.x; l < p.count; l += kRowThreads) {
                float v[8] = {};
                if (some) {
                    const Raw<TI> q = STAGED ? staged<TI>(slice, room, l) : load_group(z, p, p.first + l, a.V);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = dense(element(q, j));
                }
                store_group(dz, p, p.first + l, a.V, a.wide, v);
            }
            __syncthreads();
            // the elements of the teacher's entries and the target: a warp each, over what was just written
            for (uint32_t k = some ? warp : a.K + 1; k <= a.K; k += kRowWarps) {
                if (k == a.K ? !hard : !soft) continue;
                const uint32_t i = k == a.K ? y : (uint32_t)idx[k];
                if (!mine(i)) continue;
                float q = 0.0f;
                bool first = true;
                for (uint32_t j = lane; soft && j < a.K; j += 32) {
                    if ((uint32_t)idx[j] != i) continue;
                    q += prob(j);
                    first &= j >= k;
                }
                if (!__all_sync(kAll, first)) continue;  // an earlier entry, or the target's, does it
                q = warp_sum(q);
                if (lane == 0) put(dz + i, dense(logit(i)) - gq * q - (i == y ? gy : 0.0f));
            }
        }
        __syncthreads();  // the slice is free
    }
    cluster_barrier();  // no block ends while another reads its record
}

template <typename TI, typename TO, bool TWO>
cudaError_t launch(const DistillArgs& a, cudaStream_t s) {
    constexpr bool kGrad = !std::is_same<TO, void>::value;
    DeviceInfo di{};
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    const uint64_t groups = ((uint64_t)a.V + 14) / 8;  // whatever the row's alignment
    constexpr uint64_t kGroupBytes = 8 * sizeof(TI);
    // as many blocks as let a few of them share an SM, more where the rows do not fill the GPU
    uint32_t blocks = 1;
    while (blocks < 16 && groups * kGroupBytes > blocks * 68ull * 1024) blocks *= 2;
    while (blocks < 16 && (uint64_t)a.T * blocks * 2 <= (uint64_t)di.sms * 2 && groups >= blocks * 2ull * kRowThreads) blocks *= 2;
    auto kernel = distill_kernel<TI, TO, TWO, false>;
    size_t smem = 0;
    uint32_t room = 0;
    int clusters = 0;
    for (;; blocks /= 2) {
        const uint64_t need = (groups + blocks - 1) / blocks + 1;
        const bool fits = kGrad && need * kGroupBytes <= kRowSmem;
        kernel = fits ? distill_kernel<TI, TO, TWO, kGrad> : distill_kernel<TI, TO, TWO, false>;
        room = fits ? (uint32_t)need : 0;
        smem = fits ? need * kGroupBytes : 0;
        e = resident_clusters(reinterpret_cast<const void*>(kernel), blocks, smem, &clusters);
        if (e != cudaSuccess) return e;
        if (clusters > 0 || blocks == 1) break;
    }
    const uint64_t most = 0x7fffffffull / 16;
    const uint32_t grid = (uint32_t)(a.T < most ? a.T : most) * blocks;
    return launch_early(kernel, grid, kRowThreads, smem, blocks, s, a, room);
}

template <typename TI, typename TO>
cudaError_t launch_two(const DistillArgs& a, cudaStream_t s) {
    return a.use_soft && a.use_hard && a.ct != kLog2e ? launch<TI, TO, true>(a, s) : launch<TI, TO, false>(a, s);
}
template <typename TI>
cudaError_t launch_type(const DistillArgs& a, int ddtype, cudaStream_t s) {
    if (!a.dz) return launch_two<TI, void>(a, s);
    return ddtype == 0 ? launch_two<TI, float>(a, s) : launch_two<TI, uint16_t>(a, s);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, int dtype, int ddtype, cudaStream_t s) {
    return dtype == 0 ? launch_type<float>(a, ddtype, s) : launch_type<uint16_t>(a, ddtype, s);
}

}  // namespace s2
