// The loss of a softmax layer against a teacher's top logits, and its gradient.
//
// With q = softmax(t / T) over the teacher's entries, p = softmax(z / T) and
// r = softmax(z) over a row of V logits, y its target:
//   loss = soft * sum_k q_k (log q_k - log p_{i_k}) - hard * log r_y
//   dz_i = soft / T * (p_i - sum over k with i_k = i of q_k) + hard * (r_i - [i = y])
// Only two sums over the row are needed for all of it, of exp((z - max) / T) and
// of exp(z - max), so the row is read once: its cluster of blocks keeps it in
// shared memory while the sums are joined, and writes the gradient from there.
// The teacher's entries and the target are put right afterwards, one by one: the
// dense part is the same for every element.
//
// A thread reads only what it copied itself, so it asks for the next row's
// groups as soon as it has taken a group for the last time: loads go on while
// sums are joined and gradients stored.
//
// Bound by HBM (a logit is read once, its gradient written once) and near it by
// instructions: two exponentials a logit and pass, in pairs of floats.
#include <cfloat>
#include <type_traits>

#include "s2_internal.h"
#include "s2_launch.cuh"
#include "s2_rows.cuh"

namespace s2 {
namespace {

using namespace rows;

constexpr int kRowThreads = 384;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kResident = 3;  // blocks on an SM
constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.69314718055994530942;
constexpr int kSlots = 4;             // teacher's entries of a lane of the first warp
constexpr uint32_t kFew = 32 * kSlots;  // up to here that warp sees to them by itself

// exp2(z * c - k) with k = max * c rounded needs one rounding; where max is near
// the end of the floats (a row of nothing but a type's lowest value) the product
// may be infinite, and (z - max) * c is taken instead.
struct Base {
    float max, k;
    bool plain;
};
__device__ __forceinline__ Base base_of(float max, float c, float limit) {
    const bool plain = fabsf(max) < limit;
    return {max, plain ? __fmul_rn(max, c) : 0.0f, plain};  // (k as it is: not fused into a difference)
}
__device__ __forceinline__ float power(const Base& b, float z, float c) { return ex2(b.plain ? fmaf(z, c, -b.k) : (z - b.max) * c); }
// What a sum taken over `from` is multiplied with to be one over `to`, a base at least as large.
__device__ __forceinline__ float factor(const Base& from, const Base& to, float c) {
    if (!to.plain) return ex2((from.max - to.max) * c);
    return from.plain ? ex2(from.k - to.k) : 0.0f;
}
// log of the sum of exp((z - max) / T) from that of the powers: k is not max * c exactly.
__device__ __forceinline__ double log_sum(float sum, const Base& b, float c) {
    if (sum == 0.0f) return 0.0;  // a row of nothing: its loss is infinite already
    return (double)logf(sum) - (b.plain ? (double)fmaf(b.max, c, -b.k) * kLn2 : 0.0);
}

// What a block knows of its part of a row.
struct Record {
    float max;         // of its logits (lowest finite number where it has none)
    float soft, hard;  // sums of the powers of (z - max) / T, z - max
    float cross;       // sum of q (log q - (z - ref) / T) over the teacher's entries here
    float mass;        // sum of their q
    float ref;         // what stands for max in `cross`
    float target;      // the target's logit
    uint32_t flags;    // 1: the target is here, 2: the row has a soft term, 4: a hard one
};

struct Sums {
    float max, a, b;
};

// Joins the sums of the lanes of a warp.
template <bool TWO>
__device__ __forceinline__ Sums join(const Sums& s, float c, float limit) {
    Sums r;
    r.max = warp_max(s.max);
    r.a = warp_sum(s.a * factor(base_of(s.max, c, limit), base_of(r.max, c, limit), c));
    r.b = TWO ? warp_sum(s.b * factor(base_of(s.max, kLog2e, limit), base_of(r.max, kLog2e, limit), kLog2e)) : r.a;
    return r;
}

// The teacher's entries of one row that a thread has seen: largest logit, sum of powers over it.
struct Teacher {
    float max, sum;
};
__device__ __forceinline__ void see(Teacher& t, float v, float ct) {
    const float m = fmaxf(t.max, v);
    t.sum = t.sum * ex2((t.max - m) * ct) + ex2((v - m) * ct);
    t.max = m;
}
__device__ __forceinline__ Teacher join(const Teacher& t, float ct) {
    Teacher r;
    r.max = warp_max(t.max);
    r.sum = warp_sum(t.sum * ex2((t.max - r.max) * ct));
    return r;
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
    *p = h;
}
__device__ __forceinline__ void put8(float* p, const float2* v) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}
__device__ __forceinline__ void put8(uint16_t* p, const float2* v) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[j].y), "f"(v[j].x));
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A gradient's eight elements of local group l of its row. wide: dz is aligned as the logits are.
template <typename TI, typename TO>
__device__ __forceinline__ void store_group(TO* dz, const Part<TI>& p, uint32_t l, uint32_t V, bool wide, const float2* v) {
    if (wide && p.inner(l)) {
        put8(dz + p.index(l, 0), v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t i = p.index(l, j);
        if (i >= 0 && i < (int64_t)V) put(dz + i, j % 2 ? v[j / 2].y : v[j / 2].x);
    }
}

// A row's entries as they lie in memory, fetched two rows ahead. A lane reads
// what it copied itself: entries lane, lane + 32, ...
struct Fetched {
    uint32_t i[kFew];
    float t[kFew];
    uint32_t y[32];
};
__device__ __forceinline__ void fetch(Fetched& f, const DistillArgs& a, uint64_t row, bool few) {
    const uint32_t lane = threadIdx.x % 32;
    if (row >= a.T) return;
    if (few)
        for (uint32_t k = lane; k < a.K; k += 32) {
            copy4(f.i + k, a.idx + row * a.K + k);
            copy4(f.t + k, a.t + row * a.K + k);
        }
    if (a.use_hard) copy4(f.y + lane, a.targets + row);
}

// What a lane of the last warp knows of a row's entries and target before the
// row's sums. In shared memory, a lane's own (21 words: no two lanes meet a
// bank): in registers it would be carried through the other warps' loops.
struct Entries {
    uint32_t i[kSlots];
    float t[kSlots], z[kSlots];  // z: of those in this block
    Teacher all;
    float inv_sum;  // 1 / all.sum
    float ref;      // the largest z here
    float cross, mass;
    float target;   // the target's logit, where it is here
    uint32_t y;
    uint32_t flags;  // as in a record

    __device__ __forceinline__ float prob(int s, float ct) const { return ex2((t[s] - all.max) * ct) * inv_sum; }
    // The loads of what `f` names; finish() is called after a while.
    template <typename TI>
    __device__ __forceinline__ void begin(const Fetched& f, const DistillArgs& a, bool alive, const TI* zr, const Part<TI>& p, bool few) {
        const uint32_t lane = threadIdx.x % 32;
        y = alive && a.use_hard ? f.y[lane] : 0xffffffffu;
        const bool has = p.holds(y, a.V);
        flags = (uint32_t)has | (y < a.V ? 4u : 0u);
        float v[kSlots + 1];
        v[kSlots] = has ? to_float(zr[y]) : 0.0f;
        uint32_t at[kSlots];
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            const uint32_t k = s * 32 + lane;
            const bool there = alive && few && k < a.K;
            at[s] = there ? f.i[k] : 0xffffffffu;
            t[s] = there ? f.t[k] : 0.0f;
            v[s] = p.holds(at[s], a.V) ? to_float(zr[at[s]]) : -FLT_MAX;
        }
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            i[s] = at[s];
            z[s] = v[s];
        }
        target = v[kSlots];
    }
    template <typename TI>
    __device__ __forceinline__ void finish(const DistillArgs& a, bool alive, const Part<TI>& p, bool few) {
        cross = mass = ref = 0.0f;
        if (!alive || !few) return;
        Teacher sum{-FLT_MAX, 0.0f};
        float top = -FLT_MAX, part = 0.0f, weight = 0.0f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            if (i[s] < a.V) see(sum, t[s], a.ct);
            top = fmaxf(top, z[s]);
        }
        sum = join(sum, a.ct);
        top = warp_max(top);
        const float inv = 1.0f / sum.sum, log_sum = logf(sum.sum);
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            const float q = ex2((t[s] - sum.max) * a.ct) * inv;
            if (!p.holds(i[s], a.V) || q == 0.0f) continue;
            part += q * ((t[s] - sum.max) * a.inv_t - log_sum - (z[s] - top) * a.inv_t);
            weight += q;
        }
        all = sum;
        inv_sum = inv;
        ref = top;
        if (sum.sum == 0.0f) return;  // no entry of weight
        cross = warp_sum(part);
        mass = warp_sum(weight);
        flags |= 2u;
    }
};

// All warps but the last go over the logits; the last one sees to the teacher's
// entries and the target, joins the block's sums and passes them on.
constexpr uint32_t kDense = kRowThreads - 32;
constexpr uint32_t kLast = kRowWarps - 1;

// The last warp waits until the others have stored a row; they go on.
__device__ __forceinline__ void stored() { asm volatile("bar.arrive 1, %0;" ::"n"(kRowThreads) : "memory"); }
__device__ __forceinline__ void stored_wait() { asm volatile("bar.sync 1, %0;" ::"n"(kRowThreads) : "memory"); }

// TO: the gradient's type, void for the loss alone. TWO: both sums are needed
// and differ. STAGED: the block's part of a row fits in shared memory (`room`
// groups); else it is read again from global memory.
template <typename TI, typename TO, bool TWO, bool STAGED>
__global__ void __launch_bounds__(kRowThreads, kResident) distill_kernel(const DistillArgs a, uint32_t room, uint32_t log2_blocks, float limit) {
    constexpr bool kGrad = !std::is_same<TO, void>::value;
    extern __shared__ uint4 slice[];
    __shared__ Sums warp_sums[kRowWarps];
    __shared__ Teacher warp_teacher[kRowWarps];
    __shared__ float2 warp_cross[kRowWarps];
    __shared__ Record records[2];
    __shared__ Entries entries[2][32];
    __shared__ Fetched fetched[2];
    stream_order();
    const uint32_t blocks = 1u << log2_blocks, rank = blocks > 1 ? cluster_rank() : 0;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const float c = a.use_soft ? a.ct : kLog2e;  // of the first sum
    const bool many = a.use_soft && a.K > kFew, few = a.use_soft && !many;
    const uint64_t rows = gridDim.x >> log2_blocks;
    auto row_at = [&](uint64_t row) { return static_cast<const TI*>(a.z) + row * a.ld; };
    auto weight_of = [&](uint64_t row) { return a.row_weight ? a.row_weight[row] : 1.0f; };

    uint64_t row = blockIdx.x >> log2_blocks;
    float weight = row < a.T ? weight_of(row) : 0.0f;
    Part<TI> p = part_of(row_at(row < a.T ? row : 0), a.V, rank, log2_blocks);
    if (warp == kLast) {
        fetch(fetched[0], a, row, few);
        copies_done();
        if (row < a.T) {
            entries[0][lane].begin(fetched[0], a, weight != 0.0f, row_at(row), p, few);
            entries[0][lane].finish(a, weight != 0.0f, p, few);
        }
        fetch(fetched[1], a, row + rows, few);
    } else if (STAGED && weight != 0.0f) {
        stage(slice, room, p, a.V, threadIdx.x, kDense);
    }
    for (uint32_t turn = 0; row < a.T; row += rows, turn ^= 1) {
        const bool alive = weight != 0.0f;
        Entries& e = entries[turn][lane];  // the last warp's
        // the row after this one
        const uint64_t next = row + rows;
        const float next_weight = next < a.T ? weight_of(next) : 0.0f;
        const TI* z = row_at(row);
        Part<TI> np = part_of(row_at(next < a.T ? next : row), a.V, rank, log2_blocks);
        const uint32_t next_count = next_weight != 0.0f ? np.count : 0;

        Sums s{-FLT_MAX, 0.0f, 0.0f};
        if (warp != kLast) {
            if (STAGED) copies_done();
            if (alive) {
                // the warp's largest first: its lanes then share a base, and no sum is ever moved to another
                auto group = [&](uint32_t l) { return STAGED ? staged<TI>(slice, room, l) : load_group(p, l, a.V); };
#pragma unroll 4
                for (uint32_t l = threadIdx.x; l < p.count; l += kDense) s.max = fmaxf(s.max, group_max(group(l)));
                s.max = warp_max(s.max);
                const Base ba = base_of(s.max, c, limit), bb = base_of(s.max, kLog2e, limit);
                Two sa = two(0.0f, 0.0f), sb = sa;
                auto add = [&](const Raw<TI>& r) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Two v = element2(r, j);
                        const float2 x = apart(fma2(v, two(c, c), two(-ba.k, -ba.k)));
                        sa = add2(sa, two(ex2(x.x), ex2(x.y)));
                        if (TWO) {
                            const float2 w = apart(fma2(v, two(kLog2e, kLog2e), two(-bb.k, -bb.k)));
                            sb = add2(sb, two(ex2(w.x), ex2(w.y)));
                        }
                    }
                };
                uint32_t l = threadIdx.x;
                if (ba.plain && bb.plain) {
                    if (!kGrad && STAGED) {  // a group is taken for the last time: the next row's takes its place
                        if (l == 0 && np.lo && l < p.count) {
                            add(group(l));
                            if (l < next_count) stage_group(slice, room, np, l, a.V);
                            l += kDense;
                        }
                        const uint32_t fast = min(p.count, next_count ? np.lo + np.n : 0);
#pragma unroll 2
                        for (; l < fast; l += kDense) {
                            add(group(l));
                            stage_inner(slice, room, np, l);
                        }
                    }
#pragma unroll 2
                    for (; l < p.count; l += kDense) {
                        add(group(l));
                        if (!kGrad && STAGED && l < next_count) stage_group(slice, room, np, l, a.V);
                    }
                } else {
                    for (; l < p.count; l += kDense) {
                        const Raw<TI> r = group(l);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x = element(r, 2 * j), w = element(r, 2 * j + 1);
                            sa = add2(sa, two(power(ba, x, c), power(ba, w, c)));
                            if (TWO) sb = add2(sb, two(power(bb, x, kLog2e), power(bb, w, kLog2e)));
                        }
                        if (!kGrad && STAGED && l < next_count) stage_group(slice, room, np, l, a.V);
                    }
                }
                const float2 ha = apart(sa), hb = apart(sb);
                s.a = ha.x + ha.y;
                s.b = hb.x + hb.y;
            }
            if (!kGrad && STAGED)  // (a part may have a group more than the one before it)
                for (uint32_t l = threadIdx.x; l < next_count; l += kDense)
                    if (!alive || l >= p.count) stage_group(slice, room, np, l, a.V);
            s.a = warp_sum(s.a);
            s.b = TWO ? warp_sum(s.b) : s.a;
            if (lane == 0) warp_sums[warp] = s;
        }
        const int32_t* idx = a.idx + row * a.K;
        const float* t = a.t + row * a.K;
        Teacher tea{-FLT_MAX, 0.0f};
        if (many && alive) {
            for (uint32_t k = threadIdx.x; k < a.K; k += kRowThreads)
                if ((uint32_t)idx[k] < a.V) see(tea, t[k], a.ct);
            tea = join(tea, a.ct);
            if (lane == 0) warp_teacher[warp] = tea;
        }
        __syncthreads();
        if (warp == kLast || many) {  // the block's
            s = lane < kLast ? warp_sums[lane] : Sums{-FLT_MAX, 0.0f, 0.0f};
            s = join<TWO>(s, c, limit);
        }
        float inv_tsum = 0.0f;
        auto prob = [&](float v) { return ex2((v - tea.max) * a.ct) * inv_tsum; };
        if (many) {  // every warp has a share of the entries
            float cross = 0.0f, mass = 0.0f;
            if (alive) tea = join(lane < kRowWarps ? warp_teacher[lane] : Teacher{-FLT_MAX, 0.0f}, a.ct);
            const bool some = !(tea.sum == 0.0f);
            inv_tsum = 1.0f / tea.sum;
            if (some) {
                const float log_tsum = logf(tea.sum);
                for (uint32_t k = threadIdx.x; k < a.K; k += kRowThreads) {
                    const uint32_t i = (uint32_t)idx[k];
                    const float q = prob(t[k]);
                    if (!p.holds(i, a.V) || q == 0.0f) continue;
                    cross += q * ((t[k] - tea.max) * a.inv_t - log_tsum - (to_float(z[i]) - s.max) * a.inv_t);
                    mass += q;
                }
            }
            cross = warp_sum(cross);
            mass = warp_sum(mass);
            if (lane == 0) warp_cross[warp] = make_float2(cross, mass);
            __syncthreads();
            if (warp == kLast) {
                const float2 w = lane < kRowWarps ? warp_cross[lane] : make_float2(0.0f, 0.0f);
                e.cross = warp_sum(w.x);
                e.mass = warp_sum(w.y);
                e.ref = s.max;
                e.flags |= some ? 2u : 0u;
            }
        }
        if (warp == kLast && lane == 0)
            records[turn] = {s.max, s.a, s.b, e.cross, e.mass, e.ref, e.target, e.flags};
        // (only the last warp has something to hand over: the others' stores need not be waited for)
        if (blocks == 1) {
            __syncthreads();
        } else {
            if (warp == kLast) cluster_arrive();
            else cluster_arrive_relaxed();
            cluster_wait();
        }
        // of the row, in every warp: a lane reads a block's record
        Sums r{-FLT_MAX, 0.0f, 0.0f};
        uint32_t flags = 0;
        const uint32_t from = peer(&records[turn], lane < blocks ? lane : 0);
        if (lane < blocks) {
            r = {peer_float(from), peer_float(from + 4), peer_float(from + 8)};
            flags = peer_u32(from + 28);
        }
        const bool soft = __any_sync(kAll, flags & 2), hard = __any_sync(kAll, flags & 4);  // (every block says the same)
        const Sums w = join<TWO>(r, c, limit);
        const Base ba = base_of(w.max, c, limit), bb = base_of(w.max, kLog2e, limit);
        if (warp == kLast && rank == 0) {
            double sum = 0.0;
            if (lane < blocks) {
                const float rc = peer_float(from + 12), rm = peer_float(from + 16), rr = peer_float(from + 20), rt = peer_float(from + 24);
                if (soft) sum += (double)a.soft * ((double)rc + (rm == 0.0f ? 0.0 : (double)rm * (((double)w.max - rr) * a.inv_t + log_sum(w.a, ba, c))));
                if (flags & 1) sum += (double)a.hard * ((double)w.max - rt + log_sum(w.b, TWO ? bb : ba, TWO ? kLog2e : c));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            if (lane == 0) a.loss[row] = soft || hard ? (float)(sum * weight) : 0.0f;
        }
        auto ahead = [&] {  // the last warp's: the next row's entries, and the fetching of those of the row after it
            copies_done();
            if (next < a.T) entries[turn ^ 1][lane].begin(fetched[turn ^ 1], a, next_weight != 0.0f, row_at(next), np, few);
            fetch(fetched[turn], a, next + rows, few);
        };
        if constexpr (kGrad) {
            TO* dz = static_cast<TO*>(a.dz) + row * a.ldd;
            const float g = weight * a.scale;
            const float gq = soft ? g * a.soft * a.inv_t : 0.0f, gy = hard ? g * a.hard : 0.0f;
            float ca = w.a == 0.0f ? 0.0f : gq / w.a, cb = w.b == 0.0f ? 0.0f : gy / w.b;
            if (!TWO) ca += cb;
            const bool some = soft || hard;
            auto dense = [&](float v) {
                const float x = ca * power(ba, v, c);
                return TWO ? fmaf(cb, power(bb, v, kLog2e), x) : x;
            };
            if (warp == kLast) {
                ahead();
            } else {
                auto dense8 = [&](const Raw<TI>& q, float2* v) {  // where both bases are plain
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Two x = element2(q, j);
                        const float2 u = apart(fma2(x, two(c, c), two(-ba.k, -ba.k)));
                        Two d = mul2(two(ca, ca), two(ex2(u.x), ex2(u.y)));
                        if (TWO) {
                            const float2 f = apart(fma2(x, two(kLog2e, kLog2e), two(-bb.k, -bb.k)));
                            d = fma2(two(cb, cb), two(ex2(f.x), ex2(f.y)), d);
                        }
                        v[j] = apart(d);
                    }
                };
                const bool plain = ba.plain && bb.plain && some;
                auto any = [&](uint32_t l) {  // any group of this row or the next
                    if (l < p.count) {
                        float2 v[4] = {};
                        if (some) {
                            const Raw<TI> q = STAGED ? staged<TI>(slice, room, l) : load_group(p, l, a.V);
                            if (plain) {
                                dense8(q, v);
                            } else {
#pragma unroll
                                for (int j = 0; j < 4; ++j) v[j] = make_float2(dense(element(q, 2 * j)), dense(element(q, 2 * j + 1)));
                            }
                        }
                        store_group(dz, p, l, a.V, a.wide, v);
                    }
                    if (STAGED && l < next_count) stage_group(slice, room, np, l, a.V);
                };
                const uint32_t both = max(p.count, STAGED ? next_count : 0);
                uint32_t l = threadIdx.x;
                if (STAGED && plain && a.wide) {  // groups in the midst of both rows
                    if (l == 0 && (p.lo | np.lo) && l < both) {
                        any(l);
                        l += kDense;
                    }
                    TO* at = dz + p.index(0, 0);
                    const uint32_t mid = p.lo + p.n, fast = next_count ? min(mid, np.lo + np.n) : 0;
#pragma unroll 2
                    for (; l < fast; l += kDense) {
                        float2 v[4];
                        dense8(staged<TI>(slice, room, l), v);
                        stage_inner(slice, room, np, l);
                        put8(at + (uint64_t)l * 8, v);
                    }
                    if (!next_count) {
#pragma unroll 2
                        for (; l < mid; l += kDense) {
                            float2 v[4];
                            dense8(staged<TI>(slice, room, l), v);
                            put8(at + (uint64_t)l * 8, v);
                        }
                    }
                }
                for (; l < both; l += kDense) any(l);
            }
            // the elements of the entries and the target are stored again, behind the dense ones
            if (many || warp == kLast) stored_wait();
            else stored();
            if (many && soft) {
                for (uint32_t k = warp; k < a.K; k += kRowWarps) {  // a warp each
                    const uint32_t i = (uint32_t)idx[k];
                    if (!p.holds(i, a.V)) continue;
                    const uint32_t y = a.use_hard ? (uint32_t)a.targets[row] : 0xffffffffu;
                    float sum = 0.0f;
                    bool first = true;
                    for (uint32_t j = lane; j < a.K; j += 32) {
                        if ((uint32_t)idx[j] != i) continue;
                        sum += prob(t[j]);
                        first &= j >= k;
                    }
                    if (!__all_sync(kAll, first)) continue;
                    sum = warp_sum(sum);
                    if (lane == 0) put(dz + i, dense(to_float(z[i])) - gq * sum - (i == y ? gy : 0.0f));
                }
            }
            if (warp == kLast) {
                if (few && soft) {
#pragma unroll
                    for (int k = 0; k < kSlots; ++k) {
                        uint32_t todo = __ballot_sync(kAll, p.holds(e.i[k], a.V));
                        while (todo) {
                            const int at = __ffs(todo) - 1;
                            todo &= todo - 1;
                            const uint32_t i = __shfl_sync(kAll, e.i[k], at);
                            // an entry that stands before it sees to the others of its index
                            float sum = 0.0f;
                            bool first = true;
#pragma unroll
                            for (int o = 0; o < kSlots; ++o) {
                                const uint32_t same = __ballot_sync(kAll, e.i[o] == i);
                                if (o < k) first &= same == 0;
                                if (o == k) first &= (same & ((1u << at) - 1)) == 0;
                                if (e.i[o] == i) sum += e.prob(o, a.ct);
                            }
                            if (!first) continue;
                            sum = warp_sum(sum);
                            if ((int)lane == at) put(dz + i, dense(e.z[k]) - gq * sum - (i == e.y ? gy : 0.0f));
                        }
                    }
                }
                if (e.flags & 1) {  // the target, where no entry has seen to it
                    bool listed = false;
                    if (few && soft) {
#pragma unroll
                        for (int k = 0; k < kSlots; ++k) listed |= e.i[k] == e.y;
                    } else if (many && soft) {
                        for (uint32_t j = lane; j < a.K; j += 32) listed |= (uint32_t)idx[j] == e.y;
                    }
                    if (!__any_sync(kAll, listed) && lane == 0) put(dz + e.y, dense(e.target) - gy);
                }
                if (next < a.T) entries[turn ^ 1][lane].finish(a, next_weight != 0.0f, np, few);
            }
        } else if (warp == kLast) {
            ahead();
            if (next < a.T) entries[turn ^ 1][lane].finish(a, next_weight != 0.0f, np, few);
        }
        weight = next_weight;
        p = np;
    }
    if (blocks > 1) cluster_barrier();  // no block ends while another reads its record
}

template <typename TI, typename TO, bool TWO>
cudaError_t launch(const DistillArgs& a, cudaStream_t s) {
    const uint64_t groups = ((uint64_t)a.V + 14) / 8;  // whatever the row's alignment
    constexpr uint64_t kGroupBytes = 8 * sizeof(TI);
    // The number of blocks that share a row: the fewest groups that a block goes
    // through in all, a row counting kRowCost of them more for the joining of its sums.
    constexpr uint64_t kRowCost = 1000;
    uint64_t best = ~0ull;
    uint32_t blocks = 0, room = 0, clusters = 0, log2_blocks = 0;
    auto kernel = distill_kernel<TI, TO, TWO, false>;
    for (uint32_t b = 1; b <= 16; b *= 2) {
        const uint64_t need = (groups + b - 1) / b + 1;
        const uint64_t smem = smem_of(need * kGroupBytes);
        const bool fits = smem <= 66 * 1024;  // kResident times in an SM, beside 8 KB of the kernel's own
        if (!fits && b < 16) continue;
        if (b > 1 && groups < b * (uint64_t)kRowThreads / 2) break;  // too little for so many
        auto k = fits ? distill_kernel<TI, TO, TWO, true> : distill_kernel<TI, TO, TWO, false>;
        int n = 0;
        const cudaError_t e = resident_clusters(reinterpret_cast<const void*>(k), kRowThreads, b, fits ? smem : 0, &n);
        if (e != cudaSuccess) return e;
        if (n < 1) continue;
        const uint64_t cost = ((uint64_t)a.T + n - 1) / n * (need + kRowCost);
        if (cost >= best) continue;
        best = cost;
        blocks = b;
        room = fits ? (uint32_t)need : 0;
        clusters = (uint32_t)n;
        kernel = k;
    }
    if (blocks == 0) {  // clusters of sixteen do not fit on this device: rows are read again
        int n = 0;
        blocks = 8;
        const cudaError_t e = resident_clusters(reinterpret_cast<const void*>(kernel), kRowThreads, blocks, 0, &n);
        if (e != cudaSuccess) return e;
        clusters = n > 0 ? n : 1;
    }
    while ((1u << log2_blocks) < blocks) ++log2_blocks;
    const float c = a.use_soft ? a.ct : kLog2e;
    const float limit = 1e30f / (c > kLog2e ? c : kLog2e);
    const uint32_t grid = (a.T < clusters ? a.T : clusters) * blocks;
    return launch_early(kernel, grid, kRowThreads, smem_of(room * kGroupBytes), blocks, s, a, room, log2_blocks, limit);
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
