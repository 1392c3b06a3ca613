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
// Bound by HBM (a logit is read once, its gradient written once), near it by
// exponentials (two a logit and pass), and by the time that a row's sums take to
// be joined, so every kind of work has warps of its own: most go over the logits
// and copy the next row's groups to the places of those that they took for the
// last time (a thread reads only what it copied, so no barrier is needed for
// that); one joins the sums and hands them to the cluster's other blocks; two see
// to the teacher's entries, every second row each, so that these have the time of
// two rows for loads that depend on one another. Measured: 2048 rows of 267735
// bfloat16 with 64 entries, a target and a bfloat16 gradient at temperature 2 432 us
// (5.1 TB/s of its 2.2 GB, 0.76 of a copy's rate), at 1 425, at any other, where
// each logit has two exponentials, 546; 2048 rows of 33278 bfloat16, the loss alone,
// 36 us at temperature 2 (3.8 TB/s), 34 at 1, 42 at others; 200 rows of 33278 float32
// with a float32 gradient 21.7 us, where one round of rows is loaded, summed and
// stored with nothing beside it.
#include <cfloat>
#include <type_traits>

#include "s2_internal.h"
#include "s2_launch.cuh"
#include "s2_rows.cuh"
#include "s2_tc.cuh"

namespace s2 {
namespace {

using namespace rows;

constexpr int kMaxThreads = 512;
constexpr uint32_t kMaxBlocks = 16;  // of a cluster
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// The exponentials of a logit: one where one sum is enough; two; or, where the
// temperature is 2, the one at that temperature and its square.
enum { kOne, kSquare, kBoth };

// exp2(z * c - k) with k close to max * c needs one rounding; where max is near
// the end of the floats (a row of nothing but a type's lowest value) the product
// may be infinite, and (z - max) * c is taken instead.
struct Base {
    float max, k;
    bool plain;
};
// limit: below it a logit's product with c and with log2(e) is far from infinite.
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
__device__ __forceinline__ float log_sum(float sum, const Base& b, float c) {
    if (sum == 0.0f) return 0.0f;  // a row of nothing: its loss is infinite already
    return logf(sum) - (b.plain ? fmaf(b.max, c, -b.k) * kLn2 : 0.0f);
}

// What a block knows of its part of a row: 32 bytes, two stores to another block
// (a third brings bmax, where that is not max).
struct __align__(16) Record {
    float max;         // base of its logits' sums (lowest finite number where it has none)
    float soft, hard;  // sums of the powers of (z - max) / T, z - max (z - bmax)
    uint32_t flags;    // 1: the target is here, 2: the row has a soft term, 4: a hard one
    float cross;       // sum of q (log q - (z - ref) / T) over the teacher's entries here
    float mass;        // sum of their q
    float ref;         // what stands for max in `cross`
    float target;      // the target's logit, where it is here
};

// Sums over a base. A log-sum at temperature T lies up to (T - 1) log V above the
// one at 1, so two sums that have nothing to do with one another have a base each.
struct Sums {
    float max, a, b;
    float bmax;  // of b; max but for kBoth
};
struct Three {  // all but bmax
    float max, a, b;
};

// Joins the sums of the lanes of a warp.
template <int EXPS>
__device__ __forceinline__ Sums join(const Sums& s, float c, float limit) {
    Sums r;
    r.max = warp_max(s.max);
    r.a = warp_sum(s.a * factor(base_of(s.max, c, limit), base_of(r.max, c, limit), c));
    r.bmax = EXPS == kBoth ? warp_max(s.bmax) : r.max;
    r.b = EXPS != kOne ? warp_sum(s.b * factor(base_of(s.bmax, kLog2e, limit), base_of(r.bmax, kLog2e, limit), kLog2e)) : r.a;
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

// A whole row's sums, moved to bases at its log-sums. A power is off by 2^-24 of
// its exponent, which is small for the logits that matter only there, and what is
// left of a sum is one to two: neither the gradient nor the loss depends on where
// the sums were taken. The moves are by whole factors of two, but for the rounding
// of the base, which goes to the sum.
template <int EXPS>
struct Settled {
    Base a, b;
    float sa, sb;
    bool moved;  // a and, where it has a base of its own, b

    __device__ __forceinline__ Settled(const Sums& w, float c, float inv_c, float limit)
        : a(base_of(w.max, c, limit)), b(base_of(w.bmax, kLog2e, limit)), sa(w.a), sb(w.b) {
        // (Bases below 2^20 are rounded by 2^-5 at most. At a temperature of 10^37 a
        // factor of two is more than the floats. Sums elsewhere stay where they are.)
        auto fit = [](const Base& x, float s, float inv_c) {
            return fabsf(x.k) < 0x1p20f - 128.0f && x.plain && s > 0x1p-100f && s < 0x1p100f && (fabsf(x.k) + 100.0f) * inv_c < FLT_MAX;
        };
        moved = fit(a, sa, inv_c) && (EXPS != kBoth || fit(b, sb, kLn2));
        if (!moved) return;
        const float by = move(a, sa, inv_c);
        if (EXPS == kSquare) {
            const float down = __uint_as_float((254u << 23) - (__float_as_uint(w.a) & 0x7f800000u));  // 2^-n
            sb *= down;
            sb *= down;
            sb = fmaf(sb, by, sb);
            sb = fmaf(sb, by, sb);
            b.max = a.max;
            b.k = 2.0f * a.k;
        } else if (EXPS == kBoth) {
            move(b, sb, kLn2);
        } else {
            sb = sa;
        }
    }
    // s = 2^n t: t over the base k + n. That number is rounded, by -r say, so t becomes
    // t (1 + p), p = 2^r - 1, the series of the exponential to its fourth term: the next is
    // below 2^-31 where |r| <= 2^-5.
    static __device__ __forceinline__ float move(Base& x, float& s, float inv_c) {
        const uint32_t bits = __float_as_uint(s);
        const float n = (float)((int)(bits >> 23) - 127), k = __fadd_rn(x.k, n), t = __fsub_rn(k, x.k);
        const float r = kLn2 * __fadd_rn(__fsub_rn(x.k, __fsub_rn(k, t)), __fsub_rn(n, t));
        const float by = fmaf(r * r, fmaf(r, fmaf(r, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f), r);
        s = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
        s = fmaf(s, by, s);
        x.k = k;
        x.max = k * inv_c;  // (nearly)
        return by;
    }
};

// A thread's sums over the groups that it takes, over a base that its warp shares
// at first. What is read again later is not known to be below it: a logit 2^kFar
// times as likely moves the sums to another base.
constexpr float kFar = 16.0f;
template <int EXPS>
struct Second {  // base of the second sum
    __device__ __forceinline__ void put(float) {}
    __device__ __forceinline__ float get(float first) const { return first; }
};
template <>
struct Second<kBoth> {
    float max;
    __device__ __forceinline__ void put(float m) { max = m; }
    __device__ __forceinline__ float get(float) const { return max; }
};
template <int EXPS>
struct Taken {
    float max, ka, kb;  // of the bases; both are plain, or none is and they are the same
    bool plain;
    Second<EXPS> second;
    Two sa, sb;
    __device__ __forceinline__ void rest_on(float m, float mb, float c, float limit) {
        const Base a = base_of(m, c, limit), b = base_of(EXPS == kBoth ? mb : m, kLog2e, limit);
        max = m;
        second.put(mb);
        ka = a.k;
        kb = b.k;
        plain = a.plain && b.plain;
    }
    __device__ __forceinline__ Taken(float m, float mb, float c, float limit) : sa(two(0.0f, 0.0f)), sb(sa) { rest_on(m, mb, c, limit); }
    // a base is plain
    template <typename TI>
    __device__ __forceinline__ void add(const Raw<TI>& r, float c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Two v = element2(r, j);
            const float2 x = apart(fma2(v, two(c, c), two(-ka, -ka)));
            const Two e = two(ex2(x.x), ex2(x.y));
            sa = add2(sa, e);
            if (EXPS == kSquare) sb = fma2(e, e, sb);
            if (EXPS == kBoth) {
                const float2 w = apart(fma2(v, two(kLog2e, kLog2e), two(-kb, -kb)));
                sb = add2(sb, two(ex2(w.x), ex2(w.y)));
            }
        }
    }
    template <typename TI>
    __device__ __forceinline__ void add_any(const Raw<TI>& r, float c) {
        if (plain) return add(r, c);
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            const float x = element(r, j) - max;
            sa = add2(sa, two(ex2(x * c), 0.0f));
            if (EXPS != kOne) sb = add2(sb, two(ex2(x * kLog2e), 0.0f));
        }
    }
    __device__ __noinline__ void move(float m, float c, float limit) {
        const Base a{max, ka, plain}, b{second.get(max), kb, plain};
        rest_on(m, m, c, limit);
        const float fa = factor(a, {max, ka, plain}, c), fb = factor(b, {max, kb, plain}, kLog2e);
        sa = mul2(sa, two(fa, fa));
        if (EXPS != kOne) sb = mul2(sb, two(fb, fb));
    }
    __device__ __forceinline__ Sums sums() const {
        const float2 x = apart(sa), y = apart(sb);
        return {max, x.x + x.y, y.x + y.y, second.get(max)};
    }
};

// What is the same for all of a launch, and for all of a row.
template <typename TI>
struct Rows {
    const DistillArgs& a;
    uint32_t rank, log2_blocks, room;
    float c, inv_c, limit;  // c: of the first sum
    uint64_t row, step;
    __device__ __forceinline__ const TI* logits(uint64_t r) const { return static_cast<const TI*>(a.z) + r * a.ld; }
    __device__ __forceinline__ bool there(uint64_t r) const { return r < a.T; }
    __device__ __forceinline__ float weight(uint64_t r) const { return !there(r) ? 0.0f : a.row_weight ? a.row_weight[r] : 1.0f; }
    __device__ __forceinline__ Part<TI> part(uint64_t r) const { return part_of(logits(there(r) ? r : 0), a.V, rank, log2_blocks); }
    // groups of part p that stay in shared memory
    __device__ __forceinline__ uint32_t kept(const Part<TI>& p, float weight) const { return weight != 0.0f ? min(p.count, room) : 0; }
};

// The factors of a row's gradient, from the joined sums.
template <int EXPS>
struct Factors {
    Base ba, bb;
    float ca, cb, gq, gy;  // of the powers; of the teacher's probabilities and the target
    bool some;             // the row has a term
    __device__ __forceinline__ Factors(const Settled<EXPS>& w, bool soft, bool hard, float weight, const DistillArgs& a)
        : ba(w.a), bb(w.b), some(soft || hard) {
        const float g = weight * a.scale;
        gq = soft ? g * a.soft * a.inv_t : 0.0f;
        gy = hard ? g * a.hard : 0.0f;
        ca = w.sa == 0.0f ? 0.0f : gq / w.sa;
        cb = w.sb == 0.0f ? 0.0f : gy / w.sb;
        if (EXPS == kOne) ca += cb;
    }
    __device__ __forceinline__ float dense(float v, float c) const {
        const float e = power(ba, v, c);
        if (EXPS == kSquare) return e * fmaf(cb, e, ca);
        return EXPS == kBoth ? fmaf(cb, power(bb, v, kLog2e), ca * e) : ca * e;
    }
    // the same for a group, where the bases are plain
    template <typename TI>
    __device__ __forceinline__ void dense8(const Raw<TI>& q, float c, float2* v) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Two x = element2(q, j);
            const float2 u = apart(fma2(x, two(c, c), two(-ba.k, -ba.k)));
            const Two e = two(ex2(u.x), ex2(u.y));
            Two d = mul2(e, EXPS == kSquare ? fma2(two(cb, cb), e, two(ca, ca)) : two(ca, ca));
            if (EXPS == kBoth) {
                const float2 f = apart(fma2(x, two(kLog2e, kLog2e), two(-bb.k, -bb.k)));
                d = fma2(two(cb, cb), two(ex2(f.x), ex2(f.y)), d);
            }
            v[j] = apart(d);
        }
    }
};

// A thread's sums over its groups first, first + step, ... of part p, joined in
// its warp. FREE: this is the last use of the groups in shared memory, and the
// next row's (part np) take their places.
//
// The base of the sums need not be the largest logit: any number near it serves.
// It is `guess` (and `guess_b`), the log-sum of the row before. Where the sums come
// out above 2^16 or below 2^-30 (a warp has a hundredth of a row's words, and far
// less of its probability where one word has nearly all) they are taken again, over
// the log-sum that they give; where they say nothing, over the largest logit. An
// exponent that matters is so below 32, and off by half of 2^-19 at most. (Taken as
// far away as floats reach, a row 40 below the one before it had its loss off by up
// to 6e-6. With one base for both sums every row was gone over three times from
// temperature 5 on: 2048 x 267735 bfloat16 with a gradient in 780 us instead of 546.
// Taking sums again costs rows that lie 35 to 50 apart, 2048 x 33278 loss alone, 40
// us instead of 35, and rows where one word has all but 2^-24 of the probability
// 502 instead of 437.)
template <typename TI, int EXPS, bool FREE>
__device__ __forceinline__ Sums sums_of(uint4* slice, const Rows<TI>& rw, const Part<TI>& p, uint32_t kept, const Part<TI>& np,
                                        uint32_t next_kept, float guess, float guess_b, uint32_t first, uint32_t step) {
    const float c = rw.c;
    const uint32_t room = rw.room;
    auto near = [](float v) { return v > 0x1p-30f && v < 0x1p16f; };
    auto known = [](float v) { return v > 0x1p-100f && v < 0x1p100f; };
    Taken<EXPS> sum(guess, guess_b, c, rw.limit);
    Sums s{guess, 0.0f, 0.0f, guess};
    bool good = sum.plain;
    if (good) {
#pragma unroll 2
        for (uint32_t l = first; l < kept; l += step) sum.add(staged<TI>(slice, room, l), c);
        s = sum.sums();
        s.a = warp_sum(s.a);
        s.b = EXPS != kOne ? warp_sum(s.b) : s.a;
        good = near(s.a) && (EXPS == kBoth ? near(s.b) : known(s.b));
    }
    if (!good) {
        const bool some = known(s.a) && (EXPS != kBoth || known(s.b));
        if (some) sum.rest_on(s.max + __log2f(s.a) / c, EXPS == kBoth ? s.bmax + __log2f(s.b) / kLog2e : 0.0f, c, rw.limit);
        if (!some || !sum.plain) {
            float m = -FLT_MAX;
#pragma unroll 4
            for (uint32_t l = first; l < kept; l += step) m = fmaxf(m, group_max(staged<TI>(slice, room, l)));
            m = warp_max(m);
            sum.rest_on(m, m, c, rw.limit);
        }
        sum.sa = sum.sb = two(0.0f, 0.0f);
        if (sum.plain) {
#pragma unroll 2
            for (uint32_t l = first; l < kept; l += step) sum.add(staged<TI>(slice, room, l), c);
        } else {
            for (uint32_t l = first; l < kept; l += step) sum.add_any(staged<TI>(slice, room, l), c);
        }
        s = sum.sums();
        s.a = warp_sum(s.a);
        s.b = EXPS != kOne ? warp_sum(s.b) : s.a;
    }
    if (FREE) {
        uint32_t l = first;
        if (l == 0 && np.lo && l < next_kept) {
            stage_group(slice, room, np, l, rw.a.V);
            l += step;
        }
        const uint32_t fast = min(next_kept, np.lo + np.n);
#pragma unroll 4
        for (; l < fast; l += step) stage_inner(slice, room, np, l);
        for (; l < next_kept; l += step) stage_group(slice, room, np, l, rw.a.V);
    }
    if (p.count > room) {  // what does not stay in shared memory
        const float far = kFar / c;
        auto limit_of = [&] {  // (finite: an infinite logit has to be seen)
            if (!sum.plain) return sum.max;
            return fminf(EXPS == kBoth ? fminf(sum.max + far, sum.second.get(sum.max) + kFar / kLog2e) : sum.max + far, FLT_MAX);
        };
        float above = limit_of();
        uint32_t r = first;
        if (first < kept) r += (kept - first + step - 1) / step * step;
#pragma unroll 2
        for (; r < p.count; r += step) {
            const Raw<TI> g = load_group(p, r, rw.a.V);
            const float m = group_max(g);
            if (m > above) {
                sum.move(m, c, rw.limit);
                above = limit_of();
            }
            sum.add_any(g, c);
        }
        s = join<EXPS>(sum.sums(), c, rw.limit);
    }
    return s;
}

// Stores a thread's groups of the gradient's dense part; the next row's take the
// places of those in shared memory.
template <typename TI, typename TO, int EXPS>
__device__ __forceinline__ void store_dense(TO* dz, uint4* slice, const Rows<TI>& rw, const Factors<EXPS>& f, const Part<TI>& p, uint32_t kept,
                                            const Part<TI>& np, uint32_t next_kept, uint32_t first, uint32_t step) {
    const uint32_t V = rw.a.V, room = rw.room;
    const float c = rw.c;
    const bool plain = f.ba.plain && (EXPS != kBoth || f.bb.plain) && f.some, wide = rw.a.wide;
    auto any = [&](uint32_t l) {  // any group of this row or the next
        if (l < p.count) {
            float2 v[4] = {};
            if (f.some) {
                const Raw<TI> q = l < kept ? staged<TI>(slice, room, l) : load_group(p, l, V);
                if (plain) {
                    f.dense8(q, c, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = make_float2(f.dense(element(q, 2 * j), c), f.dense(element(q, 2 * j + 1), c));
                }
            }
            store_group(dz, p, l, V, wide, v);
        }
        if (l < next_kept) stage_group(slice, room, np, l, V);
    };
    const uint32_t both = max(p.count, next_kept);
    uint32_t l = first;
    if (plain && wide) {  // groups in the midst of both rows
        if (l == 0 && (p.lo | np.lo) && l < both) {
            any(l);
            l += step;
        }
        TO* at = dz + p.index(0, 0);
        const uint32_t mid = p.lo + p.n, here = min(mid, kept), fast = next_kept ? min(here, min(np.lo + np.n, next_kept)) : 0;
#pragma unroll 2
        for (; l < fast; l += step) {
            float2 v[4];
            f.dense8(staged<TI>(slice, room, l), c, v);
            stage_inner(slice, room, np, l);
            put8(at + (uint64_t)l * 8, v);
        }
        if (!next_kept) {
#pragma unroll 2
            for (; l < here; l += step) {
                float2 v[4];
                f.dense8(staged<TI>(slice, room, l), c, v);
                put8(at + (uint64_t)l * 8, v);
            }
        }
        const uint32_t rest = max(kept, next_kept);
        for (; l < rest; l += step) any(l);
#pragma unroll 2
        for (; l < mid; l += step) {
            float2 v[4];
            f.dense8(load_inner(p, l), c, v);
            put8(at + (uint64_t)l * 8, v);
        }
    }
    for (; l < both; l += step) any(l);
}

// The row's loss, from what the lanes' blocks know; in lane 0.
template <int EXPS>
__device__ __forceinline__ float loss_of(const Record& r, const Settled<EXPS>& w, bool mine, bool soft, float weight, const DistillArgs& a, float c) {
    float sum = 0.0f;
    if (mine) {
        if (soft) sum += a.soft * (r.cross + (r.mass == 0.0f ? 0.0f : r.mass * ((w.a.max - r.ref) * a.inv_t + log_sum(w.sa, w.a, c))));
        const Base& b = EXPS != kOne ? w.b : w.a;
        if (r.flags & 1) sum += a.hard * ((b.max - r.target) + log_sum(w.sb, b, EXPS != kOne ? kLog2e : c));
    }
    return warp_sum(sum) * weight;
}

// ---- up to 256 entries -----------------------------------------------------------

constexpr int kSlots = 8;               // entries of a lane
constexpr uint32_t kFew = 32 * kSlots;
constexpr uint32_t kPlaces = 512;       // of the table that finds indices that stand twice
constexpr uint32_t kNone = 0xffffffffu;
constexpr uint32_t kRepeated = 0x80000000u;  // beside an index of the table (below 2^31)
constexpr uint32_t kHelpers = 96;       // threads that do not go over the logits

template <int EXPS>
struct SharedBases {};
template <>
struct SharedBases<kBoth> {  // bmax of the records and of the warps' sums
    float4 bases[2][kMaxBlocks];
    float sum_bases[kMaxThreads / 32];
};
template <int EXPS>
struct Shared : SharedBases<EXPS> {
    Record records[2][kMaxBlocks];  // of this row and the next, from every block
    Three sums[kMaxThreads / 32];
    float4 entries[2];              // cross, mass, ref, target
    uint32_t flags[2];
    uint32_t table[2][kPlaces];
    uint64_t full[2];               // the records are here
    uint32_t dead;
};

__device__ __forceinline__ void arrive(uint32_t barrier, uint32_t threads) {
    __syncwarp();  // the whole warp at once
    asm volatile("bar.arrive %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
}
__device__ __forceinline__ void wait(uint32_t barrier, uint32_t threads) {
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
}
// 16 bytes to another block's shared memory; its barrier counts them.
__device__ __forceinline__ void push16(uint32_t to, uint32_t barrier, const uint4& v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w), "r"(barrier)
                 : "memory");
}

// Barriers of a block: kSums: a row's sums and entries are there, and the records
// of the row before have been read (all threads; the joining warp alone waits);
// kStored + parity: the row's dense part is stored (the entries' warp waits).
constexpr uint32_t kSums = 1, kStored = 2;

// The rows of an entries' warp: what it holds of one.
template <typename TI>
struct Entries {
    uint32_t i[kSlots];
    float q[kSlots], z[kSlots];  // q: logits, then probabilities; z: of those in this block
    float target;
    uint32_t y, flags, repeated;  // repeated: a bit for each slot whose index stands twice
    bool twice, listed;

    __device__ __forceinline__ void fetch(const Rows<TI>& rw, uint64_t row) {
        const DistillArgs& a = rw.a;
        const uint32_t lane = threadIdx.x % 32;
        const bool there = rw.there(row);
        y = there && a.use_hard ? (uint32_t)a.targets[row] : kNone;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            const uint32_t k = s * 32 + lane;
            const bool some = there && a.use_soft && k < a.K;
            i[s] = some ? (uint32_t)a.idx[row * a.K + k] : kNone;
            q[s] = some ? a.t[row * a.K + k] : 0.0f;
        }
    }
    // The logits that belong to what fetch() brought.
    __device__ __forceinline__ void gather(const Rows<TI>& rw, uint64_t row, const Part<TI>& p) {
        const TI* zr = rw.logits(row);
        const bool has = p.holds(y, rw.a.V);
        flags = (uint32_t)has | (y < rw.a.V ? 4u : 0u);
        target = has ? to_float(zr[y]) : 0.0f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) z[s] = p.holds(i[s], rw.a.V) ? to_float(zr[i[s]]) : -FLT_MAX;
    }
    // Probabilities, and this block's part of the soft term: cross, mass, ref, target.
    __device__ __forceinline__ float4 finish(const Rows<TI>& rw, const Part<TI>& p, uint32_t* table, bool grad) {
        const DistillArgs& a = rw.a;
        const uint32_t lane = threadIdx.x % 32, V = a.V;
        twice = listed = false;
        repeated = 0;
        if (!a.use_soft) return make_float4(0.0f, 0.0f, 0.0f, target);
        float most = -FLT_MAX, top = -FLT_MAX, sum = 0.0f, cross = 0.0f, mass = 0.0f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            if (i[s] < V) most = fmaxf(most, q[s]);
            top = fmaxf(top, z[s]);
        }
        most = warp_max(most);
        top = warp_max(top);
        float x[kSlots];
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            x[s] = q[s] - most;
            q[s] = i[s] < V ? ex2(x[s] * a.ct) : 0.0f;
            sum += q[s];
            listed |= i[s] == y && i[s] < V;
        }
        sum = warp_sum(sum);
        if (!(sum == 0.0f)) {
            flags |= 2u;
            const float inv = 1.0f / sum, log_all = logf(sum);
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                q[s] *= inv;
                if (!p.holds(i[s], V) || q[s] == 0.0f) continue;
                cross += q[s] * (x[s] * a.inv_t - log_all - (z[s] - top) * a.inv_t);
                mass += q[s];
            }
            cross = warp_sum(cross);
            mass = warp_sum(mass);
        }
        listed = __any_sync(kAll, listed) && (flags & 2u);
        if (grad) {  // each index into a table of its own, where another of the same would be found
            for (uint32_t t = lane; t < kPlaces; t += 32) table[t] = kNone;
            __syncwarp();
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                if (i[s] >= V) continue;
                uint32_t at = (i[s] * 0x9E3779B1u) >> 23;  // (half full at most)
                for (uint32_t tries = 0; tries < kPlaces; ++tries) {
                    const uint32_t old = atomicCAS(table + at, kNone, i[s]);
                    if (old == kNone) break;
                    if ((old & ~kRepeated) == i[s]) {
                        atomicOr(table + at, kRepeated);
                        twice = true;
                        break;
                    }
                    at = (at + 1) % kPlaces;
                }
            }
            twice = __any_sync(kAll, twice);
            if (twice) {  // all entries of such an index have to know
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    if (i[s] >= V) continue;
                    uint32_t at = (i[s] * 0x9E3779B1u) >> 23;
                    for (uint32_t tries = 0; tries < kPlaces && (table[at] & ~kRepeated) != i[s]; ++tries) at = (at + 1) % kPlaces;
                    repeated |= (table[at] >> 31) << s;
                }
            }
        }
        return make_float4(cross, mass, top, target);
    }
    // The gradient's elements at the entries and the target, over their dense part.
    template <typename TO, int EXPS>
    __device__ __forceinline__ void correct(TO* dz, const Rows<TI>& rw, const Factors<EXPS>& f, const Part<TI>& p, bool soft) const {
        const uint32_t lane = threadIdx.x % 32, V = rw.a.V;
        if (soft) {
#pragma unroll
            for (int s = 0; s < kSlots; ++s)
                if (p.holds(i[s], V) && !(repeated >> s & 1)) put(dz + i[s], f.dense(z[s], rw.c) - f.gq * q[s] - (i[s] == y ? f.gy : 0.0f));
        }
        if (soft && twice) {
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                uint32_t todo = __ballot_sync(kAll, p.holds(i[s], V) && (repeated >> s & 1));
                while (todo) {
                    const int at = __ffs(todo) - 1;
                    todo &= todo - 1;
                    const uint32_t which = __shfl_sync(kAll, i[s], at);
                    // an entry that stands before it sees to the others of its index
                    float sum = 0.0f;
                    bool first = true;
#pragma unroll
                    for (int o = 0; o < kSlots; ++o) {
                        const uint32_t same = __ballot_sync(kAll, i[o] == which);
                        if (o < s) first &= same == 0;
                        if (o == s) first &= (same & ((1u << at) - 1)) == 0;
                        if (i[o] == which) sum += q[o];
                    }
                    if (!first) continue;
                    sum = warp_sum(sum);
                    if ((int)lane == at) put(dz + which, f.dense(z[s], rw.c) - f.gq * sum - (which == y ? f.gy : 0.0f));
                }
            }
        }
        if ((flags & 1u) && !listed && lane == 0) put(dz + y, f.dense(target, rw.c) - f.gy);
    }
};

// TO: the gradient's type, void for the loss alone. EXPS: a logit's
// exponentials. `room` groups of the block's part of a row stay in shared memory;
// what lies behind them is read again.
template <typename TI, typename TO, int EXPS>
__global__ void __launch_bounds__(kMaxThreads, 2) distill_kernel(const DistillArgs a, uint32_t room, uint32_t log2_blocks, float limit, uint32_t* faults) {
    constexpr bool kGrad = !std::is_same<TO, void>::value;
    extern __shared__ uint4 slice[];
    __shared__ Shared<EXPS> sh;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, threads = blockDim.x, dense_threads = threads - kHelpers;
    const uint32_t blocks = 1u << log2_blocks;
    if (threadIdx.x == 0) {
        tc::bar_init(tc::smem_u32(&sh.full[0]), 1);
        tc::bar_init(tc::smem_u32(&sh.full[1]), 1);
        tc::bar_fence_init();
        sh.dead = 0;
    }
    if (blocks > 1) cluster_barrier();  // before another block's records come
    else __syncthreads();
    stream_order();
    Rows<TI> rw{a, blocks > 1 ? cluster_rank() : 0, log2_blocks, room, a.use_soft ? a.ct : kLog2e, a.use_soft ? 1.0f / a.ct : kLn2, limit, blockIdx.x >> log2_blocks, gridDim.x >> log2_blocks};
    const tc::Wait wt{&sh.dead, faults};
    // Waits for the records of the cluster's n-th row and joins them. (Should a
    // wait run out, the rows go on with what is there: nothing else depends on it.)
    auto joined = [&](uint32_t n, Record& r, bool& soft, bool& hard) {
        __syncwarp();
        tc::bar_wait(tc::smem_u32(&sh.full[n & 1]), (n >> 1) & 1, wt);
        r = {-FLT_MAX, 0.0f, 0.0f, 0u, 0.0f, 0.0f, 0.0f, 0.0f};
        if (lane < blocks) r = sh.records[n & 1][lane];
        float bmax = r.max;
        if constexpr (EXPS == kBoth) bmax = lane < blocks ? sh.bases[n & 1][lane].x : bmax;
        soft = __any_sync(kAll, r.flags & 2u);  // (every block says the same)
        hard = __any_sync(kAll, r.flags & 4u);
        return Settled<EXPS>(join<EXPS>({r.max, r.soft, r.hard, bmax}, rw.c, limit), rw.c, rw.inv_c, limit);
    };

    if (threadIdx.x < dense_threads) {
        float weight = rw.weight(rw.row), next_weight = rw.weight(rw.row + rw.step);
        Part<TI> p = rw.part(rw.row);
        float guess = FLT_MAX, guess_b = FLT_MAX;  // none yet
        for (uint32_t l = threadIdx.x, n = rw.kept(p, weight); l < n; l += dense_threads) stage_group(slice, room, p, l, a.V);
        for (uint32_t n = 0; rw.there(rw.row); ++n, rw.row += rw.step) {
            const float after = rw.weight(rw.row + 2 * rw.step);
            const Part<TI> np = rw.part(rw.row + rw.step);
            const uint32_t kept = rw.kept(p, weight), next_kept = rw.kept(np, next_weight);
            Sums s{-FLT_MAX, 0.0f, 0.0f, -FLT_MAX};
            copies_done();
            if (weight != 0.0f) {
                s = sums_of<TI, EXPS, !kGrad>(slice, rw, p, kept, np, next_kept, guess, guess_b, threadIdx.x, dense_threads);
            } else if (!kGrad) {
                for (uint32_t l = threadIdx.x; l < next_kept; l += dense_threads) stage_group(slice, room, np, l, a.V);
            }
            if (lane == 0) {
                sh.sums[warp] = {s.max, s.a, s.b};
                if constexpr (EXPS == kBoth) sh.sum_bases[warp] = s.bmax;
            }
            arrive(kSums, threads);
            Record r;
            bool soft, hard;
            const Settled<EXPS> w = joined(n, r, soft, hard);
            if (w.moved) {  // the next row's
                guess = w.a.max;
                guess_b = w.b.max;
            }
            if constexpr (kGrad) {
                const Factors<EXPS> f(w, soft, hard, weight, a);
                store_dense(static_cast<TO*>(a.dz) + rw.row * a.ldd, slice, rw, f, p, kept, np, next_kept, threadIdx.x, dense_threads);
                arrive(kStored + (n & 1), dense_threads + 32);
            }
            weight = next_weight;
            next_weight = after;
            p = np;
        }
    } else if (threadIdx.x < dense_threads + 32) {  // joins
        for (uint32_t n = 0; rw.there(rw.row); ++n, rw.row += rw.step) {
            const float weight = rw.weight(rw.row);
            wait(kSums, threads);
            const bool some = lane < dense_threads / 32;
            const Three mine = some ? sh.sums[lane] : Three{-FLT_MAX, 0.0f, 0.0f};
            float bmax = mine.max;
            if constexpr (EXPS == kBoth) bmax = some ? sh.sum_bases[lane] : bmax;
            const Sums s = join<EXPS>({mine.max, mine.a, mine.b, bmax}, rw.c, limit);
            const float4 e = sh.entries[n & 1];
            const uint32_t at = tc::smem_u32(&sh.records[n & 1][rw.rank]), bar = tc::smem_u32(&sh.full[n & 1]);
            if (lane == 0) tc::bar_expect(bar, blocks * (uint32_t)(sizeof(Record) + (EXPS == kBoth ? sizeof(float4) : 0)));
            __syncwarp();
            if (lane < blocks) {
                uint32_t to, of;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(lane));
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(of) : "r"(bar), "r"(lane));
                push16(to, of, make_uint4(__float_as_uint(s.max), __float_as_uint(s.a), __float_as_uint(s.b), sh.flags[n & 1]));
                push16(to + 16, of, make_uint4(__float_as_uint(e.x), __float_as_uint(e.y), __float_as_uint(e.z), __float_as_uint(e.w)));
                if constexpr (EXPS == kBoth) {
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(tc::smem_u32(&sh.bases[n & 1][rw.rank])), "r"(lane));
                    push16(to, of, make_uint4(__float_as_uint(s.bmax), 0, 0, 0));
                }
            }
            Record r;
            bool soft, hard;
            const Settled<EXPS> w = joined(n, r, soft, hard);
            if (rw.rank == 0) {
                const float loss = loss_of<EXPS>(r, w, lane < blocks, soft, weight, a, rw.c);
                if (lane == 0) a.loss[rw.row] = soft || hard ? loss : 0.0f;
            }
        }
    } else {  // entries of every second row
        const uint32_t parity = warp - dense_threads / 32 - 1;
        const uint64_t first = rw.row;
        Entries<TI> e;
        if (parity == 1 && rw.there(first)) arrive(kSums, threads);
        rw.row += parity * rw.step;
        e.fetch(rw, rw.row);
        for (uint32_t n = parity; rw.there(rw.row); n += 2, rw.row += 2 * rw.step) {
            const float weight = rw.weight(rw.row);
            const Part<TI> p = rw.part(rw.row);
            float4 own = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (weight != 0.0f) {
                e.gather(rw, rw.row, p);
                own = e.finish(rw, p, sh.table[parity], kGrad);
            } else {
                e.flags = e.repeated = 0;
                e.listed = e.twice = false;
            }
            if (lane == 0) {
                sh.entries[parity] = own;
                sh.flags[parity] = e.flags;
            }
            __syncwarp();
            if (n > 0) tc::bar_wait(tc::smem_u32(&sh.full[(n - 1) & 1]), ((n - 1) >> 1) & 1, wt);  // kSums of that row is over
            arrive(kSums, threads);
            Record r;
            bool soft, hard;
            const Settled<EXPS> w = joined(n, r, soft, hard);
            if (rw.there(rw.row + rw.step)) arrive(kSums, threads);
            if constexpr (kGrad) {
                const Factors<EXPS> f(w, soft, hard, weight, a);
                wait(kStored + parity, dense_threads + 32);
                if (f.some) e.correct(static_cast<TO*>(a.dz) + rw.row * a.ldd, rw, f, p, soft);
            }
            e.fetch(rw, rw.row + 2 * rw.step);
        }
    }
    __syncwarp();
    if (blocks > 1) cluster_barrier();  // no block ends while another's records are on their way to it
}

// ---- more entries ------------------------------------------------------------------

// Every warp has a share of the entries, row by row: no table holds them, and an
// index that stands twice is found by going through the list for each.
template <typename TI, typename TO, int EXPS>
__global__ void __launch_bounds__(kMaxThreads, 2) distill_many_kernel(const DistillArgs a, uint32_t room, uint32_t log2_blocks, float limit, uint32_t*) {
    constexpr bool kGrad = !std::is_same<TO, void>::value;
    extern __shared__ uint4 slice[];
    __shared__ Sums warp_sums[kMaxThreads / 32];
    __shared__ float2 warp_teacher[kMaxThreads / 32], warp_cross[kMaxThreads / 32];
    __shared__ Record records[2];
    __shared__ float bases[2];
    stream_order();
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, threads = blockDim.x, warps = threads / 32;
    const uint32_t blocks = 1u << log2_blocks;
    const Rows<TI> rw{a, blocks > 1 ? cluster_rank() : 0, log2_blocks, room, a.ct, 1.0f / a.ct, limit, blockIdx.x >> log2_blocks, gridDim.x >> log2_blocks};
    uint32_t turn = 0;
    for (uint64_t row = rw.row; rw.there(row); row += rw.step, turn ^= 1) {
        const float weight = rw.weight(row);
        const bool alive = weight != 0.0f;
        const Part<TI> p = rw.part(row);
        const TI* z = rw.logits(row);
        const uint32_t kept = rw.kept(p, weight);
        const int32_t* idx = a.idx + row * a.K;
        const float* t = a.t + row * a.K;
        const uint32_t y = alive && a.use_hard ? (uint32_t)a.targets[row] : kNone;
        for (uint32_t l = threadIdx.x; l < kept; l += threads) stage_group(slice, room, p, l, a.V);
        // log-sum of the entries: largest, and sum over it
        float most = -FLT_MAX, sum = 0.0f;
        if (alive)
            for (uint32_t k = threadIdx.x; k < a.K; k += threads)
                if ((uint32_t)idx[k] < a.V) {
                    const float m = fmaxf(most, t[k]);
                    sum = sum * ex2((most - m) * a.ct) + ex2((t[k] - m) * a.ct);
                    most = m;
                }
        auto join_teacher = [&](float& m, float& v) {
            const float to = warp_max(m);
            v = warp_sum(v * ex2((m - to) * a.ct));
            m = to;
        };
        join_teacher(most, sum);
        copies_done();
        Sums s{-FLT_MAX, 0.0f, 0.0f, -FLT_MAX};
        if (alive) s = sums_of<TI, EXPS, false>(slice, rw, p, kept, p, 0, FLT_MAX, FLT_MAX, threadIdx.x, threads);
        if (lane == 0) {
            warp_sums[warp] = s;
            warp_teacher[warp] = make_float2(most, sum);
        }
        __syncthreads();
        s = join<EXPS>(lane < warps ? warp_sums[lane] : Sums{-FLT_MAX, 0.0f, 0.0f, -FLT_MAX}, rw.c, limit);
        most = lane < warps ? warp_teacher[lane].x : -FLT_MAX;
        sum = lane < warps ? warp_teacher[lane].y : 0.0f;
        join_teacher(most, sum);
        const bool some = !(sum == 0.0f);
        const float inv = 1.0f / sum, log_all = logf(sum);
        auto prob = [&](uint32_t k) { return ex2((t[k] - most) * a.ct) * inv; };
        float cross = 0.0f, mass = 0.0f;
        if (some)
            for (uint32_t k = threadIdx.x; k < a.K; k += threads) {
                const uint32_t i = (uint32_t)idx[k];
                if (!p.holds(i, a.V)) continue;
                const float q = prob(k);
                if (q == 0.0f) continue;
                cross += q * ((t[k] - most) * a.inv_t - log_all - (to_float(z[i]) - s.max) * a.inv_t);
                mass += q;
            }
        cross = warp_sum(cross);
        mass = warp_sum(mass);
        if (lane == 0) warp_cross[warp] = make_float2(cross, mass);
        __syncthreads();
        const bool has = p.holds(y, a.V);
        if (warp == 0) {
            cross = warp_sum(lane < warps ? warp_cross[lane].x : 0.0f);
            mass = warp_sum(lane < warps ? warp_cross[lane].y : 0.0f);
            if (lane == 0) {
                records[turn] = {s.max, s.a, s.b, (uint32_t)has | (some ? 2u : 0u) | (y < a.V ? 4u : 0u), cross, mass, s.max, has ? to_float(z[y]) : 0.0f};
                bases[turn] = s.bmax;
            }
        }
        cluster_barrier();
        Record r{-FLT_MAX, 0.0f, 0.0f, 0u, 0.0f, 0.0f, 0.0f, 0.0f};
        float bmax = r.max;
        if (lane < blocks) {
            const uint32_t at = peer(&records[turn], lane);
            r = {peer_float(at), peer_float(at + 4), peer_float(at + 8), peer_u32(at + 12), peer_float(at + 16), peer_float(at + 20), peer_float(at + 24), peer_float(at + 28)};
            bmax = EXPS == kBoth ? peer_float(peer(&bases[turn], lane)) : r.max;
        }
        const bool hard = y < a.V;
        const Settled<EXPS> w(join<EXPS>({r.max, r.soft, r.hard, bmax}, rw.c, limit), rw.c, rw.inv_c, limit);
        if (rw.rank == 0 && warp == 0) {
            const float loss = loss_of<EXPS>(r, w, lane < blocks, some, weight, a, rw.c);
            if (lane == 0) a.loss[row] = some || hard ? loss : 0.0f;
        }
        if constexpr (kGrad) {
            TO* dz = static_cast<TO*>(a.dz) + row * a.ldd;
            const Factors<EXPS> f(w, some, hard, weight, a);
            store_dense(dz, slice, rw, f, p, kept, p, 0, threadIdx.x, threads);
            __syncthreads();  // the elements below are stored again
            for (uint32_t k = warp; k <= a.K; k += warps) {  // a warp each, the target behind the entries
                if (k == a.K ? !has : !some) continue;
                const uint32_t i = k == a.K ? y : (uint32_t)idx[k];
                if (!p.holds(i, a.V)) continue;
                float q = 0.0f;
                bool first = true;
                for (uint32_t j = lane; some && j < a.K; j += 32) {
                    if ((uint32_t)idx[j] != i) continue;
                    q += prob(j);
                    first &= j >= k;
                }
                if (!__all_sync(kAll, first)) continue;  // an entry before it has seen to it
                q = warp_sum(q);
                if (lane == 0) put(dz + i, f.dense(to_float(z[i]), rw.c) - f.gq * q - (i == y ? f.gy : 0.0f));
            }
            __syncthreads();
        }
    }
    cluster_barrier();  // no block ends while another reads its record
}

// How a row is spread: threads of a block, blocks on an SM, shared memory of a
// block's part of a row. Estimated nanoseconds of a round of rows, fitted to rows
// of 1000 to 267735 in every spread: launching and joining the sums, then 62 bytes of
// logits and gradient a nanosecond on an SM, 16 where the logits are read again.
// (2048 x 267735 bfloat16 with its gradient: three blocks of an SM and eight of a row
// 434 us; two and eight 472, two and four 506. 300 x 60000 bfloat16, the loss alone:
// two of an SM and one of a row 11, three and two 18. One row of 1000: 288 threads a
// block 3.8 us, 1024 5.3, and such blocks were the best nowhere.)
struct Spread {
    uint32_t threads, per_sm, smem;
    double join_ns;
};
constexpr Spread kSpreads[2] = {{512, 2, 104 * 1024, 5500.0}, {288, 3, 66 * 1024, 4500.0}};
constexpr double kBytesNs = 62.0, kAgainNs = 16.0;

template <typename TI, typename TO, int EXPS>
cudaError_t launch(const DistillArgs& a, uint32_t* faults, cudaStream_t s) {
    const uint64_t groups = ((uint64_t)a.V + 14) / 8;  // whatever the row's alignment
    constexpr uint64_t kGroupBytes = 8 * sizeof(TI);
    constexpr double kMoved = kGroupBytes + (std::is_same<TO, void>::value ? 0.0 : std::is_same<TO, float>::value ? 32.0 : 16.0);
    DeviceInfo di{};
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    auto kernel = a.use_soft && a.K > kFew ? distill_many_kernel<TI, TO, EXPS> : distill_kernel<TI, TO, EXPS>;
    double best = 0.0;
    uint32_t blocks = 0, log2_blocks = 0, room = 0, clusters = 0, threads = 0, smem = 0;
    for (const Spread& w : kSpreads) {
        for (uint32_t b = 1, log2 = 0; b <= kMaxBlocks; b *= 2, ++log2) {
            if (b > 1 && groups < b * (uint64_t)w.threads / 2) break;  // too little for so many
            const uint64_t need = (groups + b - 1) / b + 1, most = w.smem / kGroupBytes, keep = need < most ? need : most;
            const uint32_t bytes = (uint32_t)smem_of(keep * kGroupBytes);
            int n = 0;
            e = resident_clusters(reinterpret_cast<const void*>(kernel), w.threads, b, bytes, &n);
            if (e != cudaSuccess) return e;
            if (n < 1) continue;
            const uint64_t rounds = ((uint64_t)a.T + n - 1) / n, all = ((uint64_t)a.T * b + di.sms - 1) / di.sms;
            const double per_sm = (double)(all < w.per_sm ? all : w.per_sm);
            const double ns = (double)rounds * (w.join_ns + per_sm * kMoved * ((double)keep / kBytesNs + (double)(need - keep) / kAgainNs));
            if (blocks && ns >= best) continue;
            best = ns;
            blocks = b;
            log2_blocks = log2;
            room = (uint32_t)keep;
            clusters = (uint32_t)n;
            threads = w.threads;
            smem = bytes;
        }
    }
    if (blocks == 0) return cudaErrorInvalidConfiguration;
    const float c = a.use_soft ? a.ct : kLog2e;
    const float limit = 1e30f / (c > kLog2e ? c : kLog2e);
    const uint32_t grid = (a.T < clusters ? a.T : clusters) * blocks;
    return launch_early(kernel, grid, threads, smem, blocks, s, a, room, log2_blocks, limit, faults);
}

template <typename TI, typename TO>
cudaError_t launch_two(const DistillArgs& a, uint32_t* faults, cudaStream_t s) {
    if (!a.use_soft || !a.use_hard || a.ct == kLog2e) return launch<TI, TO, kOne>(a, faults, s);
    return 2.0f * a.ct == kLog2e ? launch<TI, TO, kSquare>(a, faults, s) : launch<TI, TO, kBoth>(a, faults, s);
}
template <typename TI>
cudaError_t launch_type(const DistillArgs& a, int ddtype, uint32_t* faults, cudaStream_t s) {
    if (!a.dz) return launch_two<TI, void>(a, faults, s);
    return ddtype == 0 ? launch_two<TI, float>(a, faults, s) : launch_two<TI, uint16_t>(a, faults, s);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, int dtype, int ddtype, cudaStream_t s) {
    uint32_t* faults = nullptr;
    const cudaError_t e = tc::wait_fault_word(&faults);
    if (e != cudaSuccess) return e;
    return dtype == 0 ? launch_type<float>(a, ddtype, faults, s) : launch_type<uint16_t>(a, ddtype, faults, s);
}

}  // namespace s2
