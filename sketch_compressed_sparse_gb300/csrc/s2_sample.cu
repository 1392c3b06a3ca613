// The next token of a row of logits from one given random number: temperature,
// top-k, top-p and min-p.
//
// With l_max the row's largest logit a token's weight is exp((l - l_max) / T). In
// the order of the logits (equal ones by index) the three filters each keep a
// beginning, so what is kept is given by one border: the logits above a value,
// and of those equal to it the indices below a limit. The token is the first
// kept index at which the running sum of the kept weights passes u times their
// sum.
//
// Which token that is depends on sums of up to V weights being right to far more
// than a float: among 267,735 tokens of like weight a sum that is off by 2^-24
// of itself moves every third border past its neighbour. A weight is therefore
// computed to about 2^-35 of itself and rounded to a multiple of 2^-43 of the
// largest (fewer bits where V is above 2^19), and weights are added as 64-bit
// integers: sums are exact and do not depend on their order.
//
// A cluster of blocks keeps the row in shared memory (or reads it again where it
// does not fit) and goes over it a few times: for the maximum; for each of top-k
// and top-p a histogram of counts or weights over 512 ranges of logits, one of 512
// parts of the range that holds the border, and a list of the few tokens in that
// part, which are ranked against one another; and for the token the sums of its
// runs of 256 tokens. Where many tokens fall into one part (equal logits, a range
// without end) the border's bits are found nine at a time.
#include <cfloat>

#include "s2_internal.h"
#include "s2_launch.cuh"
#include "s2_rows.cuh"

namespace s2 {
namespace {

using namespace rows;

constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kBins = kRowThreads;   // one per thread
constexpr int kChunks = kRowThreads; // runs of tokens, one per thread
constexpr uint32_t kList = 256;      // tokens that are ranked against one another
constexpr float kPerOctave = 16.0f;  // ranges of logits per factor of two of weight
constexpr int kBits = 43;            // of a weight of 1

// 2^(j/32) * 2^43, rounded
__device__ const uint64_t kRoots[32] = {
    0x80000000000ull, 0x82cd8698ac3ull, 0x85aac367cc5ull, 0x88980e8092eull,
    0x8b95c1e3ea9ull, 0x8ea4398b45dull, 0x91c3d373ab1ull, 0x94f4efa8fefull,
    0x9837f0518dcull, 0x9b8d39b9d55ull, 0x9ef5326091aull, 0xa27043030c5ull,
    0xa5fed6a9b15ull, 0xa9a15ab4ea8ull, 0xad583eea42aull, 0xb123f581d2bull,
    0xb504f333f9eull, 0xb8fbaf47630ull, 0xbd08a39f581ull, 0xc12c4cca667ull,
    0xc5672a11550ull, 0xc9b9bd866e3ull, 0xce248c151f8ull, 0xd2a81d91f13ull,
    0xd744fccad6aull, 0xdbfbb797dafull, 0xe0ccdeec2a9ull, 0xe5b906e77c8ull,
    0xeac0c6e7dd2ull, 0xefe4b99bdceull, 0xf5257d15248ull, 0xfa83b2db723ull,
};

// A row's settings, and what follows from them.
struct Settings {
    float ch, cl;     // log2(e) / temperature, in two floats
    float bins;       // ranges per unit of logit, by weight
    double min_p;     // temperature * log(min_p)
    bool greedy, use_min_p;
    uint32_t top_k;   // 0: off
    float top_p;      // 1: off
    float u;
};

struct Listed {
    float v;
    uint32_t i;
    uint64_t w;
};

struct Shared {
    uint64_t roots[32];
    uint64_t hist[2][kBins];
    Listed list[kList], all[kList];
    uint64_t scan[kRowWarps];
    uint64_t best[2];    // largest logit's key and the complement of its index
    uint32_t finite[2];  // tokens above -infinity
    uint32_t listed;
    uint64_t total;      // weight kept in this block
    uint64_t warp_best[kRowWarps];
    uint32_t warp_finite[kRowWarps];
    Settings set;
    uint64_t before;     // of the bin that was found
    uint32_t bin;
    float border_v;
    uint32_t border_i;
};

// Bits in the order of the numbers; both zeros are one.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// floor(f * z), or the ceiling, for a float f in [0, 1).
__device__ uint64_t times(float f, uint64_t z, bool up) {
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const uint64_t m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const uint32_t s = 150 - (e ? e : 1);  // f = m * 2^-s, 24 < s
    const uint64_t lo = z * m, hi = __umul64hi(z, m);
    uint64_t q = 0;
    bool rest = (lo | hi) != 0;
    if (s < 64) {
        q = lo >> s | hi << (64 - s);  // (24 bits of hi: nothing is lost)
        rest = (lo << (64 - s)) != 0;
    } else if (s < 128) {
        q = hi >> (s - 64);
        rest = lo != 0 || (s > 64 && (hi << (128 - s)) != 0);
    }
    return q + (up && rest);
}

// A row as the blocks of a cluster share it.
template <typename TI, bool STAGED>
struct Row {
    const uint4* slice;
    uint32_t room;
    Part<TI> p;
    uint32_t V;
    uint32_t span;    // 256-token steps per run
    uint32_t chunks;  // runs of this block

    // f(values of eight neighbours) of local group l
    template <typename F>
    __device__ __forceinline__ void one(uint32_t l, F f) const {
        const Raw<TI> r = STAGED ? staged<TI>(slice, room, l) : load_group(p, l, V);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = element(r, j);
        f(v);
    }
    // f(values, local group) for every group of run `chunk` that this lane holds
    template <typename F>
    __device__ __forceinline__ void run(uint32_t chunk, F f) const {
        for (uint32_t s = 0; s < span; ++s) {
            const uint32_t l = (chunk * span + s) * 32 + threadIdx.x % 32;
            if (l < p.count) one(l, [&](const float* v) { f(v, l); });
        }
    }
    // for every group of the block, each once
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        for (uint32_t c = threadIdx.x / 32; c < chunks; c += kRowWarps) run(c, f);
    }
    __device__ __forceinline__ uint32_t index(uint32_t l, int j) const { return (uint32_t)p.index(l, j); }
};

// What is kept: logits above v, and those equal to it with an index below i.
struct Border {
    float v;
    uint32_t i;
    __device__ __forceinline__ bool keeps(float x, uint32_t at) const { return x > v || (x == v && at < i); }
};

// A token's weight, to about 2^-35 of itself. (d, dl) is l - l_max exactly, (y, e)
// that times log2(e) / T, and y = (32 n + j) / 32 + r with |r| <= 1/64, so that
//   2^(y + e) = 2^n * 2^(j/32) * exp(ln 2 * (r + e)).
// Adding a float whose last place is the wanted unit turns a float into a whole
// number of those units. (The products and sums are spelt out so that none is fused.)
struct Weigher {
    const uint64_t* roots;
    float max, ch, cl;
    int shift;  // bits fewer than kBits
    __device__ __forceinline__ uint64_t operator()(float l) const {
        constexpr float kStep32 = 1.5f * 262144.0f;      // last place 2^-5
        constexpr float kStep28 = 1.5f / 32.0f;          // last place 2^-28
        constexpr float kStep35 = 1.5f / 4096.0f;        // last place 2^-35
        constexpr double kLn2 = 0.69314718055994530942;
        constexpr float kLnHi = (float)kLn2, kLnLo = (float)(kLn2 - (double)kLnHi);
        constexpr float c2 = (float)(kLn2 * kLn2 / 2), c3 = (float)(kLn2 * kLn2 * kLn2 / 6),
                        c4 = (float)(kLn2 * kLn2 * kLn2 * kLn2 / 24), c5 = (float)(kLn2 * kLn2 * kLn2 * kLn2 * kLn2 / 120);
        if (max == __uint_as_float(0x7f800000u)) return l == max ? 1ull << (kBits - shift) : 0;
        const float d = __fadd_rn(l, -max);
        const float y = __fmul_rn(d, ch);
        if (!(y > -(float)(kBits + 2))) return 0;  // (-infinity and NaN too)
        const float back = __fadd_rn(d, -l);  // what d took for -max
        const float dl = __fadd_rn(__fadd_rn(l, -__fadd_rn(d, -back)), __fadd_rn(-max, -back));
        const float e = __fmaf_rn(dl, ch, __fmaf_rn(d, cl, __fmaf_rn(d, ch, -y)));
        const float t = __fadd_rn(y, kStep32);
        const int n = __float_as_int(t) - __float_as_int(kStep32);
        const float r = __fadd_rn(y, -__fadd_rn(t, -kStep32));
        const float x = __fadd_rn(r, e);
        const float a = __fmul_rn(r, kLnHi);
        float small = __fmaf_rn(e, kLnHi, __fmaf_rn(r, kLnLo, __fmaf_rn(r, kLnHi, -a)));
        small = __fmaf_rn(__fmul_rn(x, x), __fmaf_rn(x, __fmaf_rn(x, __fmaf_rn(x, c5, c4), c3), c2), small);
        const float ta = __fadd_rn(a, kStep28);
        const float tb = __fadd_rn(__fadd_rn(small, __fadd_rn(a, -__fadd_rn(ta, -kStep28))), kStep35);
        const int q = (__float_as_int(ta) - __float_as_int(kStep28)) * 128 + (__float_as_int(tb) - __float_as_int(kStep35));
        const uint64_t root = roots[n & 31];
        const uint64_t w = root + (uint64_t)(((int64_t)(uint32_t)(root >> 12) * q) >> 23);  // q is in units of 2^-35
        const int s = shift - (n >> 5);
        return s ? (w + (1ull << (s - 1))) >> s : w;
    }
};

__device__ __forceinline__ uint64_t warp_scan(uint64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint64_t u = __shfl_up_sync(kAll, v, o);
        if (threadIdx.x % 32 >= o) v += u;
    }
    return v;
}
// Sum of the values of this thread and those before it; *total: of all.
__device__ __forceinline__ uint64_t block_scan(Shared& sh, uint64_t v, uint64_t* total) {
    v = warp_scan(v);
    __syncthreads();  // the last scan's sums have been read
    if (threadIdx.x % 32 == 31) sh.scan[threadIdx.x / 32] = v;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (uint32_t i = 0; i < kRowWarps; ++i) {
        const uint64_t s = sh.scan[i];
        if (i < threadIdx.x / 32) before += s;
        all += s;
    }
    *total = all;
    return before + v;
}

__device__ __forceinline__ void add64(uint64_t* at, uint64_t v) {
    uint32_t* w = reinterpret_cast<uint32_t*>(at);
    const uint32_t lo = (uint32_t)v, old = atomicAdd(w, lo);
    const uint32_t hi = (uint32_t)(v >> 32) + (old + lo < old);
    if (hi) atomicAdd(w + 1, hi);
}

// Finds the bin in which the sum over the bins of all blocks reaches `target`
// (from 1 to that sum), and takes off what lies before it. bin_of(v) is a
// group's element's bin, or kBins; measure(v) what it counts. `target_of(total)`
// gives the target. The same answer in every block.
template <typename R, typename BinOf, typename Measure, typename TargetOf>
__device__ __forceinline__ uint32_t find_bin(Shared& sh, const R& row, const Border& from, uint32_t& turn, uint32_t blocks, BinOf bin_of,
                                             Measure measure, TargetOf target_of, uint64_t* target) {
    uint64_t* hist = sh.hist[turn++ & 1];
    hist[threadIdx.x] = 0;
    __syncthreads();
    row.each([&](const float* v, uint32_t l) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!from.keeps(v[j], row.index(l, j))) continue;
            const uint32_t b = bin_of(v[j]);
            if (b < kBins) {
                const uint64_t m = measure(v[j]);
                if (m) add64(hist + b, m);
            }
        }
    });
    cluster_barrier();
    uint64_t sum = 0;
    for (uint32_t r = 0; r < blocks; ++r) sum += peer_u64(peer(hist + threadIdx.x, r));
    uint64_t total;
    const uint64_t upto = block_scan(sh, sum, &total);
    const uint64_t goal = target_of(total);
    if (upto >= goal && upto - sum < goal) {
        sh.bin = threadIdx.x;
        sh.before = upto - sum;
    }
    __syncthreads();
    *target = goal - sh.before;
    return sh.bin;
}

// The border of the shortest beginning of what `from` keeps that measures
// target_of(what all of it measures) or more. `scale`: ranges per unit of logit.
template <typename R, typename Measure, typename TargetOf>
__device__ Border narrow(Shared& sh, const R& row, Border from, uint32_t& turn, uint32_t blocks, float top, float scale, Measure measure,
                         TargetOf target_of) {
    uint64_t target;
    auto range = [&](float v) { return fminf((top - v) * scale, (float)(kBins - 1)); };  // larger logits first
    const uint32_t bin = find_bin(sh, row, from, turn, blocks,
                                  [&](float v) { return (uint32_t)__float2int_rn(range(v)); }, measure, target_of, &target);
    auto left = [&](uint64_t) { return target; };
    // a part of the range; the last range has no end
    uint32_t part = kBins;
    auto part_of_range = [&](float v) { return (uint32_t)__float2int_rn(fminf(fmaxf((range(v) - (float)bin + 0.5f) * (kBins - 1), 0.0f), kBins - 1)); };
    auto in_range = [&](float v) { return (uint32_t)__float2int_rn(range(v)) == bin; };
    if (bin < kBins - 1)
        part = find_bin(sh, row, from, turn, blocks, [&](float v) { return in_range(v) ? part_of_range(v) : kBins; }, measure, left, &target);
    auto member = [&](float v) { return in_range(v) && (part == kBins || part_of_range(v) == part); };

    // few: rank them against one another
    if (part < kBins) {
        if (threadIdx.x == 0) sh.listed = 0;
        __syncthreads();
        row.each([&](const float* v, uint32_t l) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t i = row.index(l, j);
                if (!from.keeps(v[j], i) || !member(v[j])) continue;
                const uint32_t at = atomicAdd(&sh.listed, 1u);
                if (at < kList) sh.list[at] = {v[j], i, measure(v[j])};
            }
        });
        cluster_barrier();
        uint32_t n = 0, most = 0;
        for (uint32_t r = 0; r < blocks; ++r) {
            const uint32_t c = peer_u32(peer(&sh.listed, r));
            if (c <= kList && n + c <= kList)
                for (uint32_t k = threadIdx.x; k < c; k += kRowThreads) {
                    const uint32_t at = peer(sh.list + k, r);
                    sh.all[n + k] = {peer_float(at), peer_u32(at + 4), peer_u64(at + 8)};
                }
            n = c > kList || n > kList ? kList + 1 : n + c;
            most = n;
        }
        __syncthreads();
        if (most <= kList) {
            for (uint32_t k = threadIdx.x; k < n; k += kRowThreads) {
                const Listed me = sh.all[k];
                uint64_t before = 0;
                for (uint32_t j = 0; j < n; ++j) {
                    const Listed o = sh.all[j];
                    if (o.v > me.v || (o.v == me.v && o.i < me.i)) before += o.w;
                }
                if (before < target && before + me.w >= target) {
                    sh.border_v = me.v;
                    sh.border_i = me.i + 1;
                }
            }
            __syncthreads();
            const Border b{sh.border_v, sh.border_i};
            __syncthreads();
            return b;
        }
    }
    // many: the border's key, nine bits at a time
    uint32_t prefix = 0;
    constexpr int kShift[4] = {23, 14, 5, 0};
#pragma unroll 1
    for (int s = 0; s < 4; ++s) {
        const int shift = kShift[s], bits = s < 3 ? 9 : 5;
        const uint32_t found = find_bin(sh, row, from, turn, blocks,
                                        [&](float v) {
                                            const uint32_t k = key_of(v);
                                            // (a shift of 32 bits would be none)
                                            if (!member(v) || (s > 0 && k >> (shift + bits) != prefix)) return (uint32_t)kBins;
                                            return ((1u << bits) - 1) - ((k >> shift) & ((1u << bits) - 1));
                                        },
                                        measure, left, &target);
        prefix = prefix << bits | (((1u << bits) - 1) - found);
    }
    // `need` of the equal logits, by index
    const float v = of_key(prefix);
    const uint64_t each = measure(v), need = (target + each - 1) / each;
    uint64_t count = 0;
    for (uint32_t c = threadIdx.x / 32; c < row.chunks; c += kRowWarps) {
        uint32_t mine = 0;
        row.run(c, [&](const float* x, uint32_t l) {
#pragma unroll
            for (int j = 0; j < 8; ++j) mine += x[j] == v && from.keeps(x[j], row.index(l, j));
        });
        mine = __reduce_add_sync(kAll, mine);
        if (threadIdx.x % 32 == 0) sh.hist[turn & 1][c] = mine;
    }
    __syncthreads();
    uint64_t* counts = sh.hist[turn++ & 1];
    count = threadIdx.x < row.chunks ? counts[threadIdx.x] : 0;
    uint64_t total;
    const uint64_t upto = block_scan(sh, count, &total);
    if (threadIdx.x == 0) {
        sh.total = total;
        sh.border_i = 0;
    }
    cluster_barrier();
    uint64_t before = 0;
    for (uint32_t r = 0; r < cluster_rank(); ++r) before += peer_u64(peer(&sh.total, r));
    const uint64_t want = need > before ? need - before : 0;  // of this block
    if (want > upto - count && want <= upto) {
        sh.bin = threadIdx.x;
        sh.before = want - (upto - count);
    }
    __syncthreads();
    if (want > 0 && want <= total && threadIdx.x < 32) {
        uint64_t seen = 0;
        const uint64_t goal = sh.before;
        // (every lane of the warp takes every step)
        for (uint32_t s = 0; s < row.span; ++s) {
            const uint32_t l = (sh.bin * row.span + s) * 32 + threadIdx.x;
            uint32_t hit = 0;
            if (l < row.p.count) {
                row.one(l, [&](const float* x) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) hit |= (uint32_t)(x[j] == v && from.keeps(x[j], row.index(l, j))) << j;
                });
            }
            const uint64_t mine = warp_scan((uint64_t)__popc(hit));
            const uint64_t first = seen + mine - __popc(hit);
            if (goal > first && goal <= first + __popc(hit)) {
                uint32_t k = (uint32_t)(goal - first);
                for (int j = 0; j < 8; ++j)
                    if (hit >> j & 1 && --k == 0) sh.border_i = row.index(l, j) + 1;
            }
            seen += __shfl_sync(kAll, mine, 31);
        }
    }
    cluster_barrier();
    // one block has found it
    uint32_t i = 0;
    for (uint32_t r = 0; r < blocks; ++r) i = max(i, peer_u32(peer(&sh.border_i, r)));
    cluster_barrier();  // read by all before it is written again
    return {v, i};
}

template <typename TI, bool STAGED>
__global__ void __launch_bounds__(kRowThreads, 2) sample_kernel(const SampleArgs a, uint32_t room, uint32_t log2_blocks, int shift) {
    extern __shared__ uint4 slice[];
    __shared__ Shared sh;
    stream_order();
    const uint32_t blocks = 1u << log2_blocks, rank = cluster_rank();
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x < 32) sh.roots[threadIdx.x] = kRoots[threadIdx.x];
    uint32_t turn = 0, parity = 0;
    for (uint64_t at = blockIdx.x / blocks; at < a.T; at += gridDim.x >> log2_blocks, parity ^= 1) {
        Row<TI, STAGED> row;
        row.slice = slice;
        row.room = room;
        row.p = part_of(static_cast<const TI*>(a.z) + at * a.ld, a.V, rank, log2_blocks);
        row.V = a.V;
        row.span = (row.p.count + 32 * kChunks - 1) / (32 * kChunks);
        if (row.span == 0) row.span = 1;
        row.chunks = (row.p.count + 32 * row.span - 1) / (32 * row.span);
        if (STAGED) stage(slice, room, row.p, a.V, threadIdx.x, kRowThreads);
        if (threadIdx.x == kRowThreads - 1) {
            Settings s;
            const float t = a.temperature ? a.temperature[at] : 1.0f;
            s.greedy = !(t >= FLT_MIN);
            const double c = 1.4426950408889634074 / (double)t;
            s.ch = (float)c;
            s.cl = (float)(c - (double)s.ch);
            s.bins = kPerOctave * s.ch;
            s.top_k = a.top_k && a.top_k[at] > 0 ? (uint32_t)a.top_k[at] : 0;
            const float p = a.top_p ? a.top_p[at] : 1.0f;
            s.top_p = p < 1.0f ? fmaxf(p, 0.0f) : 1.0f;
            const float m = a.min_p ? a.min_p[at] : 0.0f;
            s.use_min_p = m > 0.0f;
            s.min_p = s.use_min_p ? (double)t * log((double)fminf(m, 1.0f)) : 0.0;
            const float u = a.u[at];
            s.u = u > 0.0f ? fminf(u, 1.0f - FLT_EPSILON / 2) : 0.0f;
            sh.set = s;
        }
        if (STAGED) copies_done();

        // the largest logit, the first of equals; how many tokens there are
        uint64_t best = 0;
        uint32_t finite = 0;
        row.each([&](const float* v, uint32_t l) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!(v[j] > minus_inf())) continue;
                ++finite;
                const uint64_t k = (uint64_t)key_of(v[j]) << 32 | (uint32_t)~row.index(l, j);
                best = k > best ? k : best;
            }
        });
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(kAll, best, o);
            best = other > best ? other : best;
        }
        finite = __reduce_add_sync(kAll, finite);
        if (lane == 0) {
            sh.warp_best[warp] = best;
            sh.warp_finite[warp] = finite;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (uint32_t w = 1; w < kRowWarps; ++w) {
                best = sh.warp_best[w] > best ? sh.warp_best[w] : best;
                finite += sh.warp_finite[w];
            }
            sh.best[parity] = best;
            sh.finite[parity] = finite;
        }
        cluster_barrier();
        best = 0;
        finite = 0;
        for (uint32_t r = 0; r < blocks; ++r) {
            const uint64_t b = peer_u64(peer(&sh.best[parity], r));
            best = b > best ? b : best;
            finite += peer_u32(peer(&sh.finite[parity], r));
        }
        const Settings set = sh.set;
        const bool first = finite == 0 || set.greedy || set.top_k == 1 || set.top_p == 0.0f;
        if (first) {  // nothing to draw; the same in every block
            if (rank == 0 && threadIdx.x == 0) a.tokens[at] = finite ? (int32_t)~(uint32_t)best : -1;
            __syncthreads();
            continue;
        }
        const float max = of_key((uint32_t)(best >> 32));
        const Weigher weigh{sh.roots, max, set.ch, set.cl, shift};
        Border border{minus_inf(), 0};
        if (set.top_k && set.top_k < finite)
            border = narrow(sh, row, border, turn, blocks, max, kPerOctave * 1.44269504f, [](float) { return (uint64_t)1; },
                            [&](uint64_t) { return (uint64_t)set.top_k; });
        if (set.top_p < 1.0f)
            border = narrow(sh, row, border, turn, blocks, max, set.bins, weigh, [&](uint64_t total) {
                const uint64_t goal = times(set.top_p, total, true);
                return goal ? goal : 1;
            });
        if (set.use_min_p) {  // weight >= min_p: l >= l_max + T log(min_p), from the next float on
            const double least = (double)max + set.min_p;
            float f = (float)least;
            if ((double)f < least) f = of_key(key_of(f) + 1);
            const uint32_t k = key_of(f) - 1;
            const float below = of_key(k == 0x7fffffffu ? k - 1 : k);  // (that key would be the other zero)
            if (below > border.v || (below == border.v && border.i > 0)) border = {below, 0};
        }

        // the sums of this block's runs
        for (uint32_t c = warp; c < row.chunks; c += kRowWarps) {
            uint64_t w = 0;
            row.run(c, [&](const float* v, uint32_t l) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (border.keeps(v[j], row.index(l, j))) w += weigh(v[j]);
            });
#pragma unroll
            for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(kAll, w, o);
            if (lane == 0) sh.hist[turn & 1][c] = w;
        }
        __syncthreads();
        const uint64_t mine = threadIdx.x < row.chunks ? sh.hist[turn & 1][threadIdx.x] : 0;
        ++turn;
        uint64_t total;
        const uint64_t upto = block_scan(sh, mine, &total);
        if (threadIdx.x == 0) sh.total = total;
        cluster_barrier();
        uint64_t before = 0, all = 0;
        for (uint32_t r = 0; r < blocks; ++r) {
            const uint64_t t = peer_u64(peer(&sh.total, r));
            if (r < rank) before += t;
            all += t;
        }
        const uint64_t goal = times(set.u, all, false);  // the token: the first whose running sum passes it
        const bool here = goal >= before && goal - before < total;
        if (here && goal - before >= upto - mine && goal - before < upto) {
            sh.bin = threadIdx.x;
            sh.before = goal - before - (upto - mine);
        }
        __syncthreads();
        if (here && warp == 0) {
            uint64_t seen = 0;
            const uint64_t left = sh.before;
            for (uint32_t s = 0; s < row.span; ++s) {
                const uint32_t l = (sh.bin * row.span + s) * 32 + lane;
                uint64_t w[8], sum = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 0;
                if (l < row.p.count)
                    row.one(l, [&](const float* v) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            w[j] = border.keeps(v[j], row.index(l, j)) ? weigh(v[j]) : 0;
                            sum += w[j];
                        }
                    });
                const uint64_t scan = warp_scan(sum);
                uint64_t run = seen + scan - sum;
                if (left >= run && left < run + sum) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (left >= run && left < run + w[j]) a.tokens[at] = (int32_t)row.index(l, j);
                        run += w[j];
                    }
                }
                seen += __shfl_sync(kAll, scan, 31);
            }
        }
        __syncthreads();  // the slice and the sums are free
    }
    cluster_barrier();  // no block ends while another reads its shared memory
}

template <typename TI>
cudaError_t launch(const SampleArgs& a, cudaStream_t s) {
    DeviceInfo di{};
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    const uint64_t groups = ((uint64_t)a.V + 14) / 8;  // whatever the row's alignment
    constexpr uint64_t kGroupBytes = 8 * sizeof(TI);
    // as many blocks as let a few of them share an SM, more where the rows do not fill the GPU
    uint32_t blocks = 1;
    while (blocks < 16 && groups * kGroupBytes > blocks * 80ull * 1024) blocks *= 2;
    while (blocks < 16 && (uint64_t)a.T * blocks * 2 <= (uint64_t)di.sms * 2 && groups >= blocks * 2ull * kRowThreads) blocks *= 2;
    auto kernel = sample_kernel<TI, false>;
    size_t smem = 0;
    uint32_t room = 0;
    int clusters = 0;
    for (;; blocks /= 2) {
        const uint64_t need = (groups + blocks - 1) / blocks + 1;
        const bool fits = smem_of(need * kGroupBytes) <= kRowSmem && need <= 32ull * kChunks;
        kernel = fits ? sample_kernel<TI, true> : sample_kernel<TI, false>;
        room = fits ? (uint32_t)need : 0;
        smem = fits ? smem_of(need * kGroupBytes) : 0;
        e = resident_clusters(reinterpret_cast<const void*>(kernel), kRowThreads, blocks, smem, &clusters);
        if (e != cudaSuccess) return e;
        if (clusters > 0 || blocks == 1) break;
    }
    uint32_t log2_blocks = 0;
    while ((1u << log2_blocks) < blocks) ++log2_blocks;
    int shift = 0;  // sums of V weights stay below 2^63
    while ((1ull << (62 - kBits + shift)) < a.V) ++shift;
    const uint64_t most = 0x7fffffffull / 16;
    const uint32_t grid = (uint32_t)(a.T < most ? a.T : most) * blocks;
    return launch_early(kernel, grid, kRowThreads, smem, blocks, s, a, room, log2_blocks, shift);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int dtype, cudaStream_t s) {
    return dtype == 0 ? launch<float>(a, s) : launch<uint16_t>(a, s);
}

}  // namespace s2
