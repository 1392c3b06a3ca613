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
// integers: sums are exact and do not depend on their order. A token below half
// of that unit weighs 0 and is not drawn, not even with u = 0: among the words of a
// row at a low temperature most are like that, and no user means one of them.
//
// A cluster of blocks keeps the row in shared memory (what does not fit is read
// again) and goes over it a few times: for the maximum; for each of top-k and
// top-p a histogram of counts or weights over 256 ranges of logits, one of 256
// parts of the range that holds the border, and a list of the few tokens in that
// part, which are ranked against one another; and for the token the sums of its
// runs of tokens. Where many tokens fall into one part (equal logits, a range
// without end) the border's bits are found eight at a time. The passes behind the
// first ones look at the largest of eight neighbours and leave most of them alone.
//
// Few rows are bound by the passes' barriers (a cluster's takes 1 to 2 us), many by
// instructions: a weight takes about 35, where a row that nothing filters weighs
// each token once and top-p with every token twice. Measured: a row of 33278
// bfloat16 with top-p 20 us; 24 rows of 267735 float32 of all kinds of settings 62 to
// 81, by what the settings are, 256 rows 378 to 385; of 256 rows 113 the largest
// alone, 141 with min-p, 270 with no filter, 247 with top-k 50, 460 with top-k 1000 and
// top-p, 739 with top-p alone (460 at temperature 0.6). To read them takes 41. (Two fifths of the issue slots are used; exact
// ends of ranges as floats, found once, spare top-p alone 10 % and cost every row
// with top-k and every single row more.)
#include <cfloat>

#include "s2_internal.h"
#include "s2_launch.cuh"
#include "s2_rows.cuh"

namespace s2 {
namespace {

using namespace rows;

constexpr uint32_t kThreads = 384;
constexpr uint32_t kPerSm = 2;      // blocks
constexpr uint32_t kBins = 256;     // a thread each
constexpr uint32_t kList = 128;     // tokens that are ranked against one another
constexpr uint32_t kQueue = 768;    // groups that a pass over few of them takes
constexpr float kPerOctave = 8.0f;  // ranges of logits per factor of two of weight
constexpr int kBits = 43;           // of a weight of 1
static_assert(kBins <= kThreads && kList <= kThreads, "a thread for each");

// 2^(j/32) in two floats
__device__ const float2 kRoots[32] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}, {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f},
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
};

struct Shared {
    float2 roots[32];
    uint64_t hist[2][kBins];
    Listed list[kList];
    union {
        struct {
            Listed all[kList];
            uint64_t weight[kList];
        };
        uint32_t queue[kQueue];  // groups that a pass looks into
        float picked[kThreads / 32][64];
    };
    uint32_t queued;
    uint64_t scan[kThreads / 32];
    float warp_max[kThreads / 32];
    float top[2];        // this block's largest logit
    uint32_t lowest[2];  // the lowest index of the row's largest
    uint32_t listed, lowest_key, highest_key;  // of the tokens that are ranked
    uint64_t total;      // weight kept in this block
    Settings set[2];     // of this row and the next
    uint64_t before, inside;  // of the bin that was found
    uint32_t bin;
    Listed border;
};

// Bits in the order of the numbers; both zeros are one.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// The nearest whole number of a float from 0 to 2^22 (adding 1.5 * 2^23 leaves it in
// the low bits; the conversion takes four times as long).
__device__ __forceinline__ uint32_t whole_of(float v) { return (uint32_t)(__float_as_int(__fadd_rn(v, 12582912.0f)) - 0x4b400000); }

// floor(f * z), or the ceiling, for a float f in [0, 1).
__device__ uint64_t times(float f, uint64_t z, bool up) {
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const uint64_t m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const uint32_t s = 150 - (e ? e : 1);  // f = m * 2^-s, 24 <= s
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

// What is kept: logits above v, and those equal to it with an index below i.
struct Border {
    float v;
    uint32_t i;
    __device__ __forceinline__ bool keeps(float x, uint32_t at) const { return (x > v) | ((x == v) & (at < i)); }
};

// A row as the blocks of a cluster share it.
template <typename TI>
struct Row {
    const uint4* slice;
    uint32_t room, kept;  // groups of the block's part in shared memory
    Part<TI> p;
    uint32_t V;
    uint32_t size;    // groups of a run
    uint32_t chunks;  // runs of this block, at most kBins

    __device__ __forceinline__ Raw<TI> group(uint32_t l) const { return l < kept ? staged<TI>(slice, room, l) : load_group(p, l, V); }
    // f(group, local index) for every group of the block, each once
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll 2
        for (uint32_t l = threadIdx.x; l < kept; l += kThreads) f(staged<TI>(slice, room, l), l);
        uint32_t l = threadIdx.x;
        if (l < kept) l += (kept - l + kThreads - 1) / kThreads * kThreads;
        for (; l < p.count; l += kThreads) f(load_group(p, l, V), l);
    }
    // Queues the groups that hold a logit above `least` or equal to it; their
    // number, more than kQueue where not all have a place. All threads, behind a
    // barrier.
    template <typename S>
    __device__ __forceinline__ uint32_t queue_up(S& sh, float least) const {
        if (threadIdx.x == 0) sh.queued = 0;
        __syncthreads();
        const uint32_t lane = threadIdx.x % 32;
#pragma unroll 2
        for (uint32_t first = threadIdx.x - lane; first < p.count; first += kThreads) {
            const uint32_t l = first + lane;
            const bool hit = l < p.count && group_max(group(l)) >= least;
            const uint32_t hits = __ballot_sync(kAll, hit);
            if (!hits) continue;
            uint32_t at = 0;
            if (lane == 0) at = atomicAdd(&sh.queued, (uint32_t)__popc(hits));
            at = __shfl_sync(kAll, at, 0);
            if (at > kQueue) break;  // too many already
            at += __popc(hits & ((1u << lane) - 1));
            if (hit && at < kQueue) sh.queue[at] = l;
        }
        __syncthreads();
        return sh.queued;
    }
    // f(group, local index) for every group that holds a logit above `least` or
    // equal to it. Where they are few, most lanes of a warp would wait for one that
    // looks into its group: such groups are queued first, and every thread takes its
    // own from the queue. `all`: there are no few. All threads, behind a barrier.
    template <typename S, typename F>
    __device__ __forceinline__ void above(S& sh, float least, bool all, F f) const {
        bool direct = all || p.count <= kThreads;
        uint32_t n = direct ? 0 : queue_up(sh, least);
        if (n > kQueue) direct = true;
        if (direct) n = p.count;
        for (uint32_t q = threadIdx.x; q < n; q += kThreads) {
            const uint32_t l = direct ? q : sh.queue[q];
            const Raw<TI> r = group(l);
            if (!direct || group_max(r) >= least) f(r, l);
        }
    }
    // f(logit) for every one of the block's for which pick(logit, index) holds, all of
    // them at `least` or above: where they are some in a hundred and f takes long, 32
    // are collected at a time. All threads.
    template <typename S, typename Pick, typename F>
    __device__ __forceinline__ void picked(S& sh, float least, Pick pick, F f) const {
        const uint32_t lane = threadIdx.x % 32;
        float* mine = sh.picked[threadIdx.x / 32];
        uint32_t n = 0;
        for (uint32_t first = threadIdx.x - lane; first < p.count; first += kThreads) {
            const uint32_t l = first + lane;
            Raw<TI> r{};
            uint32_t here = 0;
            if (l < p.count) {
                r = group(l);
                if (group_max(r) >= least) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) here |= (uint32_t)pick(element(r, j), index(l, j)) << j;
                }
            }
            if (!__any_sync(kAll, here)) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool hit = here >> j & 1;
                const uint32_t hits = __ballot_sync(kAll, hit);
                if (hit) mine[n + __popc(hits & ((1u << lane) - 1))] = element(r, j);
                n += __popc(hits);
                if (n < 32) continue;
                __syncwarp();
                f(mine[lane]);
                const float rest = mine[32 + lane];
                __syncwarp();
                n -= 32;
                if (lane < n) mine[lane] = rest;
            }
        }
        __syncwarp();
        if (lane < n) f(mine[lane]);
    }
    // The lane's groups of run `chunk`: f(local index) for lane, lane + 32, ..., in as
    // many steps for every lane; the index is past the block's groups where there is none.
    template <typename F>
    __device__ __forceinline__ void run(uint32_t chunk, F f) const {
        for (uint32_t s = 0; s < size; s += 32) {
            const uint32_t i = s + threadIdx.x % 32, l = chunk * size + i;
            f(i < size && l < p.count ? l : 0xffffffffu);
        }
    }
    __device__ __forceinline__ uint32_t index(uint32_t l, int j) const { return (uint32_t)p.index(l, j); }
};

// Weights, to about 2^-35 of themselves. (D, Dl) is l_max - l exactly, (PY, -e)
// that times log2(e) / T, and -PY = (32 n + j) / 32 - R with |R| <= 1/64, so that
//   2^(-PY + e) = 2^n * 2^(j/32) * exp(ln 2 * (e - R)).
// Adding a float whose last place is the wanted unit turns a float into a whole
// number of those units: a weight is hi * 2^-22 + lo * 2^-43. Two tokens at a time.
// (Products and sums are single instructions: none is fused into another.)
struct Weigher {
    const float2* roots;
    float max, ch, cl;
    int shift;  // bits fewer than kBits
    float none;  // down to it weights are below 2^-40

    __device__ __forceinline__ void pair(float l0, float l1, int* hi, int* lo) const {
        constexpr float kStep32 = 1.5f * 262144.0f;   // last place 2^-5
        constexpr float kStep22 = 3.0f;               // last place 2^-22
        constexpr float kStep43 = 1.5f / 1048576.0f;  // last place 2^-43
        constexpr double kLn2 = 0.69314718055994530942;
        constexpr float kLnHi = (float)kLn2, kLnLo = (float)(kLn2 - (double)kLnHi);
        constexpr float c2 = (float)(kLn2 * kLn2 / 2), c3 = (float)(kLn2 * kLn2 * kLn2 / 6),
                        c4 = (float)(kLn2 * kLn2 * kLn2 * kLn2 / 24), c5 = (float)(kLn2 * kLn2 * kLn2 * kLn2 * kLn2 / 120);
        auto both = [](float v) { return two(v, v); };
        const Two minus = both(-1.0f), M = both(max);
        // (what is not kept, NaN and -infinity among it, is moved to where it does no harm)
        const Two l = two(fmaxf(l0, none), fmaxf(l1, none));
        const Two D = fma2(l, minus, M), back = add2(D, both(-max));
        const Two Dl = fma2(add2(l, back), minus, fma2(fma2(back, minus, D), minus, M));
        const Two PY = mul2(D, both(ch));
        const Two e = fma2(Dl, both(-ch), fma2(D, both(-cl), fma2(D, both(-ch), PY)));
        const Two t = fma2(PY, minus, both(kStep32));
        const Two R = add2(PY, add2(t, both(-kStep32)));
        const Two na = mul2(R, both(kLnHi)), a = mul2(R, both(-kLnHi)), x = fma2(R, minus, e);
        Two small = fma2(e, both(kLnHi), fma2(R, both(-kLnLo), fma2(R, both(-kLnHi), na)));
        small = fma2(mul2(x, x), fma2(x, fma2(x, fma2(x, both(c5), both(c4)), both(c3)), both(c2)), small);
        const float2 ft = apart(t);
        const int n0 = __float_as_int(ft.x) - __float_as_int(kStep32), n1 = __float_as_int(ft.y) - __float_as_int(kStep32);
        const float2 r0 = roots[n0 & 31], r1 = roots[n1 & 31];
        const Two by = two(__int_as_float(((n0 >> 5) + 127 - shift) << 23), __int_as_float(((n1 >> 5) + 127 - shift) << 23));
        const Two root = mul2(two(r0.x, r1.x), by), rest = mul2(two(r0.y, r1.y), by);
        const Two p = mul2(root, a), pe = fma2(root, a, mul2(root, na)), s = add2(root, p);
        const Two wl = add2(add2(fma2(rest, a, fma2(root, small, pe)), rest), fma2(fma2(root, minus, s), minus, p));
        const Two v = add2(s, wl), under = fma2(fma2(s, minus, v), minus, wl);
        const Two th = add2(v, both(kStep22));
        const Two tl = add2(add2(fma2(add2(th, both(-kStep22)), minus, v), under), both(kStep43));
        const float2 h = apart(th), w = apart(tl);
        hi[0] = __float_as_int(h.x) - __float_as_int(kStep22);
        hi[1] = __float_as_int(h.y) - __float_as_int(kStep22);
        lo[0] = __float_as_int(w.x) - __float_as_int(kStep43);
        lo[1] = __float_as_int(w.y) - __float_as_int(kStep43);
    }
    __device__ __forceinline__ static uint64_t whole(int hi, int lo) { return (uint64_t)(((int64_t)hi << 21) + lo); }
    // A weight by itself, of a logit that is not below `none`.
    __device__ __noinline__ uint64_t operator()(float l) const {
        if (max == __uint_as_float(0x7f800000u)) return l == max ? 1ull << (kBits - shift) : 0;
        int hi[2], lo[2];
        pair(l, l, hi, lo);
        return whole(hi[0], lo[0]);
    }
    // Of a group: f(element, its number, weight), a weight of 0 where use(element, number) does not hold.
    template <typename TI, typename Use, typename F>
    __device__ __forceinline__ void group(const Raw<TI>& r, Use use, F f) const {
        if (max == __uint_as_float(0x7f800000u)) {
#pragma unroll 1
            for (int j = 0; j < 8; ++j)
                if (use(element(r, j), j)) f(element(r, j), j, (*this)(element(r, j)));
            return;
        }
        int hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) pair(element(r, j), element(r, j + 1), hi + j, lo + j);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f(element(r, j), j, use(element(r, j), j) ? whole(hi[j], lo[j]) : 0);
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
    const uint64_t mine = threadIdx.x % 32 < kThreads / 32 ? sh.scan[threadIdx.x % 32] : 0, upto = warp_scan(mine);
    *total = __shfl_sync(kAll, upto, 31);
    const uint64_t before = __shfl_sync(kAll, upto - mine, threadIdx.x / 32);
    return before + v;
}

// Adds to a sum in shared memory, nothing where v is 0. (No branches: most lanes add.)
__device__ __forceinline__ void add64(uint64_t* at, uint64_t v) {
    asm volatile(
        "{.reg .pred p; .reg .u32 lo, hi, old, sum;\n"
        "mov.b64 {lo, hi}, %1;\n"
        "setp.ne.u32 p, lo, 0;\n"
        "mov.u32 old, 0;\n"
        "@p atom.shared.add.u32 old, [%0], lo;\n"
        "add.cc.u32 sum, old, lo;\n"
        "addc.u32 hi, hi, 0;\n"
        "setp.ne.u32 p, hi, 0;\n"
        "@p red.shared.add.u32 [%0 + 4], hi;}" ::"r"((uint32_t)__cvta_generic_to_shared(at)),
        "l"(v)
        : "memory");
}
__device__ __forceinline__ void count32(uint64_t* at, uint32_t v) {  // (a block has fewer than 2^32)
    asm volatile(
        "{.reg .pred p; setp.ne.u32 p, %1, 0;\n"
        "@p red.shared.add.u32 [%0], %1;}" ::"r"((uint32_t)__cvta_generic_to_shared(at)),
        "r"(v)
        : "memory");
}

// What a row's threads share and agree on.
template <typename TI>
struct Team {
    Shared& sh;
    const Row<TI>& row;
    uint32_t blocks, rank;
    float top;  // the row's largest logit
    uint32_t& turn;

    // Finds the bin in which the sum over the bins of all blocks reaches the goal
    // goal_of(total), from 1 to that sum; *goal: what is left of it in that bin,
    // *inside: what lies in it. fill(hist) adds this block's part. The same answer in
    // every block.
    template <typename Fill, typename GoalOf>
    __device__ __forceinline__ uint32_t find_bin(Fill fill, GoalOf goal_of, uint64_t* goal, uint64_t* inside = nullptr) const {
        uint64_t* hist = sh.hist[turn++ & 1];
        if (threadIdx.x < kBins) hist[threadIdx.x] = 0;
        __syncthreads();
        fill(hist);
        cluster_barrier();
        const uint64_t sum = threadIdx.x < kBins ? sum_of_blocks(hist + threadIdx.x, blocks) : 0;
        uint64_t total;
        const uint64_t upto = block_scan(sh, sum, &total);
        const uint64_t want = goal_of(total);
        if (upto >= want && upto - sum < want) {
            sh.bin = threadIdx.x;
            sh.before = upto - sum;
            sh.inside = sum;
        }
        __syncthreads();
        *goal = want - sh.before;
        if (inside) *inside = sh.inside;
        return sh.bin;
    }
    // The sum of the blocks' totals, and of those before this one. (A lane reads a block's.)
    __device__ __forceinline__ void totals(uint64_t* before, uint64_t* all) const {
        const uint32_t lane = threadIdx.x % 32;
        const uint64_t mine = lane < blocks ? peer_u64(peer(&sh.total, lane)) : 0;
        uint64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 16; o *= 2) {
            const uint64_t u = __shfl_up_sync(kAll, upto, o);
            if (lane >= o) upto += u;
        }
        *all = __shfl_sync(kAll, upto, 15);
        *before = __shfl_sync(kAll, upto - mine, rank);
    }
};

// How tokens are measured: counted, or weighed.
struct Count {
    static constexpr bool kWeighed = false;
    __device__ __forceinline__ uint64_t operator()(float) const { return 1; }
    template <typename TI, typename Use, typename F>
    __device__ __forceinline__ void group(const Raw<TI>& r, Use use, F f) const {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f(element(r, j), j, (uint64_t)use(element(r, j), j));
    }
};
struct Weigh : Weigher {
    static constexpr bool kWeighed = true;
};
template <typename Measure>
__device__ __forceinline__ void count_in(uint64_t* at, uint64_t m) {
    if (Measure::kWeighed) add64(at, m);
    else count32(at, (uint32_t)m);
}

// A float not above any logit of range `bin` or one before it: that range ends half a
// range on, and a difference is rounded by 2^-24 of the larger of its numbers.
__device__ __forceinline__ float below_range(float top, uint32_t bin, float scale) {
    const float by = ((float)bin + 0.75f) / scale;
    return (top - by) - (fabsf(top) + by) * 0x1p-21f;
}

// The border of the shortest beginning of what `from` keeps that measures
// goal_of(what all of it measures) or more. `scale`: ranges per unit of logit.
// `least`: no token below it belongs to that beginning. `kept_most`: `from` keeps
// no more tokens than this (so few that they are all ranked). `dense`: it keeps
// most of them.
template <typename TI, typename Measure, typename GoalOf>
__device__ Border narrow(const Team<TI>& team, Border from, float scale, float least, uint64_t kept_most, bool dense, const Measure& measure, GoalOf goal_of) {
    Shared& sh = team.sh;
    const Row<TI>& row = team.row;
    const float top = team.top;
    uint64_t goal = 0, inside = 0;
    const bool rank_all = kept_most <= kList;
    auto range = [&](float v) { return fminf((top - v) * scale, (float)(kBins - 1)); };  // larger logits first
    auto range_of = [&](float v) { return whole_of(range(v)); };
    auto kept = [&](uint32_t l) { return [&row, &from, l](float v, int j) { return from.keeps(v, row.index(l, j)); }; };
    uint32_t bin = 0;
    if (!rank_all)
        bin = team.find_bin(
            [&](uint64_t* hist) {
                row.above(sh, fmaxf(least, from.v), dense, [&](const Raw<TI>& r, uint32_t l) {
                    measure.group(r, kept(l), [&](float v, int, uint64_t m) { count_in<Measure>(hist + range_of(v), m); });
                });
            },
            goal_of, &goal, &inside);
    auto left = [&](uint64_t) { return goal; };
    // a part of the range; the last range has no end
    uint32_t part = kBins;
    auto part_of_range = [&](float v) { return whole_of(fminf(fmaxf((range(v) - (float)bin + 0.5f) * (kBins - 1), 0.0f), kBins - 1)); };
    const float low = bin < kBins - 1 && !rank_all ? fmaxf(from.v, below_range(top, bin, scale)) : from.v;
    const bool few = rank_all || (!Measure::kWeighed && inside <= kList);
    if (bin < kBins - 1 && !few)
        part = team.find_bin(
            [&](uint64_t* hist) {
                auto in_bin = [&](float v, uint32_t i) { return from.keeps(v, i) & (range_of(v) == bin); };
                auto add = [&](float v) { count_in<Measure>(hist + part_of_range(v), measure(v)); };
                row.picked(sh, low, in_bin, add);
            },
            left, &goal);
    auto member = [&](float v) { return rank_all | ((range_of(v) == bin) & ((part == kBins) | (part_of_range(v) == part))); };

    // few: rank them against one another
    if (part < kBins || few) {
        if (rank_all) cluster_barrier();  // the last list has been read by all (else find_bin saw to it)
        if (threadIdx.x == 0) {
            sh.listed = 0;
            sh.lowest_key = 0xffffffffu;
            sh.highest_key = 0;
        }
        __syncthreads();
        uint32_t lowest = 0xffffffffu, highest = 0;
        row.above(sh, low, false, [&](const Raw<TI>& r, uint32_t l) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = element(r, j);
                const uint32_t i = row.index(l, j);
                if (!(from.keeps(v, i) & member(v))) continue;
                const uint32_t at = atomicAdd(&sh.listed, 1u), k = key_of(v);
                if (at < kList) sh.list[at] = {v, i};
                lowest = min(lowest, k);
                highest = max(highest, k);
            }
        });
        lowest = __reduce_min_sync(kAll, lowest);
        highest = __reduce_max_sync(kAll, highest);
        if (threadIdx.x % 32 == 0 && lowest <= highest) {
            atomicMin(&sh.lowest_key, lowest);
            atomicMax(&sh.highest_key, highest);
        }
        cluster_barrier();
        // each warp takes some blocks' lists to their places behind one another
        const uint32_t lane = threadIdx.x % 32, c = min(lane < team.blocks ? peer_u32(peer(&sh.listed, lane)) : 0, kList + 1);
        uint32_t upto = c;
#pragma unroll
        for (int o = 1; o < 16; o *= 2) {
            const uint32_t u = __shfl_up_sync(kAll, upto, o);
            if (lane >= o) upto += u;
        }
        const uint32_t n = __shfl_sync(kAll, upto, 15);
        if (n <= kList)
            for (uint32_t r = threadIdx.x / 32; r < team.blocks; r += kThreads / 32) {
                const uint32_t many = __shfl_sync(kAll, c, r), first = __shfl_sync(kAll, upto - c, r);
                for (uint32_t k = lane; k < many; k += 32) {
                    const uint32_t at = peer(sh.list + k, r);
                    const Listed e{peer_float(at), peer_u32(at + 4)};
                    sh.all[first + k] = e;
                    sh.weight[first + k] = measure(e.v);
                }
            }
        __syncthreads();
        if (n <= kList) {
            if (rank_all) {
                uint64_t total = 0;
#pragma unroll 8
                for (uint32_t j = 0; j < n; ++j) total += sh.weight[j];
                goal = goal_of(total);
            }
            if (threadIdx.x < n) {
                const Listed me = sh.all[threadIdx.x];
                uint64_t before = 0;
#pragma unroll 8
                for (uint32_t j = 0; j < n; ++j) {
                    const Listed o = sh.all[j];
                    const uint64_t w = sh.weight[j];
                    before += o.v > me.v || (o.v == me.v && o.i < me.i) ? w : 0;
                }
                if (before < goal && before + sh.weight[threadIdx.x] >= goal) sh.border = {me.v, me.i + 1};
            }
            __syncthreads();
            const Border b{sh.border.v, sh.border.i};
            __syncthreads();
            return b;
        }
    }
    // many: the border's key, eight bits at a time, unless all have the same
    uint32_t prefix = 0;
    int shift = 24;
    if (part < kBins || few) {
        const uint32_t lane = threadIdx.x % 32;
        const uint32_t lowest = __reduce_min_sync(kAll, lane < team.blocks ? peer_u32(peer(&sh.lowest_key, lane)) : 0xffffffffu);
        prefix = __reduce_max_sync(kAll, lane < team.blocks ? peer_u32(peer(&sh.highest_key, lane)) : 0u);
        if (lowest == prefix) shift = -8;
        else prefix = 0;
    }
#pragma unroll 1
    for (; shift >= 0; shift -= 8) {
        const uint32_t found = team.find_bin(
            [&](uint64_t* hist) {
                row.above(sh, low, false, [&](const Raw<TI>& r, uint32_t l) {
#pragma unroll 1
                    for (int j = 0; j < 8; ++j) {
                        const float v = element(r, j);
                        const uint32_t k = key_of(v);
                        if (!from.keeps(v, row.index(l, j)) || !member(v) || (shift < 24 && k >> (shift + 8) != prefix)) continue;
                        count_in<Measure>(hist + (255u - (k >> shift & 255u)), measure(v));
                    }
                });
            },
            left, &goal);
        prefix = prefix << 8 | (255u - found);
    }
    // `need` of the equal logits, by index
    const float v = of_key(prefix);
    const uint64_t each = measure(v), need = (goal + each - 1) / each;
    uint64_t* counts = sh.hist[team.turn++ & 1];
    auto hits = [&](const Raw<TI>& r, uint32_t l) {
        uint32_t hit = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) hit |= (uint32_t)(element(r, j) == v && from.keeps(v, row.index(l, j))) << j;
        return hit;
    };
    for (uint32_t c = threadIdx.x / 32; c < row.chunks; c += kThreads / 32) {
        uint32_t mine = 0;
        row.run(c, [&](uint32_t l) { mine += l < row.p.count ? __popc(hits(row.group(l), l)) : 0; });
        mine = __reduce_add_sync(kAll, mine);
        if (threadIdx.x % 32 == 0) counts[c] = mine;
    }
    __syncthreads();
    const uint64_t count = threadIdx.x < row.chunks ? counts[threadIdx.x] : 0;
    uint64_t total;
    const uint64_t upto = block_scan(sh, count, &total);
    if (threadIdx.x == 0) {
        sh.total = total;
        sh.border.i = 0;
    }
    cluster_barrier();
    uint64_t before, all;
    team.totals(&before, &all);
    const uint64_t want = need > before ? need - before : 0;  // of this block
    if (want > upto - count && want <= upto) {
        sh.bin = threadIdx.x;
        sh.before = want - (upto - count);
    }
    __syncthreads();
    if (want > 0 && want <= total && threadIdx.x < 32) {
        uint64_t seen = 0;
        const uint64_t goal_here = sh.before;
        row.run(sh.bin, [&](uint32_t l) {
            const uint32_t hit = l < row.p.count ? hits(row.group(l), l) : 0;
            const uint64_t mine = warp_scan((uint64_t)__popc(hit));
            const uint64_t first = seen + mine - __popc(hit);
            if (goal_here > first && goal_here <= first + __popc(hit)) {
                uint32_t k = (uint32_t)(goal_here - first);
                for (int j = 0; j < 8; ++j)
                    if (hit >> j & 1 && --k == 0) sh.border.i = row.index(l, j) + 1;
            }
            seen += __shfl_sync(kAll, mine, 31);
        });
    }
    cluster_barrier();
    // one block has found it
    const uint32_t lane = threadIdx.x % 32;
    const uint32_t i = __reduce_max_sync(kAll, lane < team.blocks ? peer_u32(peer(&sh.border.i, lane)) : 0);
    cluster_barrier();  // read by all before it is written again
    return {v, i};
}

// A logit that at least `k` of the row's are not below, from the largest of eight
// neighbours each (one atomic instead of eight); -infinity where that is not known.
template <typename TI>
__device__ __forceinline__ float at_least(const Team<TI>& team, uint64_t k, float scale) {
    const Row<TI>& row = team.row;
    const float top = team.top;
    // (too near to all of them; and where a thread has few groups, a pass for this takes longer than it spares)
    if (k > row.V / 16 || row.p.groups(row.V) < 8ull * kThreads * team.blocks) return minus_inf();
    uint64_t goal, groups = 0;
    const uint32_t bin = team.find_bin(
        [&](uint64_t* hist) {
            row.each([&](const Raw<TI>& r, uint32_t) {
                const float m = group_max(r);
                if (m > minus_inf()) atomicAdd(reinterpret_cast<uint32_t*>(hist + whole_of(fminf((top - m) * scale, (float)(kBins - 1)))), 1u);
            });
        },
        [&](uint64_t total) {
            groups = total;
            return total < k ? total : k;
        },
        &goal);
    return bin < kBins - 1 && groups >= k ? below_range(top, bin, scale) : minus_inf();
}

template <typename TI>
__global__ void __launch_bounds__(kThreads, kPerSm) sample_kernel(const SampleArgs a, uint32_t room, uint32_t log2_blocks, int shift) {
    extern __shared__ uint4 slice[];
    __shared__ Shared sh;
    stream_order();
    const uint32_t blocks = 1u << log2_blocks, rank = blocks > 1 ? cluster_rank() : 0;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = kThreads / 32;
    if (threadIdx.x < 32) sh.roots[threadIdx.x] = kRoots[threadIdx.x];
    uint32_t turn = 0, parity = 0;
    const uint64_t step = gridDim.x >> log2_blocks;
    auto part = [&](uint64_t at) { return part_of(static_cast<const TI*>(a.z) + at * a.ld, a.V, rank, log2_blocks); };
    // Row `at` on its way to shared memory, and its settings.
    auto begin = [&](uint64_t at, uint32_t slot) {
        if (at >= a.T) return;
        const Part<TI> p = part(at);
        const uint32_t kept = min(p.count, room);
        for (uint32_t l = threadIdx.x; l < kept; l += kThreads) stage_group(slice, room, p, l, a.V);
        if (threadIdx.x == kThreads - 1) {
            Settings s;
            const float t = a.temperature ? a.temperature[at] : 1.0f;
            s.greedy = !(t >= FLT_MIN);
            // log2(e) / t in two floats: a quotient, and that of its remainder (64-bit division is slow here)
            constexpr double kLog2e = 1.4426950408889634074;
            constexpr float kHigh = (float)kLog2e, kLow = (float)(kLog2e - (double)kHigh);
            s.ch = __fdiv_rn(kHigh, t);
            s.cl = t < 0x1p100f ? __fdiv_rn(__fmaf_rn(-s.ch, t, kHigh) + kLow, t) : 0.0f;  // (beyond, a remainder below the floats)
            s.bins = kPerOctave * s.ch;
            s.top_k = a.top_k && a.top_k[at] > 0 ? (uint32_t)a.top_k[at] : 0;
            const float p = a.top_p ? a.top_p[at] : 1.0f;
            s.top_p = p < 1.0f ? fmaxf(p, 0.0f) : 1.0f;
            const float m = a.min_p ? a.min_p[at] : 0.0f;
            s.use_min_p = m > 0.0f;
            s.min_p = s.use_min_p ? (double)t * log((double)fminf(m, 1.0f)) : 0.0;
            const float u = a.u[at];
            s.u = u > 0.0f ? fminf(u, 1.0f - FLT_EPSILON / 2) : 0.0f;
            sh.set[slot] = s;
        }
    };
    begin(blockIdx.x >> log2_blocks, 0);
    for (uint64_t at = blockIdx.x >> log2_blocks; at < a.T; at += step, parity ^= 1) {
        Row<TI> row;
        row.slice = slice;
        row.room = room;
        row.p = part(at);
        row.kept = min(row.p.count, room);
        row.V = a.V;
        row.size = max(1u, (row.p.count + kBins - 1) / kBins);
        copies_done();

        // the largest logit
        float top = minus_inf();
        row.each([&](const Raw<TI>& r, uint32_t) { top = fmaxf(top, group_max(r)); });
        top = rows::warp_max(top);
        if (lane == 0) sh.warp_max[warp] = top;
        __syncthreads();  // (and what every thread copied is there for all)
        if (warp == 0) {
            top = rows::warp_max(lane < warps ? sh.warp_max[lane] : minus_inf());
            if (lane == 0) sh.top[parity] = top;
        }
        cluster_barrier();
        top = rows::warp_max(lane < blocks ? peer_float(peer(&sh.top[parity], lane)) : minus_inf());
        const Settings set = sh.set[parity];
        const bool filtered = set.top_k || set.top_p < 1.0f || set.use_min_p;
        row.chunks = (row.p.count + row.size - 1) / row.size;
        if (top == minus_inf() || set.greedy || set.top_k == 1 || set.top_p == 0.0f) {  // nothing to draw; the same in every block
            if (threadIdx.x == 0) sh.lowest[parity] = 0xffffffffu;
            __syncthreads();
            if (top > minus_inf())
                row.above(sh, top, false, [&](const Raw<TI>& r, uint32_t l) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (element(r, j) == top) atomicMin(&sh.lowest[parity], row.index(l, j));
                });
            cluster_barrier();
            begin(at + step, parity ^ 1);
            if (rank == 0 && warp == 0) {
                const uint32_t i = __reduce_min_sync(kAll, lane < blocks ? peer_u32(peer(&sh.lowest[parity], lane)) : 0xffffffffu);
                if (lane == 0) a.tokens[at] = (int32_t)i;  // -1 where there is none
            }
            __syncthreads();
            continue;
        }
        const Team<TI> team{sh, row, blocks, rank, top, turn};
        Weigh weigh;
        weigh.roots = sh.roots;
        weigh.max = top;
        weigh.ch = set.ch;
        weigh.cl = set.cl;
        weigh.shift = shift;
        weigh.none = fmaxf(top - fminf(60.0f / set.ch, FLT_MAX), -FLT_MAX);
        // What weighs next to nothing is left out from the start; where the floats
        // below the largest do (a tiny temperature), so is all but that.
        Border border = weigh.none < top ? Border{weigh.none, 0} : Border{top, 0xffffffffu};
        if (set.top_k && set.top_k < a.V) {
            const float scale = kPerOctave * 1.44269504f;
            const float least = at_least(team, set.top_k, scale);
            border = narrow(team, border, scale, least, ~0ull, least == minus_inf(), Count{}, [&](uint64_t total) { return total < set.top_k ? total : (uint64_t)set.top_k; });
        }
        if (set.top_p < 1.0f)
            border = narrow(team, border, set.bins, minus_inf(), set.top_k ? set.top_k : ~0ull, !set.top_k, weigh, [&](uint64_t total) {
                const uint64_t goal = times(set.top_p, total, true);
                return goal ? goal : 1;
            });
        if (set.use_min_p) {  // weight >= min_p: l >= l_max + T log(min_p), from the next float on
            if (threadIdx.x == 0) {
                const double least = (double)top + set.min_p;
                float f = (float)least;
                if ((double)f < least) f = of_key(key_of(f) + 1);
                const uint32_t k = key_of(f) - 1;
                sh.border.v = of_key(k == 0x7fffffffu ? k - 1 : k);  // (that key would be the other zero)
            }
            __syncthreads();
            const float below = sh.border.v;
            if (below > border.v || (below == border.v && border.i > 0)) border = {below, 0};
        }

        // the sums of this block's runs
        uint64_t* sums = sh.hist[turn++ & 1];
        auto sum_of = [&](const Raw<TI>& r, auto use) {
            uint64_t w = 0;
            weigh.group(r, use, [&](float, int, uint64_t m) { w += m; });
            return w;
        };
        auto kept = [&](uint32_t l) { return [&row, &border, l](float v, int j) { return border.keeps(v, row.index(l, j)); }; };
        const bool small = row.p.count <= kThreads;
        const uint32_t few = small ? row.p.count : filtered ? row.queue_up(sh, border.v) : kQueue + 1;
        if (few <= kQueue) {
            if (threadIdx.x < kBins) sums[threadIdx.x] = 0;
            __syncthreads();
            for (uint32_t q = threadIdx.x; q < few; q += kThreads) {
                const uint32_t l = small ? q : sh.queue[q];
                add64(sums + l / row.size, sum_of(row.group(l), kept(l)));
            }
        } else {  // many groups that would meet in one sum: a warp's steps are a run's
            row.size = (row.size + 31) / 32 * 32;
            row.chunks = (row.p.count + row.size - 1) / row.size;
            const float least = border.i ? border.v : of_key(key_of(border.v) + 1);
            const bool tied = border.i - 1 < 0xfffffffeu;  // the index decides between those equal to border.v
            for (uint32_t c = warp; c < row.chunks; c += warps) {
                uint64_t w = 0;
                row.run(c, [&](uint32_t l) {
                    if (l >= row.p.count) return;
                    const Raw<TI> r = row.group(l);
                    bool equal = false;
                    w += sum_of(r, [&](float v, int) {
                        equal |= v == border.v;
                        return v >= least;
                    });
                    if (tied && equal) {  // those behind the border, taken off again
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (element(r, j) == border.v && row.index(l, j) >= border.i) w -= weigh(border.v);
                    }
                });
#pragma unroll
                for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(kAll, w, o);
                if (lane == 0) sums[c] = w;
            }
        }
        __syncthreads();
        begin(at + step, parity ^ 1);  // (what follows reads few of this row's logits once more)
        const uint64_t mine = threadIdx.x < row.chunks ? sums[threadIdx.x] : 0;
        uint64_t total;
        const uint64_t upto = block_scan(sh, mine, &total);
        if (threadIdx.x == 0) sh.total = total;
        cluster_barrier();
        uint64_t before, all;
        team.totals(&before, &all);
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
            row.run(sh.bin, [&](uint32_t l) {
                uint64_t w[8], sum = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 0;
                if (l < row.p.count)
                    weigh.group(load_group(row.p, l, a.V), [&](float v, int j) { return border.keeps(v, row.index(l, j)); },
                                [&](float, int j, uint64_t m) {
                                    w[j] = m;
                                    sum += m;
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
            });
        }
        __syncthreads();  // the sums are free
    }
    cluster_barrier();  // no block ends while another reads its shared memory
}

// How a row is spread: over a cluster of up to sixteen blocks, two on an SM, that
// go through their rows one after the other. A row costs kRowNs on each of its
// blocks and a group kGroupNs of its SM, kAgain times as much where it is read
// again in every pass, and the slowest of a few rows kRows more than most. Rows of
// all kinds of settings, in us, over two, four, eight and sixteen blocks:
//   24 x 267735 float32 222, 103, 66, 63; 256 x 267735 582, 410, 379, 558;
//   256 x 33278 91, 94, 137, 328; one row of 33278 41, 29, 22, 21.
// Blocks of 512 threads, with fewer registers each, 68, 390, 84 and 23; of 320 64,
// 420, 93 and 21; three of 320 with less shared memory 70, 375, 92 and 22; one of 640
// 78, 404, 104 and 21.
constexpr uint32_t kPartSmem = 100 * 1024;  // of a block's part of a row
constexpr double kRowNs = 22000.0, kGroupNs = 6.25, kAgain = 2.0, kRows = 0.5;

template <typename TI>
cudaError_t launch(const SampleArgs& a, cudaStream_t s) {
    DeviceInfo di{};
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    const uint64_t groups = ((uint64_t)a.V + 14) / 8;  // whatever the row's alignment
    constexpr uint64_t kGroupBytes = 8 * sizeof(TI);
    const void* kernel = reinterpret_cast<const void*>(sample_kernel<TI>);
    double best = 0.0;
    uint32_t blocks = 0, log2_blocks = 0, room = 0, clusters = 0, smem = 0;
    for (uint32_t b = 1, log2 = 0; b <= 16; b *= 2, ++log2) {
        if (b > 1 && groups < b * (uint64_t)kThreads / 2) break;  // too little for so many
        const uint64_t need = (groups + b - 1) / b + 1, most = kPartSmem / kGroupBytes, keep = need < most ? need : most;
        const uint32_t bytes = (uint32_t)smem_of(keep * kGroupBytes);
        int n = 0;
        e = resident_clusters(kernel, kThreads, b, bytes, &n);
        if (e != cudaSuccess) return e;
        if (n < 1) continue;
        const uint64_t on = ((uint64_t)a.T * b + di.sms - 1) / di.sms;
        const double per_sm = (double)(on < kPerSm ? on : kPerSm), rounds = kRows + (a.T > (uint32_t)n ? (double)a.T / n : 1.0);
        const double ns = rounds * (kRowNs + per_sm * kGroupNs * ((double)keep + kAgain * (double)(need - keep)));
        if (blocks && ns >= best) continue;
        best = ns;
        blocks = b;
        log2_blocks = log2;
        room = (uint32_t)keep;
        clusters = (uint32_t)n;
        smem = bytes;
    }
    if (blocks == 0) return cudaErrorInvalidConfiguration;
    int shift = 0;  // sums of V weights stay below 2^63
    while ((1ull << (62 - kBits + shift)) < a.V) ++shift;
    const uint32_t grid = (a.T < clusters ? a.T : clusters) * blocks;
    return launch_early(sample_kernel<TI>, grid, kThreads, smem, blocks, s, a, room, log2_blocks, shift);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int dtype, cudaStream_t s) {
    return dtype == 0 ? launch<float>(a, s) : launch<uint16_t>(a, s);
}

}  // namespace s2
