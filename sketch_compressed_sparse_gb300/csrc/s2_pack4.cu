// 4-bit packing (MXFP4): e2m1 codes, two to a byte, with one power-of-two scale
// for each 32 elements of a row, and the way back.
//
// The scale of a block is 2^e with the least e >= -125 for which no element
// exceeds 6 * 2^e (6 is e2m1's largest number). With the largest element's bits
// (1.m * 2^(E-127)) that is e = E - 129, plus 1 where 1.m exceeds 1.5 = 6 / 2^2,
// and the stored byte is e + 127. A power of two makes x * 2^-e exact (but where
// it is far below the smallest code), so a code is one rounding away from its
// element, and code * 2^e is exact in float32 and in bfloat16.
//
// Both directions are bound by HBM: an element is read once and written once.
// A lane holds neighbours of four rows of a tile of 128 x 128 elements, 32 rows
// apart: their scale words are then 16 neighbouring bytes of the tile, and it has
// four or eight independent loads in flight. Packing takes 32 bytes of a row a
// lane, eight floats or sixteen bfloat16 (with eight bfloat16 twice the shuffles
// and addresses, 267735 x 1024 in 202 us instead of 101).
#include "s2_internal.h"
#include "s2_launch.cuh"

namespace s2 {
namespace {

constexpr int kTile = 128;           // rows and columns of a tile of scales
constexpr int kRows = 4;             // rows of a lane
constexpr uint32_t kTileBytes = 512;
constexpr uint32_t kMinByte = 2;     // e >= -125
constexpr uint32_t kInf = 0x7f800000u;

// What a warp works on: rows of one tile, LANES lanes and 128 / LANES elements a
// lane to a row, 32 / LANES rows at a time.
struct Item {
    uint64_t row;    // the lane's first row; the others are 32, 64 and 96 below
    uint32_t col;    // the lane's first column
    int left;        // columns from there to the row's end
    uint64_t scale;  // the four words of scale bytes of the lane's rows
};
template <int LANES>
__device__ __forceinline__ Item item(uint64_t at, uint32_t tcols, uint32_t cols) {
    constexpr uint32_t kAtOnce = 32 / LANES, kBands = 32 / kAtOnce;  // of a tile's first 32 rows
    const uint32_t lane = threadIdx.x % 32, sub = lane % LANES;
    // neighbouring warps take neighbouring tiles of the same rows
    const uint64_t band = at / tcols;
    const uint32_t tcol = (uint32_t)(at - band * tcols);
    const uint64_t trow = band / kBands;
    const uint32_t r = (uint32_t)(band % kBands) * kAtOnce + lane / LANES;
    Item it;
    it.row = trow * kTile + r;
    it.col = tcol * kTile + sub * (kTile / LANES);
    it.left = (int)cols - (int)it.col;
    it.scale = (trow * tcols + tcol) * kTileBytes + r * 16;
    return it;
}

// A lane's elements of a row, eight words as they lie in memory: eight floats or
// sixteen bfloat16. Those past the row's end are 0.
template <typename T>
struct Raw {
    static constexpr int kPer = 32 / sizeof(T);
    uint32_t w[8];
    __device__ __forceinline__ float value(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    // Bits of the largest magnitude as a float's; above every number's where there is a NaN.
    __device__ __forceinline__ uint32_t amax() const {
        uint32_t m = 0;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        } else {
            m = w[0] & 0x7fff7fffu;
#pragma unroll
            for (int i = 1; i < 8; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
            return max(m & 0xffff0000u, m << 16);
        }
    }
};
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load(const T* p, int left) {
    Raw<T> r;
    if (VEC && left >= Raw<T>::kPer) {
        const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
        r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
        return r;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r.w[i] = 0;
        if constexpr (sizeof(T) == 4) {
            if (i < left) r.w[i] = p[i];
        } else {
            if (2 * i < left) r.w[i] = p[2 * i];
            if (2 * i + 1 < left) r.w[i] |= (uint32_t)p[2 * i + 1] << 16;
        }
    }
    return r;
}

// Eight codes as a word, the first in the lowest half byte: to nearest, ties to
// even, the sign kept.
__device__ __forceinline__ uint32_t codes8(const float* q) {
    uint32_t r;
    asm("{.reg .b8 a, b, c, d;\n"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        "mov.b32 %0, {a, b, c, d};}"
        : "=r"(r)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return r;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) pack4_kernel(Pack4Args a) {
    constexpr int kPer = Raw<T>::kPer, kLanes = kTile / kPer, kBlock = 32 / kPer;  // lanes of a row, of a block
    stream_order();
    const uint64_t at = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / 32;
    if (at >= a.items) return;  // whole warps
    const Item it = item<kLanes>(at, a.tcols, a.cols);
    const T* x = static_cast<const T*>(a.x);
    Raw<T> v[kRows];
    uint32_t word[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const uint64_t row = it.row + 32 * i;
        const bool there = row < a.rows && it.left > 0;
        v[i] = load<T, VEC>(x + (there ? row * a.ldx + it.col : 0), there ? it.left : 0);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const uint64_t row = it.row + 32 * i;
        uint32_t m = v[i].amax();
#pragma unroll
        for (int o = 1; o < kBlock; o *= 2) m = max(m, __shfl_xor_sync(kFull, m, o));
        const bool special = m >= kInf;
        uint32_t b = (uint32_t)max((int)((m + 0x3fffffu) >> 23) - 2, (int)kMinByte);
        const float inv = special ? 0.0f : __uint_as_float((254u - b) << 23);
        uint32_t c[kPer / 8];
#pragma unroll
        for (int h = 0; h < kPer / 8; ++h) {
            float q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = v[i].value(8 * h + j) * inv;
            c[h] = codes8(q);
        }
        if (special) {
            b = 255;
#pragma unroll
            for (int h = 0; h < kPer / 8; ++h) c[h] = 0;
        }
        const bool there = row < a.rows && it.left > 0;
        if (!there) b = 127;  // past the end
        if (there) {
            uint8_t* p = a.codes + row * a.ldc + it.col / 2;
            if (it.left >= kPer) {
                if constexpr (kPer == 16) *reinterpret_cast<uint2*>(p) = make_uint2(c[0], c[1]);
                else *reinterpret_cast<uint32_t*>(p) = c[0];
            } else {
                for (int j = 0; 2 * j < it.left; ++j) p[j] = (uint8_t)(c[j / 4] >> (8 * (j % 4)));
            }
        }
        // the bytes of the row's four blocks, kBlock lanes apart, as one word in its first lane
        uint32_t w = b;
        w |= __shfl_xor_sync(kFull, b, kBlock) << 8;
        word[i] = __byte_perm(w, __shfl_xor_sync(kFull, w, 2 * kBlock), 0x5410);
    }
    if (threadIdx.x % kLanes == 0)
        *reinterpret_cast<uint4*>(a.scales + it.scale) = make_uint4(word[0], word[1], word[2], word[3]);
}

// The numbers of eight codes, exactly.
__device__ __forceinline__ void values8(uint32_t codes, float* v) {
    uint32_t h[4];
    asm("{.reg .b8 a, b, c, d;\n"
        "mov.b32 {a, b, c, d}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n"
        "cvt.rn.f16x2.e2m1x2 %3, d;}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(v[2 * j]), "=f"(v[2 * j + 1]) : "r"(h[j]));
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float scale_of(uint32_t b) {
    // byte 0 stands for 2^-127, a subnormal float; byte 255 for NaN
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fffffffu : b << 23);
}

// Rows on 16 bytes: eight neighbours a lane.
template <typename T>
__global__ void __launch_bounds__(kThreads) unpack4_kernel(Unpack4Args a) {
    constexpr int kLanes = 16, kPer = 8;
    stream_order();
    const uint64_t at = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / 32;
    if (at >= a.items) return;
    const Item it = item<kLanes>(at, a.tcols, a.cols);
    if (it.left <= 0) return;
    uint32_t c[kRows];
    const uint4 s4 = *reinterpret_cast<const uint4*>(a.scales + it.scale);
    const uint32_t s[kRows] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const uint64_t row = it.row + 32 * i;
        c[i] = 0;
        if (row >= a.rows) continue;
        const uint8_t* p = a.codes + row * a.ldc + it.col / 2;
        if (it.left >= kPer) {
            c[i] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            for (int j = 0; 2 * j < it.left; ++j) c[i] |= (uint32_t)p[j] << (8 * j);
        }
    }
    T* out = static_cast<T*>(a.out);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const uint64_t row = it.row + 32 * i;
        if (row >= a.rows) break;
        const float f = scale_of((s[i] >> (8 * (threadIdx.x % kLanes / 4))) & 255u);
        float v[kPer];
        values8(c[i], v);
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] *= f;
        T* o = out + row * a.ldo + it.col;
        if constexpr (sizeof(T) == 4) {
            if (it.left >= kPer) {
                reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (j < it.left) o[j] = v[j];
            }
        } else {
            const uint4 w = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
            if (it.left >= kPer) {
                *reinterpret_cast<uint4*>(o) = w;
            } else {
                const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (j < it.left) o[j] = (uint16_t)(h[j / 2] >> (16 * (j % 2)));
            }
        }
    }
}

// Rows that start anywhere: every sixteenth element a lane, so that the half-warp's
// stores of two or four bytes still run along the row (20000 x 4095 bfloat16 in
// 65 us; with eight neighbours a lane 227).
template <typename T>
__global__ void __launch_bounds__(kThreads) unpack4_any_kernel(Unpack4Args a) {
    constexpr int kLanes = 16, kPer = 8;
    stream_order();
    const uint64_t at = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / 32;
    if (at >= a.items) return;
    const Item it = item<kLanes>(at, a.tcols, a.cols);
    const uint32_t sub = threadIdx.x % kLanes, tile = it.col - sub * kPer;  // the tile's first column
    const uint4 s4 = *reinterpret_cast<const uint4*>(a.scales + it.scale);
    const uint32_t s[kRows] = {s4.x, s4.y, s4.z, s4.w};
    T* out = static_cast<T*>(a.out);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const uint64_t row = it.row + 32 * i;
        if (row >= a.rows) break;
        const uint8_t* p = a.codes + row * a.ldc + tile / 2 + sub / 2;
        T* o = out + row * a.ldo + tile + sub;
        uint32_t c = 0;  // the lane's eight codes
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (tile + sub + j * kLanes < a.cols) c |= ((uint32_t)p[j * (kLanes / 2)] >> (4 * (sub % 2)) & 15u) << (4 * j);
        float v[kPer];
        values8(c, v);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (tile + sub + j * kLanes >= a.cols) continue;
            const float q = v[j] * scale_of(s[i] >> (8 * (j / 2)) & 255u);  // two steps of sixteen are a block
            if constexpr (sizeof(T) == 4) o[j * kLanes] = q;
            else o[j * kLanes] = (uint16_t)bf16x2(q, 0.0f);
        }
    }
}

// Rows start on 16 bytes.
inline bool vector_rows(const void* p, uint64_t ld, uint64_t rows, uint64_t esz) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * esz % 16 == 0);
}
inline uint32_t blocks_of(uint64_t items) { return (uint32_t)((items + kThreads / 32 - 1) / (kThreads / 32)); }

}  // namespace

cudaError_t launch_pack4(const Pack4Args& m, int dtype, cudaStream_t s) {
    Pack4Args a = m;
    a.items = a.tiles * (dtype == 0 ? 16 : 8);
    const bool vec = vector_rows(a.x, a.ldx, a.rows, dtype == 0 ? 4 : 2);
    auto kernel = dtype == 0 ? (vec ? pack4_kernel<uint32_t, true> : pack4_kernel<uint32_t, false>)
                             : (vec ? pack4_kernel<uint16_t, true> : pack4_kernel<uint16_t, false>);
    return launch_early(kernel, blocks_of(a.items), kThreads, 0, 0, s, a);
}

cudaError_t launch_unpack4(const Unpack4Args& a, int dtype, cudaStream_t s) {
    const bool vec = vector_rows(a.out, a.ldo, a.rows, dtype == 0 ? 4 : 2);
    if (dtype == 0) return launch_early(vec ? unpack4_kernel<float> : unpack4_any_kernel<float>, blocks_of(a.items), kThreads, 0, 0, s, a);
    return launch_early(vec ? unpack4_kernel<uint16_t> : unpack4_any_kernel<uint16_t>, blocks_of(a.items), kThreads, 0, 0, s, a);
}

}  // namespace s2
