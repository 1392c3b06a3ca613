// 8-bit packing: e4m3 codes with one power-of-two scale for each block of 128
// elements of a row, or of 128 x 128 elements, and the way back.
//
// The scale of a block is 2^e with the least e >= -117 for which no finite
// element of the block exceeds 448 * 2^e (448 is e4m3's largest number). With
// the float's bits (1.m * 2^(E-127)) that is e = E - 135, plus 1 where 1.m
// exceeds 1.75 = 448 / 2^8, and the stored byte is e + 127. A power of two
// makes x * 2^-e exact, so a code is one rounding away from its element, and
// makes code * 2^e exact in float32 and in bfloat16 (the bound -117 keeps the
// smallest code times 2^e a normal number).
//
// Both directions are bound by HBM: an element is read once and written once.
// They come near it only with few instructions per element, so the special
// numbers cost nothing where there are none: maxima ignore NaN, and only a
// block whose maximum is infinite goes through its elements again. Measured, of
// the 6.79 TB/s of a plain copy: 8192 x 4096 bfloat16 packed in 17.6 us (0.85),
// unpacked in 17.0 us (0.88); float32 25.2 us (0.98) and 26.0 us (0.95); rows of
// 4095 bfloat16 30 and 29 us; 33278 x 512 float32 in both orders 19.7 us (0.77;
// its 1040 tiles are 2.3 rounds of the 456 that are resident).
//
// Sixteen lanes hold one row's block (see column()); where rows do not start on
// 16 bytes a lane holds every sixteenth element, so that its accesses of two or
// four bytes still run along the row together with its neighbours'.
#include <cuda_bf16.h>

#include "s2_internal.h"
#include "s2_launch.cuh"

namespace s2 {
namespace {

constexpr int kBlk = 128;
constexpr int kPer = 8;               // elements per lane
constexpr int kLanes = kBlk / kPer;   // lanes per block of a row
constexpr int kMinByte = 10;          // e >= -117
constexpr uint32_t kInf = 0x7f800000u;

// Eight elements as they lie in memory.
template <typename T>
struct Raw {
    uint32_t w[2 * sizeof(T)];
};

// Element i as a float.
__device__ __forceinline__ float value(const Raw<float>& r, int i) { return __uint_as_float(r.w[i]); }
__device__ __forceinline__ float value(const Raw<uint16_t>& r, int i) {
    return __uint_as_float(i % 2 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
}
__device__ __forceinline__ void put(Raw<float>& r, int i, float x) { r.w[i] = __float_as_uint(x); }
__device__ __forceinline__ void put(Raw<uint16_t>& r, int i, uint16_t x) { r.w[i / 2] |= (uint32_t)x << (16 * (i % 2)); }

// Column of a lane's element i within its block, and whether all of a lane's
// columns lie before `left`. VEC: rows start on 16 bytes, and a lane holds
// eight neighbours of 16 bits or twice four of 32 bits, so that each 16-byte
// access of the half-warp is 256 bytes of a row.
template <typename T, bool VEC>
__device__ __forceinline__ uint32_t column(uint32_t sub, int i) {
    return !VEC ? sub + i * kLanes : sizeof(T) == 2 ? sub * 8 + i : sub * 4 + i % 4 + i / 4 * 64;
}
template <typename T>
__device__ __forceinline__ bool whole(uint32_t sub, int left) {
    return left > (int)column<T, true>(sub, kPer - 1);
}

// A lane's elements of the block of a row that begins at p; `left` columns
// exist from there on (the others read as 0). VEC: p is 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load8(const T* p, uint32_t sub, int left) {
    Raw<T> r;
    if (VEC && whole<T>(sub, left)) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            const uint4 a = *reinterpret_cast<const uint4*>(p + column<T, true>(sub, 4 * i));
            r.w[4 * i] = a.x;
            r.w[4 * i + 1] = a.y;
            r.w[4 * i + 2] = a.z;
            r.w[4 * i + 3] = a.w;
        }
        return r;
    }
#pragma unroll
    for (int i = 0; i < (int)(2 * sizeof(T)); ++i) r.w[i] = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if ((int)column<T, VEC>(sub, i) < left) put(r, i, p[column<T, VEC>(sub, i)]);
    return r;
}

// Bits of the largest magnitude among the eight, NaN aside.
__device__ __forceinline__ uint32_t amax_bits(const Raw<float>& r) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = fmaxf(m, fabsf(__uint_as_float(r.w[i])));
    return __float_as_uint(m);
}
__device__ __forceinline__ uint32_t amax_bits(const Raw<uint16_t>& r) {
    __nv_bfloat162 m = __float2bfloat162_rn(0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&r.w[i])));
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
    return max(w & 0xffff0000u, w << 16);
}
// Of the finite ones.
template <typename T>
__device__ __forceinline__ uint32_t finite_amax_bits(const Raw<T>& r) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t b = __float_as_uint(value(r, i)) & 0x7fffffffu;
        m = max(m, b < kInf ? b : 0u);
    }
    return m;
}

__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    return (uint32_t)max((int)((amax + 0x1fffffu) >> 23) - 8, kMinByte);
}

// The eight codes of a block with scale byte b. A code is e4m3's nearest (ties
// to even); NaN becomes NaN, and so do infinities, which the conversion alone
// would saturate (special: the block has some).
template <typename T>
__device__ __forceinline__ uint2 codes8(const Raw<T>& r, uint32_t b, bool special) {
    const float inv = __uint_as_float((254u - b) << 23);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo = value(r, 2 * i) * inv, hi = value(r, 2 * i + 1) * inv;
        if (special) {
            if (fabsf(lo) == __uint_as_float(kInf)) lo = __uint_as_float(0x7fffffffu);
            if (fabsf(hi) == __uint_as_float(kInf)) hi = __uint_as_float(0x7fffffffu);
        }
        uint16_t q;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(hi), "f"(lo));
        h[i] = q;
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ uint8_t byte_of(uint2 c, int i) { return (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i % 4))); }

// A lane's codes to the block that begins at p (8-byte aligned), and from there.
template <typename T, bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, uint2 c, uint32_t sub, int left) {
    if (VEC && whole<T>(sub, left)) {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint2*>(p + column<T, true>(sub, 0)) = c;
        } else {
            *reinterpret_cast<uint32_t*>(p + column<T, true>(sub, 0)) = c.x;
            *reinterpret_cast<uint32_t*>(p + column<T, true>(sub, 4)) = c.y;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if ((int)column<T, VEC>(sub, i) < left) p[column<T, VEC>(sub, i)] = byte_of(c, i);
}
template <typename T, bool VEC>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, uint32_t sub, int left) {
    if (VEC && whole<T>(sub, left)) {
        if constexpr (sizeof(T) == 2) return *reinterpret_cast<const uint2*>(p + column<T, true>(sub, 0));
        return make_uint2(*reinterpret_cast<const uint32_t*>(p + column<T, true>(sub, 0)),
                          *reinterpret_cast<const uint32_t*>(p + column<T, true>(sub, 4)));
    }
    uint2 c = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if ((int)column<T, VEC>(sub, i) < left) (i < 4 ? c.x : c.y) |= (uint32_t)p[column<T, VEC>(sub, i)] << (8 * (i % 4));
    return c;
}

// Blocks of a row in flight per half-warp: 8192 x 4096 bfloat16 packed in 19.2 us
// with two, 20.6 with four; rows of 4095 unpacked in 31 and 40 us (launches one after the other).
constexpr int kItems = 2;

// One half-warp per block of a row, kItems of them in flight.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) pack_rows_kernel(Pack8Args a) {
    stream_order();
    const uint32_t sub = threadIdx.x % kLanes;
    const uint64_t first = ((uint64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes) * kItems;
    const T* x = static_cast<const T*>(a.x);
    Raw<T> v[kItems];
    uint64_t row[kItems];
    uint32_t col[kItems];
    int left[kItems];
    uint32_t r = first < a.items ? (uint32_t)first / a.nblk : 0, blk = first < a.items ? (uint32_t)first - r * a.nblk : 0;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        row[i] = r;
        col[i] = blk * kBlk;
        left[i] = first + i < a.items ? (int)(a.cols - col[i]) : 0;
        v[i] = load8<T, VEC>(x + row[i] * a.ldx + col[i], sub, left[i]);
        if (++blk == a.nblk) {
            blk = 0;
            ++r;
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        uint32_t m = amax_bits(v[i]);
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
        const bool special = __any_sync(kFull, m == kInf);
        if (special) {
            m = finite_amax_bits(v[i]);
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
        }
        const uint32_t b = scale_byte(m);
        store_codes<T, VEC>(a.codes + row[i] * a.ldc + col[i], codes8(v[i], b, special), sub, left[i]);
        if (sub == 0 && left[i]) a.scales[first + i] = (uint8_t)b;
    }
}

// 4 x 4 bytes: word i holds row i; afterwards word j holds column j.
__device__ __forceinline__ void transpose4(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    const uint32_t a = __byte_perm(r0, r1, 0x5140), b = __byte_perm(r2, r3, 0x5140);
    const uint32_t c = __byte_perm(r0, r1, 0x7362), d = __byte_perm(r2, r3, 0x7362);
    r0 = __byte_perm(a, b, 0x5410);
    r1 = __byte_perm(a, b, 0x7632);
    r2 = __byte_perm(c, d, 0x5410);
    r3 = __byte_perm(c, d, 0x7632);
}

// Place of the 16 bytes of rows 16 u to 16 u + 15 of column col in the
// transposed tile in shared memory: shifted among the eight of a column so
// that lanes that hold columns 8 or 1 apart meet different banks.
__device__ __forceinline__ uint32_t turned_at(uint32_t col, uint32_t u) {
    return col * kBlk + ((u ^ col ^ (col / 8)) % 8) * 16;
}

// One block of threads per 128 x 128 tile: each half-warp holds eight whole
// rows of it in registers, so the tile is read once; the transposed codes
// turn 8 x 8 bytes in registers and pass through shared memory.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) pack_tiles_kernel(Pack8Args a) {
    stream_order();
    __shared__ uint32_t warp_max[kThreads / 32];
    __shared__ __align__(16) uint8_t turned[kBlk * kBlk];
    const uint32_t sub = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
    const uint32_t trow = blockIdx.x / a.nblk, tcol = blockIdx.x - trow * a.nblk;
    const uint64_t r0 = (uint64_t)trow * kBlk + grp * kPer;
    const int left = (int)(a.cols - tcol * kBlk);
    const int rvalid = (int)min((uint64_t)kPer, a.rows > r0 ? a.rows - r0 : 0);
    const T* x = static_cast<const T*>(a.x) + (rvalid ? r0 : 0) * a.ldx + tcol * kBlk;
    Raw<T> v[kPer];
    uint32_t m = 0;
    // (the whole tile exists nearly always: its loads carry no conditions)
    if (rvalid == kPer) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = load8<T, VEC>(x + i * a.ldx, sub, left);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = load8<T, VEC>(x + (i < rvalid ? i : 0) * a.ldx, sub, i < rvalid ? left : 0);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = max(m, amax_bits(v[i]));
    m = __reduce_max_sync(kFull, m);
    if (threadIdx.x % 32 == 0) warp_max[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, warp_max[i]);
    const bool special = m == kInf;  // the same in the whole block of threads
    if (special) {
        m = 0;
        for (int i = 0; i < kPer; ++i) m = max(m, finite_amax_bits(v[i]));
        m = __reduce_max_sync(kFull, m);
        __syncthreads();
        if (threadIdx.x % 32 == 0) warp_max[threadIdx.x / 32] = m;
        __syncthreads();
        for (int i = 0; i < kThreads / 32; ++i) m = max(m, warp_max[i]);
    }
    const uint32_t b = scale_byte(m);
    uint2 c[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        c[i] = codes8(v[i], b, special);
        if (i < rvalid) store_codes<T, VEC>(a.codes + (r0 + i) * a.ldc + tcol * kBlk, c[i], sub, left);
    }
    if (threadIdx.x == 0) {
        a.scales[(uint64_t)trow * a.nblk + tcol] = (uint8_t)b;
        if (a.codes_t) a.scales_t[(uint64_t)tcol * a.nrow_blk + trow] = (uint8_t)b;
    }
    if (!a.codes_t) return;
    transpose4(c[0].x, c[1].x, c[2].x, c[3].x);
    transpose4(c[4].x, c[5].x, c[6].x, c[7].x);
    transpose4(c[0].y, c[1].y, c[2].y, c[3].y);
    transpose4(c[4].y, c[5].y, c[6].y, c[7].y);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const uint2 w = j < 4 ? make_uint2(c[j].x, c[j + 4].x) : make_uint2(c[j - 4].y, c[j].y);
        *reinterpret_cast<uint2*>(turned + turned_at(column<T, VEC>(sub, j), grp / 2) + grp % 2 * 8) = w;
    }
    __syncthreads();
    const int down = (int)min((uint64_t)kBlk, a.rows - (uint64_t)trow * kBlk);
#pragma unroll
    for (int i = 0; i < kBlk * kBlk / 16 / kThreads; ++i) {
        const uint32_t t = threadIdx.x + i * kThreads, col = t / 8, at = (t % 8) * 16;
        if (tcol * kBlk + col >= a.cols) continue;
        const uint8_t* s = turned + turned_at(col, t % 8);
        uint8_t* d = a.codes_t + (uint64_t)(tcol * kBlk + col) * a.ldct + (uint64_t)trow * kBlk + at;
        if ((int)at + 16 <= down) {
            *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(s);
        } else {
            for (int j = 0; (int)at + j < down; ++j) d[j] = s[j];
        }
    }
}

// Two e4m3 codes to two floats, exactly.
__device__ __forceinline__ float2 decode2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    float2 f;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) unpack_kernel(Unpack8Args a) {
    stream_order();
    const uint32_t sub = threadIdx.x % kLanes;
    const uint64_t first = ((uint64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes) * kItems;
    T* out = static_cast<T*>(a.out);
    uint2 c[kItems];
    uint32_t b[kItems], col[kItems];
    uint64_t row[kItems];
    int left[kItems];
    uint32_t r = first < a.items ? (uint32_t)first / a.nblk : 0, blk = first < a.items ? (uint32_t)first - r * a.nblk : 0;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        row[i] = r;
        col[i] = blk * kBlk;
        left[i] = first + i < a.items ? (int)(a.cols - col[i]) : 0;
        const uint8_t* p = a.codes + row[i] * a.ldc + col[i];
        c[i] = load_codes<T, VEC>(p, sub, left[i]);
        b[i] = left[i] ? a.scales[(row[i] >> a.row_shift) * a.nblk + blk] : 127u;
        if (++blk == a.nblk) {
            blk = 0;
            ++r;
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        // byte 0 stands for 2^-127, a subnormal float; byte 255 for NaN
        const float s = __uint_as_float(b[i] == 0 ? 0x00400000u : b[i] == 255 ? 0x7fffffffu : b[i] << 23);
        float f[kPer];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 d = decode2((j < 2 ? c[i].x : c[i].y) >> (16 * (j % 2)));
            f[2 * j] = d.x * s;
            f[2 * j + 1] = d.y * s;
        }
        T* o = out + row[i] * a.ldo + col[i];
        const bool all = VEC && whole<T>(sub, left[i]);
        if constexpr (sizeof(T) == 4) {
            if (all) {
                *reinterpret_cast<float4*>(o + column<T, true>(sub, 0)) = make_float4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4*>(o + column<T, true>(sub, 4)) = make_float4(f[4], f[5], f[6], f[7]);
            } else {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if ((int)column<T, VEC>(sub, j) < left[i]) o[column<T, VEC>(sub, j)] = f[j];
            }
        } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = bf16x2(f[2 * j], f[2 * j + 1]);
            if (all) {
                *reinterpret_cast<uint4*>(o + column<T, true>(sub, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if ((int)column<T, VEC>(sub, j) < left[i]) o[column<T, VEC>(sub, j)] = (uint16_t)(w[j / 2] >> (16 * (j % 2)));
            }
        }
    }
}

inline bool vec16(const void* p, uint64_t ld, size_t esz) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * esz % 16 == 0;
}

}  // namespace

cudaError_t launch_pack8(const Pack8Args& a, int dtype, bool tiles, cudaStream_t s) {
    const bool vec = vec16(a.x, a.ldx, dtype == 0 ? 4 : 2);
    const uint32_t per = (uint32_t)(kThreads / kLanes * kItems), grid = tiles ? a.nrow_blk * a.nblk : (a.items - 1) / per + 1;
    auto launch = [&](auto kernel) { return launch_early(kernel, grid, kThreads, 0, 0, s, a); };
    if (tiles && dtype == 0) return vec ? launch(pack_tiles_kernel<float, true>) : launch(pack_tiles_kernel<float, false>);
    if (tiles) return vec ? launch(pack_tiles_kernel<uint16_t, true>) : launch(pack_tiles_kernel<uint16_t, false>);
    if (dtype == 0) return vec ? launch(pack_rows_kernel<float, true>) : launch(pack_rows_kernel<float, false>);
    return vec ? launch(pack_rows_kernel<uint16_t, true>) : launch(pack_rows_kernel<uint16_t, false>);
}

cudaError_t launch_unpack8(const Unpack8Args& a, int dtype, cudaStream_t s) {
    const bool vec = vec16(a.out, a.ldo, dtype == 0 ? 4 : 2);
    const uint32_t per = (uint32_t)(kThreads / kLanes * kItems), grid = (a.items - 1) / per + 1;
    auto launch = [&](auto kernel) { return launch_early(kernel, grid, kThreads, 0, 0, s, a); };
    if (dtype == 0) return vec ? launch(unpack_kernel<float, true>) : launch(unpack_kernel<float, false>);
    return vec ? launch(unpack_kernel<uint16_t, true>) : launch(unpack_kernel<uint16_t, false>);
}

}  // namespace s2
