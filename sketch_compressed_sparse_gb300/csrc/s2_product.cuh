// What the products of packed matrices share: the way of their sums from tensor
// memory to Y [M][N] (y, ldy, M and dtype, 0 float32 or 1 bfloat16, of A).
#pragma once

#include "s2_tc.cuh"

namespace s2 {
namespace tc {

__device__ __forceinline__ uint16_t to_bf16(float v) {
    uint16_t h;  // the one rounding to 16 bits: Y's own type
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
    return h;
}

template <typename A>
__device__ __forceinline__ void store(const A& a, uint32_t t, uint32_t f, float v) {
    const uint64_t at = (uint64_t)t * a.ldy + f;
    if (a.dtype == 0) static_cast<float*>(a.y)[at] = v;
    else static_cast<uint16_t*>(a.y)[at] = to_bf16(v);
}

// Feature f of sixteen neighbouring tokens, from t on.
template <typename A>
__device__ __forceinline__ void store16(const A& a, uint32_t t, uint32_t f, const uint32_t* r) {
    if (t + 16 > a.M) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (t + j < a.M) store(a, t + j, f, __uint_as_float(r[j]));
    } else if (a.dtype == 0) {
        float* p = static_cast<float*>(a.y) + (uint64_t)t * a.ldy + f;
#pragma unroll
        for (int j = 0; j < 16; ++j, p += a.ldy) *p = __uint_as_float(r[j]);
    } else {
        uint16_t* p = static_cast<uint16_t*>(a.y) + (uint64_t)t * a.ldy + f;
#pragma unroll
        for (int j = 0; j < 16; ++j, p += a.ldy) *p = to_bf16(__uint_as_float(r[j]));
    }
}

// 16 columns of an accumulator and, if there are any, of the sum of the chunks before.
__device__ __forceinline__ void load_sums16(uint32_t acc, uint32_t sum, bool before, uint32_t* r) {
    uint32_t q[16];
    tmem_ld16(acc, r);
    if (before) tmem_ld16(sum, q);
    wait_ld16(r);
    if (before) {
        wait_ld16(q);
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(q[j]) + __uint_as_float(r[j]));
    }
}

}  // namespace tc
}  // namespace s2
