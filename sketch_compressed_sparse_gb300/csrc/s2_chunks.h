// How the stages of a long sum are divided into chunks. (Plain C++: tests
// compile this file by itself.)
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define S2_BOTH __host__ __device__ __forceinline__
#else
#define S2_BOTH inline
#endif

namespace s2 {

// Chunks of at most `most` stages that `stages` stages need.
S2_BOTH uint32_t chunk_count(uint32_t stages, uint32_t most) { return (stages + most - 1) / most; }

// The stage that chunk c (of `chunks`) ends before. (In 64 bits: the product of
// the two numbers passes 2^32 from 217,000 stages in chunks of 11 on.)
S2_BOTH uint32_t chunk_end(uint32_t stages, uint32_t chunks, uint32_t c) {
    return (uint32_t)((uint64_t)stages * (c + 1) / chunks);
}

}  // namespace s2
