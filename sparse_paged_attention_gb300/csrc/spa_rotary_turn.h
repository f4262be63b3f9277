// spa_rotary_turn.h - a position times a frequency, as the fraction of a turn that it is.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define SPA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SPA_HOST_DEVICE inline
#endif

namespace spa {

// The upper 32 bits of pos * turns modulo 2^64: the fraction of a turn in [-1/2, 1/2), in units of 2^-32 (cut off,
// not rounded).  Unsigned, because the product is meant to wrap, and a signed one must not.
SPA_HOST_DEVICE int32_t turn_of(int32_t pos, int64_t turns) {
  return (int32_t)(uint32_t)(((uint64_t)(int64_t)pos * (uint64_t)turns) >> 32);
}

}  // namespace spa
