// Eight elements at a time, for the kernels that norm, rotate and append.
#pragma once

#include "kv.h"

namespace palu {

// eight consecutive elements: as they lie in memory, and as four packed pairs of fp32 values
template <typename T> struct Vec8 {
  uint4 r[sizeof(T) / 2];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const T*>(base) + i);
#pragma unroll
    for (int k = 0; k < int(sizeof(T) / 2); ++k) r[k] = p[k];
  }
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    uint4* p = reinterpret_cast<uint4*>(static_cast<T*>(base) + i);
#pragma unroll
    for (int k = 0; k < int(sizeof(T) / 2); ++k) p[k] = r[k];
  }
  __device__ __forceinline__ void get(uint64_t (&x)[4]) const {
    const T* e = reinterpret_cast<const T*>(r);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = pair(to_f32(e[2 * j]), to_f32(e[2 * j + 1]));
  }
  __device__ __forceinline__ void set(const uint64_t (&x)[4]) {
    T* e = reinterpret_cast<T*>(r);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = unpair(x[j]);
      e[2 * j] = from_f32<T>(v.x);
      e[2 * j + 1] = from_f32<T>(v.y);
    }
  }
};

}  // namespace palu
