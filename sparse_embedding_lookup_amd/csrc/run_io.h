// run_io.h -- runs of neighbouring elements of a row, widened to fp32 and back.  A run needs
// the alignment of its elements only (the memory pipeline takes any), and never reaches past
// the elements it is told of.
#pragma once

#include <type_traits>

#include "ctr_internal.h"

namespace ctr {

template <int TY>
constexpr int kEltSize = TY == kEltF32 ? 4 : 2;

template <int TY>
__device__ __forceinline__ void store_elt(void* p, int64_t i, float v) {
  if constexpr (TY == kEltF32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)to_half<TY, false>(v, 0u);
}

// N elements as they are stored (one element, or whole 4-byte words).
template <int TY, int N>
struct Run {
  static constexpr int kWords = (N * kEltSize<TY> + 3) / 4;
  static_assert(N == 1 || N * kEltSize<TY> % 4 == 0, "whole words");
  uint32_t u[kWords];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (N == 1) {
      if constexpr (TY == kEltF32) u[0] = static_cast<const uint32_t*>(p)[i];
      else u[0] = static_cast<const uint16_t*>(p)[i];
    } else {
      __builtin_memcpy(u, static_cast<const char*>(p) + i * kEltSize<TY>, sizeof(u));
    }
  }
  // The first `there` of them; the others zero.
  __device__ __forceinline__ void load_some(const void* p, int64_t i, int there) {
    if (there >= N) {
      load(p, i);
      return;
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) u[w] = 0u;
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < there) {
        if constexpr (TY == kEltF32) u[e] = static_cast<const uint32_t*>(p)[i + e];
        else u[e / 2] |= (uint32_t) static_cast<const uint16_t*>(p)[i + e] << (e & 1 ? 16 : 0);
      }
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (TY == kEltF32) return __uint_as_float(u[e]);
    else return e & 1 ? half_hi<TY>(u[e / 2]) : half_lo<TY>(u[e / 2]);
  }
};

template <int TY, int N>
__device__ __forceinline__ void store_run(void* p, int64_t i, const float* v) {
  if constexpr (N == 1) {
    store_elt<TY>(p, i, v[0]);
  } else {
    uint32_t u[Run<TY, N>::kWords];
#pragma unroll
    for (int w = 0; w < Run<TY, N>::kWords; ++w) {
      if constexpr (TY == kEltF32) u[w] = __float_as_uint(v[w]);
      else u[w] = to_half<TY, false>(v[2 * w], 0u) | (to_half<TY, false>(v[2 * w + 1], 0u) << 16);
    }
    __builtin_memcpy(static_cast<char*>(p) + i * kEltSize<TY>, u, sizeof(u));
  }
}
template <int TY, int N>
__device__ __forceinline__ void store_some(void* p, int64_t i, const float* v, int there) {
  if (there >= N) {
    store_run<TY, N>(p, i, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (e < there) store_elt<TY>(p, i + e, v[e]);
}

// f(std::integral_constant<int, the element type>).
template <typename F>
hipError_t for_type(int dtype, F f) {
  if (dtype == kEltF32) return f(std::integral_constant<int, kEltF32>{});
  if (dtype == kEltBF16) return f(std::integral_constant<int, kEltBF16>{});
  return f(std::integral_constant<int, kEltF16>{});
}

}  // namespace ctr
