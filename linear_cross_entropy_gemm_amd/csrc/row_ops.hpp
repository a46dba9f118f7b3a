// Helpers of the row-wise operators around the vocabulary head (layer norm,
// dropout, sampling): vectors that need no alignment beyond their element's,
// and sums over a 64-lane wave.
#pragma once

#include "device_common.hpp"

namespace flce {

// 16 bytes of consecutive elements at any element address.  gfx950 serves
// global accesses at any byte address under the HSA ABI, so a row of odd
// length or odd stride still moves 16 bytes per load; only a vector that
// crosses the end of its row is moved element by element.
template <typename T> struct RowVec;
template <> struct RowVec<bf16> {
  static constexpr int E = 8;
  typedef __bf16 type __attribute__((ext_vector_type(8)));
  typedef __bf16 mem __attribute__((ext_vector_type(8), aligned(2)));
};
template <> struct RowVec<float> {
  static constexpr int E = 4;
  typedef float type __attribute__((ext_vector_type(4)));
  typedef float mem __attribute__((ext_vector_type(4), aligned(4)));
};

// Elements [col, col + E) of the row p of n elements; those at n and beyond
// read as `fill`.
template <typename T>
__device__ __forceinline__ typename RowVec<T>::type load_row(const T* p, int64_t col, int64_t n, float fill = 0.0f) {
  constexpr int E = RowVec<T>::E;
  typename RowVec<T>::type v;
  if (col + E <= n) {
    v = *reinterpret_cast<const typename RowVec<T>::mem*>(p + col);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = (T)fill;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (col + e < n) v[e] = p[col + e];
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void store_row(T* p, int64_t col, int64_t n, typename RowVec<T>::type v) {
  constexpr int E = RowVec<T>::E;
  if (col + E <= n) {
    *reinterpret_cast<typename RowVec<T>::mem*>(p + col) = v;
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (col + e < n) p[col + e] = v[e];
  }
}

// Sum over the wave's 64 lanes in a fixed order (every lane active): adds
// within 16 lanes by data-parallel moves, then the four groups' totals.
template <int ctrl>
__device__ __forceinline__ float dpp_f32(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_f32(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
__device__ __forceinline__ float wave_sum(float x) {
  x += dpp_f32<0xB1>(x);    // lane ^ 1
  x += dpp_f32<0x4E>(x);    // lane ^ 2
  x += dpp_f32<0x141>(x);   // mirror within 8
  x += dpp_f32<0x140>(x);   // mirror within 16
  return (lane_f32(x, 0) + lane_f32(x, 16)) + (lane_f32(x, 32) + lane_f32(x, 48));
}

}  // namespace flce
