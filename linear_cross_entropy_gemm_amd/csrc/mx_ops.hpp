// The block formats of the OCP Microscaling specification (v1.0): 32 elements
// along a row share a scale 2^(code - 127) (E8M0, code 255 is NaN); elements
// are E4M3 (8 bits) or E2M1 (4 bits).  The scale is the least power of two
// under which no element of the block passes the format's largest value.
#pragma once

#include "row_ops.hpp"

namespace flce {

constexpr int kMxBlock = 32;

// Largest magnitude of a block, as bits (ordered like the magnitudes; NaN is
// above infinity): this lane's E elements and those of the other lanes of its
// aligned group of 32 / E.  Every lane of the wave is active.
template <int E>
__device__ __forceinline__ uint32_t block_max_bits(const float (&y)[E]) {
  static_assert(E == 4 || E == 8, "4 or 8 lanes hold a block");
  auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) m = larger(m, __builtin_bit_cast(uint32_t, y[e]) & 0x7FFFFFFFu);
  m = larger(m, dpp_u32<0xB1>(m));               // lane ^ 1
  m = larger(m, dpp_u32<0x4E>(m));               // lane ^ 2
  if (E == 4) m = larger(m, dpp_u32<0x141>(m));  // mirror within 8
  return m;
}

// Scale codes for a block's largest magnitude: 448 = 1.75 2^8, 6 = 1.5 2^2.
template <int kExp, uint32_t kMant>
__device__ __forceinline__ uint32_t mx_code(uint32_t max_bits) {
  if (max_bits >= 0x7F800000u) return 255;
  const int c = (int)(max_bits >> 23) - kExp + ((max_bits & 0x7FFFFFu) > kMant ? 1 : 0);
  return c > 0 ? (uint32_t)c : 0u;
}
__device__ __forceinline__ uint32_t mx8_code(uint32_t max_bits) { return mx_code<8, 0x600000u>(max_bits); }
__device__ __forceinline__ uint32_t mx4_code(uint32_t max_bits) { return mx_code<2, 0x400000u>(max_bits); }

// 1 / scale, exact: the codes of finite blocks stop at 253 (of no use with 255).
__device__ __forceinline__ float mx_inverse(uint32_t code) {
  return __builtin_bit_cast(float, (254u - code) << 23);
}

// E elements as E4M3 at [col, col + E) of a row of n bytes (rounded to nearest
// even; every element of a block without a scale is NaN).
template <int E>
__device__ __forceinline__ void store_e4m3(uint8_t* p, int col, int n, const float (&y)[E], uint32_t code) {
  const float inv = mx_inverse(code);
  uint32_t w[E / 4];
#pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * q] * inv, y[4 * q + 1] * inv, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * q + 2] * inv, y[4 * q + 3] * inv, v, true);
    w[q] = code == 255 ? 0x7F7F7F7Fu : (uint32_t)v;
  }
  if (col + E <= n) {
    typedef uint32_t mem __attribute__((ext_vector_type(E / 4), aligned(1)));
    mem v;
#pragma unroll
    for (int q = 0; q < E / 4; ++q) v[q] = w[q];
    *reinterpret_cast<mem*>(p + col) = v;
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (col + e < n) p[col + e] = (uint8_t)(w[e / 4] >> 8 * (e % 4));
  }
}

}  // namespace flce
