// Helpers of the row-wise operators around the vocabulary head (norms,
// dropout, sampling): vectors that need no alignment beyond their element's,
// sums over a 64-lane wave and over a row's threads, and launch shapes.
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

// The same in two steps, for loads that stay under way: load_clamped reads a
// whole vector at `col`, or the row's last whole one where that would cross or
// lie past the row's end (rows of at least one vector); row_tail, at the
// vector's use, moves the elements that belong to it down and clears the rest.
template <typename T>
__device__ __forceinline__ typename RowVec<T>::type load_clamped(const T* p, int col, int n) {
  constexpr int E = RowVec<T>::E;
  if (n < E) return load_row(p, col, n);
  return *reinterpret_cast<const typename RowVec<T>::mem*>(p + (col + E <= n ? col : n - E));
}
template <typename T>
__device__ __forceinline__ void row_tail(typename RowVec<T>::type& v, int col, int n) {
  constexpr int E = RowVec<T>::E;
  const int over = n < E ? 0 : col + E - n;   // (shorter rows were read element by element)
  if (!__builtin_amdgcn_ballot_w64(over > 0)) return;
  u32x4 x = __builtin_bit_cast(u32x4, v);
  if (over >= E) x = u32x4{0, 0, 0, 0};
  const int k = over > 0 ? over * (8 / E) : 0;   // in halves of 2 bytes (bf16: elements)
  if (k & 4) x = u32x4{x[2], x[3], 0, 0};
  if (k & 2) x = u32x4{x[1], x[2], x[3], 0};
  if (k & 1) x = u32x4{x[0] >> 16 | x[1] << 16, x[1] >> 16 | x[2] << 16, x[2] >> 16 | x[3] << 16, x[3] >> 16};
  v = __builtin_bit_cast(typename RowVec<T>::type, x);
}

template <typename T>
__device__ __forceinline__ void store_row(T* p, int64_t col, int64_t n, typename RowVec<T>::type v) {
  constexpr int E = RowVec<T>::E;
  if (col + E <= n) {
    *reinterpret_cast<typename RowVec<T>::mem*>(p + col) = v;
  } else if (col < n) {
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

__device__ __forceinline__ float wave_max(float x) {   // no NaN
  x = __builtin_fmaxf(x, dpp_f32<0xB1>(x));
  x = __builtin_fmaxf(x, dpp_f32<0x4E>(x));
  x = __builtin_fmaxf(x, dpp_f32<0x141>(x));
  x = __builtin_fmaxf(x, dpp_f32<0x140>(x));
  return __builtin_fmaxf(__builtin_fmaxf(lane_f32(x, 0), lane_f32(x, 16)),
                         __builtin_fmaxf(lane_f32(x, 32), lane_f32(x, 48)));
}

template <int ctrl>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x) {
  auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  x = larger(x, dpp_u32<0xB1>(x));
  x = larger(x, dpp_u32<0x4E>(x));
  x = larger(x, dpp_u32<0x141>(x));
  x = larger(x, dpp_u32<0x140>(x));
  auto lane = [=](int l) { return (uint32_t)__builtin_amdgcn_readlane((int)x, l); };
  return larger(larger(lane(0), lane(16)), larger(lane(32), lane(48)));
}

__device__ __forceinline__ uint32_t wave_sum_u32(uint32_t x) {
  x += dpp_u32<0xB1>(x);
  x += dpp_u32<0x4E>(x);
  x += dpp_u32<0x141>(x);
  x += dpp_u32<0x140>(x);
  auto lane = [=](int l) { return (uint32_t)__builtin_amdgcn_readlane((int)x, l); };
  return (lane(0) + lane(16)) + (lane(32) + lane(48));
}

// How many lower lanes are set in `mask`.
__device__ __forceinline__ int lane_rank(unsigned long long mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// The same on 64-bit values, moved by halves.
typedef unsigned long long u64;
template <int ctrl>
__device__ __forceinline__ u64 dpp_u64(u64 x) {
  return (u64)dpp_u32<ctrl>((uint32_t)(x >> 32)) << 32 | dpp_u32<ctrl>((uint32_t)x);
}
__device__ __forceinline__ u64 lane_u64(u64 x, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), lane);
  return (u64)hi << 32 | lo;
}
__device__ __forceinline__ u64 wave_sum_u64(u64 x) {
  x += dpp_u64<0xB1>(x);
  x += dpp_u64<0x4E>(x);
  x += dpp_u64<0x141>(x);
  x += dpp_u64<0x140>(x);
  return (lane_u64(x, 0) + lane_u64(x, 16)) + (lane_u64(x, 32) + lane_u64(x, 48));
}
__device__ __forceinline__ u64 wave_min_u64(u64 x) {
  auto less = [](u64 a, u64 b) { return a < b ? a : b; };
  x = less(x, dpp_u64<0xB1>(x));
  x = less(x, dpp_u64<0x4E>(x));
  x = less(x, dpp_u64<0x141>(x));
  x = less(x, dpp_u64<0x140>(x));
  return less(less(lane_u64(x, 0), lane_u64(x, 16)), less(lane_u64(x, 32), lane_u64(x, 48)));
}
__device__ __forceinline__ double wave_sum_f64(double x) {
  auto bits = [](double v) { return __builtin_bit_cast(u64, v); };
  auto val = [](u64 v) { return __builtin_bit_cast(double, v); };
  x += val(dpp_u64<0xB1>(bits(x)));
  x += val(dpp_u64<0x4E>(bits(x)));
  x += val(dpp_u64<0x141>(bits(x)));
  x += val(dpp_u64<0x140>(bits(x)));
  return (val(lane_u64(bits(x), 0)) + val(lane_u64(bits(x), 16))) +
         (val(lane_u64(bits(x), 32)) + val(lane_u64(bits(x), 48)));
}
// Inclusive sum over the lanes in order; `all` gets the whole sum.
__device__ __forceinline__ u64 wave_scan_u64(u64 x, u64& all) {
  x += dpp_u64<0x111>(x);   // from 1, 2, 4, 8 lanes below within 16
  x += dpp_u64<0x112>(x);
  x += dpp_u64<0x114>(x);
  x += dpp_u64<0x118>(x);
  const u64 a = lane_u64(x, 15), b = a + lane_u64(x, 31), c = b + lane_u64(x, 47);
  const int lane = threadIdx.x & 63;
  x += lane < 16 ? 0 : lane < 32 ? a : lane < 48 ? b : c;
  all = lane_u64(x, 63);
  return x;
}

__device__ __forceinline__ uint32_t wave_scan_u32(uint32_t x, uint32_t& all) {
  x += dpp_u32<0x111>(x);
  x += dpp_u32<0x112>(x);
  x += dpp_u32<0x114>(x);
  x += dpp_u32<0x118>(x);
  auto lane = [](uint32_t v, int l) { return (uint32_t)__builtin_amdgcn_readlane((int)v, l); };
  const uint32_t a = lane(x, 15), b = a + lane(x, 31), c = b + lane(x, 47);
  const int l = threadIdx.x & 63;
  x += l < 16 ? 0 : l < 32 ? a : l < 48 ? b : c;
  all = lane(x, 63);
  return x;
}

// The parameter's vector of a thread; absent parameters read as `fill`.
template <typename WT, int E>
__device__ __forceinline__ void load_param(float (&out)[E], const void* p, int col, int H, float fill) {
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = fill;
  if (!p) return;
  constexpr int W = RowVec<WT>::E;
  constexpr int step = W < E ? W : E;   // a narrower row vector takes part of a parameter vector
#pragma unroll
  for (int q = 0; q < E / step; ++q) {
    const int c = col + q * step;
    if (W <= E) {
      const typename RowVec<WT>::type v = load_row(static_cast<const WT*>(p), c, H, fill);
#pragma unroll
      for (int e = 0; e < step; ++e) out[q * step + e] = to_f32(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < step; ++e)
        if (c + e < H) out[e] = to_f32(static_cast<const WT*>(p)[c + e]);
    }
  }
}

// Sums of N values over the kRow threads of a row (every thread gets them).
// Rows wider than a wave go through LDS; `buf` alternates between calls so
// that one barrier per call is enough.
template <int N> using SumLds = float[2][N][16];
template <int kRow, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], SumLds<N>& lds, int& buf) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (kRow == 64) return;
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) lds[buf][i][w] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < kRow / 64; ++k) v[i] += lds[buf][i][k];
  }
  buf ^= 1;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The longest rows kept in registers: 2048 vectors of 16 bytes.
constexpr int64_t kMaxRegVecs = 2048;

inline int64_t row_vecs(int64_t H, int64_t elem_bytes) { return ceil_div(H, 16 / elem_bytes); }

// Work-groups for `sets` of rows, at most `most`: as few as leave every one
// the same number of steps.
inline int64_t even_grid(int64_t sets, int64_t most) {
  if (sets <= most) return sets;
  return ceil_div(sets, ceil_div(sets, most));
}

}  // namespace flce
