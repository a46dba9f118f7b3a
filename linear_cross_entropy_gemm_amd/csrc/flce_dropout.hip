// Dropout whose mask is regenerated, never stored (flce_dropout).
//
//   y_i = [r_i +] (u_i >= floor(p 2^32) ? x_i / (1 - p) : 0)
//
// u_i is word i % 4 of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011) on the counter
// (i / 4 low, i / 4 high, offset low, offset high) under the key (seed low,
// seed high).  A word depends on the element's index alone, so the backward
// pass is the same map on the upstream gradient, and any launch shape gives
// the same mask.
//
// Bound by memory: the generator's twenty 64-bit multiplications per four
// elements run beside the loads.  470 MB in and 470 MB out take 159 us (5.9
// TB/s, the plain copy's rate), and 7 rounds instead of 10, or 16 bits per
// element instead of 32, take as long.  One vector per thread, without a loop:
// two or four of them in a row read 5 to 10% slower (5.7 and 5.5 TB/s).
#include <cmath>

#include "flce_internal.hpp"
#include "row_ops.hpp"

namespace flce {

namespace {

constexpr int kDropThreads = 256;

struct DropArgs {
  const void* x;
  const void* residual;   // null: none
  void* y;
  int64_t n;
  uint32_t threshold;     // words below it are dropped
  int drop_all;           // p = 1
  float scale;            // 1 / (1 - p)
  uint32_t k0, k1;
  uint64_t offset;
  const uint64_t* offset_dev;   // added to `offset` when not null
};

// Each round multiplies two words to 64 bits and mixes the halves with the
// other two words and the round key.
__device__ __forceinline__ u32x4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// One 16-byte vector per thread (8 bf16 or 4 fp32, two calls or one of the
// generator).
template <typename T, bool kResidual>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(DropArgs p) {
  constexpr int E = RowVec<T>::E;
  typedef typename RowVec<T>::type vec_t;
  const int64_t i = ((int64_t)blockIdx.x * kDropThreads + threadIdx.x) * E;
  if (i >= p.n) return;
  vec_t v = load_row(static_cast<const T*>(p.x), i, p.n);
  vec_t r = v;
  if (kResidual) r = load_row(static_cast<const T*>(p.residual), i, p.n);
  uint64_t off = p.offset;
  if (p.offset_dev) off += *p.offset_dev;
#pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    const uint64_t blk = (uint64_t)i / 4 + q;
    const u32x4 w = philox((uint32_t)blk, (uint32_t)(blk >> 32), (uint32_t)off, (uint32_t)(off >> 32), p.k0, p.k1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool keep = w[e] >= p.threshold && !p.drop_all;
      const float x = keep ? to_f32(v[4 * q + e]) : 0.0f;   // a dropped infinity or NaN leaves no trace
      // one rounding of r + x / (1 - p) to fp32, one to the storage dtype
      v[4 * q + e] = (T)(kResidual ? __builtin_fmaf(x, p.scale, to_f32(r[4 * q + e])) : x * p.scale);
    }
  }
  store_row(static_cast<T*>(p.y), i, p.n, v);
}

template <typename T>
void launch_dropout(const DropArgs& p, hipStream_t stream) {
  const int64_t per = (int64_t)kDropThreads * RowVec<T>::E;
  const unsigned grid = (unsigned)((p.n + per - 1) / per);
  if (p.residual)
    dropout_kernel<T, true><<<grid, kDropThreads, 0, stream>>>(p);
  else
    dropout_kernel<T, false><<<grid, kDropThreads, 0, stream>>>(p);
}

// y may be an input itself, and must not overlap it otherwise.
bool partly_over(const void* in, const void* out, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out);
  return a != b && a < b + bytes && b < a + bytes;
}

}  // namespace

}  // namespace flce

extern "C" int flce_dropout(const void* x, const void* residual, void* y, int64_t n, double p, uint64_t seed,
                            uint64_t offset, const uint64_t* offset_dev, hipStream_t stream, int dtype) {
  using namespace flce;
  if (dtype != FLCE_DTYPE_BF16 && dtype != FLCE_DTYPE_F32) return FLCE_EINVAL;
  if (n < 0 || !(p >= 0.0 && p <= 1.0)) return FLCE_EINVAL;
  const uintptr_t es = dtype == FLCE_DTYPE_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(offset_dev) % 8 != 0) return FLCE_EINVAL;
  if (n > 0 && (!x || !y)) return FLCE_EINVAL;
  if (reinterpret_cast<uintptr_t>(x) % es != 0 || reinterpret_cast<uintptr_t>(y) % es != 0 ||
      reinterpret_cast<uintptr_t>(residual) % es != 0)
    return FLCE_EINVAL;
  if (n > (int64_t(1) << 33)) return FLCE_EUNSUPPORTED;   // a launch holds fewer than 2^32 threads
  if (n == 0) return FLCE_OK;
  const size_t bytes = (size_t)n * es;
  if (partly_over(x, y, bytes) || (residual && partly_over(residual, y, bytes))) return FLCE_EINVAL;
  DropArgs a;
  a.x = x;
  a.residual = residual;
  a.y = y;
  a.n = n;
  a.drop_all = p >= 1.0;
  a.threshold = a.drop_all ? 0xFFFFFFFFu : (uint32_t)(p * 4294967296.0);
  a.scale = a.drop_all ? 0.0f : (float)(1.0 / (1.0 - p));
  a.k0 = (uint32_t)seed;
  a.k1 = (uint32_t)(seed >> 32);
  a.offset = offset;
  a.offset_dev = offset_dev;
  ProfileScope ps(FLCE_KERNEL_DROPOUT, stream);
  if (dtype == FLCE_DTYPE_BF16)
    launch_dropout<bf16>(a, stream);
  else
    launch_dropout<float>(a, stream);
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}
