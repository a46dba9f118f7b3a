// What the sampler (flce_sample.hip) and the verification of drafted tokens
// (flce_verify.hip) share: keys, exact weights and parameters of a row of
// logits, and sums over a work-group.  sample_rows.hpp explains them.
#pragma once

#include <type_traits>

#include "flce_internal.hpp"
#include "row_ops.hpp"
#include "sample_rule.hpp"

namespace flce {

constexpr uint32_t kKeyNegInf = 0x007FFFFFu;
constexpr int kSmall = 2048;         // rows one wave holds
constexpr int kGroup = 64;           // logits per stored maximum
constexpr int kPieceGroups = kPiece / kGroup;
constexpr int kSlots = 128;          // bins of z per piece; the last holds the rest
constexpr int kScanThreads = 256;

constexpr double kInfMax = 1e300;   // stands for an infinite maximum

// A row's distribution after the filters: the kept logits are those whose
// composite reaches `cut` and whose integer weight reaches min-p's.
struct RowStat {
  u64 cut;
  u64 sum;         // of their integer weights
  uint32_t kmax;   // key of the row's maximum
  uint32_t live;   // 0: nothing to draw (no logit above -inf, or a parameter out of range)
};

struct SampleArgs {
  const void* z;
  int64_t ld;      // elements
  const float* u;
  int64_t N, V;
  flce_sample_params_t prm;
  int s;           // weights are multiples of 2^-s
  int64_t* tokens;
  float* logprobs;
  // left by the scan (rows longer than kSmall)
  int pieces;
  uint32_t* pmax;   // [N][pieces] key of the piece's maximum
  double* psum;     // [N][pieces] its weight relative to that maximum
  uint32_t* gmax;   // [N][pieces][kPieceGroups] keys
  u64* hist;        // [N][pieces][kSlots]
};

// Statistics of two sets of rows instead of tokens (kStats): the first n1 rows
// are z's with a parameter for every per1 of them, the others z2's.  (A type of
// its own: a kernel's arguments are copied to every lane's scratch memory for the
// functions that are not inlined, 1 us of a drawn token, 3 of 64.)
struct StatsArgs : SampleArgs {
  RowStat* stats;
  const void* z2;
  int64_t ld2, n1;
  uint32_t per1, per2;
  flce_sample_params_t prm2;
};
template <bool kStats>
using RowArgs = std::conditional_t<kStats, StatsArgs, SampleArgs>;

template <typename T, bool kStats>
__device__ __forceinline__ const T* row_logits(const RowArgs<kStats>& a, int64_t row) {
  if constexpr (kStats) {
    if (row >= a.n1) return static_cast<const T*>(a.z2) + (row - a.n1) * a.ld2;
  }
  return static_cast<const T*>(a.z) + row * a.ld;
}

__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.0f : kNegInf; }   // NaN, -0

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __builtin_bit_cast(float, k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Coefficients of P, held in scalar registers: they feed the multiply-adds
// directly there, where literals take two moves each.  The empty asm keeps
// the compiler from seeing their values.
struct ExpCoef {
  double c[8];
  __device__ __forceinline__ void load() {
    const double v[8] = {0x1.62e42fef9cc69p-1,  0x1.ebfbdff82a733p-3,  0x1.c6b08da70cce5p-5,  0x1.3b2ab70ad2596p-7,
                         0x1.5d87759834f12p-10, 0x1.4308c7183804ap-13, 0x1.00c0e4e161930p-16, 0x1.63b2d79cc14d7p-20};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = v[i];
      asm("" : "+s"(c[i]));
    }
  }
};

// A row's parameters and the weights they define.
struct RowParams {
  double t, p, q, zmax, rate;   // rate = log2(e) / t
  ExpCoef coef;
  int64_t k;
  float u, xmin;
  bool ok;

  __device__ __forceinline__ void set_max(float m) {
    zmax = m < __builtin_inff() ? (double)m : kInfMax;
    xmin = (float)((double)m - t * (0.69314718055994530942 * 0.8 * 0x1p30));
  }
};

template <bool kStats>
__device__ __forceinline__ RowParams row_params(const RowArgs<kStats>& a, int64_t row) {
  RowParams r;
  const flce_sample_params_t* of = &a.prm;
  if constexpr (kStats) {
    const bool second = row >= a.n1;
    if (second) of = &a.prm2;
    row = second ? (uint32_t)(row - a.n1) / a.per2 : (uint32_t)row / a.per1;
  }
  const flce_sample_params_t& prm = *of;
  const float t = prm.temperature_rows ? prm.temperature_rows[row] : prm.temperature;
  const float p = prm.top_p_rows ? prm.top_p_rows[row] : prm.top_p;
  const float q = prm.min_p_rows ? prm.min_p_rows[row] : prm.min_p;
  r.k = prm.top_k_rows ? prm.top_k_rows[row] : prm.top_k;
  r.u = 0.0f;
  if constexpr (!kStats) r.u = a.u[row];
  r.ok = t >= 0.0f && t < __builtin_inff() && p > 0.0f && p <= 1.0f && q >= 0.0f && q <= 1.0f && r.k >= 0 &&
         r.u >= 0.0f && r.u < 1.0f;
  r.t = t;
  r.p = p;
  r.q = q;
  r.set_max(0.0f);
  r.rate = 1.4426950408889634074 / r.t;
  r.coef.load();
  return r;
}

// How a row's candidates are found.
enum Mode { kGreedy, kTopK, kMinP, kTopP, kAll };
__device__ __forceinline__ Mode mode_of(const RowParams& r, int64_t V) {
  if (r.t == 0.0) return kGreedy;
  if (r.k > 0 && r.k < V) return kTopK;
  if (r.q > 0.0) return kMinP;
  return r.p < 1.0 ? kTopP : kAll;
}

// Bins of z, 1/8 of min(t, 3/2) wide, by whole-number floats ascending with z.
// Differences of two are exact below kBinLimit.
constexpr float kBinLimit = 8388608.0f;   // 2^23
__device__ __forceinline__ float bin_scale(const RowParams& r) {
  const double a = 8.0 / (r.t < 1.5 ? r.t : 1.5);
  return (float)(a < 1e30 ? a : 1e30);
}
__device__ __forceinline__ float bin_of(float x, float alpha) { return __builtin_floorf(x * alpha); }
// The least float in bin b or above: within a few steps of b / alpha.
__device__ __forceinline__ float bin_edge(float b, float alpha) {
  uint32_t k = key_of(clean(b / alpha)) + 8;
  for (int i = 0; i < 32 && bin_of(value_of(k - 1), alpha) >= b; ++i) --k;
  return value_of(k);
}

// 2^(d rate) as 2^(n + f), |f| <= 1/2 and |d rate| < 2^31: adding 1.5 2^52
// leaves n in the low bits, 2^f = 1 + f P(f) with P through the Chebyshev
// nodes (relative error 2^-38.8; exactly 1 at d = 0), n put into the exponent.
__device__ __forceinline__ double exp2_of(double d, double rate, const ExpCoef& k) {
  const double big = __builtin_fma(d, rate, 0x1.8p52);
  const double f = __builtin_fma(d, rate, -(big - 0x1.8p52));
  double v = k.c[7];
#pragma unroll
  for (int i = 6; i >= 0; --i) v = __builtin_fma(v, f, k.c[i]);
  return __builtin_amdgcn_ldexp(__builtin_fma(v, f, 1.0), (int)(uint32_t)__builtin_bit_cast(u64, big));
}
// exp((x - max) / t) in any row: the maximum may be infinite (zmax is 1e300
// then), so the exponent is clamped.
__device__ __forceinline__ double weight_any(float x, const RowParams& r) {
  const double y = ((double)x - r.zmax) * r.rate;
  return exp2_of(__builtin_fmin(__builtin_fmax(y, -1000.0), 0.0), 1.0, r.coef);
}
// In ordinary rows the clamp is one fp32 maximum: xmin lies 0.8 2^30 in the
// exponent below the row's maximum, and takes NaN and -inf too.
__device__ __forceinline__ bool ordinary(float m, const RowParams& r) {
  return (double)__builtin_fabsf(m) < r.t * 0x1p48 && r.t < 1e20;
}
__device__ __forceinline__ double weight(float x, const RowParams& r) {
  return exp2_of((double)__builtin_fmaxf(x, r.xmin) - r.zmax, r.rate, r.coef);
}

// round(w 2^s) for w <= 1, s <= 51: adding 2^52 leaves the integer in the
// mantissa.
__device__ __forceinline__ u64 fixed(double w, double scale) {
  return __builtin_bit_cast(u64, __builtin_fma(w, scale, 0x1p52)) & 0xFFFFFFFFFFFFFull;
}

__device__ __forceinline__ double scale_of(const SampleArgs& a) {
  return __builtin_bit_cast(double, (u64)(1023 + a.s) << 52);
}

// The least integer weight that min-p keeps (a weight of 0 is never drawn).
__device__ __forceinline__ u64 floor_weight(const RowParams& r, double scale) {
  const u64 f = (u64)ceil(r.q * scale);
  return f < 1 ? 1 : f;
}

// The share of a sum that u (or p) asks for, as a running-sum target.
__device__ __forceinline__ u64 draw_target(float u, u64 sum) {
  const u64 t = (u64)((double)u * (double)sum);
  return t < sum ? t : sum - 1;
}
__device__ __forceinline__ u64 share(double p, u64 sum) {
  const u64 n = (u64)ceil(p * (double)sum);
  return n < 1 ? 1 : n > sum ? sum : n;
}

// A row's result; `weight_sum` is the kept set's.  Its logarithm starts
// from the hardware's fp32 one and takes one step of log s = log a + log(1 +
// (s / a - 1)), where the rest is below 1e-6.
__device__ __forceinline__ void emit(const SampleArgs& a, int64_t row, int64_t tok, float x, const RowParams& r,
                                     double weight_sum) {
  a.tokens[row] = tok;
  if (!a.logprobs) return;
  const double l2 = (double)__builtin_amdgcn_logf((float)weight_sum);
  const double e = __builtin_fma(weight_sum, exp2_of(-l2, 1.0, r.coef), -1.0);
  const double ls = __builtin_fma(l2, 0.69314718055994530942, e - 0.5 * e * e);
  const double y = __builtin_fmin(((double)x - r.zmax) * r.rate, 0.0);
  a.logprobs[row] = (float)(__builtin_fma(y, 0.69314718055994530942, -ls));
}
__device__ __forceinline__ void emit_none(const SampleArgs& a, int64_t row) {
  a.tokens[row] = -1;
  if (a.logprobs) a.logprobs[row] = kNegInf;
}

__device__ __forceinline__ int bits_of(u64 x) { return x ? 64 - __builtin_clzll(x) : 0; }

// Sums over a work-group of TH threads.
template <int TH>
struct GroupScratch {
  u64 wsum[TH / 64];
};

// Exclusive sum of x over the threads in order; `all` gets the whole sum.
template <int TH>
__device__ __forceinline__ u64 group_scan(u64 x, u64& all, GroupScratch<TH>& sh) {
  u64 sum;
  const u64 inc = wave_scan_u64(x, sum);
  if (TH > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh.wsum[w] = sum;
    __syncthreads();
    // every wave scans the waves' sums
    const int lane = threadIdx.x & 63;
    const u64 inc_w = wave_scan_u64(lane < TH / 64 ? sh.wsum[lane] : 0, sum);
    all = sum;
    return (w ? lane_u64(inc_w, w - 1) : 0) + inc - x;
  }
  all = sum;
  return inc - x;
}

// ---------------------------------------------------------------------------
// Candidates as composites that order them by descending logit, then
// ascending index.

__device__ __forceinline__ u64 composite(uint32_t key, int64_t i) { return (u64)key << 32 | (uint32_t)~(uint32_t)i; }
__device__ __forceinline__ uint32_t key_in(u64 c) { return (uint32_t)(c >> 32); }
__device__ __forceinline__ int64_t index_in(u64 c) { return (int64_t)(uint32_t)~(uint32_t)c; }
__device__ __forceinline__ float value_in(u64 c) { return value_of(key_in(c)); }

// What flce_sample.hip does for others: the workspace of N rows of V logits
// (total 0: not supported), the arguments that follow from it, and the checks of
// parameters.
struct SampleLayout {
  int64_t pieces;
  size_t psum, hist, gmax, total;   // byte offsets (pmax at 0)
};
SampleLayout sample_layout(int64_t N, int64_t V);
void sample_args(SampleArgs& a, int64_t N, int64_t V, const SampleLayout& l, void* workspace);
bool sample_params_ok(const flce_sample_params_t& q);

}  // namespace flce
