// Drawing a token from each row of logits (flce_sample): temperature, top-k,
// top-p and min-p filters, then the inverse of the distribution function in
// index order at a given random number.
//
// Weights are integers: W = round(2^s exp((z - max) / t)), with s chosen so
// that a row's sum stays below 2^62.  Sums of integers are exact, so the order
// of atomics changes no decision and the same call gives the same bits; the
// rounding, 2^-(s+1) per token next to the largest token's 1, is far below
// what a 24-bit random number or an fp32 probability resolves (s is 44 at a
// vocabulary of 2^18).  Where a row is split into pieces, a piece's weights are
// relative to its own maximum: their sum (of integers in the bins, of doubles
// in a fixed order without them) is brought to the row's by a rounded 64-bit
// product, so the ways through the kernels agree to about 2^-38 of the row's
// weight, not to the bit.  The exponential is taken in 64 bits (relative error
// 2^-38.8) for the same reason: an fp32 one moves the borders between tokens
// of a flat row by more than their spacing warrants.
//
// Rows of up to 2048 logits stay in one wave's registers
// (sample_small_kernel).  A longer row passes through the chip once, in
// pieces of 8192 logits spread over the work-groups of sample_scan_kernel,
// which leaves behind what decides where the answer lies:
//   * the maximum of each 64 logits and of the piece;
//   * with top-p alone: the piece's weight by bins of z, 1/8 of min(t, 3/2) wide,
//     counted down from the piece's maximum (bins are aligned in z, so bins
//     of different pieces add up);
//   * without any filter, or with min-p: the piece's weight.
// sample_pick_kernel (one work-group per row) then looks only where it has
// to:
//   * top-k: the k-th largest of the 64-logit maxima bounds the k-th logit
//     from below, so every candidate lies in a group whose maximum reaches it;
//   * min-p: the candidates reach the maximum + t ln q;
//   * top-p alone: the bin in which the weight from above reaches p of the
//     row's: the candidates are the logits from that bin up where those are
//     few, and the bin's own logits where the kept set is most of a flat row;
//   * then one wave compares up to 64 candidates with each other, or a search
//     in LDS finds the cuts among up to 12288, or, in a flat row, the weights
//     of one piece are summed in index order.
// What bounds them: the scan the memory where no weights are needed (256 rows
// of 202048 bf16 logits, 103 MB, in 19 us: 5.4 TB/s, a plain copy's rate);
// where they are it takes 46 us, 58 with the bins, of which 17 64-bit
// operations per logit explain 22 at the vector units' nominal rate; the pick the latency of one row's steps (11
// to 17 us on a short list, of which a third is waiting for memory and a third
// for instructions that no earlier work-group fetched; 42 us in a flat row of
// 129279 fp32 logits, 61 us in 256 flat rows of 202048 bf16 ones, half of it
// reading the row once more).
// Rows for which that does not work out (a list that overflows, a cut below
// the bins) take the searches over the whole row at the end of the kernel: one
// row of 202048 bf16 logits then takes 95 us with min-p, 260 with top-p and 210
// with top-k, 256 rows 155, 355 and 270.  Normal logits come to that with min-p
// 0.05 at a standard deviation (over t) of 0.8, with top-p 0.9 at 0.6, with
// top-k at k above 12288.
//
// Values are compared through keys, 32-bit integers in the order of the
// logits (equal zeros share a key, NaN counts as -inf).  The kept set of
// every filter is "key above K, or key K and index at most I", so a filter
// is a search for (K, I).
#include <cmath>

#include "flce_internal.hpp"
#include "row_ops.hpp"

namespace flce {

namespace {

constexpr uint32_t kKeyNegInf = 0x007FFFFFu;
constexpr int kSmall = 2048;         // rows one wave holds
constexpr int kPiece = 8192;         // logits per work-group of the scan
constexpr int kGroup = 64;           // logits per stored maximum
constexpr int kPieceGroups = kPiece / kGroup;
constexpr int kSlots = 128;          // bins of z per piece; the last holds the rest
constexpr int kScanThreads = 256;

constexpr double kInfMax = 1e300;   // stands for an infinite maximum

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

__device__ __forceinline__ RowParams row_params(const SampleArgs& a, int64_t row) {
  RowParams r;
  const float t = a.prm.temperature_rows ? a.prm.temperature_rows[row] : a.prm.temperature;
  const float p = a.prm.top_p_rows ? a.prm.top_p_rows[row] : a.prm.top_p;
  const float q = a.prm.min_p_rows ? a.prm.min_p_rows[row] : a.prm.min_p;
  r.k = a.prm.top_k_rows ? a.prm.top_k_rows[row] : a.prm.top_k;
  r.u = a.u[row];
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

// Draws from n <= 64 candidates, one per lane of a wave (c = 0 beyond them),
// that hold every token at least as likely as the least of them.  top-p is a
// share of the candidates' weight after top-k, or of `row_sum` where that is
// not 0.  A candidate's rank and the weights before it come from comparing it
// with every other one.
__device__ __forceinline__ void pick_in_wave(const SampleArgs& a, int64_t row, u64 c, int n, const RowParams& r,
                                             bool top_k, u64 row_sum) {
  const double scale = scale_of(a);
  u64 f = c ? fixed(weight(value_in(c), r), scale) : 0;
  int rank = 0;
  u64 above = 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const bool more = lane_u64(c, i) > c;
    rank += more ? 1 : 0;
    above += more ? lane_u64(f, i) : 0;
  }
  if (top_k && rank >= r.k) f = 0;
  if (r.p < 1.0) {
    const u64 all = wave_sum_u64(f);
    if (above >= share(r.p, row_sum ? row_sum : all)) f = 0;
  }
  if (f < floor_weight(r, scale)) f = 0;
  u64 before = 0, sum = 0;   // in index order
#pragma unroll 1
  for (u64 left = __builtin_amdgcn_ballot_w64(f != 0); left; left &= left - 1) {
    const int i = __builtin_ctzll(left);
    const u64 w = lane_u64(f, i);
    sum += w;
    before += (uint32_t)lane_u64(c, i) > (uint32_t)c ? w : 0;   // indices are complemented
  }
  const u64 target = draw_target(r.u, sum);
  if (before <= target && target < before + f)   // one lane
    emit(a, row, index_in(c), value_in(c), r, (double)sum / scale);
}

// Rows of up to 64 kPer logits, any parameters: one wave per row, no LDS, lane
// l holding the logits [l kPer, (l + 1) kPer).  Every cut is found bit by bit
// of its key, from counts and sums over the wave, until one key is left.  1024
// rows of 1000 bf16 logits: 8 us without filters, 14 with top-p, 18 with top-k
// and top-p, bound by the searches' instructions.
template <typename T, int kPer>
__global__ __launch_bounds__(256) void sample_small_kernel(SampleArgs a) {
  constexpr int low = sizeof(T) == 2 ? 16 : 0, E = RowVec<T>::E;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= a.N) return;
  RowParams r = row_params(a, row);
  const T* z = static_cast<const T*>(a.z) + row * a.ld;
  float x[kPer];
  if (kPer == 1) {
    x[0] = lane < a.V ? clean(to_f32(z[lane])) : kNegInf;
  } else {
#pragma unroll
    for (int j = 0; j < kPer; j += E) {
      const typename RowVec<T>::type v = load_row(z, lane * kPer + j, a.V, kNegInf);
#pragma unroll
      for (int e = 0; e < E && j + e < kPer; ++e) x[j + e] = clean(to_f32(v[e]));
    }
  }
  float m = x[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) m = __builtin_fmaxf(m, x[j]);
  m = wave_max(m);
  if (!r.ok || m == kNegInf) {
    if (lane == 0) emit_none(a, row);
    return;
  }
  r.set_max(m);
  if (r.t == 0.0) {   // the first maximum
    int at = kPer;
#pragma unroll
    for (int j = kPer - 1; j >= 0; --j) at = x[j] == m ? j : at;
    const int l = __builtin_ctzll(__builtin_amdgcn_ballot_w64(at < kPer));
    if (lane == l) emit(a, row, lane * kPer + at, m, r, 1.0);
    return;
  }
  uint32_t key[kPer];   // 0: not kept
#pragma unroll
  for (int j = 0; j < kPer; ++j) key[j] = x[j] > kNegInf ? key_of(x[j]) : 0;
  auto count = [&](uint32_t from) {
    uint32_t n = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) n += key[j] >= from ? 1u : 0u;
    return wave_sum_u32(n);
  };
  // the largest kept key K for which reaches(K, count from K) holds (it holds
  // for all keys below, and for the least); where the test is the count, the
  // search ends when one key is left (counting beside the sums of weights
  // costs as much as the passes it saves: 19 against 18 us at V = 1000, fp32)
  auto search = [&](auto reaches, bool counted) {
    uint32_t K = 0, top = 0, at_least = 2, above = 0;   // K <= result < top (0: no bound)
    if (counted) at_least = count(1);
#pragma unroll 1
    for (int b = 31; b >= low && at_least - above > 1; --b) {
      const uint32_t c = K | 1u << b, n = counted ? count(c) : above + 2;
      if (reaches(c, n)) {
        K = c;
        at_least = n;
      } else {
        top = c;
        above = counted ? n : above;
      }
    }
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool in = key[j] >= K && (top == 0 || key[j] < top);
      best = in && key[j] > best ? key[j] : best;
    }
    return wave_max_u32(best);
  };
  // Of the kept logits with key K, only the first `n` in index order stay;
  // smaller keys go.
  auto cut_at = [&](uint32_t K, u64 n) {
    uint32_t ties = 0, before;
#pragma unroll
    for (int j = 0; j < kPer; ++j) ties += key[j] == K ? 1u : 0u;
    before = wave_scan_u32(ties, before) - ties;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool tie = key[j] == K;
      key[j] = key[j] < K || (tie && before >= n) ? 0 : key[j];
      before += tie ? 1u : 0u;
    }
  };
  if (r.k > 0 && r.k < a.V && count(1) > (u64)r.k) {
    const uint32_t k = (uint32_t)r.k;
    const uint32_t K = search([=](uint32_t, uint32_t n) { return n >= k; }, true);
    cut_at(K, k - count(K + 1));
  }
  const double scale = scale_of(a);
  u64 w[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) w[j] = key[j] ? fixed(weight_any(x[j], r), scale) : 0;
  if (r.p < 1.0) {
    auto mass = [&](uint32_t from) {
      u64 s = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) s += key[j] >= from ? w[j] : 0;
      return wave_sum_u64(s);
    };
    const u64 need = share(r.p, mass(1));
    const uint32_t K = search([&](uint32_t c, uint32_t) { return mass(c) >= need; }, false);
    const u64 rest = need - mass(K + 1), each = fixed(weight_any(value_of(K), r), scale);
    cut_at(K, (rest + each - 1) / each);
  }
  const u64 least = floor_weight(r, scale);
  u64 own = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    w[j] = key[j] && w[j] >= least ? w[j] : 0;
    own += w[j];
  }
  u64 sum;
  u64 run = wave_scan_u64(own, sum) - own;
  const u64 target = draw_target(r.u, sum);
  if (run <= target && target < run + own) {   // one lane
    int at = 0;
    float xt = x[0];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (run <= target) {
        at = j;
        xt = x[j];
      }
      run += w[j];
    }
    emit(a, row, lane * kPer + at, xt, r, (double)sum / scale);
  }
}

// ---------------------------------------------------------------------------
// Maximum over aligned groups of 8 or 16 lanes.
template <int kLanes> __device__ __forceinline__ float lanes_max(float x) {
  x = __builtin_fmaxf(x, dpp_f32<0xB1>(x));
  x = __builtin_fmaxf(x, dpp_f32<0x4E>(x));
  x = __builtin_fmaxf(x, dpp_f32<0x141>(x));
  if (kLanes == 16) x = __builtin_fmaxf(x, dpp_f32<0x140>(x));
  return x;
}

// One piece of one row per work-group: the only pass over all logits.
template <typename T>
__global__ __launch_bounds__(kScanThreads) void sample_scan_kernel(SampleArgs a) {
  constexpr int E = RowVec<T>::E, kVec = kPiece / (kScanThreads * E), kLanes = kGroup / E;
  constexpr int kWaves = kScanThreads / 64;
  __shared__ float wmax[kWaves];
  __shared__ double wsum[kWaves];
  constexpr int kRest = 16;
  __shared__ u64 hist[kWaves][kSlots + kRest - 1];
  const int64_t row_i = blockIdx.x / a.pieces;
  const int piece = blockIdx.x % a.pieces;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const T* z = static_cast<const T*>(a.z) + row_i * a.ld;
  const int64_t base = (int64_t)piece * kPiece;
  typename RowVec<T>::type v[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) v[j] = load_row(z, base + (j * kScanThreads + t) * E, a.V, kNegInf);
  RowParams r = row_params(a, row_i);
  const int64_t out = row_i * a.pieces + piece;
  float m = kNegInf;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    float g = to_f32(v[j][0]);   // the maximum passes over NaN
#pragma unroll
    for (int e = 1; e < E; ++e) g = __builtin_fmaxf(g, to_f32(v[j][e]));
    g = clean(lanes_max<kLanes>(g));
    if (t % kLanes == 0) a.gmax[out * kPieceGroups + (j * kScanThreads + t) / kLanes] = key_of(g);
    m = __builtin_fmaxf(m, g);
  }
  m = wave_max(m);
  if (lane == 0) wmax[w] = m;
  const Mode mode = mode_of(r, a.V);
  if (mode == kTopP)
    for (int i = lane; i < kSlots + kRest - 1; i += 64) hist[w][i] = 0;
  __syncthreads();
  m = wmax[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) m = __builtin_fmaxf(m, wmax[i]);
  if (t == 0) a.pmax[out] = key_of(m);
  if (!r.ok || mode == kGreedy || mode == kTopK || (mode == kMinP && r.p >= 1.0)) return;
  if (!ordinary(m, r)) {   // nothing beside the rest of an ordinary row
    if (t == 0) a.psum[out] = 0.0;
    if (mode == kTopP && t < kSlots) a.hist[out * kSlots + t] = 0;
    return;
  }
  r.set_max(m);
  if (mode != kTopP) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) sum += weight(to_f32(v[j][e]), r);
    sum = wave_sum_f64(sum);
    if (lane == 0) wsum[w] = sum;
    __syncthreads();
    if (t == 0) a.psum[out] = ((wsum[0] + wsum[1]) + wsum[2]) + wsum[3];
    return;
  }
  const double scale = scale_of(a);
  const float alpha = bin_scale(r);
  const float top = bin_of(m, alpha);
  // what lies below the bins is most of a peaked row: 16 places share it
  const float spread = (float)(kSlots - 1 + lane % kRest);
#pragma unroll
  for (int j = 0; j < kVec; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = to_f32(v[j][e]);
      const u64 f = fixed(weight(x, r), scale);
      const int d = (int)__builtin_fminf(top - bin_of(x, alpha), spread);
      if (f) atomicAdd(&hist[w][d], f);
    }
  __syncthreads();
  if (t < kSlots) {
    u64 h = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      h += hist[i][t];
      if (t == kSlots - 1)
        for (int j = 1; j < kRest; ++j) h += hist[i][t + j];
    }
    a.hist[out * kSlots + t] = h;
  }
}

// ---------------------------------------------------------------------------
// Kept by a filter: keys above `key`, and `key` itself up to index `idx`.
struct Cut {
  uint32_t key;
  int64_t idx;
  __device__ __forceinline__ bool keeps(int64_t i, uint32_t k) const { return k > key || (k == key && i <= idx); }
};

// The values from `from` up to (not including) `to`, +inf for no limit; NaN
// is none of them.  accepted() turns vectors into a mask of their elements;
// bit() gives the element (vector and position) of a mask's bit.
template <typename T> struct Interval;
template <> struct Interval<float> {
  float from, to;
  bool open;
  __device__ __forceinline__ Interval(float f, float t) : from(f), to(t), open(t == __builtin_inff()) {}
  template <int N> __device__ __forceinline__ uint32_t accepted(const typename RowVec<float>::type (&v)[N]) const {
    uint32_t mask = 0;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = v[j][e];
        mask |= (x >= from && (open || x < to) ? 1u : 0u) << (j * 4 + e);
      }
    return mask;
  }
  static __device__ __forceinline__ int bit(int b, int) { return b; }
  static __device__ __forceinline__ uint32_t bits_of_vector(int j) { return 0xFu << (4 * j); }
};
// bf16 pairs as 16-bit keys: with d = key - least, d < width where the
// saturating difference width - d is not 0; two elements per instruction.
template <> struct Interval<bf16> {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
  u16x2 least, width;
  // the first 16-bit key whose value is at least x (zeros of both signs are
  // one value: the lower key of the two)
  static __device__ __forceinline__ uint32_t ceil_key(float x) {
    const uint32_t k = key_of(clean(x));
    const uint32_t k16 = k >> 31 ? (uint32_t)(((u64)k + 0xFFFFu) >> 16) : k >> 16;
    return k16 == 0x8000u ? 0x7FFFu : k16;
  }
  __device__ __forceinline__ Interval(float from, float to) {
    const uint32_t a = ceil_key(from), b = to == __builtin_inff() ? 0xFF81u : ceil_key(to);
    least = (uint16_t)a;
    width = (uint16_t)(b > a ? b - a : 0);
  }
  template <int N> __device__ __forceinline__ uint32_t accepted(const typename RowVec<bf16>::type (&v)[N]) const {
    uint32_t mask = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const u32x4 w = __builtin_bit_cast(u32x4, v[j]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i16x2 s = __builtin_bit_cast(i16x2, (uint32_t)w[q]);
        const u16x2 sign = __builtin_bit_cast(u16x2, (i16x2)(s >> 15));
        const u16x2 key = __builtin_bit_cast(u16x2, s) ^ (sign | (uint16_t)0x8000);
        const u16x2 d = key - least;
        uint32_t in;   // (spelled out: the compiler would make two compares and selects of it)
        asm("v_pk_sub_u16 %0, %1, %2 clamp\n\tv_pk_min_u16 %0, %0, 1 op_sel_hi:[1,0]" : "=v"(in) : "v"(width), "v"(d));
        mask = mask << 1 | in;
      }
    }
    return mask;
  }
  // bit 15 - p (first of a pair) or 31 - p (second) of a full mask of four
  // vectors is pair p
  static __device__ __forceinline__ int bit(int b, int n) { return 2 * (4 * n - 1 - (b & 15)) + (b >> 4); }
  static __device__ __forceinline__ uint32_t bits_of_vector(int j) { return 0x000F000Fu << (12 - 4 * j); }
};

// A row's work-group of TH threads: its shared memory, and what it does.  1024
// threads have the shortest way through one row; 512, with half the list,
// leave room for two rows on a compute unit.
template <int TH>
struct Picker {
static constexpr int kRowThreads = TH, kRowWaves = TH / 64;
static constexpr int kBinBits = TH == 1024 ? 11 : 10, kBins = 1 << kBinBits;   // bits of a key per search pass
static constexpr int kList = 12 * TH;                             // candidates (8 bytes each)
static constexpr int kMaxPieces = TH == 1024 ? (1 << 24) / kPiece : 256;
static constexpr int kGroupBatch = 4 * TH;                        // groups looked through at a time
static_assert(kBins == 2 * TH, "find_bin gives every thread two bins");

struct RowShared {
  u64 hist[kBins];
  GroupScratch<kRowThreads> scratch;
  u64 above;
  uint32_t digit;
  uint32_t kmax[kRowWaves];
  int64_t idx;
};

struct PickShared {
  RowShared row;
  u64 list[kList];                    // composites
  u64 cmass[kMaxPieces];              // kept weight per piece
  double factor[kMaxPieces];          // weight of each piece's maximum
  u64 slot[kSlots];
  u64 sum;
  uint16_t glist[kGroupBatch];        // accepted groups of a batch
  int groups;
  int count;
  int found;
};

static __device__ __forceinline__ u64 group_sum(u64 x, RowShared& sh) {
  u64 all;
  group_scan<kRowThreads>(x, all, sh.scratch);
  return all;
}

// The bin, from the highest down, at which the running sum reaches `need`
// (1 <= need <= the sum); `above` gets the sum of the bins over it, plus what
// it held.  `need_of` maps the whole sum to `need`.
template <typename G>
static __device__ __forceinline__ uint32_t find_bin(G need_of, u64& above, RowShared& sh) {
  const int top = kBins - 1 - 2 * threadIdx.x;
  const u64 a = sh.hist[top], b = sh.hist[top - 1];
  u64 all;
  const u64 exc = group_scan<kRowThreads>(a + b, all, sh.scratch) + above, inc = exc + a + b;
  const u64 need = need_of(all);
  if (exc < need && need <= inc) {   // one thread
    const bool first = need <= exc + a;
    sh.digit = (uint32_t)(first ? top : top - 1);
    sh.above = first ? exc : exc + a;
  }
  __syncthreads();
  above = sh.above;
  return sh.digit;
}

static __device__ __forceinline__ void clear_bins(RowShared& sh) {
  __syncthreads();
  sh.hist[threadIdx.x] = 0;
  sh.hist[threadIdx.x + kRowThreads] = 0;
  __syncthreads();
}

// A row of V logits: every wave of the work-group owns a consecutive part of
// it, so sums over waves are sums in index order.
template <typename T>
struct Row {
  static constexpr int E = RowVec<T>::E;
  const T* z;
  int64_t V, begin, end;

  __device__ __forceinline__ Row(const T* p, int64_t v) : z(p), V(v) {
    const int64_t per = (v + kRowWaves * 64 * E - 1) / (kRowWaves * 64 * E) * (64 * E);
    begin = (int64_t)(threadIdx.x >> 6) * per;
    end = begin + per < v ? begin + per : v;
  }

  // f(index, value) over this thread's elements of its wave's part, four
  // loads under way.
  template <typename F> __device__ __forceinline__ void each(F f) const {
    constexpr int kUnroll = 4;
    for (int64_t c = begin + (threadIdx.x & 63) * E; c < end; c += 64 * E * kUnroll) {
      typename RowVec<T>::type v[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
        if (c + j * 64 * E < end) v[j] = load_row(z, c + j * 64 * E, V);
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
        if (c + j * 64 * E < end) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (c + j * 64 * E + e < V) f(c + j * 64 * E + e, clean(to_f32(v[j][e])));
        }
    }
  }

  // The first index at which the running sum of f (u64, in index order)
  // exceeds the target that `target_of` makes of the whole sum; `sum` gets
  // that.  -1 if there is none.
  template <typename F, typename G>
  __device__ __forceinline__ int64_t locate(F f, G target_of, u64& sum, RowShared& sh) const {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    u64 s = 0;
    each([&](int64_t i, float x) { s += f(i, x); });
    s = wave_sum_u64(s);
    __syncthreads();
    if (lane == 0) sh.scratch.wsum[w] = s;
    if (threadIdx.x == 0) sh.idx = -1;
    __syncthreads();
    u64 before = 0;
    sum = 0;
    for (int i = 0; i < kRowWaves; ++i) {
      if (i < w) before += sh.scratch.wsum[i];
      sum += sh.scratch.wsum[i];
    }
    const u64 target = target_of(sum);
    if (before <= target && target < before + s) {   // one wave
      for (int64_t b = begin; b < end; b += 64 * E) {
        const int64_t c = b + lane * E;
        u64 own[E], part = 0;
        const typename RowVec<T>::type v = load_row(z, c, V);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          own[e] = c + e < V ? f(c + e, clean(to_f32(v[e]))) : 0;
          part += own[e];
        }
        u64 all;
        const u64 inc = wave_scan_u64(part, all);
        if (target < before + all) {
          u64 run = before + inc - part;
          if (run <= target && target < run + part) {   // one lane
            int64_t at = c;
#pragma unroll
            for (int e = 0; e < E; ++e) {
              run += own[e];
              if (run <= target) at = c + e + 1;
            }
            sh.idx = at;
          }
          break;
        }
        before += all;
      }
    }
    __syncthreads();
    return sh.idx;
  }

  // The key K at which the sum of f over keys above K is below `need` and
  // the sum with K reaches it; `above` receives the former.  `need_of` maps
  // the sum over everything to `need` (1 <= need <= that sum).  One pass of
  // kBinBits key bits after another, the passes after the first over the keys that
  // share K's leading bits.
  template <typename F, typename G>
  __device__ __forceinline__ uint32_t search(F f, G need_of, u64& above, RowShared& sh) const {
    constexpr int low = sizeof(T) == 2 ? 16 : 0;   // a bf16 key's last 16 bits follow from its first
    uint32_t prefix = 0;
    u64 need = 0;
    above = 0;
    int hi = 32;
    while (hi > low) {
      const int bits = hi - low < kBinBits ? hi - low : kBinBits, lo = hi - bits;
      clear_bins(sh);
      each([&](int64_t i, float x) {
        const uint32_t k = key_of(x);
        if (hi == 32 || (k >> hi) == prefix) {
          const u64 w = f(i, x);
          if (w) atomicAdd(&sh.hist[(k >> lo) & ((1u << bits) - 1)], w);
        }
      });
      __syncthreads();
      const uint32_t d = find_bin([&](u64 all) { return hi == 32 ? need = need_of(all) : need; }, above, sh);
      prefix = (hi == 32 ? 0u : prefix << bits) | d;
      hi = lo;
    }
    if (low == 0) return prefix;
    return prefix << 16 | ((prefix & 0x8000u) ? 0u : 0xFFFFu);
  }
};

// The candidates of a row in LDS.
template <typename T>
struct Candidates {
  static constexpr int low = sizeof(T) == 2 ? 16 : 0;
  PickShared& sh;
  int n;
  uint32_t kmin;   // of the listed keys, without their last `low` bits
  int ib, bits;    // bits of an index, and of a packed composite

  template <typename F> __device__ __forceinline__ void each(F f) const {
    for (int i = threadIdx.x; i < n; i += kRowThreads) f(sh.list[i]);
  }

  // Packs composites into as few bits as the listed keys and the row's
  // indices need.
  __device__ __forceinline__ void measure(int64_t V) {
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    each([&](u64 c) {
      const uint32_t k = key_in(c) >> low;
      lo = k < lo ? k : lo;
      hi = k > hi ? k : hi;
    });
    lo = ~wave_max_u32(~lo);
    hi = wave_max_u32(hi);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh.row.scratch.wsum[threadIdx.x >> 6] = (u64)hi << 32 | lo;
    __syncthreads();
    for (int i = 0; i < kRowWaves; ++i) {
      const u64 v = sh.row.scratch.wsum[i];
      lo = (uint32_t)v < lo ? (uint32_t)v : lo;
      hi = (uint32_t)(v >> 32) > hi ? (uint32_t)(v >> 32) : hi;
    }
    kmin = lo;
    ib = bits_of((u64)V);
    bits = bits_of(hi - lo) + ib;
  }
  __device__ __forceinline__ u64 mask() const { return ((u64)1 << ib) - 1; }
  __device__ __forceinline__ u64 pack(u64 c) const {
    return (u64)((key_in(c) >> low) - kmin) << ib | (mask() - (u64)index_in(c));
  }
  __device__ __forceinline__ u64 unpack(u64 p) const {
    uint32_t k = (uint32_t)(p >> ib) + kmin;
    if (low) k = k << 16 | ((k & 0x8000u) ? 0u : 0xFFFFu);
    return composite(k, (int64_t)(mask() - (p & mask())));
  }

  // The value X of `part` (`width` bits) at which the sum of f over
  // candidates with a larger part is below `need` and the sum with X reaches
  // it; kBinBits bits per pass.
  template <typename P, typename F> __device__ __forceinline__ u64 search(P part, int width, F f, u64 need) const {
    RowShared& r = sh.row;
    u64 prefix = 0, above = 0;
    for (int hi = width; hi > 0;) {
      const int b = hi < kBinBits ? hi : kBinBits, lo = hi - b;
      clear_bins(r);
      each([&](u64 c) {
        const u64 x = part(c);
        if (x >> hi == prefix) {
          const u64 w = f(c);
          if (w) atomicAdd(&r.hist[(x >> lo) & ((1u << b) - 1)], w);
        }
      });
      __syncthreads();
      prefix = prefix << b | find_bin([=](u64) { return need; }, above, r);
      hi = lo;
    }
    return prefix;
  }

  // Collects the logits from `from` up to (not including) `to` (+inf: no
  // limit) out of the groups whose maximum reaches `from`; false if they
  // overflow the list.
  __device__ __forceinline__ bool collect(const T* z, int64_t V, const uint32_t* gmax, float from, float to) {
    const uint32_t least = key_of(clean(from));
    const Interval<T> in(from, to);
    constexpr int E = RowVec<T>::E, kLanes = kGroup / E, kPass = kRowThreads / kLanes, kUnroll = 4;
    const int t = threadIdx.x, lane = t & 63;
    const int groups = (int)((V + kGroup - 1) / kGroup);
    __syncthreads();
    if (t == 0) sh.count = 0;
    for (int g0 = 0; g0 < groups; g0 += kGroupBatch) {
      // the accepted groups of a batch, in any order
      __syncthreads();
      if (t == 0) sh.groups = 0;
      __syncthreads();
      bool live[kGroupBatch / kRowThreads];
      u64 hit[kGroupBatch / kRowThreads];
      int total = 0;
#pragma unroll
      for (int j = 0; j < kGroupBatch / kRowThreads; ++j) {
        const int g = g0 + j * kRowThreads + t;
        live[j] = g < groups && gmax[g] >= least;
      }
#pragma unroll
      for (int j = 0; j < kGroupBatch / kRowThreads; ++j) {
        hit[j] = __builtin_amdgcn_ballot_w64(live[j]);
        total += __builtin_popcountll(hit[j]);
      }
      if (total) {
        int at = 0;
        if (lane == 0) at = atomicAdd(&sh.groups, total);
        at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
        for (int j = 0; j < kGroupBatch / kRowThreads; ++j) {
          if (live[j]) sh.glist[at + lane_rank(hit[j])] = (uint16_t)(j * kRowThreads + t);
          at += __builtin_popcountll(hit[j]);
        }
      }
      __syncthreads();
      // kLanes lanes take a group, kUnroll groups in a row; a lane's accepted
      // logits are the bits of a mask, and the list first holds where they are
      const int ng = sh.groups, before = sh.count;
      __syncthreads();
      // (loads without a branch stay under way: lanes past the last group read
      // the first again, and a vector across the row's end is read once more)
      struct Batch {
        typename RowVec<T>::type v[kUnroll];
        uint32_t ok;   // mask bits of the vectors that are groups
        bool edge;
      } cur, nxt;
      auto place = [&](int i) { return (g0 + (int)sh.glist[i < ng ? i : 0]) * kGroup + (t % kLanes) * E; };
      auto load = [&](Batch& to, int i0) {
        to.ok = 0;
        to.edge = false;
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
          const int i = i0 + j * kPass, c = place(i);
          to.ok |= i < ng ? Interval<T>::bits_of_vector(j) : 0u;
          to.edge |= c + E > V;
          to.v[j] = *reinterpret_cast<const typename RowVec<T>::mem*>(z + (c + E <= V ? c : V - E));
        }
      };
      if (ng > 0) load(nxt, t / kLanes);
      for (int i0 = t / kLanes; i0 - t / kLanes < ng; i0 += kPass * kUnroll) {
        cur = nxt;
        if (i0 - t / kLanes + kPass * kUnroll < ng) load(nxt, i0 + kPass * kUnroll);
        if (__builtin_amdgcn_ballot_w64(cur.edge)) {
#pragma unroll 1
          for (int j = 0; j < kUnroll; ++j) {
            const typename RowVec<T>::type x = load_row(z, place(i0 + j * kPass), V, kNegInf);
#pragma unroll
            for (int q = 0; q < kUnroll; ++q)
              if (q == j) cur.v[q] = x;
          }
        }
        uint32_t mask = in.template accepted<kUnroll>(cur.v) & cur.ok;
        uint32_t all;
        const uint32_t mine = (uint32_t)__builtin_popcount(mask);
        int pos = (int)(wave_scan_u32(mine, all) - mine);
        if (!all) continue;
        int at = 0;
        if (lane == 0) at = atomicAdd(&sh.count, (int)all);
        pos += __builtin_amdgcn_readfirstlane(at);
        const uint32_t code = (uint32_t)i0 << 16 | (uint32_t)(t % kLanes) << 8;
        while (__builtin_amdgcn_ballot_w64(mask != 0)) {
          if (mask && pos < kList) sh.list[pos] = code + (uint32_t)__builtin_ctz(mask);
          ++pos;
          mask &= mask - 1;
        }
      }
      __syncthreads();
      n = sh.count;
      if (n > kList) return false;
      // places to composites
#pragma unroll 4
      for (int i = before + t; i < n; i += kRowThreads) {
        const uint32_t code = (uint32_t)sh.list[i];
        const int b = Interval<T>::bit((int)(code & 255u), kUnroll);
        const int g = sh.glist[(int)(code >> 16) + b / E * kPass];
        const int64_t at = (int64_t)(g0 + g) * kGroup + (int)(code >> 8 & 255u) * E + b % E;
        sh.list[i] = composite(key_of(clean(to_f32(z[at]))), at);
      }
    }
    __syncthreads();
    return true;
  }
};

// Within the piece at `base`: the first index at which the running sum of f
// (in index order) exceeds `target`; a target at or past the piece's sum is
// taken as its last counted element.  -1 if the piece counts nothing.
template <typename T, typename F>
static __device__ __forceinline__ int64_t locate_in_piece(const T* z, int64_t V, int64_t base, F f, u64 target,
                                                          RowShared& sh) {
  constexpr int E = RowVec<T>::E, kVec = kPiece / (kRowThreads * E);
  const int64_t c = base + (int64_t)threadIdx.x * E * kVec;
  u64 own[kVec * E], part = 0;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const typename RowVec<T>::type v = load_row(z, c + j * E, V, kNegInf);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      own[j * E + e] = c + j * E + e < V ? f(c + j * E + e, clean(to_f32(v[e]))) : 0;
      part += own[j * E + e];
    }
  }
  u64 all;
  u64 run = group_scan<kRowThreads>(part, all, sh.scratch);
  if (all == 0) return -1;
  if (target >= all) target = all - 1;
  if (run <= target && target < run + part) {   // one thread
    int64_t at = c;
#pragma unroll
    for (int e = 0; e < kVec * E; ++e) {
      run += own[e];
      if (run <= target) at = c + e + 1;
    }
    sh.idx = at;
  }
  __syncthreads();
  return sh.idx;
}

// sh.factor[i] = weight of piece i's maximum (0 where the piece is masked).
static __device__ __forceinline__ void piece_factors(const SampleArgs& a, int64_t row_i, const RowParams& r,
                                                     PickShared& sh) {
  __syncthreads();
  for (int i = threadIdx.x; i < a.pieces; i += kRowThreads) {
    const uint32_t k = a.pmax[row_i * a.pieces + i];
    sh.factor[i] = k > kKeyNegInf ? weight(value_of(k), r) : 0.0;
  }
  __syncthreads();
}

// An integer weight relative to a piece's maximum, relative to the row's.
static __device__ __forceinline__ u64 rescale(u64 h, double factor) {
  return factor == 1.0 ? h : (u64)((double)h * factor + 0.5);
}
static __device__ __forceinline__ u64 piece_weight(double psum, double factor, double scale) {
  return (u64)(psum * factor * scale + 0.5);
}

// The listed candidates (which hold every token at least as likely as the
// least of them): by one wave, or searched where they are more.
template <typename T>
static __device__ __forceinline__ void pick_from_list(const SampleArgs& a, int64_t row_i, Candidates<T>& list,
                                               const RowParams& r, bool top_k, u64 row_sum, PickShared& sh) {
  top_k = top_k && r.k < list.n;
  if (list.n <= 64) {
    if (threadIdx.x < 64)
      pick_in_wave(a, row_i, (int)threadIdx.x < list.n ? sh.list[threadIdx.x] : 0, list.n, r, top_k, row_sum);
    return;
  }
  const double scale = scale_of(a);
  list.measure(a.V);
  auto wt = [&](u64 c) { return weight(value_in(c), r); };
  auto pack = [&](u64 c) { return list.pack(c); };
  u64 cut = 0;   // composites from here on are kept
  if (top_k) cut = list.unpack(list.search(pack, list.bits, [](u64) { return (u64)1; }, (u64)r.k));
  if (r.p < 1.0) {
    auto f = [&](u64 c) { return c >= cut ? fixed(wt(c), scale) : 0; };
    u64 s = 0;
    list.each([&](u64 c) { s += f(c); });
    s = group_sum(s, sh.row);
    const u64 need = share(r.p, row_sum ? row_sum : s);
    if (need <= s) {   // else the share reaches below the list
      const u64 c = list.unpack(list.search(pack, list.bits, f, need));
      cut = c > cut ? c : cut;
    }
  }
  const u64 least = floor_weight(r, scale);
  auto mass = [&](u64 c) {
    const u64 w = c >= cut ? fixed(wt(c), scale) : 0;
    return w >= least ? w : (u64)0;
  };
  u64 s = 0;
  list.each([&](u64 c) { s += mass(c); });
  s = group_sum(s, sh.row);
  // in index order: the larger its complement, the earlier an index
  const u64 at = list.search([&](u64 c) { return list.mask() - (u64)index_in(c); }, list.ib, mass,
                             draw_target(r.u, s) + 1);
  const int64_t tok = (int64_t)(list.mask() - at);
  if (threadIdx.x == 0)
    emit(a, row_i, tok, clean(to_f32(static_cast<const T*>(a.z)[row_i * a.ld + tok])), r, (double)s / scale);
}

// Top-k or min-p: false if the candidates overflow the list.
template <typename T>
static __device__ __forceinline__ bool pick_bounded(const SampleArgs& a, const T* z, int64_t row_i, const RowParams& r,
                                                    uint32_t km, Mode mode, PickShared& sh) {
  const uint32_t* gmax = a.gmax + row_i * a.pieces * kPieceGroups;
  uint32_t bound = kKeyNegInf + 1;   // candidates' keys from here on
  u64 row_sum = 0;
  if (mode == kTopK) {
    // the k-th largest of the group maxima, or of all logits where there are
    // too few groups or a short row's bound would be loose (with k above a
    // quarter of the groups, more than 1.15 k logits reach it), by its key's
    // distance from the row's maximum: in steps of 2^13 (a thousandth of a
    // binade; 2^14 with fewer bins) over two binades, or to the first bits
    const int groups = (int)((a.V + kGroup - 1) / kGroup);
    const bool by_group = r.k <= (a.V <= 4 * kPiece ? groups / 4 : groups);
    uint32_t* bins = reinterpret_cast<uint32_t*>(sh.row.hist);
    for (int step = 24 - kBinBits; step < 32; step += 8) {
      auto count = [&](uint32_t key) {
        const uint32_t d = (km - key) >> step;
        if (d < kBins - 1) atomicAdd(&bins[d], 1u);
      };
      clear_bins(sh.row);
      if (by_group) {
        for (int i = threadIdx.x; i < groups; i += kRowThreads) count(gmax[i]);
      } else {
        Row<T>(z, a.V).each([&](int64_t, float x) { count(key_of(x)); });
      }
      __syncthreads();
      u64 all;
      const uint32_t x = bins[2 * threadIdx.x], y = bins[2 * threadIdx.x + 1];
      const u64 exc = group_scan<kRowThreads>(x + y, all, sh.row.scratch);
      if ((u64)r.k > all) continue;   // further down: coarser steps
      if (exc < (u64)r.k && (u64)r.k <= exc + x + y)   // one thread
        sh.found = 2 * threadIdx.x + ((u64)r.k <= exc + x ? 0 : 1);
      __syncthreads();
      const uint32_t d = (uint32_t)sh.found;
      const uint32_t reach = ((d + 1) << step) - 1;
      if (km - (kKeyNegInf + 1) > reach) bound = km - reach;
      break;
    }
  } else {
    // w >= q: a little below max + t ln q, by what the weights' rounding lets
    // through (2^-37 of a weight, one unit of an integer) and then by fp32's;
    // the exact test follows
    const double unit = 1.0 / scale_of(a), q = r.q > unit ? r.q : unit;
    const double zq = r.zmax + r.t * (log(q) - 0x1p-37 - unit / q);
    const float x = (float)(zq - 1e-6 * (__builtin_fabs(zq) + __builtin_fabs(r.zmax)));
    const uint32_t b = key_of(clean(x));
    bound = b > bound ? b : bound;
    if (r.p < 1.0) {
      piece_factors(a, row_i, r, sh);
      const double scale = scale_of(a);
      for (int i = 0; i < a.pieces; ++i)
        row_sum += piece_weight(a.psum[row_i * a.pieces + i], sh.factor[i], scale);
    }
  }
  Candidates<T> list{sh, 0, 0, 0, 0};
  if (!list.collect(z, a.V, gmax, value_of(bound), __builtin_inff())) return false;
  pick_from_list(a, row_i, list, r, mode == kTopK, row_sum, sh);
  return true;
}

// No filter, or top-p alone: the pieces' weights above the cut, then the
// piece that holds the answer; a short list where the kept set is small.
// False if the cut lies below the bins or its bin overflows the list.
template <typename T>
static __device__ __forceinline__ bool pick_by_pieces(const SampleArgs& a, const T* z, int64_t row_i, const RowParams& r,
                                                      uint32_t km, Mode mode, PickShared& sh) {
  const double scale = scale_of(a);
  const uint32_t* pmax = a.pmax + row_i * a.pieces;
  Cut cut{0u, a.V};
  piece_factors(a, row_i, r, sh);
  if (mode == kTopP) {
    const float alpha = bin_scale(r), top = bin_of(value_of(km), alpha);
    if (!(__builtin_fabsf(top) < kBinLimit)) return false;
    const uint32_t* gmax = a.gmax + row_i * a.pieces * kPieceGroups;
    // f(piece, row's bin, weight) over the pieces' bins; slot j of a piece is
    // the row's bin j + (row's top - piece's top), kSlots - 1 is the rest
    auto each_slot = [&](auto f) {
      const int j = threadIdx.x % kSlots;
#pragma unroll 4
      for (int i = threadIdx.x / kSlots; i < a.pieces; i += kRowThreads / kSlots) {
        const u64 h = a.hist[(row_i * a.pieces + i) * kSlots + j];
        const float d = (float)j + (top - bin_of(value_of(pmax[i]), alpha));
        const int slot = j < kSlots - 1 ? (int)__builtin_fminf(d, (float)(kSlots - 1)) : kSlots - 1;
        f(i, slot, rescale(h, sh.factor[i]));
      }
    };
    for (int i = threadIdx.x; i < kSlots; i += kRowThreads) sh.slot[i] = 0;
    __syncthreads();
    each_slot([&](int, int slot, u64 w) {
      if (w) atomicAdd(&sh.slot[slot], w);
    });
    __syncthreads();
    // the bin at which the sum from above reaches p of the whole
    u64 all;
    const int t = threadIdx.x;
    const u64 own = t < kSlots ? sh.slot[t] : 0;
    const u64 exc = group_scan<kRowThreads>(own, all, sh.row.scratch);
    const u64 need = share(r.p, all);
    if (exc < need && need <= exc + own) {   // one thread
      sh.found = t;
      sh.sum = exc;
    }
    __syncthreads();
    const int border = sh.found;
    const u64 above = sh.sum;
    if (border == kSlots - 1) return false;
    const float bin = top - (float)border;
    const float from = bin_edge(bin, alpha), to = bin_edge(bin + 1.0f, alpha);
    Candidates<T> list{sh, 0, 0, 0, 0};
    // every logit above the border bin weighs at least what its upper edge
    // does: few of them make a short list together with the bin
    if ((double)above <= weight(to, r) * scale * (kList / 4) && list.collect(z, a.V, gmax, from, __builtin_inff())) {
      pick_from_list(a, row_i, list, r, false, all, sh);
      return true;
    }
    if (!list.collect(z, a.V, gmax, from, to)) return false;
    auto wt = [&](u64 c) { return fixed(weight(value_in(c), r), scale); };
    u64 s = 0;
    list.each([&](u64 c) { s += wt(c); });
    s = group_sum(s, sh.row);
    if (s == 0) return false;
    const u64 rest = need - above;
    list.measure(a.V);
    const u64 c =
        list.unpack(list.search([&](u64 x) { return list.pack(x); }, list.bits, wt, rest < s ? rest : s));
    cut = Cut{key_in(c), index_in(c)};
    // the kept weight by pieces
    for (int i = threadIdx.x; i < a.pieces; i += kRowThreads) sh.cmass[i] = 0;
    __syncthreads();
    list.each([&](u64 x) {
      if (x >= c) atomicAdd(&sh.cmass[index_in(x) / kPiece], wt(x));
    });
    each_slot([&](int i, int slot, u64 w) {   // a wave's slots are of one piece
      const u64 sum = wave_sum_u64(slot < border ? w : 0);
      if (sum && (threadIdx.x & 63) == 0) atomicAdd(&sh.cmass[i], sum);
    });
  } else {
    for (int i = threadIdx.x; i < a.pieces; i += kRowThreads)
      sh.cmass[i] = piece_weight(a.psum[row_i * a.pieces + i], sh.factor[i], scale);
  }
  __syncthreads();
  const int i2 = 2 * threadIdx.x;
  const u64 m0 = i2 < a.pieces ? sh.cmass[i2] : 0, m1 = i2 + 1 < a.pieces ? sh.cmass[i2 + 1] : 0;
  u64 sum;
  const u64 exc = group_scan<kRowThreads>(m0 + m1, sum, sh.row.scratch);
  u64 target = draw_target(r.u, sum);
  if (exc <= target && target < exc + m0 + m1) {   // one thread
    const bool first = target < exc + m0;
    sh.found = first ? i2 : i2 + 1;
    sh.sum = target - (first ? exc : exc + m0);
  }
  __syncthreads();
  target = sh.sum;
  int64_t tok = -1;
  auto mass = [&](int64_t i, float x) { return cut.keeps(i, key_of(x)) ? fixed(weight(x, r), scale) : (u64)0; };
  // (a piece whose logits all round to nothing passes on to the next)
  for (int i = sh.found; i < a.pieces && tok < 0; ++i, target = 0)
    tok = locate_in_piece(z, a.V, (int64_t)i * kPiece, mass, target, sh.row);
  if (tok < 0) return false;
  if (threadIdx.x == 0) emit(a, row_i, tok, clean(to_f32(z[tok])), r, (double)sum / scale);
  return true;
}

// Any parameters, by passes over the whole row.  A function of its own, with
// its arguments by value: inlined or by reference it would put what the
// common paths hold in registers on the stack.
template <typename T>
static __device__ __attribute__((noinline)) void pick_whole_row(SampleArgs a, const T* z, int64_t row_i, RowParams r,
                                                         RowShared& sh) {
  const Row<T> row(z, a.V);
  const double scale = scale_of(a);
  Cut cut{0u, a.V};
  // the ties at the border go to the lowest indices
  auto tie_index = [&](uint32_t key, u64 count) {
    u64 n;
    const int64_t i = row.locate([&](int64_t, float x) { return (u64)(key_of(x) == key); },
                                 [=](u64) { return count - 1; }, n, sh);
    return i < 0 ? a.V : i;
  };
  if (r.k > 0 && r.k < a.V) {
    const u64 k = (u64)r.k;
    u64 above;
    cut.key = row.search([](int64_t, float) { return (u64)1; }, [=](u64) { return k; }, above, sh);
    cut.idx = tie_index(cut.key, k - above);
  }
  if (r.p < 1.0) {
    u64 above, need = 0;
    const Cut in = cut;
    const uint32_t key =
        row.search([&](int64_t i, float x) { return in.keeps(i, key_of(x)) ? fixed(weight_any(x, r), scale) : 0; },
                   [&](u64 all) { return need = share(r.p, all); }, above, sh);
    const u64 each = fixed(weight_any(value_of(key), r), scale);
    const int64_t i = tie_index(key, (need - above + each - 1) / each);
    cut.idx = key == cut.key && cut.idx < i ? cut.idx : i;
    cut.key = key;
  }
  const u64 least = floor_weight(r, scale);
  u64 sum;
  const int64_t tok = row.locate(
      [&](int64_t i, float x) {
        const u64 w = cut.keeps(i, key_of(x)) ? fixed(weight_any(x, r), scale) : 0;
        return w >= least ? w : (u64)0;
      },
      [&](u64 s) { return draw_target(r.u, s); }, sum, sh);
  if (threadIdx.x == 0) emit(a, row_i, tok, clean(to_f32(z[tok])), r, (double)sum / scale);
}

template <typename T>
static __device__ __forceinline__ void run(const SampleArgs& a, PickShared& sh) {
  const int64_t row_i = blockIdx.x;
  RowParams r = row_params(a, row_i);
  const T* z = static_cast<const T*>(a.z) + row_i * a.ld;
  const uint32_t* pmax = a.pmax + row_i * a.pieces;
  uint32_t km = 0;
  for (int i = threadIdx.x; i < a.pieces; i += kRowThreads) km = pmax[i] > km ? pmax[i] : km;
  km = wave_max_u32(km);
  if ((threadIdx.x & 63) == 0) sh.row.kmax[threadIdx.x >> 6] = km;
  if (threadIdx.x == 0) sh.found = a.pieces;
  __syncthreads();
  for (int i = 0; i < kRowWaves; ++i) km = sh.row.kmax[i] > km ? sh.row.kmax[i] : km;
  if (!r.ok || km <= kKeyNegInf) {
    if (threadIdx.x == 0) emit_none(a, row_i);
    return;
  }
  r.set_max(value_of(km));
  const Mode mode = mode_of(r, a.V);
  bool done = false;
  if (mode == kGreedy) {
    // the first piece that holds the maximum, then the first index in it
    for (int i = threadIdx.x; i < a.pieces; i += kRowThreads)
      if (pmax[i] == km) atomicMin(&sh.found, i);
    __syncthreads();
    const int64_t tok = locate_in_piece(z, a.V, (int64_t)sh.found * kPiece,
                                        [&](int64_t, float x) { return (u64)(key_of(x) == km); }, 0, sh.row);
    if (threadIdx.x == 0) emit(a, row_i, tok, value_of(km), r, 1.0);
    done = true;
  } else if (!ordinary(value_of(km), r)) {
  } else if (mode == kTopK || mode == kMinP) {
    done = pick_bounded(a, z, row_i, r, km, mode, sh);
  } else {
    done = pick_by_pieces(a, z, row_i, r, km, mode, sh);
  }
  if (!done) pick_whole_row(a, z, row_i, r, sh.row);
}
};

// One row per work-group; at most 128 registers, so that 512 threads fit twice.
template <typename T, int TH>
__global__ __launch_bounds__(TH) __attribute__((amdgpu_waves_per_eu(4))) void sample_pick_kernel(SampleArgs a) {
  __shared__ typename Picker<TH>::PickShared sh;
  Picker<TH>::template run<T>(a, sh);
}

// Two rows at a time on a compute unit where there are more rows than compute
// units and a flat row's border bin still fits the shorter list.  1024 rows of
// 4000 bf16 logits, 512 against 1024 threads: k = 50 and p = 0.95 on peaked
// rows 31 against 53 us, p = 0.9 on flat ones 45 against 76 us, no filter 22
// against 30 us.
template <typename T>
void launch_pick(const SampleArgs& a, hipStream_t st) {
  if (a.N > 256 && a.V <= 65536)
    sample_pick_kernel<T, 512><<<(unsigned)a.N, 512, 0, st>>>(a);
  else
    sample_pick_kernel<T, 1024><<<(unsigned)a.N, 1024, 0, st>>>(a);
}

template <typename T>
void launch_small(const SampleArgs& a, hipStream_t st) {
  const unsigned g = (unsigned)((a.N + 3) / 4);
  if (a.V <= 64) sample_small_kernel<T, 1><<<g, 256, 0, st>>>(a);
  else if (a.V <= 512) sample_small_kernel<T, 8><<<g, 256, 0, st>>>(a);
  else if (a.V <= 1024) sample_small_kernel<T, 16><<<g, 256, 0, st>>>(a);
  else sample_small_kernel<T, 32><<<g, 256, 0, st>>>(a);
}

// Workspace: what the scan leaves, for rows longer than kSmall.
struct SampleLayout {
  int64_t pieces;
  size_t psum, hist, gmax, total;   // byte offsets (pmax at 0); total 0: not supported
};

SampleLayout sample_layout(int64_t N, int64_t V) {
  SampleLayout l{(V + kPiece - 1) / kPiece, 0, 0, 0, 0};
  // launches of fewer than 2^32 threads
  if (N > (int64_t(1) << 21) || V > (int64_t(1) << 24) || N * l.pieces > (int64_t(1) << 23)) return l;
  if (V <= kSmall) {
    l.total = 256;
    return l;
  }
  auto pad = [](size_t b) { return (b + 255) & ~size_t(255); };
  const size_t n = (size_t)(N * l.pieces);
  l.psum = pad(n * 4);
  l.hist = l.psum + pad(n * 8);
  l.gmax = l.hist + pad(n * kSlots * 8);
  l.total = l.gmax + pad(n * kPieceGroups * 4);
  if (l.total < 256) l.total = 256;   // no rows
  return l;
}

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

}  // namespace flce

extern "C" size_t flce_sample_workspace_size(int64_t N, int64_t V, int dtype) {
  if ((dtype != FLCE_DTYPE_BF16 && dtype != FLCE_DTYPE_F32) || N < 0 || V < 1) return 0;
  return flce::sample_layout(N, V).total;
}

extern "C" int flce_sample(const void* logits, int64_t ld_logits, const float* u, int64_t N, int64_t V,
                           const flce_sample_params_t* params, int64_t* tokens, float* logprobs, hipStream_t stream,
                           int dtype, void* workspace, size_t workspace_bytes) {
  using namespace flce;
  if (dtype != FLCE_DTYPE_BF16 && dtype != FLCE_DTYPE_F32) return FLCE_EINVAL;
  if (N < 0 || V < 1 || !params) return FLCE_EINVAL;
  const uintptr_t es = dtype == FLCE_DTYPE_BF16 ? 2 : 4;
  const flce_sample_params_t& q = *params;
  if (!q.temperature_rows && !(q.temperature >= 0.0f && std::isfinite(q.temperature))) return FLCE_EINVAL;
  if (!q.top_k_rows && q.top_k < 0) return FLCE_EINVAL;
  if (!q.top_p_rows && !(q.top_p > 0.0f && q.top_p <= 1.0f)) return FLCE_EINVAL;
  if (!q.min_p_rows && !(q.min_p >= 0.0f && q.min_p <= 1.0f)) return FLCE_EINVAL;
  if (!on(q.temperature_rows, 4) || !on(q.top_k_rows, 8) || !on(q.top_p_rows, 4) || !on(q.min_p_rows, 4))
    return FLCE_EINVAL;
  if (!on(logprobs, 4) || !on(workspace, 256)) return FLCE_EINVAL;
  if (N > 0 && (!logits || !u || !tokens || !workspace)) return FLCE_EINVAL;
  if (!on(logits, es) || !on(u, 4) || !on(tokens, 8) || ld_logits < 0) return FLCE_EINVAL;
  const SampleLayout l = sample_layout(N, V);
  if (l.total == 0) return FLCE_EUNSUPPORTED;
  if (N == 0) return FLCE_OK;
  if (workspace_bytes < l.total) return FLCE_EWORKSPACE;
  SampleArgs a;
  a.z = logits;
  a.ld = ld_logits;
  a.u = u;
  a.N = N;
  a.V = V;
  a.prm = q;
  int bits = 0;
  while ((int64_t(1) << bits) < V) ++bits;
  a.s = 62 - bits < 51 ? 62 - bits : 51;
  a.tokens = tokens;
  a.logprobs = logprobs;
  char* ws = static_cast<char*>(workspace);
  a.pieces = (int)l.pieces;
  a.pmax = reinterpret_cast<uint32_t*>(ws);
  a.psum = reinterpret_cast<double*>(ws + l.psum);
  a.hist = reinterpret_cast<u64*>(ws + l.hist);
  a.gmax = reinterpret_cast<uint32_t*>(ws + l.gmax);
  if (V <= kSmall) {
    ProfileScope ps(FLCE_KERNEL_SAMPLE_PICK, stream);
    if (dtype == FLCE_DTYPE_BF16)
      launch_small<bf16>(a, stream);
    else
      launch_small<float>(a, stream);
    return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
  }
  {
    ProfileScope ps(FLCE_KERNEL_SAMPLE_SCAN, stream);
    const unsigned g = (unsigned)(N * l.pieces);
    if (dtype == FLCE_DTYPE_BF16)
      sample_scan_kernel<bf16><<<g, kScanThreads, 0, stream>>>(a);
    else
      sample_scan_kernel<float><<<g, kScanThreads, 0, stream>>>(a);
  }
  {
    ProfileScope ps(FLCE_KERNEL_SAMPLE_PICK, stream);
    if (dtype == FLCE_DTYPE_BF16)
      launch_pick<bf16>(a, stream);
    else
      launch_pick<float>(a, stream);
  }
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}
