// Drawing a token from each row of logits (flce_sample): temperature, top-k,
// top-p and min-p filters, then the inverse of the distribution function in
// index order at a given random number.
//
// Weights are integers: W = round(2^s exp((z - max) / t)), with s chosen so
// that a row's sum stays below 2^62.  Sums of integers are exact, so neither
// the order of atomics nor the split of a row changes a decision; the
// rounding, 2^-(s+1) per token next to the largest token's 1, is far below
// what a 24-bit random number or an fp32 probability resolves (s is 44 at a
// vocabulary of 2^18).  The exponential is taken in 64 bits for the same
// reason: an fp32 one moves the borders between tokens of a flat row by more
// than their spacing warrants.
//
// A row passes through the chip once, in pieces of 8192 logits spread over
// the work-groups of sample_scan_kernel, which leaves behind what decides
// where the answer lies:
//   * the maximum of each 64 logits and of the piece;
//   * with top-p alone: the piece's weight by bins of z, 1/8 of min(t, 1) wide,
//     counted down from the piece's maximum (bins are aligned in z, so bins
//     of different pieces add up);
//   * without any filter, or with min-p: the piece's weight.
// sample_pick_kernel (one work-group per row) then looks only where it has
// to:
//   * top-k: the k-th largest of the 64-logit maxima bounds the k-th logit
//     from below, so every candidate lies in a group whose maximum reaches it;
//   * min-p: the candidates reach the maximum + t ln q;
//   * top-p alone: the bin in which the weight from above reaches p of the
//     row's; only that bin's logits decide where the cut falls;
//   * then a search in the list of candidates (LDS), or, where the kept set
//     is most of a flat row, one piece whose weights are summed in order.
// Rows for which that does not work out (a list that overflows, a cut below
// the bins) take the searches over the whole row at the end of the kernel.
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

typedef unsigned long long u64;

constexpr int kRowThreads = 1024;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kBins = 2048;          // 11 bits of a key per search pass
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;
constexpr int kPiece = 8192;         // logits per work-group of the scan
constexpr int kGroup = 64;           // logits per stored maximum
constexpr int kPieceGroups = kPiece / kGroup;
constexpr int kSlots = 128;          // bins of z per piece; the last holds the rest
constexpr int kList = 8192;          // candidates per row (64 KB of LDS)
constexpr int kScanThreads = 256;

struct SampleArgs {
  const void* z;
  int64_t ld;      // elements
  const float* u;
  int64_t N, V;
  flce_sample_params_t prm;
  int s;           // weights are multiples of 2^-s
  int64_t* tokens;
  float* logprobs;
  // left by the scan (rows longer than one piece)
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

// A row's parameters and the weights they define.
struct RowParams {
  double t, p, q, zmax;
  int64_t k;
  float u;
  bool ok;
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
  r.zmax = 0.0;
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

// Bins of z: 1/8 of min(t, 1) wide, ascending with z.
__device__ __forceinline__ float bin_scale(const RowParams& r) {
  return r.t < 1.0 ? (float)(8.0 / r.t < 1e30 ? 8.0 / r.t : 1e30) : 8.0f;
}
__device__ __forceinline__ int bin_of(float x, float alpha) {
  return (int)__builtin_floorf(__builtin_fminf(__builtin_fmaxf(x * alpha, -0x1p30f), 0x1p30f));
}

// exp((z - max) / t); 1 for the maximum itself, also where it is infinite.
__device__ __forceinline__ double weight(float x, const RowParams& r) {
  const double z = (double)x;
  return z == r.zmax ? 1.0 : exp((z - r.zmax) / r.t);
}

// round(w 2^s) for w <= 1, s <= 51: adding 2^52 leaves the integer in the
// mantissa.
__device__ __forceinline__ u64 fixed(double w, double scale) {
  return __builtin_bit_cast(u64, __builtin_fma(w, scale, 0x1p52)) - __builtin_bit_cast(u64, 0x1p52);
}

__device__ __forceinline__ u64 wave_sum_u64(u64 x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ u64 wave_scan_u64(u64 x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const u64 y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  return x;
}

struct RowShared {
  u64 hist[kBins];
  u64 wsum[kRowWaves];
  u64 above, total;
  uint32_t digit;
  uint32_t kmax[kRowWaves];
  int64_t idx;
};

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

  // f(index, value) over this thread's elements of its wave's part.
  template <typename F> __device__ __forceinline__ void each(F f) const {
    for (int64_t c = begin + (threadIdx.x & 63) * E; c < end; c += 64 * E) {
      const typename RowVec<T>::type v = load_row(z, c, V);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (c + e < V) f(c + e, clean(to_f32(v[e])));
    }
  }

  // The first index at which the running sum of f (u64, in index order)
  // exceeds `target`, or -1.  All threads get it.
  template <typename F> __device__ int64_t locate(F f, u64 target, RowShared& sh) const {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    u64 s = 0;
    each([&](int64_t i, float x) { s += f(i, x); });
    s = wave_sum_u64(s);
    __syncthreads();
    if (lane == 0) sh.wsum[w] = s;
    if (threadIdx.x == 0) sh.idx = -1;
    __syncthreads();
    u64 before = 0;
    for (int i = 0; i < w; ++i) before += sh.wsum[i];
    if (before <= target && target < before + s) {   // one wave
      for (int64_t b = begin; b < end; b += 64 * E) {
        const int64_t c = b + lane * E;
        u64 own[E], sum = 0;
        const typename RowVec<T>::type v = load_row(z, c, V);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          own[e] = c + e < V ? f(c + e, clean(to_f32(v[e]))) : 0;
          sum += own[e];
        }
        const u64 inc = wave_scan_u64(sum);
        const u64 all = __shfl(inc, 63);
        if (target < before + all) {
          u64 run = before + inc - sum;
          if (run <= target && target < run + sum) {   // one lane
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
  // 11 key bits after another, the passes after the first over the keys that
  // share K's leading bits.
  template <typename F, typename G> __device__ uint32_t search(F f, G need_of, u64& above, RowShared& sh) const {
    constexpr int low = sizeof(T) == 2 ? 16 : 0;   // a bf16 key's last 16 bits follow from its first
    uint32_t prefix = 0;
    u64 over = 0, need = 0;
    int hi = 32;
    while (hi > low) {
      const int bits = hi - low < 11 ? hi - low : 11, lo = hi - bits;
      for (int i = threadIdx.x; i < kBins; i += kRowThreads) sh.hist[i] = 0;
      __syncthreads();
      each([&](int64_t i, float x) {
        const uint32_t k = key_of(x);
        if (hi == 32 || (k >> hi) == prefix) {
          const u64 w = f(i, x);
          if (w) atomicAdd(&sh.hist[(k >> lo) & ((1u << bits) - 1)], w);
        }
      });
      __syncthreads();
      // running sums from the highest bin down: thread i holds the bins
      // kBins - 1 - 2 i and the one below it
      const int top = kBins - 1 - 2 * threadIdx.x;
      const u64 a = sh.hist[top], b = sh.hist[top - 1];
      u64 inc = wave_scan_u64(a + b);
      if ((threadIdx.x & 63) == 63) sh.wsum[threadIdx.x >> 6] = inc;
      __syncthreads();
      u64 before = 0, all = 0;
      for (int i = 0; i < kRowWaves; ++i) {
        if (i < (int)(threadIdx.x >> 6)) before += sh.wsum[i];
        all += sh.wsum[i];
      }
      if (hi == 32) need = need_of(all);
      inc += before + over;
      const u64 exc = inc - a - b;
      if (exc < need && need <= inc) {   // one thread
        const bool first = need <= exc + a;
        sh.digit = (uint32_t)(first ? top : top - 1);
        sh.above = first ? exc : exc + a;
      }
      __syncthreads();
      prefix = (hi == 32 ? 0u : prefix << bits) | sh.digit;
      over = sh.above;
      __syncthreads();
      hi = lo;
    }
    above = over;
    if (low == 0) return prefix;
    return prefix << 16 | ((prefix & 0x8000u) ? 0u : 0xFFFFu);
  }
};

// Kept by a filter: keys above `key`, and `key` itself up to index `idx`.
struct Cut {
  uint32_t key;
  int64_t idx;
  __device__ __forceinline__ bool keeps(int64_t i, uint32_t k) const { return k > key || (k == key && i <= idx); }
};

__device__ __forceinline__ double wave_sum_f64(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

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
  __shared__ u64 hist[kWaves][kSlots];
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
    float g = clean(to_f32(v[j][0]));
#pragma unroll
    for (int e = 1; e < E; ++e) g = __builtin_fmaxf(g, clean(to_f32(v[j][e])));
    g = lanes_max<kLanes>(g);
    if (t % kLanes == 0) a.gmax[out * kPieceGroups + (j * kScanThreads + t) / kLanes] = key_of(g);
    m = __builtin_fmaxf(m, g);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, o));
  if (lane == 0) wmax[w] = m;
  const Mode mode = mode_of(r, a.V);
  if (mode == kTopP)
    for (int i = t; i < kWaves * kSlots; i += kScanThreads) hist[i / kSlots][i % kSlots] = 0;
  __syncthreads();
  m = wmax[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) m = __builtin_fmaxf(m, wmax[i]);
  if (t == 0) a.pmax[out] = key_of(m);
  if (!r.ok || mode == kGreedy || mode == kTopK || (mode == kMinP && r.p >= 1.0)) return;
  if (m == kNegInf) {
    if (t == 0) a.psum[out] = 0.0;
    if (mode == kTopP && t < kSlots) a.hist[out * kSlots + t] = 0;
    return;
  }
  r.zmax = (double)m;
  if (mode != kTopP) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) sum += weight(clean(to_f32(v[j][e])), r);
    sum = wave_sum_f64(sum);
    if (lane == 0) wsum[w] = sum;
    __syncthreads();
    if (t == 0) a.psum[out] = ((wsum[0] + wsum[1]) + wsum[2]) + wsum[3];
    return;
  }
  const double scale = __builtin_bit_cast(double, (u64)(1023 + a.s) << 52);
  const float alpha = bin_scale(r);
  const int top = bin_of(m, alpha);
#pragma unroll
  for (int j = 0; j < kVec; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = clean(to_f32(v[j][e]));
      const u64 f = fixed(weight(x, r), scale);
      const int d = top - bin_of(x, alpha);
      if (f) atomicAdd(&hist[w][d < kSlots ? d : kSlots - 1], f);
    }
  __syncthreads();
  u64 h = 0;
  if (t < kSlots) {
#pragma unroll
    for (int i = 0; i < kWaves; ++i) h += hist[i][t];
    a.hist[out * kSlots + t] = h;
  }
  const u64 all = wave_sum_u64(h);
  __syncthreads();
  if (lane == 0) hist[0][w] = all;
  __syncthreads();
  if (t == 0) a.psum[out] = (double)(hist[0][0] + hist[0][1]) / scale;
}

struct PickShared {
  RowShared row;
  u64 list[kList];                  // composites, see Candidates
  union {
    u64 cmass[kPiece / 4];          // kept list weight per piece (at most 2^24 / 8192 = 2048)
    double dmass[kPiece / 4];
  };
  double factor[kPiece / 4];        // weight of each piece's maximum
  double slot[kSlots];
  double dsum[kRowWaves];
  u64 usum[kRowWaves];
  int count;
  int found;
};

__device__ __forceinline__ int bits_of(u64 x) { return x ? 64 - __builtin_clzll(x) : 0; }

// Sum over the work-group, all threads get it.
__device__ __forceinline__ u64 group_sum_u64(u64 x, PickShared& sh) {
  x = wave_sum_u64(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.usum[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0;
  for (int i = 0; i < kRowWaves; ++i) x += sh.usum[i];
  return x;
}

// The candidates of a row: composites that order them by descending logit,
// then ascending index (a larger composite comes first).
template <typename T>
struct Candidates {
  static constexpr int low = sizeof(T) == 2 ? 16 : 0;
  PickShared& sh;
  uint32_t kmin;     // lower bound of the keys, without their last `low` bits
  int ib;            // bits of an index
  int bits;          // bits of a composite
  int n;

  __device__ __forceinline__ u64 pack(uint32_t key, int64_t i) const {
    return (u64)((key >> low) - kmin) << ib | (((u64)1 << ib) - 1 - (u64)i);
  }
  __device__ __forceinline__ int64_t index(u64 c) const { return (int64_t)(((u64)1 << ib) - 1 - (c & (((u64)1 << ib) - 1))); }
  __device__ __forceinline__ uint32_t key(u64 c) const {
    const uint32_t k = (uint32_t)(c >> ib) + kmin;
    if (low == 0) return k;
    return k << 16 | ((k & 0x8000u) ? 0u : 0xFFFFu);
  }
  __device__ __forceinline__ float value(u64 c) const { return value_of(key(c)); }

  template <typename F> __device__ __forceinline__ void each(F f) const {
    for (int i = threadIdx.x; i < n; i += kRowThreads) f(sh.list[i]);
  }

  // The value X of `part` (`width` bits) at which the sum of f over
  // candidates with a larger part is below `need` and the sum with X reaches
  // it; 11 bits per pass.
  template <typename P, typename F> __device__ u64 search(P part, int width, F f, u64 need) const {
    RowShared& r = sh.row;
    u64 prefix = 0, over = 0;
    int hi = width;
    while (hi > 0) {
      const int b = hi < 11 ? hi : 11, lo = hi - b;
      __syncthreads();
      r.hist[threadIdx.x] = 0;
      r.hist[threadIdx.x + kRowThreads] = 0;
      __syncthreads();
      each([&](u64 c) {
        const u64 x = part(c);
        if (x >> hi == prefix) {
          const u64 w = f(c);
          if (w) atomicAdd(&r.hist[(x >> lo) & ((1u << b) - 1)], w);
        }
      });
      __syncthreads();
      const int top = kBins - 1 - 2 * threadIdx.x;
      const u64 u = r.hist[top], v = r.hist[top - 1];
      u64 inc = wave_scan_u64(u + v);
      if ((threadIdx.x & 63) == 63) r.wsum[threadIdx.x >> 6] = inc;
      __syncthreads();
      for (int i = 0; i < (int)(threadIdx.x >> 6); ++i) inc += r.wsum[i];
      inc += over;
      const u64 exc = inc - u - v;
      if (exc < need && need <= inc) {   // one thread
        const bool first = need <= exc + u;
        r.digit = (uint32_t)(first ? top : top - 1);
        r.above = first ? exc : exc + u;
      }
      __syncthreads();
      prefix = prefix << b | r.digit;
      over = r.above;
      hi = lo;
    }
    __syncthreads();
    return prefix;
  }

  // Collects the logits that `take(key, value)` accepts out of the groups
  // whose maximum `group(key)` accepts; false if they overflow the list.
  template <typename G, typename F>
  __device__ bool collect(const T* z, int64_t V, const uint32_t* gmax, G group, F take) {
    constexpr int E = RowVec<T>::E, kUnroll = 4;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    __syncthreads();
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    const int64_t stride = (int64_t)kRowThreads * E;
    for (int64_t b = (int64_t)w * 64 * E; b < V; b += stride * kUnroll) {
      bool live[kUnroll];
      typename RowVec<T>::type v[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int64_t c = b + j * stride + lane * E;
        live[j] = c < V && (!gmax || group(gmax[c / kGroup]));
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
        if (live[j]) v[j] = load_row(z, b + j * stride + lane * E, V);
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        if (!__builtin_amdgcn_ballot_w64(live[j])) continue;
        const int64_t c = b + j * stride + lane * E;
        uint32_t k[E];
        u64 hit[E];
        int total = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float x = live[j] && c + e < V ? clean(to_f32(v[j][e])) : kNegInf;
          k[e] = key_of(x);
          hit[e] = __builtin_amdgcn_ballot_w64(live[j] && c + e < V && take(k[e], x));
          total += __builtin_popcountll(hit[e]);
        }
        if (!total) continue;
        int at = 0;
        if (lane == 0) at = atomicAdd(&sh.count, total);
        at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int pos = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(hit[e] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)hit[e], 0));
          if ((hit[e] >> lane & 1) && pos < kList) sh.list[pos] = pack(k[e], c + e);
          at += __builtin_popcountll(hit[e]);
        }
      }
    }
    __syncthreads();
    n = sh.count;
    return n <= kList;
  }
};

// Within the piece at `base`: the first index at which the running sum of f
// (in index order) exceeds `target`; a target at or past the piece's sum is
// taken as its last counted element.  -1 if the piece counts nothing.
template <typename T, typename F>
__device__ int64_t locate_in_piece(const T* z, int64_t V, int64_t base, F f, u64 target, PickShared& sh) {
  constexpr int E = RowVec<T>::E, kVec = kPiece / (kRowThreads * E);
  const int64_t c = base + (int64_t)threadIdx.x * E * kVec;
  u64 own[kVec * E], sum = 0;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const typename RowVec<T>::type v = load_row(z, c + j * E, V, kNegInf);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      own[j * E + e] = c + j * E + e < V ? f(c + j * E + e, clean(to_f32(v[e]))) : 0;
      sum += own[j * E + e];
    }
  }
  const u64 inc = wave_scan_u64(sum);
  const int w = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 63) sh.usum[w] = inc;
  __syncthreads();
  u64 before = 0, all = 0;
  for (int i = 0; i < kRowWaves; ++i) {
    if (i < w) before += sh.usum[i];
    all += sh.usum[i];
  }
  if (all == 0) return -1;
  if (target >= all) target = all - 1;
  u64 run = before + inc - sum;
  if (run <= target && target < run + sum) {   // one thread
    int64_t at = c;
#pragma unroll
    for (int e = 0; e < kVec * E; ++e) {
      run += own[e];
      if (run <= target) at = c + e + 1;
    }
    sh.row.idx = at;
  }
  __syncthreads();
  return sh.row.idx;
}

// sh.factor[i] = weight of piece i's maximum (0 where the piece is masked).
__device__ __forceinline__ void piece_factors(const SampleArgs& a, int64_t row_i, const RowParams& r, PickShared& sh) {
  __syncthreads();
  for (int i = threadIdx.x; i < a.pieces; i += kRowThreads) {
    const uint32_t k = a.pmax[row_i * a.pieces + i];
    sh.factor[i] = k > kKeyNegInf ? weight(value_of(k), r) : 0.0;
  }
  __syncthreads();
}

// Top-k, min-p, or any filter on a row of one piece: the candidates in a
// list.  False if they overflow it.
template <typename T>
__device__ bool pick_from_list(const SampleArgs& a, const T* z, int64_t row_i, const RowParams& r, uint32_t km,
                               double scale, Mode mode, const uint32_t* gmax, PickShared& sh, int64_t& tok,
                               double& total) {
  constexpr int low = sizeof(T) == 2 ? 16 : 0;
  const int ib = bits_of((u64)a.V);
  uint32_t bound = kKeyNegInf + 1;   // candidates' keys from here on
  if (gmax && mode == kTopK) {
    // the k-th largest group maximum, to the first 11 bits of its key
    const int groups = a.pieces * kPieceGroups;
    if (r.k > groups - groups / 8) return false;
    RowShared& s = sh.row;
    __syncthreads();
    s.hist[threadIdx.x] = 0;
    s.hist[threadIdx.x + kRowThreads] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < groups; i += kRowThreads) atomicAdd(&s.hist[gmax[i] >> 21], (u64)1);
    __syncthreads();
    const int top = kBins - 1 - 2 * threadIdx.x;
    const u64 u = s.hist[top], v = s.hist[top - 1];
    u64 inc = wave_scan_u64(u + v);
    if ((threadIdx.x & 63) == 63) s.wsum[threadIdx.x >> 6] = inc;
    __syncthreads();
    for (int i = 0; i < (int)(threadIdx.x >> 6); ++i) inc += s.wsum[i];
    const u64 exc = inc - u - v, k = (u64)r.k;
    if (exc < k && k <= inc) s.digit = (uint32_t)(k <= exc + u ? top : top - 1);
    __syncthreads();
    const uint32_t b = s.digit << 21;
    bound = b > bound ? b : bound;
  } else if (gmax) {
    // w >= q: a little below max + t ln q in fp32, the exact test follows
    const double zq = r.zmax + r.t * log(r.q);
    const float x = (float)(zq - 1e-6 * (__builtin_fabs(zq) + __builtin_fabs(r.zmax)));
    const uint32_t b = key_of(clean(x));
    bound = b > bound ? b : bound;
  }
  Candidates<T> list{sh, bound >> low, ib, 0, 0};
  list.bits = bits_of((km >> low) - list.kmin) + ib;
  if (!list.collect(z, a.V, gmax, [=](uint32_t k) { return k >= bound; },
                    [=](uint32_t k, float) { return k >= bound; }))
    return false;
  auto wt = [&](u64 c) { return weight(list.value(c), r); };
  auto self = [](u64 c) { return c; };
  u64 cut = 0;
  if (mode == kTopK && (u64)r.k < (u64)list.n)
    cut = list.search(self, list.bits, [](u64) { return (u64)1; }, (u64)r.k);
  if (r.p < 1.0) {
    u64 s = 0;
    list.each([&](u64 c) { s += c >= cut ? fixed(wt(c), scale) : 0; });
    s = group_sum_u64(s, sh);
    // the weight that p is a share of: the top-k's, or the whole row's
    double all = (double)s;
    if (mode == kMinP && gmax) {
      piece_factors(a, row_i, r, sh);
      all = 0.0;
      for (int i = 0; i < a.pieces; ++i) all += a.psum[row_i * a.pieces + i] * sh.factor[i];
      all *= scale;
    }
    u64 need = (u64)ceil(r.p * all);
    if (need < 1) need = 1;
    if (need < s || (need == s && !(mode == kMinP && gmax))) {
      const u64 c2 = list.search(self, list.bits, [&](u64 c) { return c >= cut ? fixed(wt(c), scale) : 0; }, need);
      cut = c2 > cut ? c2 : cut;
    }
  }
  auto mass = [&](u64 c) {
    if (c < cut) return (u64)0;
    const double w = wt(c);
    return w >= r.q ? fixed(w, scale) : (u64)0;
  };
  u64 s = 0;
  list.each([&](u64 c) { s += mass(c); });
  s = group_sum_u64(s, sh);
  u64 target = (u64)((double)r.u * (double)s);
  if (target >= s) target = s - 1;
  // in index order: the larger its complement, the earlier an index
  const u64 mask = ((u64)1 << ib) - 1;
  const u64 at = list.search([=](u64 c) { return c & mask; }, ib, mass, target + 1);
  tok = (int64_t)(mask - at);
  total = (double)s / scale;
  return true;
}

// No filter, or top-p alone on a long row: the pieces' weights above the cut,
// then the piece that holds the answer.  False if the cut lies below the bins
// or its bin overflows the list.
template <typename T>
__device__ bool pick_by_pieces(const SampleArgs& a, const T* z, int64_t row_i, const RowParams& r, uint32_t km,
                               double scale, Mode mode, PickShared& sh, int64_t& tok, double& total) {
  constexpr int low = sizeof(T) == 2 ? 16 : 0;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint32_t* pmax = a.pmax + row_i * a.pieces;
  const double* psum = a.psum + row_i * a.pieces;
  Cut cut{0u, a.V};
  auto mass = [&](int64_t i, float x) { return cut.keeps(i, key_of(x)) ? fixed(weight(x, r), scale) : (u64)0; };
  if (a.pieces == 1) {   // no scan ran: the row is the piece
    u64 s = 0;
    for (int64_t c = threadIdx.x; c < a.V; c += kRowThreads) s += mass(c, clean(to_f32(z[c])));
    s = group_sum_u64(s, sh);
    tok = locate_in_piece(z, a.V, 0, mass, (u64)((double)r.u * (double)s), sh);
    total = (double)s / scale;
    return true;
  }
  piece_factors(a, row_i, r, sh);
  int border = 0;
  const float alpha = bin_scale(r);
  const int top = bin_of(value_of(km), alpha);
  const u64* hist = a.hist + row_i * a.pieces * kSlots;
  if (mode == kTopP) {
    double all = 0.0;
    for (int i = 0; i < a.pieces; ++i) all += psum[i] * sh.factor[i];
    // the row's bins: slot j of piece i is bin (top - its top) + j
    if (threadIdx.x < kSlots) {
      double s = 0.0;
      if (threadIdx.x < kSlots - 1)
        for (int i = 0; i < a.pieces; ++i) {
          if (pmax[i] <= kKeyNegInf) continue;
          const int64_t j = (int64_t)threadIdx.x - ((int64_t)top - bin_of(value_of(pmax[i]), alpha));
          if (j >= 0) s += (double)hist[i * kSlots + j] / scale * sh.factor[i];
        }
      sh.slot[threadIdx.x] = s;
    }
    __syncthreads();
    const double need = r.p * all;
    if (threadIdx.x == 0) {
      double run = 0.0;
      int b = 0;
      for (; b < kSlots - 1; ++b) {
        if (run + sh.slot[b] >= need) break;
        run += sh.slot[b];
      }
      sh.found = b;
      sh.dsum[0] = run;
    }
    __syncthreads();
    border = sh.found;
    const double above = sh.dsum[0];
    if (border == kSlots - 1) return false;
    Candidates<T> list{sh, 0, bits_of((u64)a.V), 0, 0};
    list.kmin = 0;
    list.bits = 32 - low + list.ib;
    const int64_t bin = (int64_t)top - border;
    if (!list.collect(z, a.V, a.gmax + row_i * a.pieces * kPieceGroups,
                      [=](uint32_t k) { return bin_of(value_of(k), alpha) >= bin; },
                      [=](uint32_t, float x) { return bin_of(x, alpha) == bin; }))
      return false;
    auto wt = [&](u64 c) { return fixed(weight(list.value(c), r), scale); };
    u64 s = 0;
    list.each([&](u64 c) { s += wt(c); });
    s = group_sum_u64(s, sh);
    if (s == 0) return false;
    const double rest = ceil((need - above) * scale);
    u64 n = rest < 1.0 ? 1 : (u64)rest;
    if (n > s) n = s;
    const u64 c = list.search([](u64 x) { return x; }, list.bits, wt, n);
    cut = Cut{list.key(c), list.index(c)};
    // the kept part of the border bin, by pieces
    __syncthreads();
    for (int i = threadIdx.x; i < a.pieces; i += kRowThreads) sh.cmass[i] = 0;
    __syncthreads();
    list.each([&](u64 x) {
      if (x >= c) atomicAdd(&sh.cmass[list.index(x) / kPiece], wt(x));
    });
    __syncthreads();
    for (int i = w; i < a.pieces; i += kRowWaves) {
      const double f = sh.factor[i];
      double s2 = 0.0;
      if (f != 0.0) {
        const int64_t shift = (int64_t)top - bin_of(value_of(pmax[i]), alpha);
        for (int j = lane; j < kSlots - 1; j += 64)
          if (shift + j < border) s2 += (double)hist[i * kSlots + j];
      }
      s2 = wave_sum_f64(s2);
      if (lane == 0) sh.dmass[i] = ((double)sh.cmass[i] + s2 * f) / scale;
    }
  } else {
    for (int i = threadIdx.x; i < a.pieces; i += kRowThreads) sh.dmass[i] = psum[i] * sh.factor[i];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < a.pieces; ++i) s += sh.dmass[i];
    const double target = (double)r.u * s;
    double run = 0.0;
    int at = -1, last = 0;
    for (int i = 0; i < a.pieces; ++i) {
      if (sh.dmass[i] > 0.0) last = i;
      if (at < 0) {
        if (run + sh.dmass[i] > target) at = i;
        else run += sh.dmass[i];
      }
    }
    if (at < 0) {   // rounding at the very end: the last counted element
      at = last;
      run = 0.0;
      sh.dsum[1] = s;
    } else {
      sh.dsum[1] = target - run;
    }
    sh.dsum[0] = s;
    sh.found = at;
  }
  __syncthreads();
  total = sh.dsum[0];
  u64 target = (u64)(sh.dsum[1] * scale);
  tok = -1;
  // a piece whose weights all round to nothing passes on to the next
  for (int i = sh.found; i < a.pieces && tok < 0; ++i, target = 0)
    tok = locate_in_piece(z, a.V, (int64_t)i * kPiece, mass, target, sh);
  return tok >= 0;
}

// One row per work-group.
template <typename T>
__global__ __launch_bounds__(kRowThreads) void sample_pick_kernel(SampleArgs a) {
  __shared__ PickShared ps;
  RowShared& sh = ps.row;
  const int64_t row_i = blockIdx.x;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  RowParams r = row_params(a, row_i);
  const Row<T> row(static_cast<const T*>(a.z) + row_i * a.ld, a.V);

  const uint32_t* pmax = a.pmax + row_i * a.pieces;
  const uint32_t* gmax = a.pieces > 1 ? a.gmax + row_i * a.pieces * kPieceGroups : nullptr;
  uint32_t km = 0;
  if (a.pieces > 1) {
    for (int i = threadIdx.x; i < a.pieces; i += kRowThreads) km = pmax[i] > km ? pmax[i] : km;
  } else {
    row.each([&](int64_t, float x) {
      const uint32_t k = key_of(x);
      km = k > km ? k : km;
    });
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t y = __shfl_xor(km, o);
    km = y > km ? y : km;
  }
  if (lane == 0) sh.kmax[w] = km;
  __syncthreads();
  km = 0;
  for (int i = 0; i < kRowWaves; ++i) km = sh.kmax[i] > km ? sh.kmax[i] : km;

  int64_t tok = -1;
  double lp = -__builtin_inf();
  if (r.ok && km > kKeyNegInf) {
    const double scale = __builtin_bit_cast(double, (u64)(1023 + a.s) << 52);
    r.zmax = (double)value_of(km);
    const Mode mode = mode_of(r, a.V);
    double total = 0.0;   // weight of the kept set
    bool done = false;
    if (mode == kGreedy) {
      // the first piece that holds the maximum, then the first index in it
      if (threadIdx.x == 0) ps.found = a.pieces;
      __syncthreads();
      if (a.pieces > 1)
        for (int i = threadIdx.x; i < a.pieces; i += kRowThreads)
          if (pmax[i] == km) atomicMin(&ps.found, i);
      __syncthreads();
      const int64_t at = a.pieces > 1 ? ps.found : 0;
      tok = locate_in_piece(row.z, a.V, at * kPiece, [&](int64_t, float x) { return (u64)(key_of(x) == km); }, 0, ps);
      done = true;
    } else if (mode == kAll || (mode == kTopP && a.pieces > 1)) {
      done = pick_by_pieces(a, row.z, row_i, r, km, scale, mode, ps, tok, total);
    } else {
      done = pick_from_list(a, row.z, row_i, r, km, scale, mode, gmax, ps, tok, total);
    }
    if (mode == kGreedy) {
      lp = 0.0;
    } else if (done) {
      const double z = (double)clean(to_f32(row.z[tok]));
      lp = (z == r.zmax ? 0.0 : (z - r.zmax) / r.t) - log(total);
    } else {
      Cut cut{0u, a.V};
      // the ties at the border go to the lowest indices
      auto tie_index = [&](uint32_t key, u64 count) {
        const int64_t i = row.locate([&](int64_t, float x) { return (u64)(key_of(x) == key); }, count - 1, sh);
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
        const uint32_t key = row.search(
            [&](int64_t i, float x) { return in.keeps(i, key_of(x)) ? fixed(weight(x, r), scale) : 0; },
            [&](u64 all) {
              const u64 n = (u64)ceil(r.p * (double)all);
              return need = n < 1 ? 1 : n > all ? all : n;
            },
            above, sh);
        const u64 each = fixed(weight(value_of(key), r), scale);
        const int64_t i = tie_index(key, (need - above + each - 1) / each);
        cut.idx = key == cut.key && cut.idx < i ? cut.idx : i;
        cut.key = key;
      }
      auto mass = [&](int64_t i, float x) {
        if (!cut.keeps(i, key_of(x))) return (u64)0;
        const double wt = weight(x, r);
        return wt >= r.q ? fixed(wt, scale) : (u64)0;
      };
      u64 s = 0;
      row.each([&](int64_t i, float x) { s += mass(i, x); });
      s = wave_sum_u64(s);
      __syncthreads();
      if (lane == 0) sh.wsum[w] = s;
      __syncthreads();
      s = 0;
      for (int i = 0; i < kRowWaves; ++i) s += sh.wsum[i];
      u64 target = (u64)((double)r.u * (double)s);
      if (target >= s) target = s - 1;
      tok = row.locate(mass, target, sh);
      const double z = (double)clean(to_f32(row.z[tok]));
      lp = (z == r.zmax ? 0.0 : (z - r.zmax) / r.t) - log((double)s / scale);
    }
  }
  if (threadIdx.x == 0) {
    a.tokens[row_i] = tok;
    if (a.logprobs) a.logprobs[row_i] = (float)lp;
  }
}

// Workspace: what the scan leaves, for rows longer than one piece.
struct SampleLayout {
  int64_t pieces;
  size_t psum, hist, gmax, total;   // byte offsets (pmax at 0); total 0: not supported
};

SampleLayout sample_layout(int64_t N, int64_t V) {
  SampleLayout l{(V + kPiece - 1) / kPiece, 0, 0, 0, 0};
  // launches of fewer than 2^32 threads
  if (N > (int64_t(1) << 21) || V > (int64_t(1) << 24) || N * l.pieces > (int64_t(1) << 23)) return l;
  if (l.pieces == 1) {
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
  if (a.pieces > 1) {
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
      sample_pick_kernel<bf16><<<(unsigned)N, kRowThreads, 0, stream>>>(a);
    else
      sample_pick_kernel<float><<<(unsigned)N, kRowThreads, 0, stream>>>(a);
  }
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}
