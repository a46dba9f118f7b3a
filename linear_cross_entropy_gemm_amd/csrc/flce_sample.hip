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

struct SampleArgs {
  const void* z;
  int64_t ld;      // elements
  const float* u;
  int64_t N, V;
  flce_sample_params_t prm;
  int s;           // weights are multiples of 2^-s
  int64_t* tokens;
  float* logprobs;
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

// One row per work-group, any parameters.
template <typename T>
__global__ __launch_bounds__(kRowThreads) void sample_row_kernel(SampleArgs a) {
  __shared__ RowShared sh;
  const int64_t row_i = blockIdx.x;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  RowParams r = row_params(a, row_i);
  const Row<T> row(static_cast<const T*>(a.z) + row_i * a.ld, a.V);

  uint32_t km = 0;
  row.each([&](int64_t, float x) {
    const uint32_t k = key_of(x);
    km = k > km ? k : km;
  });
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
    if (r.t == 0.0) {
      tok = row.locate([&](int64_t, float x) { return (u64)(key_of(x) == km); }, 0, sh);
      lp = 0.0;
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

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

}  // namespace flce

extern "C" size_t flce_sample_workspace_size(int64_t N, int64_t V, int dtype) {
  if ((dtype != FLCE_DTYPE_BF16 && dtype != FLCE_DTYPE_F32) || N < 0 || V < 1) return 0;
  if (N > (int64_t(1) << 22) || V > (int64_t(1) << 24)) return 0;
  return 256;
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
  if (N > (int64_t(1) << 22) || V > (int64_t(1) << 24)) return FLCE_EUNSUPPORTED;
  if (N == 0) return FLCE_OK;
  if (workspace_bytes < flce_sample_workspace_size(N, V, dtype)) return FLCE_EWORKSPACE;
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
  ProfileScope ps(FLCE_KERNEL_SAMPLE, stream);
  if (dtype == FLCE_DTYPE_BF16)
    sample_row_kernel<bf16><<<(unsigned)N, kRowThreads, 0, stream>>>(a);
  else
    sample_row_kernel<float><<<(unsigned)N, kRowThreads, 0, stream>>>(a);
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}
