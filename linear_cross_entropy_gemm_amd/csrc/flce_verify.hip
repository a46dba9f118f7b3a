// Verification of drafted tokens against the target's distribution from given
// random numbers (flce_verify), with the sampler's temperature and filters.
//
// Sequence b has K drafted tokens x_i (the first len_b of them), the draft's
// distributions q_i that they were drawn from and the target's p_0 .. p_K:
//   n = the first i with i >= len_b or u_i q_i(x_i) >= p_i(x_i)
//   tokens = x_0 .. x_{n-1} and one drawn from r = max(p_n - q_n, 0) (from p_n
//   where the draft had ended)
// which leaves every token distributed as if drawn from p.
//
//   1. the sampler's scan and pick leave each row's cut and sum of weights
//      instead of a token (sample_rows.hpp): all 2K + 1 rows of a sequence at
//      once, since a row's turn is known only after the rows before it
//   2. verify_count_kernel: n from K pairs of logits, a wave per sequence, and
//      what is known with it: the accepted tokens
//   3. verify_residual_kernel: the weight of r by pieces of 4096
//   4. verify_draw_kernel: the piece in which the running sum passes u, and the
//      token in it, in index order
// What bounds them (MI355X, us): 64 sequences of 4 on 129279 fp32 logits, each with
// parameters of its own (298 MB): scan 50, its memory; rows 26, one work-group's
// chain of steps each; count 6, residual 17, draw 9.  32 of 7 on 202048 bf16 logits
// without filters (194 MB): scan 82, where the vector units are busy 82% of the
// time with 26 instructions a logit, half of them the 64-bit exponential's; rows
// 5, count 6, residual 24, draw 9.  One sequence of 4 with k = 50 and p = 0.95: 4,
// 14, 7 (residual and count), 6, each kernel the latency of its steps.
// A distribution's values are formed from the logits again where they are
// needed: 64-bit exponentials over a row's sum; r goes into integers of 2^-51,
// whose sums are exact in any order.
#include <cmath>

#include "sample_rows.hpp"

namespace flce {

namespace {

constexpr int kVerThreads = 256;
constexpr int kVerPiece = 4096;
constexpr double kVerScale = 0x1p51;
constexpr int64_t kMaxDrafted = 1024;

struct VerifyArgs {
  StatsArgs s;   // rows, parameters and what the sampler's kernels left
  bool drafts;    // the draft's logits are given (else its tokens are certain)
  const int64_t* x;
  const int64_t* lens;   // null: K
  const float* u;
  const float* u_draw;
  int64_t B;
  int K, pieces;
  int* n;        // [B]
  u64* rsum;     // [B][pieces] of r
  u64* psum;     // [B][pieces] of p
  int64_t* tokens;
  int64_t* accepted;
  float* logprobs;
};

// A row's distribution.
template <typename T>
struct Dist {
  RowParams r;
  const T* z;
  u64 cut, least;
  double scale, inv;   // probability = weight * inv
  bool live, plain;

  __device__ __forceinline__ Dist(const StatsArgs& a, int64_t row) : r(row_params<true>(a, row)) {
    const RowStat st = a.stats[row];
    z = row_logits<T, true>(a, row);
    live = st.live != 0;
    cut = live ? st.cut : ~(u64)0;
    scale = scale_of(a);
    least = floor_weight(r, scale);
    const float m = value_of(st.kmax);
    r.set_max(m);
    plain = ordinary(m, r);
    inv = r.t == 0.0 ? 1.0 : scale / (double)st.sum;
  }
  __device__ __forceinline__ bool reaches(float x) const { return key_of(x) >= key_in(cut); }
  // (weights that round to 0 in the sums' unit count here, where a token is
  // judged, and have no part in what is drawn; 2^-1000 stands for 0)
  __device__ __forceinline__ double prob(int64_t i, float x) const {
    if (!live || composite(key_of(x), i) < cut || !(x > kNegInf)) return 0.0;
    if (r.t == 0.0) return 1.0;
    const double w = plain ? weight(x, r) : weight_any(x, r);
    if (w < 0x1p-900 || (r.q > 0.0 && fixed(w, scale) < least)) return 0.0;
    return w * inv;
  }
  // of E consecutive ones
  template <int E>
  __device__ __forceinline__ void probs(double (&out)[E], int64_t i, const float (&x)[E]) const {
    if (live && plain && r.t != 0.0) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const double w = weight(x[e], r);
        const bool in = composite(key_of(x[e]), i + e) >= cut && w >= 0x1p-900;
        out[e] = in ? w : 0.0;
      }
      if (r.q > 0.0) {
#pragma unroll
        for (int e = 0; e < E; ++e) out[e] = fixed(out[e], scale) < least ? 0.0 : out[e];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) out[e] *= inv;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) out[e] = prob(i + e, x[e]);
    }
  }
  __device__ __forceinline__ double prob(int64_t i) const { return prob(i, clean(to_f32(z[i]))); }
  __device__ __forceinline__ float logprob(int64_t i) const {
    if (r.t == 0.0) return 0.0f;
    const double y = __builtin_fmin(((double)clean(to_f32(z[i])) - r.zmax) * r.rate, 0.0);
    return (float)(y * 0.69314718055994530942 + log(inv));
  }
};

__device__ __forceinline__ int64_t target_row(const VerifyArgs& v, int64_t b, int i) { return b * (v.K + 1) + i; }
__device__ __forceinline__ int64_t draft_row(const VerifyArgs& v, int64_t b, int i) { return v.s.n1 + b * v.K + i; }

__device__ __forceinline__ int drafted(const VerifyArgs& v, int64_t b) {
  if (!v.lens) return v.K;
  const int64_t n = v.lens[b];
  return n < 0 ? 0 : n > v.K ? v.K : (int)n;
}

// How many drafted tokens of sequence b are accepted: one wave, a lane per
// position.  With `put` the outputs that are known then are written: all but
// the token that is drawn.
template <typename T>
__device__ __forceinline__ int count_accepted(const VerifyArgs& v, int64_t b, bool put) {
  const int len = drafted(v, b), lane = threadIdx.x & 63;
  int n = len;
#pragma unroll 1
  for (int i0 = 0; i0 < len && n == len; i0 += 64) {
    const int i = i0 + lane;
    bool ok = false;
    int64_t x = -1;
    float lp = kNegInf;
    if (i < len) {
      x = v.x[b * v.K + i];
      const float u = v.u[b * v.K + i];
      if (x >= 0 && x < v.s.V && u >= 0.0f && u < 1.0f) {
        const Dist<T> at(v.s, target_row(v, b, i));
        const double p = at.prob(x);
        const double q = v.drafts ? Dist<T>(v.s, draft_row(v, b, i)).prob(x) : 1.0;
        ok = (double)u * q < p;
        if (put && v.logprobs) lp = at.logprob(x);
      }
    }
    const unsigned long long bad = ~__builtin_amdgcn_ballot_w64(ok);
    if (bad) {
      n = i0 + __builtin_ctzll(bad);
      if (n > len) n = len;
    }
    if (put && i < n) {
      v.tokens[target_row(v, b, i)] = x;
      if (v.logprobs) v.logprobs[target_row(v, b, i)] = lp;
    }
  }
  if (put) {
    for (int i = n + 1 + lane; i <= v.K; i += 64) {
      v.tokens[target_row(v, b, i)] = -1;
      if (v.logprobs) v.logprobs[target_row(v, b, i)] = kNegInf;
    }
    if (lane == 0) {
      v.n[b] = n;
      v.accepted[b] = n;
    }
  }
  return n;
}

// The weights that sequence b's last token is drawn from, behind n accepted
// ones.
template <typename T>
struct Residual {
  Dist<T> p, q;
  bool with_q;      // the draft's distribution
  int64_t certain;  // its certain token, -1: none

  __device__ __forceinline__ Residual(const VerifyArgs& v, int64_t b, int n)
      : p(v.s, target_row(v, b, n)),
        q(v.s, v.drafts && n < drafted(v, b) ? draft_row(v, b, n) : target_row(v, b, n)) {
    const bool on = n < drafted(v, b);
    with_q = on && v.drafts;
    certain = on && !v.drafts ? v.x[b * v.K + n] : -1;
  }
  // both integer weights of E logits from index i on; no branches among them in
  // ordinary rows
  template <int E>
  __device__ __forceinline__ void weights(int64_t i, const typename RowVec<T>::type& zp,
                                          const typename RowVec<T>::type& zq, u64 (&rw)[E], u64 (&pw)[E]) const {
    float x[E], y[E];
    bool any = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] = clean(to_f32(zp[e]));
      y[e] = clean(to_f32(zq[e]));
      any |= p.reaches(x[e]);
      rw[e] = pw[e] = 0;
    }
    if (!__builtin_amdgcn_ballot_w64(any)) return;
    double a[E], c[E];
    p.probs(a, i, x);
#pragma unroll
    for (int e = 0; e < E; ++e) c[e] = 0.0;
    if (with_q) q.probs(c, i, y);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (i + e == certain) c[e] = 1.0;
      pw[e] = fixed(a[e], kVerScale);
      rw[e] = fixed(__builtin_fmax(a[e] - c[e], 0.0), kVerScale);
    }
  }
};

// One wave per sequence.
template <typename T>
__global__ __launch_bounds__(64) void verify_count_kernel(VerifyArgs v) {
  count_accepted<T>(v, blockIdx.x, true);
}

// With kCount every work-group finds n by itself.
template <typename T, bool kCount>
__global__ __launch_bounds__(kVerThreads) void verify_residual_kernel(VerifyArgs v) {
  constexpr int E = RowVec<T>::E, kVec = kVerPiece / (kVerThreads * E);
  __shared__ u64 part[2][kVerThreads / 64];
  __shared__ int n_of;
  const int64_t b = blockIdx.x / v.pieces;
  const int piece = blockIdx.x % v.pieces;
  int n;
  if (kCount) {
    if (threadIdx.x < 64) {
      n = count_accepted<T>(v, b, piece == 0);
      if (threadIdx.x == 0) n_of = n;
    }
    __syncthreads();
    n = n_of;
  } else {
    n = v.n[b];
  }
  const Residual<T> res(v, b, n);
  u64 rs = 0, ps = 0;
  if (res.p.live) {
    const int64_t base = (int64_t)piece * kVerPiece + threadIdx.x * E;
    typename RowVec<T>::type zp[kVec], zq[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int64_t c = base + j * kVerThreads * E;
      zp[j] = load_row(res.p.z, c, v.s.V, kNegInf);
      zq[j] = zp[j];
      if (res.with_q) zq[j] = load_row(res.q.z, c, v.s.V, kNegInf);
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      u64 rw[E], pw[E];
      res.weights(base + j * kVerThreads * E, zp[j], zq[j], rw, pw);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        rs += rw[e];
        ps += pw[e];
      }
    }
  }
  rs = wave_sum_u64(rs);
  ps = wave_sum_u64(ps);
  if ((threadIdx.x & 63) == 0) {
    part[0][threadIdx.x >> 6] = rs;
    part[1][threadIdx.x >> 6] = ps;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    v.rsum[b * v.pieces + piece] = part[0][0] + part[0][1] + part[0][2] + part[0][3];
    v.psum[b * v.pieces + piece] = part[1][0] + part[1][1] + part[1][2] + part[1][3];
  }
}

// One vector of the piece per thread.
template <typename T>
__global__ __launch_bounds__(kVerPiece / RowVec<T>::E) void verify_draw_kernel(VerifyArgs v) {
  constexpr int E = RowVec<T>::E, TH = kVerPiece / E;
  __shared__ GroupScratch<TH> scratch;
  __shared__ int found;
  __shared__ u64 rest;
  const int64_t b = blockIdx.x;
  const int t = threadIdx.x, n = v.n[b];
  const float u = v.u_draw[b];
  const Residual<T> res(v, b, n);
  const int64_t at = target_row(v, b, n);
  // consecutive pieces per thread; p itself where nothing is left of r
  const int per = (v.pieces + TH - 1) / TH;
  const u64* sums = v.rsum + b * v.pieces;
  u64 own = 0, all = 0, before = 0;
  for (int way = 0; way < 2; ++way) {
    if (way) sums = v.psum + b * v.pieces;
    own = 0;
    for (int i = t * per; i < (t + 1) * per && i < v.pieces; ++i) own += sums[i];
    before = group_scan<TH>(own, all, scratch);
    if (all) break;
  }
  const bool from_p = sums != v.rsum + b * v.pieces;
  if (!all || !(u >= 0.0f && u < 1.0f)) {
    if (t == 0) {
      v.tokens[at] = -1;
      if (v.logprobs) v.logprobs[at] = kNegInf;
    }
    return;
  }
  const u64 target = draw_target(u, all);
  if (before <= target && target < before + own) {   // one thread
    int i = t * per;
    for (; target >= before + sums[i]; ++i) before += sums[i];
    found = i;
    rest = target - before;
  }
  __syncthreads();
  const int64_t c = (int64_t)found * kVerPiece + t * E;
  const typename RowVec<T>::type zp = load_row(res.p.z, c, v.s.V, kNegInf);
  typename RowVec<T>::type zq = zp;
  if (res.with_q) zq = load_row(res.q.z, c, v.s.V, kNegInf);
  u64 rw[E], pw[E];
  res.weights(c, zp, zq, rw, pw);
  own = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) own += from_p ? pw[e] : rw[e];
  before = group_scan<TH>(own, all, scratch);
  if (before <= rest && rest < before + own) {   // one thread
    int64_t x = c;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      before += from_p ? pw[e] : rw[e];
      if (before <= rest) x = c + e + 1;
    }
    v.tokens[at] = x;
    if (v.logprobs) v.logprobs[at] = res.p.logprob(x);
  }
}

template <typename T>
void launch_verify(const VerifyArgs& v, hipStream_t stream) {
  // The sequences' accepted counts by themselves, or again in every work-group
  // where all of those are on the chip at once: 7 us against 5 + 6 with one
  // sequence of 4 tokens (202048 logits); with 32 of 7 it was 37 against 6 + 32,
  // of which the weights take less now (24).
  const unsigned g = (unsigned)(v.B * v.pieces);
  if (g <= 1024) {
    ProfileScope ps(FLCE_KERNEL_VERIFY_RESIDUAL, stream);
    verify_residual_kernel<T, true><<<g, kVerThreads, 0, stream>>>(v);
  } else {
    {
      ProfileScope ps(FLCE_KERNEL_VERIFY_COUNT, stream);
      verify_count_kernel<T><<<(unsigned)v.B, 64, 0, stream>>>(v);
    }
    ProfileScope ps(FLCE_KERNEL_VERIFY_RESIDUAL, stream);
    verify_residual_kernel<T, false><<<g, kVerThreads, 0, stream>>>(v);
  }
  ProfileScope ps(FLCE_KERNEL_VERIFY_DRAW, stream);
  verify_draw_kernel<T><<<(unsigned)v.B, kVerPiece / RowVec<T>::E, 0, stream>>>(v);
}

struct VerifyLayout {
  SampleLayout rows;
  int64_t pieces;
  size_t stats, n, rsum, psum, total;   // total 0: not supported
};

VerifyLayout verify_layout(int64_t B, int64_t K, int64_t V, bool drafts) {
  VerifyLayout l{};
  if (B > (int64_t(1) << 21) || K > kMaxDrafted) return l;
  const int64_t R = B * (drafts ? 2 * K + 1 : K + 1);
  l.rows = sample_layout(R, V);
  l.pieces = ceil_div(V, kVerPiece);
  if (l.rows.total == 0 || B * l.pieces >= (int64_t(1) << 24)) return l;   // launches of fewer than 2^32 threads
  auto pad = [](size_t b) { return (b + 255) & ~size_t(255); };
  l.stats = pad(l.rows.total);
  l.n = l.stats + pad((size_t)R * sizeof(RowStat));
  l.rsum = l.n + pad((size_t)B * 4);
  l.psum = l.rsum + pad((size_t)(B * l.pieces) * 8);
  l.total = l.psum + pad((size_t)(B * l.pieces) * 8);
  return l;
}

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

}  // namespace flce

extern "C" size_t flce_verify_workspace_size(int64_t B, int64_t K, int64_t V, int dtype, int with_draft) {
  if ((dtype != FLCE_DTYPE_BF16 && dtype != FLCE_DTYPE_F32) || B < 0 || K < 0 || V < 1) return 0;
  return flce::verify_layout(B, K, V, with_draft != 0).total;
}

extern "C" int flce_verify(const void* target, int64_t ld_target, const void* draft, int64_t ld_draft,
                           const int64_t* draft_tokens, const int64_t* draft_lens, const float* u, const float* u_draw,
                           int64_t B, int64_t K, int64_t V, const flce_sample_params_t* params,
                           const flce_sample_params_t* draft_params, int64_t* tokens, int64_t* accepted,
                           float* logprobs, hipStream_t stream, int dtype, void* workspace, size_t workspace_bytes) {
  using namespace flce;
  if (dtype != FLCE_DTYPE_BF16 && dtype != FLCE_DTYPE_F32) return FLCE_EINVAL;
  if (B < 0 || K < 0 || V < 1 || !params) return FLCE_EINVAL;
  const uintptr_t es = dtype == FLCE_DTYPE_BF16 ? 2 : 4;
  if (!draft_params) draft_params = params;
  if (!sample_params_ok(*params) || !sample_params_ok(*draft_params)) return FLCE_EINVAL;
  if (!on(target, es) || !on(draft, es) || !on(draft_tokens, 8) || !on(draft_lens, 8) || !on(u, 4) ||
      !on(u_draw, 4) || !on(tokens, 8) || !on(accepted, 8) || !on(logprobs, 4) || !on(workspace, 256))
    return FLCE_EINVAL;
  if (ld_target < 0 || (draft && ld_draft < 0)) return FLCE_EINVAL;
  if (B > 0 && (!target || !u_draw || !tokens || !accepted || !workspace)) return FLCE_EINVAL;
  if (B > 0 && K > 0 && (!draft_tokens || !u)) return FLCE_EINVAL;
  const bool drafts = draft && K > 0;
  const VerifyLayout l = verify_layout(B, K, V, drafts);
  if (l.total == 0) return FLCE_EUNSUPPORTED;
  if (B == 0) return FLCE_OK;
  if (workspace_bytes < l.total) return FLCE_EWORKSPACE;
  char* ws = static_cast<char*>(workspace);
  VerifyArgs v{};
  StatsArgs& a = v.s;
  a.z = target;
  a.ld = ld_target;
  a.z2 = draft;
  a.ld2 = ld_draft;
  a.n1 = B * (K + 1);
  a.per1 = (uint32_t)(K + 1);
  a.per2 = (uint32_t)(K > 0 ? K : 1);
  a.prm = *params;
  a.prm2 = *draft_params;
  a.stats = reinterpret_cast<RowStat*>(ws + l.stats);
  sample_args(a, B * (drafts ? 2 * K + 1 : K + 1), V, l.rows, ws);
  v.drafts = drafts;
  v.x = draft_tokens;
  v.lens = draft_lens;
  v.u = u;
  v.u_draw = u_draw;
  v.B = B;
  v.K = (int)K;
  v.pieces = (int)l.pieces;
  v.n = reinterpret_cast<int*>(ws + l.n);
  v.rsum = reinterpret_cast<u64*>(ws + l.rsum);
  v.psum = reinterpret_cast<u64*>(ws + l.psum);
  v.tokens = tokens;
  v.accepted = accepted;
  v.logprobs = logprobs;
  launch_rows<true>(a, stream, dtype, FLCE_KERNEL_VERIFY_SCAN, FLCE_KERNEL_VERIFY_ROWS);
  if (dtype == FLCE_DTYPE_BF16)
    launch_verify<bf16>(v, stream);
  else
    launch_verify<float>(v, stream);
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}
