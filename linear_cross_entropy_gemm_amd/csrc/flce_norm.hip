// Layer norm over the last dimension, forward (flce_layer_norm_fwd) and
// backward (flce_layer_norm_bwd).  Row x of H values, weight w, bias b:
//
//   mean = avg x, var = avg (x - mean)^2, rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   g = dy w,  dx = rstd (g - avg g - xh avg(g xh))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
//   ln_fwd_kernel    the row stays in registers: one read, one write
//   ln_bwd_kernel    the rows x and dy stay in registers; each thread keeps
//                    dw and db of its columns in registers over all rows of
//                    its group and stores them once
//   ln_*_wide_kernel rows too long for registers: several passes over a row
//   ln_param_grad_kernel  dw and db of wide rows, by columns
//   ln_reduce_kernel sum of the groups' dw and db in a fixed order
//
// Bound by memory, at 75 to 100% of the rate of torch's plain copy (launch_fwd
// lists the shapes): forward 8192 x 6656 bf16 in 50 us (4.4 TB/s), backward in
// 75 us (4.4 TB/s, 5 us of it the reduction).  The wide rows read x three
// times forward and x and dy three times backward, partly out of the caches:
// 4096 x 16384 fp32 in 145 us (3.7 TB/s of one read and one write) and 292 us
// (2.8 TB/s), so a row one vector beyond the registers takes 65 and 164 us
// where 4096 x 8192 fp32 takes 55 and 83.  A persistent work-group keeps the
// parameters and the next row in registers; the loads of the next row must
// not wait on a branch, so a vector past the row's end is read from inside the
// row and put right when it is used (a branch per vector cost a tenth).
#include <cmath>

#include "flce_internal.hpp"
#include "row_ops.hpp"

namespace flce {

namespace {

// Statistics, sums and products are fp32; y, dx, dw and db are rounded to
// their storage dtype once, at the store.
struct LnFwdArgs {
  const void* x;
  const void* weight;   // null: 1
  const void* bias;     // null: 0
  void* y;
  float* mean;          // may be null
  float* rstd;          // may be null
  int64_t M, ldx, ldy;  // strides in elements
  int H;
  float eps;
};

struct LnBwdArgs {
  const void* dy;
  const void* x;
  const void* weight;
  const float* mean;
  const float* rstd;
  void* dx;             // null: not needed
  float* partial;       // [groups][2][H]: dw, then db; null: not needed
  int64_t M, ldy, ldx, ldg;
  int H;
};

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

// Mean and 1 / standard deviation of a row from its waves' own: a wave's mean
// and sum of squared deviations from it need no barrier, and
//   mean = sum n_w mean_w / H,  sum of squares = sum (q_w + n_w (mean_w - mean)^2)
// joins them behind one.  A mean is kept in two parts throughout, the rounded
// one that the deviations were taken from and what its rounding left over: one
// fp32 number for a wave's mean would move every y of a row at 1e5 standard
// deviations from zero by 3e-3, the two parts leave 4e-7.
// kRow threads hold a row in kVec vectors each; a work-group holds kRows
// rows (more than one only where a row is one wave) and walks over the rows
// in steps of the grid, the next row's loads issued before the current row's
// sums.
template <typename T, typename WT, int kRow, int kVec, int kRows, int kEu>
__global__ __launch_bounds__(kRow* kRows) __attribute__((amdgpu_waves_per_eu(kEu))) void ln_fwd_kernel(LnFwdArgs p) {
  static_assert(kRow == 64 || kRows == 1, "a work-group barrier must see one row");
  constexpr int E = RowVec<T>::E, kWaves = kRow / 64;
  typedef typename RowVec<T>::type vec_t;
  __shared__ float lds[2][3][kWaves];
  int buf = 0;
  const int t = threadIdx.x % kRow, wave = t >> 6;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kRow;
  if (row >= p.M) return;   // whole waves (kRow = 64) or the whole work-group
  vec_t cur[kVec], nxt[kVec];
  auto load = [&](vec_t (&to)[kVec], int64_t from) {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      to[i] = load_clamped(static_cast<const T*>(p.x) + from * p.ldx, (t + i * kRow) * E, p.H);
  };
  // elements that wave w holds
  auto count = [&](int w) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int left = p.H - (w * 64 + i * kRow) * E;
      n += left < 0 ? 0 : left < 64 * E ? left : 64 * E;
    }
    return (float)n;
  };
  load(cur, row);
  float w[kVec][E], b[kVec][E];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    load_param<WT>(w[i], p.weight, (t + i * kRow) * E, p.H, 1.0f);
    load_param<WT>(b[i], p.bias, (t + i * kRow) * E, p.H, 0.0f);
  }
  const float inv = 1.0f / (float)p.H, mine = count(wave), inv_mine = mine > 0.0f ? 1.0f / mine : 0.0f;
  for (; row < p.M; row += step) {
    if (row + step < p.M) load(nxt, row + step);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      row_tail<T>(cur[i], (t + i * kRow) * E, p.H);
#pragma unroll
      for (int e = 0; e < E; ++e) s = __builtin_fmaf(to_f32(cur[i][e]), inv_mine, s);   // a sum could overflow
    }
    const float m0 = wave_sum(s);
    // squares of the deviations, and the deviations' own average: what the
    // rounding of m0 left over is taken out of both results (as a sum, the
    // half of a row's deviations that has one sign could overflow)
    float d1 = 0.0f, d2 = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int left = p.H - (t + i * kRow) * E;
      if (__builtin_amdgcn_ballot_w64(left < E)) {   // the row ends in this wave's vectors
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float x = e < left ? to_f32(cur[i][e]) - m0 : 0.0f;
          d1 = __builtin_fmaf(x, inv_mine, d1);
          d2 = __builtin_fmaf(x, x, d2);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float x = to_f32(cur[i][e]) - m0;
          d1 = __builtin_fmaf(x, inv_mine, d1);
          d2 = __builtin_fmaf(x, x, d2);
        }
      }
    }
    const float rest0 = wave_sum(d1), q0 = __builtin_fmaf(-(rest0 * mine), rest0, wave_sum(d2));
    // the row's mean is m + rest
    float m = m0, rest = rest0, q = q0;
    if (kRow > 64) {
      if ((threadIdx.x & 63) == 0) {
        lds[buf][0][wave] = m0;
        lds[buf][1][wave] = rest0;
        lds[buf][2][wave] = q0;
      }
      __syncthreads();
      m = lds[buf][0][0];   // deviations of the waves' means from the first's rounded one
      auto from_first = [&](int i) { return (lds[buf][0][i] - m) + lds[buf][1][i]; };
      rest = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) rest = __builtin_fmaf(count(i) * inv, from_first(i), rest);
      q = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        const float d = from_first(i) - rest, n = count(i);
        q += n > 0.0f ? __builtin_fmaf(n * d, d, lds[buf][2][i]) : 0.0f;
      }
      buf ^= 1;
    }
    const float var = q * inv;
    const float rstd = 1.0f / sqrtf((var > 0.0f ? var : var == var ? 0.0f : var) + p.eps);
    T* yr = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      vec_t o;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float xh = ((to_f32(cur[i][e]) - m) - rest) * rstd;
        o[e] = (T)__builtin_fmaf(xh, w[i][e], b[i][e]);
      }
      store_row(yr, (t + i * kRow) * E, p.H, o);
    }
    if (t == 0) {
      if (p.mean) p.mean[row] = m + rest;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) cur[i] = nxt[i];
  }
}

constexpr int kWide = 1024;

// Rows too long for registers: mean, deviations and output in three passes
// over the row (the second and third mostly out of the L2).
template <typename T, typename WT>
__global__ __launch_bounds__(kWide) void ln_fwd_wide_kernel(LnFwdArgs p) {
  constexpr int E = RowVec<T>::E;
  typedef typename RowVec<T>::type vec_t;
  __shared__ SumLds<1> lds1;
  __shared__ SumLds<2> lds2;
  int buf = 0, buf2 = 0;
  const float inv = 1.0f / (float)p.H;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.ldx;
    float s[1] = {0.0f};
    for (int c = threadIdx.x * E; c < p.H; c += kWide * E) {
      const vec_t v = load_row(xr, c, p.H);
#pragma unroll
      for (int e = 0; e < E; ++e) s[0] = __builtin_fmaf(to_f32(v[e]), inv, s[0]);
    }
    row_sums<kWide>(s, lds1, buf);
    const float mean0 = s[0];
    float dev[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x * E; c < p.H; c += kWide * E) {
      const vec_t v = load_row(xr, c, p.H);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = c + e < p.H ? to_f32(v[e]) - mean0 : 0.0f;
        dev[0] = __builtin_fmaf(d, inv, dev[0]);
        dev[1] = __builtin_fmaf(d, d, dev[1]);
      }
    }
    row_sums<kWide>(dev, lds2, buf2);
    const float rest = dev[0];
    const float var = __builtin_fmaf(-rest, rest, dev[1] * inv);
    const float rstd = 1.0f / sqrtf((var > 0.0f ? var : var == var ? 0.0f : var) + p.eps);
    T* yr = static_cast<T*>(p.y) + row * p.ldy;
    for (int c = threadIdx.x * E; c < p.H; c += kWide * E) {
      const vec_t v = load_row(xr, c, p.H);
      float w[E], b[E];
      load_param<WT>(w, p.weight, c, p.H, 1.0f);
      load_param<WT>(b, p.bias, c, p.H, 0.0f);
      vec_t o;
#pragma unroll
      for (int e = 0; e < E; ++e)
        o[e] = (T)__builtin_fmaf(((to_f32(v[e]) - mean0) - rest) * rstd, w[e], b[e]);
      store_row(yr, c, p.H, o);
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mean0 + rest;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
}

template <typename T, typename WT, int kRow, int kVec, int kRows, int kEu>
__global__ __launch_bounds__(kRow* kRows) __attribute__((amdgpu_waves_per_eu(kEu))) void ln_bwd_kernel(LnBwdArgs p) {
  static_assert(kRow == 64 || kRows == 1, "a work-group barrier must see one row");
  constexpr int E = RowVec<T>::E;
  typedef typename RowVec<T>::type vec_t;
  __shared__ SumLds<2> lds;
  int buf = 0;
  const int t = threadIdx.x % kRow, sub = threadIdx.x / kRow;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + sub;
  struct Rows {
    vec_t x[kVec], d[kVec];
    float mean, rstd;
  } cur, nxt;
  auto load = [&](Rows& to, int64_t from) {
    to.mean = p.mean[from];
    to.rstd = p.rstd[from];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      to.x[i] = load_clamped(static_cast<const T*>(p.x) + from * p.ldx, (t + i * kRow) * E, p.H);
      to.d[i] = load_clamped(static_cast<const T*>(p.dy) + from * p.ldy, (t + i * kRow) * E, p.H);
    }
  };
  if (row < p.M) load(cur, row);
  float w[kVec][E], dw[kVec][E], db[kVec][E];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    load_param<WT>(w[i], p.weight, (t + i * kRow) * E, p.H, 1.0f);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[i][e] = db[i][e] = 0.0f;
  }
  const float inv = 1.0f / (float)p.H;
  for (; row < p.M; row += step) {
    if (row + step < p.M) load(nxt, row + step);
    // columns past the row's end hold dy = 0 and add nothing to any sum
    float s[2] = {0.0f, 0.0f}, xh[kVec][E];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      row_tail<T>(cur.x[i], (t + i * kRow) * E, p.H);
      row_tail<T>(cur.d[i], (t + i * kRow) * E, p.H);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = to_f32(cur.d[i][e]), g = d * w[i][e];
        xh[i][e] = (to_f32(cur.x[i][e]) - cur.mean) * cur.rstd;
        s[0] += g;
        s[1] = __builtin_fmaf(g, xh[i][e], s[1]);
        dw[i][e] = __builtin_fmaf(d, xh[i][e], dw[i][e]);
        db[i][e] += d;
      }
    }
    if (p.dx) {
      row_sums<kRow>(s, lds, buf);
      const float m1 = s[0] * inv, m2 = s[1] * inv * cur.rstd;
      T* gr = static_cast<T*>(p.dx) + row * p.ldg;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        vec_t o;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float g = __builtin_fmaf(to_f32(cur.d[i][e]), w[i][e], -m1);
          o[e] = (T)__builtin_fmaf(g, cur.rstd, -(xh[i][e] * m2));
        }
        store_row(gr, (t + i * kRow) * E, p.H, o);
      }
    }
    cur = nxt;
  }
  if (!p.partial) return;
  float* out = p.partial + (int64_t)blockIdx.x * 2 * p.H;
  if constexpr (kRows > 1) {
    // the work-group's waves add up their columns in order
    __shared__ float acc[kRows][2][kVec * E][kRow];
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        acc[sub][0][i * E + e][t] = dw[i][e];
        acc[sub][1][i * E + e][t] = db[i][e];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.H; c += kRow * kRows) {
      const int which = c >= p.H, col = which ? c - p.H : c;
      const int v = col / E, th = v % kRow, k = v / kRow * E + col % E;
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) s += acc[r][which][k][th];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const int col = (t + i * kRow) * E + e;
        store_row<float>(out, col, p.H, f32x4{dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]});
        store_row<float>(out + p.H, col, p.H, f32x4{db[i][e], db[i][e + 1], db[i][e + 2], db[i][e + 3]});
      }
  }
}

// dx of rows too long for registers: the two sums, then the output.
template <typename T, typename WT>
__global__ __launch_bounds__(kWide) void ln_bwd_wide_kernel(LnBwdArgs p) {
  constexpr int E = RowVec<T>::E;
  typedef typename RowVec<T>::type vec_t;
  __shared__ SumLds<2> lds;
  int buf = 0;
  const float inv = 1.0f / (float)p.H;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dr = static_cast<const T*>(p.dy) + row * p.ldy;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x * E; c < p.H; c += kWide * E) {
      const vec_t x = load_row(xr, c, p.H), d = load_row(dr, c, p.H);
      float w[E];
      load_param<WT>(w, p.weight, c, p.H, 1.0f);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float g = to_f32(d[e]) * w[e];
        s[0] += g;
        s[1] = __builtin_fmaf(g, (to_f32(x[e]) - mean) * rstd, s[1]);
      }
    }
    row_sums<kWide>(s, lds, buf);
    const float m1 = s[0] * inv, m2 = s[1] * inv;
    T* gr = static_cast<T*>(p.dx) + row * p.ldg;
    for (int c = threadIdx.x * E; c < p.H; c += kWide * E) {
      const vec_t x = load_row(xr, c, p.H), d = load_row(dr, c, p.H);
      float w[E];
      load_param<WT>(w, p.weight, c, p.H, 1.0f);
      vec_t o;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float xh = (to_f32(x[e]) - mean) * rstd;
        o[e] = (T)((__builtin_fmaf(to_f32(d[e]), w[e], -m1) - xh * m2) * rstd);
      }
      store_row(gr, c, p.H, o);
    }
  }
}

// dw and db of wide rows: thread = one column, group y takes every
// gridDim.y-th row.
template <typename T>
__global__ __launch_bounds__(256) void ln_param_grad_kernel(LnBwdArgs p) {
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col >= p.H) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < p.M; row += gridDim.y) {
    const float d = to_f32(static_cast<const T*>(p.dy)[row * p.ldy + col]);
    const float x = to_f32(static_cast<const T*>(p.x)[row * p.ldx + col]);
    dw = __builtin_fmaf(d, (x - p.mean[row]) * p.rstd[row], dw);
    db += d;
  }
  float* out = p.partial + (int64_t)blockIdx.y * 2 * p.H;
  out[col] = dw;
  out[p.H + col] = db;
}

// Sum of the groups' partials: 64 columns per work-group, 16 waves over the
// groups, joined in order.
template <typename WT>
__global__ __launch_bounds__(1024) void ln_reduce_kernel(const float* partial, int groups, int H, WT* dw, WT* db) {
  __shared__ float lds[16][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < 2 * H) {
    // eight loads under way, added in order
    int g = wv;
    for (; g + 7 * 16 < groups; g += 8 * 16) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = partial[(int64_t)(g + i * 16) * 2 * H + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; g < groups; g += 16) s += partial[(int64_t)g * 2 * H + c];
  }
  lds[wv][lane] = s;
  __syncthreads();
  if (wv == 0 && c < 2 * H) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += lds[i][lane];
    if (c < H) {
      if (dw) dw[c] = (WT)s;
    } else if (db) {
      db[c - H] = (WT)s;
    }
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The longest rows kept in registers: 2048 vectors of 16 bytes.
constexpr int64_t kMaxRegVecs = 2048;

int64_t row_vecs(int64_t H, int dtype) { return ceil_div(H, dtype == FLCE_DTYPE_BF16 ? 8 : 4); }

// Work-groups for `sets` of rows, at most `most`: as few as leave every one
// the same number of steps.
int64_t even_grid(int64_t sets, int64_t most) {
  if (sets <= most) return sets;
  return ceil_div(sets, ceil_div(sets, most));
}

// Groups of rows that ln_bwd_kernel (or ln_param_grad_kernel) sums dw and db
// over, one partial each.
int64_t bwd_groups(int64_t M, int64_t H, int dtype) {
  const int64_t v = row_vecs(H, dtype);
  if (v <= 64) return even_grid(ceil_div(M, 4), 1024);
  if (v <= 128) return even_grid(ceil_div(M, 4), 512);
  if (v <= 256) return even_grid(ceil_div(M, 4), 256);
  if (v <= 1024) return even_grid(M, 512);
  if (v <= kMaxRegVecs) return even_grid(M, 256);
  return M < 64 ? M : 64;
}

// Threads, vectors per thread and resident work-groups by the row's length in
// vectors of 16 bytes, as measured on 134 MB of bf16 rows with fp32 parameters
// (kernel alone, TB/s of rows read and written; next best shape in brackets; a
// plain copy reaches 5.3; H = 5003 is fp32, 82 MB):
//   H      512       1024      2048      4096      6656      5003      16384
//   fwd    4.9       5.1       5.1       5.0       4.3       4.3       4.0
//          [4.7]     [4.6]     [5.0]     [4.8]     [3.9]     [4.3]     [4.1, 1024 threads]
//   bwd    5.2       5.4       5.1       4.9       4.5       4.6       4.1
//          [4.8]     [4.8]     [4.9]     [4.9]     [4.3]     [4.1]     [3.0]
// What they lose to the copy is the wait between a row's last load and its
// first store, which the registers for more rows in flight would hide.  As it
// is, the bf16 forward shapes of three and four vectors spill 104 to 152 scalar
// registers (into vector ones) and <bf16, bf16, 256, 4> two vector registers
// to memory; asking the compiler for more resident waves spills more of those
// and costs more (fwd 4.3 to 2.4).
template <typename T, typename WT>
void launch_fwd(const LnFwdArgs& p, int dtype, hipStream_t st) {
  const int64_t v = row_vecs(p.H, dtype);
  auto grid = [&](int rows, int64_t most) { return (unsigned)even_grid(ceil_div(p.M, rows), most); };
  if (v <= 64) ln_fwd_kernel<T, WT, 64, 1, 4, 1><<<grid(4, 4096), 256, 0, st>>>(p);
  else if (v <= 128) ln_fwd_kernel<T, WT, 64, 2, 4, 1><<<grid(4, 1024), 256, 0, st>>>(p);
  else if (v <= 256) ln_fwd_kernel<T, WT, 64, 4, 4, 1><<<grid(4, 512), 256, 0, st>>>(p);
  else if (v <= 512) ln_fwd_kernel<T, WT, 128, 4, 1, 1><<<grid(1, 1536), 128, 0, st>>>(p);
  else if (v <= 1024) ln_fwd_kernel<T, WT, 256, 4, 1, 3><<<grid(1, 768), 256, 0, st>>>(p);
  else if (v <= 1536) ln_fwd_kernel<T, WT, 512, 3, 1, 1><<<grid(1, 512), 512, 0, st>>>(p);
  else if (v <= kMaxRegVecs) ln_fwd_kernel<T, WT, 512, 4, 1, 1><<<grid(1, 256), 512, 0, st>>>(p);
  else ln_fwd_wide_kernel<T, WT><<<grid(1, 65536), kWide, 0, st>>>(p);
}

template <typename T, typename WT>
void launch_bwd(const LnBwdArgs& p, int dtype, hipStream_t st) {
  const int64_t v = row_vecs(p.H, dtype);
  const unsigned g = (unsigned)bwd_groups(p.M, p.H, dtype);
  if (v <= 64) ln_bwd_kernel<T, WT, 64, 1, 4, 1><<<g, 256, 0, st>>>(p);
  else if (v <= 128) ln_bwd_kernel<T, WT, 64, 2, 4, 1><<<g, 256, 0, st>>>(p);
  else if (v <= 256) ln_bwd_kernel<T, WT, 64, 4, 4, 1><<<g, 256, 0, st>>>(p);
  else if (v <= 512) ln_bwd_kernel<T, WT, 256, 2, 1, 1><<<g, 256, 0, st>>>(p);
  else if (v <= 1024) ln_bwd_kernel<T, WT, 256, 4, 1, 2><<<g, 256, 0, st>>>(p);
  else if (v <= 1536) ln_bwd_kernel<T, WT, 512, 3, 1, 1><<<g, 512, 0, st>>>(p);
  else if (v <= kMaxRegVecs) ln_bwd_kernel<T, WT, 512, 4, 1, 1><<<g, 512, 0, st>>>(p);
  else {
    if (p.dx) ln_bwd_wide_kernel<T, WT><<<(unsigned)(p.M < 65536 ? p.M : 65536), kWide, 0, st>>>(p);
    if (p.partial) ln_param_grad_kernel<T><<<dim3((unsigned)ceil_div(p.H, 256), g), 256, 0, st>>>(p);
  }
}

bool dtype_ok(int d) { return d == FLCE_DTYPE_BF16 || d == FLCE_DTYPE_F32; }
uintptr_t size_of(int d) { return d == FLCE_DTYPE_BF16 ? 2 : 4; }
bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Sizes shared by both directions; rows of 1 to 2^21 elements.
int check_sizes(int64_t M, int64_t H, int dtype, int w_dtype) {
  if (!dtype_ok(dtype) || !dtype_ok(w_dtype) || M < 0 || H < 1) return FLCE_EINVAL;
  if (M >= (int64_t(1) << 31) || H > (int64_t(1) << 21)) return FLCE_EUNSUPPORTED;
  return FLCE_OK;
}

}  // namespace

}  // namespace flce

extern "C" int flce_layer_norm_fwd(const void* x, int64_t ld_x, const void* weight, const void* bias, int64_t M,
                                   int64_t H, float eps, void* y, int64_t ld_y, float* mean, float* rstd,
                                   hipStream_t stream, int dtype, int w_dtype) {
  using namespace flce;
  const int rc = check_sizes(M, H, dtype, w_dtype);
  if (rc != FLCE_OK) return rc;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return FLCE_EINVAL;
  const uintptr_t es = size_of(dtype), ws = size_of(w_dtype);
  if (!on(weight, ws) || !on(bias, ws) || !on(mean, 4) || !on(rstd, 4)) return FLCE_EINVAL;
  if (M == 0) return FLCE_OK;
  if (!x || !y || !on(x, es) || !on(y, es)) return FLCE_EINVAL;
  if (ld_x < 0 || (M > 1 && ld_y < H)) return FLCE_EINVAL;
  if (x == y && M > 1 && ld_x != ld_y) return FLCE_EINVAL;
  LnFwdArgs p{x, weight, bias, y, mean, rstd, M, ld_x, ld_y, (int)H, eps};
  ProfileScope ps(FLCE_KERNEL_LAYER_NORM, stream);
  if (dtype == FLCE_DTYPE_BF16)
    w_dtype == FLCE_DTYPE_BF16 ? launch_fwd<bf16, bf16>(p, dtype, stream) : launch_fwd<bf16, float>(p, dtype, stream);
  else
    w_dtype == FLCE_DTYPE_BF16 ? launch_fwd<float, bf16>(p, dtype, stream) : launch_fwd<float, float>(p, dtype, stream);
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}

extern "C" size_t flce_layer_norm_bwd_workspace_size(int64_t M, int64_t H, int dtype) {
  using namespace flce;
  if (check_sizes(M, H, dtype, dtype) != FLCE_OK) return 0;
  const int64_t g = bwd_groups(M, H, dtype);
  const size_t bytes = (size_t)(g < 1 ? 1 : g) * 2 * (size_t)H * 4;
  return (bytes + 255) & ~size_t(255);
}

extern "C" int flce_layer_norm_bwd(const void* grad_y, int64_t ld_gy, const void* x, int64_t ld_x,
                                   const void* weight, const float* mean, const float* rstd, int64_t M, int64_t H,
                                   void* grad_x, int64_t ld_gx, void* grad_weight, void* grad_bias,
                                   hipStream_t stream, int dtype, int w_dtype, void* workspace,
                                   size_t workspace_bytes) {
  using namespace flce;
  const int rc = check_sizes(M, H, dtype, w_dtype);
  if (rc != FLCE_OK) return rc;
  const uintptr_t es = size_of(dtype), ws = size_of(w_dtype);
  const bool params = grad_weight || grad_bias;
  if (M == 0 && !params) return FLCE_OK;
  if (!on(weight, ws) || !on(grad_weight, ws) || !on(grad_bias, ws)) return FLCE_EINVAL;
  if (M > 0) {
    if (!grad_y || !x || !mean || !rstd) return FLCE_EINVAL;
    if (!on(grad_y, es) || !on(x, es) || !on(grad_x, es) || !on(mean, 4) || !on(rstd, 4)) return FLCE_EINVAL;
    if (ld_gy < 0 || ld_x < 0 || (grad_x && M > 1 && ld_gx < H)) return FLCE_EINVAL;
    if (grad_x && (grad_x == grad_y || grad_x == x)) return FLCE_EINVAL;
  }
  if (params) {
    if (!workspace || !on(workspace, 256)) return FLCE_EINVAL;
    if (workspace_bytes < flce_layer_norm_bwd_workspace_size(M, H, dtype)) return FLCE_EWORKSPACE;
  }
  float* partial = params ? static_cast<float*>(workspace) : nullptr;
  if (M > 0 && (grad_x || params)) {
    LnBwdArgs p{grad_y, x, weight, mean, rstd, grad_x, partial, M, ld_gy, ld_x, ld_gx, (int)H};
    ProfileScope ps(FLCE_KERNEL_LAYER_NORM_BWD, stream);
    if (dtype == FLCE_DTYPE_BF16)
      w_dtype == FLCE_DTYPE_BF16 ? launch_bwd<bf16, bf16>(p, dtype, stream)
                                 : launch_bwd<bf16, float>(p, dtype, stream);
    else
      w_dtype == FLCE_DTYPE_BF16 ? launch_bwd<float, bf16>(p, dtype, stream)
                                 : launch_bwd<float, float>(p, dtype, stream);
  }
  if (params) {
    const int groups = M > 0 ? (int)bwd_groups(M, H, dtype) : 0;   // no rows: zero gradients
    const unsigned g = (unsigned)ceil_div(2 * H, 64);
    ProfileScope ps(FLCE_KERNEL_LAYER_NORM_REDUCE, stream);
    if (w_dtype == FLCE_DTYPE_BF16)
      ln_reduce_kernel<bf16><<<g, 1024, 0, stream>>>(partial, groups, (int)H, static_cast<bf16*>(grad_weight),
                                                     static_cast<bf16*>(grad_bias));
    else
      ln_reduce_kernel<float><<<g, 1024, 0, stream>>>(partial, groups, (int)H, static_cast<float*>(grad_weight),
                                                      static_cast<float*>(grad_bias));
  }
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}
