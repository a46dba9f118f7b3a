// RMS norm over the last dimension with the residual's addition: forward
// (flce_rms_norm_fwd), forward with an 8-bit output (flce_rms_norm_mx) and
// backward (flce_rms_norm_bwd).  Row x of H values, residual r, weight w:
//
//   s = x + r, rounded to the stream's type (it is what the next block reads)
//   rstd = 1 / sqrt(avg s^2 + eps),  y = s rstd (w + offset)
//   xh = s rstd,  g = dy (w + offset)
//   dx = rstd (g - xh avg(g xh)) + ds,  dw = sum over rows of dy xh
//
//   rms_fwd_kernel   the row stays in registers: x and r read once, s and y
//                    written once
//   rms_bwd_kernel   the rows s, dy and ds stay in registers; each thread keeps
//                    dw of its columns over all rows of its group
//   rms_*_wide_kernel rows too long for registers: two passes over a row
//   rms_param_grad_kernel  dw of wide rows, by columns
//   rms_reduce_kernel sum of the groups' dw in a fixed order
//
// What bounds them is memory: 8192 x 6656 bf16 with a residual 66 us forward (436
// MB, 6.5 TB/s), 82 backward with the stream's gradient (78 and 81 among calls on
// other data, which find nothing in the caches); 8192 x 7168 to 8 bits 68 (413
// MB); 4099 x 5003 fp32 backward, rows at odd addresses, 47 (246 MB).  One row of
// 6656 takes 3.3, its call through the binding 12.
//
// 8 bits: a block of 32 elements of y shares a scale, the least power of two
// s with max|y| / s <= 448 (the largest E4M3 value), from the bits of the
// maximum; y goes from fp32 to E4M3 in one rounding.
#include <cmath>

#include "flce_internal.hpp"
#include "mx_ops.hpp"
#include "row_ops.hpp"

namespace flce {

namespace {

// Sums and products are fp32; s, y and the gradients are rounded to their
// storage dtype once.
struct RmsFwdArgs {
  const void* x;
  const void* residual;   // null: none
  const void* weight;     // null: 1 (the offset is not added)
  void* sum;              // s (with a residual)
  void* y;
  uint8_t* scales;        // 8-bit output: y holds E4M3
  float* rstd;            // may be null
  int64_t M, ldx, ldr, lds, ldy, ldsc;   // strides in elements
  int H;
  float eps, offset;
  int past;               // see past_caches
};

struct RmsBwdArgs {
  const void* dy;
  const void* s;
  const void* ds;         // null: none
  const void* weight;
  const float* rstd;
  void* dx;               // null: not needed
  float* partial;         // [groups][H]; null: not needed
  int64_t M, ldy, lds, ldd, ldx;
  int H;
  float offset;
  int past;
};

// Rows that pass through the caches before anything can read them again: of a
// call that moves more than the last-level cache's 256 MB.  Stored as such
// they leave it to the loads: 8192 x 6656 bf16 forward with a residual takes 67
// us, 82 without (436 MB; a loop that only copies two arrays to two others 82);
// below the border there is no difference (268 MB: 44 and 45), and the next
// kernel finds the rows in the cache.
inline bool past_caches(int64_t bytes) { return bytes > int64_t(256) << 20; }
template <typename T>
__device__ __forceinline__ void put_vec(T* p, int64_t col, int64_t n, const typename RowVec<T>::type& v, bool past) {
  if (past && col + RowVec<T>::E <= n)
    __builtin_nontemporal_store(v, reinterpret_cast<typename RowVec<T>::mem*>(p + col));
  else
    store_row(p, col, n, v);
}

// A vector that is converted again at its next use: the compiler holds the
// fp32 values, twice the registers, over a barrier otherwise.
template <typename V>
__device__ __forceinline__ void hold_packed(V& v) {
  u32x4 x = __builtin_bit_cast(u32x4, v);
  asm volatile("" : "+v"(x));
  v = __builtin_bit_cast(V, x);
}

template <typename WT, int E>
__device__ __forceinline__ void load_weight(float (&out)[E], const void* p, int col, int H, float offset) {
  load_param<WT>(out, p, col, H, 1.0f);
  if (p) {
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] += offset;
  }
}

// One vector of y: in the storage dtype, or as E4M3 under its block's scale.
// kLanes neighbouring lanes hold a block, and every lane of the wave is active.
template <typename T, bool kMx8>
__device__ __forceinline__ void put_row(const RmsFwdArgs& p, int64_t row, int col, const float (&y)[RowVec<T>::E]) {
  constexpr int E = RowVec<T>::E;
  if constexpr (kMx8) {
    const uint32_t code = mx8_code(block_max_bits<E>(y));
    uint8_t* out = static_cast<uint8_t*>(p.y) + row * p.ldy;
    store_e4m3<E>(out, col, p.H, y, code);
    if (col % 32 == 0 && col < p.H) p.scales[row * p.ldsc + col / 32] = (uint8_t)code;
  } else {
    typename RowVec<T>::type o;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = (T)y[e];
    put_vec(static_cast<T*>(p.y) + row * p.ldy, col, p.H, o, p.past);
  }
}

template <typename T, bool kRes>
__device__ __forceinline__ void add_residual(typename RowVec<T>::type& x, const typename RowVec<T>::type& r) {
  if constexpr (kRes) {
#pragma unroll
    for (int e = 0; e < RowVec<T>::E; ++e) x[e] = (T)(to_f32(x[e]) + to_f32(r[e]));
  }
}

// kRow threads hold a row in kVec vectors each; a work-group holds kRows rows
// (more than one only where a row is one wave) and walks over the rows in
// steps of the grid, the next row's loads issued before the current row's sum.
template <typename T, typename WT, int kRow, int kVec, int kRows, bool kRes, bool kMx8>
__global__ __launch_bounds__(kRow* kRows) void rms_fwd_kernel(RmsFwdArgs p) {
  static_assert(kRow == 64 || kRows == 1, "a work-group barrier must see one row");
  constexpr int E = RowVec<T>::E;
  typedef typename RowVec<T>::type vec_t;
  __shared__ SumLds<1> lds;
  int buf = 0;
  const int t = threadIdx.x % kRow;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kRow;
  if (row >= p.M) return;   // whole waves (kRow = 64) or the whole work-group
  struct Rows {
    vec_t x[kVec], r[kRes ? kVec : 1];
  } cur, nxt;
  auto load = [&](Rows& to, int64_t from) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      to.x[i] = load_clamped(static_cast<const T*>(p.x) + from * p.ldx, (t + i * kRow) * E, p.H);
      if constexpr (kRes)
        to.r[i] = load_clamped(static_cast<const T*>(p.residual) + from * p.ldr, (t + i * kRow) * E, p.H);
    }
  };
  load(cur, row);
  float w[kVec][E];
#pragma unroll
  for (int i = 0; i < kVec; ++i) load_weight<WT>(w[i], p.weight, (t + i * kRow) * E, p.H, p.offset);
  const float inv = 1.0f / (float)p.H;
  for (; row < p.M; row += step) {
    if (row + step < p.M) load(nxt, row + step);
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int col = (t + i * kRow) * E;
      if constexpr (kRes) add_residual<T, kRes>(cur.x[i], cur.r[i]);
      row_tail<T>(cur.x[i], col, p.H);
      if constexpr (kRes) put_vec(static_cast<T*>(p.sum) + row * p.lds, col, p.H, cur.x[i], p.past);
#pragma unroll
      for (int e = 0; e < E; ++e) q[0] = __builtin_fmaf(to_f32(cur.x[i][e]), to_f32(cur.x[i][e]), q[0]);
    }
    row_sums<kRow>(q, lds, buf);
    const float rstd = 1.0f / sqrtf(__builtin_fmaf(q[0], inv, p.eps));
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = (to_f32(cur.x[i][e]) * rstd) * w[i][e];
      put_row<T, kMx8>(p, row, (t + i * kRow) * E, y);
    }
    if (t == 0 && p.rstd) p.rstd[row] = rstd;
    cur = nxt;
  }
}

constexpr int kWide = 1024;

// Rows too long for registers: s and its squares, then y from s again (out of
// the caches; a thread reads back what it wrote itself).
template <typename T, typename WT, bool kRes, bool kMx8>
__global__ __launch_bounds__(kWide) void rms_fwd_wide_kernel(RmsFwdArgs p) {
  constexpr int E = RowVec<T>::E;
  typedef typename RowVec<T>::type vec_t;
  __shared__ SumLds<1> lds;
  int buf = 0;
  const float inv = 1.0f / (float)p.H;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.ldx;
    T* sr = static_cast<T*>(p.sum) + row * p.lds;
    float q[1] = {0.0f};
    for (int c = threadIdx.x * E; c < p.H; c += kWide * E) {
      vec_t v = load_row(xr, c, p.H);
      if constexpr (kRes) {
        add_residual<T, kRes>(v, load_row(static_cast<const T*>(p.residual) + row * p.ldr, c, p.H));
        store_row(sr, c, p.H, v);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) q[0] = __builtin_fmaf(to_f32(v[e]), to_f32(v[e]), q[0]);
    }
    row_sums<kWide>(q, lds, buf);
    const float rstd = 1.0f / sqrtf(__builtin_fmaf(q[0], inv, p.eps));
    for (int base = 0; base < p.H; base += kWide * E) {   // (no lane leaves: blocks span lanes)
      const int c = base + threadIdx.x * E;
      const vec_t v = load_row(kRes ? sr : xr, c, p.H);
      float w[E], y[E];
      load_weight<WT>(w, p.weight, c, p.H, p.offset);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = c + e < p.H ? (to_f32(v[e]) * rstd) * w[e] : 0.0f;
      put_row<T, kMx8>(p, row, c, y);
    }
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
  }
}

template <typename T, typename WT, int kRow, int kVec, int kRows, bool kDs>
__global__ __launch_bounds__(kRow* kRows) void rms_bwd_kernel(RmsBwdArgs p) {
  static_assert(kRow == 64 || kRows == 1, "a work-group barrier must see one row");
  constexpr int E = RowVec<T>::E;
  typedef typename RowVec<T>::type vec_t;
  // The row in use and the next one, in turn (moving one to the other's place
  // waits for its loads: 8192 x 6656 bf16 takes 87 us then, 81 so; a third row
  // brings nothing).  Two vectors of bf16 each and 1024 threads: the next row has
  // no registers left (4096 x 16384: 107 us without it, 218 with it in scratch
  // memory).
  constexpr int kRing = E == 8 && kRow * kVec == kMaxRegVecs ? 1 : 2;
  __shared__ SumLds<1> lds;
  int buf = 0;
  const int t = threadIdx.x % kRow, sub = threadIdx.x / kRow;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + sub;
  struct Rows {
    vec_t s[kVec], d[kVec], a[kDs ? kVec : 1];
    float rstd;
  } ring[kRing];
  auto load = [&](Rows& to, int64_t from) {
    to.rstd = p.rstd[from];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      to.s[i] = load_clamped(static_cast<const T*>(p.s) + from * p.lds, (t + i * kRow) * E, p.H);
      to.d[i] = load_clamped(static_cast<const T*>(p.dy) + from * p.ldy, (t + i * kRow) * E, p.H);
      if constexpr (kDs) to.a[i] = load_clamped(static_cast<const T*>(p.ds) + from * p.ldd, (t + i * kRow) * E, p.H);
    }
  };
  if (row < p.M) load(ring[0], row);
  float w[kVec][E], dw[kVec][E];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    load_weight<WT>(w[i], p.weight, (t + i * kRow) * E, p.H, p.offset);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[i][e] = 0.0f;
  }
  const float inv = 1.0f / (float)p.H;
  auto use = [&](Rows& cur) {
    // columns past the row's end hold dy = 0 and add nothing to any sum
    float m[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      row_tail<T>(cur.s[i], (t + i * kRow) * E, p.H);
      row_tail<T>(cur.d[i], (t + i * kRow) * E, p.H);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = to_f32(cur.d[i][e]), xh = to_f32(cur.s[i][e]) * cur.rstd;
        m[0] = __builtin_fmaf(d * w[i][e], xh, m[0]);
        dw[i][e] = __builtin_fmaf(d, xh, dw[i][e]);
      }
    }
    if (p.dx) {
      row_sums<kRow>(m, lds, buf);
      const float m2 = m[0] * inv;
      T* gr = static_cast<T*>(p.dx) + row * p.ldx;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        vec_t o;
        hold_packed(cur.s[i]);
        hold_packed(cur.d[i]);
        if constexpr (kDs) row_tail<T>(cur.a[i], (t + i * kRow) * E, p.H);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float xh = to_f32(cur.s[i][e]) * cur.rstd;
          const float g = __builtin_fmaf(-xh, m2, to_f32(cur.d[i][e]) * w[i][e]);
          o[e] = (T)(kDs ? __builtin_fmaf(g, cur.rstd, to_f32(cur.a[i][e])) : g * cur.rstd);
        }
        put_vec(gr, (t + i * kRow) * E, p.H, o, p.past);
      }
    }
  };
  while (row < p.M) {
#pragma unroll
    for (int j = 0; j < kRing; ++j) {
      if (row >= p.M) break;
      if (kRing == 2 && row + step < p.M) load(ring[(j + 1) % kRing], row + step);
      use(ring[j]);
      if (kRing == 1 && row + step < p.M) load(ring[0], row + step);
      row += step;
    }
  }
  if (!p.partial) return;
  float* out = p.partial + (int64_t)blockIdx.x * p.H;
  if constexpr (kRows > 1) {
    // the work-group's waves add up their columns in order
    __shared__ float acc[kRows][kVec * E][kRow];
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[sub][i * E + e][t] = dw[i][e];
    __syncthreads();
    for (int c = threadIdx.x; c < p.H; c += kRow * kRows) {
      const int v = c / E, th = v % kRow, k = v / kRow * E + c % E;
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) s += acc[r][k][th];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int e = 0; e < E; e += 4)
        store_row<float>(out, (t + i * kRow) * E + e, p.H, f32x4{dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]});
  }
}

// dx of rows too long for registers: the sum, then the output.
template <typename T, typename WT>
__global__ __launch_bounds__(kWide) void rms_bwd_wide_kernel(RmsBwdArgs p) {
  constexpr int E = RowVec<T>::E;
  typedef typename RowVec<T>::type vec_t;
  __shared__ SumLds<1> lds;
  int buf = 0;
  const float inv = 1.0f / (float)p.H;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const T* sr = static_cast<const T*>(p.s) + row * p.lds;
    const T* dr = static_cast<const T*>(p.dy) + row * p.ldy;
    const float rstd = p.rstd[row];
    float m[1] = {0.0f};
    for (int c = threadIdx.x * E; c < p.H; c += kWide * E) {
      const vec_t s = load_row(sr, c, p.H), d = load_row(dr, c, p.H);
      float w[E];
      load_weight<WT>(w, p.weight, c, p.H, p.offset);
#pragma unroll
      for (int e = 0; e < E; ++e) m[0] = __builtin_fmaf(to_f32(d[e]) * w[e], to_f32(s[e]) * rstd, m[0]);
    }
    row_sums<kWide>(m, lds, buf);
    const float m2 = m[0] * inv;
    T* gr = static_cast<T*>(p.dx) + row * p.ldx;
    for (int c = threadIdx.x * E; c < p.H; c += kWide * E) {
      const vec_t s = load_row(sr, c, p.H), d = load_row(dr, c, p.H);
      vec_t a = s;
      if (p.ds) a = load_row(static_cast<const T*>(p.ds) + row * p.ldd, c, p.H);
      float w[E];
      load_weight<WT>(w, p.weight, c, p.H, p.offset);
      vec_t o;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float g = __builtin_fmaf(-(to_f32(s[e]) * rstd), m2, to_f32(d[e]) * w[e]);
        o[e] = (T)__builtin_fmaf(g, rstd, p.ds ? to_f32(a[e]) : 0.0f);
      }
      store_row(gr, c, p.H, o);
    }
  }
}

// dw of wide rows: thread = one column, group y takes every gridDim.y-th row.
template <typename T>
__global__ __launch_bounds__(256) void rms_param_grad_kernel(RmsBwdArgs p) {
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col >= p.H) return;
  float dw = 0.0f;
  for (int64_t row = blockIdx.y; row < p.M; row += gridDim.y) {
    const float d = to_f32(static_cast<const T*>(p.dy)[row * p.ldy + col]);
    dw = __builtin_fmaf(d, to_f32(static_cast<const T*>(p.s)[row * p.lds + col]) * p.rstd[row], dw);
  }
  p.partial[(int64_t)blockIdx.y * p.H + col] = dw;
}

// Sum of the groups' partials: 32 columns per work-group, 32 slices of the
// groups, joined in order.
template <typename WT>
__global__ __launch_bounds__(1024) void rms_reduce_kernel(const float* partial, int groups, int H, WT* dw) {
  __shared__ float lds[32][33];
  const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < H) {
    // eight loads under way, added in order
    int g = sl;
    for (; g + 7 * 32 < groups; g += 8 * 32) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = partial[(int64_t)(g + i * 32) * H + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; g < groups; g += 32) s += partial[(int64_t)g * H + c];
  }
  lds[sl][lane] = s;
  __syncthreads();
  if (sl == 0 && c < H) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += lds[i][lane];
    dw[c] = (WT)s;
  }
}

// Groups of rows that rms_bwd_kernel (or rms_param_grad_kernel) sums dw over,
// one partial each.
int64_t bwd_groups(int64_t M, int64_t H, int dtype) {
  const int64_t v = row_vecs(H, dtype == FLCE_DTYPE_BF16 ? 2 : 4);
  if (v <= 64) return even_grid(ceil_div(M, 4), 1024);
  if (v <= 128) return even_grid(ceil_div(M, 4), 512);
  if (v <= 512) return even_grid(M, 512);
  if (v <= kMaxRegVecs) return even_grid(M, 256);
  return M < 64 ? M : 64;
}

// Threads and vectors a row, as measured (us): 8192 x 6656 bf16 with a residual
// 67 by 512 x 2, 69 by 256 x 4, 66 by 1024 x 1 (with an 8-bit output, 8192 x
// 7168: 67, 72, 82); one row of 6656 3.3, 4.1, 3.2.
template <typename T, typename WT, bool kRes, bool kMx8>
void launch_fwd(const RmsFwdArgs& p, hipStream_t st) {
  const int64_t v = row_vecs(p.H, sizeof(T));
  auto grid = [&](int rows, int64_t most) { return (unsigned)even_grid(ceil_div(p.M, rows), most); };
  if (v <= 64) rms_fwd_kernel<T, WT, 64, 1, 4, kRes, kMx8><<<grid(4, 4096), 256, 0, st>>>(p);
  else if (v <= 128) rms_fwd_kernel<T, WT, 64, 2, 4, kRes, kMx8><<<grid(4, 1024), 256, 0, st>>>(p);
  else if (v <= 256) rms_fwd_kernel<T, WT, 64, 4, 4, kRes, kMx8><<<grid(4, 512), 256, 0, st>>>(p);
  else if (v <= 512) rms_fwd_kernel<T, WT, 128, 4, 1, kRes, kMx8><<<grid(1, 1536), 128, 0, st>>>(p);
  else if (v <= 1024) rms_fwd_kernel<T, WT, 512, 2, 1, kRes, kMx8><<<grid(1, 512), 512, 0, st>>>(p);
  else if (v <= kMaxRegVecs) rms_fwd_kernel<T, WT, 1024, 2, 1, kRes, kMx8><<<grid(1, 512), 1024, 0, st>>>(p);
  else rms_fwd_wide_kernel<T, WT, kRes, kMx8><<<grid(1, 65536), kWide, 0, st>>>(p);
}

// As measured (us, with rms_reduce_kernel, before a row's registers took turns):
// 8192 x 6656 bf16 with ds 85 by 1024 x 1 and 256 groups, 93 by 512 x 2 and 512,
// 111 by 256 x 4 and 512; 16384 x 2048 46 by 256 x 1 and 512 groups, 56 by four
// rows of 64 x 4; 4099 x 5003 fp32 48 by 1024 x 2, 55 by 512 x 4.  Now 82, 48, 47.
template <typename T, typename WT, bool kDs>
void launch_bwd(const RmsBwdArgs& p, int dtype, hipStream_t st) {
  const int64_t v = row_vecs(p.H, sizeof(T));
  const unsigned g = (unsigned)bwd_groups(p.M, p.H, dtype);
  if (v <= 64) rms_bwd_kernel<T, WT, 64, 1, 4, kDs><<<g, 256, 0, st>>>(p);
  else if (v <= 128) rms_bwd_kernel<T, WT, 64, 2, 4, kDs><<<g, 256, 0, st>>>(p);
  else if (v <= 256) rms_bwd_kernel<T, WT, 256, 1, 1, kDs><<<g, 256, 0, st>>>(p);
  else if (v <= 512) rms_bwd_kernel<T, WT, 256, 2, 1, kDs><<<g, 256, 0, st>>>(p);
  else if (v <= 1024) rms_bwd_kernel<T, WT, 1024, 1, 1, kDs><<<g, 1024, 0, st>>>(p);
  else if (v <= kMaxRegVecs) rms_bwd_kernel<T, WT, 1024, 2, 1, kDs><<<g, 1024, 0, st>>>(p);
  else {
    if (p.dx) rms_bwd_wide_kernel<T, WT><<<(unsigned)(p.M < 65536 ? p.M : 65536), kWide, 0, st>>>(p);
    if (p.partial) rms_param_grad_kernel<T><<<dim3((unsigned)ceil_div(p.H, 256), g), 256, 0, st>>>(p);
  }
}

bool dtype_ok(int d) { return d == FLCE_DTYPE_BF16 || d == FLCE_DTYPE_F32; }
uintptr_t size_of(int d) { return d == FLCE_DTYPE_BF16 ? 2 : 4; }
bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_sizes(int64_t M, int64_t H, int dtype, int w_dtype) {
  if (!dtype_ok(dtype) || !dtype_ok(w_dtype) || M < 0 || H < 1) return FLCE_EINVAL;
  if (M >= (int64_t(1) << 31) || H > (int64_t(1) << 21)) return FLCE_EUNSUPPORTED;
  return FLCE_OK;
}

// What both forward entries check and launch.
template <bool kMx8>
int rms_fwd(RmsFwdArgs p, int64_t H, hipStream_t stream, int dtype, int w_dtype) {
  const int rc = check_sizes(p.M, H, dtype, w_dtype);
  if (rc != FLCE_OK) return rc;
  if (!(p.eps > 0.0f) || !std::isfinite(p.eps) || !std::isfinite(p.offset)) return FLCE_EINVAL;
  const uintptr_t es = size_of(dtype), os = kMx8 ? 1 : es;
  if (!on(p.weight, size_of(w_dtype)) || !on(p.rstd, 4)) return FLCE_EINVAL;
  if (p.M == 0) return FLCE_OK;
  if (!p.x || !p.y || !on(p.x, es) || !on(p.y, os) || (kMx8 && !p.scales)) return FLCE_EINVAL;
  if ((p.residual == nullptr) != (p.sum == nullptr) || !on(p.residual, es) || !on(p.sum, es)) return FLCE_EINVAL;
  if (p.ldx < 0 || (p.residual && p.ldr < 0)) return FLCE_EINVAL;
  if (p.M > 1 && (p.ldy < H || (p.sum && p.lds < H) || (kMx8 && p.ldsc < ceil_div(H, 32)))) return FLCE_EINVAL;
  if (p.y == p.sum) return FLCE_EINVAL;
  // an output in the place of an input: row by row, in the same type
  const void* out[2] = {p.y, p.sum};
  const int64_t ld[2] = {p.ldy, p.lds};
  for (int i = 0; i < 2; ++i) {
    if (!out[i]) continue;
    const bool at_x = out[i] == p.x, at_r = out[i] == p.residual;
    if (kMx8 && i == 0 && (at_x || at_r)) return FLCE_EINVAL;
    if (p.M > 1 && ((at_x && ld[i] != p.ldx) || (at_r && ld[i] != p.ldr))) return FLCE_EINVAL;
  }
  p.past = past_caches(p.M * H * (int64_t)((p.residual ? 3 : 1) * es + os));
  ProfileScope ps(FLCE_KERNEL_RMS_NORM, stream);
  const bool b = dtype == FLCE_DTYPE_BF16, wb = w_dtype == FLCE_DTYPE_BF16;
  if (p.residual) {
    if (b) wb ? launch_fwd<bf16, bf16, true, kMx8>(p, stream) : launch_fwd<bf16, float, true, kMx8>(p, stream);
    else wb ? launch_fwd<float, bf16, true, kMx8>(p, stream) : launch_fwd<float, float, true, kMx8>(p, stream);
  } else {
    if (b) wb ? launch_fwd<bf16, bf16, false, kMx8>(p, stream) : launch_fwd<bf16, float, false, kMx8>(p, stream);
    else wb ? launch_fwd<float, bf16, false, kMx8>(p, stream) : launch_fwd<float, float, false, kMx8>(p, stream);
  }
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}

}  // namespace

}  // namespace flce

extern "C" int flce_rms_norm_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, const void* weight,
                                 float offset, int64_t M, int64_t H, float eps, void* y, int64_t ld_y, void* sum,
                                 int64_t ld_s, float* rstd, hipStream_t stream, int dtype, int w_dtype) {
  flce::RmsFwdArgs p{x, residual, weight, sum, y, nullptr, rstd, M, ld_x, ld_r, ld_s, ld_y, 0, (int)H, eps, offset, 0};
  return flce::rms_fwd<false>(p, H, stream, dtype, w_dtype);
}

extern "C" int flce_rms_norm_mx(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, const void* weight,
                                 float offset, int64_t M, int64_t H, float eps, void* y, int64_t ld_y, void* scales,
                                 int64_t ld_scales, void* sum, int64_t ld_s, float* rstd, hipStream_t stream,
                                 int dtype, int w_dtype) {
  flce::RmsFwdArgs p{x,    residual, weight, sum,  y,         static_cast<uint8_t*>(scales), rstd, M,
                     ld_x, ld_r,     ld_s,   ld_y, ld_scales, (int)H,                        eps,  offset, 0};
  return flce::rms_fwd<true>(p, H, stream, dtype, w_dtype);
}

extern "C" size_t flce_rms_norm_bwd_workspace_size(int64_t M, int64_t H, int dtype) {
  using namespace flce;
  if (check_sizes(M, H, dtype, dtype) != FLCE_OK) return 0;
  const int64_t g = bwd_groups(M, H, dtype);
  return ((size_t)(g < 1 ? 1 : g) * (size_t)H * 4 + 255) & ~size_t(255);
}

extern "C" int flce_rms_norm_bwd(const void* grad_y, int64_t ld_gy, const void* s, int64_t ld_s, const void* grad_s,
                                 int64_t ld_gs, const void* weight, float offset, const float* rstd, int64_t M,
                                 int64_t H, void* grad_x, int64_t ld_gx, void* grad_weight, hipStream_t stream,
                                 int dtype, int w_dtype, void* workspace, size_t workspace_bytes) {
  using namespace flce;
  const int rc = check_sizes(M, H, dtype, w_dtype);
  if (rc != FLCE_OK) return rc;
  const uintptr_t es = size_of(dtype), ws = size_of(w_dtype);
  if (!std::isfinite(offset)) return FLCE_EINVAL;
  if (M == 0 && !grad_weight) return FLCE_OK;
  if (!on(weight, ws) || !on(grad_weight, ws)) return FLCE_EINVAL;
  if (M > 0) {
    if (!grad_y || !s || !rstd) return FLCE_EINVAL;
    if (!on(grad_y, es) || !on(s, es) || !on(grad_s, es) || !on(grad_x, es) || !on(rstd, 4)) return FLCE_EINVAL;
    if (ld_gy < 0 || ld_s < 0 || (grad_s && ld_gs < 0) || (grad_x && M > 1 && ld_gx < H)) return FLCE_EINVAL;
    if (grad_x && (grad_x == grad_y || grad_x == s || grad_x == grad_s)) return FLCE_EINVAL;
  }
  if (grad_weight) {
    if (!workspace || !on(workspace, 256)) return FLCE_EINVAL;
    if (workspace_bytes < flce_rms_norm_bwd_workspace_size(M, H, dtype)) return FLCE_EWORKSPACE;
  }
  float* partial = grad_weight ? static_cast<float*>(workspace) : nullptr;
  if (M > 0 && (grad_x || grad_weight)) {
    RmsBwdArgs p{grad_y, s, grad_x ? grad_s : nullptr, weight, rstd, grad_x, partial, M, ld_gy, ld_s, ld_gs, ld_gx,
                 (int)H, offset, past_caches(M * H * (int64_t)(es * (2 + (grad_x ? 1 : 0) + (grad_s ? 1 : 0))))};
    ProfileScope ps(FLCE_KERNEL_RMS_NORM_BWD, stream);
    const bool b = dtype == FLCE_DTYPE_BF16, wb = w_dtype == FLCE_DTYPE_BF16;
    if (p.ds) {
      if (b) wb ? launch_bwd<bf16, bf16, true>(p, dtype, stream) : launch_bwd<bf16, float, true>(p, dtype, stream);
      else wb ? launch_bwd<float, bf16, true>(p, dtype, stream) : launch_bwd<float, float, true>(p, dtype, stream);
    } else {
      if (b) wb ? launch_bwd<bf16, bf16, false>(p, dtype, stream) : launch_bwd<bf16, float, false>(p, dtype, stream);
      else wb ? launch_bwd<float, bf16, false>(p, dtype, stream) : launch_bwd<float, float, false>(p, dtype, stream);
    }
  }
  if (grad_weight) {
    const int groups = M > 0 ? (int)bwd_groups(M, H, dtype) : 0;   // no rows: a zero gradient
    const unsigned g = (unsigned)ceil_div(H, 32);
    ProfileScope ps(FLCE_KERNEL_RMS_NORM_REDUCE, stream);
    if (w_dtype == FLCE_DTYPE_BF16)
      rms_reduce_kernel<bf16><<<g, 1024, 0, stream>>>(partial, groups, (int)H, static_cast<bf16*>(grad_weight));
    else
      rms_reduce_kernel<float><<<g, 1024, 0, stream>>>(partial, groups, (int)H, static_cast<float*>(grad_weight));
  }
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}
