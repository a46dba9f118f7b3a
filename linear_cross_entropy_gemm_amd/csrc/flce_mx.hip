// Products with 4-bit weights in the E2M1 block format (flce_logits_mx), and
// the packing of weights into it (flce_pack_mx).
//
//   z = cap(m x W^T),  W_vk = code_vk 2^(scale_v,k/32 - 127)
//
// A decoding step reads the whole projection for a few tokens: V Kp 17 / 32
// bytes (Kp: H padded to 128) where bf16 weights take 2 V H.  The weights pass
// through registers once, from memory straight into the form that the matrix
// instructions take: a lane's 16-byte load is one block of 32 along a row, its
// scale one byte, and the hardware's conversion makes pairs of bf16 of it
// (exactly: 2 significant bits times a power of two).  The order along K is
// free as long as both operands agree, so element j of lane group g in step k
// stands for column 128 k + 32 g + j on both sides.
//
// The tokens' rows are brought to bf16 fragments in LDS: bf16 as they are,
// E4M3 times its power of two (4 significant bits: exact), fp32 as three bf16
// parts of 8 bits each (exact: 24 bits).  Products are exact in fp32 and sums
// are fp32.
#include <cmath>

#include "flce_internal.hpp"
#include "mx_ops.hpp"

namespace flce {

namespace {

constexpr int kStep = 128;      // columns of one step: four lane groups of one block
constexpr int kThreads = 256;   // four waves, each with rows of its own

enum XKind { kXBf16, kXF32, kXMx8 };

struct MxArgs {
  const void* x;
  const uint8_t* xs;   // scales of 8-bit rows
  const uint8_t* w;    // [V][Kp / 2]
  const uint8_t* ws;   // [V][Kp / 32]
  void* z;
  int64_t ldx, ldxs, ldz;   // elements
  int64_t N, V;
  int H, steps;   // steps = Kp / 128
  float softcap, mult;
  int out_bf16;   // z in bf16, else fp32
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));

// 8 elements of a weight row (one dword of codes) as bf16.
__device__ __forceinline__ bf16x8v weights8(uint32_t codes, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 8 values as kParts bf16 parts each (one is enough for what has 8 bits).
// Cut, not rounded: the rest is exact and no part passes the largest float.
template <int kParts>
__device__ __forceinline__ void cut_parts(const float (&v)[8], u32x4 (&out)[kParts]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[kParts] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x = v[2 * i + h];
      const bool special = !(__builtin_fabsf(x) < __builtin_inff());
      if (x != x) x = __builtin_nanf("");
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
        const uint32_t b = __builtin_bit_cast(uint32_t, x) & 0xFFFF0000u;
        w[q] |= h ? b : b >> 16;
        x = special ? 0.0f : x - __builtin_bit_cast(float, b);
      }
    }
#pragma unroll
    for (int q = 0; q < kParts; ++q) out[q][i] = w[q];
  }
}

// 8 elements of a token's row from column k on, as they come from memory
// (load: rows of at least 8, k anything: what lies past the row's end is read
// from inside it and put right by parts(), so that no load waits on a branch),
// and as bf16 parts.
template <XKind kX> struct XVec;
template <> struct XVec<kXBf16> {
  typename RowVec<bf16>::type v;
  __device__ __forceinline__ void load(const MxArgs& p, int64_t n, int k) {
    v = load_clamped_vec(static_cast<const bf16*>(p.x) + n * p.ldx, k, p.H);
  }
  __device__ __forceinline__ void parts(u32x4 (&out)[1], int k, int H) {
    row_tail<bf16>(v, k, H);
    out[0] = __builtin_bit_cast(u32x4, v);
  }
};
template <> struct XVec<kXF32> {
  f32x4 v[2];
  __device__ __forceinline__ void load(const MxArgs& p, int64_t n, int k) {
    const float* r = static_cast<const float*>(p.x) + n * p.ldx;
    v[0] = load_clamped_vec(r, k, p.H);
    v[1] = load_clamped_vec(r, k + 4, p.H);
  }
  __device__ __forceinline__ void parts(u32x4 (&out)[3], int k, int H) {
    row_tail<float>(v[0], k, H);
    row_tail<float>(v[1], k + 4, H);
    const float x[8] = {v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]};
    cut_parts(x, out);
  }
};
template <> struct XVec<kXMx8> {
  u32x2 v;
  uint32_t code;
  __device__ __forceinline__ void load(const MxArgs& p, int64_t n, int k) {
    typedef uint32_t mem __attribute__((ext_vector_type(2), aligned(1)));
    const int at = k + 8 <= p.H ? k : p.H - 8, block = k < p.H ? k / kMxBlock : 0;
    const mem m = *reinterpret_cast<const mem*>(static_cast<const uint8_t*>(p.x) + n * p.ldx + at);
    v = u32x2{m[0], m[1]};
    code = p.xs[n * p.ldxs + block];
  }
  __device__ __forceinline__ void parts(u32x4 (&out)[1], int k, int H) {
    const int over = k + 8 - H;
    u64 x = (u64)v[1] << 32 | v[0];
    if (over > 0) x = over >= 8 ? 0 : x >> 8 * over;
    // (past the row's end the scale is 1: what is there must not turn into NaN)
    const float s = __builtin_bit_cast(float, (k < H ? code : 127u) << 23);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t half = (uint32_t)(x >> 32 * (q / 2));
      const bf16x2 b = q & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(half, s, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(half, s, false);
      out[0][q] = __builtin_bit_cast(uint32_t, b);
    }
  }
};

template <typename T>
__device__ __forceinline__ void store_logits(T* p, int64_t left, const float (&v)[4]) {
  typedef T mem __attribute__((ext_vector_type(4), aligned(sizeof(T))));
  if (left >= 4) {
    *reinterpret_cast<mem*>(p) = mem{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < left) p[i] = (T)v[i];
  }
}

// A wave's tile of logits: lane (r, g) holds token r of each tile of 16 and
// four consecutive vocabulary entries of each.
template <int kRt, int kNt>
__device__ __forceinline__ void put_logits(const MxArgs& p, int64_t n0, int64_t v0, const f32x4 (&acc)[kRt][kNt]) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const bool capped = p.softcap > 0.0f;
  const CapSeries cap(p.mult, capped ? 1.0f / p.softcap : 0.0f, p.softcap);
#pragma unroll
  for (int n = 0; n < kNt; ++n) {
    const int64_t tok = n0 + n * 16 + r;
    if (tok >= p.N) continue;
#pragma unroll
    for (int i = 0; i < kRt; ++i) {
      const int64_t v = v0 + i * 16 + g * 4;
      if (v >= p.V) continue;
      float z[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = capped ? softcap_value(acc[i][n][e], cap) : acc[i][n][e] * p.mult;
      if (p.out_bf16) store_logits(static_cast<bf16*>(p.z) + tok * p.ldz + v, p.V - v, z);
      else store_logits(static_cast<float*>(p.z) + tok * p.ldz + v, p.V - v, z);
    }
  }
}

// A wave's weights on their way through its registers: kRt tiles of 16 rows,
// a chunk of four steps.  A row's scales come four steps (16 bytes) at a time:
// byte by byte the loads take longer than those of the codes (153 against 110
// us for 202048 rows of 6656).
template <int kRt>
struct WeightStream {
  const uint8_t *wp[kRt], *sp[kRt];
  u32x4 w[4][kRt], sc[kRt], sc_next[kRt];
  int steps, shift;

  __device__ __forceinline__ void start(const MxArgs& p, int64_t v0) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    steps = p.steps;
#pragma unroll
    for (int i = 0; i < kRt; ++i) {
      const int64_t v = v0 + i * 16 + r, at = v < p.V ? v : p.V - 1;
      wp[i] = p.w + at * p.steps * 64 + g * 16;
      sp[i] = p.ws + at * p.steps * 4;
    }
  }
  __device__ __forceinline__ void load(int s, int step) {
    const int at = step < steps ? step : steps - 1;
#pragma unroll
    for (int i = 0; i < kRt; ++i) w[s][i] = *reinterpret_cast<const u32x4*>(wp[i] + at * 64);
  }
  // the scales of steps c to c + 3; the last 16 bytes of the row where it ends
  // before (rows of four steps or more)
  __device__ __forceinline__ void load_scales(int c) {
    typedef uint32_t mem __attribute__((ext_vector_type(4), aligned(4)));
    const int at = c + 4 <= steps ? c : steps - 4;
#pragma unroll
    for (int i = 0; i < kRt; ++i) {
      const mem m = *reinterpret_cast<const mem*>(sp[i] + at * 4);
      sc_next[i] = u32x4{m[0], m[1], m[2], m[3]};
    }
  }
  __device__ __forceinline__ void take_scales(int c) {
    const int d = c + 4 <= steps ? 0 : c + 4 - steps;   // the same for every lane
#pragma unroll
    for (int i = 0; i < kRt; ++i) {
      u32x4 x = sc_next[i];
      if (d & 2) x = u32x4{x[2], x[3], 0, 0};
      if (d & 1) x = u32x4{x[1], x[2], x[3], 0};
      sc[i] = x;
    }
  }
  // eight columns of step s as bf16: dword j of the block
  __device__ __forceinline__ float scale(int s, int i) const {
    const int g = (threadIdx.x & 63) >> 4;
    return __builtin_bit_cast(float, (sc[i][s] >> 8 * g & 255u) << 23);
  }
};

constexpr int kMaxResident = 80 * 1024;   // bytes of LDS for the tokens' rows: two work-groups on a compute unit

// A token's row in LDS: its columns in order, padded by 16 bytes so that the
// 16 rows a wave reads at a time start in different banks.
__host__ __device__ constexpr int row_bytes(int columns) { return columns * 2 + 16; }

// Up to 16 tokens whose rows stay in LDS as a whole: they are brought there
// once, and then the weights stream through without a barrier.
template <XKind kX, int kRt>
__global__ __launch_bounds__(512) void mx_logits_resident_kernel(MxArgs p) {
  constexpr int kParts = kX == kXF32 ? 3 : 1;
  extern __shared__ __align__(16) uint8_t rows[];   // [parts][N][row]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t v0 = ((int64_t)blockIdx.x * 8 + wave) * (16 * kRt);
  WeightStream<kRt> ws;
  ws.start(p, v0);
#pragma unroll
  for (int s = 0; s < 4; ++s) ws.load(s, s);
  ws.load_scales(0);
  const int stride = row_bytes(p.steps * kStep), vecs = p.steps * 16;
  const int part = (int)p.N * stride;
  for (int n = 0; n < p.N; ++n)
    for (int kv = threadIdx.x; kv < vecs; kv += 512) {
      XVec<kX> x;
      u32x4 parts[kParts];
      x.load(p, n, kv * 8);
      x.parts(parts, kv * 8, p.H);
#pragma unroll
      for (int q = 0; q < kParts; ++q) *reinterpret_cast<u32x4*>(rows + q * part + n * stride + kv * 16) = parts[q];
    }
  __syncthreads();
  ws.take_scales(0);
  const uint8_t* mine = rows + (r < p.N ? r : p.N - 1) * stride + g * 64;
  f32x4 acc[kRt][1];
#pragma unroll
  for (int i = 0; i < kRt; ++i) acc[i][0] = f32x4{0, 0, 0, 0};
  for (int c = 0; c < p.steps; c += 4) {
    ws.load_scales(c + 4);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (c + s < p.steps) {
        float sc[kRt];
#pragma unroll
        for (int i = 0; i < kRt; ++i) sc[i] = ws.scale(s, i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf16x8v b[kParts];
#pragma unroll
          for (int q = 0; q < kParts; ++q)
            b[q] = *reinterpret_cast<const bf16x8v*>(mine + q * part + (c + s) * 256 + j * 16);
#pragma unroll
          for (int i = 0; i < kRt; ++i) {
            const bf16x8v a = weights8(ws.w[s][i][j], sc[i]);
#pragma unroll
            for (int q = 0; q < kParts; ++q)
              acc[i][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[q], acc[i][0], 0, 0, 0);
          }
        }
      }
      ws.load(s, c + 4 + s);
    }
    ws.take_scales(c + 4);
  }
  put_logits<kRt, 1>(p, 0, v0, acc);
}

// Any number of tokens, kNt tiles of 16 a work-group: their rows pass through
// LDS in chunks of kSt steps, double buffered, one barrier a chunk.
template <XKind kX, int kRt, int kNt, int kSt>
__global__ __launch_bounds__(kThreads) void mx_logits_kernel(MxArgs p) {
  constexpr int kParts = kX == kXF32 ? 3 : 1;
  constexpr int kVecs = kSt * 16;                            // vectors of 8 columns in a chunk
  constexpr int kItems = kNt * 16 * kVecs / kThreads;        // of them, per thread
  constexpr int kStride = row_bytes(kSt * kStep);
  __shared__ __align__(16) uint8_t rows[2][kParts][kNt * 16][kStride];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.y * (16 * kNt);
  const int64_t v0 = ((int64_t)blockIdx.x * 4 + wave) * (16 * kRt);
  WeightStream<kRt> ws;
  ws.start(p, v0);
  XVec<kX> xv[kItems];
  auto load_x = [&](int step0) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int idx = t + i * kThreads;
      const int64_t n = n0 + idx / kVecs;
      xv[i].load(p, n < p.N ? n : p.N - 1, step0 * kStep + idx % kVecs * 8);
    }
  };
  auto stage_x = [&](int buf, int step0) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int idx = t + i * kThreads;
      u32x4 parts[kParts];
      xv[i].parts(parts, step0 * kStep + idx % kVecs * 8, p.H);
#pragma unroll
      for (int q = 0; q < kParts; ++q)
        *reinterpret_cast<u32x4*>(&rows[buf][q][idx / kVecs][idx % kVecs * 16]) = parts[q];
    }
  };
  load_x(0);
#pragma unroll
  for (int s = 0; s < 4; ++s) ws.load(s, s);
  ws.load_scales(0);
  stage_x(0, 0);
  f32x4 acc[kRt][kNt];
#pragma unroll
  for (int i = 0; i < kRt; ++i)
#pragma unroll
    for (int j = 0; j < kNt; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  ws.take_scales(0);
  __syncthreads();
  int buf = 0;
  for (int c = 0; c < p.steps; c += 4) {
    ws.load_scales(c + 4);
#pragma unroll
    for (int h = 0; h < 4; h += kSt, buf ^= 1) {
      load_x(c + h + kSt);
#pragma unroll
      for (int s = h; s < h + kSt; ++s) {
        if (c + s < p.steps) {
          float sc[kRt];
#pragma unroll
          for (int i = 0; i < kRt; ++i) sc[i] = ws.scale(s, i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            bf16x8v a[kRt];
#pragma unroll
            for (int i = 0; i < kRt; ++i) a[i] = weights8(ws.w[s][i][j], sc[i]);
#pragma unroll
            for (int q = 0; q < kParts; ++q)
#pragma unroll
              for (int n = 0; n < kNt; ++n) {
                const bf16x8v b = *reinterpret_cast<const bf16x8v*>(&rows[buf][q][n * 16 + r][(s - h) * 256 + g * 64 + j * 16]);
#pragma unroll
                for (int i = 0; i < kRt; ++i)
                  acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b, acc[i][n], 0, 0, 0);
              }
          }
        }
        ws.load(s, c + 4 + s);
      }
      stage_x(buf ^ 1, c + h + kSt);
      __syncthreads();
    }
    ws.take_scales(c + 4);
  }
  put_logits<kRt, kNt>(p, n0, v0, acc);
}

// A row of fewer than 8 elements, as parts.
template <XKind kX, int kParts>
__device__ __forceinline__ void load_few(const MxArgs& p, int64_t n, int k, u32x4 (&out)[kParts]) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = 0.0f;
    if (k + e >= p.H) continue;
    const int64_t at = n * p.ldx + k + e;
    if (kX == kXBf16) x[e] = to_f32(static_cast<const bf16*>(p.x)[at]);
    else if (kX == kXF32) x[e] = static_cast<const float*>(p.x)[at];
    else x[e] = __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(p.x)[at], 0) * mx_scale(p.xs[n * p.ldxs]);
  }
  cut_parts(x, out);
}

// Rows of less than four steps: nothing to stream.  A wave has 16 vocabulary
// entries and 16 tokens and reads both from memory.
template <XKind kX>
__global__ __launch_bounds__(kThreads) void mx_logits_short_kernel(MxArgs p) {
  constexpr int kParts = kX == kXF32 ? 3 : 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t v0 = ((int64_t)blockIdx.x * 4 + wave) * 16, n0 = (int64_t)blockIdx.y * 16;
  const int64_t v = v0 + r < p.V ? v0 + r : p.V - 1, n = n0 + r < p.N ? n0 + r : p.N - 1;
  f32x4 acc[1][1] = {{{0, 0, 0, 0}}};
  for (int s = 0; s < p.steps; ++s) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p.w + (v * p.steps + s) * 64 + g * 16);
    const float scale = __builtin_bit_cast(float, (uint32_t)p.ws[(v * p.steps + s) * 4 + g] << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = s * kStep + g * 32 + j * 8;
      XVec<kX> x;
      u32x4 parts[kParts];
      if (p.H >= 8) {
        x.load(p, n, k);
        x.parts(parts, k, p.H);
      } else {
        load_few<kX>(p, n, k, parts);
      }
      const bf16x8v a = weights8(w[j], scale);
#pragma unroll
      for (int q = 0; q < kParts; ++q)
        acc[0][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8v, parts[q]), acc[0][0], 0, 0, 0);
    }
  }
  put_logits<1, 1>(p, n0, v0, acc);
}

template <XKind kX>
void launch_logits(const MxArgs& p, hipStream_t st) {
  constexpr int kParts = kX == kXF32 ? 3 : 1;
  auto grid = [&](int rows, int tokens) {
    return dim3((unsigned)ceil_div(p.V, rows), (unsigned)ceil_div(p.N, tokens));
  };
  if (p.steps < 4) {
    mx_logits_short_kernel<kX><<<grid(64, 16), kThreads, 0, st>>>(p);
    return;
  }
  const int64_t resident = p.N * kParts * row_bytes(p.steps * kStep);
  if (p.N <= 16 && resident <= kMaxResident)
    mx_logits_resident_kernel<kX, 2><<<grid(256, 16), 512, (size_t)resident, st>>>(p);
  else if (p.N <= 16)
    mx_logits_kernel<kX, 2, 1, 2><<<grid(128, 16), kThreads, 0, st>>>(p);
  else if (p.N <= 32)
    mx_logits_kernel<kX, 2, 2, 2><<<grid(128, 32), kThreads, 0, st>>>(p);
  else
    mx_logits_kernel<kX, 2, 4, 1><<<grid(128, 64), kThreads, 0, st>>>(p);
}

// Nearest E2M1 code, ties to the even one.
__device__ __forceinline__ uint32_t e2m1_code(float x) {
  const float a = __builtin_fabsf(x);
  const uint32_t c = (uint32_t)(a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) +
                     (a > 5.0f);
  return c | (x < 0.0f && c ? 8u : 0u);
}

// Eight columns per thread, four threads per block; a row has `vecs` of them,
// a multiple of 16.
template <typename T>
__global__ __launch_bounds__(256) void pack_mx_kernel(const T* W, int64_t ld, int64_t total, int H, int vecs,
                                                      uint32_t* packed, uint8_t* scales) {
  constexpr int E = RowVec<T>::E;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool in = i < total;   // no lane leaves: blocks span lanes
  const int64_t row = in ? i / vecs : 0;
  const int k = in ? (int)(i % vecs) * 8 : H;
  float w[8];
#pragma unroll
  for (int q = 0; q < 8 / E; ++q) {
    const typename RowVec<T>::type v = load_row(W + row * ld, k + q * E, H);
#pragma unroll
    for (int e = 0; e < E; ++e) w[q * E + e] = to_f32(v[e]);
  }
  const uint32_t code = mx4_code(block_max_bits<8>(w));
  if (!in) return;
  const float inv = mx_inverse(code);
  uint32_t out = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) out |= (code == 255 ? 0u : e2m1_code(w[e] * inv)) << (4 * e);
  packed[i] = out;
  if (k % kMxBlock == 0) scales[i / 4] = (uint8_t)code;
}

uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

}  // namespace

}  // namespace flce

extern "C" int flce_pack_mx(const void* W, int64_t ld_w, int64_t V, int64_t H, void* packed, void* scales,
                            hipStream_t stream, int dtype) {
  using namespace flce;
  if ((dtype != FLCE_DTYPE_BF16 && dtype != FLCE_DTYPE_F32) || V < 0 || H < 1) return FLCE_EINVAL;
  if (V > (int64_t(1) << 24) || H > (int64_t(1) << 21)) return FLCE_EUNSUPPORTED;
  const int64_t vecs = ceil_div(H, kStep) * (kStep / 8), total = V * vecs;
  if (total > (int64_t(1) << 31)) return FLCE_EUNSUPPORTED;   // a launch holds fewer than 2^32 threads
  if (V == 0) return FLCE_OK;
  if (!W || !packed || !scales || addr(W) % (dtype == FLCE_DTYPE_BF16 ? 2 : 4) || addr(packed) % 16) return FLCE_EINVAL;
  if (ld_w < 0) return FLCE_EINVAL;
  ProfileScope ps(FLCE_KERNEL_PACK_MX, stream);
  const unsigned g = (unsigned)ceil_div(total, 256);
  if (dtype == FLCE_DTYPE_BF16)
    pack_mx_kernel<bf16><<<g, 256, 0, stream>>>(static_cast<const bf16*>(W), ld_w, total, (int)H, (int)vecs,
                                                static_cast<uint32_t*>(packed), static_cast<uint8_t*>(scales));
  else
    pack_mx_kernel<float><<<g, 256, 0, stream>>>(static_cast<const float*>(W), ld_w, total, (int)H, (int)vecs,
                                                 static_cast<uint32_t*>(packed), static_cast<uint8_t*>(scales));
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}

extern "C" int flce_logits_mx(const void* x, int64_t ld_x, const void* x_scales, int64_t ld_xs, const void* packed,
                              const void* scales, int64_t N, int64_t H, int64_t V, float softcap_T, float multiplier,
                              void* logits, int64_t ld_logits, hipStream_t stream, int x_dtype, int dtype) {
  using namespace flce;
  if (x_dtype != FLCE_DTYPE_BF16 && x_dtype != FLCE_DTYPE_F32 && x_dtype != FLCE_DTYPE_MX8) return FLCE_EINVAL;
  if ((dtype != FLCE_DTYPE_BF16 && dtype != FLCE_DTYPE_F32) || N < 0 || H < 1 || V < 1) return FLCE_EINVAL;
  if (!std::isfinite(softcap_T) || !std::isfinite(multiplier)) return FLCE_EINVAL;
  if (softcap_T > 0.0f && (!std::isfinite(1.0f / softcap_T) || !std::isfinite(multiplier / softcap_T)))
    return FLCE_EINVAL;
  if (N > (int64_t(1) << 20) || V > (int64_t(1) << 24) || H > (int64_t(1) << 21)) return FLCE_EUNSUPPORTED;
  if (N == 0) return FLCE_OK;
  const bool mx8 = x_dtype == FLCE_DTYPE_MX8;
  const uintptr_t es = mx8 ? 1 : x_dtype == FLCE_DTYPE_BF16 ? 2 : 4, os = dtype == FLCE_DTYPE_BF16 ? 2 : 4;
  if (!x || !packed || !scales || !logits || (mx8 != (x_scales != nullptr))) return FLCE_EINVAL;
  if (addr(x) % es || addr(packed) % 16 || addr(logits) % os) return FLCE_EINVAL;
  if (ld_x < 0 || (mx8 && ld_xs < 0) || (N > 1 && ld_logits < V)) return FLCE_EINVAL;
  MxArgs p{x, static_cast<const uint8_t*>(x_scales), static_cast<const uint8_t*>(packed),
           static_cast<const uint8_t*>(scales), logits, ld_x, ld_xs, ld_logits, N, V, (int)H,
           (int)ceil_div(H, kStep), softcap_T > 0.0f ? softcap_T : 0.0f, multiplier, dtype == FLCE_DTYPE_BF16};
  ProfileScope ps(FLCE_KERNEL_LOGITS_MX, stream);
  if (mx8) launch_logits<kXMx8>(p, stream);
  else if (x_dtype == FLCE_DTYPE_BF16) launch_logits<kXBf16>(p, stream);
  else launch_logits<kXF32>(p, stream);
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}
