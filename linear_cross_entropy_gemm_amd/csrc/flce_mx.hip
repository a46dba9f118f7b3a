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

// 8 elements of a token's row from column k on, as they come from memory.
template <XKind kX> struct XVec;
template <> struct XVec<kXBf16> {
  u32x4 v;
  __device__ __forceinline__ void load(const MxArgs& p, int64_t n, int k) {
    v = __builtin_bit_cast(u32x4, load_row(static_cast<const bf16*>(p.x) + n * p.ldx, k, p.H));
  }
  __device__ __forceinline__ void clear() { v = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void parts(u32x4 (&out)[1]) const { out[0] = v; }
};
template <> struct XVec<kXF32> {
  f32x4 v[2];
  __device__ __forceinline__ void load(const MxArgs& p, int64_t n, int k) {
    const float* r = static_cast<const float*>(p.x) + n * p.ldx;
    v[0] = load_row(r, k, p.H);
    v[1] = load_row(r, k + 4, p.H);
  }
  __device__ __forceinline__ void clear() { v[0] = v[1] = f32x4{0, 0, 0, 0}; }
  // cut, not rounded: the rest is exact and no part passes the largest float
  __device__ __forceinline__ void parts(u32x4 (&out)[3]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[3] = {0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = v[i / 2][2 * (i & 1) + h];
        const bool special = !(__builtin_fabsf(x) < __builtin_inff());
        if (x != x) x = __builtin_nanf("");
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const uint32_t b = __builtin_bit_cast(uint32_t, x) & 0xFFFF0000u;
          w[q] |= h ? b : b >> 16;
          x = special ? 0.0f : x - __builtin_bit_cast(float, b);
        }
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) out[q][i] = w[q];
    }
  }
};
template <> struct XVec<kXMx8> {
  u32x2 v;
  uint32_t code;
  __device__ __forceinline__ void load(const MxArgs& p, int64_t n, int k) {
    typedef uint32_t mem __attribute__((ext_vector_type(2), aligned(1)));
    const uint8_t* r = static_cast<const uint8_t*>(p.x) + n * p.ldx;
    v = u32x2{0, 0};
    if (k + 8 <= p.H) {
      const mem m = *reinterpret_cast<const mem*>(r + k);
      v = u32x2{m[0], m[1]};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < p.H) v[e / 4] |= (uint32_t)r[k + e] << 8 * (e % 4);
    }
    code = k < p.H ? p.xs[n * p.ldxs + k / kMxBlock] : 0u;
  }
  __device__ __forceinline__ void clear() { v = u32x2{0, 0}; code = 0; }
  __device__ __forceinline__ void parts(u32x4 (&out)[1]) const {
    const float s = __builtin_bit_cast(float, code << 23);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bf16x2 b = q & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[q / 2], s, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[q / 2], s, false);
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

// kRt tiles of 16 rows a wave, kNt tiles of 16 tokens, chunks of kSt steps.
// The tokens' chunk is double buffered in LDS (one barrier a chunk); a wave's
// weights of the next chunk are requested as soon as their registers are free.
template <XKind kX, int kRt, int kNt, int kSt, typename OT>
__global__ __launch_bounds__(kThreads) void mx_logits_kernel(MxArgs p) {
  constexpr int kParts = kX == kXF32 ? 3 : 1;
  constexpr int kVecs = kSt * 16;                            // vectors of 8 columns in a chunk
  constexpr int kItems = kNt * 16 * kVecs / kThreads;        // of them, per thread
  __shared__ u32x4 frag[2][kParts][kNt][kSt * 4][64];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.y * (16 * kNt);
  const int64_t v0 = ((int64_t)blockIdx.x * 4 + wave) * (16 * kRt);
  const uint8_t *wp[kRt], *sp[kRt];
#pragma unroll
  for (int i = 0; i < kRt; ++i) {
    const int64_t v = v0 + i * 16 + r, at = v < p.V ? v : p.V - 1;
    wp[i] = p.w + at * p.steps * 64 + g * 16;
    sp[i] = p.ws + at * p.steps * 4 + g;
  }
  u32x4 w[kSt][kRt];
  uint32_t sc[kSt][kRt];
  auto load_w = [&](int s, int step) {
    const int at = step < p.steps ? step : p.steps - 1;
#pragma unroll
    for (int i = 0; i < kRt; ++i) {
      w[s][i] = *reinterpret_cast<const u32x4*>(wp[i] + at * 64);
      sc[s][i] = sp[i][at * 4];
    }
  };
  XVec<kX> xv[kItems];
  auto load_x = [&](int step0) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int idx = t + i * kThreads, kv = idx % kVecs;
      const int64_t n = n0 + idx / kVecs;
      const int k = step0 * kStep + kv * 8;
      if (n < p.N && k < p.H) xv[i].load(p, n, k);
      else xv[i].clear();
    }
  };
  auto stage_x = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int idx = t + i * kThreads, kv = idx % kVecs, n = idx / kVecs;
      // vector kv: step kv / 16, lane group kv / 4 % 4, dword kv % 4 of its block
      u32x4 parts[kParts];
      xv[i].parts(parts);
#pragma unroll
      for (int q = 0; q < kParts; ++q)
        frag[buf][q][n / 16][kv / 16 * 4 + kv % 4][kv / 4 % 4 * 16 + n % 16] = parts[q];
    }
  };
  load_x(0);
#pragma unroll
  for (int s = 0; s < kSt; ++s) load_w(s, s);
  stage_x(0);
  f32x4 acc[kRt][kNt];
#pragma unroll
  for (int i = 0; i < kRt; ++i)
#pragma unroll
    for (int j = 0; j < kNt; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  __syncthreads();
  int buf = 0;
  for (int c = 0; c < p.steps; c += kSt, buf ^= 1) {
    const bool more = c + kSt < p.steps;
    if (more) load_x(c + kSt);
#pragma unroll
    for (int s = 0; s < kSt; ++s) {
      if (c + s < p.steps) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf16x8v a[kRt];
#pragma unroll
          for (int i = 0; i < kRt; ++i) a[i] = weights8(w[s][i][j], __builtin_bit_cast(float, sc[s][i] << 23));
#pragma unroll
          for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int n = 0; n < kNt; ++n) {
              const bf16x8v b = __builtin_bit_cast(bf16x8v, frag[buf][q][n][s * 4 + j][lane]);
#pragma unroll
              for (int i = 0; i < kRt; ++i)
                acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b, acc[i][n], 0, 0, 0);
            }
        }
      }
      if (more) load_w(s, c + kSt + s);
    }
    if (more) stage_x(buf ^ 1);
    __syncthreads();
  }
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
      store_logits(static_cast<OT*>(p.z) + tok * p.ldz + v, p.V - v, z);
    }
  }
}

template <XKind kX, typename OT>
void launch_logits(const MxArgs& p, hipStream_t st) {
  auto grid = [&](int rt, int nt) {
    return dim3((unsigned)ceil_div(p.V, 64 * rt), (unsigned)ceil_div(p.N, 16 * nt));
  };
  if (p.N <= 16)
    mx_logits_kernel<kX, 2, 1, 2, OT><<<grid(2, 1), kThreads, 0, st>>>(p);
  else if (p.N <= 32)
    mx_logits_kernel<kX, 2, 2, 2, OT><<<grid(2, 2), kThreads, 0, st>>>(p);
  else
    mx_logits_kernel<kX, 2, 4, 1, OT><<<grid(2, 4), kThreads, 0, st>>>(p);
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
           (int)ceil_div(H, kStep), softcap_T > 0.0f ? softcap_T : 0.0f, multiplier};
  ProfileScope ps(FLCE_KERNEL_LOGITS_MX, stream);
  if (dtype == FLCE_DTYPE_BF16) {
    if (mx8) launch_logits<kXMx8, bf16>(p, stream);
    else if (x_dtype == FLCE_DTYPE_BF16) launch_logits<kXBf16, bf16>(p, stream);
    else launch_logits<kXF32, bf16>(p, stream);
  } else {
    if (mx8) launch_logits<kXMx8, float>(p, stream);
    else if (x_dtype == FLCE_DTYPE_BF16) launch_logits<kXBf16, float>(p, stream);
    else launch_logits<kXF32, float>(p, stream);
  }
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}
