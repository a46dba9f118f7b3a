// Products with 4-bit weights in the E2M1 block format (flce_logits_mx), and
// the packing of weights into it (flce_pack_mx).
//
//   z = cap(m x W^T),  W_vk = code_vk 2^(scale_v,k/32 - 127)
//
// A decoding step reads the whole projection for a few tokens: V Kp 17 / 32
// bytes (Kp: H padded to 128) where bf16 weights take 2 V H.  The weights pass
// through registers once and are never converted: the scaled matrix
// instruction takes E2M1 rows with a scale for every 32 elements as they lie in
// memory, next to E4M3 rows with theirs.  So the tokens are brought to E4M3
// parts, each under the block's scale times a power of two: one for rows that are
// in 8 bits already, two for bf16 (8 significant bits), five for fp32, and for bf16
// where the logits are fp32.
//
// What the instruction keeps (measured with single products): it adds the 8
// products of columns 8 i to 8 i + 7 down to 2^-13 of the largest, the 16 sums
// and the accumulator down to 2^-23 of the largest, and cuts off the rest.  Where
// the tokens are 8-bit or bf16 a product's loss, at most 2^-13 of its group's
// largest, is a sixteenth of what half a step of that bf16 element stands for
// (2^-9).  An element above 2^-14 of its block's largest has exact bf16 parts, a
// smaller one to 2^-22 of that largest; sums of random rows end within 4e-6 of
// themselves, with a few columns 300 times the others within 1e-4.  Five parts are
// digits: whole numbers to 16 times the largest's exponent less 3, then base 32.
// Products of digits and E2M1 are whole numbers of halves to 96, which the
// instruction adds exactly; elements are held to 2^-24 of their block's largest,
// and sums of random rows end within 3e-7.
//
// (Conversion of the weights to bf16 pairs and plain bf16 products took 114 us
// of the vector and matrix units for 1 x 6656 x 202048, as long as the memory
// takes for the weights, and 180 together.)
#include <cmath>

#include "flce_internal.hpp"
#include "mx_ops.hpp"

namespace flce {

namespace {

// Loads that go straight to LDS: lane l's 16 (or 4) bytes at offset `at` of the
// buffer land at LDS address lds + 16 l (4 l); zeros past the buffer's end.
// Written as assembly so that the compiler does not make every later LDS read
// wait for them: the kernel waits by counts.
typedef uint32_t u32x4s __attribute__((ext_vector_type(4)));
constexpr uint32_t kPastBuffer = 0x80000000u;
__device__ __forceinline__ u32x4s buffer_of(const uint8_t* base, int64_t bytes) {   // the same in every lane
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return settled(u32x4s{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a),
                        (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) & 0xFFFFu,
                        (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)bytes), 0x00020000u});
}
__device__ __forceinline__ void dma16(const u32x4s& from, uint32_t lds, uint32_t at) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               : : "v"(at), "s"(from), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void dma4(const u32x4s& from, uint32_t lds, uint32_t at) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               : : "v"(at), "s"(from), "{m0}"(lds) : "memory");
}
// Waits until at most n of the wave's memory accesses are under way, and until
// none of its LDS accesses is; no access moves across either.
template <int n>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(n) : "memory");
}
// Work-group barrier behind which this wave's LDS accesses are done (its loads
// to LDS only as far as it waited for them).
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory"); }
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }
__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) {
  return (uint32_t)__builtin_amdgcn_readfirstlane(
      (uint32_t)reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint8_t*)p));
}

constexpr int kStep = 128;      // columns of one matrix instruction: four lane groups of one block
constexpr int64_t kMostRow = int64_t(1) << 21;   // bytes between rows that are read through a buffer's 32-bit offsets

typedef int i32x4v __attribute__((ext_vector_type(4)));
typedef int i32x8v __attribute__((ext_vector_type(8)));

struct MxArgs {
  // the tokens: raw rows (inline split), or parts [P][N][ldx] and codes [N][ldxs]
  const void* x;
  const uint8_t* xs;
  int64_t ldx, ldxs;   // elements, bytes
  const uint8_t* w;    // [V][Kp / 2]
  const uint8_t* ws;   // [V][Kp / 32]
  void* z;
  int64_t ldz;         // elements
  int64_t N, V;
  int H, steps;        // steps = Kp / 128
  float softcap, mult;
  int out_bf16;        // z in bf16, else fp32
};

// acc += A B^T over 128 columns: A 16 rows of E2M1 (lane (r, g): row r, block g),
// B 16 rows of E4M3 (lane (r, g): row r, columns 16 g to 16 g + 15 and 64 + 16 g
// to 64 + 16 g + 15), byte kByte of sa and sb the scale of block g of the lane's
// row.  The empty asm keeps the sums in accumulation registers and the operands
// alive past the instruction: the compiler may give the result the registers of
// its 4-bit operand otherwise, which the hardware still reads while it writes.
template <int kByte>
__device__ __forceinline__ void mx_mma(f32x4& acc, const u32x4& a, const i32x8v& b, uint32_t sa, uint32_t sb) {
  const i32x8v wide = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide, b, acc, 4, 0, kByte, (int)sa, kByte, (int)sb);
  asm("" : "+a"(acc) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mx_mma(int byte, f32x4& acc, const u32x4& a, const i32x8v& b, uint32_t sa,
                                       uint32_t sb) {
  if (byte == 0) mx_mma<0>(acc, a, b, sa, sb);   // (byte is a constant where this is used)
  else if (byte == 1) mx_mma<1>(acc, a, b, sa, sb);
  else if (byte == 2) mx_mma<2>(acc, a, b, sa, sb);
  else mx_mma<3>(acc, a, b, sa, sb);
}

// Parts of a token, and how far part q's code lies below the block's.  fp32 rows
// have five whose elements are whole numbers up to 16, digits of base 32 (see the
// top), kept in units down to 2^-9, E4M3's last: part q's unit is 2^-min(5 q, 9),
// and its code has only the rest to go.
constexpr int kDigits = 5;
template <int kParts>
__device__ __forceinline__ constexpr uint32_t part_down(int q) {
  return kParts == kDigits ? (5 * q > 9 ? 5 * q - 9 : 0) : 4 * q;
}

// Their steps are summed by themselves, smallest part first, and added to the
// sums so far by the vector unit, which rounds to nearest.  (Two parts and one
// would gain nothing: on constant operands 320 x 4096 x 128256 takes 283 us and 212
// that way where it takes 262 and 190.)
template <int kParts>
__device__ __forceinline__ f32x4 step_sums(const f32x4& acc) {
  return kParts == kDigits ? f32x4{0, 0, 0, 0} : acc;
}
template <int kParts>
__device__ __forceinline__ void add_step(f32x4& acc, const f32x4& sum) {
  acc = kParts == kDigits ? acc + sum : sum;
}

// Four steps' scales of a row (four bytes each) -> those of the lane's own
// block, a byte per step.
__device__ __forceinline__ uint32_t own_scales(const u32x4& x) {
  const uint32_t g = (threadIdx.x & 63) >> 4;
  const uint32_t lo = __builtin_amdgcn_perm(x[1], x[0], 0x0c0c0400u + g * 0x0101u);
  const uint32_t hi = __builtin_amdgcn_perm(x[3], x[2], 0x04000c0cu + g * 0x01010000u);
  return lo | hi;
}

// 8 values of a block, whose other values are with the other three lanes of an
// aligned group of four, as E4M3 parts; returns the block's code.  Codes below
// the last part's part_down are raised to it, so that no part's is negative.
template <int kParts>
__device__ __forceinline__ uint32_t split8(const float (&v)[8], u32x2 (&out)[kParts]) {
  const uint32_t bits = block_max_bits<8>(v);
  uint32_t code = kParts == kDigits ? bits >> 23 : mx8_code(bits);
  if (kParts == kDigits) code = code == 255 ? 255 : code < 3 ? 0 : code - 3;   // the largest: 8 to 16 units
  if (code < part_down<kParts>(kParts - 1)) code = part_down<kParts>(kParts - 1);
  const float inv = code == 255 ? 1.0f : mx_inverse(code);
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = code == 255 ? 0.0f : v[e] * inv;   // a block without a scale is NaN by its code
  // next to the largest float no part may round the sum up to 2^128
  const float top = code == 247 ? 240.0f : 448.0f;
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    float y[8];
    if constexpr (kParts == kDigits) {
      const float unit = 1.0f / (float)(1 << (5 * p < 9 ? 5 * p : 9));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = rintf(x[e]);
        y[e] = d * unit;
        x[e] = (x[e] - d) * 32.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __builtin_amdgcn_fmed3f(x[e], -top, top);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h], y[4 * h + 1], 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h + 2], y[4 * h + 3], w, true);
      out[p][h] = (uint32_t)w;
      if (kParts != kDigits && p + 1 < kParts) {
        x[4 * h] = (x[4 * h] - __builtin_amdgcn_cvt_f32_fp8(w, 0)) * 16.0f;
        x[4 * h + 1] = (x[4 * h + 1] - __builtin_amdgcn_cvt_f32_fp8(w, 1)) * 16.0f;
        x[4 * h + 2] = (x[4 * h + 2] - __builtin_amdgcn_cvt_f32_fp8(w, 2)) * 16.0f;
        x[4 * h + 3] = (x[4 * h + 3] - __builtin_amdgcn_cvt_f32_fp8(w, 3)) * 16.0f;
      }
    }
  }
  return code;
}

template <typename T>
__device__ __forceinline__ void load8(float (&v)[8], const T* row, int k, int H) {
  constexpr int E = RowVec<T>::E;
#pragma unroll
  for (int q = 0; q < 8 / E; ++q) {
    const typename RowVec<T>::type x = load_row(row, k + q * E, H);
#pragma unroll
    for (int e = 0; e < E; ++e) v[q * E + e] = to_f32(x[e]);
  }
}

// Parts and codes of rows that the products read from a workspace: one vector
// of 8 columns per thread, `vecs` (a multiple of 16) in a row.
template <typename T, int kParts>
__global__ __launch_bounds__(256) void mx_split_kernel(const T* x, int64_t ldx, int64_t N, int H, int vecs,
                                                       uint8_t* parts, int64_t ldp, uint8_t* codes, int64_t ldc) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= N * vecs) return;   // whole groups of 16 lanes
  const int64_t n = i / vecs;
  const int kv = (int)(i % vecs);
  float v[8];
  u32x2 out[kParts];
  load8(v, x + n * ldx, kv * 8, H);
  const uint32_t code = split8<kParts>(v, out);
#pragma unroll
  for (int p = 0; p < kParts; ++p) *reinterpret_cast<u32x2*>(parts + (p * N + n) * ldp + kv * 8) = out[p];
  if (kv % 4 == 0) codes[n * ldc + kv / 4] = (uint8_t)code;
}

// Rows in 8 bits, padded to whole steps.
__global__ __launch_bounds__(256) void mx_copy_kernel(const uint8_t* x, int64_t ldx, const uint8_t* xs, int64_t ldxs,
                                                      int64_t N, int H, int vecs, uint8_t* parts, int64_t ldp,
                                                      uint8_t* codes, int64_t ldc) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= N * vecs) return;
  const int64_t n = i / vecs;
  const int k = (int)(i % vecs) * 8;
  u32x2 v = {0, 0};
  if (k + 8 <= H) {
    typedef uint32_t mem __attribute__((ext_vector_type(2), aligned(1)));
    const mem m = *reinterpret_cast<const mem*>(x + n * ldx + k);
    v = u32x2{m[0], m[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e < H) v[e / 4] |= (uint32_t)x[n * ldx + k + e] << 8 * (e % 4);
  }
  *reinterpret_cast<u32x2*>(parts + n * ldp + k) = v;
  if (k % kMxBlock == 0) codes[n * ldc + k / kMxBlock] = k < H ? xs[n * ldxs + k / kMxBlock] : 127;
}

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

__device__ __forceinline__ i32x8v token_columns(const uint8_t* p) {
  const i32x4v a = *reinterpret_cast<const i32x4v*>(p), b = *reinterpret_cast<const i32x4v*>(p + 64);
  return i32x8v{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Bytes of a row of codes: whole groups of four steps.
__host__ __device__ constexpr int code_bytes(int steps) { return (steps + 3) / 4 * 16; }

// A token's part in LDS: its columns in order, padded by 16 bytes so that the
// 16 rows that a wave reads at a time start in different banks.
__host__ __device__ constexpr int part_bytes(int steps) { return steps * kStep + 16; }

// A wave's weights in LDS: a group of four steps (16 rows of 256 bytes) with its
// scales (16 rows of 16 bytes).
constexpr int kGroupBytes = 4096 + 256;

constexpr int kLdsMost = 160 * 1024;

// Up to 16 tokens that stay in LDS as a whole, brought there once; then the
// weights stream through every wave's own place without a barrier, tile after
// tile of 16 rows (tile blockIdx.x + gridDim.x (wave + waves i)): once a group is in
// registers the next one's loads are issued, and its products hide them together
// with the other waves'.
//
// The loads go straight to LDS, 16 lanes to 256 bytes of a row, four rows a
// load: straight to the lanes that need them (a lane a row, 64 different lines
// a load) the address units take as long as the memory.  Piece k (16 bytes) of
// row r lands at k ^ r, so that the 16 rows that a wave reads at a time lie in
// different banks.
template <int kParts, bool kInline>
__global__ __launch_bounds__(1024) void mx_logits_stream_kernel(MxArgs p, int tiles) {
  extern __shared__ __align__(16) uint8_t lds[];   // parts [kParts][N][part_bytes], codes [N][code_bytes], groups
  const int threads = blockDim.x, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = threads >> 6;
  const int N = (int)p.N, row = part_bytes(p.steps), part = N * row, crow = code_bytes(p.steps);
  uint8_t* codes = lds + kParts * part;
  uint8_t* group = codes + N * crow + wave * kGroupBytes;
  const uint32_t to = lds_address(group);

  // where the next group's loads come from
  const int w_row = p.steps * 64, s_row = p.steps * 4;
  const uint32_t s_off = (uint32_t)((lane >> 2) * s_row + (lane & 3) * 4);
  int tile_in = blockIdx.x + gridDim.x * wave, c_in = 0;
  const int tile_step = gridDim.x * waves;
  u32x4s from_w, from_s;
  auto set_tile = [&]() {
    const int64_t v = (int64_t)tile_in * 16;
    const int64_t rows = tile_in < tiles ? (p.V - v < 16 ? p.V - v : 16) : 0;
    from_w = buffer_of(p.w + (rows ? v : 0) * w_row, rows * w_row);
    from_s = buffer_of(p.ws + (rows ? v : 0) * s_row, rows * s_row);
  };
  auto load_group = [&]() {   // (of what lies past the row's end the scales are not used, the codes not read)
    dma4(from_s, to + 4096, s_off + c_in * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * i + (lane >> 4), piece = (lane & 15) ^ row;
      dma16(from_w, to + i * 1024, c_in + (piece >> 2) < p.steps ? row * w_row + c_in * 64 + piece * 16 : kPastBuffer);
    }
    c_in += 4;
    if (c_in >= p.steps) {
      c_in = 0;
      tile_in += tile_step;
      set_tile();
    }
  };
  set_tile();
  load_group();

  if constexpr (kInline) {
    const int vecs = p.steps * 16;
    for (int n = 0; n < N; ++n)
      for (int kv = threadIdx.x; kv < vecs; kv += threads) {   // groups of four lanes leave together
        float v[8];
        u32x2 out[kParts];
        load8(v, static_cast<const bf16*>(p.x) + n * p.ldx, kv * 8, p.H);
        const uint32_t code = split8<kParts>(v, out);
#pragma unroll
        for (int q = 0; q < kParts; ++q) *reinterpret_cast<u32x2*>(lds + q * part + n * row + kv * 8) = out[q];
        if (kv % 4 == 0) codes[n * crow + kv / 4] = (uint8_t)code;
      }
  } else {
    const uint8_t* x = static_cast<const uint8_t*>(p.x);
    const int vecs = p.steps * 8;
    for (int n = 0; n < kParts * N; ++n)
      for (int kv = threadIdx.x; kv < vecs; kv += threads)
        *reinterpret_cast<u32x4*>(lds + n * row + kv * 16) = *reinterpret_cast<const u32x4*>(x + n * p.ldx + kv * 16);
    for (int i = threadIdx.x; i < N * p.steps; i += threads) {
      const int n = i / p.steps, s = i % p.steps;
      const uint8_t* from = p.xs + n * p.ldxs + s * 4;
      *reinterpret_cast<uint32_t*>(codes + n * crow + s * 4) = *reinterpret_cast<const uint32_t*>(from);
    }
  }
  __syncthreads();

  const int n = r < N ? r : N - 1;
  const uint8_t* mine = lds + n * row + g * 16;
  const uint8_t* my_codes = codes + n * crow;
  for (int tile = blockIdx.x + gridDim.x * wave; tile < tiles; tile += tile_step) {
    f32x4 acc[1][1] = {{{0, 0, 0, 0}}};
    for (int c = 0; c < p.steps; c += 4) {
      wait_loads<0>();
      const uint32_t scale = own_scales(*reinterpret_cast<const u32x4*>(group + 4096 + r * 16));
      const uint32_t xc = own_scales(*reinterpret_cast<const u32x4*>(my_codes + c * 4));
      u32x4 a[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) a[s] = *reinterpret_cast<const u32x4*>(group + r * 256 + (((s * 4 + g) ^ r) * 16));
      wait_lds();   // what was read is in registers: its place may be loaded again
      load_group();
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (c + s < p.steps) {
          f32x4 sum = step_sums<kParts>(acc[0][0]);
#pragma unroll
          for (int q = kParts - 1; q >= 0; --q)
            mx_mma(s, sum, a[s], token_columns(mine + q * part + (c + s) * kStep), scale,
                   xc - part_down<kParts>(q) * 0x01010101u);
          add_step<kParts>(acc[0][0], sum);
        }
      }
    }
    put_logits<1, 1>(p, 0, (int64_t)tile * 16, acc);
  }
  wait_loads<0>();   // nothing may land in LDS that is no longer this work-group's
}

// More tokens: a work-group of kWv x kWt waves has kWv kRt tiles of 16
// vocabulary entries by kWt kNt tiles of 16 tokens, kRt x kNt a wave.  A stage is
// kU steps of both, its weights' rows (64 kU bytes) and its tokens' (128 kU bytes
// of each part), in a ring of kStages in LDS; the scales of a group of four steps
// come a group ahead.  One barrier a stage: behind it everyone's loads of the
// stage are there, and the one before it is free.  Rows are swizzled by pieces of
// 16 bytes, so that no bank serves two of the 16 rows that a wave reads at a
// time.  Loads that do not divide evenly among the waves are done twice, alike.
template <int kParts, int kWv, int kWt, int kRt, int kNt, int kU, int kStages>
struct TileShape {
  static constexpr int waves = kWv * kWt, rows = kWv * kRt * 16, tokens = kWt * kNt * 16;
  static constexpr int w_pieces = 4 * kU, x_pieces = 8 * kU;          // of a row in a stage
  static constexpr int w_at_once = 64 / w_pieces, x_at_once = 64 / x_pieces;   // rows a load
  static constexpr int w_loads = rows / w_at_once, x_part = tokens / x_at_once, x_loads = kParts * x_part;
  static constexpr int s_loads = (rows + tokens) / 16;
  static constexpr int w_each = (w_loads + waves - 1) / waves, x_each = (x_loads + waves - 1) / waves;
  static constexpr int s_each = (s_loads + waves - 1) / waves, each = w_each + x_each;
  static constexpr int w_bytes = rows * 64 * kU, x_bytes = tokens * kStep * kU, stage = w_bytes + kParts * x_bytes;
  static constexpr int s_bytes = (rows + tokens) * 16;
  static constexpr int lds = kStages * stage + 2 * s_bytes;
  static constexpr int group = 4 / kU;   // stages of a group
  static_assert(lds <= kLdsMost, "a work-group's stages fit a compute unit");
  static_assert(group > kStages - 2, "a group's scales are there with its first stage");
  __device__ static constexpr int w_swizzle(int row) { return row / (4 / kU) % w_pieces; }
  __device__ static constexpr int x_swizzle(int row) { return kU == 1 ? row / 2 % 8 : row % 16; }
  // loads of this wave that may be under way when stage `i` of a group is needed:
  // the stages behind it, and the scales that one of those began with
  static constexpr int behind(int i) {
    int n = (kStages - 2) * each;
    for (int d = 1; d <= kStages - 2; ++d) n += (i + group * 4 - d) % group == 0 ? s_each : 0;
    return n;
  }
};

template <typename S, int i = 0>
__device__ __forceinline__ void wait_stage(int which) {
  if constexpr (i < S::group) {
    if (which == i) wait_loads<S::behind(i)>();   // (a constant where this is used)
    else wait_stage<S, i + 1>(which);
  }
}

template <int kParts, int kWv, int kWt, int kRt, int kNt, int kU, int kStages>
__global__ __launch_bounds__(64 * kWv * kWt) void mx_logits_tile_kernel(MxArgs p, int row_blocks, int token_blocks) {
  typedef TileShape<kParts, kWv, kWt, kRt, kNt, kU, kStages> S;
  extern __shared__ __align__(16) uint8_t lds[];   // stages, then two groups' scales: rows', tokens'
  // the token blocks of a row block follow each other on one XCD, which reads
  // the weights once
  const int local = blockIdx.x / 8, rb = local / token_blocks * 8 + blockIdx.x % 8, tb = local % token_blocks;
  if (rb >= row_blocks) return;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wv = wave / kWt, wt = wave % kWt;
  const int64_t v0 = (int64_t)rb * S::rows, n0 = (int64_t)tb * S::tokens;
  const int rows = (int)(p.V - v0 < S::rows ? p.V - v0 : S::rows);
  const int tokens = (int)(p.N - n0 < S::tokens ? p.N - n0 : S::tokens);
  const int w_row = p.steps * 64, s_row = p.steps * 4, x_row = (int)p.ldx, c_row = (int)p.ldxs;
  const u32x4s from_w = buffer_of(p.w + v0 * w_row, (int64_t)rows * w_row);
  const u32x4s from_s = buffer_of(p.ws + v0 * s_row, (int64_t)rows * s_row);
  // (the tokens' rows may lie closer than their length, or all be one)
  const int64_t x_bytes = (tokens - 1) * p.ldx + (int64_t)p.steps * kStep;
  const u32x4s from_c = buffer_of(p.xs + n0 * p.ldxs, (tokens - 1) * p.ldxs + p.steps * 4);
  u32x4s from_x[S::x_each];   // the part that the wave's m-th load is of
#pragma unroll
  for (int m = 0; m < S::x_each; ++m) {
    const int q = (wave + m * S::waves) % S::x_loads / S::x_part;
    from_x[m] = buffer_of(static_cast<const uint8_t*>(p.x) + (q * p.N + n0) * p.ldx, x_bytes);
  }
  const uint32_t at = lds_address(lds), at_s = at + kStages * S::stage;

  // offsets of the wave's loads in step 0, and the steps that their pieces are of
  uint32_t w_off[S::w_each], x_off[S::x_each];
  int w_step[S::w_each], x_step[S::x_each];
#pragma unroll
  for (int m = 0; m < S::w_each; ++m) {
    const int row = (wave + m * S::waves) % S::w_loads * S::w_at_once + lane / S::w_pieces;
    const int piece = lane % S::w_pieces ^ S::w_swizzle(row % 16);
    w_off[m] = (uint32_t)(row * w_row + piece * 16);
    w_step[m] = piece / 4;
  }
#pragma unroll
  for (int m = 0; m < S::x_each; ++m) {
    const int row = (wave + m * S::waves) % S::x_loads % S::x_part * S::x_at_once + lane / S::x_pieces;
    const int piece = lane % S::x_pieces ^ S::x_swizzle(row % 16);
    x_off[m] = (uint32_t)(row * x_row + piece * 16);
    x_step[m] = piece / 8;
  }
  auto load_stage = [&](int step, uint32_t to) {
#pragma unroll
    for (int m = 0; m < S::w_each; ++m) {
      const int i = (wave + m * S::waves) % S::w_loads;
      dma16(from_w, to + i * 1024, step + w_step[m] < p.steps ? w_off[m] + step * 64 : kPastBuffer);
    }
#pragma unroll
    for (int m = 0; m < S::x_each; ++m) {
      const int i = (wave + m * S::waves) % S::x_loads;
      dma16(from_x[m], to + S::w_bytes + i * 1024, step + x_step[m] < p.steps ? x_off[m] + step * kStep : kPastBuffer);
    }
  };
  auto load_scales = [&](int c, uint32_t to) {   // (what lies past a row's end is not used)
#pragma unroll
    for (int m = 0; m < S::s_each; ++m) {
      const int i = (wave + m * S::waves) % S::s_loads, j = i - S::rows / 16;
      if (j < 0) dma4(from_s, to + i * 256, (uint32_t)((16 * i + (lane >> 2)) * s_row + c * 4 + (lane & 3) * 4));
      else dma4(from_c, to + i * 256, (uint32_t)((16 * j + (lane >> 2)) * c_row + c * 4 + (lane & 3) * 4));
    }
  };

  load_scales(0, at_s);
#pragma unroll
  for (int t = 0; t < kStages - 1; ++t) load_stage(t * kU, at + t * S::stage);
  const uint8_t* my_w = lds + (wv * kRt * 16 + r) * 64 * kU;
  const uint8_t* my_x = lds + S::w_bytes + (wt * kNt * 16 + r) * kStep * kU;
  const int w_sw = S::w_swizzle(r), x_sw = S::x_swizzle(r);
  const uint8_t* my_s = lds + kStages * S::stage + (wv * kRt * 16 + r) * 16;
  const uint8_t* my_c = lds + kStages * S::stage + S::rows * 16 + (wt * kNt * 16 + r) * 16;
  f32x4 acc[kRt][kNt];
#pragma unroll
  for (int i = 0; i < kRt; ++i)
#pragma unroll
    for (int j = 0; j < kNt; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  int use = 0, fill = (kStages - 1) * S::stage, group = 0;   // offsets of the stage in use and the one to be filled
  for (int c = 0; c < p.steps; c += 4, group ^= 1) {
    uint32_t scale[kRt], code[kNt];
#pragma unroll
    for (int h = 0; h < S::group; ++h) {
      wait_stage<S>(h);
      lds_barrier();
      if (h == 0) {
        load_scales(c + 4, at_s + (group ^ 1) * S::s_bytes);
#pragma unroll
        for (int i = 0; i < kRt; ++i)
          scale[i] = own_scales(*reinterpret_cast<const u32x4*>(my_s + group * S::s_bytes + i * 256));
#pragma unroll
        for (int n = 0; n < kNt; ++n)
          code[n] = own_scales(*reinterpret_cast<const u32x4*>(my_c + group * S::s_bytes + n * 256));
      }
      load_stage(c + (h + kStages - 1) * kU, at + fill);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int s = h * kU + u;
        if (c + s >= p.steps) continue;
        u32x4 a[kRt];
#pragma unroll
        for (int i = 0; i < kRt; ++i)
          a[i] = *reinterpret_cast<const u32x4*>(my_w + use + i * 16 * 64 * kU + ((u * 4 + g) ^ w_sw) * 16);
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
          f32x4 sum[kRt];
#pragma unroll
          for (int i = 0; i < kRt; ++i) sum[i] = step_sums<kParts>(acc[i][n]);
#pragma unroll
          for (int q = kParts - 1; q >= 0; --q) {
            const uint8_t* x = my_x + use + q * S::x_bytes + n * 16 * kStep * kU;
            const i32x4v lo = *reinterpret_cast<const i32x4v*>(x + ((u * 8 + g) ^ x_sw) * 16);
            const i32x4v hi = *reinterpret_cast<const i32x4v*>(x + ((u * 8 + g + 4) ^ x_sw) * 16);
            const i32x8v b = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
            for (int i = 0; i < kRt; ++i)
              mx_mma(s, sum[i], a[i], b, scale[i], code[n] - part_down<kParts>(q) * 0x01010101u);
          }
#pragma unroll
          for (int i = 0; i < kRt; ++i) add_step<kParts>(acc[i][n], sum[i]);
        }
      }
      use = use + S::stage == kStages * S::stage ? 0 : use + S::stage;
      fill = fill + S::stage == kStages * S::stage ? 0 : fill + S::stage;
    }
  }
  wait_loads<0>();   // nothing may land in LDS that is no longer this work-group's
  put_logits<kRt, kNt>(p, n0 + wt * kNt * 16, v0 + wv * kRt * 16, acc);
}

// LDS of the streaming kernel's tokens.
int64_t stream_tokens(int64_t N, int64_t steps, int parts) {
  return N * (parts * part_bytes((int)steps) + code_bytes((int)steps));
}

// One work-group on each of the 256 compute units; waves so that every one has
// about as many tiles as the others.
template <int kParts, bool kInline>
void launch_stream(const MxArgs& p, int waves, hipStream_t st) {
  const int64_t tiles = ceil_div(p.V, 16);
  const int64_t bytes = stream_tokens(p.N, p.steps, kParts) + waves * kGroupBytes;
  const unsigned g = (unsigned)(tiles < 256 ? tiles : 256);
  mx_logits_stream_kernel<kParts, kInline><<<g, waves * 64, (size_t)bytes, st>>>(p, (int)tiles);
}

template <int kParts, int kWv, int kWt, int kRt, int kNt, int kU, int kStages>
void launch_tiles(const MxArgs& p, hipStream_t st) {
  typedef TileShape<kParts, kWv, kWt, kRt, kNt, kU, kStages> S;
  const int64_t rb = ceil_div(p.V, S::rows), tb = ceil_div(p.N, S::tokens);
  mx_logits_tile_kernel<kParts, kWv, kWt, kRt, kNt, kU, kStages>
      <<<(unsigned)(ceil_div(rb, 8) * 8 * tb), 64 * S::waves, S::lds, st>>>(p, (int)rb, (int)tb);
}

// Kernels by size, as measured on random rows and weights (us; floors: the weights'
// bytes at 6.1 TB/s; the products at the 4.0 PFLOP/s that this instruction reaches
// on random operands, twice as many for bf16).
// Streaming, 1 x 6656 x 202048 bf16: 121 with one group of four steps under way in
// each of 10 waves (floor 117); two and three groups took 1 and 6 more, pieces of 64
// bytes 13 more.  With few tiles and four waves 1 x 8192 x 1000 takes 13 with one
// group and 14 with three or more: its time is the way from launch to sum.
// Tiles (waves along V x along N, tiles of 16 a wave, steps x stages), in order
// (2 parts at the first four, 1 at the others):
//                        16 x 6656  24 x 6656  320 x 4096  64 x 8192  320 x 4096  24 x 7168
//                        x 202048   x 202048   x 128256    x 1000     x 128256    x 129280
//   8x1 2x1 2x3          156        220        552         26         526         134
//   4x1 2x2 2x3          161        170        493         25         298         98
//   4x2 4x2 1x2          200        204        274         55         205         118
//   4x2 2x4 1x2          315        321        377         54         203         123
//   floor, memory        117        117        59          1          59          81
//   floor, products      21         32         168         1          84          11
// One part by the last two, x 4096 x 128256: 84 and 97 at 65 tokens, 129 and 125 at
// 129, 138 and 155 at 200, 286 and 318 at 512.
// The large ones are bound by the matrix units, which are busy 57% of 2.0 GHz: 2.47
// PFLOP/s of 8-bit products at 320 bf16 tokens, two for each.  A second work-group
// on the compute unit is worth more than deeper rings (two stages 260, four stages
// and one work-group 334, on constant operands, which leave the clock higher) and
// than the next stage's operands read into registers ahead of the products (two
// work-groups of four waves 311, one of eight 326, likewise).
template <int kParts>
void launch_products(const MxArgs& p, bool raw, hipStream_t st) {
  const int64_t left = kLdsMost - stream_tokens(p.N, p.steps, kParts);
  if (p.N <= 16 && left >= 4 * kGroupBytes) {
    int64_t most = left / kGroupBytes;
    if (most > 12) most = 12;
    const int64_t tiles = ceil_div(p.V, 16);
    int waves = (int)ceil_div(tiles, 256 * ceil_div(tiles, 256 * most));
    if (waves < 4) waves = 4;   // they also bring the tokens to LDS
    if constexpr (kParts > 1) {
      if (raw) {
        launch_stream<kParts, true>(p, waves, st);
        return;
      }
    }
    launch_stream<kParts, false>(p, waves, st);
    return;
  }
  if constexpr (kParts == kDigits) {
    // Up to 16 tokens, 8 x 4096 x 128256: 65, by 32 tokens 85.  33 to 48 tokens:
    // one work-group of 48 on a compute unit, or two of 32 with half the rows; a
    // round of the former lasts as long as 1.6 of the latter.
    // 48 x 4096 by 48 and by 32: x 32000 55 and 43 (1 round and 1), x 36000 55 and 62
    // (1 and 2), x 80000 114 and 104 (2 and 3), x 104000 118 and 135 (2 and 4), x 150000
    // 178 and 191 (3 and 5); 33 x 1001 x 50001 21 and 25.
    const int64_t by48 = ceil_div(ceil_div(p.V, 256), 256), by32 = ceil_div(2 * ceil_div(p.V, 128), 512);
    if (p.N <= 16) launch_tiles<kDigits, 4, 1, 2, 1, 2, 2>(p, st);
    else if (p.N > 32 && p.N <= 48 && 5 * by32 >= 8 * by48) launch_tiles<kDigits, 8, 1, 2, 3, 1, 2>(p, st);
    else launch_tiles<kDigits, 4, 1, 2, 2, 1, 2>(p, st);
  } else {
    // (few tiles: rather more of them, for the other compute units)
    const bool few = ceil_div(p.V, 256) * ceil_div(p.N, 64) < 256;
    if (p.N <= 16) launch_tiles<kParts, 8, 1, 2, 1, 2, 3>(p, st);
    else if (p.N <= 32 || few) launch_tiles<kParts, 4, 1, 2, 2, 2, 3>(p, st);
    else if (kParts == 1 && p.N > 64) launch_tiles<1, 4, 2, 2, 4, 1, 2>(p, st);
    else launch_tiles<kParts, 4, 2, 4, 2, 1, 2>(p, st);
  }
}

// Tokens in parts: how many, and how they lie in the workspace.
struct MxTokens {
  int parts;
  size_t codes, total;   // byte offsets in the workspace (parts at 0)
  int64_t ldp, ldc;
};

// bf16 rows are digits too where the logits are fp32: what the matrix unit cuts
// from products of their E4M3 parts ends below a bf16 logit's last bit, not below an
// fp32 one's (7e-5 of the logits where one channel in 100 is 300 times the others;
// 1e-7 so).  Its price, us: 1 x 6656 x 202048 131 for 121, 16 185 for 159, 320 x 4096
// x 128256 709 for 292.
MxTokens mx_tokens(int64_t N, int64_t H, int x_dtype, int dtype) {
  MxTokens t{};
  const int64_t steps = ceil_div(H, kStep);
  t.parts = x_dtype == FLCE_DTYPE_MX8 ? 1 : x_dtype == FLCE_DTYPE_BF16 && dtype == FLCE_DTYPE_BF16 ? 2 : kDigits;
  t.ldp = steps * kStep;
  t.ldc = code_bytes((int)steps);
  t.codes = (size_t)(t.parts * N * t.ldp);
  t.total = (t.codes + (size_t)(N * t.ldc) + 255) & ~size_t(255);
  if (t.total < 256) t.total = 256;
  return t;
}

bool mx_sizes_ok(int64_t N, int64_t H, int x_dtype) {
  return (x_dtype == FLCE_DTYPE_BF16 || x_dtype == FLCE_DTYPE_F32 || x_dtype == FLCE_DTYPE_MX8) && N >= 0 && H >= 1;
}

// Nearest E2M1 code, ties to the even one.
__device__ __forceinline__ uint32_t e2m1_code(float x) {
  const float a = __builtin_fabsf(x);
  const uint32_t c = (uint32_t)(a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) +
                     (a > 5.0f);
  return c | (x < 0.0f && c ? 8u : 0u);
}

// Eight columns per thread, four threads per block; a row has `vecs` of them,
// a multiple of 16.  Done once for a projection; 202048 x 6656 takes 996 us from
// bf16 and 1087 from fp32 (floors at 6.1 TB/s 558 and 999): a thread has one load of
// 16 bytes under way, or two, which reach 3.4 and 5.6 TB/s.
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
  if (!W || !packed || !scales || addr(W) % (dtype == FLCE_DTYPE_BF16 ? 2 : 4) || addr(packed) % 16 ||
      addr(scales) % 4)
    return FLCE_EINVAL;
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

extern "C" size_t flce_logits_mx_workspace_size(int64_t N, int64_t H, int x_dtype) {
  using namespace flce;
  if (!mx_sizes_ok(N, H, x_dtype) || N > (int64_t(1) << 20) || H > (int64_t(1) << 21)) return 0;
  return mx_tokens(N, H, x_dtype, FLCE_DTYPE_F32).total;   // enough for either type of logits
}

extern "C" int flce_logits_mx(const void* x, int64_t ld_x, const void* x_scales, int64_t ld_xs, const void* packed,
                              const void* scales, int64_t N, int64_t H, int64_t V, float softcap_T, float multiplier,
                              void* logits, int64_t ld_logits, hipStream_t stream, int x_dtype, int dtype,
                              void* workspace, size_t workspace_bytes) {
  using namespace flce;
  if (!mx_sizes_ok(N, H, x_dtype) || (dtype != FLCE_DTYPE_BF16 && dtype != FLCE_DTYPE_F32) || V < 1) return FLCE_EINVAL;
  if (!std::isfinite(softcap_T) || !std::isfinite(multiplier)) return FLCE_EINVAL;
  if (softcap_T > 0.0f && (!std::isfinite(1.0f / softcap_T) || !std::isfinite(multiplier / softcap_T)))
    return FLCE_EINVAL;
  if (N > (int64_t(1) << 20) || V > (int64_t(1) << 24) || H > (int64_t(1) << 21)) return FLCE_EUNSUPPORTED;
  const int64_t steps = ceil_div(H, kStep), vecs = steps * 16;
  // a launch holds fewer than 2^32 threads (16 logits a thread of the products)
  if (N * vecs > (int64_t(1) << 31) || N * V > (int64_t(1) << 35)) return FLCE_EUNSUPPORTED;
  if (N == 0) return FLCE_OK;
  const bool mx8 = x_dtype == FLCE_DTYPE_MX8;
  const uintptr_t es = mx8 ? 1 : x_dtype == FLCE_DTYPE_BF16 ? 2 : 4, os = dtype == FLCE_DTYPE_BF16 ? 2 : 4;
  if (!x || !packed || !scales || !logits || !workspace || (mx8 != (x_scales != nullptr))) return FLCE_EINVAL;
  if (addr(x) % es || addr(packed) % 16 || addr(scales) % 4 || addr(logits) % os || addr(workspace) % 256)
    return FLCE_EINVAL;
  if (ld_x < 0 || (mx8 && ld_xs < 0) || (N > 1 && ld_logits < V)) return FLCE_EINVAL;
  const MxTokens t = mx_tokens(N, H, x_dtype, dtype);
  if (workspace_bytes < t.total) return FLCE_EWORKSPACE;
  uint8_t* parts = static_cast<uint8_t*>(workspace);
  uint8_t* codes = parts + t.codes;
  // rows in 8 bits that are whole groups of four steps are read where they are;
  // one or two bf16 rows are split by the work-groups (a launch less)
  const bool ready = mx8 && H % (4 * kStep) == 0 && ld_x <= kMostRow && ld_xs <= kMostRow && ld_x % 16 == 0 &&
                     ld_xs % 16 == 0 && addr(x) % 16 == 0 && addr(x_scales) % 16 == 0;
  const bool raw =
      x_dtype == FLCE_DTYPE_BF16 && N <= 2 && stream_tokens(N, steps, t.parts) <= kLdsMost - 4 * kGroupBytes;
  MxArgs p{parts, codes, t.ldp, t.ldc, static_cast<const uint8_t*>(packed), static_cast<const uint8_t*>(scales), logits,
           ld_logits, N, V, (int)H, (int)steps, softcap_T > 0.0f ? softcap_T : 0.0f, multiplier,
           dtype == FLCE_DTYPE_BF16};
  if (ready || raw) {
    p.x = x;
    p.xs = static_cast<const uint8_t*>(x_scales);
    p.ldx = ld_x;
    p.ldxs = ld_xs;
  } else {
    ProfileScope ps(FLCE_KERNEL_SPLIT_MX, stream);
    const unsigned g = (unsigned)ceil_div(N * vecs, 256);
    if (mx8)
      mx_copy_kernel<<<g, 256, 0, stream>>>(static_cast<const uint8_t*>(x), ld_x, static_cast<const uint8_t*>(x_scales),
                                            ld_xs, N, (int)H, (int)vecs, parts, t.ldp, codes, t.ldc);
    else if (x_dtype == FLCE_DTYPE_BF16 && t.parts == 2)
      mx_split_kernel<bf16, 2><<<g, 256, 0, stream>>>(static_cast<const bf16*>(x), ld_x, N, (int)H, (int)vecs, parts,
                                                      t.ldp, codes, t.ldc);
    else if (x_dtype == FLCE_DTYPE_BF16)
      mx_split_kernel<bf16, kDigits><<<g, 256, 0, stream>>>(static_cast<const bf16*>(x), ld_x, N, (int)H, (int)vecs,
                                                            parts, t.ldp, codes, t.ldc);
    else
      mx_split_kernel<float, kDigits><<<g, 256, 0, stream>>>(static_cast<const float*>(x), ld_x, N, (int)H, (int)vecs,
                                                             parts, t.ldp, codes, t.ldc);
  }
  ProfileScope ps(FLCE_KERNEL_LOGITS_MX, stream);
  if (t.parts == 1) launch_products<1>(p, false, stream);
  else if (t.parts == 2) launch_products<2>(p, raw, stream);
  else launch_products<kDigits>(p, raw, stream);
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}
