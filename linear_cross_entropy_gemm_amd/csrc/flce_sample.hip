// Drawing a token from each row of logits (flce_sample): temperature, top-k,
// top-p and min-p filters, then the inverse of the distribution function in
// index order at a given random number.
//
// The kernels and their reasons are in sample_rows.hpp.
#include <cmath>

#include "sample_rows.hpp"

namespace flce {

namespace {

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

// Workspace: what the scan leaves, for rows longer than kSmall.
SampleLayout sample_layout(int64_t N, int64_t V) {
  SampleLayout l{(V + kPiece - 1) / kPiece, 0, 0, 0, 0};
  // launches of fewer than 2^32 threads
  if (N > (int64_t(1) << 21) || V > kMaxVocab || N * l.pieces > (int64_t(1) << 23)) return l;
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

void sample_args(SampleArgs& a, int64_t N, int64_t V, const SampleLayout& l, void* workspace) {
  a.N = N;
  a.V = V;
  int bits = 0;
  while ((int64_t(1) << bits) < V) ++bits;
  a.s = 62 - bits < 51 ? 62 - bits : 51;
  char* ws = static_cast<char*>(workspace);
  a.pieces = (int)l.pieces;
  a.pmax = reinterpret_cast<uint32_t*>(ws);
  a.psum = reinterpret_cast<double*>(ws + l.psum);
  a.hist = reinterpret_cast<u64*>(ws + l.hist);
  a.gmax = reinterpret_cast<uint32_t*>(ws + l.gmax);
}

// The scalar parameters' ranges and the per-row arrays' alignment.
bool sample_params_ok(const flce_sample_params_t& q) {
  if (!q.temperature_rows && !(q.temperature >= 0.0f && std::isfinite(q.temperature))) return false;
  if (!q.top_k_rows && q.top_k < 0) return false;
  if (!q.top_p_rows && !(q.top_p > 0.0f && q.top_p <= 1.0f)) return false;
  if (!q.min_p_rows && !(q.min_p >= 0.0f && q.min_p <= 1.0f)) return false;
  return on(q.temperature_rows, 4) && on(q.top_k_rows, 8) && on(q.top_p_rows, 4) && on(q.min_p_rows, 4);
}

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
  if (!sample_params_ok(*params)) return FLCE_EINVAL;
  if (!on(logprobs, 4) || !on(workspace, 256)) return FLCE_EINVAL;
  if (N > 0 && (!logits || !u || !tokens || !workspace)) return FLCE_EINVAL;
  if (!on(logits, es) || !on(u, 4) || !on(tokens, 8) || ld_logits < 0) return FLCE_EINVAL;
  const SampleLayout l = sample_layout(N, V);
  if (l.total == 0) return FLCE_EUNSUPPORTED;
  if (N == 0) return FLCE_OK;
  if (workspace_bytes < l.total) return FLCE_EWORKSPACE;
  SampleArgs a{};
  a.z = logits;
  a.ld = ld_logits;
  a.u = u;
  a.prm = *params;
  a.tokens = tokens;
  a.logprobs = logprobs;
  sample_args(a, N, V, l, workspace);
  launch_rows<false>(a, stream, dtype, FLCE_KERNEL_SAMPLE_SCAN, FLCE_KERNEL_SAMPLE_PICK);
  return hipGetLastError() == hipSuccess ? FLCE_OK : FLCE_EDEVICE;
}
