// How many threads pick a row's cut or token (sample_rows.hpp), and how many
// pieces of a row their work-group's arrays hold.  Host code alone, so that the
// rule can be tested without a GPU.
#pragma once

#include <stdint.h>

namespace flce {

constexpr int kPiece = 8192;                          // logits per work-group of the scan
constexpr int64_t kMaxVocab = int64_t(1) << 24;

// Pieces that a work-group of `threads` has room for: two a thread, every row's
// with 1024 threads; a quarter of that with 512, of which two work-groups share a
// compute unit's memory (rows up to 2097152).
constexpr int picker_pieces(int threads) { return threads == 1024 ? (int)(kMaxVocab / kPiece) : threads / 2; }

// 512 threads, two rows at a time on a compute unit, where there are more rows
// than compute units and either a flat row's border bin still fits the shorter
// list or (`any_list`) the list need not hold it.  1024 rows of 4000 bf16 logits,
// 512 against 1024 threads: k = 50 and p = 0.95 on peaked rows 31 against 53 us, p
// = 0.9 on flat ones 45 against 76 us, no filter 22 against 30 us.
constexpr int picker_threads(int64_t rows, int64_t V, bool any_list) {
  const int64_t pieces = (V + kPiece - 1) / kPiece;
  return rows > 256 && pieces <= picker_pieces(512) && (V <= 65536 || any_list) ? 512 : 1024;
}

}  // namespace flce
