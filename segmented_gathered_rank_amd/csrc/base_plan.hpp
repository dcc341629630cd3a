// How a batch of the 4-bit and gated base products is cut between the
// row-streaming and the tiled kernels (host arithmetic, no device code; also
// built by the host unit tests).
#pragma once

#include <algorithm>
#include <cstdint>

namespace lora {

// Storage of W^T ([h_out] rows along h_in).
enum class WKind : int {
  kBf16,    // bf16
  kFp8,     // OCP e4m3 codes, one float scale per row
  kInt4,    // 4-bit codes q: s (q - z), s and z per row and group of `group` k (no z array: 8)
  kTable4   // 4-bit codes q: s T[q], T a 16-entry bf16 codebook
};
constexpr bool is_w4(WKind k) { return k == WKind::kInt4 || k == WKind::kTable4; }

constexpr int kRowsTokens = 64;            // tokens of one row-streaming workgroup at most; longer batches run in chunks
constexpr int32_t kRowsMaxTokens = 32768;  // longest batch of those kernels: the finish has a grid row for each token

// A batch's first `tiles` tokens take tiles (fused_gemm.hpp), the `rows` after
// them stream W's rows (rows_kernels.hpp); either may be 0.
struct BatchCut {
  int32_t tiles, rows;
};

// What the cut depends on.  adapters: the pool's slots, or 0 for a call without ids.
struct BaseShape {
  WKind kind;
  int n_proj;
  int32_t h_in, h_out;
  int32_t adapters, max_rank;
};

// The kernels' measured costs in microseconds.
//
// With ids.  Rows: 10 to start, 0.4 for each 10^6 weights and chunk of 64 tokens,
// 6 for each 10^6 base sums written and read.  Tiles: 35 to start (with the
// shrink), 0.032 for each k of every round of 256 tiles, and 12 for each projection
// and 16 ranks past the first 16 that an adapter may have (a tile meets two or
// three adapters where the batch has runs).  The host does not see the ids, and a
// batch whose neighbours differ costs tiles about 4 for each round, projection and
// 16 ranks of every adapter that a tile may meet: 0.2 is charged of it, as if one
// batch in twenty were such, so that where the ways are close rows, which take
// any order alike, are taken.  Measured, rows against tiles:
// 4096x4096 4-bit 58 / 156 at 512 tokens, 97 / 157 at 1000; 4096 -> 2 x 12288 bf16
// 204 / 127 at 256; 768 -> 2 x 2304 4-bit 42 / 60 at 512, 69 / 64 at 1000; 2048 ->
// 2 x 8192 fp8, ranks up to 64, 84 / 143 at 256, 140 / 145 at 512.  With unlike
// neighbours of 64 adapters: the third shape 98 / 553 at 1000, the second 209 / 697.
//
// Without ids there is no shrink, no expand and, on rows, no finish unless h_in is
// split.  Rows: 10, 0.33, 0.2 or 0.19 for each 10^6 weights of 16, 8 or 4 bits and
// chunk, and 1 for each 10^6 base sums.  Tiles: 15, and 0.03 for each k of every
// round.  Measured, rows against tiles: 4096 -> 2 x 12288 bf16 172 / 98 at 256
// tokens, 505 / 207 at 1000; 2048 -> 2 x 8192 fp8 60 / 70 at 512, 115 / 72 at 1000;
// 4096x4096 4-bit 50 / 141 at 1000, 100 / 149 at 2048; 768 -> 2 x 2304 4-bit
// 35 / 44 at 1000, 54 / 47 at 2048.
//
// A few tokens past a multiple of 256 may add a round of tiles for a batch's rest
// that rows take in less: 4096 -> 2 x 8192 fp8, 2111 tokens as 2048 + 63 take 343
// us, where 2304, as many tiles as 2111 alone would be, take 416.
inline double rows_cost(const BaseShape& b, int32_t n) {
  const double cols = static_cast<double>(b.n_proj) * b.h_out;
  const double chunks = static_cast<double>((static_cast<int64_t>(n) + kRowsTokens - 1) / kRowsTokens);
  if (b.adapters == 0) {
    const double per = b.kind == WKind::kBf16 ? 0.33e-6 : b.kind == WKind::kFp8 ? 0.2e-6 : 0.19e-6;
    return 10.0 + per * cols * b.h_in * chunks + 1e-6 * n * cols;
  }
  return 10.0 + 0.4e-6 * cols * b.h_in * chunks + 6e-6 * n * cols;
}
inline double tiles_cost(const BaseShape& b, int32_t n) {
  const int64_t cols = static_cast<int64_t>(b.n_proj) * b.h_out;
  const int64_t n_tiles = (static_cast<int64_t>(n) + 255) / 256 * ((cols + 255) / 256);
  const double rounds = static_cast<double>((n_tiles + 255) / 256);
  if (b.adapters == 0) return 15.0 + 0.03 * b.h_in * rounds;
  const int units = b.n_proj * std::min(b.adapters, 256) * ((b.max_rank + 15) / 16);   // that a tile may meet
  return 35.0 + 12.0 * b.n_proj * ((b.max_rank - 1) / 16) + (0.032 * b.h_in + 0.2 * units) * rounds;
}

inline BatchCut cut_batch(const BaseShape& b, int32_t n) {
  if (n <= kRowsTokens) return {0, n};
  const double rows = rows_cost(b, n), tiles = tiles_cost(b, n);
  const int32_t tail = n % 256, whole = n - tail;
  if (tail > 0 && whole > 0 && tiles_cost(b, whole) + rows_cost(b, tail) < std::min(rows, tiles)) return {whole, tail};
  return rows < tiles && n <= kRowsMaxTokens ? BatchCut{0, n} : BatchCut{n, 0};
}

}  // namespace lora
