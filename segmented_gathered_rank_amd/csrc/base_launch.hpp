// Launches of the base-product kernels (arguments checked by the caller).
#pragma once

#include "base_args.hpp"

namespace lora {

// A checked call of the 4-bit or gated entry points.
struct BaseCall {
  PoolView pv;
  WKind kind;
  int32_t group;          // 4-bit: 32, 64 or 128
  bool glu;
  WView w[2];
  const __bf16* x;
  const int32_t* ids;     // null: no adapters
  __bf16* y;
  int64_t ld_x, ld_w, ld_y;   // ld_w in bytes
  int32_t n, h_in, h_out;
  int32_t module[2];
  int32_t act;
  size_t ws_bytes;
  float* ws;              // may be null without ids; its size then bounds the split of h_in
};

// Workspace of the row-streaming kernels: the base sums of each split of h_in,
// and t, of every token.
constexpr int kRowsMaxSplits = 8;
inline size_t rows_bytes(int splits, int n_proj, int32_t n_tokens, int64_t h_out) {
  return sizeof(float) * n_proj * static_cast<size_t>(n_tokens) * static_cast<size_t>(splits * h_out + kMaxRank);
}
// What a call uses when it is given as much as it can use (adapters: 0 without ids).
size_t rows_ws_bytes(WKind kind, int n_proj, int32_t n_tokens, int32_t adapters, int32_t h_in, int32_t h_out);

// Workspace of the tiled kernels: t of every token from each split of h_in.
// The splits fill the GPU once, with 64 tokens and at least 256 k to each
// workgroup; the tiles add them up.
constexpr int kTilesMaxSplits = 4;
inline int tiles_splits(int32_t n_tokens, int32_t h_in) {
  const int64_t chunks = (static_cast<int64_t>(n_tokens) + 63) / 64;
  int s = static_cast<int>(256 / chunks);
  if (s > kTilesMaxSplits) s = kTilesMaxSplits;
  if (s > h_in / 256) s = h_in / 256;
  return s < 1 ? 1 : s;
}
inline size_t tiles_ws_bytes(int n_proj, int32_t n_tokens, int32_t h_in) {
  return sizeof(float) * n_proj * static_cast<size_t>(n_tokens) * kMaxRank * tiles_splits(n_tokens, h_in);
}

lora_status launch_shrink(const BaseCall& c, int splits, hipStream_t s);  // rows.hip: t of every token into c.ws
lora_status launch_rows(const BaseCall& c, hipStream_t s);    // rows.hip
lora_status launch_tiles(const BaseCall& c, hipStream_t s);   // tiles.hip
bool tiles_fit(bool glu, int32_t n_tokens, int32_t h_out);

}  // namespace lora
