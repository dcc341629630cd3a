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
  float* ws;              // rows path with ids: rows_ws_bytes(...)
};

// Workspace of the row-streaming kernels: base sums and t of every token.
inline size_t rows_ws_bytes(int32_t n_proj, int32_t n_tokens, int64_t h_out) {
  return sizeof(float) * n_proj * static_cast<size_t>(n_tokens) * static_cast<size_t>(h_out + kMaxRank);
}

lora_status launch_rows(const BaseCall& c, hipStream_t s);    // rows.hip
lora_status launch_tiles(const BaseCall& c, hipStream_t s);   // tiles.hip

}  // namespace lora
