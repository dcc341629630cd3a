// Launches of the tiled base product (fused_gemm.hpp) with 4-bit weights or
// the gate.
#include "base_launch.hpp"
#include "fused_gemm.hpp"

namespace lora {
namespace {

template <WKind WK, bool GLU, bool G32>
void launch(const FusedArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.n_tiles + 7) / 8 * 8));
  if (a.ids) hipLaunchKernelGGL((k_fused_gemm<FgLora::kGiven, WK, GLU, G32>), grid, dim3(kFgThreads), 0, s, a);
  else hipLaunchKernelGGL((k_fused_gemm<FgLora::kNone, WK, GLU, G32>), grid, dim3(kFgThreads), 0, s, a);
}

template <WKind WK, bool GLU>
void by_group(const FusedArgs& a, int32_t group, hipStream_t s) {
  if (group == 32) launch<WK, GLU, true>(a, s);
  else launch<WK, GLU, false>(a, s);
}

int64_t n_tiles(bool glu, int32_t n, int32_t h_out) {
  const int tc = glu ? kFgGluCols : kFgBN;
  return (static_cast<int64_t>(n) + kFgBM - 1) / kFgBM * ((h_out + tc - 1) / tc);
}

}  // namespace

// 512 threads to a tile, and to 64 tokens of the shrink: within a launch's 2^32 - 1.
bool tiles_fit(bool glu, int32_t n, int32_t h_out) {
  return n <= (1 << 28) && n_tiles(glu, n, h_out) <= (int64_t(1) << 22);
}

lora_status launch_tiles(const BaseCall& c, hipStream_t s) {
  FusedArgs a{};
  a.pv = c.pv;
  a.x = c.x;
  a.w[0] = c.w[0];
  a.w[1] = c.w[1];
  a.ids = c.ids;
  a.y = c.y;
  a.t = c.ids ? c.ws : nullptr;
  a.t_splits = tiles_splits(c.n, c.h_in);
  a.ld_x = c.ld_x;
  a.ld_w = c.ld_w;
  a.ld_y = c.ld_y;
  a.n = c.n;
  a.h_in = c.h_in;
  a.h_out = c.h_out;
  a.module[0] = c.module[0];
  a.module[1] = c.module[1];
  a.act = c.act;
  a.group_shift = c.group == 128 ? 2 : c.group == 64 ? 1 : 0;
  const int tc = c.glu ? kFgGluCols : kFgBN;
  a.n_ct = (c.h_out + tc - 1) / tc;
  a.n_tiles = static_cast<int32_t>(n_tiles(c.glu, c.n, c.h_out));
  if (c.glu) {
    switch (c.kind) {
      case WKind::kBf16: launch<WKind::kBf16, true, false>(a, s); break;
      case WKind::kFp8: launch<WKind::kFp8, true, false>(a, s); break;
      case WKind::kInt4: by_group<WKind::kInt4, true>(a, c.group, s); break;
      case WKind::kTable4: by_group<WKind::kTable4, true>(a, c.group, s); break;
    }
  } else if (c.kind == WKind::kInt4) {
    by_group<WKind::kInt4, false>(a, c.group, s);
  } else {
    by_group<WKind::kTable4, false>(a, c.group, s);
  }
  return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // namespace lora
