// Launches of the row-streaming base product (rows_kernels.hpp).
#include "base_launch.hpp"
#include "rows_kernels.hpp"

namespace lora {
namespace {

template <WKind WK, int G, int TB, bool GLU>
void launch(const RowsArgs& base, hipStream_t s) {
  constexpr int CB = GLU ? 2 : 1;
  RowsArgs a = base;
  a.n_blocks = a.h_out / (16 * (GLU ? CB / 2 : CB));
  const unsigned gx = static_cast<unsigned>(a.n_units + (a.n_blocks + 7) / 8 * 8);
  const unsigned gy = static_cast<unsigned>((a.n + kRowsTokens - 1) / kRowsTokens);
  hipLaunchKernelGGL((k_rows<WK, G, TB, CB, GLU>), dim3(gx, gy), dim3(kRowsThreads), 0, s, a);
}

template <WKind WK, int G, bool GLU>
void by_tokens(const RowsArgs& a, hipStream_t s) {
  if (a.n <= 16) launch<WK, G, 1, GLU>(a, s);
  else if (a.n <= 32) launch<WK, G, 2, GLU>(a, s);
  else launch<WK, G, 4, GLU>(a, s);
}

template <WKind WK, bool GLU>
void by_group(const RowsArgs& a, int32_t group, hipStream_t s) {
  if (group == 32) by_tokens<WK, 32, GLU>(a, s);
  else if (group == 64) by_tokens<WK, 64, GLU>(a, s);
  else by_tokens<WK, 128, GLU>(a, s);
}

}  // namespace

lora_status launch_rows(const BaseCall& c, hipStream_t s) {
  RowsArgs a{};
  a.pv = c.pv;
  a.w[0] = c.w[0];
  a.w[1] = c.w[1];
  a.x = c.x;
  a.ids = c.ids;
  a.y = c.y;
  a.ld_x = c.ld_x;
  a.ld_w = c.ld_w;
  a.ld_y = c.ld_y;
  a.n = c.n;
  a.h_in = c.h_in;
  a.h_out = c.h_out;
  a.module[0] = c.module[0];
  a.module[1] = c.module[1];
  a.act = c.act;
  const int n_proj = c.glu ? 2 : 1;
  if (c.ids) {
    a.part = c.ws;
    a.t = c.ws + static_cast<int64_t>(n_proj) * c.n * c.h_out;
    const int units = (c.n < kRowsTokens ? c.n : kRowsTokens) * n_proj * ((c.pv.max_rank + 15) / 16);
    a.n_units = (units + 7) / 8 * 8;
  }
  if (c.glu) {
    switch (c.kind) {
      case WKind::kBf16: by_tokens<WKind::kBf16, 0, true>(a, s); break;
      case WKind::kFp8: by_tokens<WKind::kFp8, 0, true>(a, s); break;
      case WKind::kInt4: by_group<WKind::kInt4, true>(a, c.group, s); break;
      case WKind::kTable4: by_group<WKind::kTable4, true>(a, c.group, s); break;
    }
  } else if (c.kind == WKind::kInt4) {
    by_group<WKind::kInt4, false>(a, c.group, s);
  } else {
    by_group<WKind::kTable4, false>(a, c.group, s);
  }
  if (hipGetLastError() != hipSuccess) return LORA_ERR_HIP;
  if (c.ids) {
    const dim3 grid((c.h_out / 4 + kFinishThreads - 1) / kFinishThreads, c.n);
    if (c.glu) hipLaunchKernelGGL((k_rows_finish<true>), grid, dim3(kFinishThreads), 0, s, a);
    else hipLaunchKernelGGL((k_rows_finish<false>), grid, dim3(kFinishThreads), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // namespace lora
