// Launches of the row-streaming base product (rows_kernels.hpp).
#include <algorithm>

#include "base_launch.hpp"
#include "rows_kernels.hpp"

namespace lora {
namespace {

constexpr int kRowsCB = 2;   // 16-row blocks of W^T to a wave of k_rows

struct RowsPlan {
  int tb;        // 16-token blocks of a workgroup: 1 to 4
  bool x_lds;    // k_rows, else k_mid
  int blocks;    // base workgroups of one split and chunk
  int chunks;    // of 16 * tb tokens
  int splits;    // of h_in over workgroups
  int units;     // shrink workgroups of one chunk
};

// Workgroups that the GPU holds at a time: k_rows two to a CU, k_mid one.
constexpr int kRowsResident = 512;
constexpr int kMidResident = 256;
constexpr int kShrinkUnits = 128;   // shrink workgroups of a launch, about

// adapters: how many different ones the batch may hold (0: a call without ids).
RowsPlan rows_plan(WKind kind, int n_proj, int32_t n, int32_t adapters, int32_t h_in, int32_t h_out, size_t ws_bytes) {
  RowsPlan p{};
  p.tb = n > 48 ? 4 : (n + 15) / 16;
  p.chunks = (n + 16 * p.tb - 1) / (16 * p.tb);
  // Each takes an adapter and projection at a time.  The chunks of a longer batch
  // have runs, as a rule, and workgroups without work are not free: 512 tokens in
  // runs of 128, 4096 -> 4096 56 us a call with 16 to a chunk, 68 with 64; 1000
  // tokens, 768 -> 2 x 2304 66 and 74.
  p.units = (std::min(std::min({n, 16 * p.tb, adapters}) * n_proj, std::max(kShrinkUnits / p.chunks, 16)) + 7) / 8 * 8;
  // the split of h_in with the least rounds of workgroups times steps of each,
  // at `step` microseconds a step, 4 to start a workgroup, and the sums' way
  // through the workspace (a call, split against unsplit: 64 tokens, 4096 ->
  // 4096 4-bit 19 us in 8 splits against 61; 33 tokens, 4096 -> 2 x 12288 4-bit 34
  // in 2 against 51)
  auto split = [&](int cols, int steps, int min_steps, int resident, double step) {
    p.blocks = (h_out * n_proj + cols - 1) / cols;
    const double sums = 2e-6 * n * n_proj * h_out;
    double best = 0.0;
    p.splits = 0;
    for (int s = 1; s <= kRowsMaxSplits && (s == 1 || s * min_steps <= steps); ++s) {
      if (s > 1 && rows_bytes(s, n_proj, n, h_out) > ws_bytes) break;
      const int64_t wgs = static_cast<int64_t>(p.blocks) * p.chunks * s;
      const double cost = static_cast<double>((wgs + resident - 1) / resident) * ((steps + s - 1) / s * step + 4.0) +
                          s * sums;
      if (p.splits == 0 || cost < best) {
        best = cost;
        p.splits = s;
      }
    }
  };
  const int ks = is_w4(kind) ? 128 : kind == WKind::kFp8 ? 64 : 32, steps = (h_in + ks - 1) / ks;
  if (p.tb == 1) {
    split(16 * kRowsCB, steps, kRowsWaves, kRowsResident, 1.0 / kRowsWaves);
    const int range = ((steps + p.splits - 1) / p.splits + 1) * ks;   // at most, of one workgroup
    p.x_lds = n * rows_x_stride(range) <= kRowsXBytes;
  }
  // beside the shrink: 64 tokens, 64 adapters of ranks 8 to 64, 2048 -> 2 x 8192 fp8
  // 34 us a call with rounds of 128, 41 of 256; 50 tokens, 32 adapters of rank 64,
  // 4096 -> 2 x 4096 bf16 42 with 192, 54 with 256; 177 tokens in runs of 29, 4160 ->
  // 5440 48 with 192, 52 with 208
  const int beside = adapters == 0 ? 0 : p.chunks > 1 ? kShrinkUnits / 2 : p.units;
  if (!p.x_lds) split(32 * kMidWaves, (h_in + 127) / 128, 2, kMidResident - beside, 1.5);
  return p;
}

template <WKind WK, int G, bool GLU>
void by_tokens(const RowsArgs& base, const RowsPlan& p, hipStream_t s) {
  RowsArgs a = base;
  a.n_blocks = p.blocks;
  const dim3 grid(static_cast<unsigned>((a.n_units + (a.n_blocks + 7) / 8 * 8) * p.chunks), 1, p.splits);
  const dim3 wg(kRowsThreads), wg_mid(kMidThreads);
  if (p.x_lds) hipLaunchKernelGGL((k_rows<WK, G, kRowsCB, GLU>), grid, wg, 0, s, a);
  else if (p.tb == 1) hipLaunchKernelGGL((k_mid<WK, G, 1, GLU>), grid, wg_mid, 0, s, a);
  else if (p.tb == 2) hipLaunchKernelGGL((k_mid<WK, G, 2, GLU>), grid, wg_mid, 0, s, a);
  else if (p.tb == 3) hipLaunchKernelGGL((k_mid<WK, G, 3, GLU>), grid, wg_mid, 0, s, a);
  else hipLaunchKernelGGL((k_mid<WK, G, 4, GLU>), grid, wg_mid, 0, s, a);
}

template <WKind WK, bool GLU>
void by_group(const RowsArgs& a, const RowsPlan& p, int32_t group, hipStream_t s) {
  if (group == 32) by_tokens<WK, 32, GLU>(a, p, s);
  else if (group == 64) by_tokens<WK, 64, GLU>(a, p, s);
  else by_tokens<WK, 128, GLU>(a, p, s);
}

RowsArgs rows_args(const BaseCall& c) {
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
  return a;
}

}  // namespace

size_t rows_ws_bytes(WKind kind, int n_proj, int32_t n, int32_t adapters, int32_t h_in, int32_t h_out) {
  return rows_bytes(rows_plan(kind, n_proj, n, adapters, h_in, h_out, SIZE_MAX).splits, n_proj, n, h_out);
}

lora_status launch_shrink(const BaseCall& c, int splits, hipStream_t s) {
  RowsArgs a = rows_args(c);
  a.t = c.ws;
  const dim3 grid((c.n + kRowsTokens - 1) / kRowsTokens, splits);
  hipLaunchKernelGGL(k_long_shrink, grid, dim3(kRowsThreads), 0, s, a, c.glu ? 2 : 1);
  return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

lora_status launch_rows(const BaseCall& c, hipStream_t s) {
  RowsArgs a = rows_args(c);
  const int n_proj = c.glu ? 2 : 1;
  const RowsPlan p = rows_plan(c.kind, n_proj, c.n, c.ids ? c.pv.n_slots : 0, c.h_in, c.h_out, c.ws_bytes);
  a.splits = p.splits;
  if (c.ids || p.splits > 1) a.part = c.ws;
  if (c.ids) {
    a.t = c.ws + static_cast<int64_t>(p.splits) * n_proj * c.n * c.h_out;
    a.n_units = p.units;
  }
  if (c.glu) {
    switch (c.kind) {
      case WKind::kBf16: by_tokens<WKind::kBf16, 0, true>(a, p, s); break;
      case WKind::kFp8: by_tokens<WKind::kFp8, 0, true>(a, p, s); break;
      case WKind::kInt4: by_group<WKind::kInt4, true>(a, p, c.group, s); break;
      case WKind::kTable4: by_group<WKind::kTable4, true>(a, p, c.group, s); break;
    }
  } else if (c.kind == WKind::kInt4) {
    by_group<WKind::kInt4, false>(a, p, c.group, s);
  } else {
    by_group<WKind::kTable4, false>(a, p, c.group, s);
  }
  if (hipGetLastError() != hipSuccess) return LORA_ERR_HIP;
  if (a.part) {
    const dim3 grid((c.h_out + kFinishCols - 1) / kFinishCols, c.n);
    if (c.glu) hipLaunchKernelGGL((k_rows_finish<true>), grid, dim3(kFinishThreads), 0, s, a);
    else hipLaunchKernelGGL((k_rows_finish<false>), grid, dim3(kFinishThreads), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // namespace lora
