// C ABI of the base products with 4-bit weights and of the gated feed-forward
// product: argument checks and path selection.
#include <algorithm>
#include <cstdlib>

#include "base_launch.hpp"
#include "fused_gemm.hpp"
#include "pool.hpp"

using namespace lora;

namespace {

// Workspace that a call with ids needs at least: the parts of a cut batch run one
// after the other and share it.  (A shorter one than lora_fused_workspace_bytes
// only limits the split of h_in.)
size_t ws_need(const BatchCut& cut, int n_proj, int64_t h_in, int64_t h_out) {
  return std::max(cut.rows > 0 ? rows_bytes(1, n_proj, cut.rows, h_out) : 0,
                  cut.tiles > 0 ? tiles_ws_bytes(n_proj, cut.tiles, static_cast<int32_t>(h_in)) : 0);
}

BaseShape shape_of(const lora_pool* p, int32_t module, WKind kind, int n_proj, bool with_ids) {
  return BaseShape{kind, n_proj, static_cast<int32_t>(p->h_in[module]), static_cast<int32_t>(p->h_out[module]),
                   with_ids ? p->n_slots : 0, p->max_rank};
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Checks of everything but the weights, for one projection or a pair.
lora_status check_base(const lora_pool* p, const int32_t* module, int n_proj, const void* x, int64_t ld_x,
                       int32_t n_tokens, const void* y, int64_t ld_y) {
  if (!p || n_tokens < 0) return LORA_ERR_ARG;
  for (int i = 0; i < n_proj; ++i)
    if (module[i] < 0 || module[i] >= p->n_modules) return LORA_ERR_ARG;
  if (p->dtype != LORA_BF16) return LORA_ERR_DTYPE;
  const int64_t h_in = p->h_in[module[0]], h_out = p->h_out[module[0]];
  if (n_proj == 2 && (p->h_in[module[1]] != h_in || p->h_out[module[1]] != h_out)) return LORA_ERR_SHAPE;
  if (h_in / p->page_elems > kFgMaxPpr || p->n_slots > kFgMaxSlots) return LORA_ERR_SHAPE;
  if (!x || !y) return LORA_ERR_ARG;
  if (ld_x < h_in || ld_y < h_out) return LORA_ERR_ARG;
  // a tile's 256 rows of x are addressed with 32-bit byte offsets (widths are 2^20 at most in any pool)
  if (ld_x > (int64_t(1) << 22)) return LORA_ERR_SHAPE;
  if (!aligned(x, 16) || ld_x % 8 != 0 || !aligned(y, 8) || ld_y % 4 != 0) return LORA_ERR_ARG;
  return LORA_OK;
}

lora_status check_rows_of_w(const void* w, int64_t ld_bytes, int64_t row_bytes) {
  if (!w || !aligned(w, 16) || ld_bytes % 16 != 0 || ld_bytes < row_bytes) return LORA_ERR_ARG;
  return ld_bytes > (int64_t(1) << 23) ? LORA_ERR_SHAPE : LORA_OK;   // a tile's 256 rows: 32-bit offsets
}

lora_status check_w4(const lora_pool* p, int32_t module, const lora_w4* w) {
  if (!w) return LORA_ERR_ARG;
  const int64_t h_in = p->h_in[module], h_out = p->h_out[module];
  if (w->group != 32 && w->group != 64 && w->group != 128) return LORA_ERR_ARG;
  if (h_in % w->group != 0) return LORA_ERR_SHAPE;
  const lora_status st = check_rows_of_w(w->codes, w->ld_codes, h_in / 2);
  if (st != LORA_OK) return st;
  if (!w->scale || !aligned(w->scale, 8) || w->ld_scale % 4 != 0 || w->ld_scale < h_out) return LORA_ERR_ARG;
  if ((w->zero && w->table) || !aligned(w->zero, 4) || !aligned(w->table, 4)) return LORA_ERR_ARG;
  return LORA_OK;
}

WView view_of(const lora_w4* w) {
  return WView{w->codes, w->scale, w->zero, static_cast<const uint32_t*>(w->table), w->ld_scale};
}

// A call whose arguments passed: fills the shared fields and launches.
lora_status base_call(const lora_pool* p, BaseCall& c, const int32_t* module, const void* x, int64_t ld_x,
                      const int32_t* ids, int32_t n_tokens, void* y, int64_t ld_y, void* ws, size_t ws_bytes,
                      void* stream) {
  const int n_proj = c.glu ? 2 : 1;
  const int64_t h_out = p->h_out[module[0]];
  if (ws_bytes > 0 && (!ws || !aligned(ws, 16))) return LORA_ERR_ARG;
  if (n_tokens == 0) return LORA_OK;
  const int64_t h_in = p->h_in[module[0]];
  const BatchCut cut = cut_batch(shape_of(p, module[0], c.kind, n_proj, ids != nullptr), n_tokens);
  if (cut.tiles > 0 && !tiles_fit(c.glu, cut.tiles, static_cast<int32_t>(h_out))) return LORA_ERR_SHAPE;
  if (ids && ws_bytes < ws_need(cut, n_proj, h_in, h_out)) return LORA_ERR_WORKSPACE;
  DeviceGuard g(p->device);
  if (!g.ok) return LORA_ERR_HIP;
  c.pv = p->view();
  c.x = static_cast<const __bf16*>(x);
  c.ids = ids;
  c.y = static_cast<__bf16*>(y);
  c.ld_x = ld_x;
  c.ld_y = ld_y;
  c.n = n_tokens;
  c.h_in = static_cast<int32_t>(h_in);
  c.h_out = static_cast<int32_t>(h_out);
  c.module[0] = module[0];
  c.module[1] = module[n_proj - 1];
  c.ws = static_cast<float*>(ws);
  c.ws_bytes = ws_bytes;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (cut.tiles > 0) {
    c.n = cut.tiles;
    if (ids) {
      const lora_status st = launch_shrink(c, tiles_splits(c.n, c.h_in), s);
      if (st != LORA_OK) return st;
    }
    const lora_status st = launch_tiles(c, s);
    if (st != LORA_OK || cut.rows == 0) return st;
    c.x += cut.tiles * ld_x;
    c.y += cut.tiles * ld_y;
    if (ids) c.ids += cut.tiles;
  }
  c.n = cut.rows;
  return launch_rows(c, s);
}

bool bad_act(lora_act act) { return act != LORA_ACT_SILU && act != LORA_ACT_GELU && act != LORA_ACT_GELU_TANH; }

}  // namespace

extern "C" {

size_t lora_fused_workspace_bytes(const lora_pool* p, int32_t module, int32_t n_proj, int32_t n_tokens) {
  if (!p || module < 0 || module >= p->n_modules || n_proj < 1 || n_proj > 2 || n_tokens < 1) return 0;
  const int32_t h_in = static_cast<int32_t>(p->h_in[module]), h_out = static_cast<int32_t>(p->h_out[module]);
  size_t most = 0;   // over the kinds of weights and with or without ids, as the call is not known
  for (WKind kind : {WKind::kBf16, WKind::kFp8, WKind::kInt4})
    for (bool with_ids : {false, true}) {
      const BatchCut cut = cut_batch(shape_of(p, module, kind, n_proj, with_ids), n_tokens);
      if (cut.tiles > 0 && with_ids) most = std::max(most, tiles_ws_bytes(n_proj, cut.tiles, h_in));
      if (cut.rows > 0) most = std::max(most, rows_ws_bytes(kind, n_proj, cut.rows, with_ids ? p->n_slots : 0, h_in, h_out));
    }
  return most;
}

int32_t lora_fused_tile_tokens(const lora_pool* p, int32_t module, int32_t n_proj, int32_t w_bits, int32_t n_tokens,
                               int32_t with_ids) {
  if (!p || module < 0 || module >= p->n_modules || n_proj < 1 || n_proj > 2 || n_tokens < 0 ||
      (w_bits != 4 && w_bits != 8 && w_bits != 16))
    return -1;
  const WKind kind = w_bits == 4 ? WKind::kInt4 : w_bits == 8 ? WKind::kFp8 : WKind::kBf16;
  return cut_batch(shape_of(p, module, kind, n_proj, with_ids != 0), n_tokens).tiles;
}

lora_status lora_fused_gemm_w4(const lora_pool* p, int32_t module, const void* x, int64_t ld_x, const lora_w4* w,
                               const int32_t* ids, int32_t n_tokens, void* y, int64_t ld_y, void* ws,
                               size_t ws_bytes, void* stream) {
  lora_status st = check_base(p, &module, 1, x, ld_x, n_tokens, y, ld_y);
  if (st == LORA_OK) st = check_w4(p, module, w);
  if (st != LORA_OK) return st;
  BaseCall c{};
  c.kind = w->table ? WKind::kTable4 : WKind::kInt4;
  c.group = w->group;
  c.w[0] = view_of(w);
  c.ld_w = w->ld_codes;
  return base_call(p, c, &module, x, ld_x, ids, n_tokens, y, ld_y, ws, ws_bytes, stream);
}

lora_status lora_fused_glu(const lora_pool* p, int32_t module_gate, int32_t module_up, const void* x, int64_t ld_x,
                           const void* w_gate, const void* w_up, int64_t ld_w, const int32_t* ids, int32_t n_tokens,
                           lora_act act, void* h, int64_t ld_h, void* ws, size_t ws_bytes, void* stream) {
  const int32_t module[2] = {module_gate, module_up};
  lora_status st = check_base(p, module, 2, x, ld_x, n_tokens, h, ld_h);
  if (st != LORA_OK) return st;
  if (bad_act(act) || ld_w < 0 || ld_w > (int64_t(1) << 40)) return LORA_ERR_ARG;
  for (const void* w : {w_gate, w_up}) {
    st = check_rows_of_w(w, 2 * ld_w, 2 * p->h_in[module_gate]);
    if (st != LORA_OK) return st;
  }
  BaseCall c{};
  c.kind = WKind::kBf16;
  c.glu = true;
  c.act = act;
  c.w[0].w = w_gate;
  c.w[1].w = w_up;
  c.ld_w = 2 * ld_w;
  return base_call(p, c, module, x, ld_x, ids, n_tokens, h, ld_h, ws, ws_bytes, stream);
}

lora_status lora_fused_glu_fp8w(const lora_pool* p, int32_t module_gate, int32_t module_up, const void* x,
                                int64_t ld_x, const void* w8_gate, const void* w8_up, int64_t ld_w,
                                const float* scale_gate, const float* scale_up, const int32_t* ids, int32_t n_tokens,
                                lora_act act, void* h, int64_t ld_h, void* ws, size_t ws_bytes, void* stream) {
  const int32_t module[2] = {module_gate, module_up};
  lora_status st = check_base(p, module, 2, x, ld_x, n_tokens, h, ld_h);
  if (st != LORA_OK) return st;
  if (bad_act(act)) return LORA_ERR_ARG;
  for (const void* w : {w8_gate, w8_up}) {
    st = check_rows_of_w(w, ld_w, p->h_in[module_gate]);
    if (st != LORA_OK) return st;
  }
  if (!scale_gate || !scale_up || !aligned(scale_gate, 16) || !aligned(scale_up, 16)) return LORA_ERR_ARG;
  BaseCall c{};
  c.kind = WKind::kFp8;
  c.glu = true;
  c.act = act;
  c.w[0].w = w8_gate;
  c.w[1].w = w8_up;
  c.w[0].scale = scale_gate;
  c.w[1].scale = scale_up;
  c.ld_w = ld_w;
  return base_call(p, c, module, x, ld_x, ids, n_tokens, h, ld_h, ws, ws_bytes, stream);
}

lora_status lora_fused_glu_w4(const lora_pool* p, int32_t module_gate, int32_t module_up, const void* x, int64_t ld_x,
                              const lora_w4* gate, const lora_w4* up, const int32_t* ids, int32_t n_tokens,
                              lora_act act, void* h, int64_t ld_h, void* ws, size_t ws_bytes, void* stream) {
  const int32_t module[2] = {module_gate, module_up};
  lora_status st = check_base(p, module, 2, x, ld_x, n_tokens, h, ld_h);
  if (st != LORA_OK) return st;
  if (bad_act(act)) return LORA_ERR_ARG;
  for (const lora_w4* w : {gate, up}) {
    st = check_w4(p, module_gate, w);
    if (st != LORA_OK) return st;
  }
  if (gate->group != up->group || gate->ld_codes != up->ld_codes || (gate->table != nullptr) != (up->table != nullptr))
    return LORA_ERR_SHAPE;
  BaseCall c{};
  c.kind = gate->table ? WKind::kTable4 : WKind::kInt4;
  c.group = gate->group;
  c.glu = true;
  c.act = act;
  c.w[0] = view_of(gate);
  c.w[1] = view_of(up);
  c.ld_w = gate->ld_codes;
  return base_call(p, c, module, x, ld_x, ids, n_tokens, h, ld_h, ws, ws_bytes, stream);
}

}  // extern "C"
