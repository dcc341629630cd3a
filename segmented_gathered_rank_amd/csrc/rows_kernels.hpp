// Base product for few tokens (decode): y^T = W^T x^T streamed once over W,
// with the adapters' shrink in the same launch.
//
// The weights are all there is to read (n_tokens flops pairs for each), so the
// kernel is a stream of W^T rows: a workgroup takes 16 * CB rows (output
// columns), its 8 waves split h_in between them, and each lane reads 16 bytes
// of one row at a time.  The products run on v_mfma_f32_16x16x32_bf16 with a
// W^T row block as the A operand and 16 tokens as the B operand: with few
// tokens most of the matrix work is on repeated columns, but the matrix cores
// are idle otherwise and the vector ALU is left to the widening of the codes.
// The waves' sums meet in LDS, in wave order, so the result does not depend
// on timing.
//
// 4-bit codes.  A lane's 16 bytes are 32 codes of one row; an exchange of
// words between the four lane groups (v_permlane32_swap, v_permlane16_swap: a
// 4 x 4 transpose) turns them into the A operands of four MFMAs over 32
// consecutive k each, so that every group of 32, 64 or 128 k is whole MFMAs.
// Those run on the codes' exact integers (or the codebook's values), and the
// group's sum is scaled once in fp32.  A zero point z enters as
// s (sum q x - z sum x), with sum x from one more MFMA whose A operand is
// all ones.
//
// Adapters.  t = s_a x A_a^T is the same kind of product with A's rank rows
// as the weights; its workgroups come first in the grid, one for each
// 16-row block of each token's adapter (the first token of an adapter does
// the work for all of the batch's tokens that share it; the others' leave at
// once).  Base sums and t then go through the workspace to a second, small
// kernel that adds t B, applies the gate and rounds once.
#pragma once

#include "base_args.hpp"

namespace lora {

constexpr int kRowsWaves = 8;
constexpr int kRowsThreads = 64 * kRowsWaves;
constexpr int kRowsTokens = 64;    // tokens of one workgroup; longer batches run as chunks of this many
constexpr int kRowsMaxPpr = 32;    // A pages per rank row
constexpr int kRowsTRow = kMaxRank;

struct RowsArgs {
  PoolView pv;
  WView w[2];             // one projection, or gate and up
  const __bf16* x;        // [n][ld_x]
  const int32_t* ids;     // [n] or null
  __bf16* y;              // [n][ld_y], written
  float* part;            // [projection][n][h_out] base sums, with adapters
  float* t;               // [projection][n][kRowsTRow] scaled shrink results, with adapters
  int64_t ld_x, ld_w, ld_y;   // ld_w in bytes
  int32_t n, h_in, h_out;
  int32_t module[2];
  int32_t act;
  int32_t n_units;        // shrink workgroups ahead of the base's (a multiple of 8)
  int32_t n_blocks;       // base workgroups
};

template <WKind WK> struct RowsLoad;   // one 16-byte load of a row, as MFMA A operands
template <> struct RowsLoad<WKind::kBf16> { static constexpr int kK = 32, kFrags = 1; };
template <> struct RowsLoad<WKind::kFp8> { static constexpr int kK = 64, kFrags = 2; };
template <> struct RowsLoad<WKind::kInt4> { static constexpr int kK = 128, kFrags = 4; };
template <> struct RowsLoad<WKind::kTable4> { static constexpr int kK = 128, kFrags = 4; };

__device__ __forceinline__ f32x4 rows_mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Word f of lane group q becomes word q of lane group f.
__device__ __forceinline__ u32x4 rows_transpose4(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{static_cast<uint32_t>(c[0]), static_cast<uint32_t>(c[1]), static_cast<uint32_t>(d[0]),
               static_cast<uint32_t>(d[1])};
}

struct RowsShrinkShared {
  int32_t pid[16][kRowsMaxPpr];
  int32_t tok[kRowsTokens];
  f32x4 red[kRowsWaves][64];
};

// t of one 16-row block of the adapter of token `tok0 + i`, for every token of
// the chunk with that adapter.  Whole workgroup; returns early where another
// unit does the work.
__device__ __forceinline__ void rows_shrink(const RowsArgs& a, RowsShrinkShared& sh, int unit, int n_proj, int tok0,
                                            int m) {
  // uniform: the matrix instructions ignore the execution mask, so what they
  // depend on must be a branch of the whole wave
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rbs = (a.pv.max_rank + 15) >> 4;
  const int i = unit / (n_proj * rbs), rest = unit - i * (n_proj * rbs);
  const int p = rest / rbs, rb = rest - p * rbs;
  if (i >= m) return;
  const int mine = lane < m ? a.ids[tok0 + lane] : -1;
  const int id = __builtin_amdgcn_readlane(mine, i);
  if (id < 0 || id >= a.pv.n_slots) return;
  const uint64_t same = __ballot(mine == id);
  if ((same & ((uint64_t(1) << i) - 1)) != 0) return;   // an earlier token's unit does it
  const SlotEntry e = a.pv.entries[static_cast<int64_t>(id) * a.pv.n_modules + a.module[p]];
  if (e.rank <= 16 * rb) return;
  const int n_tok = __popcll(same);
  if (wave == 0 && mine == id) sh.tok[__popcll(same & ((uint64_t(1) << lane) - 1))] = lane;
  const int h = static_cast<int>(a.pv.page_elems), ppr = a.h_in / h;
  for (int q = threadIdx.x; q < 16 * ppr; q += kRowsThreads) {
    const int r = q / ppr, kp = q - r * ppr, j = 16 * rb + r;
    sh.pid[r][kp] = j < e.rank ? a.pv.page_ids[e.a_off + j * ppr + kp] : a.pv.zero_page;
  }
  __syncthreads();
  const int l16 = lane & 15, lq = lane >> 4;
  const __bf16* pages = static_cast<const __bf16*>(a.pv.pages);
  const int n32 = a.h_in >> 5;
  const int s0 = n32 * wave / kRowsWaves, s1 = n32 * (wave + 1) / kRowsWaves;
  for (int tb = 0; 16 * tb < n_tok; ++tb) {
    const int tok = sh.tok[min(16 * tb + l16, n_tok - 1)];
    const __bf16* xr = a.x + static_cast<int64_t>(tok0 + tok) * a.ld_x + 8 * lq;
    f32x4 acc{0.f, 0.f, 0.f, 0.f};
    int kp = 32 * s0 / h, off = 32 * s0 - kp * h;
    constexpr int U = 8;
    for (int s = s0; s < s1; s += U) {
      bf16x8 af[U], xf[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // past the wave's end the last step is read again and not used
        const int su = min(s + u, s1 - 1);
        const __bf16* ap = pages + static_cast<int64_t>(sh.pid[l16][kp]) * h + off + 8 * lq;
        af[u] = *reinterpret_cast<const bf16x8*>(ap);
        xf[u] = *reinterpret_cast<const bf16x8*>(xr + 32 * su);
        if (su + 1 < s1) {
          off += 32;
          if (off == h) { off = 0; ++kp; }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s + u < s1) acc = rows_mfma(af[u], xf[u], acc);
    }
    sh.red[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
      f32x4 v = sh.red[0][lane];
#pragma unroll
      for (int w = 1; w < kRowsWaves; ++w) v += sh.red[w][lane];
      if (16 * tb + l16 < n_tok) {
        float* to = a.t + (static_cast<int64_t>(p) * a.n + tok0 + tok) * kRowsTRow + 16 * rb + 4 * lq;
        *reinterpret_cast<f32x4*>(to) = v * e.scale;
      }
    }
    __syncthreads();
  }
}

// WK: storage of W.  G: k of one 4-bit group (else 0).  TB: 16-token blocks.
// CB: 16-row blocks of W^T a workgroup takes; with GLU half of them gate
// rows and half up rows of the same output columns.
template <WKind WK, int G, int TB, int CB, bool GLU>
__global__ __launch_bounds__(kRowsThreads) void k_rows(RowsArgs a) {
  constexpr int F = RowsLoad<WK>::kFrags, KS = RowsLoad<WK>::kK;
  constexpr bool W4 = is_w4(WK);
  constexpr int NS = W4 ? 128 / G : 1;           // scales of one load
  constexpr int U = W4 && G == 32 ? 2 : 4;       // loads of each row in flight, twice over
  constexpr int NP = GLU ? 2 : 1;
  constexpr int CPB = CB / NP;                   // column blocks
  union Shared {
    RowsShrinkShared shrink;
    f32x4 red[kRowsWaves][CB * TB][64];
  };
  __shared__ Shared sh;
  const int tok0 = blockIdx.y * kRowsTokens, m = min(a.n - tok0, kRowsTokens);
  if (static_cast<int>(blockIdx.x) < a.n_units) {
    rows_shrink(a, sh.shrink, blockIdx.x, NP, tok0, m);
    return;
  }
  // consecutive column blocks on one XCD, so that they share lines of the scales in its L2
  const int b = blockIdx.x - a.n_units, per = (a.n_blocks + 7) >> 3;
  const int blk = (b & 7) * per + (b >> 3);
  if (blk >= a.n_blocks) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int col0 = blk * (16 * CPB);

  const char* wp[CB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
    wp[cb] = static_cast<const char*>(a.w[GLU ? cb & 1 : 0].w) +
             static_cast<int64_t>(col0 + 16 * (GLU ? cb >> 1 : cb) + l16) * a.ld_w;
  const __bf16* xp[TB];
#pragma unroll
  for (int tb = 0; tb < TB; ++tb) xp[tb] = a.x + static_cast<int64_t>(tok0 + min(16 * tb + l16, m - 1)) * a.ld_x;
  W4Table tab[NP];
  if constexpr (WK == WKind::kTable4) {
#pragma unroll
    for (int p = 0; p < NP; ++p) tab[p].load(a.w[p].table);
  }

  const int steps = (a.h_in + KS - 1) / KS;
  const int s0 = steps * wave / kRowsWaves, s1 = steps * (wave + 1) / kRowsWaves;
  // a row's last load may reach past its end (h_in an odd multiple of 64 under
  // KS = 128): it is moved back into the row and x is zero there
  const int last = (W4 ? a.h_in / 2 : WK == WKind::kFp8 ? a.h_in : 2 * a.h_in) - 16;

  struct Batch {
    u32x4 w[U][CB];
    u32x2 s[W4 ? U : 1][NS][W4 ? CB : 1];
    uint32_t z[W4 ? U : 1][NS][W4 ? CB : 1];
  };
  auto load = [&](Batch& t, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int su = min(s + u, s1 - 1);
      const int at = min(su * 64 + 16 * lq, last);
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) t.w[u][cb] = ld16<true>(reinterpret_cast<const u32x4*>(wp[cb] + at));
      if constexpr (W4) {
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const int g = min(su * NS + j, a.h_in / G - 1);
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) {
            const WView& w = a.w[GLU ? cb & 1 : 0];
            const int64_t o = g * w.ld_scale + col0 + 16 * (GLU ? cb >> 1 : cb) + 4 * lq;
            t.s[u][j][cb] = *reinterpret_cast<const u32x2*>(static_cast<const __bf16*>(w.scale) + o);
            if (G < 128 && su * NS + j > g) t.s[u][j][cb] = u32x2{0u, 0u};   // past the last group
            t.z[u][j][cb] = 0x08080808u;
            if (WK == WKind::kInt4 && w.zero) t.z[u][j][cb] = *reinterpret_cast<const uint32_t*>(w.zero + o);
          }
        }
      }
    }
  };

  f32x4 acc[CB][TB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) acc[cb][tb] = f32x4{0.f, 0.f, 0.f, 0.f};
  const f32x4 none{0.f, 0.f, 0.f, 0.f};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});

  auto compute = [&](const Batch& t, int u, int s) {
    // x of this load: F pieces of 8 k
    bf16x8 xf[F][TB];
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int k = W4 ? s * KS + 32 * f + 8 * lq : s * KS + 8 * F * lq + 8 * f;
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
        if constexpr (W4) {
          const bool in = k < a.h_in;
          u32x4 v = *reinterpret_cast<const u32x4*>(xp[tb] + (in ? k : 0));
          if (!in) v = u32x4{0u, 0u, 0u, 0u};
          xf[f][tb] = __builtin_bit_cast(bf16x8, v);
        } else {
          xf[f][tb] = *reinterpret_cast<const bf16x8*>(xp[tb] + k);
        }
      }
    }
    if constexpr (!W4) {
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        const u32x4 v = t.w[u][cb];
        if constexpr (WK == WKind::kBf16) {
#pragma unroll
          for (int tb = 0; tb < TB; ++tb)
            acc[cb][tb] = rows_mfma(__builtin_bit_cast(bf16x8, v), xf[0][tb], acc[cb][tb]);
        } else {
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            u32x4 o;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * f + j], 1.0f, false);
              const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * f + j], 1.0f, true);
              o[2 * j] = __builtin_bit_cast(uint32_t, lo);
              o[2 * j + 1] = __builtin_bit_cast(uint32_t, hi);
            }
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
              acc[cb][tb] = rows_mfma(__builtin_bit_cast(bf16x8, o), xf[f][tb], acc[cb][tb]);
          }
        }
      }
    } else {
      f32x4 xs[NS][TB];   // sum of x over each group: every row of the product with ones
      if constexpr (WK == WKind::kInt4) {
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int tb = 0; tb < TB; ++tb)
            xs[f * NS / 4][tb] = rows_mfma(ones, xf[f][tb], f % (4 / NS) == 0 ? none : xs[f * NS / 4][tb]);
      }
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        const u32x4 v = rows_transpose4(t.w[u][cb]);
        f32x4 sum[TB];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const bf16x8 wf = w4_widen<WK>(v[f], tab[GLU ? cb & 1 : 0]);
#pragma unroll
          for (int tb = 0; tb < TB; ++tb)
            sum[tb] = rows_mfma(wf, xf[f][tb], f % (4 / NS) == 0 ? none : sum[tb]);
          if (f % (4 / NS) == 4 / NS - 1) {   // the group ends here: scale its sum
            const int j = f * NS / 4;
            const u32x2 s2 = t.s[u][j][cb];
            const f32x4 sc{bf16lo(s2.x), bf16hi(s2.x), bf16lo(s2.y), bf16hi(s2.y)};
            const uint32_t zw = t.z[u][j][cb];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float z = static_cast<float>((zw >> (8 * e)) & 0xFFu);
#pragma unroll
              for (int tb = 0; tb < TB; ++tb) {
                float g = sum[tb][e];
                if constexpr (WK == WKind::kInt4) g = fmaf(-z, xs[j][tb][0], g);
                acc[cb][tb][e] = fmaf(sc[e], g, acc[cb][tb][e]);
              }
            }
          }
        }
      }
    }
  };

  if (s0 < s1) {
    Batch cur, nxt;
    load(cur, s0);
    for (int s = s0; s < s1; s += U) {
      if (s + U < s1) load(nxt, s + U);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s + u < s1) compute(cur, u, s + u);
      cur = nxt;
    }
  }

  // ---- the waves' sums, in wave order
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) sh.red[wave][cb * TB + tb][lane] = acc[cb][tb];
  __syncthreads();
  auto total = [&](int cb, int tb, int l) {
    f32x4 v = sh.red[0][cb * TB + tb][l];
#pragma unroll
    for (int w = 1; w < kRowsWaves; ++w) v += sh.red[w][cb * TB + tb][l];
    if constexpr (WK == WKind::kFp8) {
      const int c = col0 + 16 * (GLU ? cb >> 1 : cb) + 4 * (l >> 4);
      v *= *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.w[GLU ? cb & 1 : 0].scale) + c);
    }
    return v;
  };
  if (a.part) {
    for (int it = threadIdx.x; it < CB * TB * 64; it += kRowsThreads) {
      const int cb = it / (TB * 64), tb = (it >> 6) % TB, l = it & 63;
      const int tok = 16 * tb + (l & 15), c = col0 + 16 * (GLU ? cb >> 1 : cb) + 4 * (l >> 4);
      if (tok < m) {
        float* to = a.part + (static_cast<int64_t>(GLU ? cb & 1 : 0) * a.n + tok0 + tok) * a.h_out + c;
        *reinterpret_cast<f32x4*>(to) = total(cb, tb, l);
      }
    }
  } else {
    for (int it = threadIdx.x; it < CPB * TB * 64; it += kRowsThreads) {
      const int cp = it / (TB * 64), tb = (it >> 6) % TB, l = it & 63;
      const int tok = 16 * tb + (l & 15), c = col0 + 16 * cp + 4 * (l >> 4);
      if (tok < m) {
        f32x4 v = total(GLU ? 2 * cp : cp, tb, l);
        if constexpr (GLU) {
          const f32x4 up = total(2 * cp + 1, tb, l);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = glu_act(a.act, v[e]) * up[e];
        }
        __bf16 o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = static_cast<__bf16>(v[e]);
        *reinterpret_cast<u32x2*>(a.y + (tok0 + static_cast<int64_t>(tok)) * a.ld_y + c) =
            __builtin_bit_cast(u32x2, o);
      }
    }
  }
}

// y = base sums + t B (and the gate), rounded once.  One thread per token and
// 4 columns; a token's rank rows are read 8 at a time.
constexpr int kFinishThreads = 128;
template <bool GLU>
__global__ __launch_bounds__(kFinishThreads) void k_rows_finish(RowsArgs a) {
  constexpr int NP = GLU ? 2 : 1;
  const int tok = blockIdx.y;
  const int c = 4 * (blockIdx.x * kFinishThreads + threadIdx.x);
  if (c >= a.h_out) return;
  const int id = a.ids[tok];
  f32x4 v[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p)
    v[p] = *reinterpret_cast<const f32x4*>(a.part + (static_cast<int64_t>(p) * a.n + tok) * a.h_out + c);
  if (id >= 0 && id < a.pv.n_slots) {
    const int h = static_cast<int>(a.pv.page_elems), ppr = a.h_out / h;
    const int cp = c / h, off = c - cp * h;
    const __bf16* pages = static_cast<const __bf16*>(a.pv.pages);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const SlotEntry e = a.pv.entries[static_cast<int64_t>(id) * a.pv.n_modules + a.module[p]];
      const float* t = a.t + (static_cast<int64_t>(p) * a.n + tok) * kRowsTRow;
      for (int j0 = 0; j0 < e.rank; j0 += 8) {
        u32x2 b[8];
        float tj[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int jj = min(j0 + j, e.rank - 1);
          const int pid = a.pv.page_ids[e.b_off + jj * ppr + cp];
          b[j] = *reinterpret_cast<const u32x2*>(pages + static_cast<int64_t>(pid) * h + off);
          tj[j] = t[jj];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < e.rank) {
            v[p][0] = fmaf(tj[j], bf16lo(b[j].x), v[p][0]);
            v[p][1] = fmaf(tj[j], bf16hi(b[j].x), v[p][1]);
            v[p][2] = fmaf(tj[j], bf16lo(b[j].y), v[p][2]);
            v[p][3] = fmaf(tj[j], bf16hi(b[j].y), v[p][3]);
          }
      }
    }
  }
  __bf16 o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = static_cast<__bf16>(GLU ? glu_act(a.act, v[0][e]) * v[NP - 1][e] : v[0][e]);
  *reinterpret_cast<u32x2*>(a.y + static_cast<int64_t>(tok) * a.ld_y + c) = __builtin_bit_cast(u32x2, o);
}

}  // namespace lora
