// Base products for short batches (decode): y^T = W^T x^T with W streamed once
// for every 64 tokens, and the adapters' shrink in the same launch.
//
// The weights are nearly all there is to read (2 n_tokens flops for each), so
// the kernels are streams of W^T rows (output columns), each lane reading 16
// bytes of one row at a time.  The products run on v_mfma_f32_16x16x32_bf16 with
// a 16-row block of W^T as the A operand and 16 tokens as the B operand: with
// few tokens most of the matrix work is on repeated columns, but the matrix cores
// are idle otherwise and the vector ALU is left to the widening of the codes.
// Up to 16 tokens whose x fits in LDS run on k_rows, whose waves split h_in;
// more on k_mid, whose waves each take rows of their own and share x.  Where the
// columns alone do not fill the GPU, workgroups split h_in too.  Waves' and
// splits' sums are added in their order, so the result does not depend on timing.
//
// 4-bit codes.  A lane's 16 bytes are 32 codes of one row; an exchange of
// words between the four lane groups (v_permlane32_swap, v_permlane16_swap: a
// 4 x 4 transpose) turns them into the A operands of four MFMAs over 32
// consecutive k each, so that every group of 32, 64 or 128 k is whole MFMAs.
// Those run on the codes' exact integers (or the codebook's values), and the
// group's sum is scaled once in fp32.  A zero point z enters as
// s (sum q x - z sum x), with the sum of x over the group formed beside it.
//
// Adapters.  t = s_a x A_a^T is the same kind of product with A's rank rows
// as the weights; its workgroups come first in the grid, one for each distinct
// adapter of a chunk's tokens and projection.  Base sums and t then go
// through the workspace to a second, small kernel (k_rows_finish) that adds t B,
// applies the gate and rounds once.  A call without adapters writes y from the
// first kernel unless h_in is split.
#pragma once

#include "base_args.hpp"

namespace lora {

constexpr int kRowsWaves = 8;
constexpr int kRowsThreads = 64 * kRowsWaves;
constexpr int kMidWaves = 8;       // waves of k_mid that multiply
constexpr int kMidMovers = 4;      // and that bring x
constexpr int kMidCols = 32 * kMidWaves;   // rows of W^T of a workgroup
constexpr int kMidThreads = 64 * (kMidWaves + kMidMovers);
constexpr int kRowsMaxPpr = kMaxFusedRowPages;   // A pages per rank row
constexpr int kRowsTRow = kMaxRank;

constexpr int kRowsXBytes = 64 * 1024;   // x in LDS: two workgroups to a CU

// Bytes from token to token of x in LDS: 16 more than the row, so that the
// tokens of one k start in different banks.
__host__ __device__ constexpr int rows_x_stride(int k) { return 2 * k + 16; }

struct RowsArgs {
  PoolView pv;
  WView w[2];             // one projection, or gate and up
  const __bf16* x;        // [n][ld_x]
  const int32_t* ids;     // [n] or null
  __bf16* y;              // [n][ld_y], written
  float* part;            // [split][projection][n][h_out] base sums, with adapters or several splits
  float* t;               // [projection][n][kRowsTRow] scaled shrink results, with adapters
  int64_t ld_x, ld_w, ld_y;   // ld_w in bytes
  int32_t n, h_in, h_out;
  int32_t module[2];
  int32_t act;
  int32_t n_units;        // shrink workgroups ahead of the base's (a multiple of 8)
  int32_t n_blocks;       // base workgroups of one split
  int32_t splits;         // of h_in, over workgroups (gridDim.z)
};

template <WKind WK> struct RowsLoad;   // one 16-byte load of a row, as MFMA A operands
template <> struct RowsLoad<WKind::kBf16> { static constexpr int kK = 32, kFrags = 1; };
template <> struct RowsLoad<WKind::kFp8> { static constexpr int kK = 64, kFrags = 2; };
template <> struct RowsLoad<WKind::kInt4> { static constexpr int kK = 128, kFrags = 4; };
template <> struct RowsLoad<WKind::kTable4> { static constexpr int kK = 128, kFrags = 4; };

__device__ __forceinline__ f32x4 rows_mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Loads written before this are issued before what follows: the compiler would
// otherwise move them down to their first use.
__device__ __forceinline__ void rows_issue() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Where the zero points are read: where there are none, from the scales (twice
// their bytes), and not used.  A load under a condition would make every step
// wait for the loads before it, as the other side writes the same register.
__device__ __forceinline__ const uint8_t* rows_zeros(const WView& w) {
  return w.zero ? w.zero : static_cast<const uint8_t*>(w.scale);
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

// The d-th distinct adapter (in order of first use) of a chunk whose lanes hold
// the tokens' ids: its id and the lanes that have it, or false.
__device__ __forceinline__ bool rows_distinct(int mine, bool valid, int d, int* id, uint64_t* same) {
  uint64_t left = __ballot(valid);
  for (; left != 0; --d) {
    *id = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    *same = __ballot(valid && mine == *id);
    if (d == 0) return true;
    left &= ~*same;
  }
  return false;
}

template <int T, int NW>   // 16-token blocks a pass over K takes at most, waves
struct RowsShrinkShared {
  int32_t pid[kMaxRank][kRowsMaxPpr];
  int32_t tok[kRowsTokens];
  f32x4 red[NW][T][64];
};

// t of the rbs 16-row blocks of adapter e from block rb0 on, for the n_tok tokens
// listed in sh.tok.  Each block goes to an equal share of the waves, which split
// h_in.
template <int T, int TM, int NW>
__device__ __forceinline__ void rows_shrink_entry(const RowsArgs& a, RowsShrinkShared<TM, NW>& sh, const SlotEntry& e,
                                                  int p, int rb0, int rbs, int tok0, int n_tok, int lane, int wave) {
  constexpr int U = T == 1 ? 8 : 4;
  const int l16 = lane & 15, lq = lane >> 4;
  const int h = static_cast<int>(a.pv.page_elems);
  const __bf16* pages = static_cast<const __bf16*>(a.pv.pages);
  const int share = NW / rbs, rb = wave / share, part = wave - rb * share;
  const int n32 = a.h_in >> 5;
  const int s0 = n32 * part / share, s1 = rb < rbs ? n32 * (part + 1) / share : s0;   // waves left over: nothing
  const int row = min(16 * rb + l16, kMaxRank - 1);
  int tok[T];
  const __bf16* xr[T];
  f32x4 acc[T];
#pragma unroll
  for (int tb = 0; tb < T; ++tb) {
    tok[tb] = sh.tok[min(16 * tb + l16, n_tok - 1)];
    xr[tb] = a.x + static_cast<int64_t>(tok0 + tok[tb]) * a.ld_x + 8 * lq;
    acc[tb] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  int kp = 32 * s0 / h, off = 32 * s0 - kp * h;
  for (int s = s0; s < s1; s += U) {
    u32x4 af[U];
    bf16x8 xf[U][T];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // past the wave's end the last step is read again and A counts as zero: a
      // branch around the products would pull the loads into it, one by one
      const int su = min(s + u, s1 - 1);
      af[u] = *reinterpret_cast<const u32x4*>(pages + static_cast<int64_t>(sh.pid[row][kp]) * h + off + 8 * lq);
#pragma unroll
      for (int tb = 0; tb < T; ++tb) xf[u][tb] = *reinterpret_cast<const bf16x8*>(xr[tb] + 32 * su);
      if (su + 1 < s1) {
        off += 32;
        if (off == h) { off = 0; ++kp; }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t live = s + u < s1 ? ~0u : 0u;
      const bf16x8 av = __builtin_bit_cast(bf16x8, af[u] & u32x4{live, live, live, live});
#pragma unroll
      for (int tb = 0; tb < T; ++tb) acc[tb] = rows_mfma(av, xf[u][tb], acc[tb]);
    }
  }
#pragma unroll
  for (int tb = 0; tb < T; ++tb) sh.red[wave][tb][lane] = acc[tb];
  __syncthreads();
  for (int it = wave; it < rbs * T; it += NW) {
    const int b = it / T, tb = it - b * T, i = 16 * tb + l16;
    if (i >= n_tok) continue;
    f32x4 v = sh.red[b * share][tb][lane];
    for (int w = 1; w < share; ++w) v += sh.red[b * share + w][tb][lane];
    float* to = a.t + (static_cast<int64_t>(p) * a.n + tok0 + sh.tok[i]) * kRowsTRow + 16 * (rb0 + b) + 4 * lq;
    *reinterpret_cast<f32x4*>(to) = v * e.scale;
  }
}

// Shrink unit `unit` of the chunk of tokens tok0 .. tok0 + m - 1: a distinct
// adapter and projection, or one 16-row block of it where the chunk has so few
// adapters that the grid's units go round (177 tokens in runs of 29, 4160 ->
// 5440, ranks up to 64: 49 us a call, 65 with whole adapters; 64 tokens, 64
// adapters of ranks 8 to 64, 2048 -> 2 x 8192: 34 us with whole adapters against
// 40 with a workgroup for each block).  Whole workgroup; false when the chunk has
// no such adapter (nor any later one).
template <int TM, int NW>
__device__ __forceinline__ bool rows_shrink(const RowsArgs& a, RowsShrinkShared<TM, NW>& sh, int unit, int n_proj,
                                            int tok0, int m) {
  // uniform: the matrix instructions ignore the execution mask, so what they
  // depend on must be a branch of the whole wave
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mine = lane < m ? a.ids[tok0 + lane] : -1;
  const bool valid = mine >= 0 && mine < a.pv.n_slots;
  int id;
  uint64_t same;
  int per = (a.pv.max_rank + 15) >> 4;   // units of an adapter and projection
  if (per > 1 && rows_distinct(mine, valid, a.n_units / (n_proj * per), &id, &same)) per = 1;
  const int d = unit / (n_proj * per), rest = unit - d * (n_proj * per);
  const int p = rest / per, rb0 = rest - p * per;
  if (!rows_distinct(mine, valid, d, &id, &same)) return false;
  const SlotEntry e = a.pv.entries[static_cast<int64_t>(id) * a.pv.n_modules + a.module[p]];
  const int rank = __builtin_amdgcn_readfirstlane(e.rank);   // uniform, as `wave` is
  const int rbs = per > 1 ? 1 : (rank + 15) >> 4;            // row blocks of this unit
  if (rank <= 16 * rb0) return true;
  const int n_tok = __popcll(same);
  if (wave == 0 && (same >> lane & 1)) sh.tok[__popcll(same & ((uint64_t(1) << lane) - 1))] = lane;
  const int ppr = a.h_in / static_cast<int>(a.pv.page_elems);
  for (int q = threadIdx.x; q < 16 * rbs * ppr; q += 64 * NW) {
    const int r = q / ppr, kp = q - r * ppr, j = 16 * rb0 + r;
    sh.pid[r][kp] = j < e.rank ? a.pv.page_ids[e.a_off + j * ppr + kp] : a.pv.zero_page;
  }
  __syncthreads();
  if (TM == 1 || n_tok <= 16) rows_shrink_entry<1, TM, NW>(a, sh, e, p, rb0, rbs, tok0, n_tok, lane, wave);
  else rows_shrink_entry<TM, TM, NW>(a, sh, e, p, rb0, rbs, tok0, n_tok, lane, wave);
  return true;
}

// The units of a chunk that workgroup `first` of its a.n_units takes.  (Where
// there is one unit to a workgroup, asking for another would cost 1 to 2 us: 64
// tokens, 4096 -> 4096, 17.9 against 16 us.)
template <int TM, int NW>
__device__ __forceinline__ void rows_shrink_all(const RowsArgs& a, RowsShrinkShared<TM, NW>& sh, int first, int n_proj,
                                                int tok0, int m) {
  const int most = min(m, a.pv.n_slots) * n_proj;
  for (int unit = first; rows_shrink<TM, NW>(a, sh, unit, n_proj, tok0, m);) {
    unit += a.n_units;
    if (unit >= most) break;
    __syncthreads();
  }
}

// t of every token of a long batch, for the tiled kernels.  A workgroup takes 64
// tokens and one split of h_in: x goes through LDS 256 k at a time (read once
// for up to kLsUnits units of 16 rank rows, in whole 256-byte runs: the 16-row
// fragments of x, 64 bytes a row at a power-of-two stride, read straight from
// memory took four times as long), wave w multiplies k 32 w .. + 32 of it by
// every unit's rows for all 64 tokens, and each unit's tokens are picked when
// t is written: [split][projection][n][kRowsTRow].
constexpr int kLsUnits = 4;
constexpr int kLsK = 256;

__global__ __launch_bounds__(kRowsThreads) void k_long_shrink(RowsArgs a, int n_proj) {
  struct Shared {
    union {
      alignas(16) unsigned char x[2][kRowsTokens * kLsK * 2];
      f32x4 red[kRowsWaves][4][64];
    };
    int32_t pid[kLsUnits][16][kRowsMaxPpr];
    int32_t unit_of[kLsUnits];     // id, projection and rank block of the pass's units
    int32_t unit_p[kLsUnits], unit_rb[kLsUnits];
  };
  __shared__ Shared sh;
  const int tok0 = blockIdx.x * kRowsTokens, m = min(a.n - tok0, kRowsTokens);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int h = static_cast<int>(a.pv.page_elems), ppr = a.h_in / h;
  const __bf16* pages = static_cast<const __bf16*>(a.pv.pages);
  const int steps = (a.h_in + kLsK - 1) / kLsK;
  const int s0 = steps * blockIdx.y / gridDim.y, s1 = steps * (blockIdx.y + 1) / gridDim.y;
  const int mine = lane < m ? a.ids[tok0 + lane] : -1;
  const bool valid = mine >= 0 && mine < a.pv.n_slots;
  uint64_t left = __ballot(valid);   // lanes whose adapters are still to come

  // x: thread moves pieces of 16 bytes, 32 threads to a token's 512 bytes
  const int xc = tid & 31;
  const __bf16* xsrc[4];
  int xdst[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int r = (tid >> 5) + 16 * q;
    xsrc[q] = a.x + static_cast<int64_t>(tok0 + min(r, m - 1)) * a.ld_x;
    xdst[q] = r * (2 * kLsK) + ((xc ^ (r & 15)) << 4);
  }
  u32x4 xr[4];
  auto load_x = [&](int s) {
    const int k = s * kLsK + 8 * xc;
#pragma unroll
    for (int q = 0; q < 4; ++q) xr[q] = *reinterpret_cast<const u32x4*>(xsrc[q] + (k < a.h_in ? k : 0));
  };
  auto store_x = [&](int s, int buf) {
    const bool in = s * kLsK + 8 * xc < a.h_in;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (!in) xr[q] = u32x4{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4*>(sh.x[buf] + xdst[q]) = xr[q];
    }
  };

  int p = 0, rb = 0;   // where the listing of units stands within the first adapter left
  for (;;) {
    // ---- the pass's units
    int n_units = 0;
    __syncthreads();   // the previous pass's reads are done
    while (left != 0 && n_units < kLsUnits) {
      const int id = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
      const int rank = a.pv.entries[static_cast<int64_t>(id) * a.pv.n_modules + a.module[p]].rank;
      if (16 * rb < rank) {
        if (tid == 0) {
          sh.unit_of[n_units] = id;
          sh.unit_p[n_units] = p;
          sh.unit_rb[n_units] = rb;
        }
        ++n_units;
        ++rb;
      } else {
        rb = 0;
        if (++p == n_proj) {
          p = 0;
          left &= ~__ballot(valid && mine == id);
        }
      }
    }
    if (n_units == 0) return;
    if (s0 < s1) load_x(s0);
    __syncthreads();
    for (int q = tid; q < n_units * 16 * ppr; q += kRowsThreads) {
      const int u = q / (16 * ppr), rest = q - u * 16 * ppr, r = rest / ppr, kp = rest - r * ppr;
      const SlotEntry e = a.pv.entries[static_cast<int64_t>(sh.unit_of[u]) * a.pv.n_modules + a.module[sh.unit_p[u]]];
      const int j = 16 * sh.unit_rb[u] + r;
      sh.pid[u][r][kp] = j < e.rank ? a.pv.page_ids[e.a_off + j * ppr + kp] : a.pv.zero_page;
    }
    if (s0 < s1) store_x(s0, 0);
    __syncthreads();

    // ---- the wave's k of the split
    f32x4 acc[kLsUnits][4];
#pragma unroll
    for (int u = 0; u < kLsUnits; ++u)
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) acc[u][tb] = f32x4{0.f, 0.f, 0.f, 0.f};
    bf16x8 af[kLsUnits];
    auto load_a = [&](int s) {
      const int k = min(s * kLsK + 32 * wave, a.h_in - 32);   // past the end x is zero
      const int kp = k / h, off = k - kp * h + 8 * lq;
#pragma unroll
      for (int u = 0; u < kLsUnits; ++u)
        af[u] = *reinterpret_cast<const bf16x8*>(
            pages + static_cast<int64_t>(sh.pid[min(u, n_units - 1)][l16][kp]) * h + off);
    };
    if (s0 < s1) load_a(s0);
    for (int s = s0; s < s1; ++s) {
      const int buf = (s - s0) & 1;
      bf16x8 av[kLsUnits];
#pragma unroll
      for (int u = 0; u < kLsUnits; ++u) av[u] = af[u];
      if (s + 1 < s1) {
        load_x(s + 1);
        load_a(s + 1);
      }
      rows_issue();
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const bf16x8 xf = *reinterpret_cast<const bf16x8*>(sh.x[buf] + (16 * tb + l16) * (2 * kLsK) +
                                                           (((4 * wave + lq) ^ l16) << 4));
#pragma unroll
        for (int u = 0; u < kLsUnits; ++u) acc[u][tb] = rows_mfma(av[u], xf, acc[u][tb]);
      }
      if (s + 1 < s1) store_x(s + 1, buf ^ 1);
      __syncthreads();
    }

    // ---- the waves' sums of each unit, in wave order
    for (int u = 0; u < n_units; ++u) {
#pragma unroll
      for (int v = 0; v < kLsUnits; ++v)
        if (u == v) {
#pragma unroll
          for (int tb = 0; tb < 4; ++tb) sh.red[wave][tb][lane] = acc[v][tb];
        }
      __syncthreads();
      if (wave < 4) {
        f32x4 v = sh.red[0][wave][lane];
#pragma unroll
        for (int w = 1; w < kRowsWaves; ++w) v += sh.red[w][wave][lane];
        const int tok = 16 * wave + l16, id = sh.unit_of[u], up = sh.unit_p[u];
        if (tok < m && a.ids[tok0 + tok] == id) {
          const float scale = a.pv.entries[static_cast<int64_t>(id) * a.pv.n_modules + a.module[up]].scale;
          const int64_t row = (static_cast<int64_t>(blockIdx.y) * n_proj + up) * a.n + tok0 + tok;
          *reinterpret_cast<f32x4*>(a.t + row * kRowsTRow + 16 * sh.unit_rb[u] + 4 * lq) = v * scale;
        }
      }
      __syncthreads();
    }
  }
}

// Four columns of a token's base sums of one projection, to the workspace.
__device__ __forceinline__ void rows_put_part(const RowsArgs& a, int n_proj, int p, int tok, int c, f32x4 v) {
  const int64_t row = static_cast<int64_t>(blockIdx.z * n_proj + p) * a.n + tok;
  *reinterpret_cast<f32x4*>(a.part + row * a.h_out + c) = v;
}

// Four columns of a token's output: v, or act(v) * up.
template <bool GLU>
__device__ __forceinline__ void rows_put(const RowsArgs& a, int tok, int c, f32x4 v, f32x4 up) {
  __bf16 o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = static_cast<__bf16>(GLU ? glu_act(a.act, v[e]) * up[e] : v[e]);
  *reinterpret_cast<u32x2*>(a.y + static_cast<int64_t>(tok) * a.ld_y + c) = __builtin_bit_cast(u32x2, o);
}

// Sixteen e4m3 codes' half h (8 codes) widened to bf16, exactly.
__device__ __forceinline__ bf16x8 rows_fp8(u32x4 v, int h) {
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * h + j], 1.0f, false);
    const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * h + j], 1.0f, true);
    o[2 * j] = __builtin_bit_cast(uint32_t, lo);
    o[2 * j + 1] = __builtin_bit_cast(uint32_t, hi);
  }
  return __builtin_bit_cast(bf16x8, o);
}

// Up to 16 tokens whose x fits in LDS.  WK: storage of W.  G: k of one 4-bit
// group (else 0).  CB: 16-row blocks of W^T a workgroup takes; with GLU half of
// them gate rows and half up rows of the same output columns.
//
// h_in is split between gridDim.z workgroups and their waves, each of which
// reads U loads of each of its rows one batch ahead of the products.  x waits
// in LDS: loads return in order, so x loaded in between would hold up W.
// Bound by the read of W: bf16, 1 token, 4096 -> 2 x 11264 36 us (5.1 TB/s);
// 4-bit with zero points, 1 token, 8192 -> 28672 35 us (3.5 TB/s, where the
// widening's and scaling's instructions are as long as the read); small layers
// by the launch (4-bit, 768 -> 768 5.4 us).
template <WKind WK, int G, int CB, bool GLU>
__global__ __launch_bounds__(kRowsThreads) void k_rows(RowsArgs a) {
  constexpr int F = RowsLoad<WK>::kFrags, KS = RowsLoad<WK>::kK;
  constexpr bool W4 = is_w4(WK);
  constexpr int NS = W4 ? 128 / G : 1;           // scales of one load
  constexpr int U = 8 / F > 4 ? 4 : 8 / F;       // loads of a row in one batch
  constexpr int NP = GLU ? 2 : 1;
  constexpr int CPB = CB / NP;                   // column blocks
  union Shared {
    RowsShrinkShared<1, kRowsWaves> shrink;
    f32x4 red[kRowsWaves][CB][64];
    unsigned char x[kRowsXBytes];
  };
  __shared__ Shared sh;
  const int m = a.n;   // at most 16
  if (static_cast<int>(blockIdx.x) < a.n_units) {
    if (blockIdx.z == 0) (void)rows_shrink<1, kRowsWaves>(a, sh.shrink, blockIdx.x, NP, 0, m);
    return;
  }
  // consecutive column blocks on one XCD, so that they share lines of the scales in its L2
  const int b = blockIdx.x - a.n_units, per = (a.n_blocks + 7) >> 3;
  const int blk = (b & 7) * per + (b >> 3);
  if (blk >= a.n_blocks) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int col0 = blk * (16 * CPB);
  auto proj = [](int cb) { return GLU ? cb & 1 : 0; };
  auto col = [&](int cb) { return col0 + 16 * (GLU ? cb >> 1 : cb); };

  const char* wp[CB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
    wp[cb] = static_cast<const char*>(a.w[proj(cb)].w) + static_cast<int64_t>(col(cb) + l16) * a.ld_w;
  W4Table tab[NP];
  if constexpr (WK == WKind::kTable4) {
#pragma unroll
    for (int p = 0; p < NP; ++p) tab[p].load(a.w[p].table);
  }

  const int steps = (a.h_in + KS - 1) / KS;
  const int parts = kRowsWaves * gridDim.z, part = kRowsWaves * blockIdx.z + wave;
  const int s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
  const int g0 = steps * (kRowsWaves * blockIdx.z) / parts;   // the workgroup's first step
  // a row's last load may reach past its end (h_in an odd multiple of 64 under
  // KS = 128): it is moved back into the row and x is zero there
  const int last = (W4 ? a.h_in / 2 : WK == WKind::kFp8 ? a.h_in : 2 * a.h_in) - 16;
  // With one group to a 128-k load, the load's words meet the k that the lane
  // itself holds (x is read at any offset); else the words are exchanged so
  // that each product covers 32 consecutive k.
  constexpr bool SWAP = W4 && G < 128;

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
            const WView& w = a.w[proj(cb)];
            const int64_t o = g * w.ld_scale + col(cb) + 4 * lq;
            t.s[u][j][cb] = *reinterpret_cast<const u32x2*>(static_cast<const __bf16*>(w.scale) + o);
            if constexpr (WK == WKind::kInt4) t.z[u][j][cb] = *reinterpret_cast<const uint32_t*>(rows_zeros(w) + o);
          }
        }
      }
    }
  };

  f32x4 acc[CB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb) acc[cb] = f32x4{0.f, 0.f, 0.f, 0.f};
  const f32x4 none{0.f, 0.f, 0.f, 0.f};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
  const int x_row = rows_x_stride((steps * (kRowsWaves * (blockIdx.z + 1)) / parts - g0) * KS);   // bytes

  auto compute = [&](const Batch& t, int u, int s) {
    bf16x8 xf[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int k = SWAP ? 32 * f + 8 * lq : 8 * F * lq + 8 * f;
      xf[f] = *reinterpret_cast<const bf16x8*>(sh.x + min(l16, m - 1) * x_row + 2 * ((s - g0) * KS + k));
    }
    if constexpr (!W4) {
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        const u32x4 v = t.w[u][cb];
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const bf16x8 wf = WK == WKind::kBf16 ? __builtin_bit_cast(bf16x8, v) : rows_fp8(v, f);
          acc[cb] = rows_mfma(wf, xf[f], acc[cb]);
        }
      }
    } else {
      f32x4 xs[NS];   // sum of x over each group: every row of the product with ones
      if constexpr (WK == WKind::kInt4) {
#pragma unroll
        for (int f = 0; f < 4; ++f)
          xs[f * NS / 4] = rows_mfma(ones, xf[f], f % (4 / NS) == 0 ? none : xs[f * NS / 4]);
      }
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        const u32x4 v = SWAP ? rows_transpose4(t.w[u][cb]) : t.w[u][cb];
        f32x4 sum;
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const bf16x8 wf = w4_widen<WK, true>(v[f], tab[proj(cb)]);
          sum = rows_mfma(wf, xf[f], f % (4 / NS) == 0 ? none : sum);
          if (f % (4 / NS) == 4 / NS - 1) {   // the group ends here: scale its sum
            const int j = f * NS / 4;
            const u32x2 s2 = t.s[u][j][cb];
            const f32x4 sc{bf16lo(s2.x), bf16hi(s2.x), bf16lo(s2.y), bf16hi(s2.y)};
            const uint32_t zw = WK == WKind::kInt4 && a.w[proj(cb)].zero ? t.z[u][j][cb] : 0x08080808u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float z = static_cast<float>((zw >> (8 * e)) & 0xFFu);
              float g = sum[e];
              if constexpr (WK == WKind::kInt4) g = fmaf(-z, xs[j][0], g);
              acc[cb][e] = fmaf(sc[e], g, acc[cb][e]);
            }
          }
        }
      }
    }
  };

  Batch cur, nxt;
  if (s0 < s1) load(cur, s0);
  {
    // x of the workgroup's k, in the order the widened codes come in; zero past h_in
    const int k0 = g0 * KS, len = steps * (kRowsWaves * (blockIdx.z + 1)) / parts * KS - k0;
    for (int i = threadIdx.x; i < m * (len >> 3); i += kRowsThreads) {
      const int r = i / (len >> 3), k = 8 * (i - r * (len >> 3));
      u32x4 v{0u, 0u, 0u, 0u};
      if (k0 + k < a.h_in)
        v = *reinterpret_cast<const u32x4*>(a.x + static_cast<int64_t>(r) * a.ld_x + k0 + k);
      if constexpr (WK == WKind::kInt4) v = w4_xl_order(v);
      *reinterpret_cast<u32x4*>(sh.x + r * x_row + 2 * k) = v;
    }
    __syncthreads();
  }
  int s = s0;
  for (; s + U <= s1; s += U) {
    if (s + U < s1) load(nxt, s + U);
#pragma unroll
    for (int u = 0; u < U; ++u) compute(cur, u, s + u);
    cur = nxt;
  }
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (s + u < s1) compute(cur, u, s + u);

  // ---- the waves' sums, in wave order
  __syncthreads();   // x is read: its place is the sums'
#pragma unroll
  for (int cb = 0; cb < CB; ++cb) sh.red[wave][cb][lane] = acc[cb];
  __syncthreads();
  auto total = [&](int cb, int l) {
    f32x4 v = sh.red[0][cb][l];
#pragma unroll
    for (int w = 1; w < kRowsWaves; ++w) v += sh.red[w][cb][l];
    if constexpr (WK == WKind::kFp8)
      v *= *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.w[proj(cb)].scale) + col(cb) + 4 * (l >> 4));
    return v;
  };
  if (a.part) {
    for (int it = threadIdx.x; it < CB * 64; it += kRowsThreads) {
      const int cb = it >> 6, l = it & 63, tok = l & 15;
      if (tok < m) rows_put_part(a, NP, proj(cb), tok, col(cb) + 4 * (l >> 4), total(cb, l));
    }
  } else {
    for (int it = threadIdx.x; it < CPB * 64; it += kRowsThreads) {
      const int cp = it >> 6, l = it & 63, tok = l & 15;
      if (tok < m)
        rows_put<GLU>(a, tok, col0 + 16 * cp + 4 * (l >> 4), total(NP * cp, l), total(NP * cp + NP - 1, l));
    }
  }
}

// More tokens, or an x past LDS: 16 * TB tokens to a workgroup, 8 waves of two
// 16-row blocks of W^T each, and 4 waves that bring x.  The 8 share x, 128 k at
// a time through two LDS buffers, so that its reads from L2 (two bytes a token
// and k for every workgroup) stay below W's, and read their own rows of W
// straight into registers, D - 1 steps ahead.  Loads return in order, so waves
// that waited for x would wait for all of W's steps too: that is why other waves
// bring it.  What bounds the kernel is a mix: the vector ALU issues in 39% of the
// SIMDs' cycles (MFMA busy 17%), and three waves to a SIMD, all that the registers
// allow, leave the rest to barriers and loads.  So the bringing waves also put x in
// the order the widening likes, form the sums of it that the zero points multiply
// and bring the scales, and a fragment of x that was read from LDS meets two
// blocks (33 tokens, 4-bit, 4096 -> 2 x 12288, without adapters: 30 to 31 us when
// tried; one block to a wave 34 to 42, 4 or 16 waves and other depths no better).  With GLU a wave takes a gate block and the up block of the
// same columns.  Measured: that case with zero points and adapters 29 us
// (1.8 TB/s of codes and scales).
//
// x in LDS: rows of 256 bytes whose 16-byte chunks are XORed with the row, so
// that the 16 rows of a fragment read cover all banks once.
template <WKind WK, int G, int TB, bool GLU>
__global__ __launch_bounds__(kMidThreads, 3) void k_mid(RowsArgs a) {
  constexpr int F = RowsLoad<WK>::kFrags, KS = 128;
  constexpr bool W4 = is_w4(WK), Z = WK == WKind::kInt4;
  constexpr int L = 4 / F;                       // loads of a row in one step
  constexpr int NS = W4 ? 128 / G : 1;           // scales of one step
  constexpr int CB = 2;
  constexpr int D = 3;                           // steps of W in registers
  constexpr int DX = 4;                          // steps of x in a moving thread's registers
  constexpr int NP = GLU ? 2 : 1;
  // With one group to a step, a 4-bit load's words meet the k that the lane
  // itself holds; else they are exchanged so that each product covers 32
  // consecutive k.
  constexpr bool SWAP = W4 && G < 128;
  struct Stage {
    alignas(16) unsigned char x[16 * TB * 256];
    float xs[Z ? NS : 1][Z ? 16 * TB : 1];
    u32x2 sc[W4 ? NS : 1][W4 ? kMidCols / 4 : 1];      // scales and zero points of the workgroup's W^T rows,
    uint32_t zp[Z ? NS : 1][Z ? kMidCols / 4 : 1];     // 4 rows to an element
  };
  union Shared {
    RowsShrinkShared<TB, kMidThreads / 64> shrink;
    Stage st[2];
  };
  __shared__ Shared sh;
  // the grid's first a.n_units workgroups of each chunk shrink; then come the
  // base's, an XCD's (every eighth) with all chunks of a column block side by
  // side, so that its L2 holds the block's W for them
  const int chunks = (a.n + 16 * TB - 1) / (16 * TB), per = (a.n_blocks + 7) >> 3;
  int b = blockIdx.x - a.n_units * chunks;
  if (b < 0) {
    const int chunk = blockIdx.x / a.n_units, at = chunk * 16 * TB;
    if (blockIdx.z == 0)
      rows_shrink_all<TB, kMidThreads / 64>(a, sh.shrink, blockIdx.x - chunk * a.n_units, NP, at,
                                            min(a.n - at, 16 * TB));
    return;
  }
  const int xcd = b & 7;
  b >>= 3;
  const int blk = xcd * per + b / chunks, tok0 = (b % chunks) * 16 * TB, m = min(a.n - tok0, 16 * TB);
  if (blk >= a.n_blocks) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  // the wave's output columns; may start past h_out: such a wave computes and does not store
  const int col0 = (blk * kMidWaves + wave) * (16 * CB / NP);
  auto proj = [](int cb) { return GLU ? cb : 0; };
  auto col = [&](int cb) { return GLU ? col0 : col0 + 16 * cb; };
  const char* wp[CB];   // uniform; lanes add 32-bit offsets
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
    wp[cb] = static_cast<const char*>(a.w[proj(cb)].w) + min(col(cb), a.h_out - 16) * a.ld_w;
  const uint32_t w_lane = static_cast<uint32_t>(l16 * a.ld_w) + 16 * lq;
  W4Table tab[NP];
  if constexpr (WK == WKind::kTable4) {
#pragma unroll
    for (int p = 0; p < NP; ++p) tab[p].load(a.w[p].table);
  }
  const int steps = (a.h_in + KS - 1) / KS, parts = gridDim.z;
  const int s0 = steps * blockIdx.z / parts, n_steps = steps * (blockIdx.z + 1) / parts - s0;
  // The column blocks start at different steps and wrap around: rows are a
  // power of two apart as a rule, so workgroups that walked h_in in step would
  // all read the same few memory channels at a time.
  const int turn = blk % max(n_steps, 1);
  auto step_at = [&](int i) {
    i = min(i, n_steps - 1) + turn;
    return s0 + (i < n_steps ? i : i - n_steps);
  };
  const int row_bytes = W4 ? a.h_in / 2 : WK == WKind::kFp8 ? a.h_in : 2 * a.h_in;

  struct Step {
    u32x4 w[L][CB];
  };
  // A step of 4-bit codes is half a line of each row, so the line has to stay for
  // the next step: plain loads (33 tokens, 4096 -> 2 x 12288 29 us, 33 with
  // streaming ones).  A step of 8 or 16 bits is whole lines: streaming, so that
  // the adapters' pages stay (64 tokens, 2048 -> 2 x 8192 fp8: the finish 12 us
  // against 14).
  auto load_w = [&](Step& t, int s) {
#pragma unroll
    for (int l = 0; l < L; ++l) {
      // a row's last load may reach past its end (h_in an odd multiple of 64): it
      // is moved back into the row, and x is zero there
      const int at = s * (64 * L) + 64 * l, over = max(at + 16 * lq + 16 - row_bytes, 0);
      const uint32_t off = w_lane + static_cast<uint32_t>(at - over);   // the row's start or later: no wrap
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) t.w[l][cb] = ld16<!W4>(reinterpret_cast<const u32x4*>(wp[cb] + off));
    }
  };
  if (wave >= kMidWaves) {
    // ---- x: thread mt of the moving waves takes chunk mt % 16 of rows mt / 16, + RP, ...
    constexpr int RP = 4 * kMidMovers, XP = 16 * TB / RP;
    const int mt = tid - 64 * kMidWaves, xchunk = mt & 15, xrow = mt >> 4;
    const __bf16* xsrc[XP];
#pragma unroll
    for (int q = 0; q < XP; ++q)
      xsrc[q] = a.x + static_cast<int64_t>(tok0 + min(xrow + RP * q, m - 1)) * a.ld_x + 8 * xchunk;
    u32x4 xr[DX][XP];
    // and of the step's scales element mt % 64 of group mt / 64
    const int sj = mt >> 6, sp = mt & 63;
    const int sproj = GLU ? sp >> 5 : 0;
    const int scol = min(GLU ? blk * (kMidCols / 2) + 4 * (sp & 31) : blk * kMidCols + 4 * sp, a.h_out - 4);
    const WView& sw = a.w[sproj];
    u32x2 sr[DX];
    uint32_t zr[DX];
    auto load_s = [&](int d, int s) {
      if (!W4 || sj >= NS) return;   // whole waves
      const int64_t o = static_cast<int64_t>(min(s * NS + sj, a.h_in / max(G, 1) - 1)) * sw.ld_scale + scol;
      sr[d] = *reinterpret_cast<const u32x2*>(static_cast<const __bf16*>(sw.scale) + o);
      if constexpr (Z) zr[d] = *reinterpret_cast<const uint32_t*>(rows_zeros(sw) + o);
    };
    auto store_s = [&](int d, Stage& st) {
      if (!W4 || sj >= NS) return;
      st.sc[sj][sp] = sr[d];
      if constexpr (Z) st.zp[sj][sp] = sw.zero ? zr[d] : 0x08080808u;
    };
    auto load_x = [&](u32x4 (&r)[XP], int s) {
      const int k = s * KS + 8 * xchunk < a.h_in ? s * KS : 0;
#pragma unroll
      for (int q = 0; q < XP; ++q) r[q] = *reinterpret_cast<const u32x4*>(xsrc[q] + k);
    };
    auto store_x = [&](const u32x4 (&r)[XP], int s, Stage& st) {
      const bool in = s * KS + 8 * xchunk < a.h_in;   // past h_in (the last step's second half): zero
#pragma unroll
      for (int q = 0; q < XP; ++q) {
        u32x4 v = r[q];
        if (!in) v = u32x4{0u, 0u, 0u, 0u};
        *reinterpret_cast<u32x4*>(st.x + (xrow + RP * q) * 256 + ((xchunk ^ ((xrow + RP * q) & 15)) << 4)) =
            Z ? w4_xl_order(v) : v;
        if constexpr (Z) {
          float f = ((bf16lo(v.x) + bf16hi(v.x)) + (bf16lo(v.y) + bf16hi(v.y))) +
                    ((bf16lo(v.z) + bf16hi(v.z)) + (bf16lo(v.w) + bf16hi(v.w)));
          f += xor_lane<1>(f);
          f += xor_lane<2>(f);
          if constexpr (G >= 64) f += xor_lane<4>(f);
          if constexpr (G >= 128) f += xor_lane<8>(f);
          if ((xchunk & (G / 8 - 1)) == 0) st.xs[xchunk / (G / 8)][xrow + RP * q] = f;
        }
      }
    };
#pragma unroll
    for (int d = 0; d < DX; ++d) {
      load_x(xr[d], step_at(d));
      load_s(d, step_at(d));
    }
    rows_issue();
    store_x(xr[0], step_at(0), sh.st[0]);
    store_s(0, sh.st[0]);
    for (int s = 0; s < n_steps; s += DX) {   // DX is even: buffers and ring slots come round together
#pragma unroll
      for (int i = 0; i < DX; ++i) {
        if (s + i >= n_steps) break;
        __syncthreads();   // x of step s + i is there; the other buffer's readers are done
        load_x(xr[i % DX], step_at(s + i + DX));
        load_s(i % DX, step_at(s + i + DX));
        rows_issue();
        store_x(xr[(i + 1) % DX], step_at(s + i + 1), sh.st[(i + 1) & 1]);   // past the end: not read
        store_s((i + 1) % DX, sh.st[(i + 1) & 1]);
      }
    }
    return;
  }

  f32x4 acc[CB][TB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) acc[cb][tb] = f32x4{0.f, 0.f, 0.f, 0.f};
  const f32x4 none{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](const Step& t, const Stage& st) {
    auto x_at = [&](int tb, int f) {
      const int chunk = F == 2 ? 8 * (f >> 1) + 2 * lq + (f & 1) : W4 && !SWAP ? 4 * lq + f : 4 * f + lq;
      return *reinterpret_cast<const bf16x8*>(st.x + (16 * tb + l16) * 256 + ((chunk ^ l16) << 4));
    };
    if constexpr (!W4) {
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        bf16x8 wf[CB];
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
          wf[cb] = WK == WKind::kBf16 ? __builtin_bit_cast(bf16x8, t.w[f / F][cb]) : rows_fp8(t.w[f / F][cb], f % F);
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
          const bf16x8 xf = x_at(tb, f);
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) acc[cb][tb] = rows_mfma(wf[cb], xf, acc[cb][tb]);
        }
      }
    } else {
      u32x4 v[CB];
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) v[cb] = SWAP ? rows_transpose4(t.w[0][cb]) : t.w[0][cb];
      f32x4 sum[CB][TB];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        bf16x8 wf[CB];
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) wf[cb] = w4_widen<WK, true>(v[cb][f], tab[proj(cb)]);
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
          const bf16x8 xf = x_at(tb, f);
#pragma unroll
          for (int cb = 0; cb < CB; ++cb)
            sum[cb][tb] = rows_mfma(wf[cb], xf, f % (4 / NS) == 0 ? none : sum[cb][tb]);
        }
        if (f % (4 / NS) == 4 / NS - 1) {   // the group ends here: scale its sum
          const int j = f * NS / 4;
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) {
            const int piece = GLU ? cb * (kMidCols / 8) + 4 * wave + lq : 8 * wave + 4 * cb + lq;
            const u32x2 s2 = st.sc[j][piece];
            const f32x4 sc{bf16lo(s2.x), bf16hi(s2.x), bf16lo(s2.y), bf16hi(s2.y)};
            f32x4 nz = none;
            if constexpr (Z) {
              const uint32_t zw = st.zp[j][piece];
#pragma unroll
              for (int e = 0; e < 4; ++e) nz[e] = -static_cast<float>((zw >> (8 * e)) & 0xFFu);
            }
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
              const float xs = Z ? st.xs[j][16 * tb + l16] : 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[cb][tb][e] =
                    fmaf(sc[e], Z ? fmaf(nz[e], xs, sum[cb][tb][e]) : sum[cb][tb][e], acc[cb][tb][e]);
            }
          }
        }
      }
    }
  };

  Step ring[D];
#pragma unroll
  for (int d = 0; d < D - 1; ++d) load_w(ring[d], step_at(d));
  constexpr int TURN = D % 2 ? 2 * D : D;   // ring slots and LDS buffers both come round
  for (int s = 0; s < n_steps; s += TURN) {
#pragma unroll
    for (int i = 0; i < TURN; ++i) {
      if (s + i >= n_steps) break;
      __syncthreads();
      load_w(ring[(i + D - 1) % D], step_at(s + i + D - 1));
      rows_issue();
      compute(ring[i % D], sh.st[i & 1]);
    }
  }

#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
    if constexpr (WK == WKind::kFp8) {
      const f32x4 sc = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.w[proj(cb)].scale) +
                                                       min(col(cb), a.h_out - 16) + 4 * lq);
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) acc[cb][tb] *= sc;
    }
#pragma unroll
  for (int tb = 0; tb < TB; ++tb) {
    if (16 * tb + l16 >= m) continue;
    const int tok = tok0 + 16 * tb + l16;
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      const int c = col(cb) + 4 * lq;
      if (c >= a.h_out) continue;
      if (a.part) rows_put_part(a, NP, proj(cb), tok, c, acc[cb][tb]);
      else if (!GLU || cb == 0) rows_put<GLU>(a, tok, c, acc[cb][tb], acc[CB - 1][tb]);
    }
  }
}

// y = base sums + t B (and the gate), rounded once.  A workgroup takes one token
// and kFinishCols columns; its four waves take every fourth rank row, 8 columns
// to a lane, so that a rank of 64 is two rounds of 8 rows for each wave, and
// their sums meet in LDS in wave order.  What bounds it is the chain of reads
// (id, entry, page ids, B), so the page ids and t of all rank rows are read at
// once and the projections' chains run side by side: 2.9 us for one token and
// 768 columns, 4.3 for 64 tokens of rank 16 and 4096, 12 for 64 of ranks 8 to 64
// and 2 x 8192.
constexpr int kFinishWaves = 4;
constexpr int kFinishThreads = 64 * kFinishWaves;
constexpr int kFinishCols = 64 * 8;
template <bool GLU>
__global__ __launch_bounds__(kFinishThreads) void k_rows_finish(RowsArgs a) {
  constexpr int NP = GLU ? 2 : 1;
  __shared__ f32x4 red[kFinishWaves][NP][2][64];
  const int tok = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = blockIdx.x * kFinishCols + 8 * lane;
  const bool in = c < a.h_out;   // h_out is a multiple of 64: all 8 columns or none
  const int id = a.ids ? a.ids[tok] : -1;
  f32x4 v[NP][2];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    v[p][0] = v[p][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    // the splits' sums: split z to wave z % kFinishWaves
    for (int z = wave; in && z < a.splits; z += kFinishWaves) {
      const f32x4* from = reinterpret_cast<const f32x4*>(
          a.part + (static_cast<int64_t>(z * NP + p) * a.n + tok) * a.h_out + c);
      v[p][0] += from[0];
      v[p][1] += from[1];
    }
  }
  if (in && id >= 0 && id < a.pv.n_slots) {
    const int h = static_cast<int>(a.pv.page_elems), ppr = a.h_out / h;
    const int cp = c / h, off = c - cp * h;
    const __bf16* pages = static_cast<const __bf16*>(a.pv.pages);
    SlotEntry e[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) e[p] = a.pv.entries[static_cast<int64_t>(id) * a.pv.n_modules + a.module[p]];
    const int most = max(e[0].rank, e[NP - 1].rank);
    constexpr int R = 8;   // rank rows of one round of a wave
    for (int j0 = wave; j0 < most; j0 += R * kFinishWaves) {
      int32_t pid[NP][R];
      float t[NP][R];
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int j = j0 + r * kFinishWaves;
          // rows past the rank read the zero page, whatever t is there counts as zero
          pid[p][r] = j < e[p].rank ? a.pv.page_ids[e[p].b_off + j * ppr + cp] : a.pv.zero_page;
          t[p][r] = j < e[p].rank ? a.t[(static_cast<int64_t>(p) * a.n + tok) * kRowsTRow + j] : 0.f;
        }
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        u32x4 b[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
          b[r] = *reinterpret_cast<const u32x4*>(pages + static_cast<int64_t>(pid[p][r]) * h + off);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[p][q >> 1][2 * (q & 1)] = fmaf(t[p][r], bf16lo(b[r][q]), v[p][q >> 1][2 * (q & 1)]);
            v[p][q >> 1][2 * (q & 1) + 1] = fmaf(t[p][r], bf16hi(b[r][q]), v[p][q >> 1][2 * (q & 1) + 1]);
          }
      }
    }
  }
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int q = 0; q < 2; ++q) red[wave][p][q][lane] = v[p][q];
  __syncthreads();
  if (wave >= 2 || !in) return;   // wave q writes columns 4 q .. + 4 of each lane's
  f32x4 o[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    o[p] = red[0][p][wave][lane];
#pragma unroll
    for (int w = 1; w < kFinishWaves; ++w) o[p] += red[w][p][wave][lane];
  }
  rows_put<GLU>(a, tok, c + 4 * wave, o[0], o[NP - 1]);
}

}  // namespace lora
