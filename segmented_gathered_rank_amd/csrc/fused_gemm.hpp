// Base product and adapter term in one matrix-core kernel:
//   y_i = x_i W + s_a (x_i A_a^T) B_a
// for a batch whose tokens come in runs of one adapter, such as prefills.
// The study page's section "The kernel trick: gather, do not merge" runs the
// shared base matmul once and then applies each adapter's low-rank update; its
// FLOP count puts the update at about 2r/d of the base.  Computing both in one
// pass over x gets close to that: the shrink reads the x tiles the base
// product has already staged, and the expand adds into the base accumulators
// before y is written once.
//
// Tile: 256 tokens x 256 output columns, 8 waves, each 128 tokens x 64
// columns, on v_mfma_f32_16x16x32_bf16 with fp32 accumulation.  The product
// is formed transposed (Y^T = W^T X^T: the A operand is a row of W^T, the B
// operand a token row of x), so each lane's four accumulators are four
// consecutive output columns of one token, stored as one 8-byte write.  K
// advances 64 per step through two LDS buffers; global_load_lds moves the x,
// W^T and adapter-A tiles straight from memory into LDS (no register
// staging), 16-byte chunks XOR-swizzled by row so fragment reads are
// conflict-free.  The next step's loads are in flight while the current
// step's MFMAs run.
//
// Adapter units.  At tile start the workgroup collects the distinct adapters
// of its 256 tokens (ascending slot order) and cuts each into units of 16
// rank rows.  The first one or two units ride along with the base product:
// their A rows are staged with each step, and wave (wm, wn) computes
// t^T = A_u X^T for tokens 128 wm + 32 wn .. +32 from x fragments it already
// holds.  A tile with more units (several adapters, or ranks above 32) runs
// a further pass over K per unit that computes t alone.  During
// the last step of a pass the units' B rows for the tile's columns are
// fetched into the idle LDS buffer.  After the pass t is masked to the tokens
// of each unit's adapter, scaled, split into two bf16 parts (hi + lo carry 16
// significand bits) and multiplied by B on the same MFMA shape into the base
// accumulators.  Rows an adapter does not have read the pool's zero page.
//
// Given t (FgLora::kGiven).  The callers that have a workspace compute t of
// every token first (k_long_shrink: x is read once more, 2 bytes for every
// 2 h_out flops), and the tile only expands: no rank rows ride along, so the
// K loop is the plain product's, and a tile's further units cost an expand
// instead of another pass over K.
//
// Gated pass (GLU): h = act(x Wg + term) * (x Wu + term).  A tile is 256 tokens
// x 128 output columns of both projections: of a wave's four 16-column blocks
// two are gate columns and two are the up columns of the same outputs, so the
// activation and the product happen on the lane's own accumulators and only h
// is written.  An adapter's units are those of its two modules; a unit's B rows
// are zero in the other projection's blocks.
//
// 4-bit codes.  A weight s (q - z) has up to 13 significand bits, so rounding
// it to bf16 on the way into LDS would add an error of the size of y's own
// rounding.  Instead LDS holds the exact integers q - z (or the codebook's
// values), the MFMAs of one 64-k step (32 for groups of 32) start from zero,
// and their sum is added to the accumulators times the group's scale in fp32:
// one vector FMA per accumulator and step, next to two MFMAs of 16 clocks per
// four of them.
#pragma once

#include <type_traits>

#include "base_args.hpp"
#include "common.hpp"

namespace lora {

constexpr int kFgThreads = 512;
constexpr int kFgWaves = kFgThreads / 64;
constexpr int kFgBM = 256;        // tokens per tile
constexpr int kFgBN = 256;        // output columns per tile
constexpr int kFgBK = 64;         // k per pipeline step
constexpr int kFgTileBytes = kFgBM * kFgBK * 2;   // one [256][64] bf16 tile
constexpr int kFgPassUnits = 2;   // 16-rank units per pass over K, at most
constexpr int kFgMaxPpr = kMaxFusedRowPages;   // A pages per rank row (h_in / page_elems) at most
constexpr int kFgMaxBpages = 8;   // B pages a tile's 256 columns touch, at most (page >= 64)
constexpr int kFgMaxSlots = 8192; // slot ids a tile's bitmap covers
constexpr int kFgMaxUnits = kFgBM * 4;   // 256 distinct adapters x 4 units (rank 64), per projection
constexpr int kFgGluCols = kFgBN / 2;    // output columns per tile of a gated pass
constexpr int kFgTRow = 144;      // bytes per token row of the t exchange (128 + 16: no bank conflicts)
constexpr int kFgBOff = 16384;    // B rows in the idle stage buffer's second half, after T

#ifndef LORA_FG_SWIZZLE
#define LORA_FG_SWIZZLE 1
#endif

struct FusedArgs {
  PoolView pv;
  const __bf16* x;        // [n][ld_x]
  WView w[2];             // W^T of the projection, or of gate and up: row c = weights of output column c
  const int32_t* ids;     // [n]; unused by the base-only kernel
  __bf16* y;              // [n][ld_y], written
  const float* t;         // given t: [split][projection][n][kMaxRank], scaled, zero past the rank in its last 16
  int64_t ld_x, ld_w, ld_y;   // ld_w in bytes
  int32_t n, h_in, h_out;
  int32_t module[2];
  int32_t act;            // gated pass: lora_act
  int32_t t_splits;       // given t: to be added up
  int32_t group_shift;    // 4-bit: log2(group / 32)
  int32_t n_ct;           // column tiles
  int32_t n_tiles;        // row tiles x column tiles
};

// XOR key of row r's 16-byte chunks in a [rows][64] bf16 LDS tile, and the
// byte offset of logical chunk c (0..7) of row r.  A fragment read has 16
// lanes on 16 consecutive rows at the same logical chunk; with this key any 8
// consecutive rows from an even row, and any 16 from a multiple of 16, hit
// distinct 16-byte bank groups, so the read is conflict-free whether the LDS
// serves 128 or 256 bytes per clock.
__device__ __forceinline__ int fg_swz_key(int r) {
#if LORA_FG_SWIZZLE == 1
  return ((r >> 1) & 7) ^ ((r & 1) << 2);
#else
  return r & 7;
#endif
}
__device__ __forceinline__ int fg_swz(int r, int c) { return r * 128 + ((c ^ fg_swz_key(r)) << 4); }

typedef __attribute__((address_space(3))) void* lds_ptr_t;
__device__ __forceinline__ lds_ptr_t fg_lds_ptr(void* p) {
  return reinterpret_cast<lds_ptr_t>(reinterpret_cast<uintptr_t>(p));
}

// Each lane's 16 bytes at `from` to LDS at the wave's `to` + 16 * lane.  (A
// function of its own: the builtin's size is checked against the target, which
// fails silently for a dependent expression in the host's pass.)
__device__ __forceinline__ void fg_load16(const void* from, void* to) {
  __builtin_amdgcn_global_load_lds(from, fg_lds_ptr(to), 16, 0, 0);
}

// Projections of one pass.
constexpr int fg_np(bool glu) { return glu ? 2 : 1; }

template <bool GLU, bool W4>
struct FgShared {
  // two pipeline stages of [256][64] bf16 x and W^T tiles; after a pass the
  // idle one holds t (first half) and the units' B rows (second half)
  alignas(16) unsigned char stage[2][2][kFgTileBytes];
  alignas(16) unsigned char astage[2][kFgPassUnits * 16 * kFgBK * 2];   // adapter A rows per stage
  int32_t ids[kFgBM];
  uint32_t bitmap[kFgMaxSlots / 32];
  int32_t dslot[kFgBM];            // distinct adapters of the tile, ascending
  SlotEntry dent[fg_np(GLU)][kFgBM];           // their entries
  uint16_t unit[fg_np(GLU) * kFgMaxUnits];     // (distinct index << 3) | (projection << 2) | unit of 16 ranks
  int32_t pid[kFgPassUnits][16][kFgMaxPpr];        // A pages of the pass's units
  int32_t bpid[kFgPassUnits][16][kFgMaxBpages];    // B pages of the pass's units over the tile's columns
  int32_t wsum[kFgWaves];
  int32_t spoilt;                  // a unit's B is not finite somewhere in the tile's columns
  alignas(8) uint16_t wscale[W4 ? 2 : 1][W4 ? 2 : 1][W4 ? kFgBN : 1];   // 4-bit: scales of a stage's two half steps
};

// Exclusive prefix sum over the workgroup's threads; returns the total in *total.
__device__ __forceinline__ int fg_block_scan(int v, int32_t* wsum, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int base = 0, tot = 0;
#pragma unroll
  for (int w = 0; w < kFgWaves; ++w) {
    const int s = wsum[w];
    if (w < wave) base += s;
    tot += s;
  }
  *total = tot;
  __syncthreads();   // wsum is reused by the next scan
  return base + incl - v;
}

__device__ __forceinline__ bf16x8 fg_lds8(const unsigned char* base, int off) {
  return *reinterpret_cast<const bf16x8*>(base + off);
}

template <int V>
using fg_int = std::integral_constant<int, V>;

// Two OCP e4m3 codes (the low or high half of w) widened to two bf16 values.
// Every e4m3 value has at most 4 significant bits and an exponent inside
// bf16's range, so the widening is exact (scale 1).
__device__ __forceinline__ uint32_t fg_e4m3x2_to_bf16x2(uint32_t w, bool high) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
  return __builtin_bit_cast(uint32_t, v);
}

// Where a pass takes its adapters' t from: no adapters, the shrink riding along
// with the base product, or computed before.
enum class FgLora : int { kNone, kRide, kGiven };

// WK: storage of W^T.  kFp8: e4m3 codes with a
// scale per output column (W8A16: the codes are widened to bf16 on their way
// into LDS, exactly, and the column scale multiplies the base product before
// the adapter term is added).  G32: 4-bit groups of 32 (else 64 or more).
template <FgLora L, WKind WK, bool GLU = false, bool G32 = false>
__global__ __launch_bounds__(kFgThreads, 1) void k_fused_gemm(FusedArgs a) {
  constexpr bool LORA = L != FgLora::kNone;
  constexpr bool W8 = WK == WKind::kFp8, W4 = is_w4(WK);
  constexpr int NP = fg_np(GLU);
  constexpr int TC = GLU ? kFgGluCols : kFgBN;   // output columns per tile
  __shared__ FgShared<GLU, W4> sh;
  constexpr int CB = 4;   // 16-column blocks per wave
  constexpr int SB = 2;   // 16-token shrink blocks per wave
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // uniform: LDS bases in scalar registers
  const int wm = wave >> 2, wn = wave & 3;   // tokens 128 wm .. +128, columns 64 wn .. +64
  const int l16 = lane & 15, lq = lane >> 4;

  // tile of this workgroup: the tiles one XCD takes are consecutive, so the
  // column tiles of a token tile share its x rows in that XCD's L2
  const int per_xcd = gridDim.x >> 3;
  const int tile = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if (tile >= a.n_tiles) return;
  int rt, ct;
  if constexpr (GLU) {
    // two projections' columns to a row tile: taken four row tiles at a time, so
    // that the tiles an XCD runs together read a quarter of the weights from the
    // other caches (4096 tokens, 4096 -> 2 x 12288: 838 -> 790 us)
    constexpr int kRows = 4;
    const int r0 = tile / (kRows * a.n_ct) * kRows, rows = min(kRows, (a.n + kFgBM - 1) / kFgBM - r0);
    const int in = tile - r0 * a.n_ct;
    ct = in / rows;
    rt = r0 + in - ct * rows;
  } else {
    rt = tile / a.n_ct;
    ct = tile - rt * a.n_ct;
  }
  const int row0 = rt * kFgBM, col0 = ct * TC;
  const int nk = a.h_in / kFgBK;

  // ---- staging: per K step each wave moves 4 blocks of 8 rows x 128 B of
  // the x tile and 4 of the W^T tile straight into LDS (lane i lands at byte
  // 16 i of its block).  Lane i fetches the logical chunk that the swizzle
  // puts at its LDS position: row 8 b + i / 8, physical chunk i % 8.  Rows
  // past the end repeat the last row (their results are never stored).
  const int lr = lane >> 3;
  const char* xbase = reinterpret_cast<const char*>(a.x + static_cast<int64_t>(row0) * a.ld_x);
  // row r of the W^T tile is output column col0 + wcol(r) of projection wproj(r):
  // in a gated pass the rows alternate between 32 gate and 32 up columns
  auto wproj = [](int r) { return GLU ? (r >> 5) & 1 : 0; };
  auto wcol = [](int r) { return GLU ? ((r >> 6) << 5) + (r & 31) : r; };
  const char* wbase = static_cast<const char*>(a.w[wproj(8 * wave)].w) + static_cast<int64_t>(col0) * a.ld_w;
  uint32_t xoff[4], woff[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int r = 8 * (wave + 8 * q) + lr;
    const int lc = (lane & 7) ^ fg_swz_key(r);
    xoff[q] = static_cast<uint32_t>((min(r, a.n - 1 - row0) * a.ld_x + 8 * lc) * 2);
    woff[q] = static_cast<uint32_t>(min(wcol(r), a.h_out - 1 - col0) * a.ld_w + 16 * lc);
  }
  auto load_x = [&](int kt, int buf) {
    const char* xb = xbase + kt * (kFgBK * 2);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      fg_load16(xb + xoff[q], sh.stage[buf][0] + 1024 * (wave + 8 * q));
  };
  auto load_w = [&](int kt, int buf) {
    const char* wb = wbase + kt * (kFgBK * 2);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      fg_load16(wb + woff[q], sh.stage[buf][1] + 1024 * (wave + 8 * q));
  };
  // W8: each thread moves two 16-byte pieces of e4m3 codes per K step (rows
  // i / 4 of the tile, k 16 (i % 4) .. +16, for i = tid, tid + 512) through
  // registers, widened to four bf16 chunks in the same swizzled layout
  const uint8_t* w8base = static_cast<const uint8_t*>(a.w[wproj(16 * wave)].w) + static_cast<int64_t>(col0) * a.ld_w;
  uint32_t w8off[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = tid + kFgThreads * q;
    const int r = i >> 2;
    w8off[q] = static_cast<uint32_t>(min(wcol(r), a.h_out - 1 - col0) * a.ld_w + 16 * (i & 3));
  }
  u32x4 w8reg[2];
  auto issue_w8 = [&](int kt) {
#pragma unroll
    for (int q = 0; q < 2; ++q) w8reg[q] = *reinterpret_cast<const u32x4*>(w8base + kt * kFgBK + w8off[q]);
  };
  auto store_w8 = [&](int buf) {
    unsigned char* Ws = sh.stage[buf][1];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = tid + kFgThreads * q;
      const int r = i >> 2, c = 2 * (i & 3);
      const u32x4 v = w8reg[q];
      const u32x4 lo{fg_e4m3x2_to_bf16x2(v.x, false), fg_e4m3x2_to_bf16x2(v.x, true),
                     fg_e4m3x2_to_bf16x2(v.y, false), fg_e4m3x2_to_bf16x2(v.y, true)};
      const u32x4 hi{fg_e4m3x2_to_bf16x2(v.z, false), fg_e4m3x2_to_bf16x2(v.z, true),
                     fg_e4m3x2_to_bf16x2(v.w, false), fg_e4m3x2_to_bf16x2(v.w, true)};
      *reinterpret_cast<u32x4*>(Ws + fg_swz(r, c)) = lo;
      *reinterpret_cast<u32x4*>(Ws + fg_swz(r, c + 1)) = hi;
    }
  };
  // 4-bit: each thread moves one 16-byte piece of codes per K step (32 k of row
  // tid / 2) through registers, with its scale and zero point, and writes four
  // bf16 chunks in the same swizzled layout
  const int r4 = tid >> 1, half4 = tid & 1;
  const WView& wv4 = a.w[wproj(32 * wave)];
  const int col4 = col0 + min(wcol(r4), a.h_out - 1 - col0);
  const uint8_t* w4base = static_cast<const uint8_t*>(wv4.w) + static_cast<int64_t>(col4) * a.ld_w + 16 * half4;
  u32x4 w4reg;
  uint16_t w4s = 0;
  uint8_t w4z = 8;
  W4Table w4tab;
  if constexpr (WK == WKind::kTable4) w4tab.load(wv4.table);
  auto issue_w4 = [&](int kt) {
    w4reg = *reinterpret_cast<const u32x4*>(w4base + kt * (kFgBK / 2));
    const int64_t o = static_cast<int64_t>((2 * kt + half4) >> a.group_shift) * wv4.ld_scale + col4;
    w4s = static_cast<const uint16_t*>(wv4.scale)[o];
    if (WK == WKind::kInt4 && wv4.zero) w4z = wv4.zero[o];
  };
  auto store_w4 = [&](int buf) {
    if constexpr (W4) {
      unsigned char* Ws = sh.stage[buf][1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 v;
        if constexpr (WK == WKind::kTable4) {
          v = w4_widen<WK>(w4reg[j], w4tab);
        } else {
          v = w4_minus(w4reg[j], static_cast<float>(w4z));
        }
        *reinterpret_cast<bf16x8*>(Ws + fg_swz(r4, 4 * half4 + j)) = v;
      }
      sh.wscale[buf][half4][r4] = w4s;
    }
  };
  load_x(0, 0);
  if constexpr (W4) {
    issue_w4(0);
    store_w4(0);
  } else if constexpr (W8) {
    issue_w8(0);
    store_w8(0);
  } else {
    load_w(0, 0);
  }

  // ---- the tile's adapters and units
  int n_units = 0;
  if constexpr (LORA) {
    int id = -1;
    if (tid < kFgBM && row0 + tid < a.n) {
      id = a.ids[row0 + tid];
      if (id < 0 || id >= a.pv.n_slots) id = -1;
    }
    const int n_words = (a.pv.n_slots + 31) >> 5;
    for (int i = tid; i < n_words; i += kFgThreads) sh.bitmap[i] = 0u;
    if (tid == 0) sh.spoilt = 0;
    __syncthreads();
    if (id >= 0) atomicOr(&sh.bitmap[id >> 5], 1u << (id & 31));
    __syncthreads();
    // distinct ids in ascending order: thread i takes bitmap word i (n_slots <= 8192)
    const uint32_t word = tid < n_words ? sh.bitmap[tid] : 0u;
    int n_dist = 0;
    int off = fg_block_scan(__popc(word), sh.wsum, &n_dist);
    for (uint32_t w = word; w; w &= w - 1) sh.dslot[off++] = tid * 32 + __ffs(w) - 1;
    if (tid < kFgBM) sh.ids[tid] = id;
    __syncthreads();
    int nu[NP] = {};
    int nus = 0;
    if (tid < n_dist) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const SlotEntry e = a.pv.entries[static_cast<int64_t>(sh.dslot[tid]) * a.pv.n_modules + a.module[p]];
        sh.dent[p][tid] = e;
        nu[p] = (max(e.rank, 0) + 15) >> 4;
        nus += nu[p];
      }
    }
    int uoff = fg_block_scan(nus, sh.wsum, &n_units);
#pragma unroll
    for (int p = 0; p < NP; ++p)
      for (int j = 0; j < nu[p]; ++j) sh.unit[uoff++] = static_cast<uint16_t>((tid << 3) | (p << 2) | j);
    __syncthreads();
  }

  const int h = static_cast<int>(a.pv.page_elems);
  const int ppr_a = a.h_in / h, ppr_b = a.h_out / h;
  const int cp0 = col0 / h;   // first B page column index of this tile
  const __bf16* pages = static_cast<const __bf16*>(a.pv.pages);

  // page ids of units u0 .. u0 + np - 1: A rows pid[u][rank row][k page], and
  // B rows bpid[u][rank row][page - cp0] over the tile's columns; the zero
  // page stands in for rows past the rank
  auto load_pids = [&](int u0, int np) {
    const int na = L == FgLora::kRide ? np * 16 * ppr_a : 0;
    for (int i = tid; i < na; i += kFgThreads) {
      const int u = i / (16 * ppr_a), rest = i - u * 16 * ppr_a;
      const int jr = rest / ppr_a, kp = rest - jr * ppr_a;
      const int un = sh.unit[u0 + u];
      const SlotEntry& e = sh.dent[(un >> 2) & (NP - 1)][un >> 3];
      const int jj = ((un & 3) << 4) + jr;
      sh.pid[u][jr][kp] = jj < e.rank ? a.pv.page_ids[e.a_off + jj * ppr_a + kp] : a.pv.zero_page;
    }
    const int ncp = (min(col0 + TC, a.h_out) - 1) / h - cp0 + 1;
    const int nb = np * 16 * ncp;
    for (int i = tid; i < nb; i += kFgThreads) {
      const int u = i / (16 * ncp), rest = i - u * 16 * ncp;
      const int jr = rest / ncp, ci = rest - jr * ncp;
      const int un = sh.unit[u0 + u];
      const SlotEntry& e = sh.dent[(un >> 2) & (NP - 1)][un >> 3];
      const int jj = ((un & 3) << 4) + jr;
      sh.bpid[u][jr][ci] = jj < e.rank ? a.pv.page_ids[e.b_off + jj * ppr_b + cp0 + ci] : a.pv.zero_page;
    }
  };
  // A rows of the pass's P units into astage: waves 0 .. 2P - 1 move one
  // block of 8 rank rows each (row 16 u + jr of the staged tile)
  const int arow = 8 * wave + lr;
  const int alc = (lane & 7) ^ fg_swz_key(arow);
  auto load_a = [&](auto P_, int kt, int buf) {
    constexpr int P = decltype(P_)::value;
    if (wave < 2 * P) {
      const int k0 = kt * kFgBK;
      const int kp = ppr_a == 1 ? 0 : k0 / h;
      const int pid = sh.pid[arow >> 4][arow & 15][kp];
      const __bf16* src = pages + static_cast<int64_t>(pid) * h + (k0 - kp * h) + 8 * alc;
      fg_load16(src, sh.astage[buf] + 1024 * wave);
    }
  };
  // B rows of the pass's P units (the first is u0) for the tile's columns into
  // dst: [u][rank row][256 W^T rows] bf16, 1 KB blocks of two rank rows; columns
  // past h_out and the other projection's read the zero page
  auto load_b = [&](auto P_, int u0, unsigned char* dst) {
    constexpr int P = decltype(P_)::value;
    const int col = col0 + wcol(8 * (lane & 31));
    const bool in_out = col < a.h_out;
    const int cp = in_out ? col / h : cp0;
    const int cin = in_out ? col - cp * h : 0;
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int b = wave + kFgWaves * q;   // block: unit b / 8, rank rows 2 (b % 8) .. +2
      const int jr = 2 * (b & 7) + (lane >> 5);
      const bool in = in_out && (!GLU || ((sh.unit[u0 + q] >> 2) & 1) == wproj(8 * (lane & 31)));
      const int pid = in ? sh.bpid[b >> 3][jr][cp - cp0] : a.pv.zero_page;
      fg_load16(pages + static_cast<int64_t>(pid) * h + cin, dst + 1024 * b);
    }
  };

  // t is zero for the tokens of other adapters, but zero times an infinity or NaN
  // in a unit's B is not.  So each lane looks at the pieces of B that it brought
  // itself, puts zero in such a value's place, and the adapter's own outputs there
  // become NaN at the end.  No barrier more; 4096 tokens, 4096 -> 2 x 12288 bf16
  // 737 -> 745 us, 2111 tokens -> 2 x 8192 fp8 326 -> 330, 4096x4096 4-bit and the
  // pass with riding units unchanged (at the products, in registers, the same
  // search cost 1.5 to 3%, and a path of its own there 350 to 640 spilled registers).
  auto keep_finite = [&](auto P_, unsigned char* dst) {
    constexpr int P = decltype(P_)::value;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the lane's pieces have landed
#pragma unroll
    for (int q = 0; q < P; ++q) {
      u32x4* at = reinterpret_cast<u32x4*>(dst + 1024 * (wave + kFgWaves * q) + 16 * lane);
      const u32x4 v = *at;
      u32x4 bad;
#pragma unroll
      for (int i = 0; i < 4; ++i)   // an exponent of all ones carries into the sign's place
        bad[i] = ((v[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
      if ((bad.x | bad.y | bad.z | bad.w) != 0) {
        *at = v & ~((bad << 1) - (bad >> 15));
        sh.spoilt = 1;
      }
    }
  };

  f32x4 acc[CB][8];
#pragma unroll
  for (int i = 0; i < CB; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  f32x4 tacc[SB][kFgPassUnits];

  // LDS rows of this lane's fragments
  const int wrow = 64 * wn + l16;    // W^T rows (output columns) of col block cb: + 16 cb
  const int xrow = 128 * wm + l16;   // x rows (tokens) of token block tb: + 16 tb
  const int srow = 128 * wm + 32 * wn + l16;   // x rows of this wave's shrink tokens: + 16 i
  unsigned char* const idle = sh.stage[nk & 1][0];   // the buffer no step of a pass's last one reads

  // One K step of the base product from 4-bit codes: the step's sums start
  // from zero and join the accumulators times their group's scale.
  static_assert(!W4 || L != FgLora::kRide, "4-bit steps carry no adapter units");
  auto step_w4 = [&](int buf) {
    if constexpr (W4) {
      const unsigned char* Xs = sh.stage[buf][0];
      const unsigned char* Ws = sh.stage[buf][1];
      bf16x8 wf[2][CB];
      f32x4 sc[G32 ? 2 : 1][CB];
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) wf[ks][cb] = fg_lds8(Ws, fg_swz(wrow + 16 * cb, 4 * ks + lq));
#pragma unroll
        for (int g = 0; g < (G32 ? 2 : 1); ++g) {
          const u32x2 v = *reinterpret_cast<const u32x2*>(&sh.wscale[buf][g][64 * wn + 16 * cb + 4 * lq]);
          sc[g][cb] = f32x4{bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y)};
        }
      }
      const f32x4 none{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int tb = 0; tb < 8; ++tb) {
        bf16x8 xf[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) xf[ks] = fg_lds8(Xs, fg_swz(xrow + 16 * tb, 4 * ks + lq));
        f32x4 sum[CB];
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
          sum[cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[0][cb], xf[0], none, 0, 0, 0);
        if constexpr (G32) {
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) acc[cb][tb] += sc[0][cb] * sum[cb];
        }
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
          sum[cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[1][cb], xf[1], G32 ? none : sum[cb], 0, 0, 0);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) acc[cb][tb] += sc[G32 ? 1 : 0][cb] * sum[cb];
        // keeps the next blocks' reads from being hoisted: registers are the limit
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // One pass over K.  BASE: the base product with the shrink of P units
  // riding along; otherwise the shrink alone.  During the last step the P
  // units' B rows go to the idle buffer.
  auto kloop = [&](auto P_, auto BASE_, int u0) {
    constexpr int P = decltype(P_)::value;
    constexpr bool BASE = decltype(BASE_)::value != 0;
#pragma unroll
    for (int i = 0; i < SB; ++i)
#pragma unroll
      for (int u = 0; u < kFgPassUnits; ++u) tacc[i][u] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto step = [&](int buf) {
      const unsigned char* Xs = sh.stage[buf][0];
      const unsigned char* Ws = sh.stage[buf][1];
      if constexpr (BASE && W4) {
        step_w4(buf);
        return;
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int c = 4 * ks + lq;
        bf16x8 xs[SB];   // x fragments of this wave's shrink tokens
        if constexpr (BASE) {
          bf16x8 wf[CB];
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) wf[cb] = fg_lds8(Ws, fg_swz(wrow + 16 * cb, c));
#pragma unroll
          for (int tb = 0; tb < 8; ++tb) {
            const bf16x8 xf = fg_lds8(Xs, fg_swz(xrow + 16 * tb, c));
#pragma unroll
            for (int cb = 0; cb < CB; ++cb)
              acc[cb][tb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[cb], xf, acc[cb][tb], 0, 0, 0);
            if constexpr (P > 0) {   // token blocks SB wn .. SB wn + SB - 1, picked without a branch
              if (tb < SB) xs[tb] = xf;
              else xs[tb % SB] = tb / SB == wn ? xf : xs[tb % SB];
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < SB; ++i) xs[i] = fg_lds8(Xs, fg_swz(srow + 16 * i, c));
        }
        if constexpr (P > 0) {
#pragma unroll
          for (int u = 0; u < P; ++u) {
            const bf16x8 af = fg_lds8(sh.astage[buf], fg_swz(16 * u + l16, c));
#pragma unroll
            for (int i = 0; i < SB; ++i)
              tacc[i][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af, xs[i], tacc[i][u], 0, 0, 0);
          }
        }
      }
    };
    // The last step is peeled so that the loop body has no branch (a branch
    // there makes the compiler shuttle the accumulators between register files).
    for (int kt = 0; kt < nk - 1; ++kt) {
      const int buf = kt & 1;
      load_x(kt + 1, buf ^ 1);   // that buffer's readers passed the last barrier
      if constexpr (BASE && !W8 && !W4) load_w(kt + 1, buf ^ 1);
      if constexpr (BASE && W8) issue_w8(kt + 1);
      if constexpr (BASE && W4) issue_w4(kt + 1);
      if constexpr (P > 0) load_a(P_, kt + 1, buf ^ 1);
      step(buf);
      if constexpr (BASE && W8) store_w8(buf ^ 1);   // widened after this step's reads of buf
      if constexpr (BASE && W4) store_w4(buf ^ 1);
      __syncthreads();
    }
    if constexpr (P > 0) load_b(P_, u0, idle + kFgTileBytes + kFgBOff);
    step((nk - 1) & 1);
    __syncthreads();   // also: the B rows have landed
  };

  // t of units u0 .. u0 + P - 1 -> LDS, masked to each unit's adapter and
  // rank rows and scaled; then acc^T += B^T_u [cols x 32] . T_u [32 x tokens]
  // where k 0..15 pair hi with ranks 0..15 and k 16..31 pair lo with them
  auto multiply_b = [&](auto P_) {
    constexpr int P = decltype(P_)::value;
    const unsigned char* T_s = idle;                           // [256 tokens][kFgTRow]
    const unsigned char* B_s = idle + kFgTileBytes + kFgBOff;  // [u][16 ranks][256 cols] bf16
#pragma unroll
    for (int u = 0; u < P; ++u) {
      bf16x8 bfr[CB];   // lane: output column wrow + 16 cb, ranks 8 (lq & 1) .. +8
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        const unsigned short* bp = reinterpret_cast<const unsigned short*>(
            B_s + u * 8192 + (8 * (lq & 1)) * 512 + 2 * (wrow + 16 * cb));
        unsigned short e[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) e[r] = bp[256 * r];
        bfr[cb] = __builtin_bit_cast(bf16x8, e);
      }
#pragma unroll
      for (int tb = 0; tb < 8; ++tb) {
        const bf16x8 tf = fg_lds8(T_s, (xrow + 16 * tb) * kFgTRow + u * 64 + 16 * lq);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
          acc[cb][tb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bfr[cb], tf, acc[cb][tb], 0, 0, 0);
      }
    }
  };
  auto expand = [&](auto P_, int u0) {
    constexpr int P = decltype(P_)::value;
    unsigned char* T_s = idle;
#pragma unroll
    for (int i = 0; i < SB; ++i) {
      const int tok = srow + 16 * i;
      const int id = sh.ids[tok];
#pragma unroll
      for (int u = 0; u < P; ++u) {
        const int un = sh.unit[u0 + u], d = un >> 3;
        float s = 0.f;
        int rows = 0;
        if (sh.dslot[d] == id) {
          const SlotEntry& e = sh.dent[(un >> 2) & (NP - 1)][d];
          s = e.scale;
          rows = e.rank - ((un & 3) << 4);
        }
        __bf16 hi[4], lo[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float t = 4 * lq + v < rows ? tacc[i][u][v] * s : 0.f;
          hi[v] = static_cast<__bf16>(t);
          lo[v] = static_cast<__bf16>(t - static_cast<float>(hi[v]));
        }
        unsigned char* trow = T_s + tok * kFgTRow + u * 64;
        *reinterpret_cast<u32x2*>(trow + 8 * lq) = __builtin_bit_cast(u32x2, hi);
        *reinterpret_cast<u32x2*>(trow + 32 + 8 * lq) = __builtin_bit_cast(u32x2, lo);
      }
    }
    keep_finite(P_, idle + kFgTileBytes + kFgBOff);
    __syncthreads();
    multiply_b(P_);
  };

  // Output column of this lane's accumulators of block cb: + 0 .. 3.
  auto out_col = [&](int cb) { return col0 + (GLU ? 32 * wn + 16 * (cb & 1) : 64 * wn + 16 * cb) + 4 * lq; };
  // W8: the base accumulators times each output column's scale (before any
  // adapter term is added).
  auto scale_base = [&]() {
    if constexpr (W8) {
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        const int col = out_col(cb);
        const float* ws = static_cast<const float*>(a.w[GLU ? cb >> 1 : 0].scale);
        const f32x4 sc = col < a.h_out ? *reinterpret_cast<const f32x4*>(ws + col) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int tb = 0; tb < 8; ++tb) acc[cb][tb] *= sc;
      }
    }
  };

  // ---- given t: the tile's units in pairs, t -> LDS as hi and lo parts
  auto expand_given = [&](int u0) {
    unsigned char* T_s = idle;
    const int np = min(n_units - u0, kFgPassUnits);
    load_pids(u0, np);
    __syncthreads();   // also: the previous pair's reads (or the K loop's) are done
    if (np == 2) load_b(fg_int<2>{}, u0, idle + kFgTileBytes + kFgBOff);
    else load_b(fg_int<1>{}, u0, idle + kFgTileBytes + kFgBOff);
    const int tok = tid >> 1, u = tid & 1;
    f32x4 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (u < np) {
      const int un = sh.unit[u0 + u];
      if (sh.dslot[un >> 3] == sh.ids[tok]) {   // rows past the batch have id -1: no slot
        const float* from =
            a.t + (static_cast<int64_t>((un >> 2) & (NP - 1)) * a.n + row0 + tok) * kMaxRank + 16 * (un & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = reinterpret_cast<const f32x4*>(from)[i];
        for (int z = 1; z < a.t_splits; ++z) {
          from += static_cast<int64_t>(NP) * a.n * kMaxRank;
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] += reinterpret_cast<const f32x4*>(from)[i];
        }
      }
    }
    if (np == 2) keep_finite(fg_int<2>{}, idle + kFgTileBytes + kFgBOff);
    else keep_finite(fg_int<1>{}, idle + kFgTileBytes + kFgBOff);
    __bf16 hi[16], lo[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      hi[i] = static_cast<__bf16>(t[i >> 2][i & 3]);
      lo[i] = static_cast<__bf16>(t[i >> 2][i & 3] - static_cast<float>(hi[i]));
    }
    unsigned char* trow = T_s + tok * kFgTRow + u * 64;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<bf16x8*>(trow + 16 * i) = *reinterpret_cast<const bf16x8*>(hi + 8 * i);
      *reinterpret_cast<bf16x8*>(trow + 32 + 16 * i) = *reinterpret_cast<const bf16x8*>(lo + 8 * i);
    }
    __syncthreads();
    if (np == 2) multiply_b(fg_int<2>{});
    else multiply_b(fg_int<1>{});
    __syncthreads();
  };

  // ---- pass 0: the base product with up to two units
  if constexpr (L == FgLora::kGiven) {
    __syncthreads();   // stage 0 has landed
    kloop(fg_int<0>{}, fg_int<1>{}, 0);
    scale_base();
    for (int u0 = 0; u0 < n_units; u0 += kFgPassUnits) expand_given(u0);
  } else if constexpr (LORA) {
    const int np0 = min(n_units, kFgPassUnits);
    if (np0 > 0) {
      load_pids(0, np0);
      __syncthreads();
    }
    if (np0 == 2) {
      load_a(fg_int<2>{}, 0, 0);
      __syncthreads();
      kloop(fg_int<2>{}, fg_int<1>{}, 0);
      scale_base();
      expand(fg_int<2>{}, 0);
    } else if (np0 == 1) {
      load_a(fg_int<1>{}, 0, 0);
      __syncthreads();
      kloop(fg_int<1>{}, fg_int<1>{}, 0);
      scale_base();
      expand(fg_int<1>{}, 0);
    } else {
      __syncthreads();
      kloop(fg_int<0>{}, fg_int<1>{}, 0);
      scale_base();
    }
    // ---- further passes, one unit at a time, shrink only
    for (int u0 = np0; u0 < n_units; ++u0) {
      __syncthreads();   // the previous pass's LDS reads are done
      load_pids(u0, 1);
      __syncthreads();
      load_x(0, 0);
      load_a(fg_int<1>{}, 0, 0);
      __syncthreads();
      kloop(fg_int<1>{}, fg_int<0>{}, u0);
      expand(fg_int<1>{}, u0);
    }
  } else {
    __syncthreads();   // stage 0 has landed (the barrier waits for the loads)
    kloop(fg_int<0>{}, fg_int<1>{}, 0);
    scale_base();
  }

  // ---- y: lane holds output columns 4 lq .. +4 of col block cb for token
  // 16 tb + l16; one rounding to bf16 per element
#pragma unroll
  for (int tb = 0; tb < 8; ++tb) {
    const int tok = row0 + xrow + 16 * tb;
    if (tok >= a.n) continue;
    __bf16* yr = a.y + static_cast<int64_t>(tok) * a.ld_y;
#pragma unroll
    for (int cb = 0; cb < (GLU ? CB / 2 : CB); ++cb) {
      const int col = out_col(cb);
      if (col >= a.h_out) continue;
      __bf16 o[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if constexpr (GLU) o[v] = static_cast<__bf16>(glu_act(a.act, acc[cb][tb][v]) * acc[cb + CB / 2][tb][v]);
        else o[v] = static_cast<__bf16>(acc[cb][tb][v]);
      }
      *reinterpret_cast<u32x2*>(yr + col) = __builtin_bit_cast(u32x2, o);
    }
  }

  // ---- outputs of adapters whose B is not finite there (rare; this wave's own
  // stores above have to land first)
  if constexpr (LORA) {
    if (sh.spoilt == 0) return;
    __threadfence();
    const int col = col0 + (GLU ? 32 * wn + (lane & 31) : 64 * wn + lane);
    if (col >= a.h_out) return;
    const int cp = col / h, cin = col - cp * h;
    for (int u = 0; u < n_units; ++u) {
      const int un = sh.unit[u], slot = sh.dslot[un >> 3];
      const SlotEntry& e = sh.dent[(un >> 2) & (NP - 1)][un >> 3];
      const int j0 = (un & 3) << 4;
      bool bad = false;
      for (int j = j0; j < min(e.rank, j0 + 16); ++j) {
        const int pid = a.pv.page_ids[e.b_off + j * ppr_b + cp];
        const uint16_t v = reinterpret_cast<const uint16_t*>(pages)[static_cast<int64_t>(pid) * h + cin];
        bad |= (v & 0x7F80) == 0x7F80;
      }
      if (!bad) continue;
      for (int t = 128 * wm; t < 128 * wm + 128; ++t)
        if (sh.ids[t] == slot)   // rows past the batch have id -1
          reinterpret_cast<uint16_t*>(a.y)[static_cast<int64_t>(row0 + t) * a.ld_y + col] = 0x7FC0;
    }
  }
}

}  // namespace lora
