// What the base-product kernels share: how the base weights are stored, the
// 4-bit codes' widening, and the gate's activations.
#pragma once

#include "base_plan.hpp"
#include "common.hpp"

namespace lora {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// The base weights of one projection.
struct WView {
  const void* w;          // rows
  const void* scale;      // fp8: float [h_out]; 4-bit: bf16 [h_in / group][ld_scale]
  const uint8_t* zero;    // 4-bit: [h_in / group][ld_scale], or null
  const uint32_t* table;  // kTable4: 16 bf16 values, two to a word
  int64_t ld_scale;
};

// Eight codes of a word (code i in bits 4i..4i+3) as bytes, in order.
__device__ __forceinline__ void w4_bytes(uint32_t w, uint32_t (&n)[2]) {
  const uint32_t e = w & 0x0F0F0F0Fu, o = (w >> 4) & 0x0F0F0F0Fu;
  n[0] = __builtin_amdgcn_perm(o, e, 0x05010400u);
  n[1] = __builtin_amdgcn_perm(o, e, 0x07030602u);
}

// Two codes 0..15 (bytes 0,1 or 2,3 of n) as two bf16 integers.  As e4m3 a
// byte c < 16 is c * 2^-9 (the subnormals and the first binade share one
// spacing), so the hardware's widening with scale 2^9 gives c exactly, at one
// instruction for two codes.
template <bool HIGH>
__device__ __forceinline__ uint32_t w4_int2(uint32_t n) {
  const bf16x2 v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(n, 512.0f, HIGH);
  return __builtin_bit_cast(uint32_t, v);
}

// A 16-entry bf16 codebook as byte planes: lo[i] holds the low bytes of
// entries 4i..4i+3, hi[i] their high bytes.
struct W4Table {
  uint32_t lo[4], hi[4];
  __device__ __forceinline__ void load(const uint32_t* t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = t[2 * i], b = t[2 * i + 1];
      lo[i] = __builtin_amdgcn_perm(b, a, 0x06040200u);
      hi[i] = __builtin_amdgcn_perm(b, a, 0x07050301u);
    }
  }
  // Four codes (bytes of n) looked up: two words of two bf16 values, in order.
  // v_perm selects among 8 bytes, so each plane takes two selections by the
  // low three bits and a third by bit 3.
  __device__ __forceinline__ u32x2 look(uint32_t n) const {
    const uint32_t s = n & 0x07070707u;
    const uint32_t b3 = ((n & 0x08080808u) >> 1) | 0x03020100u;
    const uint32_t l = __builtin_amdgcn_perm(__builtin_amdgcn_perm(lo[3], lo[2], s),
                                             __builtin_amdgcn_perm(lo[1], lo[0], s), b3);
    const uint32_t h = __builtin_amdgcn_perm(__builtin_amdgcn_perm(hi[3], hi[2], s),
                                             __builtin_amdgcn_perm(hi[1], hi[0], s), b3);
    return u32x2{__builtin_amdgcn_perm(h, l, 0x05010400u), __builtin_amdgcn_perm(h, l, 0x07030602u)};
  }
};

// Eight codes of a word as the eight bf16 integers q (kInt4) or codebook
// values (kTable4), in order of k.
// EVEN_ODD (kInt4): in the order 0 2 4 6 1 3 5 7 instead, two instructions less.
template <WKind WK, bool EVEN_ODD = false>
__device__ __forceinline__ bf16x8 w4_widen(uint32_t w, const W4Table& tab) {
  uint32_t n[2];
  if constexpr (EVEN_ODD && WK == WKind::kInt4) {
    n[0] = w & 0x0F0F0F0Fu;
    n[1] = (w >> 4) & 0x0F0F0F0Fu;
  } else {
    w4_bytes(w, n);
  }
  if constexpr (WK == WKind::kTable4) {
    const u32x2 a = tab.look(n[0]), b = tab.look(n[1]);
    return __builtin_bit_cast(bf16x8, u32x4{a.x, a.y, b.x, b.y});
  } else {
    return __builtin_bit_cast(bf16x8, u32x4{w4_int2<false>(n[0]), w4_int2<true>(n[0]), w4_int2<false>(n[1]),
                                              w4_int2<true>(n[1])});
  }
}

// Eight bf16 values in the order that EVEN_ODD widening gives the codes.
__device__ __forceinline__ u32x4 w4_xl_order(u32x4 v) {
  return u32x4{__builtin_amdgcn_perm(v.y, v.x, 0x05040100u), __builtin_amdgcn_perm(v.w, v.z, 0x05040100u),
               __builtin_amdgcn_perm(v.y, v.x, 0x07060302u), __builtin_amdgcn_perm(v.w, v.z, 0x07060302u)};
}

// Eight codes of a word as the eight bf16 integers q - z, exactly (|q - z| < 256).
__device__ __forceinline__ bf16x8 w4_minus(uint32_t w, float z) {
  uint32_t n[2], o[4];
  w4_bytes(w, n);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = n[i >> 1] >> (16 * (i & 1));
    const float a = static_cast<float>(v & 0xFFu) - z, b = static_cast<float>((v >> 8) & 0xFFu) - z;
    o[i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
  }
  return __builtin_bit_cast(bf16x8, u32x4{o[0], o[1], o[2], o[3]});
}

// The gate's activation, in fp32 (act: lora_act).
__device__ __forceinline__ float glu_act(int act, float v) {
  if (act == LORA_ACT_SILU) return v / (1.f + expf(-v));
  if (act == LORA_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678f);   // erfc: no cancellation for v << 0
  // tanh form: 0.5 v (1 + tanh(u)) = v / (1 + exp(-2u)), u = sqrt(2/pi) (v + 0.044715 v^3)
  const float u2 = 1.59576912f * (v + 0.044715f * v * v * v);
  return v / (1.f + expf(-u2));
}

}  // namespace lora
