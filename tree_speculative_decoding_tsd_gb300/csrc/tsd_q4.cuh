// The 4-bit KV cache: its number format and the helpers its kernels share.
//
// A row of d dims (one token, one head, K or V) holds d codes c in 0..15 and a bf16
// scale s for each 32 dims: value = (c - 8) s.  Rows do not depend on one another, so
// an append never touches an earlier row.  Of a group's elements the one of largest
// magnitude gets the code 0 (s has the other sign): the 16 codes reach from there to 7/8
// of it on the other side, a step of 1/8 where a symmetric format has 1/7.
//
// A 32-bit word holds the codes of eight dims, the even ones in its low half and the odd
// ones in its high half, from the lowest bits up: one mask then gives two adjacent dims
// as two fp16 numbers (a code in the lowest bits of an fp16 number is c * 2^-24, four
// bits higher c * 2^-20: exact, and taken as such by products).
#pragma once

#include "tsd_q8.cuh"

namespace tsd {

constexpr int kQ4Group = TSD_Q4_GROUP;

// Codes of a word, less 8, as fp32.
__device__ __forceinline__ void q4_values(uint32_t w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // 1024 + c in fp16; 1032 is exact, too
    const uint32_t h = ((w >> (4 * i)) & 0x000f000fu) | 0x64006400u;
    const float2 f = __half22float2(
        __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6408))));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// Smallest magnitude that a group is held for; groups below it are zeros, which keeps
// a scale's inverse finite.
constexpr float kQ4Tiny = 8.077935669463161e-28f;   // 2^-90

// Scale of a group (bf16 bits) whose largest and smallest elements are hi and lo (NaN
// where there is one): that of the larger magnitude, over -8.
__device__ __forceinline__ uint32_t q4_scale(float hi, float lo) {
  const float top = hi >= -lo ? hi : lo;
  if (!(fabsf(top) < INFINITY)) return 0x7fffu;
  if (fabsf(top) < kQ4Tiny) return 0u;
  return __bfloat16_as_ushort(__float2bfloat16_rn(top * -0.125f));
}

// Eight elements as a word of codes, given 1 / s (fp32, rounded to nearest): the nearest
// whole number to x / s, ties to even, within -8..7, plus 8.  Adding 1.5 * 2^23 + 8 rounds
// the exact product (a fused multiply-add) to a whole number in the sum's lowest bits;
// cvt.pack clamps two numbers to four bits and puts them behind those it is given.
__device__ __forceinline__ uint32_t q4_word(const float (&x)[8], float inv) {
  constexpr float kZero = 12582912.f;
  int c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __float_as_int(fmaf(x[i], inv, kZero + 8.f)) - 0x4b400000;
  uint32_t w = 0;
  auto pack = [&](int hi, int lo) {
    asm("cvt.pack.sat.u4.s32.b32 %0, %1, %2, %0;\n" : "+r"(w) : "r"(hi), "r"(lo));
  };
  pack(c[7], c[5]);
  pack(c[3], c[1]);
  pack(c[6], c[4]);
  pack(c[2], c[0]);
  return w;
}
// 1 / s; 0 for a group of zeros or one that holds a NaN, whose codes are 8.
__device__ __forceinline__ float q4_inverse(uint32_t scale) {
  return (scale & 0x7fffu) == 0u || (scale & 0x7fffu) > 0x7f80u ? 0.f : __frcp_rn(bf16_value(scale));
}

// Host: descriptors of the 4-bit calls (latent heads: valid, not implemented).
inline tsd_status q4_desc_status(const tsd_attn_desc* d, bool scaled = false) {
  if (!q8_desc_ok(d, scaled)) return TSD_ERR_INVALID_ARG;
  return d->v_aliases_k ? TSD_ERR_UNSUPPORTED : TSD_OK;
}

}  // namespace tsd
