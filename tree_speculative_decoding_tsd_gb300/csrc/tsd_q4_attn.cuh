// Shared declarations of the attention paths over the 4-bit cache.  Arguments and plan are
// those of the 8-bit cache's paths; kc, vc are the codes, ke, ve the scales (bf16).
#pragma once

#include "tsd_q4.cuh"
#include "tsd_q8_attn.cuh"
#include "tsd_tcgen05.cuh"

namespace tsd {

// Up to this many packed rows take the path with keys on the product's rows.  (12 rows of 32
// requests over 1k to 4k keys: 48 us so and 67 us on tcgen05; 16 rows: 50 and 67, of 8 requests
// over 32k keys 93 and 138 us.)
constexpr int kQ4FewRows = 16;

// Splits of a launch at most (a grid's y and z); caches near 2^31 positions have one more.
constexpr int kMaxGrid = 65535;

constexpr int kQ4F32 = kQ8Simt;                      // the path of fp32 heads

// Exponents above a tile's scales, within which its keys or values are held in fp16 (the
// scales that writes give: -92..125).
constexpr int kQ4MinExp = -96, kQ4MaxExp = 118;

// The two sums of a row have bounds of their own.  Weighted values count over 2^m, m the bound of x + E:
// small scores of large values may matter, and large scores of small values may not.  The weights' sum
// counts over 2^u, u = m - eu, which has to be near the largest x.  While all E are within this of 0, that
// is eu = 0 and the sum takes 2^(x + E - m), a key's weight for the products, times 2^-E: what the first
// factor loses (below 2^-126) is 2^-62 of the largest or less.  From the first tile on whose E is further
// off, each row has an eu of its own, and the tiles' sums are computed on their own.
constexpr int kQ4Near = 32;

// The new eu: m, eu of the keys before, m_new the bound with a tile whose largest score is x.
__device__ __forceinline__ float q4_near(float m, float eu, float m_new, float x) {
  const float e = rintf(m_new - fmaxf(m - eu, x));
  return fabsf(e) <= 127.f ? e : eu;                 // (no key yet, or scores that are not finite)
}

// 2^k / total for total >= 0, and 0 for 0, where either alone may be far from 1.
__device__ __forceinline__ float q4_over(float k, float total) {
  const int e = (int)(__float_as_uint(total) >> 23) - 127;
  return total == 0.f ? 0.f : __fdividef(ex2(k - (float)e), total * pow2i(-e));
}

void launch_q4_few(const Q8AttnArgs& a, const Q8Plan& p, int D, cudaStream_t st);
void launch_q4_f32(const Q8AttnArgs& a, const Q8Plan& p, int D, cudaStream_t st);
void launch_q4_rows(const Q8AttnArgs& a, const Q8Plan& p, int D, cudaStream_t st);

}  // namespace tsd
