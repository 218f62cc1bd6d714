// Shared declarations of the attention paths over the 4-bit cache.  Arguments and plan are
// those of the 8-bit cache's paths; kc, vc are the codes, ke, ve the scales (bf16).
#pragma once

#include "tsd_q4.cuh"
#include "tsd_q8_attn.cuh"

namespace tsd {

// Up to this many packed rows take the path with keys on the product's rows.  (12 rows of 32
// requests over 1k to 4k keys: 48 us so and 67 us on tcgen05; 16 rows: 50 and 67, of 8 requests
// over 32k keys 93 and 138 us.)
constexpr int kQ4FewRows = 16;

constexpr int kQ4F32 = kQ8Simt;                      // the path of fp32 heads

// Exponents above a tile's scales, within which its keys or values are held in fp16 (the
// scales that writes give: -92..125).
constexpr int kQ4MinExp = -96, kQ4MaxExp = 118;

void launch_q4_few(const Q8AttnArgs& a, const Q8Plan& p, int D, cudaStream_t st);
void launch_q4_f32(const Q8AttnArgs& a, const Q8Plan& p, int D, cudaStream_t st);
void launch_q4_rows(const Q8AttnArgs& a, const Q8Plan& p, int D, cudaStream_t st);

}  // namespace tsd
