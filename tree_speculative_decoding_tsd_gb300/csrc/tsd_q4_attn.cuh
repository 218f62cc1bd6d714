// Shared declarations of the attention paths over the 4-bit cache.  Arguments and plan are
// those of the 8-bit cache's paths; kc, vc are the codes, ke, ve the scales (bf16).
#pragma once

#include "tsd_q4.cuh"
#include "tsd_q8_attn.cuh"

namespace tsd {

constexpr int kQ4FewRows = 16;      // packed rows of the path for few

// Exponents above a tile's scales, within which its keys or values are held in fp16 (the
// scales that writes give: -92..125).
constexpr int kQ4MinExp = -96, kQ4MaxExp = 118;

void launch_q4_few(const Q8AttnArgs& a, const Q8Plan& p, int D, cudaStream_t st);
void launch_q4_rows(const Q8AttnArgs& a, const Q8Plan& p, int D, cudaStream_t st);

}  // namespace tsd
