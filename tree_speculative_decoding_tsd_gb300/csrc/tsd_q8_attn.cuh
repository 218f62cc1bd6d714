// Shared declarations of the attention paths over the 8-bit cache.
#pragma once

#include "tsd_q8.cuh"

namespace tsd {

struct Q8AttnArgs {
  const void* q;
  const uint8_t* kc;
  const uint8_t* vc;          // null: the value is the first dv entries of the key
  const uint8_t* ke;
  const uint8_t* ve;
  const int32_t* plen;
  const void* kt;
  const void* vt;
  const uint64_t* mask;
  void* out;
  float* lse;
  void* part_o;               // [B][Hq][nr][nsplit][dv] normalised outputs of the splits, over scale
  float2* part_meta;          // [B][Hq][nr][nsplit] (log2-sum-exp, scale)
  int32_t* err;
  CacheMap map;
  int B, R, Hq, g, M;
  int r0, nr;                 // the launch's tree rows: r0 .. r0 + nr - 1 (M = nr g packed rows)
  int nsplit, split_len, nrg, rb, tree_split;
  int split0;                 // (4-bit cache) the launch's first split
  int by_length;              // grid z is a rank in (prefix length desc, index asc) order
  float qscale;               // softmax scale * log2(e)
  long long wait_cycles;      // of a pipeline wait (kernels that poll)
};

enum Q8Path { kQ8Simt = 0, kQ8Few = 1, kQ8Rows = 2, kQ8Latent = 3 };

// Up to this many packed rows take the path with keys on lanes.  (4 rows, 16 requests
// over 20k to 32k keys: 165 us so and 179 us with the rows on lanes; 16 rows, 8 requests
// over 32k keys: 112 and 118 us, 32 over 1k to 4k: 50 and 54 us; 32 rows of them, with
// 32 columns: 59 and 56 us.)
constexpr int kQ8FewRows = 16;

struct Q8Plan {
  int path;
  int rb, nrg;                // packed rows per CTA, row groups per KV head
  int nsplit, split_len;
  int by_length;              // requests are taken longest first
  int tree_split;             // the tree rows are a split of their own, behind the prefix splits
  int part_bytes;             // element size of a split's output: 4 (fp32) or 2 (fp16)
  int small_ctas;             // (4-bit cache, few rows) several small CTAs per SM
  size_t ws_bytes;
};

// Splits that hold work for a request of prefix length P, and the positions k0 .. k1 - 1 of one of them.
// (Unsigned: P and the end of its last split may lie on either side of 2^31.)
__device__ __forceinline__ int q8_splits(const Q8AttnArgs& a, int P) {
  const int npre = P > 0 ? (int)(((uint32_t)P + a.split_len - 1u) / (uint32_t)a.split_len) : 0;
  return a.tree_split ? npre + 1 : max(npre, 1);
}
__device__ __forceinline__ int q8_first(const Q8AttnArgs& a, int P, int sp) {
  return (int)min((uint32_t)sp * a.split_len, (uint32_t)P);
}
__device__ __forceinline__ int q8_end(const Q8AttnArgs& a, int P, int k0) {
  return (int)min((uint32_t)k0 + a.split_len, (uint32_t)P);
}

bool launch_q8_few(const tsd_attn_desc& d, const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st);
bool launch_q8_rows(const tsd_attn_desc& d, const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st);
bool launch_q8_latent(const tsd_attn_desc& d, const Q8AttnArgs& a, const Q8Plan& p,
                      cudaStream_t st);

}  // namespace tsd
