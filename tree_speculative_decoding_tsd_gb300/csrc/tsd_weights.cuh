// Shared declarations of the attention-weight kernels (tsd_cache_weights).
#pragma once

#include "tsd_q8.cuh"

namespace tsd {

struct WeightArgs {
  const void* q;             // [B][R][Hq][dk]
  const void* k;             // cache rows (element type of q, or e4m3 codes)
  const uint8_t* ke;         // exponent bytes of an 8-bit cache, else null
  const int32_t* plen;
  const void* kt;            // [B][R][Hkv][dk]
  const int32_t* path;       // [B][S+1]
  const int32_t* path_len;   // [B]
  const float* lse;          // [B][R][Hq], natural log
  float* acc;                // [B][Hkv][cap]
  int32_t* pos;              // [B][Hkv][cap]
  int32_t* seen;             // [B][Hkv]
  int32_t* err;
  CacheMap map;
  int R, Hq, g, S;
  float decay;
  float qscale;              // softmax scale * log2(e)
  long long wait_cycles;     // of a pipeline wait (kernels that poll)
};

constexpr int kWeightKeys = 128;     // cached rows per tile
constexpr int kMaxPath = 17;         // 1 + S, S <= 16
constexpr float kLog2e = 1.4426950408889634f;

// Path of one request as a CTA sees it.
struct PathSmem {
  int32_t rows[kMaxPath];
  int code;
  int blind;                 // a page that only the prefix has is missing
};

// Read the path of request b and check it, its length, the capacity and the pages
// of the path's rows; the same answer on every thread and in every CTA of the
// request, so that the requests that the commit skips are skipped as a whole, and no
// others.  Returns the path length L, or minus the error code.
__device__ __forceinline__ int weight_path(const WeightArgs& a, int b, int P, PathSmem& s) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    s.code = 0x7fffffff;
    s.blind = 0;
  }
  __syncthreads();
  const int L = a.path_len[b];
  int code = 0;
  if (L < 0 || L > a.S) code = TSD_DEV_ERR_BAD_TREE;
  else if (P < 0 || (long)P + 1 + L > a.map.cap) code = TSD_DEV_ERR_CAPACITY;
  else {
    if (tid <= L) {
      const int r = a.path[(long)b * (a.S + 1) + tid];
      if (r < 0 || r >= a.R) code = TSD_DEV_ERR_BAD_TREE;
      s.rows[tid] = r;
    }
    if (a.map.page_size)
      for (int p = tid; p <= (P + L) / a.map.page_size; p += blockDim.x) {
        const int pg = a.map.page_table[(long)b * a.map.max_pages + p];
        if (pg >= 0 && pg < a.map.num_pages) continue;
        if (p < P / a.map.page_size) s.blind = 1;
        else if (code == 0) code = TSD_DEV_ERR_BAD_PAGE;
      }
  }
  if (code != 0) atomicMin(&s.code, code);
  __syncthreads();
  code = s.code;
  return code != 0x7fffffff ? -code : L;
}

// The path's rows of a request with a page of the prefix missing, whose log-sum-exps
// are not valid: no weight, and the positions that the commit's rows need.  By the
// CTA that has the path's rows, for a KV head.
static __device__ __noinline__ void unweighed_path(const WeightArgs& a, int b, int hk, int P, int L) {
  const int tid = threadIdx.x;
  const long head = (long)b * a.map.Hkv + hk, at = head * a.map.cap + P;
  if (tid <= L) {
    a.acc[at + tid] = 0.f;
    a.pos[at + tid] = a.seen[head] + tid;
  }
  __syncthreads();                       // `seen` has been read
  if (tid != 0) return;
  a.seen[head] += L + 1;
  report_error(a.err, TSD_DEV_ERR_BAD_PAGE, b);
}

bool launch_weights_tc(const tsd_attn_desc& d, const WeightArgs& a, cudaStream_t st);
bool launch_weights_latent(const tsd_attn_desc& d, const WeightArgs& a, cudaStream_t st);

}  // namespace tsd
