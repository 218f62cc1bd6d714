// What the calls that append rows to a quantised cache share: which rows a request
// appends, and the checks that make it be skipped.
#pragma once

#include "tsd_q8.cuh"

namespace tsd {

struct AppendSmem {
  int code;
  int32_t path[17];        // commit: source rows
};

constexpr int kNoCode = 0x7fffffff;

// Rows that request b appends (0 for none), or minus the error code that makes
// the request be skipped: every thread of the CTA gets the same answer.  c: its
// count, r: its path entry threadIdx.x (commit; requested with the lengths).
// A: map, rows (source rows per request), S (path length bound).
template <bool kCommit, typename A>
__device__ __forceinline__ int append_rows(const A& a, int b, int P, int c, int r, AppendSmem& s) {
  const int tid = threadIdx.x;
  if (tid == 0) s.code = kNoCode;
  __syncthreads();
  int code = 0;
  const long n = kCommit ? (long)c + 1 : c;
  if (kCommit && (c < 0 || c > a.S)) code = TSD_DEV_ERR_BAD_TREE;
  else if (!kCommit && (c < 0 || c > a.rows)) code = TSD_DEV_ERR_CAPACITY;
  else if (P < 0 || P + n > a.map.cap) code = TSD_DEV_ERR_CAPACITY;
  else {
    if (kCommit && tid < n) {
      if (r < 0 || r >= a.rows) code = TSD_DEV_ERR_BAD_TREE;
      s.path[tid] = r;
    }
    if (a.map.page_size && n > 0) {
      const int p1 = (int)((P + n - 1) / a.map.page_size);
      for (int p = P / a.map.page_size + tid; p <= p1; p += blockDim.x) {
        const int pg = a.map.page_table[(long)b * a.map.max_pages + p];
        if ((pg < 0 || pg >= a.map.num_pages) && code == 0) code = TSD_DEV_ERR_BAD_PAGE;
      }
    }
  }
  if (code != 0) atomicMin(&s.code, code);
  __syncthreads();
  code = s.code;
  return code != kNoCode ? -code : (int)n;
}

}  // namespace tsd
