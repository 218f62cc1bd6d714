// tsd_cache_weights, tsd_cache_weights_q8: attention weight that every cached
// row received from the accepted rows of a round.
//
//   acc[p] = decay * acc[p] + sum_{i <= L} sum_{h of the KV head}
//            exp(scale q_{r_i, h} . k_p - lse_{r_i, h})           p < P
//   acc[P + j] = the same sum over i >= j against scratch row r_j   j <= L
// with r_0..r_L the accepted path and lse the log-sum-exp that the attention of
// the round left.  Rows P..P+L also get their token positions, and `seen`
// advances by L + 1; the call goes between the walk and the commit.
//
// The sum over the columns (accepted rows x heads of the group) belongs to one
// cached row, so with the scores transposed (keys on lanes) no reduction
// crosses a thread.  Paths: tsd_weights_tc.cu and tsd_weights_latent.cu (tcgen05,
// bf16), and weights_simt_kernel here: fp32 inputs and what the tensor cores do not take.
// It is a blocked fp32 product: 128 keys x 32 columns per CTA and step, 64 dims
// at a time in shared memory (rows padded to 68 floats: 16-byte loads of eight
// consecutive keys then start in eight different banks); a thread owns one key
// and 16 columns, so 17 vector loads feed 64 multiply-adds.
#include <cuda_bf16.h>

#include "tsd_host.h"
#include "tsd_weights.cuh"

namespace tsd {
namespace {

constexpr int kSimtThreads = 256, kSimtCols = 32, kSimtDims = 64, kSimtPad = kSimtDims + 4;

template <typename T, int D, bool kQ8>
__global__ void __launch_bounds__(kSimtThreads)
weights_simt_kernel(const __grid_constant__ WeightArgs a) {
  __shared__ __align__(16) float sk[kWeightKeys * kSimtPad];
  __shared__ __align__(16) float sq[kSimtCols * kSimtDims];
  __shared__ float slse[kSimtCols];
  __shared__ float half_sum[kWeightKeys];
  __shared__ PathSmem path;
  grid_dependency_sync();
  const int hk = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int P = a.plen[b];
  const bool on_path = blockIdx.x == gridDim.x - 1;      // the accepted rows themselves
  const int k0 = blockIdx.x * kWeightKeys;
  if (!on_path && k0 >= P) return;
  const int L = weight_path(a, b, P, path);
  if (L < 0) {
    if (on_path && tid == 0) report_error(a.err, -L, b);
    return;
  }
  if (path.blind) {
    if (on_path) unweighed_path(a, b, hk, P, L);
    return;
  }
  const int nkeys = on_path ? L + 1 : min(kWeightKeys, P - k0);
  const int key = tid & (kWeightKeys - 1), half = tid >> 7;
  const int ncol = (L + 1) * a.g;
  float sum = 0.f;
  for (int c0 = 0; c0 < ncol; c0 += kSimtCols) {
    float s[kSimtCols / 2];
#pragma unroll
    for (int n = 0; n < kSimtCols / 2; ++n) s[n] = 0.f;
#pragma unroll 1
    for (int d0 = 0; d0 < D; d0 += kSimtDims) {
      __syncthreads();
      for (int v = tid; v < kWeightKeys * kSimtDims / 8; v += kSimtThreads) {
        const int r = v / (kSimtDims / 8), c = v % (kSimtDims / 8) * 8;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.f;
        if (r < nkeys) {
          if (on_path) {
            load8((const T*)a.kt + (((long)b * a.R + path.rows[r]) * a.map.Hkv + hk) * D + d0 + c, x);
          } else if constexpr (kQ8) {
            const uint2 w = __ldg((const uint2*)((const uint8_t*)a.k +
                                                 a.map.row(b, hk, k0 + r) * D + d0 + c));
            const float f = q8_scale(a.ke[a.map.block(b, hk, k0 + r)]);
            float lo[4], hi[4];
            q8_unpack4(w.x, lo);
            q8_unpack4(w.y, hi);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[j] = lo[j] * f;
              x[4 + j] = hi[j] * f;
            }
          } else {
            load8((const T*)a.k + a.map.row(b, hk, k0 + r) * D + d0 + c, x);
          }
        }
        *(float4*)(sk + r * kSimtPad + c) = make_float4(x[0], x[1], x[2], x[3]);
        *(float4*)(sk + r * kSimtPad + c + 4) = make_float4(x[4], x[5], x[6], x[7]);
      }
      for (int v = tid; v < kSimtCols * kSimtDims / 8; v += kSimtThreads) {
        const int n = v / (kSimtDims / 8), c = v % (kSimtDims / 8) * 8;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.f;
        if (c0 + n < ncol) {
          const int i = (c0 + n) / a.g, h = hk * a.g + (c0 + n) % a.g;
          load8((const T*)a.q + (((long)b * a.R + path.rows[i]) * a.Hq + h) * D + d0 + c, x);
        }
        *(float4*)(sq + n * kSimtDims + c) = make_float4(x[0], x[1], x[2], x[3]);
        *(float4*)(sq + n * kSimtDims + c + 4) = make_float4(x[4], x[5], x[6], x[7]);
      }
      if (d0 == 0 && tid < kSimtCols && c0 + tid < ncol) {
        const int i = (c0 + tid) / a.g, h = hk * a.g + (c0 + tid) % a.g;
        slse[tid] = a.lse[((long)b * a.R + path.rows[i]) * a.Hq + h] * kLog2e;
      }
      __syncthreads();
#pragma unroll 4
      for (int d = 0; d < kSimtDims; d += 4) {
        const float4 kv = *(const float4*)(sk + key * kSimtPad + d);
#pragma unroll
        for (int n = 0; n < kSimtCols / 2; ++n) {
          const float4 qv = *(const float4*)(sq + (half * (kSimtCols / 2) + n) * kSimtDims + d);
          s[n] = fmaf(kv.x, qv.x, s[n]);
          s[n] = fmaf(kv.y, qv.y, s[n]);
          s[n] = fmaf(kv.z, qv.z, s[n]);
          s[n] = fmaf(kv.w, qv.w, s[n]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kSimtCols / 2; ++n) {
      const int col = half * (kSimtCols / 2) + n;
      if (c0 + col < ncol && !(on_path && (c0 + col) / a.g < key))
        sum += exp2f(fmaf(s[n], a.qscale, -slse[col]));
    }
  }
  if (half == 1) half_sum[key] = sum;
  __syncthreads();
  if (half == 0 && key < nkeys) {
    sum += half_sum[key];
    const long at = ((long)b * a.map.Hkv + hk) * a.map.cap;
    if (on_path) {
      a.acc[at + P + key] = sum;
      a.pos[at + P + key] = a.seen[b * a.map.Hkv + hk] + key;
    } else {
      a.acc[at + k0 + key] = fmaf(a.decay, a.acc[at + k0 + key], sum);
    }
  }
  __syncthreads();                       // `seen` has been read
  if (on_path && tid == 0) a.seen[b * a.map.Hkv + hk] += L + 1;
}

template <typename T, int D>
void launch_simt(const tsd_attn_desc& d, const WeightArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)ceil_div(d.cap, kWeightKeys) + 1, d.Hkv, d.B);
  if (a.ke != nullptr) launch(weights_simt_kernel<T, D, true>, grid, dim3(kSimtThreads), 0, st, a);
  else launch(weights_simt_kernel<T, D, false>, grid, dim3(kSimtThreads), 0, st, a);
}

tsd_status weights_impl(const tsd_attn_desc* d, int S, const void* q, const void* k,
                        const void* kexp, bool q8, const int32_t* page_table, int max_pages,
                        int page_size, int num_pages, const int32_t* prefix_len,
                        const void* ktree, const int32_t* accept_rows, const int32_t* accept_len,
                        const float* lse, float decay, float* acc, int32_t* pos, int32_t* seen,
                        int32_t* err, tsd_stream_t stream) {
  if (!q8_desc_ok(d, true) || (((uintptr_t)err) & 3u) != 0) return TSD_ERR_INVALID_ARG;
  if (S < 1 || S > 16 || !(decay >= 0.f && decay <= 1.f) || d->Hkv > 65535)
    return TSD_ERR_INVALID_ARG;
  if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(prefix_len) || !ok_ptr(ktree) || !ok_ptr(accept_rows) ||
      !ok_ptr(accept_len) || !ok_ptr(lse) || !ok_ptr(acc) || !ok_ptr(pos) || !ok_ptr(seen) ||
      (q8 && !ok_ptr(kexp)))
    return TSD_ERR_INVALID_ARG;
  if (!paging_ok(d, page_table, max_pages, page_size, num_pages)) return TSD_ERR_INVALID_ARG;
  WeightArgs a{};
  a.q = q;
  a.k = k;
  a.ke = q8 ? (const uint8_t*)kexp : nullptr;
  a.plen = prefix_len;
  a.kt = ktree;
  a.path = accept_rows;
  a.path_len = accept_len;
  a.lse = lse;
  a.acc = acc;
  a.pos = pos;
  a.seen = seen;
  a.err = err;
  a.map = cache_map(d, page_table, max_pages, page_size, num_pages);
  a.R = d->R;
  a.Hq = d->Hq;
  a.g = d->Hq / d->Hkv;
  a.S = S;
  a.decay = decay;
  a.qscale = d->scale * kLog2e;
  a.wait_cycles = wait_budget();
  const cudaStream_t st = (cudaStream_t)stream;
  const bool f32 = d->dtype == TSD_F32;
  if (launch_weights_tc(*d, a, st) || launch_weights_latent(*d, a, st)) return cuda_status();
  if (d->dk == 576) {
    if (f32) launch_simt<float, 576>(*d, a, st);
    else launch_simt<__nv_bfloat16, 576>(*d, a, st);
  } else if (d->dk == 128) {
    if (f32) launch_simt<float, 128>(*d, a, st);
    else launch_simt<__nv_bfloat16, 128>(*d, a, st);
  } else {
    if (f32) launch_simt<float, 64>(*d, a, st);
    else launch_simt<__nv_bfloat16, 64>(*d, a, st);
  }
  return cuda_status();
}

}  // namespace
}  // namespace tsd

using namespace tsd;

extern "C" tsd_status tsd_cache_weights(const tsd_attn_desc* d, int S, const void* q,
                                        const void* kcache, const int32_t* page_table,
                                        int max_pages, int page_size, int num_pages,
                                        const int32_t* prefix_len, const void* ktree,
                                        const int32_t* accept_rows, const int32_t* accept_len,
                                        const float* lse, float decay, float* acc, int32_t* pos,
                                        int32_t* seen, int32_t* err, tsd_stream_t stream) {
  return weights_impl(d, S, q, kcache, nullptr, false, page_table, max_pages, page_size, num_pages,
                      prefix_len, ktree, accept_rows, accept_len, lse, decay, acc, pos, seen, err,
                      stream);
}

extern "C" tsd_status tsd_cache_weights_q8(const tsd_attn_desc* d, int S, const void* q,
                                           const void* kq, const void* kexp,
                                           const int32_t* page_table, int max_pages,
                                           int page_size, int num_pages,
                                           const int32_t* prefix_len, const void* ktree,
                                           const int32_t* accept_rows, const int32_t* accept_len,
                                           const float* lse, float decay, float* acc,
                                           int32_t* pos, int32_t* seen, int32_t* err,
                                           tsd_stream_t stream) {
  return weights_impl(d, S, q, kq, kexp, true, page_table, max_pages, page_size, num_pages,
                      prefix_len, ktree, accept_rows, accept_len, lse, decay, acc, pos, seen, err,
                      stream);
}
