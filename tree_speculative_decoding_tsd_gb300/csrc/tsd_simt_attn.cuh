// Tree attention over a quantised cache on the CUDA cores, in fp32, and the merge of a
// request's splits, which the tensor-core paths take, too.
//
// A CTA takes up to RB packed rows (tree rows x query heads of a KV head), one KV head and
// one split; a warp takes four keys at a time and its lanes split the dims in words of
// four.  The 4 RB dot products are summed over the lanes together, each halving of the
// lanes leaving half the products on a lane, so that a lane ends with one (row, key) and
// computes that one's exponential; the weights go back by one shuffle each.  Bound by
// instructions (RB x 2 d multiply-adds per key and about as many again), not by the
// cache's bytes.
#pragma once

#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "tsd_common.cuh"
#include "tsd_host.h"
#include "tsd_q8_attn.cuh"
#include "tsd_tcgen05.cuh"

namespace tsd {
namespace {

constexpr int kSimtThreads = 128, kSimtWarps = 4, kSimtKeys = 4;

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
  const float4 v = __ldg((const float4*)p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void store_out(float* p, float x) { *p = x; }

// Keys: how the prefix is read; its kDv <= kDk, kAlias: the value is the first kDv entries
// of the key.
template <typename T, int RB, typename Keys>
__global__ void __launch_bounds__(kSimtThreads)
simt_attn_kernel(const __grid_constant__ Q8AttnArgs a) {
  constexpr int DK = Keys::kDk, DV = Keys::kDv;
  constexpr bool ALIAS = Keys::kAlias;
  constexpr int WK = (DK / 4 + 31) / 32, WV = (DV / 4 + 31) / 32;   // words of four per lane
  __shared__ float sm_m[kSimtWarps][RB], sm_l[kSimtWarps][RB];
  __shared__ float sm_o[kSimtWarps][RB][DV];
  grid_dependency_sync();
  const int sp = blockIdx.x, hk = blockIdx.y / a.nrg, rg = blockIdx.y % a.nrg, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = min(max(a.plen[b], 0), a.map.cap);
  const int nsb = q8_splits(a, P);
  if (sp >= nsb) return;
  const int k0 = q8_first(a, P, sp), k1 = q8_end(a, P, k0);

  // the (row, key of four) that this lane's score is of; the row's maximum, the sum of
  // its keys' weights, and what the row sees
  const int mi = (lane >> 2) & (RB - 1), mu = lane & 3;
  float m = -INFINITY, l = 0.f;
  float qv[RB][WK][4], o[RB][WV][4];
  const int nrows = min(RB, a.M - rg * RB);
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const bool valid = i < nrows;
    const int p = valid ? rg * RB + i : 0;
    const int r = p / a.g, h = hk * a.g + p % a.g;
    const T* qp = (const T*)a.q + (((long)b * a.R + r) * a.Hq + h) * DK;
#pragma unroll
    for (int t = 0; t < WK; ++t) {
      const int w = lane + 32 * t;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (valid && w < DK / 4) load4(qp + 4 * w, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) qv[i][t][j] = x[j];
    }
#pragma unroll
    for (int t = 0; t < WV; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][t][j] = 0.f;
  }

  const int tr = mi < nrows ? (rg * RB + mi) / a.g : 0;
  const uint64_t rmask = tr > 0 ? a.mask[(long)b * a.R + tr] : 0ull;

  // four keys with their values (zero where there is none), the first `live` of them
  // there; for the tree, from row j0
  auto visit = [&](float (&k)[kSimtKeys][WK][4], float (&v)[kSimtKeys][WV][4], int live, bool tree,
                   int j0) {
    float s[RB * kSimtKeys];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int u = 0; u < kSimtKeys; ++u) {
        float x = 0.f;
#pragma unroll
        for (int t = 0; t < WK; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) x = fmaf(qv[i][t][j], k[u][t][j], x);
        s[i * kSimtKeys + u] = x;
      }
    const float dot = warp_reduce_scatter<RB * kSimtKeys, false>(s, lane);
    const int j = j0 + mu;
    const bool sees = mi < nrows && mu < live && (!tree || j == 0 || ((rmask >> (j - 1)) & 1ull));
    const float x = sees ? dot * a.qscale : -INFINITY;
    float mx = fmaxf(x, __shfl_xor_sync(kFull, x, 1));
    mx = fmaxf(fmaxf(mx, __shfl_xor_sync(kFull, mx, 2)), m);
    // (a score of -inf does not count, whatever its value; one that is NaN does)
    const bool counts = !(x == -INFINITY);
    const float al = mx == m ? 1.f : m == -INFINITY ? 0.f : exp2f(m - mx);
    const float p = counts ? exp2f(x - mx) : 0.f;
    m = mx;
    l = fmaf(l, al, p);
    if (__any_sync(kFull, al != 1.f)) {
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const float f = __shfl_sync(kFull, al, i * kSimtKeys);
#pragma unroll
        for (int t = 0; t < WV; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[i][t][c] *= f;
      }
    }
    const uint32_t seen = __ballot_sync(kFull, counts);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int u = 0; u < kSimtKeys; ++u) {
        if (!((seen >> (i * kSimtKeys + u)) & 1u)) continue;
        const float f = __shfl_sync(kFull, p, i * kSimtKeys + u);
#pragma unroll
        for (int t = 0; t < WV; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[i][t][c] = fmaf(f, v[u][t][c], o[i][t][c]);
      }
  };

  for (int j = k0 + warp * kSimtKeys; j < k1; j += kSimtWarps * kSimtKeys) {
    float k[kSimtKeys][WK][4], v[kSimtKeys][WV][4];
    // (four keys from a multiple of four are of one page and one block)
    const long row0 = a.map.row(b, hk, j);
    if (row0 < 0 && lane == 0) report_error(a.err, TSD_DEV_ERR_BAD_PAGE, b);
    const int live = row0 < 0 ? 0 : k1 - j;
    Keys::read(a, b, hk, j, row0, live, lane, k, v);
    visit(k, v, live, false, 0);
  }
  if (sp == nsb - 1) {
    const T* kt = (const T*)a.kt + ((long)b * a.R * a.map.Hkv + hk) * DK;
    const T* vt = ALIAS ? kt : (const T*)a.vt + ((long)b * a.R * a.map.Hkv + hk) * DV;
    constexpr int VS = ALIAS ? DK : DV;
    for (int j = warp * kSimtKeys; j < a.R; j += kSimtWarps * kSimtKeys) {
      float k[kSimtKeys][WK][4], v[kSimtKeys][WV][4];
      const int live = a.R - j;
#pragma unroll
      for (int u = 0; u < kSimtKeys; ++u) {
#pragma unroll
        for (int t = 0; t < WK; ++t) {
          const int w = lane + 32 * t;
          float x[4] = {0.f, 0.f, 0.f, 0.f};
          if (u < live && w < DK / 4) load4(kt + (long)(j + u) * a.map.Hkv * DK + 4 * w, x);
#pragma unroll
          for (int c = 0; c < 4; ++c) k[u][t][c] = x[c];
        }
#pragma unroll
        for (int t = 0; t < WV; ++t) {
          const int w = lane + 32 * t;
          float x[4] = {0.f, 0.f, 0.f, 0.f};
          if (u < live && w < DV / 4) load4(vt + (long)(j + u) * a.map.Hkv * VS + 4 * w, x);
#pragma unroll
          for (int c = 0; c < 4; ++c) v[u][t][c] = x[c];
        }
      }
      visit(k, v, live, true, j);
    }
  }

  // merge the four warps' running states
  l += __shfl_xor_sync(kFull, l, 1);
  l += __shfl_xor_sync(kFull, l, 2);
  if (lane < RB * kSimtKeys && mu == 0) {
    sm_m[warp][mi] = m;
    sm_l[warp][mi] = l;
  }
#pragma unroll
  for (int i = 0; i < RB; ++i) {
#pragma unroll
    for (int t = 0; t < WV; ++t)
      if (lane + 32 * t < DV / 4)
        *(float4*)&sm_o[warp][i][4 * (lane + 32 * t)] =
            make_float4(o[i][t][0], o[i][t][1], o[i][t][2], o[i][t][3]);
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < nrows * DV; idx += kSimtThreads) {
    const int i = idx / DV, c = idx - i * DV;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSimtWarps; ++w) mx = fmaxf(mx, sm_m[w][i]);
    float lt = 0.f, ot = 0.f;
#pragma unroll
    for (int w = 0; w < kSimtWarps; ++w) {
      const float wt = sm_m[w][i] == -INFINITY ? 0.f : exp2f(sm_m[w][i] - mx);
      lt = fmaf(sm_l[w][i], wt, lt);
      ot = fmaf(sm_o[w][i][c], wt, ot);
    }
    // (a split whose pages are all missing saw nothing: weight 0)
    const float res = mx == -INFINITY && lt == 0.f ? 0.f : ot / lt;
    const float lse2 = mx + log2f(lt);
    const int p = rg * RB + i;
    const int r = p / a.g, h = hk * a.g + p % a.g;
    const long orow = ((long)b * a.R + r) * a.Hq + h;
    if (nsb == 1) {
      store_out((T*)a.out + orow * DV + c, res);
      if (c == 0) a.lse[orow] = lse2 * 0.69314718055994531f;
    } else {
      const long prow = (((long)b * a.Hq + h) * a.R + r) * a.nsplit + sp;
      ((float*)a.part_o)[prow * DV + c] = res;
      if (c == 0) a.part_meta[prow] = make_float2(lse2, 1.f);
    }
  }
}

// W words of a split's output: four fp32, or eight fp16.
__device__ __forceinline__ void part_values(const uint4& w, float (&x)[4], float) {
  x[0] = __uint_as_float(w.x);
  x[1] = __uint_as_float(w.y);
  x[2] = __uint_as_float(w.z);
  x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void part_values(const uint2& w, float (&x)[4], __half) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *(uint2*)p = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Merge of the splits of one output row: with L_s the log2-sum-exp and c_s the
// scale of split s, out = sum_s 2^(L_s - L) c_s O_s and L = log2 sum_s 2^(L_s).
// One warp per row, four dims per lane and step.  Bounded by latency, so the outputs of the first kBatch splits are
// requested together with the sums, before any weight is known.  PT: element type
// of the splits' outputs.
template <typename T, int DV, typename PT>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ Q8AttnArgs a) {
  using Word = typename std::conditional<sizeof(PT) == 4, uint4, uint2>::type;
  constexpr int kStep = DV / 128 > 0 ? DV / 128 : 1;   // words of four dims per lane
  constexpr int kBatch = kStep > 1 ? 8 : 16;
  grid_dependency_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long row = (long)blockIdx.x * 4 + warp;
  if (row >= (long)a.B * a.nr * a.Hq) return;
  const int b = (int)(row / ((long)a.nr * a.Hq)), r = (int)((row / a.Hq) % a.nr), h = (int)(row % a.Hq);
  const long base = (((long)b * a.Hq + h) * a.nr + r) * a.nsplit;
  const long orow = ((long)b * a.R + a.r0 + r) * a.Hq + h;
  const PT* const parts = (const PT*)a.part_o + base * DV;
  const bool active = DV >= 128 || lane < DV / 4;
  // (the workspace holds nsplit entries per row; those of splits without work are
  // read, too, and left out)
  float2 meta = lane < a.nsplit ? a.part_meta[base + lane] : make_float2(-INFINITY, 0.f);
  Word w[kBatch][kStep];
#pragma unroll
  for (int s = 0; s < kBatch; ++s)
#pragma unroll
    for (int i = 0; i < kStep; ++i)
      if (s < a.nsplit && active) w[s][i] = *(const Word*)(parts + (long)s * DV + 128 * i + 4 * lane);
  const int P = min(max(a.plen[b], 0), a.map.cap);
  const int n = q8_splits(a, P);
  if (n == 1) return;                    // written by its only split
  if (lane >= n) meta.x = -INFINITY;
  float mx = meta.x;
  for (int s = lane + 32; s < n; s += 32) mx = fmaxf(mx, a.part_meta[base + s].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
  float sum = meta.x == -INFINITY ? 0.f : exp2f(meta.x - mx);
  for (int s = lane + 32; s < n; s += 32) {
    const float L = a.part_meta[base + s].x;
    if (L != -INFINITY) sum += exp2f(L - mx);
  }
  sum = warp_total(sum);
  // the weight first, then the scale: each alone may be far from 1
  float wt = meta.x == -INFINITY ? 0.f : exp2f(meta.x - mx) / sum * meta.y;
  float acc[kStep][4];
#pragma unroll
  for (int i = 0; i < kStep; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  for (int s0 = 0; s0 < n; s0 += kBatch) {
    if (s0 > 0) {
#pragma unroll
      for (int s = 0; s < kBatch; ++s)
#pragma unroll
        for (int i = 0; i < kStep; ++i)
          if (s0 + s < n && active) w[s][i] = *(const Word*)(parts + (long)(s0 + s) * DV + 128 * i + 4 * lane);
      if (s0 % 32 == 0) {
        meta = s0 + lane < n ? a.part_meta[base + s0 + lane] : make_float2(-INFINITY, 0.f);
        wt = meta.x == -INFINITY ? 0.f : exp2f(meta.x - mx) / sum * meta.y;
      }
    }
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      if (s0 + s >= n) break;            // (the same for the whole warp)
      const float ws = __shfl_sync(kFull, wt, (s0 + s) & 31);
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        float x[4];
        part_values(w[s][i], x, PT());
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(ws, x[j], acc[i][j]);
      }
    }
  }
  if (active) {
#pragma unroll
    for (int i = 0; i < kStep; ++i) store4((T*)a.out + orow * DV + 128 * i + 4 * lane, acc[i]);
  }
  if (lane == 0) a.lse[orow] = (mx + log2f(sum)) * 0.69314718055994531f;
}

template <typename T, int DV, typename PT>
void launch_combine(const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  if (p.nsplit <= 1) return;
  const long rows = (long)a.B * a.nr * a.Hq;
  launch_plain(combine_kernel<T, DV, PT>, dim3((unsigned)ceil_div(rows, 4)), dim3(128), 0, st, a);
}

template <typename T, int RB, typename Keys>
void launch_simt(const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  launch(simt_attn_kernel<T, RB, Keys>, dim3(p.nsplit, a.map.Hkv * p.nrg, a.B),
         dim3(kSimtThreads), 0, st, a);
  launch_combine<T, Keys::kDv, float>(a, p, st);
}

}  // namespace
}  // namespace tsd
