// tsd_tree_verify_attn_q8: branch-aware tree attention over an 8-bit prefix
// cache (codes and block exponents of tsd_q8.cuh) plus the scratch pad's rows
// in the element type of q.
//
// Source: "Adapting Tree-Structured Speculative Decoding to DeepSeek-V4"
// (review), research gap item 1 and "How it works" steps 3 and 5, as for
// tsd_tree_verify_attn.  With s = scale q . k, p = exp(s - m), m the running
// maximum: out = sum p v / sum p, lse = m + log sum p, in one pass over the
// keys; splits of the prefix are merged by q8_combine_kernel.
//
// Paths: tcgen05 for bf16 inputs (tsd_q8_few.cu and tsd_q8_tc.cu, heads of 64 or 128
// dims with few or more packed rows; tsd_q8_latent.cu, 576/512), and
// q8_simt_kernel here: fp32 inputs, computed in fp32 on the CUDA cores.  Its
// CTA takes up to RB packed rows, one KV head and one split; a warp takes four
// keys at a time and its lanes split the dims in words of four codes.  The 4 RB dot
// products are summed over the lanes together, each halving of the lanes leaving half
// the products on a lane, so that a lane ends with one (row, key) and computes that
// one's exponential; the weights go back by one shuffle each.  Bound by instructions
// (RB x 2 d multiply-adds per key and about as many again), not by the cache's bytes.
// 33-row trees of 4 requests of 32 heads over 1k to 4k keys: 581 us, 9.7 TFLOP/s of fp32.
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

// DV <= DK; ALIAS: the value is the first DV entries of the key.
template <typename T, int DK, int DV, int RB, bool ALIAS>
__global__ void __launch_bounds__(kSimtThreads)
q8_simt_kernel(const __grid_constant__ Q8AttnArgs a) {
  constexpr int WK = (DK / 4 + 31) / 32, WV = (DV / 4 + 31) / 32;   // words of four per lane
  __shared__ float sm_m[kSimtWarps][RB], sm_l[kSimtWarps][RB];
  __shared__ float sm_o[kSimtWarps][RB][DV];
  grid_dependency_sync();
  const int sp = blockIdx.x, hk = blockIdx.y / a.nrg, rg = blockIdx.y % a.nrg, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = min(max(a.plen[b], 0), a.map.cap);
  const int nsb = q8_splits(a, P);
  if (sp >= nsb) return;
  const int k0 = min(sp * a.split_len, P), k1 = min(P, k0 + a.split_len);

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
    uint32_t kw[kSimtKeys][WK], vw[kSimtKeys][WV];
    // (four keys from a multiple of four are of one block)
    const long row0 = a.map.row(b, hk, j);
    if (row0 < 0 && lane == 0) report_error(a.err, TSD_DEV_ERR_BAD_PAGE, b);
    const long blk = row0 < 0 ? 0 : a.map.block_at(b, hk, j, row0);
    const float fk = q8_scale(a.ke[blk]), fv = ALIAS ? fk : q8_scale(a.ve[blk]);
    const int live = row0 < 0 ? 0 : k1 - j;
#pragma unroll
    for (int u = 0; u < kSimtKeys; ++u) {
      const long row = row0 + u;
#pragma unroll
      for (int t = 0; t < WK; ++t) {
        const int w = lane + 32 * t;
        kw[u][t] = u < live && w < DK / 4 ? __ldg((const uint32_t*)(a.kc + row * DK) + w) : 0u;
      }
#pragma unroll
      for (int t = 0; t < WV; ++t) {
        const int w = lane + 32 * t;
        vw[u][t] = ALIAS ? kw[u][t]
                         : u < live && w < DV / 4 ? __ldg((const uint32_t*)(a.vc + row * DV) + w) : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < kSimtKeys; ++u) {
#pragma unroll
      for (int t = 0; t < WK; ++t) {
        q8_unpack4(kw[u][t], k[u][t]);
#pragma unroll
        for (int x = 0; x < 4; ++x) k[u][t][x] *= fk;
      }
#pragma unroll
      for (int t = 0; t < WV; ++t) {
        q8_unpack4(vw[u][t], v[u][t]);
#pragma unroll
        for (int x = 0; x < 4; ++x) v[u][t][x] *= fv;
      }
    }
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
__global__ void __launch_bounds__(128) q8_combine_kernel(const __grid_constant__ Q8AttnArgs a) {
  using Word = typename std::conditional<sizeof(PT) == 4, uint4, uint2>::type;
  constexpr int kStep = DV / 128 > 0 ? DV / 128 : 1;   // words of four dims per lane
  constexpr int kBatch = kStep > 1 ? 8 : 16;
  grid_dependency_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long row = (long)blockIdx.x * 4 + warp;
  if (row >= (long)a.B * a.R * a.Hq) return;
  const int b = (int)(row / ((long)a.R * a.Hq)), r = (int)((row / a.Hq) % a.R), h = (int)(row % a.Hq);
  const long base = (((long)b * a.Hq + h) * a.R + r) * a.nsplit;
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
    for (int i = 0; i < kStep; ++i) store4((T*)a.out + row * DV + 128 * i + 4 * lane, acc[i]);
  }
  if (lane == 0) a.lse[row] = (mx + log2f(sum)) * 0.69314718055994531f;
}

Q8Plan plan_q8(const tsd_attn_desc& d) {
  Q8Plan p{};
  const int M = d.R * (d.Hq / d.Hkv);
  if (d.dtype == TSD_BF16) {
    // tcgen05: few packed rows on the columns, more on the lanes, in equal
    // groups of at most 128 per CTA; latent heads 64 per CTA
    p.part_bytes = 2;
    if (d.v_aliases_k) {
      p.path = kQ8Latent;
      p.rb = 64;
      p.nrg = (int)ceil_div(M, 64);
    } else if (M <= kQ8FewRows) {
      p.path = kQ8Few;
      p.nrg = 1;
      p.rb = M;
    } else {
      p.path = kQ8Rows;
      p.nrg = (int)ceil_div(M, 128);
      p.rb = (int)ceil_div(M, p.nrg);
    }
    // One CTA per SM.  The split count minimises the modelled time of requests
    // that fill the cache: waves of CTAs times (tiles of a CTA + 4 for its
    // set-up and epilogue), and 5 tiles' time for the merge.
    const long units = (long)d.B * d.Hkv * p.nrg, tiles = ceil_div(d.cap, 128);
    const long lo = ceil_div(tiles, 256), hi = lo > 64 ? lo : tiles < 64 ? tiles : 64;
    long best = -1, best_per = tiles;
    for (long n = lo; n <= hi; ++n) {
      const long per = ceil_div(tiles, n);
      const long cost = ceil_div(units * ceil_div(tiles, per), 152L) * (per + 4) + (per < tiles ? 5 : 0);
      if (best < 0 || cost < best) { best = cost; best_per = per; }
    }
    p.split_len = (int)best_per * 128;
    p.nsplit = (int)ceil_div(d.cap, p.split_len);
    // short splits: the scratch rows are a split of their own, not a longer last one
    p.tree_split = p.nsplit > 1 && best_per <= 8 ? 1 : 0;
    p.nsplit += p.tree_split;
    // More CTAs than SMs and a request's keys in one: the longest requests first, so
    // that the last wave holds the shortest ones.  (32 requests over 1k to 4k keys, 16
    // rows: 57 us in the batch's order, 50 by length; 132 rows: 105 and 104 us; 16 latent
    // requests over 1k to 8k keys: 372 and 278 us; in seven splits, 16 requests over 20k
    // to 32k keys: 165 and 169 us.)
    p.by_length = p.nsplit == 1 && d.B > 1 && d.B <= 64 && units > 152;
  } else {
    p.path = kQ8Simt;
    p.part_bytes = 4;
    // packed rows of a CTA.  (Four or eight, in a graph: 52-row trees of 24 requests over
    // 60 to 88 keys 271 and 245 us, 2-row trees of 32 requests over 1k to 4k keys 372 and
    // 315 us, one 17-row tree over 2k keys 79 and 82 us; latent rows, two or four: 9-row
    // trees of 2 requests over 1000 keys 325 and 284 us.)
    p.rb = d.dk > 128 || M <= 4 ? 4 : 8;
    p.nrg = (int)ceil_div(M, p.rb);
    // about four CTAs per SM over the whole batch, splits of at least 64 keys
    long ns = ceil_div(152L * 4, (long)d.B * d.Hkv * p.nrg);
    const long most = ceil_div(d.cap, 64);
    if (ns > most) ns = most;
    p.split_len = (int)ceil_div(ceil_div(d.cap, ns), 64) * 64;        // (whole blocks)
    p.nsplit = (int)ceil_div(d.cap, p.split_len);
  }
  p.ws_bytes = p.nsplit > 1 ? (size_t)d.B * d.Hq * d.R * p.nsplit *
                                  (d.dv * (size_t)p.part_bytes + sizeof(float2))
                            : 0;
  return p;
}

template <typename T, int DV, typename PT>
void launch_combine(const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  if (p.nsplit <= 1) return;
  const long rows = (long)a.B * a.R * a.Hq;
  launch_plain(q8_combine_kernel<T, DV, PT>, dim3((unsigned)ceil_div(rows, 4)), dim3(128), 0, st, a);
}

template <typename T, int DK, int DV, int RB, bool ALIAS>
void launch_simt(const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  launch(q8_simt_kernel<T, DK, DV, RB, ALIAS>, dim3(p.nsplit, a.map.Hkv * p.nrg, a.B),
         dim3(kSimtThreads), 0, st, a);
  launch_combine<T, DV, float>(a, p, st);
}

}  // namespace
}  // namespace tsd

using namespace tsd;

extern "C" size_t tsd_verify_q8_workspace_size(const tsd_attn_desc* d) {
  if (!q8_desc_ok(d, true)) return 0;
  return plan_q8(*d).ws_bytes;
}

extern "C" tsd_status tsd_tree_verify_attn_q8(const tsd_attn_desc* d, const void* q,
                                              const void* kq, const void* vq, const void* kexp,
                                              const void* vexp, const int32_t* page_table,
                                              int max_pages, int page_size, int num_pages,
                                              const int32_t* prefix_len, const void* ktree,
                                              const void* vtree, const uint64_t* mask, void* out,
                                              float* lse, void* ws, size_t ws_bytes, int32_t* err,
                                              tsd_stream_t stream) {
  if (!q8_desc_ok(d, true) || (((uintptr_t)err) & 3u) != 0) return TSD_ERR_INVALID_ARG;
  const bool alias = d->v_aliases_k != 0;
  if (!ok_ptr(q) || !ok_ptr(kq) || !ok_ptr(kexp) || !ok_ptr(prefix_len) || !ok_ptr(ktree) ||
      !ok_ptr(mask) || !ok_ptr(out) || !ok_ptr(lse))
    return TSD_ERR_INVALID_ARG;
  if (!alias && (!ok_ptr(vq) || !ok_ptr(vexp) || !ok_ptr(vtree))) return TSD_ERR_INVALID_ARG;
  if (!paging_ok(d, page_table, max_pages, page_size, num_pages)) return TSD_ERR_INVALID_ARG;
  const Q8Plan p = plan_q8(*d);
  if ((long)d->Hkv * p.nrg > 65535 || p.nsplit > 65535) return TSD_ERR_INVALID_ARG;
  if (ws_bytes < p.ws_bytes || (p.ws_bytes > 0 && !ok_ptr(ws))) return TSD_ERR_INVALID_ARG;
  Q8AttnArgs a{};
  a.q = q;
  a.kc = (const uint8_t*)kq;
  a.vc = alias ? nullptr : (const uint8_t*)vq;
  a.ke = (const uint8_t*)kexp;
  a.ve = alias ? nullptr : (const uint8_t*)vexp;
  a.plen = prefix_len;
  a.kt = ktree;
  a.vt = alias ? nullptr : vtree;
  a.mask = mask;
  a.out = out;
  a.lse = lse;
  if (p.nsplit > 1) {
    const size_t parts = (size_t)d->B * d->Hq * d->R * p.nsplit;
    a.part_o = ws;
    a.part_meta = (float2*)((char*)ws + parts * d->dv * p.part_bytes);
  }
  a.err = err;
  a.map = cache_map(d, page_table, max_pages, page_size, num_pages);
  a.B = d->B;
  a.R = d->R;
  a.Hq = d->Hq;
  a.g = d->Hq / d->Hkv;
  a.M = d->R * a.g;
  a.nsplit = p.nsplit;
  a.split_len = p.split_len;
  a.nrg = p.nrg;
  a.rb = p.rb;
  a.tree_split = p.tree_split;
  a.by_length = p.by_length;
  a.qscale = d->scale * 1.4426950408889634f;
  a.wait_cycles = wait_budget();
  const cudaStream_t st = (cudaStream_t)stream;
  if (p.path != kQ8Simt) {
    const bool launched = p.path == kQ8Latent ? launch_q8_latent(*d, a, p, st)
                          : p.path == kQ8Few  ? launch_q8_few(*d, a, p, st)
                                              : launch_q8_rows(*d, a, p, st);
    if (!launched) return TSD_ERR_UNSUPPORTED;
    if (alias) launch_combine<__nv_bfloat16, 512, __half>(a, p, st);
    else if (d->dv == 128) launch_combine<__nv_bfloat16, 128, __half>(a, p, st);
    else launch_combine<__nv_bfloat16, 64, __half>(a, p, st);
  } else if (alias) {
    launch_simt<float, 576, 512, 4, true>(a, p, st);
  } else if (d->dk == 128) {
    if (p.rb == 8) launch_simt<float, 128, 128, 8, false>(a, p, st);
    else launch_simt<float, 128, 128, 4, false>(a, p, st);
  } else {
    if (p.rb == 8) launch_simt<float, 64, 64, 8, false>(a, p, st);
    else launch_simt<float, 64, 64, 4, false>(a, p, st);
  }
  return cuda_status();
}
