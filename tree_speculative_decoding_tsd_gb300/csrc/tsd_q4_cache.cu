// tsd_cache_write_q4, tsd_commit_path_q4, tsd_cache_read_q4: rows into the 4-bit cache,
// and back.
//
// For each request, n rows land at positions P..P+n-1 (P the prefix length): rows
// 0..n-1 of a dense [B][T] array (a prefill), or the accepted rows of the scratch pad (a
// commit; Source: "Adapting Tree-Structured Speculative Decoding to DeepSeek-V4"
// (review), "Secret weapon" and "How it works" step 6).  Per group of 32 dims:
//   x* = the element of largest magnitude,  s = bf16(-x* / 8),
//   c  = clamp(round(x / s), -8, 7) + 8;  read back: (c - 8) s
//
// Writing, two lanes hold a group, sixteen elements (two words of codes) each: a scale and
// its inverse cost as much as eight elements do, and a shuffle joins two ranges (eight elements
// a lane: 40 instead of 28 us for the prompt below).  Reading, a lane has eight elements.
//
// 4 x up to 8192 rows of 8 heads: written in 28 us (22 by the bytes; issue slots 62%, memory 59%),
// read back in 23; 32 requests of 1k to 4k rows read from pages in 50 us (47 by the bytes).
#include <cuda_bf16.h>
#include <math.h>

#include "tsd_append.cuh"
#include "tsd_host.h"
#include "tsd_q4.cuh"

namespace tsd {
namespace {

struct Q4CacheArgs {
  const void* src[2];      // K, V rows in: [B][rows][Hkv][d]
  void* dst[2];            // and out (read)
  uint32_t* codes[2];
  uint16_t* scales[2];
  int32_t* prefix_len;
  const int32_t* first;    // read: first position
  const int32_t* count;    // commit: accepted draft rows L (L + 1 rows move); else rows n
  const int32_t* path;     // commit: [B][S+1] source rows
  int32_t* err;
  CacheMap map;
  int rows, S;             // rows per request of src or dst; path length bound
};

// Threads, positions of a CTA and rows of a lane requested together (write, read).  Prompt and its
// read-back / read of 32 requests in a graph: 60 / 63 us; four rows 73 / 87, one 60 / 67; 128
// threads 62 / 66, 512 threads 69 / 79; 64 positions 65 / 69.
constexpr int kThreads = 256;
constexpr int kTokens = 32;
constexpr int kUnroll = 2;
constexpr int kPathThreads = 512;
// Appends of at most this many rows (those of a path) take one CTA per request and no second
// launch.
constexpr int kFewRows = 17;

// Sixteen elements of a row: half a group.  range: the group's largest element and minus its
// smallest (NaN if any is), from two lanes.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
struct RowF32 {
  float4 a[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = __ldg((const float4*)p + i);
  }
  template <int kHalf> __device__ __forceinline__ void values(float (&x)[8]) const {
    const float4 u = a[2 * kHalf], v = a[2 * kHalf + 1];
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
  }
  __device__ __forceinline__ float2 range() const {
    float x[8], y[8];
    values<0>(x);
    values<1>(y);
    float hi = x[0], lo = -x[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi = max_nan(max_nan(hi, x[i]), y[i]);
      lo = max_nan(max_nan(lo, -x[i]), -y[i]);
    }
    hi = max_nan(hi, __shfl_xor_sync(kFull, hi, 1));
    lo = max_nan(lo, __shfl_xor_sync(kFull, lo, 1));
    return make_float2(hi, lo);
  }
};
struct RowBf16 {
  uint4 a[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a[0] = __ldg((const uint4*)p);
    a[1] = __ldg((const uint4*)p + 1);
  }
  template <int kHalf> __device__ __forceinline__ void values(float (&x)[8]) const {
    const uint32_t w[4] = {a[kHalf].x, a[kHalf].y, a[kHalf].z, a[kHalf].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ float2 range() const {
    const uint32_t w[8] = {a[0].x, a[0].y, a[0].z, a[0].w, a[1].x, a[1].y, a[1].z, a[1].w};
    auto pair = [](const uint32_t& v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); };
    __nv_bfloat162 h = pair(w[0]), l = h;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      h = __hmax2_nan(h, pair(w[i]));
      l = __hmin2_nan(l, pair(w[i]));
    }
    // (largest, minus the smallest) side by side, for one shuffle
    l = __hneg2(l);
    __nv_bfloat162 m = __hmax2_nan(__lows2bfloat162(h, l), __highs2bfloat162(h, l));
    const uint32_t o = __shfl_xor_sync(kFull, *reinterpret_cast<const uint32_t*>(&m), 1);
    m = __hmax2_nan(m, pair(o));
    return __bfloat1622float2(m);
  }
};
template <typename T> struct RowOf { using type = RowF32; };
template <> struct RowOf<__nv_bfloat16> { using type = RowBf16; };

// Lane c (of D / 16) of a row: its sixteen elements to two words of codes and, from the first
// lane of a group, the group's scale.  All lanes of a warp take part.
template <typename Row>
__device__ __forceinline__ void put_row(const Row& r, bool live, uint32_t* codes, uint16_t* scales,
                                        int c) {
  const float2 m = r.range();
  const uint32_t s = q4_scale(m.x, -m.y);
  const float inv = q4_inverse(s);
  float x[8], y[8];
  r.template values<0>(x);
  r.template values<1>(y);
  const uint32_t w0 = inv == 0.f ? 0x88888888u : q4_word(x, inv);
  const uint32_t w1 = inv == 0.f ? 0x88888888u : q4_word(y, inv);
  if (!live) return;
  ((uint2*)codes)[c] = make_uint2(w0, w1);
  if ((c & 1) == 0) scales[c >> 1] = (uint16_t)s;
}

// Rows of head 0 of positions pos .. pos + n - 1 (n <= kTokens), for the whole CTA; a head
// further on they lie the returned distance further.
__device__ __forceinline__ long head_rows(const CacheMap& m, int b, int pos, int n, long* rows) {
  if ((int)threadIdx.x < n) rows[threadIdx.x] = m.row(b, 0, pos + threadIdx.x);
  __syncthreads();
  return m.page_size ? m.page_size : m.cap;
}

// Prefill: grid (tokens, K or V, request).  prefix_len changes only in
// q4_advance_kernel, so every CTA reads the length of before.  A warp takes kUnroll times
// 512 / D consecutive positions of a head, which it writes side by side.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) write_q4_kernel(const __grid_constant__ Q4CacheArgs a) {
  constexpr int VR = D / 16, kRows = 32 / VR, kBatch = kRows * kUnroll;
  using Row = typename RowOf<T>::type;
  __shared__ AppendSmem s;
  grid_dependency_sync();
  const int b = blockIdx.z, part = blockIdx.y, P = a.prefix_len[b], n0 = a.count[b];
  const int n = append_rows<false>(a, b, P, n0, 0, s);
  const int t0 = blockIdx.x * kTokens;
  if (t0 >= n) return;                                 // (no rows, or an error)
  __shared__ long rows[kTokens];
  const long apart = head_rows(a.map, b, P + t0, min(kTokens, n - t0), rows);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane % VR, sub = lane / VR;
  const T* const src = (const T*)a.src[part] + (long)b * a.rows * a.map.Hkv * D;
  constexpr int kPerHead = kTokens / kBatch;
  for (int i = warp; i < a.map.Hkv * kPerHead; i += kThreads / 32) {
    const int h = i / kPerHead, t = t0 + (i % kPerHead) * kBatch + sub;
    Row r[kUnroll];
    long row[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int x = min(t + u * kRows, n - 1);
      r[u].load(src + ((long)x * a.map.Hkv + h) * D + c * 16);
      row[u] = rows[x - t0] + h * apart;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      put_row(r[u], t + u * kRows < n, a.codes[part] + row[u] * (D / 8),
              a.scales[part] + row[u] * (D / kQ4Group), c);
  }
}

__global__ void __launch_bounds__(128) q4_advance_kernel(const __grid_constant__ Q4CacheArgs a) {
  __shared__ AppendSmem s;
  grid_dependency_sync();
  const int b = blockIdx.x, P = a.prefix_len[b], c = a.count[b];
  const int n = append_rows<false>(a, b, P, c, 0, s);
  if (threadIdx.x != 0) return;
  if (n < 0) report_error(a.err, -n, b);
  else a.prefix_len[b] = P + n;
}

// Few rows: one CTA per request, which reads the prefix length and advances it itself.
template <typename T, int D, bool kPath>
__global__ void __launch_bounds__(kPathThreads)
append_q4_kernel(const __grid_constant__ Q4CacheArgs a) {
  constexpr int VR = D / 16, kRows = 32 / VR;
  using Row = typename RowOf<T>::type;
  __shared__ AppendSmem s;
  grid_dependency_sync();
  const int b = blockIdx.x, P = a.prefix_len[b], c0 = a.count[b];
  const int r0 = kPath && threadIdx.x <= a.S ? a.path[(long)b * (a.S + 1) + threadIdx.x] : 0;
  const int n = append_rows<kPath>(a, b, P, c0, r0, s);  // (its barrier: the whole CTA has read P)
  if (threadIdx.x == 0) {
    if (n < 0) report_error(a.err, -n, b);
    else a.prefix_len[b] = P + n;
  }
  if (n <= 0) return;
  static_assert(kFewRows <= kTokens, "a row per thread");
  __shared__ long rows[kTokens];
  const long apart = head_rows(a.map, b, P, n, rows);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane % VR, sub = lane / VR, Hkv = a.map.Hkv;
  const int work = 2 * Hkv * n;                        // (part, head, row)
  for (int i0 = warp * kRows; i0 < work; i0 += kPathThreads / 32 * kRows) {
    const int i = i0 + sub, j = min(i, work - 1);
    const int t = j % n, h = j / n % Hkv, part = j / n / Hkv;
    Row r;
    r.load((const T*)a.src[part] + (((long)b * a.rows + (kPath ? s.path[t] : t)) * Hkv + h) * D + c * 16);
    const long row = rows[t] + h * apart;
    put_row(r, i < work, a.codes[part] + row * (D / 8), a.scales[part] + row * (D / kQ4Group), c);
  }
}

// The eight values of a word, times the scale, to p.
__device__ __forceinline__ void store_word(float* p, uint32_t w, uint32_t scale) {
  float x[8];
  q4_values(w, x);
  const float f = bf16_value(scale);
  ((float4*)p)[0] = make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
  ((float4*)p)[1] = make_float4(x[4] * f, x[5] * f, x[6] * f, x[7] * f);
}
// bf16: a code in the lowest bits of 128 is 128 + c, less 136 exactly c - 8; the product with the
// scale is rounded once, as that in fp32 (which is exact) would be.
__device__ __forceinline__ void store_word(__nv_bfloat16* p, uint32_t w, uint32_t scale) {
  const uint32_t f = scale | scale << 16;
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 x = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c),
                                     __bfloat162bfloat162(__ushort_as_bfloat16(0x4308)));
    const __nv_bfloat162 y = __hmul2(x, *reinterpret_cast<const __nv_bfloat162*>(&f));
    out[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  *(uint4*)p = make_uint4(out[0], out[1], out[2], out[3]);
}

// Positions first..first+count-1 to rows 0.. of [B][rows][Hkv][d]: as the write, the
// other way.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_q4_kernel(const __grid_constant__ Q4CacheArgs a) {
  constexpr int VR = D / 8, kRows = 32 / VR, kBatch = kRows * kUnroll;
  __shared__ int s_code;
  grid_dependency_sync();
  const int b = blockIdx.z, part = blockIdx.y, tid = threadIdx.x;
  const int P = a.prefix_len[b], p0 = a.first[b], n = a.count[b];
  if (tid == 0) s_code = kNoCode;
  __syncthreads();
  int code = 0;
  if (P < 0 || P > a.map.cap || n < 0 || n > a.rows || p0 < 0 || (long)p0 + n > P) {
    code = TSD_DEV_ERR_CAPACITY;
  } else if (a.map.page_size && n > 0) {
    for (int p = p0 / a.map.page_size + tid; p <= (p0 + n - 1) / a.map.page_size; p += kThreads) {
      const int pg = a.map.page_table[(long)b * a.map.max_pages + p];
      if (pg < 0 || pg >= a.map.num_pages) code = TSD_DEV_ERR_BAD_PAGE;
    }
  }
  if (code != 0) atomicMin(&s_code, code);
  __syncthreads();
  if (s_code != kNoCode) {
    if (tid == 0 && blockIdx.x == 0 && part == 0) report_error(a.err, s_code, b);
    return;
  }
  const int t0 = blockIdx.x * kTokens;
  if (t0 >= n) return;
  __shared__ long rows[kTokens];
  const long apart = head_rows(a.map, b, p0 + t0, min(kTokens, n - t0), rows);
  const int lane = tid & 31, warp = tid >> 5;
  const int c = lane % VR, sub = lane / VR;
  T* const dst = (T*)a.dst[part] + (long)b * a.rows * a.map.Hkv * D;
  constexpr int kPerHead = kTokens / kBatch;
  for (int i = warp; i < a.map.Hkv * kPerHead; i += kThreads / 32) {
    const int h = i / kPerHead, t = t0 + (i % kPerHead) * kBatch + sub;
    uint32_t w[kUnroll], f[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long row = rows[min(t + u * kRows, n - 1) - t0] + h * apart;
      // (Read once, past L1: 32 requests 54 us in a graph, 63 with __ldg.  Scales of fp32 rows,
      // whose stores leave more time between loads: 73 so, 87 past L1.)
      w[u] = __ldcs(a.codes[part] + row * (D / 8) + c);
      const uint16_t* const scale = a.scales[part] + row * (D / kQ4Group) + (c >> 2);
      f[u] = sizeof(T) == 2 ? __ldcg(scale) : __ldg(scale);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (t + u * kRows >= n) break;
      store_word(dst + ((long)(t + u * kRows) * a.map.Hkv + h) * D + c * 8, w[u], f[u]);
    }
  }
}

template <typename T, int D>
void launch_append(const Q4CacheArgs& a, int B, bool commit, cudaStream_t st) {
  if (commit) {
    launch(append_q4_kernel<T, D, true>, dim3(B), dim3(kPathThreads), 0, st, a);
  } else if (a.rows <= kFewRows) {
    launch(append_q4_kernel<T, D, false>, dim3(B), dim3(kPathThreads), 0, st, a);
  } else {
    const int most = a.rows < a.map.cap ? a.rows : a.map.cap;
    launch(write_q4_kernel<T, D>, dim3((unsigned)ceil_div(most, kTokens), 2, B), dim3(kThreads), 0, st, a);
    launch(q4_advance_kernel, dim3(B), dim3(128), 0, st, a);
  }
}

tsd_status cache_args(const tsd_attn_desc* d, const void* kq, const void* vq, const void* kscale,
                      const void* vscale, const int32_t* page_table, int max_pages, int page_size,
                      int num_pages, const int32_t* prefix_len, int32_t* err, Q4CacheArgs* a) {
  const tsd_status st = q4_desc_status(d);
  if (st != TSD_OK) return st;
  if (!ok_ptr(kq) || !ok_ptr(vq) || !ok_ptr(kscale) || !ok_ptr(vscale) || !ok_ptr(prefix_len) ||
      (((uintptr_t)err) & 3u) != 0 || !paging_ok(d, page_table, max_pages, page_size, num_pages))
    return TSD_ERR_INVALID_ARG;
  a->codes[0] = (uint32_t*)kq;
  a->codes[1] = (uint32_t*)vq;
  a->scales[0] = (uint16_t*)kscale;
  a->scales[1] = (uint16_t*)vscale;
  a->prefix_len = const_cast<int32_t*>(prefix_len);
  a->err = err;
  a->map = cache_map(d, page_table, max_pages, page_size, num_pages);
  return TSD_OK;
}

tsd_status append_impl(const tsd_attn_desc* d, int rows, int S, const void* k, const void* v,
                       const int32_t* path, const int32_t* count, Q4CacheArgs a, bool commit,
                       tsd_stream_t stream) {
  if (rows < 1 || (commit && (S < 1 || S > 16 || !ok_ptr(path)))) return TSD_ERR_INVALID_ARG;
  if (!ok_ptr(k) || !ok_ptr(v) || !ok_ptr(count)) return TSD_ERR_INVALID_ARG;
  a.src[0] = k;
  a.src[1] = v;
  a.count = count;
  a.path = path;
  a.rows = rows;
  a.S = S;
  const cudaStream_t st = (cudaStream_t)stream;
  const bool f32 = d->dtype == TSD_F32;
  if (d->dk == 128) {
    if (f32) launch_append<float, 128>(a, d->B, commit, st);
    else launch_append<__nv_bfloat16, 128>(a, d->B, commit, st);
  } else {
    if (f32) launch_append<float, 64>(a, d->B, commit, st);
    else launch_append<__nv_bfloat16, 64>(a, d->B, commit, st);
  }
  return cuda_status();
}

template <typename T, int D>
void launch_read(const Q4CacheArgs& a, int B, cudaStream_t st) {
  const int most = a.rows < a.map.cap ? a.rows : a.map.cap;
  launch(read_q4_kernel<T, D>, dim3((unsigned)ceil_div(most, kTokens), 2, B), dim3(kThreads), 0, st, a);
}

}  // namespace
}  // namespace tsd

using namespace tsd;

extern "C" tsd_status tsd_cache_write_q4(const tsd_attn_desc* d, int T, const void* knew,
                                         const void* vnew, const int32_t* new_len, void* kq,
                                         void* vq, void* kscale, void* vscale,
                                         const int32_t* page_table, int max_pages, int page_size,
                                         int num_pages, int32_t* prefix_len, int32_t* err,
                                         tsd_stream_t stream) {
  Q4CacheArgs a{};
  const tsd_status st = cache_args(d, kq, vq, kscale, vscale, page_table, max_pages, page_size,
                                   num_pages, prefix_len, err, &a);
  if (st != TSD_OK) return st;
  return append_impl(d, T, 0, knew, vnew, nullptr, new_len, a, false, stream);
}

extern "C" tsd_status tsd_commit_path_q4(const tsd_attn_desc* d, int S, const void* ktree,
                                         const void* vtree, const int32_t* accept_rows,
                                         const int32_t* accept_len, void* kq, void* vq,
                                         void* kscale, void* vscale, const int32_t* page_table,
                                         int max_pages, int page_size, int num_pages,
                                         int32_t* prefix_len, int32_t* err, tsd_stream_t stream) {
  Q4CacheArgs a{};
  const tsd_status st = cache_args(d, kq, vq, kscale, vscale, page_table, max_pages, page_size,
                                   num_pages, prefix_len, err, &a);
  if (st != TSD_OK) return st;
  return append_impl(d, d->R, S, ktree, vtree, accept_rows, accept_len, a, true, stream);
}

extern "C" tsd_status tsd_cache_read_q4(const tsd_attn_desc* d, int T, const void* kq,
                                        const void* vq, const void* kscale, const void* vscale,
                                        const int32_t* page_table, int max_pages, int page_size,
                                        int num_pages, const int32_t* prefix_len,
                                        const int32_t* first, const int32_t* count, void* kout,
                                        void* vout, int32_t* err, tsd_stream_t stream) {
  Q4CacheArgs a{};
  const tsd_status st = cache_args(d, kq, vq, kscale, vscale, page_table, max_pages, page_size,
                                   num_pages, prefix_len, err, &a);
  if (st != TSD_OK) return st;
  if (T < 1 || !ok_ptr(first) || !ok_ptr(count) || !ok_ptr(kout) || !ok_ptr(vout))
    return TSD_ERR_INVALID_ARG;
  a.dst[0] = kout;
  a.dst[1] = vout;
  a.first = first;
  a.count = count;
  a.rows = T;
  const cudaStream_t cs = (cudaStream_t)stream;
  const bool f32 = d->dtype == TSD_F32;
  if (d->dk == 128) {
    if (f32) launch_read<float, 128>(a, d->B, cs);
    else launch_read<__nv_bfloat16, 128>(a, d->B, cs);
  } else {
    if (f32) launch_read<float, 64>(a, d->B, cs);
    else launch_read<__nv_bfloat16, 64>(a, d->B, cs);
  }
  return cuda_status();
}
