// tsd_cache_write_q8, tsd_commit_path_q8: rows appended to the 8-bit cache.
//
// For each request, n rows land at positions P..P+n-1 (P the prefix length):
// rows 0..n-1 of a dense [B][T] array (a prefill), or the accepted rows of the
// scratch pad (a commit; Source: "Adapting Tree-Structured Speculative Decoding
// to DeepSeek-V4" (review), "Secret weapon" and "How it works" step 6: only the
// accepted path's KV is written).  Per block of 64 tokens that holds a new row
// and per head:
//   a  = max |x| over the block's new rows (finite elements)
//   e' = max(e, need(a)) if the block holds earlier rows, else need(a)
//   new codes = e4m3(x * 2^(127 - e')), earlier codes c -> e4m3(c * 2^(e - e'))
// Products with powers of two are exact in fp32, so each code is rounded once
// (an earlier code only where it becomes subnormal).
//
// Prefill: a CTA takes a (block, head, K or V); the new rows stay in registers
// between the maximum and the conversion, so the source is read once and the codes
// are written once; earlier rows are read only when the exponent grows.  Bounded by
// memory: 2 (or 4) bytes read and 1 written per element (4 x 8192 rows at most of 8
// heads: 31 us with the length's update, 22 us by the bytes).  Commit: a warp takes a
// (block, head, K or V); bounded by latency.
#include <cuda_bf16.h>

#include <type_traits>

#include "tsd_append.cuh"
#include "tsd_host.h"

namespace tsd {
namespace {

struct Q8WriteArgs {
  const void* src[2];      // K, V rows: [B][rows][Hkv][d]
  uint8_t* codes[2];
  uint8_t* exps[2];
  int32_t* prefix_len;
  const int32_t* count;    // commit: accepted draft rows L (L + 1 rows move); write: rows n
  const int32_t* path;     // commit: [B][S+1] source rows
  int32_t* err;
  CacheMap map;
  int rows, S, parts;      // source rows per request; path length bound; 1 (latent) or 2
};

// Threads of a CTA, and 8-element vectors of a block per thread.
template <int D> constexpr int kWriteThreads = D > 128 ? 512 : 256;
template <int D> constexpr int kWriteVecs = kQ8Block * D / 8 / kWriteThreads<D>;

// CTAs per SM to fit the registers to.  (4 x 8192 rows at most of 128 dims, in a graph:
// bf16 38 us at six, 40 at eight, 41 as the compiler has it; fp32 56 us at five, 57 at
// four, 61 at three.  Rows of 576 dims need the registers for their vectors.)
template <typename T, int D> constexpr int kWriteCtas = D > 128 ? 1 : sizeof(T) * D > 256 ? 5 : 6;

struct WriteSmem : AppendSmem {
  uint32_t warp_max[32];
};

// Eight elements as they are in memory, and as fp32.  `top` runs the largest magnitude
// in a form of the type's own (bf16: two at a time), `bits` gives it as fp32 bits.
struct RawF32 {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg((const uint4*)p);
    b = __ldg((const uint4*)p + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  __device__ __forceinline__ uint32_t top(uint32_t t) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, w[i] & 0x7fffffffu);
    return t;
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t t) { return t; }
};
struct RawBf16 {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg((const uint4*)p); }
  __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ uint32_t top(uint32_t t) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) t = __vmaxu2(t, w[i] & 0x7fff7fffu);
    return t;
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t t) { return max(t << 16, t & 0xffff0000u); }
};
template <typename Raw>
__device__ __forceinline__ uint2 to_codes(const Raw& raw, float f) {
  float x[8];
  raw.values(x);
  float2 y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = __fmul2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(f, f));
  return make_uint2(q8_pack4(y[0].x, y[0].y, y[1].x, y[1].y), q8_pack4(y[2].x, y[2].y, y[3].x, y[3].y));
}
// The largest finite magnitude, for a block that holds an infinity or a NaN.
constexpr uint32_t kInf = 0x7f800000u;
template <typename Raw>
__device__ __forceinline__ uint32_t finite_top(const Raw& raw, uint32_t t) {
  float x[8];
  raw.values(x);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = __float_as_uint(x[j]) & 0x7fffffffu;
    t = max(t, u < kInf ? u : 0u);
  }
  return t;
}

// Block `blk` (positions 64 blk ..) of head h of request b, part 0 (K) or 1 (V).
template <typename T, int D>
__device__ __forceinline__ void write_block(const Q8WriteArgs& a, int b, int h, int part, int blk,
                                            int P, int n, WriteSmem& s) {
  using Raw = typename std::conditional<sizeof(T) == 4, RawF32, RawBf16>::type;
  constexpr int kThreads = kWriteThreads<D>, kVecs = kWriteVecs<D>, VR = D / 8;
  const int tid = threadIdx.x;
  const int first = blk * kQ8Block;
  const int r0 = max(P - first, 0);                  // the block's earlier rows end here
  const int r1 = min(P + n - first, kQ8Block);       // and its new ones here
  Raw raw[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int r = (tid + i * kThreads) / VR, c = (tid + i * kThreads) % VR;
    raw[i].clear();
    if (r >= r0 && r < r1) {
      const int t = first + r - P;
      raw[i].load((const T*)a.src[part] + (((long)b * a.rows + t) * a.map.Hkv + h) * D + c * 8);
    }
  }
  uint8_t* const ep = a.exps[part] + a.map.block(b, h, first);
  const int e_old = r0 > 0 ? *ep : 0;
  uint8_t* const row0 = a.codes[part] + a.map.row(b, h, first) * D;
  auto block_max = [&](uint32_t x) {
    x = __reduce_max_sync(kFull, x);
    if ((tid & 31) == 0) s.warp_max[tid >> 5] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) x = max(x, s.warp_max[w]);
    return x;
  };
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) m = raw[i].top(m);
  m = block_max(Raw::bits(m));
  if (m >= kInf) {                                   // (the same in the whole CTA)
    m = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) m = finite_top(raw[i], m);
    __syncthreads();                                 // warp_max has been read
    m = block_max(m);
  }
  const int e = max(q8_need(__uint_as_float(m)), e_old);
  const float inv = q8_scale(254 - min(e, kQ8ExpMax));  // 2^(127 - e)
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = tid + i * kThreads, r = v / VR;
    if (r >= r0 && r < r1) {
      *(uint2*)(row0 + (long)v * 8) = to_codes(raw[i], inv);
    }
  }
  if (r0 > 0 && e != e_old) {
    const float f = pow2i(e_old - e);
    for (int v = tid; v < r0 * (D / 16); v += kThreads) {
      uint4 w = *(uint4*)(row0 + (long)v * 16);
      w.x = q8_rescale4(w.x, f);
      w.y = q8_rescale4(w.y, f);
      w.z = q8_rescale4(w.z, f);
      w.w = q8_rescale4(w.w, f);
      *(uint4*)(row0 + (long)v * 16) = w;
    }
  }
  // (every thread has read the exponent before the barrier that follows)
  __syncthreads();
  if (tid == 0 && (r0 == 0 || e != e_old)) *ep = (uint8_t)e;
}

// Prefill: grid (blocks, part x head, request).  prefix_len changes only in
// write_advance_kernel, so every CTA reads the length of before.
template <typename T, int D>
__global__ void __launch_bounds__(kWriteThreads<D>, kWriteCtas<T, D>)
write_q8_kernel(const __grid_constant__ Q8WriteArgs a) {
  __shared__ WriteSmem s;
  grid_dependency_sync();
  const int b = blockIdx.z, P = a.prefix_len[b], c = a.count[b];
  const int n = append_rows<false>(a, b, P, c, 0, s);
  if (n <= 0) return;
  const int blk = P / kQ8Block + blockIdx.x;
  if (blk * (long)kQ8Block >= (long)P + n) return;
  write_block<T, D>(a, b, blockIdx.y / a.parts, blockIdx.y % a.parts, blk, P, n, s);
}

__global__ void __launch_bounds__(128) write_advance_kernel(const __grid_constant__ Q8WriteArgs a) {
  __shared__ WriteSmem s;
  grid_dependency_sync();
  const int b = blockIdx.x, P = a.prefix_len[b], c = a.count[b];
  const int n = append_rows<false>(a, b, P, c, 0, s);
  if (threadIdx.x != 0) return;
  if (n < 0) report_error(a.err, -n, b);
  else a.prefix_len[b] = P + n;
}

// Commit: at most 17 rows, so at most two blocks per head and part.  One CTA per
// request, a warp per (block, head, part): the prefix length is read and advanced by
// the same CTA, and no launch or cluster is needed to order the two.  (A cluster of
// eight CTAs took as long on the device, 13.4 us with the advance inside a graph, and
// 1 us more to launch.)  Rows of up to 128 bf16 dims stay in registers between the
// maximum and the conversion; wider ones are read again, from L1.
constexpr int kCommitThreads = 512;

template <typename T, int D>
__device__ __forceinline__ void commit_block(const Q8WriteArgs& a, const WriteSmem& s, int b, int h,
                                             int part, int blk, int P, int n) {
  using Raw = typename std::conditional<sizeof(T) == 4, RawF32, RawBf16>::type;
  constexpr int VR = D / 8;                          // 8-element vectors of a row
  constexpr int kVecs = (17 * VR + 31) / 32;         // of the new rows, per lane
  constexpr bool kKeep = sizeof(T) == 2 && D <= 128;
  const int lane = threadIdx.x & 31;
  const int first = blk * kQ8Block;
  const int r0 = max(P - first, 0), r1 = min(P + n - first, kQ8Block);
  const int work = (r1 - r0) * VR;
  uint8_t* const ep = a.exps[part] + a.map.block(b, h, first);
  uint8_t* const row0 = a.codes[part] + a.map.row(b, h, first) * D;
  const int e_old = r0 > 0 ? *ep : 0;
  auto source = [&](int v) {
    const int t = first + r0 + v / VR - P;
    return (const T*)a.src[part] + (((long)b * a.rows + s.path[t]) * a.map.Hkv + h) * D + v % VR * 8;
  };
  Raw raw[kKeep ? kVecs : 1];
  uint32_t m = 0;
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      raw[i].clear();
      if (lane + 32 * i < work) raw[i].load(source(lane + 32 * i));
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) m = raw[i].top(m);
  } else {
#pragma unroll 4
    for (int v = lane; v < work; v += 32) {
      raw[0].load(source(v));
      m = raw[0].top(m);
    }
  }
  m = __reduce_max_sync(kFull, Raw::bits(m));
  if (m >= kInf) {
    m = 0;
    for (int v = lane; v < work; v += 32) {
      Raw again;
      again.load(source(v));
      m = finite_top(again, m);
    }
    m = __reduce_max_sync(kFull, m);
  }
  const int e = max(q8_need(__uint_as_float(m)), e_old);
  const float inv = q8_scale(254 - min(e, kQ8ExpMax));  // 2^(127 - e)
  auto put = [&](const Raw& w, int v) {
    *(uint2*)(row0 + ((long)r0 * VR + v) * 8) = to_codes(w, inv);
  };
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (lane + 32 * i < work) put(raw[i], lane + 32 * i);
  } else {
#pragma unroll 4
    for (int v = lane; v < work; v += 32) {
      raw[0].load(source(v));
      put(raw[0], v);
    }
  }
  if (r0 > 0 && e != e_old) {
    const float f = pow2i(e_old - e);
#pragma unroll 4
    for (int v = lane; v < r0 * (D / 16); v += 32) {
      uint4 w = *(uint4*)(row0 + (long)v * 16);
      w.x = q8_rescale4(w.x, f);
      w.y = q8_rescale4(w.y, f);
      w.z = q8_rescale4(w.z, f);
      w.w = q8_rescale4(w.w, f);
      *(uint4*)(row0 + (long)v * 16) = w;
    }
  }
  __syncwarp();                                      // (every lane has read the exponent)
  if (lane == 0 && (r0 == 0 || e != e_old)) *ep = (uint8_t)e;
}

template <typename T, int D>
__global__ void __launch_bounds__(kCommitThreads)
commit_q8_kernel(const __grid_constant__ Q8WriteArgs a) {
  __shared__ WriteSmem s;
  grid_dependency_sync();
  const int b = blockIdx.x, P = a.prefix_len[b], c = a.count[b];
  const int r = threadIdx.x <= a.S ? a.path[(long)b * (a.S + 1) + threadIdx.x] : 0;
  const int n = append_rows<true>(a, b, P, c, r, s);  // (its barrier: the whole CTA has read P)
  if (threadIdx.x == 0) {
    if (n < 0) report_error(a.err, -n, b);
    else a.prefix_len[b] = P + n;
  }
  if (n <= 0) return;
  const int blk0 = P / kQ8Block, nb = (P + n - 1) / kQ8Block - blk0 + 1;
  for (int t = threadIdx.x >> 5; t < nb * a.map.Hkv * a.parts; t += kCommitThreads / 32) {
    const int hp = t / nb;
    commit_block<T, D>(a, s, b, hp / a.parts, hp % a.parts, blk0 + t % nb, P, n);
  }
}

template <typename T, int D>
void launch_write(const Q8WriteArgs& a, int B, int nblk, bool commit, cudaStream_t st) {
  if (commit) {
    launch(commit_q8_kernel<T, D>, dim3(B), dim3(kCommitThreads), 0, st, a);
    return;
  }
  launch(write_q8_kernel<T, D>, dim3(nblk, a.map.Hkv * a.parts, B), dim3(kWriteThreads<D>), 0, st, a);
  launch(write_advance_kernel, dim3(B), dim3(128), 0, st, a);
}

tsd_status write_impl(const tsd_attn_desc* d, int rows, int S, const void* k, const void* v,
                      const int32_t* path, const int32_t* count, void* kq, void* vq, void* kexp,
                      void* vexp, const int32_t* page_table, int max_pages, int page_size,
                      int num_pages, int32_t* prefix_len, int32_t* err, bool commit,
                      tsd_stream_t stream) {
  if (!q8_desc_ok(d) || (((uintptr_t)err) & 3u) != 0) return TSD_ERR_INVALID_ARG;
  const bool alias = d->v_aliases_k != 0;
  if (rows < 1 || (commit && (S < 1 || S > 16 || !ok_ptr(path)))) return TSD_ERR_INVALID_ARG;
  if (!ok_ptr(k) || !ok_ptr(count) || !ok_ptr(kq) || !ok_ptr(kexp) || !ok_ptr(prefix_len))
    return TSD_ERR_INVALID_ARG;
  if (!alias && (!ok_ptr(v) || !ok_ptr(vq) || !ok_ptr(vexp))) return TSD_ERR_INVALID_ARG;
  if (!paging_ok(d, page_table, max_pages, page_size, num_pages)) return TSD_ERR_INVALID_ARG;
  Q8WriteArgs a{};
  a.src[0] = k;
  a.src[1] = alias ? nullptr : v;
  a.codes[0] = (uint8_t*)kq;
  a.codes[1] = alias ? nullptr : (uint8_t*)vq;
  a.exps[0] = (uint8_t*)kexp;
  a.exps[1] = alias ? nullptr : (uint8_t*)vexp;
  a.prefix_len = prefix_len;
  a.count = count;
  a.path = path;
  a.err = err;
  a.map = cache_map(d, page_table, max_pages, page_size, num_pages);
  a.rows = rows;
  a.S = S;
  a.parts = alias ? 1 : 2;
  // n rows from any position of a block span at most this many blocks, and no
  // more than the cache has
  const long span = ((long)(rows < d->cap ? rows : d->cap) + kQ8Block - 2) / kQ8Block + 1;
  const cudaStream_t st = (cudaStream_t)stream;
  const bool f32 = d->dtype == TSD_F32;
  if ((long)d->Hkv * a.parts > 65535) return TSD_ERR_INVALID_ARG;
  if (d->dk == 576) {
    if (f32) launch_write<float, 576>(a, d->B, (int)span, commit, st);
    else launch_write<__nv_bfloat16, 576>(a, d->B, (int)span, commit, st);
  } else if (d->dk == 128) {
    if (f32) launch_write<float, 128>(a, d->B, (int)span, commit, st);
    else launch_write<__nv_bfloat16, 128>(a, d->B, (int)span, commit, st);
  } else {
    if (f32) launch_write<float, 64>(a, d->B, (int)span, commit, st);
    else launch_write<__nv_bfloat16, 64>(a, d->B, (int)span, commit, st);
  }
  return cuda_status();
}

}  // namespace
}  // namespace tsd

using namespace tsd;

extern "C" tsd_status tsd_cache_write_q8(const tsd_attn_desc* d, int T, const void* knew,
                                         const void* vnew, const int32_t* new_len, void* kq,
                                         void* vq, void* kexp, void* vexp,
                                         const int32_t* page_table, int max_pages, int page_size,
                                         int num_pages, int32_t* prefix_len, int32_t* err,
                                         tsd_stream_t stream) {
  return write_impl(d, T, 0, knew, vnew, nullptr, new_len, kq, vq, kexp, vexp, page_table,
                    max_pages, page_size, num_pages, prefix_len, err, false, stream);
}

extern "C" tsd_status tsd_commit_path_q8(const tsd_attn_desc* d, int S, const void* ktree,
                                         const void* vtree, const int32_t* accept_rows,
                                         const int32_t* accept_len, void* kq, void* vq,
                                         void* kexp, void* vexp, const int32_t* page_table,
                                         int max_pages, int page_size, int num_pages,
                                         int32_t* prefix_len, int32_t* err,
                                         tsd_stream_t stream) {
  if (d == nullptr) return TSD_ERR_INVALID_ARG;
  return write_impl(d, d->R, S, ktree, vtree, accept_rows, accept_len, kq, vq, kexp, vexp,
                    page_table, max_pages, page_size, num_pages, prefix_len, err, true, stream);
}
