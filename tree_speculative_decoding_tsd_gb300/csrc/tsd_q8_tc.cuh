// Device pieces of the two tcgen05 paths over the 8-bit cache: 8-bit products,
// operand layouts, the exact splits and scalings of bf16 rows, streaming loads;
// and the host's tensor map of the K codes.
#pragma once

#include <cuda.h>

#include "tsd_q8_attn.cuh"
#include "tsd_tcgen05.cuh"

namespace tsd {
namespace {

constexpr int kKeys = 128;                      // keys per tile
constexpr uint32_t kHalf = kKeys * 128;         // [128 rows][64 fp16]: 16 KB
constexpr uint32_t kTile = 2 * kHalf;           // a widened V tile
constexpr int kRing = 4;                        // K tiles in shared memory
constexpr float kOverflow = 8.0f;               // log2 headroom of the lazy maximum
constexpr int kHeadroom = 7;                    // P's offset: 2^8 * 2^7 < 65504
constexpr int kMaxTiles = 256;                  // prefix tiles of a split
constexpr int kPrefetch = 4;                    // tiles that V's L2 prefetch runs ahead

// The request of grid index z, and its prefix length within the cache.  By length
// (batches of up to 64): the one of rank z, which warp 0 finds and leaves in `slot`.
// For the whole CTA, before its threads part.
__device__ __forceinline__ int request_at(const Q8AttnArgs& a, int z, int& P, volatile int* slot) {
  int b = z;
  if (a.by_length) {
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      const int p0 = lane < a.B ? min(max(a.plen[lane], 0), a.map.cap) : -1;
      const int p1 = lane + 32 < a.B ? min(max(a.plen[lane + 32], 0), a.map.cap) : -1;
      int r0 = 0, r1 = 0;              // requests before this lane's two: longer, or as long and earlier
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const int x = __shfl_sync(kFull, p0, j);
        r0 += x > p0 || (x == p0 && j < lane);
        r1 += x >= p1;
      }
      if (a.B > 32) {
#pragma unroll 8
        for (int j = 0; j < 32; ++j) {
          const int x = __shfl_sync(kFull, p1, j);
          r0 += x > p0;
          r1 += x > p1 || (x == p1 && j < lane);
        }
      }
      if (p0 >= 0 && r0 == z) {
        slot[0] = lane;
        slot[1] = p0;
      }
      if (p1 >= 0 && r1 == z) {
        slot[0] = lane + 32;
        slot[1] = p1;
      }
    }
    __syncthreads();
    // (a reduction's result is a uniform value, which spares registers)
    b = __reduce_max_sync(kFull, (int)slot[0]);
    P = __reduce_max_sync(kFull, (int)slot[1]);
  } else {
    P = min(max(a.plen[b], 0), a.map.cap);
  }
  return b;
}

// The kernels' pipeline waits.  kPoll: with the budget of tsd_set_wait_budget, in an
// instantiation of its own, so that the usual one has neither the budget nor the polling
// loop in its code (65-row trees over 8 x 32k keys: 321 us so, 324 us with the limit and
// the sleep as kernel arguments).
template <bool kPoll>
__device__ __forceinline__ bool phase_timed(uint32_t bar, uint32_t parity, long long budget) {
  if constexpr (kPoll) return mbar_poll(bar, parity, budget);
  else return mbar_wait(bar, parity);
}
// The same for a phase that is usually complete already: one look before the timed
// wait.
template <bool kPoll>
__device__ __forceinline__ bool phase_ready(uint32_t bar, uint32_t parity, long long budget) {
  if constexpr (kPoll) return mbar_poll(bar, parity, budget);
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok || mbar_wait(bar, parity);
}
// Whether a phase is complete, looked at early: an access to shared memory takes about
// 300 cycles while widened tiles are stored and products read theirs, which a warp
// spends on other work.
__device__ __forceinline__ bool complete(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
// One lane of a converged warp.  A warp that issues products runs its loop on all
// lanes, so that descriptors and addresses are uniform values, and issues on this
// lane.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// D (+)= A.B, 8-bit operands (e4m3), K = 32 per instruction.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}

// Byte offset of 16-byte unit u of row r in a K-major tile of D-byte rows
// (128-byte swizzle for D = 128, 64-byte swizzle for D = 64), and the matrix
// descriptor of such a tile.
template <int D>
__device__ __forceinline__ uint32_t unit_offset(int r, int u) {
  return D == 128 ? r * 128 + ((u ^ (r & 7)) << 4) : r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
}
template <int D>
__device__ __forceinline__ uint64_t row_desc(uint32_t addr) {
  if (D == 128) return smem_desc(addr, 16, 1024);
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(512 >> 4) << 32) |
         (1ull << 46) | (4ull << 61);
}

// Sixteen bf16 times f, which puts their row's largest into [128, 256), as e4m3 numbers
// hi and lo.  hi + lo = x f down to e4m3's smallest step: off by at most 2^-10, 2^-17 of
// the largest, for elements below 2^-9 of it (tsd_q8_tc.cu).
__device__ __forceinline__ void split16(const uint4 (&w)[2], float f, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4& s = w[i >> 1];
    const uint32_t a = (i & 1) ? s.z : s.x, b = (i & 1) ? s.w : s.y;
    const float x[4] = {__uint_as_float(a << 16) * f, __uint_as_float(a & 0xffff0000u) * f,
                        __uint_as_float(b << 16) * f, __uint_as_float(b & 0xffff0000u) * f};
    float y[4];
    h[i] = q8_pack4(x[0], x[1], x[2], x[3]);
    q8_unpack4(h[i], y);
    l[i] = q8_pack4(x[0] - y[0], x[1] - y[1], x[2] - y[2], x[3] - y[3]);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Running largest magnitude of bf16 pairs, the even and the odd elements apart.
__device__ __forceinline__ uint32_t top_pairs(uint32_t top, const uint4& w) {
  top = __vmaxu2(top, w.x & 0x7fff7fffu);
  top = __vmaxu2(top, w.y & 0x7fff7fffu);
  top = __vmaxu2(top, w.z & 0x7fff7fffu);
  return __vmaxu2(top, w.w & 0x7fff7fffu);
}
// The larger of the two, as fp32 bits (at least 0x7f800000: not finite).
__device__ __forceinline__ uint32_t top_of(uint32_t pairs) {
  return max(pairs << 16, pairs & 0xffff0000u);
}
// A widening thread's share of a V tile (128 keys x 16 W codes, W = 4 or 8): chunks
// of 16 codes, `T` threads.  Eight lanes that store together take four chunks of an
// even and of an odd row (W = 8: chunks 0-3 or 4-7; W = 4: two rows): eight different
// 16-byte columns of a swizzled row pair, so the stores do not conflict.  A thread's
// chunks are T / W rows apart, which keeps its addresses at fixed distances.
template <int W, int T>
struct WideShare {
  static constexpr int kCount = (kKeys * W + T - 1) / T;
  static constexpr int kStep = T / W;              // rows between a thread's chunks
  static_assert(T % (4 * W) == 0, "whole swizzle halves");
  int row, col;                                    // first chunk
  uint32_t dst0, dst1;                             // its two 16-byte units in a stage
  __device__ __forceinline__ explicit WideShare(int wt) {
    row = W == 8 ? 2 * (wt >> 4) + ((wt >> 2) & 1) : wt >> 2;
    col = W == 8 ? (wt & 3) + 4 * ((wt >> 3) & 1) : wt & 3;
    const uint32_t base = (uint32_t)((col >> 2) * kHalf + row * 128);
    const int u = 2 * (col & 3);
    dst0 = base + (uint32_t)((u ^ (row & 7)) << 4);
    dst1 = base + (uint32_t)(((u + 1) ^ (row & 7)) << 4);
  }
  // chunks of the rows below nvalid from `src`, the tile's first code of this share
  // (rows of `pitch` codes), zeros behind them
  template <int kPitch>
  __device__ __forceinline__ void load(uint4 (&r)[kCount], const uint8_t* src, int nvalid) const;
  __device__ __forceinline__ void widen(const uint4 (&r)[kCount], uint8_t* stage) const;
};

// Eight bf16 times f as fp16.
__device__ __forceinline__ uint4 scale8(const uint4& w, float f) {
  uint4 r;
  r.x = pack_half2(__uint_as_float(w.x << 16) * f, __uint_as_float(w.x & 0xffff0000u) * f);
  r.y = pack_half2(__uint_as_float(w.y << 16) * f, __uint_as_float(w.y & 0xffff0000u) * f);
  r.z = pack_half2(__uint_as_float(w.z << 16) * f, __uint_as_float(w.z & 0xffff0000u) * f);
  r.w = pack_half2(__uint_as_float(w.w << 16) * f, __uint_as_float(w.w & 0xffff0000u) * f);
  return r;
}
// fp32 exponent field of a row's largest magnitude, at least 15 so that both
// the scale and its inverse are normal numbers.
__device__ __forceinline__ int row_exponent(uint32_t top) { return max((int)(top >> 23), 15); }

template <int W, int T>
template <int kPitch>
__device__ __forceinline__ void WideShare<W, T>::load(uint4 (&r)[kCount], const uint8_t* src,
                                                      int nvalid) const {
  const uint8_t* const p = src + (long)row * kPitch + col * 16;
  if (nvalid >= kKeys) {
#pragma unroll
    for (int i = 0; i < kCount; ++i)
      if ((i + 1) * kStep <= kKeys || row + i * kStep < kKeys) r[i] = ld_stream(p + i * kStep * kPitch);
    return;
  }
#pragma unroll
  for (int i = 0; i < kCount; ++i) {
    r[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row + i * kStep < nvalid) r[i] = ld_stream(p + i * kStep * kPitch);
  }
}
template <int W, int T>
__device__ __forceinline__ void WideShare<W, T>::widen(const uint4 (&r)[kCount], uint8_t* stage) const {
#pragma unroll
  for (int i = 0; i < kCount; ++i) {
    if ((i + 1) * kStep > kKeys && row + i * kStep >= kKeys) break;    // (a short last round)
    uint32_t h[8];
    q8_half4(r[i].x, h[0], h[1]);
    q8_half4(r[i].y, h[2], h[3]);
    q8_half4(r[i].z, h[4], h[5]);
    q8_half4(r[i].w, h[6], h[7]);
    // (kStep is a multiple of 4: the swizzle of row + i kStep differs in bit 2 at most)
    const uint32_t flip = (uint32_t)((i * kStep) & 4) << 4;
    uint8_t* const d = stage + i * kStep * 128;
    *(uint4*)(d + (dst0 ^ flip)) = make_uint4(h[0], h[1], h[2], h[3]);
    *(uint4*)(d + (dst1 ^ flip)) = make_uint4(h[4], h[5], h[6], h[7]);
  }
}

// Scratch rows of (request b, head hk) in shared memory for the scan, [65][D] bf16: K
// where the first widened tile will be, V at the second one (`apart` bytes on).  N
// threads, eight per row; a thread scans what it copied itself.
template <int D>
constexpr uint32_t kTreeBytes = 65u * D * 2;

template <int D, int N>
__device__ __forceinline__ void tree_fetch(const Q8AttnArgs& a, int b, int hk, int wt, uint32_t dst,
                                           uint32_t apart) {
#pragma unroll 1
  for (int x = wt; x < a.R * 8; x += N) {
    const int j = x >> 3, c = x & 7;
    const long row = (((long)b * a.R + j) * a.map.Hkv + hk) * (D / 8) + c;
#pragma unroll
    for (int v = 0; v < D / 64; ++v) {
      const uint32_t to = dst + (uint32_t)(j * (D / 8) + c + 8 * v) * 16u;
      cp_async16(to, (const uint4*)a.kt + row + 8 * v, true);
      cp_async16(to + apart, (const uint4*)a.vt + row + 8 * v, true);
    }
  }
  asm volatile("cp.async.commit_group;\n" ::: "memory");
}

// Which rows some row sees, their factors, and (returned) this thread's largest
// exponent of a value row.
template <int D, int N>
__device__ __forceinline__ int tree_scan(const Q8AttnArgs& a, int b, int wt, const uint8_t* rows,
                                         uint32_t apart, float* kt_in, float* vt_in, float* kt_out, int* vt_u) {
  const int lane = threadIdx.x & 31;
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int r = lane + 32 * i;
    const uint64_t m = r > 0 && r < a.R ? a.mask[(long)b * a.R + r] : 0ull;
    lo |= (uint32_t)m;
    hi |= (uint32_t)(m >> 32);
  }
  asm volatile("cp.async.wait_group 0;\n" ::: "memory");
  const uint64_t seen = ((uint64_t)__reduce_or_sync(kFull, hi) << 32) | __reduce_or_sync(kFull, lo);
  int best = -1000;
#pragma unroll 1
  for (int x0 = wt - lane; x0 < a.R * 8; x0 += N) {  // (whole warps)
    const int j = (x0 + lane) >> 3, c = lane & 7;
    uint32_t kt = 0, vt = 0;
    if (j < a.R) {
      const uint4* p = (const uint4*)rows + j * (D / 8) + c;
#pragma unroll
      for (int v = 0; v < D / 64; ++v) {
        kt = top_pairs(kt, p[8 * v]);
        vt = top_pairs(vt, p[8 * v + apart / 16]);
      }
    }
    kt = top_of(kt);
    vt = top_of(vt);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      kt = max(kt, __shfl_xor_sync(kFull, kt, o));
      vt = max(vt, __shfl_xor_sync(kFull, vt, o));
    }
    if (j >= a.R) continue;
    const bool live = j == 0 || ((seen >> (j - 1)) & 1ull);
    const bool bad = kt >= 0x7f800000u || vt >= 0x7f800000u;
    const int ek = row_exponent(kt), ev = row_exponent(vt);
    if (c == 0) {
      // K: 2^(7 - (e - 127)) and its inverse; V: 2^(8 - (e - 127))
      kt_in[j] = live && !bad ? q8_scale(261 - ek) : 0.f;
      vt_in[j] = live && !bad ? q8_scale(262 - ev) : 0.f;
      kt_out[j] = bad ? __int_as_float(0x7fffffff) : q8_scale(ek - 7);
      vt_u[j] = live && !bad ? ev - 135 : -900;
    }
    if (live && !bad) best = max(best, ev - 135);
  }
  for (int j = a.R + wt; j < kKeys; j += N) {        // rows that do not exist (N > 128)
    kt_in[j] = vt_in[j] = 0.f;
    kt_out[j] = 1.f;
    vt_u[j] = -900;
  }
  return best;
}

// The packed rows of a row group as hi + lo (n_rows of them, zeros behind the
// last one) with their score factors: D / 16 lanes of the n threads per row.
template <int D>
__device__ __forceinline__ void stage_q(const Q8AttnArgs& a, int b, int hk, int row_base,
                                        int rows_here, int n_rows, int tid, int n, uint8_t* hi_tile,
                                        uint8_t* lo_tile, float* c2v) {
  constexpr int QL = D / 16;
#pragma unroll 1
  for (int x = tid; x < n_rows * QL; x += n) {       // (whole warps: n_rows is a multiple of 16)
    const int r = x / QL, c = x % QL;
    uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    uint32_t top = 0;
    if (r < rows_here) {
      const int p = row_base + r;
      const int tr = p / a.g, qh = hk * a.g + p % a.g;
      const uint4* qp =
          (const uint4*)((const __nv_bfloat16*)a.q + (((long)b * a.R + tr) * a.Hq + qh) * D) + 2 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = __ldg(qp + i);
        top = top_pairs(top, w[i]);
      }
    }
    top = top_of(top);
#pragma unroll
    for (int o = QL / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    const bool bad = top >= 0x7f800000u;
    const int e = row_exponent(top);
    uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
    if (!bad) split16(w, q8_scale(261 - e), hi, lo);
    *(uint4*)(hi_tile + unit_offset<D>(r, c)) = hi;
    *(uint4*)(lo_tile + unit_offset<D>(r, c)) = lo;
    if (c == 0) c2v[r] = bad ? __int_as_float(0x7fffffff) : a.qscale * q8_scale(e - 7);
  }
}

// The scratch rows' keys as hi + lo, and their values as fp16; rows that nobody
// sees are zeros.
template <int D>
__device__ __forceinline__ void tree_keys(const Q8AttnArgs& a, int b, int hk, int wt, int n,
                                          const float* kt_in, uint8_t* hi_tile, uint8_t* lo_tile) {
#pragma unroll 1
  for (int x = wt; x < kKeys * (D / 16); x += n) {
    const int row = x / (D / 16), u = x % (D / 16);
    uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
    const float f = kt_in[row];
    if (f != 0.f) {
      const uint4* p = (const uint4*)((const __nv_bfloat16*)a.kt +
                                      (((long)b * a.R + row) * a.map.Hkv + hk) * D) + 2 * u;
      const uint4 w[2] = {__ldg(p), __ldg(p + 1)};
      split16(w, f, hi, lo);
    }
    *(uint4*)(hi_tile + unit_offset<D>(row, u)) = hi;
    *(uint4*)(lo_tile + unit_offset<D>(row, u)) = lo;
  }
}
template <int D>
__device__ __forceinline__ void tree_values(const Q8AttnArgs& a, int b, int hk, int wt, int n,
                                            const float* vt_in, uint8_t* stage) {
#pragma unroll 2
  for (int x = wt; x < kKeys * (D / 8); x += n) {
    const int row = x / (D / 8), u = x % (D / 8);
    const float f = vt_in[row];
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (f != 0.f)
      v = scale8(__ldg((const uint4*)((const __nv_bfloat16*)a.vt +
                                      (((long)b * a.R + row) * a.map.Hkv + hk) * D) + u), f);
    *(uint4*)(stage + (u >> 3) * kHalf + row * 128 + (((u & 7) ^ (row & 7)) << 4)) = v;
  }
}

// n / d, exact and below 2^31: a function of its own, because an inlined 64-bit division
// is 100 instructions.
__device__ __noinline__ int quotient(long long n, int d) { return (int)(n / d); }

// The K tile of positions pos.. by TMA (cache row `row`, for a paged cache).  A
// tile behind the cache's or page's last row reads zeros there; rows behind the
// prefix are masked later, whatever they hold; the rows of a missing page are
// those of page 0.
__device__ __forceinline__ void load_keys(const Q8AttnArgs& a, const CUtensorMap& kmap, int b,
                                          int hk, int pos, long long row, uint32_t dst,
                                          uint32_t bytes, uint32_t full) {
  int y = pos, z = b * a.map.Hkv + hk;
  if (a.map.page_size) {
    y = (int)((uint32_t)pos % (uint32_t)a.map.page_size);
    z = row < 0 ? 0 : quotient(row - y, a.map.page_size);
  }
  mbar_expect_tx(full, bytes);
  tma_3d(dst, &kmap, 0, y, z, full);
}

// K codes of D dims as (dims, rows of a head, heads), in boxes of 128 rows and 128
// or 64 dims (swizzled to their width): rows are those of a request's head, or of a
// page's.
bool encode_keys(CUtensorMap* m, const Q8AttnArgs& a, int D, int width) {
  const long rows = a.map.page_size > 0 ? a.map.page_size : a.map.cap;
  const long heads = (a.map.page_size > 0 ? (long)a.map.num_pages : (long)a.B) * a.map.Hkv;
  if (heads > 0x7fffffffl) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)heads};
  const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)rows * D};
  const cuuint32_t box[3] = {(cuuint32_t)width, (cuuint32_t)kKeys, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(a.kc), dims, strides,
                     box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

}  // namespace tsd
