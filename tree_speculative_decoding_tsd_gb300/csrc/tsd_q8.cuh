// The 8-bit KV cache: its number format, its addressing, and the helpers its
// kernels share.
//
// A cache row holds e4m3 codes; the 64 tokens of a block share one exponent
// byte per head (K and V apart): value = code * 2^(e - 127).  A power of two
// keeps every value exact in the arithmetic that reads it, and makes a later
// change of a block's exponent exact down to e4m3's smallest step.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "tsd_common.cuh"

namespace tsd {

constexpr int kQ8Block = TSD_Q8_BLOCK;
// Exponent bytes that a write gives.  e4m3's largest value is 448 = 1.75 * 2^8,
// so e = 246 (2^119) reaches 2.98e38 and e = 10 (2^-117) keeps the smallest
// code step, 2^-9, a normal fp32 number.
constexpr int kQ8ExpMin = 10, kQ8ExpMax = 246;

// Rows of a cache, contiguous [B][Hkv][cap] or paged [num_pages][Hkv][page_size]
// (any element size), and the exponent bytes of an 8-bit one: a contiguous head
// has ceil(cap / 64) of them, a page page_size / 64 per head.
struct CacheMap {
  const int32_t* page_table;
  int max_pages, page_size, num_pages;   // page_size 0: contiguous
  int Hkv, cap;

  // Row of position pos of (request b, head h); -1 for a page outside the pool.
  __device__ __forceinline__ long row(int b, int h, int pos) const {
    if (page_size == 0) return ((long)b * Hkv + h) * cap + pos;
    const int pg = page_table[(long)b * max_pages + pos / page_size];
    if (pg < 0 || pg >= num_pages) return -1;
    return ((long)pg * Hkv + h) * page_size + pos % page_size;
  }
  // Index of the exponent byte of position pos, whose row is `row` (not -1).
  __device__ __forceinline__ long block_at(int b, int h, int pos, long row) const {
    if (page_size) return row / kQ8Block;              // (pages are whole blocks)
    return ((long)b * Hkv + h) * ((cap + kQ8Block - 1) / kQ8Block) + pos / kQ8Block;
  }
  // Index of the exponent byte of position pos; -1 for a page outside the pool.
  __device__ __forceinline__ long block(int b, int h, int pos) const {
    if (page_size == 0)
      return ((long)b * Hkv + h) * ((cap + kQ8Block - 1) / kQ8Block) + pos / kQ8Block;
    const int pg = page_table[(long)b * max_pages + pos / page_size];
    if (pg < 0 || pg >= num_pages) return -1;
    return ((long)pg * Hkv + h) * (page_size / kQ8Block) + (pos % page_size) / kQ8Block;
  }
};

// 2^(e - 127) of an exponent byte (0 gives 0, 255 infinity).
__device__ __forceinline__ float q8_scale(int e) { return __uint_as_float((uint32_t)e << 23); }

// 2^d, and 0 below 2^-126 (d <= 127).
__device__ __forceinline__ float pow2i(int d) {
  return d < -126 ? 0.f : __uint_as_float((uint32_t)(d + 127) << 23);
}

// Exponent byte that holds magnitudes up to amax (finite, >= 0): the smallest e
// with amax <= 448 * 2^(e - 127), within [kQ8ExpMin, kQ8ExpMax].  With amax =
// f * 2^x, f in [1, 2): 448 = 1.75 * 2^8, so e - 127 = x - 8, one more if f > 1.75.
__device__ __forceinline__ int q8_need(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int x = (int)(u >> 23) - 127;
  const int e = x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0) + 127;
  return min(max(e, kQ8ExpMin), kQ8ExpMax);
}

// Two values as two e4m3 codes (round to nearest even, magnitudes past 448
// saturate, NaN stays NaN); a in the low byte.
__device__ __forceinline__ uint32_t q8_pack2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d) {
  return q8_pack2(a, b) | (q8_pack2(c, d) << 16);
}
// Four codes as two pairs of fp16, exactly.
__device__ __forceinline__ void q8_half4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Four codes as fp32.
__device__ __forceinline__ void q8_unpack4(uint32_t w, float (&v)[4]) {
  uint32_t a, b;
  q8_half4(w, a, b);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  v[0] = x.x; v[1] = x.y; v[2] = y.x; v[3] = y.y;
}
// Four codes held at one exponent as codes at another: times f = 2^(old - new).
__device__ __forceinline__ uint32_t q8_rescale4(uint32_t w, float f) {
  float v[4];
  q8_unpack4(w, v);
  return q8_pack4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
}

// Eight consecutive elements as fp32 (16-byte aligned for bf16, 32 for fp32).
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg((const float4*)p), b = __ldg((const float4*)p + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = __ldg((const uint4*)p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Host: the descriptor of an 8-bit (or evictable) cache: as tsd_tree_verify_attn
// takes it, apart from the scale where `scaled` is false.
inline bool q8_desc_ok(const tsd_attn_desc* d, bool scaled = false) {
  if (d == nullptr) return false;
  if (d->B < 1 || d->B > 65535 || d->R < 1 || d->R > 65 || d->Hq < 1 || d->Hkv < 1 ||
      d->Hq % d->Hkv != 0 || d->cap < 1)
    return false;
  if (d->dtype != TSD_F32 && d->dtype != TSD_BF16) return false;
  if (scaled && (!(d->scale > 0.f) || !(d->scale < 1e30f))) return false;
  if (d->v_aliases_k) return d->dk == 576 && d->dv == 512;
  return d->dk == d->dv && (d->dk == 64 || d->dk == 128);
}

// Host: page arguments as tsd_accept_commit takes them (page_size 0, the rest
// unused, for a contiguous cache).
inline bool paging_ok(const tsd_attn_desc* d, const void* page_table, int max_pages, int page_size,
                      int num_pages) {
  if (page_size == 0) return true;
  return page_size > 0 && page_size % 128 == 0 && max_pages >= 1 && num_pages >= 1 &&
         (long)max_pages * page_size == d->cap && page_table != nullptr &&
         (((uintptr_t)page_table) & 15u) == 0;
}

inline CacheMap cache_map(const tsd_attn_desc* d, const int32_t* page_table, int max_pages,
                          int page_size, int num_pages) {
  CacheMap m{};
  m.Hkv = d->Hkv;
  m.cap = d->cap;
  if (page_size > 0) {
    m.page_table = page_table;
    m.max_pages = max_pages;
    m.page_size = page_size;
    m.num_pages = num_pages;
  }
  return m;
}

}  // namespace tsd
