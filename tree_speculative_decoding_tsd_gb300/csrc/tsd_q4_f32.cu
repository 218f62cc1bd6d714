// Path of tsd_tree_verify_attn_q4 for fp32 heads of 64 or 128 dims; packed rows are R tree rows x
// g query heads of a KV head.
//
//   S[row][key]  = Q . K_tile^T     16 rows x 8 keys x 8 dims per instruction, tf32
//   O[row][dim] += P . V_tile       16 rows x 8 dims x 8 keys
//
// Numbers.  A cached value (c - 8) s has at most 11 significant bits (3 of the code, 8 of the
// scale), so it is a tf32 number as it stands, whatever its exponent.  Q and P go as two tf32
// terms: Q off by 2^-22 of an element at most, P by 2^-23 of a weight, sums in fp32.  (fp16 or
// bf16 terms would lose the bits of small weights, and scales far below a tile's largest.)
// Scratch rows, fp32 numbers of 24 bits, go as two terms, too: off by 2^-22.  Rows of Q below
// 2^-60 are held times 2^64, so that the low terms are not subnormal.
//
// A CTA has four warps and 64, 32 or 16 rows; with fewer rows the warps share a tile's keys and
// are joined at the end.  Codes are requested a tile ahead and widened once, for all rows, into
// shared memory (16-byte units permuted by key: no reader and no writer meets a bank twice).
// The keys' order within a product is that of its accumulators, so that P stays in registers.
//
// The tensor core cuts its sums: over thousands of keys an accumulator loses a few 2^-20, always
// towards zero.  So 32 dims of a score, and 64 keys of an output, are summed there and then added
// in fp32 (6% of the time; the outputs' error is then that of plain fp32 code, before four times).
//
// What bounds it: with 64 rows the products (two of 1024 multiply-adds for each; 60% of the tensor
// pipe) and their waits, at 255 registers and two CTAs per SM.  65 rows of 64 heads over 8000
// keys: 255 us, 67 TFLOP/s; 4 x 33 rows of 32 heads over 1k to 4k keys: 181 us.  On the CUDA
// cores, with a thread's 8 x 4 scores from shared memory, whose loads bound that, 484 and 267 us;
// a warp per eight rows with keys in registers, as over the 8-bit cache, 1531 and 558.
#include <type_traits>

#include "tsd_common.cuh"
#include "tsd_host.h"
#include "tsd_q4.cuh"
#include "tsd_q4_attn.cuh"
#include "tsd_tcgen05.cuh"

namespace tsd {
namespace {

constexpr int kF32Threads = 128, kF32Keys = 64;

template <int D, int WR>
struct F32Layout {
  static constexpr int kRows = 16 * WR, KW = 4 / WR;          // rows of the CTA; warps that share a row
  static constexpr int q = kRows * D, kv = kF32Keys * D;      // floats
  static constexpr int joint = KW > 1 ? 4 * 16 * D + 4 * 32 : 0;
  static constexpr uint32_t total = 4 * (q + 2 * kv);
  static_assert(joint <= 2 * kv, "the joint lies where K and V were");
};

// 32 codes of a group times its scale: (c - 8) s, exact.
__device__ __forceinline__ void widen8(uint32_t w, float s, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (2^23 + c as a float, less 2^23 + 8)
    x[2 * i] = (__uint_as_float(0x4b000000u | (w >> 4 * i & 15u)) - 8388616.f) * s;
    x[2 * i + 1] = (__uint_as_float(0x4b000000u | (w >> (16 + 4 * i) & 15u)) - 8388616.f) * s;
  }
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x as two tf32 terms.  The high one: x cut (which does not overflow) or rounded; the low one
// rounded: the product drops its last 13 bits.
__device__ __forceinline__ void cut_terms(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) + 0x1000u;
}
__device__ __forceinline__ void near_terms(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) + 0x1000u;
}
// Places of a key's 16-byte units in shared memory.  K is read by lanes (key g, unit t), V by
// lanes (unit g, key 2 t): eight lanes that are served together differ in the low bits below.
__device__ __forceinline__ int k_turn(int key) { return (key & 1) << 2 | (key & 2) | (key >> 2 & 1); }
__device__ __forceinline__ int v_turn(int key) { return key & 7; }

template <int D, int WR>
__global__ void __launch_bounds__(kF32Threads, 2) q4_f32_kernel(const __grid_constant__ Q8AttnArgs a) {
  using L = F32Layout<D, WR>;
  constexpr int NG = D / kQ4Group, KW = L::KW;
  constexpr int kChunks = NG / 2;                  // groups of K, and of V, that a thread widens
  constexpr int NT = kF32Keys / 8 / KW;            // products' keys of a warp, by eight
  extern __shared__ __align__(16) float smem_f[];
  float* const sq = smem_f;                        // [WR][D / 8][32][4]: operands as they are taken
  float* const sk = sq + L::q;                     // [64][D]
  float* const sv = sk + L::kv;                    // [64][D]
  grid_dependency_sync();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int wr = warp % WR, key_base = (warp / WR) * (kF32Keys / KW);
  const int sp = blockIdx.x, hk = blockIdx.y / a.nrg, rg = blockIdx.y % a.nrg, b = blockIdx.z;
  const int P = min(max(a.plen[b], 0), a.map.cap);
  const int nsb = q8_splits(a, P);
  if (sp >= nsb) return;
  const int k0 = q8_first(a, P, sp), k1 = q8_end(a, P, k0);
  const int n_pre = (k1 - k0 + kF32Keys - 1) / kF32Keys;
  const int row_base = rg * a.rb, rows_here = min(a.rb, a.M - row_base);

  // a thread's groups of the next tile, and how many keys that tile has
  uint4 wk[kChunks], wv[kChunks];
  float fk[kChunks], fv[kChunks];
  int live = 0;
  auto fetch = [&](int tile) {
    const int pos = k0 + tile * kF32Keys;
    const long row0 = a.map.row(b, hk, pos);       // (64 keys from a multiple of 64 are of one page)
    if (row0 < 0 && tid == 0) report_error(a.err, TSD_DEV_ERR_BAD_PAGE, b);
    live = row0 < 0 ? 0 : min(k1 - pos, kF32Keys);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int x = warp + 4 * i, grp = x % NG, key = lane + 32 * (x / NG);
      const bool there = key < live;
      const long row = there ? row0 + key : 0;
      const uint4 none = make_uint4(0u, 0u, 0u, 0u);
      wk[i] = there ? __ldg((const uint4*)(a.kc + row * (D / 2)) + grp) : none;
      wv[i] = there ? __ldg((const uint4*)(a.vc + row * (D / 2)) + grp) : none;
      fk[i] = there ? bf16_value(__ldg((const uint16_t*)a.ke + row * NG + grp)) : 0.f;
      fv[i] = there ? bf16_value(__ldg((const uint16_t*)a.ve + row * NG + grp)) : 0.f;
    }
  };
  if (n_pre > 0) fetch(0);

  // Q: lane (g, t) takes rows g, g + 8 of a warp's and, of each 16 dims, 4 t .. 4 t + 3: the
  // first two in one product, the others in the next.
  float c2[2];                                     // factors of the scores
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 16 * wr + g + 8 * i;
    float4 w[D / 16];
    float top = 0.f, zero = 0.f;                   // (zero: NaN if an element is not finite)
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      w[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < rows_here) {
        const int pr = row_base + row, tr = pr / a.g, qh = hk * a.g + pr % a.g;
        w[j] = __ldg((const float4*)((const float*)a.q + (((long)b * a.R + tr) * a.Hq + qh) * D) + 4 * j + t);
      }
      top = fmaxf(top, fmaxf(fmaxf(fabsf(w[j].x), fabsf(w[j].y)), fmaxf(fabsf(w[j].z), fabsf(w[j].w))));
      zero += (w[j].x * 0.f + w[j].y * 0.f) + (w[j].z * 0.f + w[j].w * 0.f);
    }
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
      zero += __shfl_xor_sync(kFull, zero, x);
    }
    const bool low = top < 8.67361738e-19f;        // 2^-60
    const float f = low ? 18446744073709551616.f : 1.f;
    // (NaN for such a row: its terms would lose that)
    c2[i] = a.qscale * (low ? 5.42101086e-20f : 1.f) + zero;
    if (warp < WR) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {           // operands: (g, 2 dims), (g + 8, 2 dims)
        float* const to = sq + ((wr * (D / 8) + 2 * j) * 32 + lane) * 4 + i;
        to[0] = w[j].x * f;
        to[2] = w[j].y * f;
        to[128] = w[j].z * f;
        to[130] = w[j].w * f;
      }
    }
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) o[i][x] = 0.f;

  // a tile that lies in shared memory; `first`: the tree row of its first key
  auto visit = [&](int nv, auto tree, int first) {
    constexpr bool is_tree = decltype(tree)::value;
    if (key_base >= nv) return;
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
    const float4* const q4 = (const float4*)sq + wr * (D / 8) * 32 + lane;
    const float* const kb = sk + (key_base + g) * D;
    const int turn = k_turn(g);
#pragma unroll 1
    for (int j = 0; j < D / 16; j += 2) {
      float d[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) d[n][x] = 0.f;
#pragma unroll
      for (int y = 0; y < 2; ++y) {                // 16 dims: two products
        uint32_t hi[2][4], lo[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 q = q4[(2 * (j + y) + i) * 32];
          cut_terms(q.x, hi[i][0], lo[i][0]);
          cut_terms(q.y, hi[i][1], lo[i][1]);
          cut_terms(q.z, hi[i][2], lo[i][2]);
          cut_terms(q.w, hi[i][3], lo[i][3]);
        }
        const int unit = ((4 * (j + y) + t) ^ turn) * 4;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 k = *(const float4*)(kb + 8 * n * D + unit);
          uint32_t kx = __float_as_uint(k.x), ky = __float_as_uint(k.y), kz = __float_as_uint(k.z),
                   kw = __float_as_uint(k.w);
          if constexpr (is_tree) {
            uint32_t hx, hy, hz, hw, lx, ly, lz, lw;
            cut_terms(k.x, hx, lx);
            cut_terms(k.y, hy, ly);
            cut_terms(k.z, hz, lz);
            cut_terms(k.w, hw, lw);
            mma_tf32(d[n], lo[0], lx, ly);
            mma_tf32(d[n], lo[1], lz, lw);
            mma_tf32(d[n], hi[0], lx, ly);
            mma_tf32(d[n], hi[1], lz, lw);
            kx = hx; ky = hy; kz = hz; kw = hw;
          }
          mma_tf32(d[n], lo[0], kx, ky);
          mma_tf32(d[n], lo[1], kz, kw);
          mma_tf32(d[n], hi[0], kx, ky);
          mma_tf32(d[n], hi[1], kz, kw);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[n][x] += d[n][x];
    }
    bool raised = false;
    float al[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {                  // rows g, g + 8: keys 2 t, 2 t + 1 of every eight
      uint64_t sees = ~0ull;                       // of the tile's keys
      if constexpr (is_tree) {
        const int row = 16 * wr + g + 8 * i, tr = row < rows_here ? (row_base + row) / a.g : 0;
        const uint64_t mask = tr > 0 ? a.mask[(long)b * a.R + tr] : 0ull;
        sees = first == 0 ? mask << 1 | 1ull : mask >> 63;    // (row 0: the root; bit j - 1: row j)
      }
      float top = m[i];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int key = key_base + 8 * n + 2 * t + x;
          float& y = s[n][2 * i + x];
          y = key < nv && (!is_tree || (sees >> key & 1u)) ? y * c2[i] : -INFINITY;
          top = fmaxf(top, y);
        }
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
      al[i] = top == m[i] ? 1.f : m[i] == -INFINITY ? 0.f : ex2(m[i] - top);
      raised |= al[i] != 1.f;
      m[i] = top;
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float& y = s[n][2 * i + x];
          y = ex2(y - base);
          sum += y;
        }
      l[i] = fmaf(l[i], al[i], sum);
    }
    if (__any_sync(kFull, raised)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[i][x] *= al[x >> 1];
    }
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {             // 64 dims
      float d[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) d[i][x] = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {               // eight keys: lane t has 2 t and 2 t + 1
        uint32_t hi[4], lo[4];
        near_terms(s[n][0], hi[0], lo[0]);
        near_terms(s[n][2], hi[1], lo[1]);
        near_terms(s[n][1], hi[2], lo[2]);
        near_terms(s[n][3], hi[3], lo[3]);
        const float* const vb = sv + (key_base + 8 * n + 2 * t) * D;
#pragma unroll
        for (int u = 0; u < 2; ++u) {              // lane g has dims 4 g .. of 32
          const int unit = 16 * c + 8 * u + g;
          const float4 va = *(const float4*)(vb + (unit ^ v_turn(2 * t)) * 4);
          const float4 vc = *(const float4*)(vb + D + (unit ^ v_turn(2 * t + 1)) * 4);
          const float x0[4] = {va.x, va.y, va.z, va.w}, x1[4] = {vc.x, vc.y, vc.z, vc.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0 = __float_as_uint(x0[i]), b1 = __float_as_uint(x1[i]);
            float (&to)[4] = d[4 * u + i];
            if constexpr (is_tree) {
              uint32_t h0, h1, l0, l1;
              cut_terms(x0[i], h0, l0);
              cut_terms(x1[i], h1, l1);
              mma_tf32(to, lo, l0, l1);
              mma_tf32(to, hi, l0, l1);
              b0 = h0;
              b1 = h1;
            }
            mma_tf32(to, lo, b0, b1);
            mma_tf32(to, hi, b0, b1);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[8 * c + i][x] += d[i][x];
    }
  };

#pragma unroll 1
  for (int tile = 0; tile < n_pre; ++tile) {
    __syncthreads();                               // the tile before has been read
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int x = warp + 4 * i, grp = x % NG, key = lane + 32 * (x / NG);
      const uint32_t ck[4] = {wk[i].x, wk[i].y, wk[i].z, wk[i].w}, cv[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float y[8];
        const int unit = 8 * grp + 2 * u;
        widen8(ck[u], fk[i], y);
        *(float4*)(sk + key * D + (unit ^ k_turn(key)) * 4) = make_float4(y[0], y[1], y[2], y[3]);
        *(float4*)(sk + key * D + ((unit + 1) ^ k_turn(key)) * 4) = make_float4(y[4], y[5], y[6], y[7]);
        widen8(cv[u], fv[i], y);
        *(float4*)(sv + key * D + (unit ^ v_turn(key)) * 4) = make_float4(y[0], y[1], y[2], y[3]);
        *(float4*)(sv + key * D + ((unit + 1) ^ v_turn(key)) * 4) = make_float4(y[4], y[5], y[6], y[7]);
      }
    }
    const int nv = live;
    if (tile + 1 < n_pre) fetch(tile + 1);
    __syncthreads();
    visit(nv, std::false_type{}, 0);
  }
  if (sp == nsb - 1) {
#pragma unroll 1
    for (int j0 = 0; j0 < a.R; j0 += kF32Keys) {
      const int nv = min(a.R - j0, kF32Keys);
      __syncthreads();
      // (a row that holds a NaN or an infinity: no values, and NaN scores for those that see it)
      for (int key = warp; key < kF32Keys; key += 4) {
        constexpr int kUnits = D / 4;
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
        if (key < nv && lane < kUnits) {
          const long row = ((long)b * a.R + j0 + key) * a.map.Hkv + hk;
          k = __ldg((const float4*)((const float*)a.kt + row * D) + lane);
          v = __ldg((const float4*)((const float*)a.vt + row * D) + lane);
        }
        const float zero = (k.x * 0.f + k.y * 0.f) + (k.z * 0.f + k.w * 0.f) +
                           ((v.x * 0.f + v.y * 0.f) + (v.z * 0.f + v.w * 0.f));
        if (__any_sync(kFull, zero != 0.f)) {      // (NaN)
          k = make_float4(NAN, NAN, NAN, NAN);
          v = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (lane < kUnits) {
          *(float4*)(sk + key * D + (lane ^ k_turn(key)) * 4) = k;
          *(float4*)(sv + key * D + (lane ^ v_turn(key)) * 4) = v;
        }
      }
      __syncthreads();
      visit(nv, std::true_type{}, j0);
    }
  }

#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) l[i] += __shfl_xor_sync(kFull, l[i], x);
  float* const s_o = sk;                           // [4][16][D]
  float2* const s_ml = (float2*)(sk + 4 * 16 * D); // [4][16]
  if constexpr (KW > 1) {
    // the warps of a row, joined by the first
    __syncthreads();
    if (t == 0) {
      s_ml[warp * 16 + g] = make_float2(m[0], l[0]);
      s_ml[warp * 16 + g + 8] = make_float2(m[1], l[1]);
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = -INFINITY, sum = 0.f;
      for (int w = wr; w < 4; w += WR) top = fmaxf(top, s_ml[w * 16 + g + 8 * i].x);
      for (int w = wr; w < 4; w += WR) {
        const float2 x = s_ml[w * 16 + g + 8 * i];
        sum += x.x == -INFINITY ? (x.y != x.y ? x.y : 0.f) : ex2(x.x - top) * x.y;
      }
      f[i] = m[i] == -INFINITY ? (l[i] != l[i] ? 1.f : 0.f) : ex2(m[i] - top);
      m[i] = top;
      l[i] = sum;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[i][x] = f[x >> 1] == 0.f ? 0.f : o[i][x] * f[x >> 1];
    if (warp >= WR) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *(float4*)(s_o + ((warp * (D / 8) + i) * 32 + lane) * 4) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
    }
    __syncthreads();
    if (warp >= WR) return;
    for (int w = wr + WR; w < 4; w += WR)
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float4 x = *(const float4*)(s_o + ((w * (D / 8) + i) * 32 + lane) * 4);
        o[i][0] += x.x;
        o[i][1] += x.y;
        o[i][2] += x.z;
        o[i][3] += x.w;
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 16 * wr + g + 8 * i;
    if (row >= rows_here) continue;
    const int pr = row_base + row, tr = pr / a.g, qh = hk * a.g + pr % a.g;
    const long orow = ((long)b * a.R + tr) * a.Hq + qh;
    const long prow = (((long)b * a.Hq + qh) * a.nr + tr) * a.nsplit + sp;
    // (a split whose pages are all missing saw nothing: weight 0)
    const float inv = m[i] == -INFINITY && l[i] == 0.f ? 0.f : 1.f / l[i];
    const float lse2 = m[i] + log2f(l[i]);
    float* const dst = nsb == 1 ? (float*)a.out + orow * D : (float*)a.part_o + prow * D;
#pragma unroll
    for (int u = 0; u < D / 32; ++u)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        *(float4*)(dst + 32 * u + 8 * t + 4 * x) =
            make_float4(o[4 * u][2 * i + x] * inv, o[4 * u + 1][2 * i + x] * inv, o[4 * u + 2][2 * i + x] * inv,
                        o[4 * u + 3][2 * i + x] * inv);
    if (t == 0) {
      if (nsb == 1) a.lse[orow] = lse2 * 0.69314718055994531f;
      else a.part_meta[prow] = make_float2(lse2, 1.f);
    }
  }
}

template <int D, int WR>
void launch_f32(const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  constexpr uint32_t smem = F32Layout<D, WR>::total;
  const auto kern = q4_f32_kernel<D, WR>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  launch(kern, dim3(p.nsplit, a.map.Hkv * p.nrg, a.B), dim3(kF32Threads), smem, st, a);
}

}  // namespace

void launch_q4_f32(const Q8AttnArgs& a, const Q8Plan& p, int D, cudaStream_t st) {
  if (D == 128)
    p.rb > 32 ? launch_f32<128, 4>(a, p, st) : p.rb > 16 ? launch_f32<128, 2>(a, p, st) : launch_f32<128, 1>(a, p, st);
  else
    p.rb > 32 ? launch_f32<64, 4>(a, p, st) : p.rb > 16 ? launch_f32<64, 2>(a, p, st) : launch_f32<64, 1>(a, p, st);
}

}  // namespace tsd
