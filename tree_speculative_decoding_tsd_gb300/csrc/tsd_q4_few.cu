// Path of tsd_tree_verify_attn_q4 for bf16 heads of 64 or 128 dims with few packed rows
// (R tree rows x g query heads of a KV head): decoding, small trees.
//
//   S[key][n]  = K . Q^T      16 keys x 8 columns x 16 dims per instruction
//   O[dim][n] += V^T . P^T    16 dims x 8 columns x 16 keys
//
// Widening is what this path has to do cheaply: codes go from shared memory straight into
// the operand registers of mma.sync (tcgen05 takes operands from shared or tensor memory,
// so that every widened element would be written and read once more; the products of
// few columns are far from binding here: 26% of the tensor pipe).  A warp works alone on
// chunks of 32 keys, which it copies itself, a chunk ahead, into a ring of its own: no barrier
// between the first chunk and the last.
//
// Numbers.
//   K   a word's masked halves are fp16 numbers as they stand, c * 2^-24 or c * 2^-20
//       (tsd_q4.cuh), exact; columns of Q carry the factor between the two.  Each group
//       of 32 dims has its own product c . q in fp32, then times the group's scale; -8 sum(q)
//       times the scales comes from a small product (sums in three bf16 terms): fp32 all the way.
//   Q   fp16 times a power of two of its row, every other pair over 16: exact for elements
//       down to 2^-27 of the row's largest, off by 2^-35 of it at most below.
//   V   fp16, one fused multiply-add: (c - 8) s 2^(-E - 9), E the exponent above the chunk's
//       largest scale: 2^-12, or 2^-25 (2^-15 of the chunk's largest scale) where that is more.
//   P   fp16: 2^(x + E - m), m a running bound of x + E over the warp's keys (raised
//       where a chunk passes it by 8): 2^-12, and steps of 2^-24.  Its sum has a bound of its
//       own (kQ4Near).
//   scratch rows: fp32 on the CUDA cores, a warp per packed row, while the first chunks are
//       under way.
// Each warp's sum, bound and output are joined at the end, in fp32.
//
// What bounds it.  One token of 16 requests of 32 heads over 20k to 32k keys: 112 us, 4.4 TB/s
// (72 us by the bytes; 106 in the kernel, where no warp waits for its copies to speak of).  The
// copies alone, the arithmetic left out, take 93 us in the same graph: 17 us of that are launch,
// set-up, joint and merge.  It is issue slots (56% full over the kernel's whole time, three
// quarters within the loop), the ALU (48%; it takes an instruction in two cycles) and the
// products' latency, at four warps a scheduler.  Up to eight packed rows need 128 registers:
// sixteen warps an SM, in CTAs of eight, or of four for many short requests, so that one's start
// and end lie beside the others' chunks (one CTA of sixteen: 142 us); nine to sixteen rows 168
// registers: twelve warps, in one CTA or in three.  Tried and dropped: chunks of 16 keys with
// rings of two to five (131 us, 45 instead of 42 for 32 requests over 1k to 4k), three CTAs of
// eight warps and 80 registers (144 us), the work dealt out evenly over one CTA per slot by the
// requests' lengths (120 us, but 80 instead of 56 us for 200 requests below 900 keys and 77
// instead of 56 for 32 of 4 rows: a CTA then starts and ends once per request).
#include <algorithm>

#include "tsd_host.h"
#include "tsd_q4.cuh"
#include "tsd_q4_attn.cuh"
#include "tsd_q8_tc.cuh"

namespace tsd {
namespace {

constexpr float kNone = -3.4e38f;                  // a bound before the first key
constexpr int H = 2, kChunk = 16 * H;              // keys of a chunk: two halves, a product's rows each

template <int D, int NT, int S, int W>
struct FewLayout {
  static constexpr int NG = D / kQ4Group;
  // A row's codes, padded so that neither way of reading (K: a unit of eight rows; V: a run
  // of words of four even or four odd rows) meets a bank twice.
  static constexpr uint32_t row = D / 2 + 16;
  static constexpr uint32_t codes = kChunk * row, scales = kChunk * NG * 2;
  static constexpr uint32_t stage = 2 * codes + 2 * scales;
  static constexpr uint32_t ring = W * S * stage;
  static constexpr int pitch = D + 4;              // floats of a row in the joint
  static constexpr uint32_t joint = W * NT * 8 * pitch * 4;
  static constexpr uint32_t off_tree = ring > joint ? ring : joint;     // float [8 NT][D]
  static constexpr uint32_t off_ml = off_tree + NT * 8 * D * 4;         // float4 [W + 1][8 NT]: m, l, u
  static constexpr uint32_t off_q = off_ml + (W + 1) * NT * 8 * 16;     // uint4 [NT][NG][32]: B operands
  static constexpr uint32_t off_qs = off_q + NT * NG * 32 * 16;         // float [NT][NG][8]: -8 times their sums
  static constexpr uint32_t off_c2 = off_qs + NT * NG * 8 * 4;          // float [8 NT]: factor of the scores
  static constexpr uint32_t off_req = off_c2 + NT * 8 * 4;              // request, its length; a huge row
  static constexpr uint32_t total = off_req + 16;
  static_assert(stage % 16 == 0, "whole units");
};

__device__ __forceinline__ void cp_async_z(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst), "l"(src), "n"(N),
               "r"(there ? N : 0) : "memory");
}
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A.B, bf16.
__device__ __forceinline__ void mma_16816_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// An 8 x 8 matrix of 16-bit elements, a row on four lanes, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;\n" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <int D, int NT, int S, int W, int kCtas>
__global__ void __launch_bounds__(W * 32, kCtas)
q4_few_kernel(const __grid_constant__ Q8AttnArgs a) {
  using L = FewLayout<D, NT, S, W>;
  constexpr int NG = L::NG, NW = D / 64;           // groups; words of V per lane and key
  extern __shared__ __align__(128) uint8_t smem[];
  grid_dependency_sync();
  // (The last splits first: those that are cut short or hold the scratch rows do not end up behind
  // the others.  One token of 16 requests over 20k to 32k keys 113 -> 110 us, of 16 over 8k to 32k
  // 95 -> 90.)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int hk = blockIdx.x, sp = a.nsplit - 1 - a.split0 - blockIdx.z;
  int* const s_huge = (int*)(smem + L::off_req) + 2;  // a row from 2^117 on: its factor in two steps
  if (tid == 0) *s_huge = 0;
  int P;
  const int b = request_at(a, blockIdx.y, P, (volatile int*)(smem + L::off_req));
  const int nsb = q8_splits(a, P);
  if (sp >= nsb) return;
  const int k0 = q8_first(a, P, sp), k1 = q8_end(a, P, k0);
  const bool with_tree = sp == nsb - 1;
  __syncthreads();                                 // (s_huge)

  // ------------------------------------------------------------- the ring
  // A warp's chunks lie W * kChunk keys apart: within a page the next one is at a fixed
  // distance.
  const uint32_t ring = su32(smem) + warp * (S * L::stage);
  const int last = (k1 - k0 + kChunk - 1) / kChunk;   // chunks of the split
  const uint8_t *kp, *vp, *ksp, *vsp;                 // this lane's part of the next chunk
  int left;                                           // steps within the page
  auto point_at = [&](int c) {
    long row = 0;
    left = 0x7fffffff;
    if (c < last) {
      const int pos = k0 + c * kChunk;
      row = a.map.row(b, hk, pos);
      if (row < 0) {                                  // (the request's output is not valid)
        if (lane == 0) report_error(a.err, TSD_DEV_ERR_BAD_PAGE, b);
        row = 0;
      }
      if (a.map.page_size) left = (a.map.page_size - pos % a.map.page_size - 1) / (W * kChunk);
    }
    kp = a.kc + row * (D / 2) + lane * 16;
    vp = a.vc + row * (D / 2) + lane * 16;
    ksp = a.ke + (row + lane) * (NG * 2);
    vsp = a.ve + (row + lane) * (NG * 2);
  };
  constexpr int U = D / 32, kRowStep = 32 / U;        // units of a row, rows of a warp's copy
  constexpr int kCopies = kChunk / kRowStep;
  const uint32_t to = (uint32_t)(lane / U) * L::row + (lane % U) * 16;
  // chunk c into a slot; then on to the warp's next one
  auto request = [&](int c, int slot) {
    const uint32_t st = ring + slot * L::stage;
    const int nv = k1 - k0 - c * kChunk;
    if (nv >= kChunk) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        cp_async_z(st + to + i * kRowStep * L::row, kp + 512 * i, true);
        cp_async_z(st + L::codes + to + i * kRowStep * L::row, vp + 512 * i, true);
      }
      cp_async_small<NG * 2>(st + 2 * L::codes + lane * (NG * 2), ksp, true);
      cp_async_small<NG * 2>(st + 2 * L::codes + L::scales + lane * (NG * 2), vsp, true);
    } else if (nv > 0) {                              // rows that are not there: zeros
#pragma unroll 1
      for (int i = 0; i < kCopies; ++i) {
        const bool there = lane / U + i * kRowStep < nv;
        cp_async_z(st + to + i * kRowStep * L::row, there ? kp + 512 * i : a.kc, there);
        cp_async_z(st + L::codes + to + i * kRowStep * L::row, there ? vp + 512 * i : a.vc, there);
      }
      const bool there = lane < nv;
      cp_async_small<NG * 2>(st + 2 * L::codes + lane * (NG * 2), there ? ksp : a.ke, there);
      cp_async_small<NG * 2>(st + 2 * L::codes + L::scales + lane * (NG * 2), there ? vsp : a.ve, there);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
    if (left > 0) {
      --left;
      kp += W * kChunk * (D / 2);
      vp += W * kChunk * (D / 2);
      ksp += W * kChunk * (NG * 2);
      vsp += W * kChunk * (NG * 2);
    } else {
      point_at(c + W);
    }
  };
  point_at(warp);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) request(warp + i * W, i);

  // ------------------------------------------------------ Q as the B operand
  // lane (g, t): column g, and of each group j the dims of word 4 j + t.  In shared memory,
  // for all warps, and with it -8 * 2^-24 sum(q) of each group.
  uint4* const s_q = (uint4*)(smem + L::off_q);
  float* const s_qs = (float*)(smem + L::off_qs);
  float* const s_c2 = (float*)(smem + L::off_c2);
#pragma unroll 1
  for (int i0 = warp; i0 < NT * NG; i0 += W) {     // a warp per group
    const int nt = i0 / NG, j = i0 % NG, n = nt * 8 + g;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    uint32_t top = 0;
    if (n < a.M) {
      const int tr = a.r0 + n / a.g, qh = hk * a.g + n % a.g;
      const uint4* src = (const uint4*)((const __nv_bfloat16*)a.q + (((long)b * a.R + tr) * a.Hq + qh) * D) + t;
      w = __ldg(src + 4 * j);
#pragma unroll
      for (int i = 0; i < NG; ++i) top = top_pairs(top, __ldg(src + 4 * i));
    }
    top = top_of(top);
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    // the largest element into [2^14, 2^15)
    const bool bad = top >= 0x7f800000u;
    const int e = row_exponent(top);
    const float f = bad ? 0.f : q8_scale(268 - e);
    if (!bad && e >= 244) *s_huge = 1;
    // 2^(e - 127) of the row, over 2^14; 2^24 of the codes: 2^10 to come
    if (t == 0 && j == 0) s_c2[n] = bad ? __int_as_float(0x7fffffff) : a.qscale * q8_scale(e);
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t q[4];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float h = i & 1 ? f * 0.0625f : f;
      const uint32_t bits = bad ? 0u : in[i];
      q[i] = pack_half2(__uint_as_float(bits << 16) * h, __uint_as_float(bits & 0xffff0000u) * h);
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&q[i]));
      sum = fmaf(i & 1 ? 16.f : 1.f, y.x + y.y, sum);
    }
    s_q[i0 * 32 + lane] = make_uint4(q[0], q[1], q[2], q[3]);
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
    sum *= -8.f * 5.9604644775390625e-08f;
    if (t == 0) s_qs[i0 * 8 + g] = sum;
  }

  // --------------------------------------------------------- scratch rows
  float* const tree_o = (float*)(smem + L::off_tree);
  float4* const s_ml = (float4*)(smem + L::off_ml);
  if (with_tree) {
    constexpr int E = D / 32;                      // dims of a lane
#pragma unroll 1
    for (int n = W - 1 - warp; n < a.M; n += W) {   // (the warps that have no group of Q first)
      const int tr = a.r0 + n / a.g, qh = hk * a.g + n % a.g;
      const uint64_t mask = tr > 0 ? a.mask[(long)b * a.R + tr] : 0ull;   // (row 0: the root; bit j - 1: row j)
      auto row4 = [&](const void* base, long row, float (&x)[E]) {
        const uint32_t* p = (const uint32_t*)((const __nv_bfloat16*)base + row * D) + lane * (E / 2);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          const uint32_t v = __ldg(p + i);
          x[2 * i] = __uint_as_float(v << 16);
          x[2 * i + 1] = __uint_as_float(v & 0xffff0000u);
        }
      };
      float q[E], o[E], m = -INFINITY, l = 0.f;
      row4(a.q, ((long)b * a.R + tr) * a.Hq + qh, q);
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] = 0.f;
#pragma unroll 1
      for (int j0 = 0; j0 < a.R; j0 += 4) {
        const uint32_t four = j0 == 0 ? (uint32_t)(mask << 1) | 1u : (uint32_t)(mask >> (j0 - 1));
        if ((four & 15u) == 0u) continue;          // (the same for the whole warp)
        float k[4][E], v[4][E], s[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const long row = ((long)b * a.R + min(j0 + u, a.R - 1)) * a.map.Hkv + hk;
          row4(a.kt, row, k[u]);
          row4(a.vt, row, v[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          s[u] = 0.f;
#pragma unroll
          for (int i = 0; i < E; ++i) s[u] = fmaf(q[i], k[u][i], s[u]);
        }
#pragma unroll
        for (int o2 = 16; o2 > 0; o2 >>= 1)
#pragma unroll
          for (int u = 0; u < 4; ++u) s[u] += __shfl_xor_sync(kFull, s[u], o2);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int j = j0 + u;
          if (j >= a.R || !(four >> u & 1u)) continue;
          float x = s[u] * a.qscale;
          if (x == -INFINITY) {                    // no weight, unless an element is not finite
            float zero = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) zero += k[u][i] * 0.f + v[u][i] * 0.f;
            if (!__any_sync(kFull, zero != 0.f)) continue;
            x = __int_as_float(0x7fffffff);
          }
          const float mn = fmaxf(m, x);
          const float al = mn == m ? 1.f : ex2(m - mn), p = ex2(x - mn);
          const float p9 = p * 0.001953125f;       // 2^-9: sums of the largest values stay finite
          m = mn;
          l = fmaf(l, al, p);
#pragma unroll
          for (int i = 0; i < E; ++i) o[i] = fmaf(o[i], al, p9 * v[u][i]);
        }
      }
#pragma unroll
      for (int i = 0; i < E; ++i) tree_o[n * D + lane * E + i] = o[i];
      if (lane == 0) s_ml[W * NT * 8 + n] = make_float4(m, l, m, 0.f);
    }
  }

  // ------------------------------------------------------------ the chunks
  __syncthreads();
  const bool huge = *s_huge != 0;
  float acc[NT][NW * 4][4], m[NT][2], l[NT][2], c2[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < NW * 4; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[nt][i][x] = 0.f;
    m[nt][0] = m[nt][1] = kNone;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) c2[nt][x] = s_c2[nt * 8 + 2 * t + x] * (huge ? 1.f : 1024.f);
  }
  // The codes' offset as a product of its own: scales of a key (NG of them, bf16, as they are)
  // times the sums, each in three bf16 terms (24 bits): its rows are (term, group).
  uint32_t ob[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = 2 * t + 8 * i, term = k / NG;  // (a pair is of one term)
      float x[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        x[y] = term < 3 ? s_qs[(nt * NG + k % NG + y) * 8 + g] : 0.f;
        for (int z = 0; z < term && z < 2; ++z) x[y] -= __bfloat162float(__float2bfloat16_rn(x[y]));
      }
      ob[nt][i] = pack_bf16x2(x[0], x[1]);
    }
  const uint8_t* const mine = smem + warp * (S * L::stage);
  // The exponents of the sums' bounds, a byte for each of the lane's columns, from the first chunk on
  // whose E is far from 0 (kQ4Near).
  uint32_t eus = 0;
  float head = kOverflow;                          // (then -inf: every chunk raises the bounds)
  int slot = 0;
#pragma unroll 1
  for (int c = warp; c < last; c += W) {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(S - 2) : "memory");
    __syncwarp();
    const int nv = k1 - k0 - c * kChunk;
    request(c + (S - 1) * W, slot == 0 ? S - 1 : slot - 1);
    const uint8_t* const st = mine + slot * L::stage;
    slot = slot == S - 1 ? 0 : slot + 1;

    // scores of keys g and g + 8 of each half, columns 2 t and 2 t + 1
    float s[NT][H][4];
    const uint8_t* const kl = st + g * L::row + 4 * t;
    const uint8_t* const sl = st + 2 * L::codes + g * (NG * 2);
    uint32_t ks[2 * H][NG / 2];                    // rows g, g + 8, ..
#pragma unroll
    for (int x = 0; x < 2 * H; ++x) {
      const uint8_t* const p = sl + 8 * x * (NG * 2);
      if constexpr (NG == 4) {
        const uint2 y = *(const uint2*)p;
        ks[x][0] = y.x;
        ks[x][NG / 2 - 1] = y.y;
      } else {
        ks[x][0] = *(const uint32_t*)p;
      }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const uint32_t a0 = NG == 4 && (t & 1) ? ks[2 * h][NG / 2 - 1] : ks[2 * h][0];
      const uint32_t a1 = NG == 4 && (t & 1) ? ks[2 * h + 1][NG / 2 - 1] : ks[2 * h + 1][0];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_16816_bf16(s[nt][h], a0, a1, a0, a1, ob[nt][0], ob[nt][1]);
    }
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      uint4 q[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) q[nt] = s_q[(nt * NG + j) * 32 + lane];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const uint32_t w0 = *(const uint32_t*)(kl + 16 * h * L::row + 16 * j);
        const uint32_t w1 = *(const uint32_t*)(kl + (16 * h + 8) * L::row + 16 * j);
        const uint32_t h0 = w0 >> 8, h1 = w1 >> 8;
        const uint32_t k0w = ks[2 * h][j / 2], k1w = ks[2 * h + 1][j / 2];
        const float s0 = __uint_as_float(j & 1 ? k0w & 0xffff0000u : k0w << 16);
        const float s1 = __uint_as_float(j & 1 ? k1w & 0xffff0000u : k1w << 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_16816(d, w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u, q[nt].x, q[nt].y);
          mma_16816(d, h0 & 0x000f000fu, h1 & 0x000f000fu, h0 & 0x00f000f0u, h1 & 0x00f000f0u, q[nt].z, q[nt].w);
          float* const r = s[nt][h];
          r[0] = fmaf(d[0], s0, r[0]);
          r[1] = fmaf(d[1], s0, r[1]);
          r[2] = fmaf(d[2], s1, r[2]);
          r[3] = fmaf(d[3], s1, r[3]);
        }
      }
    }

    // the exponent above the chunk's largest value scale
    const uint8_t* const sv = st + 2 * L::codes + L::scales;
    int E;
    float down;                                    // weights as terms of the sum
    {
      constexpr int kWords = NG / 2;
      uint32_t w[kWords], top = 0;
      if constexpr (kWords == 2) {
        const uint2 y = *(const uint2*)(sv + lane * 8);
        w[0] = y.x;
        w[kWords - 1] = y.y;
      } else {
        w[0] = *(const uint32_t*)(sv + lane * 4);
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
      top = __reduce_max_sync(kFull, max(top & 0xffffu, top >> 16));
      E = (int)(top >> 7) - 126;
      // (far from 0, or scales that are not finite)
      if (__builtin_expect(top - ((126u - kQ4Near) << 7) >= (2u * kQ4Near + 1u) << 7, 0)) {
        if (top >= 0x7f80u) {
          top = 0;
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const uint32_t lo = w[i] & 0x7fffu, hi = w[i] >> 16 & 0x7fffu;
            top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
          }
          top = __reduce_max_sync(kFull, top);
        }
        E = top == 0u ? 0 : min(max((int)(top >> 7) - 126, kQ4MinExp), kQ4MaxExp);   // (zeros: at any)
        if (abs(E) > kQ4Near) head = -INFINITY;
      }
      down = q8_scale(127 - E);
    }
    const float fE = (float)E;

    // P, in the layout of the scores
    uint32_t pb[NT][H][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (huge) {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[nt][h][x] *= 1024.f;
      }
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[nt][h][x] = fmaf(s[nt][h][x], c2[nt][x & 1], fE);
      if (nv < kChunk) {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (16 * h + 8 * (x >> 1) + g >= nv) s[nt][h][x] = -INFINITY;
      }
      float top[2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
        top[x] = max3f(fmaxf(s[nt][0][x], s[nt][0][x + 2]), s[nt][1][x], s[nt][1][x + 2]);
      if (__any_sync(kFull, !(top[0] <= m[nt][0] + head) || !(top[1] <= m[nt][1] + head))) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(kFull, top[x], o));
          const float mn = fmaxf(m[nt][x], top[x]);
          const float al = ex2(m[nt][x] - mn);
          if (head < 0.f) {                          // the sum of the chunk on its own
            down = 0.f;
            const int at = 8 * (2 * nt + x);
            const float e0 = (float)(int8_t)(eus >> at), e = q4_near(m[nt][x], e0, mn, top[x] - fE);
            eus = (eus & ~(255u << at)) | ((uint32_t)(int)e & 255u) << at;
            l[nt][x] *= ex2((m[nt][x] - mn) + (e - e0));
#pragma unroll
            for (int h = 0; h < H; ++h)
              l[nt][x] += ex2((s[nt][h][x] - mn) + (e - fE)) + ex2((s[nt][h][x + 2] - mn) + (e - fE));
          } else {
            l[nt][x] *= al;
          }
          m[nt][x] = mn;
#pragma unroll
          for (int i = 0; i < NW * 4; ++i) {
            acc[nt][i][x] *= al;
            acc[nt][i][x + 2] *= al;
          }
        }
      }
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float p0 = ex2(s[nt][h][0] - m[nt][0]), p1 = ex2(s[nt][h][1] - m[nt][1]);
        const float p2 = ex2(s[nt][h][2] - m[nt][0]), p3 = ex2(s[nt][h][3] - m[nt][1]);
        sum[0] += p0 + p2;
        sum[1] += p1 + p3;
        pb[nt][h][0] = transposed(pack_half2(p0, p1));
        pb[nt][h][1] = transposed(pack_half2(p2, p3));
      }
      l[nt][0] = fmaf(sum[0], down, l[nt][0]);
      l[nt][1] = fmaf(sum[1], down, l[nt][1]);
    }

    // V: lane (g, t) takes dims 8 NW g .. of keys 2 t, 2 t + 1 and 2 t + 8, 2 t + 9 of a half
    const float up = q8_scale(127 + 15 - E);
    const uint8_t* const vl = st + L::codes + 2 * t * L::row + 4 * NW * g;
    const uint8_t* const vs = sv + 2 * t * (NG * 2) + (NG == 4 ? g >> 1 : g >> 2) * 2;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      uint32_t f0[2], f1[2], z[2], v[4][NW];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * h + 8 * i;
        const uint32_t sa = *(const uint16_t*)(vs + r * (NG * 2)), sb = *(const uint16_t*)(vs + (r + 1) * (NG * 2));
        f0[i] = pack_half2(bf16_value(sa) * up, bf16_value(sb) * up);
        f1[i] = hmul2(f0[i], 0x2c002c00u);           // 2^-4
        z[i] = hmul2(f0[i], 0x80088008u);            // -2^-21
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint8_t* const p = vl + (r + x) * L::row;
          if constexpr (NW == 2) {
            const uint2 y = *(const uint2*)p;
            v[2 * i + x][0] = y.x;
            v[2 * i + x][NW - 1] = y.y;
          } else {
            v[2 * i + x][0] = *(const uint32_t*)p;
          }
        }
      }
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        // the halves of two keys: even dims, odd dims
        uint32_t ea = __byte_perm(v[0][w], v[1][w], 0x5410), oa = __byte_perm(v[0][w], v[1][w], 0x7632);
        uint32_t eb = __byte_perm(v[2][w], v[3][w], 0x5410), ob = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t mask = i & 1 ? 0x00f000f0u : 0x000f000fu;
          const uint32_t* const f = i & 1 ? f1 : f0;
          const uint32_t a0 = hfma2(ea & mask, f[0], z[0]), a1 = hfma2(oa & mask, f[0], z[0]);
          const uint32_t a2 = hfma2(eb & mask, f[1], z[1]), a3 = hfma2(ob & mask, f[1], z[1]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_16816(acc[nt][4 * w + i], a0, a1, a2, a3, pb[nt][h][0], pb[nt][h][1]);
          if (i == 1) {
            ea >>= 8;
            oa >>= 8;
            eb >>= 8;
            ob >>= 8;
          }
        }
      }
    }
  }

  // ------------------------------------------------------------- the joint
  asm volatile("cp.async.wait_group 0;\n" ::: "memory");
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float sum = l[nt][x];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
      const float top = m[nt][x] == kNone ? -INFINITY : m[nt][x];
      const float e = (float)(int8_t)(eus >> 8 * (2 * nt + x));
      if (g == 0) s_ml[warp * NT * 8 + nt * 8 + 2 * t + x] = make_float4(top, sum, top - e, 0.f);
    }
  __syncthreads();                                 // the ring has been read
  float* const s_o = (float*)smem;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float* const dst = s_o + (warp * NT * 8 + nt * 8 + 2 * t + x) * L::pitch + 8 * NW * g;
#pragma unroll
      for (int i = 0; i < NW * 4; ++i)
        *(float2*)(dst + 2 * i) = make_float2(acc[nt][i][x], acc[nt][i][x + 2]);
    }
  // A row's W + 1 parts, on sixteen lanes: the factor of each one's output.
  static_assert(W < 16, "a lane per part");
  for (int i = tid; i < NT * 8 * 16; i += W * 32) {   // (whole warps)
    const int n = i / 16, w = i % 16;
    const bool there = w < W || (w == W && with_tree);
    const float4 ml = there ? s_ml[w * NT * 8 + n] : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    float top = ml.x, near = ml.z;                 // bounds of the products, and of the sums
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      near = fmaxf(near, __shfl_xor_sync(kFull, near, o));
    }
    // (no bound: nothing seen, or scores that are all NaN)
    const bool none = ml.x == -INFINITY;
    const float f = none ? (ml.y != ml.y ? ml.y : 0.f) : ex2(ml.x - top);
    float total = none ? f : ex2(ml.z - near) * ml.y;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
    if (there) s_ml[w * NT * 8 + n] = make_float4(f * q4_over(9.f + (top - near), total), 0.f, near, total);
  }
  __syncthreads();
  for (int i = tid; i < a.M * (D / 2); i += W * 32) {
    const int n = i / (D / 2), c = i % (D / 2) * 2;
    float2 o = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w <= W; ++w) {
      if (w == W && !with_tree) break;
      const float f = s_ml[w * NT * 8 + n].x;
      const float2 x = w < W ? *(const float2*)(s_o + (w * NT * 8 + n) * L::pitch + c)
                             : *(const float2*)(tree_o + n * D + c);
      o.x = fmaf(f, x.x, o.x);                     // (0 times an infinity of a scratch value is seen, too)
      o.y = fmaf(f, x.y, o.y);
    }
    const float lse2 = s_ml[n].z + log2f(s_ml[n].w);
    const int tr = a.r0 + n / a.g, qh = hk * a.g + n % a.g;
    if (nsb == 1) {
      const long orow = ((long)b * a.R + tr) * a.Hq + qh;
      *(uint32_t*)((__nv_bfloat16*)a.out + orow * D + c) = pack_bf16x2(o.x, o.y);
      if (c == 0) a.lse[orow] = lse2 * 0.69314718055994531f;
    } else {
      const long prow = (((long)b * a.Hq + qh) * a.nr + tr - a.r0) * a.nsplit + sp;
      *(float2*)((float*)a.part_o + prow * D + c) = o;
      if (c == 0) a.part_meta[prow] = make_float2(lse2, 1.f);
    }
  }
}

template <int D, int NT, int S, int W, int kCtas>
void launch_few(const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  const uint32_t smem = FewLayout<D, NT, S, W>::total;
  const auto kern = q4_few_kernel<D, NT, S, W, kCtas>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  for (Q8AttnArgs part = a; part.split0 < p.nsplit; part.split0 += kMaxGrid)
    launch(kern, dim3(a.map.Hkv, a.B, std::min(p.nsplit - part.split0, kMaxGrid)), dim3(W * 32), smem, st, part);
}

}  // namespace

// Up to eight packed rows, 16 warps of 128 registers per SM; more need 168 (two CTAs of eight warps
// with 128: 69 instead of 50 us for 16 rows of 32 requests over 1k to 4k keys).
void launch_q4_few(const Q8AttnArgs& a, const Q8Plan& p, int D, cudaStream_t st) {
  const bool small = p.small_ctas;
  if (D == 128) {
    if (a.M <= 8) small ? launch_few<128, 1, 2, 4, 4>(a, p, st) : launch_few<128, 1, 2, 8, 2>(a, p, st);
    else small ? launch_few<128, 2, 2, 4, 3>(a, p, st) : launch_few<128, 2, 2, 12, 1>(a, p, st);
  } else {
    if (a.M <= 8) small ? launch_few<64, 1, 3, 4, 4>(a, p, st) : launch_few<64, 1, 3, 8, 2>(a, p, st);
    else small ? launch_few<64, 2, 3, 4, 3>(a, p, st) : launch_few<64, 2, 3, 12, 1>(a, p, st);
  }
}

}  // namespace tsd
