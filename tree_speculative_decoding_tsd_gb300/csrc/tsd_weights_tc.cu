// tcgen05 path of tsd_cache_weights(_q8): bf16 heads of 64 or 128 dims with up to
// 288 columns (path rows x query heads of a KV head).
//
//   S^T[key][n] = K_tile . Q^T    M = 128 keys, N = columns (up to 256), K = d
//   acc[key]    = decay * acc[key] + sum_n 2^(S^T f_n - lse_n)
// A tensor-memory lane is a cached row and a thread owns a lane, so the sum over
// the columns stays in one thread: no reduction, no second pass, and nothing but K
// is read per key (and 8 bytes of acc).  Bound by memory: per 128-key tile 32 KB
// (bf16) or 16 KB (8-bit codes) of K arrive, while a thread's exponentials take 150 to
// 290 cycles for 36 columns.  4 requests of 8 heads, 32k bf16 rows, 36 columns: 45 us,
// 5.9 TB/s; 32 requests of 1k to 4k 8-bit rows: 29 us, as long as its longest request's
// CTA takes (splitting them further: 30 us, and 3 to 9% more where all are full).
//
// 8-bit cache: kind::f8f6f4 on the codes, Q as the sum of two e4m3 numbers, powers
// of two in fp32 (tsd_q8_tc.cu).  bf16 cache: kind::f16.
//
// Q of all columns stays in shared memory (72 KB at 288 of 128 dims); more columns, groups
// of 32 heads with 9 path rows or more, take weights_simt_kernel: 32 requests of 1k to 4k
// 8-bit rows of one KV head 56 us at 288 columns, 236 us at 320.
//
// A CTA takes a run of tiles of one (request, KV head): K tiles by TMA through a
// ring as deep as shared memory allows, two warpgroups that take the even and the
// odd tiles (a score buffer of 256 columns each), one warp that issues the products
// and one that loads.  The CTA with the last tiles also takes the path's own rows,
// first, from the scratch pad.  Every wait is bounded.
#include "tsd_host.h"
#include "tsd_q8_tc.cuh"
#include "tsd_weights.cuh"

namespace tsd {
namespace {

constexpr int kSumWarps = 8, kMma = 8, kTma = 9;
constexpr int kThreads = 10 * 32;
constexpr int kMaxCols = 288;
constexpr int kMaxRing = 12;

struct WeightSmem {        // behind the ring and Q
  float f[kMaxCols];       // factor of a column's scores
  float nl[kMaxCols];      // -log2(e) lse (-inf behind the last column)
  float kt_out[32];        // 8-bit cache: factors of the path rows
  uint64_t bars[2 * kMaxRing + 7];
  uint32_t tmem, abort;
  PathSmem path;
};

enum { BAR_FULL = 0, BAR_EMPTY = kMaxRing, BAR_S_FULL = 2 * kMaxRing, BAR_S_EMPTY = BAR_S_FULL + 2,
       BAR_FINAL = BAR_S_EMPTY + 2 };

struct WeightPlan {
  int nsplit, tiles;       // CTAs per (request, head); tiles of one
  int cols, ring;          // columns at most (a multiple of 16); K slots
};

// kBufCols: columns of a score buffer; 128 where the columns fit, so that two CTAs
// share an SM (one's set-up behind the other's work), else 256.
template <int D, bool kQ8, int kBufCols, bool kPoll>
__global__ void __launch_bounds__(kThreads, kBufCols == 128 ? 2 : 1)
weights_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ WeightArgs a,
                  WeightPlan p) {
  constexpr uint32_t kTileBytes = kWeightKeys * D * (kQ8 ? 1 : 2);
  constexpr uint32_t kRowBytes = D * (kQ8 ? 1 : 2);        // of Q (twice that: hi and lo)
  constexpr int kPathSlots = kQ8 ? 2 : 1;                   // hi and lo of the path's rows
  if (threadIdx.x == kTma * 32) tma_desc_prefetch(&kmap);
  grid_dependency_sync();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = su32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const uint32_t off_q = p.ring * kTileBytes;
  const uint32_t q_bytes = p.cols * kRowBytes;
  WeightSmem& s = *(WeightSmem*)(smem + off_q + (kQ8 ? 2 : 1) * q_bytes);
  volatile uint32_t* abort = &s.abort;
  auto bar = [&](int i) { return su32(&s.bars[i]); };
  auto wait_ready = [&](uint32_t at, uint32_t parity) {
    return phase_ready<kPoll>(at, parity, a.wait_cycles);
  };
  auto wait_timed = [&](uint32_t at, uint32_t parity) {
    return phase_timed<kPoll>(at, parity, a.wait_cycles);
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sp = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
  const int P = a.plen[b];
  const int total = P > 0 ? (min(P, a.map.cap) + kWeightKeys - 1) / kWeightKeys : 0;
  const int t0 = sp * p.tiles, n_pre = max(min(total - t0, p.tiles), 0);
  // the first CTA behind or at the end of the prefix takes the path's rows
  const bool with_path = sp == max((total + p.tiles - 1) / p.tiles - 1, 0);
  if (n_pre == 0 && !with_path) return;
  const int slots0 = with_path ? kPathSlots : 0;            // ring slots taken before the prefix
  const long head = (long)b * a.map.Hkv + hk;
  auto load_k = [&](int t) {                                // prefix tile t of this CTA
    const int pos = (t0 + t) * kWeightKeys, g = slots0 + t, sl = g % p.ring;
    int y = pos, z = (int)head;
    if (a.map.page_size) {
      const long r = max(a.map.row(b, hk, pos), 0l);        // (weight_path finds missing pages)
      y = (int)(r % a.map.page_size);
      z = (int)(r / a.map.page_size);
    }
    mbar_expect_tx(bar(BAR_FULL + sl), kTileBytes);
    if (kQ8) tma_3d(sbase + sl * kTileBytes, &kmap, 0, y, z, bar(BAR_FULL + sl));
    else tma_4d(sbase + sl * kTileBytes, &kmap, 0, y, z, 0, bar(BAR_FULL + sl));
  };
  // The first K tiles are on their way before the path is known.
  const int early = min(n_pre, p.ring - slots0);
  if (tid == kTma * 32) {
    for (int i = 0; i < p.ring; ++i) {
      mbar_init(bar(BAR_FULL + i), 1);
      mbar_init(bar(BAR_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(BAR_S_FULL + i), 1);
      mbar_init(bar(BAR_S_EMPTY + i), 4);
    }
    mbar_init(bar(BAR_FINAL), 1);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    for (int t = 0; t < early; ++t) load_k(t);
  }
  const int L = weight_path(a, b, P, s.path);
  if (L < 0 || s.path.blind) {                              // nothing is weighed
    if (L >= 0 && with_path) unweighed_path(a, b, hk, P, L);
    else if (with_path && tid == 0) report_error(a.err, -L, b);
    if (tid == kTma * 32)
      for (int t = 0; t < early; ++t) mbar_wait(bar(BAR_FULL + slots0 + t), 0);
    return;
  }
  const int ncol = (L + 1) * a.g, pad = (ncol + 15) / 16 * 16;
  const int ntiles = n_pre + (with_path ? 1 : 0);           // tile 0 is the path's, if any
  const int chunks = (pad + kBufCols - 1) / kBufCols;       // of columns

  // ---------------------------------------------------------------- set-up
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
        su32(&s.tmem)), "n"(2 * kBufCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  } else if (warp < kSumWarps) {
    // Q: the path's rows, D / 16 lanes each, 16 elements a lane
    constexpr int QL = D / 16;
    for (int x = tid; x < pad * QL; x += kSumWarps * 32) {  // (whole warps)
      const int n = x / QL, c = x % QL;
      uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      float nl = -INFINITY;
      if (n < ncol) {
        const long row = ((long)b * a.R + s.path.rows[n / a.g]) * a.Hq + hk * a.g + n % a.g;
        const uint4* qp = (const uint4*)((const __nv_bfloat16*)a.q + row * D) + 2 * c;
        w[0] = __ldg(qp);
        w[1] = __ldg(qp + 1);
        if (c == 0) nl = -a.lse[row] * kLog2e;
      }
      if constexpr (kQ8) {
        uint32_t top = top_of(top_pairs(top_pairs(0u, w[0]), w[1]));
#pragma unroll
        for (int o = QL / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
        const bool bad = top >= 0x7f800000u;
        const int e = row_exponent(top);
        uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
        if (!bad) split16(w, q8_scale(261 - e), hi, lo);
        *(uint4*)(smem + off_q + unit_offset<D>(n, c)) = hi;
        *(uint4*)(smem + off_q + q_bytes + unit_offset<D>(n, c)) = lo;
        if (c == 0) s.f[n] = bad ? __int_as_float(0x7fffffff) : a.qscale * q8_scale(e - 7);
      } else {
        // two boxes of 64 dims (D = 128), 128-byte swizzle
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int u = 2 * c + i;
          *(uint4*)(smem + off_q + (u >> 3) * (p.cols * 128u) + n * 128u + (((u & 7) ^ (n & 7)) << 4)) = w[i];
        }
        if (c == 0) s.f[n] = a.qscale;
      }
      if (c == 0) s.nl[n] = nl;
    }
    if (with_path) {
      // the path's rows as tile 0 (rows behind them: whatever was there, not used)
      for (int x = tid; x < 32 * QL; x += kSumWarps * 32) {
        const int j = x / QL, c = x % QL;
        uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (j <= L) {
          const uint4* kp = (const uint4*)((const __nv_bfloat16*)a.kt +
                                           (((long)b * a.R + s.path.rows[j]) * a.map.Hkv + hk) * D) + 2 * c;
          w[0] = __ldg(kp);
          w[1] = __ldg(kp + 1);
        }
        if constexpr (kQ8) {
          uint32_t top = top_of(top_pairs(top_pairs(0u, w[0]), w[1]));
#pragma unroll
          for (int o = QL / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
          const bool bad = top >= 0x7f800000u;
          const int e = row_exponent(top);
          uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
          if (!bad) split16(w, q8_scale(261 - e), hi, lo);
          *(uint4*)(smem + unit_offset<D>(j, c)) = hi;
          *(uint4*)(smem + kTileBytes + unit_offset<D>(j, c)) = lo;
          if (c == 0) s.kt_out[j] = bad ? __int_as_float(0x7fffffff) : q8_scale(e - 7);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int u = 2 * c + i;
            *(uint4*)(smem + (u >> 3) * (kWeightKeys * 128u) + j * 128u + (((u & 7) ^ (j & 7)) << 4)) = w[i];
          }
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s.tmem;

  // -------------------------------------------------------------- K tiles
  if (warp == kTma) {
    if (lane == 0) {
      int loaded = early;
      for (int t = loaded; t < n_pre && !*abort; ++t) {
        const int g = slots0 + t;
        if (!wait_timed(bar(BAR_EMPTY + g % p.ring), (g / p.ring - 1) & 1)) {
          *abort = 1;
          break;
        }
        load_k(t);
        ++loaded;
      }
      // no copy may be in flight when the CTA leaves
      for (int g = max(slots0 + loaded - p.ring, slots0); g < slots0 + loaded; ++g)
        mbar_wait(bar(BAR_FULL + g % p.ring), (g / p.ring) & 1);
    }
    __syncwarp();
  }

  // ------------------------------------------------------------- products
  else if (warp == kMma) {
    const bool one = elect_one();
    // (the path's slots were written before the barrier: phase 0 of theirs is
    // completed here, so that later uses count from it)
    if (one && with_path)
      for (int j = 0; j < kPathSlots; ++j) mbar_arrive(bar(BAR_FULL + j));
    __syncwarp();
    bool ok = true;
    for (int i = 0; ok && i < ntiles; ++i) {
      const bool is_path = with_path && i == 0;
      const int g = is_path ? 0 : slots0 + i - (with_path ? 1 : 0), sl = g % p.ring;
      ok = wait_ready(bar(BAR_FULL + sl), (g / p.ring) & 1);
      for (int c = 0; c < chunks; ++c) {
        const int n = min(pad - c * kBufCols, kBufCols), buf = i & 1;
        // the buffer's scores of its item before have been read
        const int before = (i >> 1) * chunks + c;           // items of this buffer so far
        if (before > 0) ok = ok && wait_ready(bar(BAR_S_EMPTY + buf), (before - 1) & 1);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        fence_after();
        const uint32_t ts = tmem + (uint32_t)(buf * kBufCols);
        const uint32_t idesc = (1u << 4) | ((uint32_t)(n >> 3) << 17) |
                               ((uint32_t)(kWeightKeys >> 4) << 24) |
                               (kQ8 ? 0u : (1u << 7) | (1u << 10));         // bf16 operands
        if (one) {
          if constexpr (kQ8) {
            for (int kp = 0; kp < (is_path ? 2 : 1); ++kp) {
              const uint64_t kd = row_desc<D>(sbase + (is_path ? kp : sl) * kTileBytes);
#pragma unroll
              for (int part = 0; part < 2; ++part) {
                const uint64_t qd = row_desc<D>(sbase + off_q + part * q_bytes + c * kBufCols * kRowBytes);
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                  mma_f8(ts, kd + 2 * kk, qd + 2 * kk, idesc, kp + part + kk == 0 ? 0u : 1u);
              }
            }
          } else {
            const uint64_t kd = smem_desc(sbase + sl * kTileBytes, 16, 1024);
            const uint64_t qd = smem_desc(sbase + off_q + c * kBufCols * 128, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_f16(ts, kd + (((kk >> 2) * (kWeightKeys * 128u) + (kk & 3) * 32) >> 4),
                      qd + (((kk >> 2) * (p.cols * 128u) + (kk & 3) * 32) >> 4), idesc,
                      kk == 0 ? 0u : 1u);
          }
          mma_commit(bar(BAR_S_FULL + buf));
          if (c == chunks - 1) {
            mma_commit(bar(BAR_EMPTY + sl));
            if (is_path && kPathSlots == 2) mma_commit(bar(BAR_EMPTY + 1));
          }
        }
        __syncwarp();
      }
    }
    if (!ok) *abort = 1;
    // every product has completed once this commit lands
    if (one) mma_commit(bar(BAR_FINAL));
    __syncwarp();
    mbar_wait(bar(BAR_FINAL), 0);
    __syncwarp();
  }

  // ----------------------------------------------------------------- sums
  else {
    const int wg = warp >> 2, key = (warp & 3) * 32 + lane;
    const uint32_t src = tmem + (uint32_t)(wg * kBufCols) + ((uint32_t)((warp & 3) * 32) << 16);
    float* const acc = a.acc + head * a.map.cap;
    int done = 0;                                           // items of this buffer
    bool ok = true;
    // this lane's row of item i, its weight so far and its factor: requested an item
    // ahead of its scores
    auto place = [&](int i) {
      return with_path && i == 0 ? P + key : (t0 + i - (with_path ? 1 : 0)) * kWeightKeys + key;
    };
    float next_old = 0.f, next_ck = 1.f;
    auto request = [&](int i) {
      const bool is_path = with_path && i == 0;
      const int pos = place(i);
      const bool mine = i < ntiles && (is_path ? key <= L : pos < P);
      next_old = mine && !is_path ? acc[pos] : 0.f;
      if (kQ8) next_ck = !mine ? 1.f : is_path ? s.kt_out[key] : q8_scale(a.ke[a.map.block(b, hk, pos)]);
    };
    request(wg);
    for (int i = wg; ok && i < ntiles; i += 2) {
      const bool is_path = with_path && i == 0;
      const int pos = place(i);
      const bool mine = is_path ? key <= L : pos < P;
      const float old = next_old, ck = next_ck;
      request(i + 2);
      const int first = is_path ? key * a.g : 0;            // row i of the path sees rows j <= i
      const float2 ck2 = make_float2(ck, ck);
      float2 s0 = make_float2(0.f, 0.f), s1 = s0;
      for (int c = 0; c < chunks; ++c, ++done) {
        const int n = min(pad - c * kBufCols, kBufCols);
        if (!__all_sync(kFull, wait_ready(bar(BAR_S_FULL + wg), done & 1))) {
          ok = false;
          break;
        }
        fence_after();
        const float* const f = s.f + c * kBufCols;
        const float* const nl = s.nl + c * kBufCols;
#pragma unroll 1
        for (int j = 0; j < n; j += 16) {
          float v[16];
          tmem_ld8(src + j, v);
          tmem_ld8(src + j + 8, v + 8);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 16; x += 4) {
            const float4 f4 = *(const float4*)(f + j + x), l4 = *(const float4*)(nl + j + x);
            float2 fa = make_float2(f4.x, f4.y), fb = make_float2(f4.z, f4.w);
            if (kQ8) {
              fa = __fmul2_rn(fa, ck2);
              fb = __fmul2_rn(fb, ck2);
            }
            const float2 xa = __ffma2_rn(make_float2(v[x], v[x + 1]), fa, make_float2(l4.x, l4.y));
            const float2 xb = __ffma2_rn(make_float2(v[x + 2], v[x + 3]), fb, make_float2(l4.z, l4.w));
            float2 ea = make_float2(ex2(xa.x), ex2(xa.y)), eb = make_float2(ex2(xb.x), ex2(xb.y));
            if (is_path) {
              const int col = c * kBufCols + j + x;
              if (col < first) ea.x = 0.f;
              if (col + 1 < first) ea.y = 0.f;
              if (col + 2 < first) eb.x = 0.f;
              if (col + 3 < first) eb.y = 0.f;
            }
            s0 = __fadd2_rn(s0, ea);
            s1 = __fadd2_rn(s1, eb);
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_S_EMPTY + wg));
      }
      if (!ok || !mine) continue;
      const float sum = (s0.x + s0.y) + (s1.x + s1.y);
      if (is_path) {
        acc[pos] = sum;
        a.pos[head * a.map.cap + pos] = a.seen[head] + key;
      } else {
        acc[pos] = fmaf(a.decay, old, sum);
      }
    }
    if (!ok && lane == 0) *abort = 1;
  }

  // --------------------------------------------------------------- teardown
  fence_before();
  __syncthreads();                                          // (`seen` has been read)
  if (tid == 0) {
    if (*abort) report_error(a.err, TSD_DEV_ERR_TIMEOUT, b);
    else if (with_path) a.seen[head] += L + 1;
  }
  fence_after();
  if (warp == kMma) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem),
                 "n"(2 * kBufCols));
  }
}

// K rows as (dims, rows of a head, heads) in boxes of 128 rows: codes whole, bf16
// in halves of 64 dims.
bool encode_cache(CUtensorMap* m, const WeightArgs& a, int B, int D, bool q8) {
  const long rows = a.map.page_size > 0 ? a.map.page_size : a.map.cap;
  const long heads = (a.map.page_size > 0 ? (long)a.map.num_pages : (long)B) * a.map.Hkv;
  if (heads > 0x7fffffffl) return false;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  if (q8) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)heads};
    const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)rows * D};
    const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)kWeightKeys, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(a.k), dims, strides, box,
                       es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)heads, (cuuint64_t)(D / 64)};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)rows * D * 2, 128};
  const cuuint32_t box[4] = {64, (cuuint32_t)kWeightKeys, 1, (cuuint32_t)(D / 64)};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.k), dims, strides,
                     box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kQ8, int kBufCols>
bool launch_d(const tsd_attn_desc& d, const WeightArgs& a, int cols, cudaStream_t st) {
  CUtensorMap m;
  if (!encode_cache(&m, a, d.B, D, kQ8)) return false;
  constexpr int kPerSm = kBufCols == 128 ? 2 : 1;
  constexpr long kSmem = 220 * 1024 / kPerSm;
  WeightPlan p{};
  p.cols = cols;
  const long tile = kWeightKeys * D * (kQ8 ? 1 : 2), q = (long)cols * D * 2;
  p.ring = (int)((kSmem - q - (long)sizeof(WeightSmem) - 1024) / tile);
  if (p.ring > kMaxRing) p.ring = kMaxRing;
  // Splits as for the attention: waves of CTAs times (tiles of a CTA and about six
  // more for its set-up).
  const long units = (long)d.B * d.Hkv, tiles = ceil_div(d.cap, kWeightKeys);
  long best = -1;
  for (long n = 1; n <= 64 && n <= tiles; ++n) {
    const long per = ceil_div(tiles, n);
    const long cost = ceil_div(units * ceil_div(tiles, per), 152L * kPerSm) * (per + 6);
    if (best < 0 || cost < best) { best = cost; p.tiles = (int)per; }
  }
  p.nsplit = (int)ceil_div(tiles, p.tiles);
  const size_t smem = (size_t)p.ring * tile + q + sizeof(WeightSmem) + 1024;
  const auto kern = a.wait_cycles < kWaitCycles ? weights_tc_kernel<D, kQ8, kBufCols, true>
                                                : weights_tc_kernel<D, kQ8, kBufCols, false>;
  // (the same for every call: another thread's may come between this and the launch)
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  launch(kern, dim3(p.nsplit, d.Hkv, d.B), dim3(kThreads), smem, st, m, a, p);
  return true;
}

template <int D, bool kQ8>
bool launch_cols(const tsd_attn_desc& d, const WeightArgs& a, cudaStream_t st) {
  const int cols = (int)ceil_div((long)(a.S + 1) * a.g, 16) * 16;
  // Up to 128 columns two CTAs share an SM: score buffers of 128 columns, half the
  // ring.  (32 requests of 1k to 4k 8-bit rows, 32 columns: 40 us in a graph so, 54 us
  // with one; 4 x 32k bf16 rows, 36 columns: 61 and 65 us.)
  return cols <= 128 ? launch_d<D, kQ8, 128>(d, a, cols, st) : launch_d<D, kQ8, 256>(d, a, cols, st);
}

}  // namespace

bool launch_weights_tc(const tsd_attn_desc& d, const WeightArgs& a, cudaStream_t st) {
  if (d.dtype != TSD_BF16 || (d.dk != 64 && d.dk != 128)) return false;
  if ((long)(a.S + 1) * a.g > kMaxCols || encode_fn() == nullptr) return false;
  if (d.dk == 128)
    return a.ke != nullptr ? launch_cols<128, true>(d, a, st) : launch_cols<128, false>(d, a, st);
  return a.ke != nullptr ? launch_cols<64, true>(d, a, st) : launch_cols<64, false>(d, a, st);
}

}  // namespace tsd
