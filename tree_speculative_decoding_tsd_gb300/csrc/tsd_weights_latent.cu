// tcgen05 path of tsd_cache_weights(_q8) for bf16 latent heads: rows of 576 dims,
// up to 2176 columns (path rows x query heads).
//
//   S^T[key][n] = K_tile . Q^T    M = 128 keys, N = 64 columns at a time, K = 576
//   acc[key]    = decay * acc[key] + sum_n 2^(S^T qscale - lse_n)
// A CTA owns 128 cached rows (or the path's own rows) and runs over all columns, so
// a row's sum stays with one thread per warpgroup and no two CTAs add to the same
// place.  The K tile is loaded once and kept in shared memory as bf16 (144 KB); Q
// comes through a ring of nine pieces of 64 columns x 64 dims (72 KB), every CTA of
// a request reading the same ones from L2.  Codes are widened to bf16 when the tile
// is loaded: code * 2^(e - 127) has 4 significant bits and is exact, and the
// tile serves up to 34 groups of columns.
//
// Bound by the tensor core: 36 products of 128 x 64 x 16 per group of columns, 48
// cycles each, against 512 cycles of exponentials in each of two warpgroups that take
// the groups in turn; and by the load of 144 KB that no other CTA on the SM covers (the
// tensor core is 19% active, 13% from codes).  16 requests of 4.5k rows, up to 5 path rows
// of 128 heads: 91 us from bf16 rows, 128 us from codes.
//
// Roles (320 threads): warps 0-7 widen or gather the tile, then sum; warp 8 issues
// the products, one thread of warp 9 loads.  Every wait is bounded.
#include "tsd_host.h"
#include "tsd_q8_tc.cuh"
#include "tsd_weights.cuh"

namespace tsd {
namespace {

constexpr int kDim = 576, kPieces = 9, kCols = 64, kMaxCols = kMaxPath * 128;
constexpr int kSumWarps = 8, kMma = 8, kTma = 9, kThreads = 10 * 32;
constexpr uint32_t kPieceK = kWeightKeys * 128, kPieceQ = kCols * 128;
constexpr uint32_t kTileK = kPieces * kPieceK;

struct LatentSmem {
  float nl[kMaxCols];            // -log2(e) lse (-inf behind the last column)
  float half[kWeightKeys];       // the second warpgroup's sums
  uint64_t bars[2 * kPieces + 6];
  uint32_t tmem, abort;
  PathSmem path;
};
constexpr uint32_t kOffQ = kTileK, kOffMisc = kOffQ + kPieces * kPieceQ;
constexpr uint32_t kTotal = kOffMisc + sizeof(LatentSmem);
static_assert(kTotal + 1024 <= 232448, "shared memory budget");

enum { BAR_Q_FULL = 0, BAR_Q_EMPTY = kPieces, BAR_S_FULL = 2 * kPieces, BAR_S_EMPTY = BAR_S_FULL + 2,
       BAR_K_FULL = BAR_S_EMPTY + 2, BAR_FINAL = BAR_K_FULL + 1 };

template <bool kQ8, bool kPoll>
__global__ void __launch_bounds__(kThreads, 1)
weights_latent_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ WeightArgs a) {
  if (threadIdx.x == kTma * 32) {
    tma_desc_prefetch(&qmap);
    if (!kQ8) tma_desc_prefetch(&kmap);
  }
  grid_dependency_sync();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = su32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  LatentSmem& s = *(LatentSmem*)(smem + kOffMisc);
  volatile uint32_t* abort = &s.abort;
  auto bar = [&](int i) { return su32(&s.bars[i]); };
  auto wait_ready = [&](uint32_t at, uint32_t parity) {
    return phase_ready<kPoll>(at, parity, a.wait_cycles);
  };
  auto wait_timed = [&](uint32_t at, uint32_t parity) {
    return phase_timed<kPoll>(at, parity, a.wait_cycles);
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int P = a.plen[b];
  const bool on_path = blockIdx.x == gridDim.x - 1;
  const int k0 = blockIdx.x * kWeightKeys;
  if (!on_path && k0 >= P) return;
  const int L = weight_path(a, b, P, s.path);
  if (L < 0) {                                              // the whole request is skipped
    if (on_path && tid == 0) report_error(a.err, -L, b);
    return;
  }
  if (s.path.blind) {
    if (on_path) unweighed_path(a, b, hk, P, L);
    return;
  }
  const int nkeys = on_path ? L + 1 : min(kWeightKeys, P - k0);
  const int ncol = (L + 1) * a.g, groups = (ncol + kCols - 1) / kCols;
  const long head = (long)b * a.map.Hkv + hk;

  // ---------------------------------------------------------------- set-up
  // piece j of column group n into the ring: runs of min(g, 64) columns are rows of
  // Q that follow one another (columns behind the last one repeat its path row)
  auto load_q = [&](int n, int j) {
    mbar_expect_tx(bar(BAR_Q_FULL + j), kPieceQ);
    const int run = min(a.g, kCols);
    for (int c = 0; c < kCols; c += run) {
      const int col = n * kCols + c;
      const long row = ((long)b * a.R + s.path.rows[min(col / a.g, L)]) * a.Hq + hk * a.g + col % a.g;
      tma_2d(sbase + kOffQ + j * kPieceQ + c * 128, &qmap, 64 * j, (int)row, bar(BAR_Q_FULL + j));
    }
  };
  if (warp == kTma) {
    if (lane == 0) {
      for (int i = 0; i < kPieces; ++i) {
        mbar_init(bar(BAR_Q_FULL + i), 1);
        mbar_init(bar(BAR_Q_EMPTY + i), 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(BAR_S_FULL + i), 1);
        mbar_init(bar(BAR_S_EMPTY + i), 4);
      }
      mbar_init(bar(BAR_K_FULL), 1);
      mbar_init(bar(BAR_FINAL), 1);
      *abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
      if (!kQ8 && !on_path) {
        int y = k0, z = (int)head;
        if (a.map.page_size) {
          const long r = a.map.row(b, hk, k0);              // (checked by weight_path)
          y = (int)(r % a.map.page_size);
          z = (int)(r / a.map.page_size);
        }
        mbar_expect_tx(bar(BAR_K_FULL), kTileK);
        for (int j = 0; j < kPieces; j += 3)
          tma_4d(sbase + j * kPieceK, &kmap, 0, y, z, j, bar(BAR_K_FULL));
      }
      for (int j = 0; j < kPieces; ++j) load_q(0, j);
    }
    __syncwarp();
  } else if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;\n" ::"r"(
        su32(&s.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  } else {
    for (int n = tid; n < groups * kCols; n += kSumWarps * 32) {
      float nl = -INFINITY;
      if (n < ncol)
        nl = -a.lse[((long)b * a.R + s.path.rows[n / a.g]) * a.Hq + hk * a.g + n % a.g] * kLog2e;
      s.nl[n] = nl;
    }
    if (on_path) {
      // the path's rows (what is behind them is not used)
      for (int x = tid; x < (L + 1) * (kDim / 8); x += kSumWarps * 32) {
        const int r = x / (kDim / 8), u = x % (kDim / 8);
        const uint4 w = __ldg((const uint4*)((const __nv_bfloat16*)a.kt +
                                             (((long)b * a.R + s.path.rows[r]) * a.map.Hkv + hk) * kDim) + u);
        *(uint4*)(smem + (u >> 3) * kPieceK + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = w;
      }
    } else if (kQ8) {
      const long row0 = a.map.row(b, hk, k0);
      const long e0 = a.map.block_at(b, hk, k0, row0);
      const float f0 = q8_scale(a.ke[e0]);
      const float f1 = nkeys > kQ8Block ? q8_scale(a.ke[e0 + 1]) : 0.f;
      const uint8_t* const codes = (const uint8_t*)a.k + row0 * kDim;
#pragma unroll 4
      for (int x = tid; x < kWeightKeys * (kDim / 16); x += kSumWarps * 32) {
        const int r = x / (kDim / 16), c = x % (kDim / 16);
        if (r >= nkeys) break;
        const uint4 w = ld_stream(codes + (long)x * 16);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
        const float f = r < kQ8Block ? f0 : f1;
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y[4];
          q8_unpack4(v[i], y);
          o[2 * i] = pack_bf16x2(y[0] * f, y[1] * f);
          o[2 * i + 1] = pack_bf16x2(y[2] * f, y[3] * f);
        }
        uint8_t* const d = smem + (c >> 2) * kPieceK + r * 128;
        const int u = 2 * (c & 3);
        *(uint4*)(d + ((u ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *(uint4*)(d + (((u + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s.tmem;

  // ------------------------------------------------------------- Q pieces
  if (warp == kTma) {
    if (lane == 0) {
      // the first piece not requested: piece j of group n
      int n = 1, j = 0;
      while (n < groups && !*abort) {
        if (!wait_timed(bar(BAR_Q_EMPTY + j), (n - 1) & 1)) {
          *abort = 1;
          break;
        }
        load_q(n, j);
        if (++j == kPieces) {
          j = 0;
          ++n;
        }
      }
      // no copy may be in flight when the CTA leaves
      for (int i = 0; i < kPieces; ++i) mbar_wait(bar(BAR_Q_FULL + i), (i < j ? n : n - 1) & 1);
      if (!kQ8 && !on_path) mbar_wait(bar(BAR_K_FULL), 0);
    }
    __syncwarp();
  }

  // ------------------------------------------------------------- products
  else if (warp == kMma) {
    constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kCols >> 3) << 17) |
                               ((uint32_t)(kWeightKeys >> 4) << 24);
    const uint64_t kd0 = smem_desc(sbase, 16, 1024), qd0 = smem_desc(sbase + kOffQ, 16, 1024);
    const bool one = elect_one();
    bool ok = kQ8 || on_path || wait_ready(bar(BAR_K_FULL), 0);
    for (int n = 0; ok && n < groups; ++n) {
      const int buf = n & 1;
      const uint32_t ts = tmem + (uint32_t)(buf * kCols);
      if (n >= 2) ok = wait_ready(bar(BAR_S_EMPTY + buf), ((n - 2) >> 1) & 1);
#pragma unroll 1
      for (int j = 0; j < kPieces; ++j) {
        ok = ok && wait_ready(bar(BAR_Q_FULL + j), n & 1);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        fence_after();
        const uint64_t kd = kd0 + (uint64_t)(j * (kPieceK >> 4)), qd = qd0 + (uint64_t)(j * (kPieceQ >> 4));
        if (one) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16(ts, kd + 2 * kk, qd + 2 * kk, idesc, j + kk == 0 ? 0u : 1u);
          mma_commit(bar(BAR_Q_EMPTY + j));
          if (j == kPieces - 1) mma_commit(bar(BAR_S_FULL + buf));
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
    const uint32_t src = tmem + (uint32_t)(wg * kCols) + ((uint32_t)((warp & 3) * 32) << 16);
    float* const acc = a.acc + head * a.map.cap;
    const bool mine = key < nkeys;
    const float old = wg == 0 && mine && !on_path ? acc[k0 + key] : 0.f;
    const int first = on_path ? key * a.g : 0;              // row i of the path sees rows j <= i
    const float2 f2 = make_float2(a.qscale, a.qscale);
    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
    bool ok = true;
    for (int n = wg; n < groups; n += 2) {
      if (!__all_sync(kFull, wait_ready(bar(BAR_S_FULL + wg), (n >> 1) & 1))) {
        ok = false;
        break;
      }
      fence_after();
      const float* const nl = s.nl + n * kCols;
#pragma unroll 2
      for (int j = 0; j < kCols; j += 16) {
        float v[16];
        tmem_ld8(src + j, v);
        tmem_ld8(src + j + 8, v + 8);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 16; x += 4) {
          const float4 l4 = *(const float4*)(nl + j + x);
          const float2 xa = __ffma2_rn(make_float2(v[x], v[x + 1]), f2, make_float2(l4.x, l4.y));
          const float2 xb = __ffma2_rn(make_float2(v[x + 2], v[x + 3]), f2, make_float2(l4.z, l4.w));
          float2 ea = make_float2(ex2(xa.x), ex2(xa.y)), eb = make_float2(ex2(xb.x), ex2(xb.y));
          if (on_path) {
            const int col = n * kCols + j + x;
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
    if (!ok && lane == 0) *abort = 1;
    const float sum = (s0.x + s0.y) + (s1.x + s1.y);
    if (wg == 1) s.half[key] = sum;
    asm volatile("bar.sync 1, 256;\n" ::: "memory");
    if (wg == 0 && mine && ok && *abort == 0) {
      const float all = sum + s.half[key];
      if (on_path) {
        acc[P + key] = all;
        a.pos[head * a.map.cap + P + key] = a.seen[head] + key;
      } else {
        acc[k0 + key] = fmaf(a.decay, old, all);
      }
    }
  }

  // --------------------------------------------------------------- teardown
  fence_before();
  __syncthreads();                                          // (`seen` has been read)
  if (tid == 0) {
    if (*abort) report_error(a.err, TSD_DEV_ERR_TIMEOUT, b);
    else if (on_path) a.seen[head] += L + 1;
  }
  fence_after();
  if (warp == kMma) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;\n" ::"r"(tmem));
  }
}

bool encode_latent(CUtensorMap* m, const WeightArgs& a, int B) {
  const long rows = a.map.page_size > 0 ? a.map.page_size : a.map.cap;
  const long heads = (a.map.page_size > 0 ? (long)a.map.num_pages : (long)B) * a.map.Hkv;
  if (heads > 0x7fffffffl) return false;
  const cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)heads, (cuuint64_t)kPieces};
  const cuuint64_t strides[3] = {(cuuint64_t)kDim * 2, (cuuint64_t)rows * kDim * 2, 128};
  const cuuint32_t box[4] = {64, (cuuint32_t)kWeightKeys, 1, 3};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.k), dims, strides,
                     box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_queries(CUtensorMap* m, const WeightArgs& a, int B) {
  const long rows = (long)B * a.R * a.Hq;
  if (rows > 0x7fffffffl) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kDim, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kDim * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)(a.g < kCols ? a.g : kCols)};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(a.q), dims, strides,
                     box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kQ8>
bool launch_latent(const tsd_attn_desc& d, const WeightArgs& a, cudaStream_t st) {
  CUtensorMap k, q;
  if (!encode_queries(&q, a, d.B)) return false;
  if (kQ8) k = q;                                           // (not used)
  else if (!encode_latent(&k, a, d.B)) return false;
  const auto kern = a.wait_cycles < kWaitCycles ? weights_latent_kernel<kQ8, true>
                                                : weights_latent_kernel<kQ8, false>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTotal + 1024);
  const dim3 grid((unsigned)ceil_div(d.cap, kWeightKeys) + 1, d.Hkv, d.B);
  launch(kern, grid, dim3(kThreads), kTotal + 1024, st, k, q, a);
  return true;
}

}  // namespace

bool launch_weights_latent(const tsd_attn_desc& d, const WeightArgs& a, cudaStream_t st) {
  if (d.dtype != TSD_BF16 || d.dk != kDim || encode_fn() == nullptr) return false;
  // a group of 64 columns is made of whole runs of a path row's heads (8 rows of a
  // swizzle pattern each, at least)
  if ((long)(a.S + 1) * a.g > kMaxCols || a.g % 8 != 0 || (a.g % kCols != 0 && kCols % a.g != 0)) return false;
  return a.ke != nullptr ? launch_latent<true>(d, a, st) : launch_latent<false>(d, a, st);
}

}  // namespace tsd
