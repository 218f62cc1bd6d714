// tcgen05 path of tsd_tree_verify_attn_q8 for bf16 latent heads: one KV head of 576
// dims whose rows are the keys and whose first 512 dims are the values, shared by
// all query heads.
//
// Products, transposed (packed query rows on the MMA's columns, 64 per CTA):
//   S^T[key][hi n | lo n] = K_tile . [Q hi | Q lo]^T   M = 128 keys, N = 128, K = 576
//   O^T[dim][n] += V_tile^T . P^T                      4 x M = 128 dims, N = 64, K = 128 keys
//
// Numbers as in tsd_q8_tc.cu: the scores from the codes as they are in the cache
// and Q as the sum of two e4m3 numbers (here side by side on the columns, so that a
// K tile is read once for both; the softmax adds them), V widened to fp16, P rounded
// to fp16, the powers of two applied to scores and probabilities in fp32.
//
// Why 64 rows and codes for the keys: the tensor memory holds O^T of 512 x 64 (256
// columns) beside two score buffers (2 x 128).  Per 128-key tile the codes arrive in
// shared memory (72 KB), the 18 products of S^T read 8 KB each, the widened values are
// written (128 KB) and the 32 products of O^T read 6 KB each: 536 KB, about 4200 cycles
// if all of it shares 128 bytes a cycle; a tile takes 5200.  (Widened keys would be 144
// KB written and 216 KB read instead of the 216 KB.)  The counters show 36% for the
// warps' own accesses, without the products' reads, and the tensor core 40% active: a
// tile's latency through the roles may bind as well.  64 x 9 rows of 128 heads over 8k
// keys: 1.51 ms, 870 TFLOP/s.
//
// Roles (768 threads): warps 0-15 softmax and epilogue (warpgroup w/4 owns 16
// columns, warp w%4 the TMEM lanes 32(w%4)..+31); warp 16 issues the products of
// S^T and owns the tensor memory, warp 17 those of O^T; one thread of warp 18 loads
// pieces of 128 dims of a K tile by TMA into a ring of three; warps 19-23 load V
// (the first 512 dims again, from L2) into registers and widen it, 128 dims at a
// time, into two stages.  P^T has two buffers.  Every wait is bounded.
#include <type_traits>

#include "tsd_common.cuh"
#include "tsd_host.h"
#include "tsd_q8_tc.cuh"

namespace tsd {
namespace {

constexpr int kDK = 576, kDV = 512, kN = 64;
constexpr int kPieces = 5;                      // of a K tile: four of 128 dims, one of 64
constexpr int kUnits = kDV / 128;               // V boxes (O^T M-tiles) of a tile
constexpr int kSlots = 3;                       // K ring
constexpr int kWG = 4, kNH = kN / kWG;
constexpr int kSoftWarps = 16, kQk = 16, kPv = 17, kTma = 18, kWide = 19, kWideWarps = 5;
constexpr int kWideThreads = kWideWarps * 32;
constexpr int kThreads = (kWide + kWideWarps) * 32;
constexpr uint32_t kPiece = kKeys * 128;        // 16 KB
constexpr uint32_t kPtBytes = 256u * kN;

constexpr uint32_t kOffK = 0;                                   // ring of K pieces
constexpr uint32_t kOffV = kOffK + kSlots * kPiece;             // two boxes [2][128 keys][64]
constexpr uint32_t kOffQ = kOffV + 2 * kTile;                   // 4 x [128][128] + [128][64] e4m3
constexpr uint32_t kOffP = kOffQ + 4 * kPiece + kPiece / 2;
constexpr uint32_t kOffM = kOffP + 2 * kPtBytes;                // float[N] each
constexpr uint32_t kOffAlpha = kOffM + 4 * kN;
constexpr uint32_t kOffNegm = kOffAlpha + 4 * kN;
constexpr uint32_t kOffShift = kOffNegm + 4 * kN;
constexpr uint32_t kOffC2 = kOffShift + 4 * kN;
constexpr uint32_t kOffRed = kOffC2 + 4 * kN;                   // float[16][NH]
constexpr uint32_t kOffRmask = kOffRed + 4 * kSoftWarps * kNH;  // u64[N]
constexpr uint32_t kOffOoff = kOffRmask + 8 * kN;               // i64[N]
constexpr uint32_t kOffRows = kOffOoff + 8 * kN;                // i64[kMaxTiles]
constexpr uint32_t kOffTree = kOffRows + 8 * kMaxTiles;         // 4 x 32 bits [128]
constexpr uint32_t kOffKex = kOffTree + 16 * kKeys;             // u8[2 kMaxTiles]
constexpr uint32_t kOffBar = kOffKex + 2 * kMaxTiles;
constexpr int kBars = 22;
constexpr uint32_t kOffFlags = kOffBar + 8 * kBars;             // tmem, abort
constexpr uint32_t kOffTop = kOffFlags + 8;
constexpr uint32_t kOffReq = kOffTop + 4 * kWideWarps;           // request, its length
constexpr uint32_t kTotal = kOffReq + 8;
static_assert(kTotal + 1024 <= 232448, "shared memory budget");

// FULL: the copy landed or the warps wrote (T_FULL: scratch rows' keys, through
// the same slots); EMPTY: read by the product.  PV_DONE: per P^T buffer.
enum { BAR_K_FULL = 0, BAR_K_EMPTY = 3, BAR_T_FULL = 6, BAR_V_FULL = 9, BAR_V_EMPTY = 11,
       BAR_S_FULL = 13, BAR_P_FULL = 15, BAR_PV_DONE = 17, BAR_O_DONE = 19, BAR_FINAL = 20 };

struct LatentMaps {
  CUtensorMap wide, last;     // K codes in boxes of 128 and of 64 dims
};

// Byte offset of 16-element unit u (0..35) of row r in a tile of pieces.
__device__ __forceinline__ uint32_t piece_offset(int r, int u) {
  return u < 32 ? (u >> 3) * kPiece + unit_offset<128>(r, u & 7)
                : 4 * kPiece + unit_offset<64>(r, u - 32);
}

template <bool kPoll>
__global__ void __launch_bounds__(kThreads, 1)
q8_latent_kernel(const __grid_constant__ LatentMaps maps, const __grid_constant__ Q8AttnArgs a) {
  if (threadIdx.x == kTma * 32) {
    tma_desc_prefetch(&maps.wide);
    tma_desc_prefetch(&maps.last);
  }
  grid_dependency_sync();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = su32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  float* m_run = (float*)(smem + kOffM);
  float* alpha = (float*)(smem + kOffAlpha);
  float* negm = (float*)(smem + kOffNegm);
  float* shiftv = (float*)(smem + kOffShift);
  float* c2v = (float*)(smem + kOffC2);
  float* red = (float*)(smem + kOffRed);
  uint64_t* rmask = (uint64_t*)(smem + kOffRmask);
  long long* ooff = (long long*)(smem + kOffOoff);
  long long* tile_row = (long long*)(smem + kOffRows);
  float* kt_in = (float*)(smem + kOffTree);
  float* vt_in = kt_in + kKeys;
  float* kt_out = vt_in + kKeys;
  int* vt_u = (int*)(kt_out + kKeys);
  uint8_t* kex = smem + kOffKex;
  volatile uint32_t* flags = (volatile uint32_t*)(smem + kOffFlags);
  int* s_top = (int*)(smem + kOffTop);
  const uint32_t bar0 = sbase + kOffBar;
  auto bar = [&](int i) { return bar0 + 8u * i; };
  auto wait_ready = [&](uint32_t at, uint32_t parity) {
    return phase_ready<kPoll>(at, parity, a.wait_cycles);
  };
  auto wait_timed = [&](uint32_t at, uint32_t parity) {
    return phase_timed<kPoll>(at, parity, a.wait_cycles);
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.y / a.nrg, rg = blockIdx.y % a.nrg, sp = blockIdx.x;
  int P;
  const int b = request_at(a, blockIdx.z, P, (volatile int*)(smem + kOffReq));
  const int nsb = q8_splits(a, P);
  if (sp >= nsb) return;
  const int k0 = q8_first(a, P, sp), k1 = q8_end(a, P, k0);
  const int n_pre = (k1 - k0 + kKeys - 1) / kKeys;
  const bool with_tree = sp == nsb - 1;
  const int ntiles = n_pre + (with_tree ? 1 : 0);
  const int row_base = rg * kN;
  const int rows_here = min(kN, a.M - row_base);
  auto valid_of = [&](int t) { return min(kKeys, k1 - (k0 + t * kKeys)); };
  auto tree_row = [&](int j) {                       // scratch row j
    return (const uint4*)((const __nv_bfloat16*)a.kt + (((long)b * a.R + j) * a.map.Hkv + hk) * kDK);
  };

  const int wt = tid - kWide * 32;
  using Share = WideShare<8, kWideThreads>;
  const Share share(wt);
  uint4 vreg[Share::kCount];
  // 128 dims from 128 u of the tile at cache row `row` (a missing page: none)
  auto load_v = [&](long row, int nvalid, int u) {
    share.load<kDK>(vreg, a.kc + (row < 0 ? 0 : row) * kDK + u * 128, row < 0 ? 0 : nvalid);
  };
  // K piece g (piece g % 5 of tile g / 5) by TMA into slot g % 3
  auto load_piece = [&](int g, long long row) {
    const int t = g / kPieces, j = g - t * kPieces, sl = g % kSlots;
    int y = k0 + t * kKeys, z = b * a.map.Hkv + hk;
    if (a.map.page_size) {
      y = (int)((uint32_t)y % (uint32_t)a.map.page_size);
      z = row < 0 ? 0 : quotient(row - y, a.map.page_size);
    }
    const uint32_t dst = sbase + kOffK + sl * kPiece, full = bar(BAR_K_FULL + sl);
    mbar_expect_tx(full, j < 4 ? kPiece : kPiece / 2);
    if (j < 4) tma_3d(dst, &maps.wide, 128 * j, y, z, full);
    else tma_3d(dst, &maps.last, 512, y, z, full);
  };

  // ---------------------------------------------------------------- set-up
  if (warp >= kWide) {
    const long r0 = n_pre > 0 ? a.map.row(b, hk, k0) : -1;
    if (n_pre > 0) load_v(r0, valid_of(0), 0);
    int top = -1000;
#pragma unroll 1
    for (int t = wt; t < n_pre; t += kWideThreads) {
      const int pos = k0 + t * kKeys;
      const long r = a.map.row(b, hk, pos);
      tile_row[t] = r;
      if (r < 0) report_error(a.err, TSD_DEV_ERR_BAD_PAGE, b);
      const long e = a.map.block_at(b, hk, pos, r);
      const int ka = r < 0 ? 127 : a.ke[e];
      const int kb = r < 0 || pos + kQ8Block >= k1 ? ka : a.ke[e + 1];
      kex[2 * t] = (uint8_t)ka;
      kex[2 * t + 1] = (uint8_t)kb;
      top = max(top, max(ka, kb) - 127);
    }
    if (with_tree) {
      // a warp per scratch row: its largest element (K), and that of its first 512
      // dims (V); which rows some row sees
      uint32_t lo = 0, hi = 0;
      for (int r = lane; r < a.R; r += 32) {
        const uint64_t m = r > 0 ? a.mask[(long)b * a.R + r] : 0ull;
        lo |= (uint32_t)m;
        hi |= (uint32_t)(m >> 32);
      }
      lo = __reduce_or_sync(kFull, lo);
      hi = __reduce_or_sync(kFull, hi);
      const uint64_t seen = ((uint64_t)hi << 32) | lo;
#pragma unroll 2
      for (int j = warp - kWide; j < kKeys; j += kWideWarps) {
        const bool live = j < a.R && (j == 0 || ((seen >> (j - 1)) & 1ull));
        uint32_t kt = 0, vt = 0;
        if (live) {
          const uint4* p = tree_row(j);
          vt = top_pairs(top_pairs(0u, __ldg(p + lane)), __ldg(p + 32 + lane));
          kt = lane < 8 ? top_pairs(vt, __ldg(p + 64 + lane)) : vt;
        }
        kt = __reduce_max_sync(kFull, top_of(kt));
        vt = __reduce_max_sync(kFull, top_of(vt));
        const bool bad = kt >= 0x7f800000u;
        const int ek = row_exponent(kt), ev = row_exponent(vt);
        if (lane == 0) {
          kt_in[j] = live && !bad ? q8_scale(261 - ek) : 0.f;
          vt_in[j] = live && !bad ? q8_scale(262 - ev) : 0.f;
          kt_out[j] = bad ? __int_as_float(0x7fffffff) : q8_scale(ek - 7);
          vt_u[j] = live && !bad ? ev - 135 : -900;
        }
        if (live && !bad) top = max(top, ev - 135);
      }
    }
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) s_top[warp - kWide] = top;
  } else if (warp < kSoftWarps) {
    // Q as hi (row n) and lo (row 64 + n) of one operand: a warp per row
#pragma unroll 2
    for (int n = warp; n < kN; n += kSoftWarps) {
      uint4 w[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (n < rows_here) {
        const int p = row_base + n;
        const int tr = p / a.g, qh = hk * a.g + p % a.g;
        const uint4* qp = (const uint4*)((const __nv_bfloat16*)a.q + (((long)b * a.R + tr) * a.Hq + qh) * kDK);
        w[0][0] = __ldg(qp + 2 * lane);
        w[0][1] = __ldg(qp + 2 * lane + 1);
        if (lane < 4) {
          w[1][0] = __ldg(qp + 64 + 2 * lane);
          w[1][1] = __ldg(qp + 64 + 2 * lane + 1);
        }
      }
      uint32_t top = top_pairs(top_pairs(0u, w[0][0]), w[0][1]);
      top = top_of(top_pairs(top_pairs(top, w[1][0]), w[1][1]));
      top = __reduce_max_sync(kFull, top);
      const bool bad = top >= 0x7f800000u;
      const int e = row_exponent(top);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int u = i == 0 ? lane : 32 + lane;
        if (i == 1 && lane >= 4) break;
        uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
        if (!bad) split16(w[i], q8_scale(261 - e), hi, lo);
        *(uint4*)(smem + kOffQ + piece_offset(n, u)) = hi;
        *(uint4*)(smem + kOffQ + piece_offset(kN + n, u)) = lo;
      }
      if (lane == 0) c2v[n] = bad ? __int_as_float(0x7fffffff) : a.qscale * q8_scale(e - 7);
    }
    for (int n = tid; n < kN; n += kSoftWarps * 32) {
      uint64_t mk = 0ull;
      if (n < rows_here) {
        const int tr = (row_base + n) / a.g;
        mk = tr > 0 ? a.mask[(long)b * a.R + tr] : 0ull;
      }
      rmask[n] = mk;
      m_run[n] = -INFINITY;
      negm[n] = 0.f;
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  } else if (warp == kTma) {
    if (lane == 0) {
      for (int i = 0; i < kSlots; ++i) {
        mbar_init(bar(BAR_K_FULL + i), 1);
        mbar_init(bar(BAR_K_EMPTY + i), 1);
        mbar_init(bar(BAR_T_FULL + i), kWideWarps);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(BAR_V_FULL + i), kWideWarps);
        mbar_init(bar(BAR_V_EMPTY + i), 1);
        mbar_init(bar(BAR_S_FULL + i), 1);
        mbar_init(bar(BAR_P_FULL + i), kSoftWarps);
        mbar_init(bar(BAR_PV_DONE + i), 1);
        mbar_init(bar(BAR_FINAL + i), 1);
      }
      mbar_init(bar(BAR_O_DONE), 1);
      flags[1] = 0;
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
      const long long r0 = a.map.page_size && n_pre > 0 ? a.map.row(b, hk, k0) : 0;
      for (int g = 0; g < kSlots && g < kPieces * n_pre; ++g) load_piece(g, r0);
    }
    __syncwarp();
  } else if (warp == kQk) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
        sbase + kOffFlags));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = flags[0];
  int U = s_top[0];
#pragma unroll
  for (int i = 1; i < kWideWarps; ++i) U = max(U, s_top[i]);
  auto tm_s = [&](int i) { return tmem + (uint32_t)(i * 2 * kN); };     // hi, then lo columns
  auto tm_o = [&](int u) { return tmem + 4u * kN + (uint32_t)(u * kN); };

  // -------------------------------------------------------------- K pieces
  if (warp == kTma) {
    if (lane == 0) {
      const int total = kPieces * n_pre;
      int loaded = min(kSlots, total);         // by the set-up
      for (int g = loaded; g < total && !flags[1]; ++g) {
        if (!wait_timed(bar(BAR_K_EMPTY + g % kSlots), (g / kSlots - 1) & 1)) {
          flags[1] = 1;
          break;
        }
        load_piece(g, tile_row[g / kPieces]);
        ++loaded;
      }
      // no copy may be in flight when the CTA leaves
      for (int sl = 0; sl < kSlots && sl < loaded; ++sl)
        mbar_wait(bar(BAR_K_FULL + sl), ((loaded - 1 - sl) / kSlots) & 1);
    }
    __syncwarp();
  }

  // -------------------------------------------------------------- widening
  else if (warp >= kWide) {
    const int tree_at = max(n_pre - 1, 0);
    bool ok = true;
    for (int t = 0; ok && t < ntiles; ++t) {
      if (with_tree && t == tree_at) {
        // the scratch rows' keys, hi pieces then lo pieces, through the K ring
#pragma unroll 1
        for (int i = 0; i < 2 * kPieces; ++i) {
          const int g = kPieces * n_pre + i, sl = g % kSlots;
          if (g >= kSlots &&
              !__all_sync(kFull, wait_timed(bar(BAR_K_EMPTY + sl), (g / kSlots - 1) & 1))) {
            ok = false;
            break;
          }
          const int j = i % kPieces, units = j < 4 ? 8 : 4;
#pragma unroll 1
          for (int x = wt; x < kKeys * units; x += kWideThreads) {
            const int r = x / units, u = x % units;
            uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
            const float f = kt_in[r];
            if (f != 0.f) {
              const uint4* p = tree_row(r) + 16 * j + 2 * u;
              const uint4 w[2] = {__ldg(p), __ldg(p + 1)};
              split16(w, f, hi, lo);
            }
            *(uint4*)(smem + kOffK + sl * kPiece +
                      (j < 4 ? unit_offset<128>(r, u) : unit_offset<64>(r, u))) = i < kPieces ? hi : lo;
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_T_FULL + sl));
        }
        if (!ok) break;
      }
#pragma unroll 1
      for (int u = 0; u < kUnits; ++u) {
        const int g = kUnits * t + u, st = g & 1;
        if (g >= 2 && !__all_sync(kFull, wait_timed(bar(BAR_V_EMPTY + st), ((g >> 1) - 1) & 1))) {
          ok = false;
          break;
        }
        uint8_t* const stage = smem + kOffV + st * kTile;
        if (t < n_pre) {
          share.widen(vreg, stage);
        } else {
#pragma unroll 2
          for (int x = wt; x < kKeys * 16; x += kWideThreads) {
            const int row = x >> 4, c = x & 15;
            const float f = vt_in[row];
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (f != 0.f) v = scale8(__ldg(tree_row(row) + 16 * u + c), f);
            *(uint4*)(stage + (c >> 3) * kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_V_FULL + st));
        const int t1 = u + 1 < kUnits ? t : t + 1, u1 = (u + 1) % kUnits;
        if (t1 < n_pre) load_v(tile_row[t1], valid_of(t1), u1);
      }
      if (__any_sync(kFull, flags[1] != 0)) break;
    }
    if (!ok) flags[1] = 1;
  }

  // ------------------------------------------------------------- scores
  else if (warp == kQk) {
    constexpr uint32_t idesc =
        (1u << 4) | ((uint32_t)(2 * kN >> 3) << 17) | ((uint32_t)(kKeys >> 4) << 24);
    const bool one = elect_one();
    // S^T (+)= K piece j in slot sl x Q piece j
    auto products = [&](uint32_t ts, int sl, int j, bool first) {
      const uint32_t k = sbase + kOffK + sl * kPiece, q = sbase + kOffQ + j * kPiece;
      if (j < 4) {
        const uint64_t kd = row_desc<128>(k), qd = row_desc<128>(q);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f8(ts, kd + 2 * kk, qd + 2 * kk, idesc, first && kk == 0 ? 0u : 1u);
      } else {
        const uint64_t kd = row_desc<64>(k), qd = row_desc<64>(q);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) mma_f8(ts, kd + 2 * kk, qd + 2 * kk, idesc, 1u);
      }
    };
    bool ok = true;
    for (int t = 0; ok && t < ntiles; ++t) {
      const int st = t & 1;
      // the buffer's scores of tile t - 2 have been read once its P is there
      if (t >= 2) ok = wait_ready(bar(BAR_P_FULL + st), ((t - 2) >> 1) & 1);
      const int n = t < n_pre ? kPieces : 2 * kPieces;
      for (int i = 0; i < n; ++i) {
        const int g = kPieces * t + i, sl = g % kSlots;
        ok = ok && (t < n_pre ? wait_ready(bar(BAR_K_FULL + sl), (g / kSlots) & 1)
                              : wait_ready(bar(BAR_T_FULL + sl), (i / kSlots) & 1));
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        fence_after();
        if (one) {
          products(tmem + (uint32_t)(st * 2 * kN), sl, i % kPieces, i == 0);
          mma_commit(bar(BAR_K_EMPTY + sl));
          if (i == n - 1) mma_commit(bar(BAR_S_FULL + st));
        }
        __syncwarp();
      }
    }
    if (!ok) flags[1] = 1;
  }

  // ------------------------------------------------------------- outputs
  else if (warp == kPv) {
    constexpr uint32_t idesc = (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(kN >> 3) << 17) |
                               ((uint32_t)(kKeys >> 4) << 24);
    const uint64_t vd0 = smem_desc(sbase + kOffV, kHalf, 1024);
    const uint64_t pd0 = smem_desc_interleave(sbase + kOffP, 128, 2048);
    const bool one = elect_one();
    bool ok = true;
    for (int t = 0; ok && t < ntiles; ++t) {
      ok = wait_ready(bar(BAR_P_FULL + (t & 1)), (t >> 1) & 1) && !flags[1];
      const uint64_t pd = pd0 + (uint64_t)((t & 1) * (kPtBytes >> 4));
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int st = u & 1;                    // (four boxes a tile)
        ok = ok && wait_ready(bar(BAR_V_FULL + st), (2 * t + (u >> 1)) & 1);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        fence_after();
        const uint64_t vd = vd0 + (uint64_t)(st * (kTile >> 4));
        const uint32_t to = tmem + 4u * kN + (uint32_t)(u * kN);
        if (one) {
          mma_f16(to, vd, pd, idesc, t == 0 ? 0u : 1u);
#pragma unroll
          for (int kk = 1; kk < kKeys / 16; ++kk)
            mma_f16_acc(to, vd + 128 * kk, pd + (uint64_t)(16 * kk), idesc);
          mma_commit(bar(BAR_V_EMPTY + st));
          if (u == kUnits - 1) {
            mma_commit(bar(BAR_PV_DONE + (t & 1)));
            if (t == ntiles - 1) mma_commit(bar(BAR_O_DONE));
          }
        }
        __syncwarp();
      }
    }
    if (!ok) flags[1] = 1;
  }

  // -------------------------------------------------------------- softmax
  else {
    const int wg = warp >> 2, q = warp & 3;
    const int key = q * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    // columns 16 wg .. + 15 of the CTA's 64: two core columns of P^T
    const int c0 = kNH * wg;
    const uint32_t pt_off = (uint32_t)key * 16u + (uint32_t)(c0 >> 3) * 2048u;
    float2 l2[kNH / 2];
#pragma unroll
    for (int i = 0; i < kNH / 2; ++i) l2[i] = make_float2(0.f, 0.f);
    bool failed = false;

    for (int t = 0; t < ntiles; ++t) {
      const int st = t & 1;
      const bool is_tree = t >= n_pre;
      const int nvalid = is_tree ? a.R : valid_of(t);
      float ck, fv;
      if (is_tree) {
        ck = kt_out[key];
        fv = pow2i(vt_u[key] - U + kHeadroom);
      } else {
        ck = q8_scale(kex[2 * t + (key >> 6)]);
        fv = pow2i((int)kex[2 * t + (key >> 6)] - 127 - U + kHeadroom);
      }
      const float2 ck2 = make_float2(ck, ck), fv2 = make_float2(fv, fv);
      const bool ok = __all_sync(kFull, wait_ready(bar(BAR_S_FULL + st), (t >> 1) & 1));
      fence_after();
      const uint32_t srow = tm_s(st) + lane_off + (uint32_t)c0;
      float v[kNH];
      if (ok) {
        float lo[kNH];
        tmem_ld8(srow, v);
        tmem_ld8(srow + 8, v + 8);
        tmem_ld8(srow + kN, lo);
        tmem_ld8(srow + kN + 8, lo + 8);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < kNH; ++i) v[i] += lo[i];
      }
#pragma unroll
      for (int i = 0; i < kNH; i += 4) {
        const float4 nm = *(const float4*)(negm + c0 + i);
        const float4 c2 = *(const float4*)(c2v + c0 + i);
        const float2 x01 = __ffma2_rn(make_float2(v[i], v[i + 1]),
                                      __fmul2_rn(make_float2(c2.x, c2.y), ck2),
                                      make_float2(nm.x, nm.y));
        const float2 x23 = __ffma2_rn(make_float2(v[i + 2], v[i + 3]),
                                      __fmul2_rn(make_float2(c2.z, c2.w), ck2),
                                      make_float2(nm.z, nm.w));
        v[i] = x01.x;
        v[i + 1] = x01.y;
        v[i + 2] = x23.x;
        v[i + 3] = x23.y;
      }
      if (is_tree || nvalid < kKeys) {
        if (key >= nvalid) {
#pragma unroll
          for (int i = 0; i < kNH; ++i) v[i] = -INFINITY;
        } else if (is_tree && key > 0) {
#pragma unroll
          for (int i = 0; i < kNH; ++i)
            if (!((rmask[c0 + i] >> (key - 1)) & 1ull)) v[i] = -INFINITY;
        }
      }
      float tmax = -INFINITY;
#pragma unroll
      for (int i = 0; i < kNH; i += 2) tmax = max3f(tmax, v[i], v[i + 1]);

      const bool local_stop = !ok || failed || flags[1] != 0;
      if (wg_bar_or(wg, local_stop || t == 0 || tmax > kOverflow)) {
        if (wg_bar_or(wg, local_stop)) {
          failed = true;
          break;
        }
#pragma unroll
        for (int e4 = 0; e4 < kNH / 4; ++e4) {
          float r4[4] = {v[4 * e4], v[4 * e4 + 1], v[4 * e4 + 2], v[4 * e4 + 3]};
          const float r = warp_reduce_scatter<4, true>(r4, lane);
          if (lane < 4) red[warp * kNH + 4 * e4 + lane] = r;
        }
        wg_bar(wg);
        if ((tid & 127) < kNH) {
          const int n = tid & 127, col = c0 + n;
          float X = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) X = fmaxf(X, red[(wg * 4 + w) * kNH + n]);
          const float m_old = m_run[col];
          float m_new, sh, al;
          if (m_old == -INFINITY) {
            m_new = X;
            sh = X == -INFINITY ? 0.f : X;
            al = 0.f;
          } else {
            sh = fmaxf(X, 0.f);
            m_new = m_old + sh;
            al = ex2(-sh);
          }
          m_run[col] = m_new;
          alpha[col] = al;
          shiftv[col] = sh;
          negm[col] = m_new == -INFINITY ? 0.f : -m_new;
        }
        wg_bar(wg);
        if (t > 0 && !__all_sync(kFull, wait_ready(bar(BAR_PV_DONE + ((t - 1) & 1)), ((t - 1) >> 1) & 1)))
          failed = true;
        fence_after();
#pragma unroll
        for (int i = 0; i < kNH; i += 2) {
          const float2 sh = *(const float2*)(shiftv + c0 + i);
          const float2 al = *(const float2*)(alpha + c0 + i);
          v[i] -= sh.x;
          v[i + 1] -= sh.y;
          l2[i / 2] = __fmul2_rn(l2[i / 2], al);
        }
        if (t > 0 && !failed) {
#pragma unroll 1
          for (int u = 0; u < kUnits; ++u)
#pragma unroll
            for (int i = 0; i < kNH; i += 8) {
              float o[8];
              const uint32_t ta = tm_o(u) + lane_off + (uint32_t)(c0 + i);
              tmem_ld8(ta, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] *= alpha[c0 + i + j];
              tmem_st8(ta, o);
            }
          tmem_wait_st();
        }
      }
      // P^T buffer st was last read by tile t - 2's products
      if (t >= 2 && !__all_sync(kFull, wait_ready(bar(BAR_PV_DONE + st), ((t - 2) >> 1) & 1)))
        failed = true;
      uint32_t w[kNH / 2];
#pragma unroll
      for (int i = 0; i < kNH / 2; ++i) {
        const float2 p = make_float2(ex2(v[2 * i]), ex2(v[2 * i + 1]));
        l2[i] = __fadd2_rn(l2[i], p);
        const float2 pv = __fmul2_rn(p, fv2);
        w[i] = pack_half2(pv.x, pv.y);
      }
      if (!failed) {
        uint8_t* pt = smem + kOffP + st * kPtBytes + pt_off;
        *(uint4*)pt = make_uint4(w[0], w[1], w[2], w[3]);
        *(uint4*)(pt + 2048) = make_uint4(w[4], w[5], w[6], w[7]);
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_P_FULL + st));
    }

    // ---------------------------------------------------------- epilogue
    failed = __any_sync(kFull, failed);
    const bool ok = !failed && __all_sync(kFull, wait_timed(bar(BAR_O_DONE), 0));
    fence_after();
    const bool stop = wg_bar_or(wg, !ok || flags[1] != 0);
    if (!stop) {
#pragma unroll
      for (int i = 0; i < kNH / 4; ++i) {
        float r4[4] = {l2[2 * i].x, l2[2 * i].y, l2[2 * i + 1].x, l2[2 * i + 1].y};
        const float r = warp_reduce_scatter<4, false>(r4, lane);
        if (lane < 4) red[warp * kNH + 4 * i + lane] = r;
      }
      wg_bar(wg);
      const float unit = pow2i(U);
      if ((tid & 127) < kNH) {
        const int n = tid & 127, col = c0 + n;
        float ls = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) ls += red[(wg * 4 + w) * kNH + n];
        alpha[col] = pow2i(-kHeadroom) / ls;
        if (col < rows_here) {
          const int p = row_base + col;
          const int tr = p / a.g, qh = hk * a.g + p % a.g;
          const float lse2 = m_run[col] + log2f(ls);
          if (nsb == 1) {
            const long orow = ((long)b * a.R + tr) * a.Hq + qh;
            ooff[col] = orow * kDV;
            a.lse[orow] = lse2 * 0.69314718055994531f;
          } else {
            const long prow = (((long)b * a.Hq + qh) * a.R + tr) * a.nsplit + sp;
            ooff[col] = prow * kDV;
            a.part_meta[prow] = make_float2(lse2, unit);
          }
        }
      }
      wg_bar(wg);
#pragma unroll 1
      for (int u = 0; u < kUnits; ++u) {
        const int d = u * 128 + key;             // O^T lane = dim
        float o[kNH];
        tmem_ld8(tm_o(u) + lane_off + (uint32_t)c0, o);
        tmem_ld8(tm_o(u) + lane_off + (uint32_t)c0 + 8, o + 8);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < kNH; ++i) {
          const int col = c0 + i;
          if (col >= rows_here) break;
          const float res = o[i] * alpha[col];
          if (nsb == 1) ((__nv_bfloat16*)a.out)[ooff[col] + d] = __float2bfloat16_rn(res * unit);
          else ((__half*)a.part_o)[ooff[col] + d] = __float2half_rn(res);
        }
      }
    }
    if (!ok && lane == 0) flags[1] = 1;
  }

  // --------------------------------------------------------------- teardown
  // Products in flight: the issuing warps wait for a commit of their own.
  if (warp == kQk || warp == kPv) {
    if (elect_one()) mma_commit(bar(BAR_FINAL + warp - kQk));
    __syncwarp();
    mbar_wait(bar(BAR_FINAL + warp - kQk), 0);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (flags[1] && tid == 0) report_error(a.err, TSD_DEV_ERR_TIMEOUT, b);
  fence_after();
  if (warp == kQk) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
  }
}

}  // namespace

bool launch_q8_latent(const tsd_attn_desc& d, const Q8AttnArgs& a, const Q8Plan& p,
                      cudaStream_t st) {
  LatentMaps m;
  if (encode_fn() == nullptr || !encode_keys(&m.wide, a, kDK, 128) ||
      !encode_keys(&m.last, a, kDK, 64))
    return false;
  const auto kern = a.wait_cycles < kWaitCycles ? q8_latent_kernel<true> : q8_latent_kernel<false>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTotal + 1024);
  launch(kern, dim3(p.nsplit, a.map.Hkv * p.nrg, a.B), dim3(kThreads), kTotal + 1024, st,
         m, a);
  return true;
}

}  // namespace tsd
