// tcgen05 path of tsd_tree_verify_attn_q8: bf16 heads of 64 or 128 dims.
//
// Products, transposed so that the packed query rows of a KV head (R tree rows
// x g query heads) are the MMA's N (a multiple of 16):
//   S^T[key][n]  = K_tile . Q^T     M = 128 keys, N = packed rows, K = d
//   O^T[dim][n] += V_tile^T . P^T   M = 128 dims, N = packed rows, K = 128 keys
// with fp32 accumulators in tensor memory (S^T twice, O^T once).
//
// Numbers.
//   S^T    kind::f8f6f4: the K tile's codes as they are in the cache, and Q as
//          the sum of two e4m3 numbers.  A bf16 row is first multiplied by the
//          power of two that puts its largest element into [128, 256); hi =
//          e4m3(x), lo = e4m3(x - hi).  x has 8 significant bits, hi 4, so
//          x - hi needs 4: hi + lo = x, except where lo falls below e4m3's
//          smallest step (elements below 2^-9 of the largest; off by at most
//          2^-10, 2^-17 of the largest).  The block's power of two (K) and the
//          row's (Q) are applied to the score in fp32.
//   tree   scratch rows of K likewise as hi + lo (four products)
//   V      fp16: a code is an fp16 number; scratch rows are scaled (largest
//          element into [2^8, 2^9): exact down to 2^-33 of it)
//   P      fp16: p * 2^(u - U + 7), u the exponent of the key's value row and U
//          the largest u of the CTA's keys: rounded to 11 bits (2^-12), p below
//          2^-32 (at the largest scale) to multiples of 2^-32.  The row sums
//          take p before it is rounded.
// A score is x = S^T * (2^k_key * scale log2(e) 2^q_n) - m_n, in fp32.
//
// Why V is widened by warps and not taken in 8 bits: kind::f8f6f4 would need P
// in 8 bits.  Two e4m3 terms as for Q do not do: P spans 2^-32..2^8, and what
// lies below 2^-17 of the largest would be lost from long flat rows.
//
// Roles: WG warpgroups of softmax and epilogue (as in tsd_verify_tc.cu:
// warpgroup w/4 owns N / WG of the columns, warp w%4 the TMEM lanes
// 32(w%4)..+31, i.e. 32 keys of a tile or 32 dims of O^T); one warp owns the
// tensor memory and issues the products; one thread loads K tiles by TMA into a
// ring of four; WW warps load V tiles straight into registers, VD tiles ahead
// (behind L2 prefetches), and widen them into two fp16 stages, laid out as the
// product reads them (rows of 64 elements, 128-byte swizzle).  P^T has two
// buffers.  mbarriers order K -> S^T -> softmax -> O^T and V -> O^T; every wait
// is bounded as in the bf16 path.
//
// Softmax with keys on lanes: the running maximum of a column is lazy.  While
// no x of a tile exceeds 8, the tile keeps the old maximum (p <= 256); else, and
// on the CTA's first tile, the warpgroup takes the tile's column maxima,
// re-centres x, and scales the sums and the O^T columns.
#include "tsd_common.cuh"
#include "tsd_host.h"
#include "tsd_q8_tc.cuh"

namespace tsd {
namespace {

// N packed rows of D dims, WG softmax warpgroups, WW widening warps.
template <int N, int D, int WG, int WW>
struct FewLayout {
  static constexpr int soft_warps = 4 * WG;
  static constexpr int threads = (soft_warps + 2 + WW) * 32;
  static constexpr uint32_t k_bytes = kKeys * D;                 // a K tile: [128 keys][D] codes
  static constexpr uint32_t q_bytes = N * D;                     // hi or lo of Q
  static constexpr uint32_t pt_bytes = 256u * N;                 // 128 keys x N fp16
  static constexpr uint32_t off_k = 0;
  static constexpr uint32_t off_v = kRing * k_bytes;
  static constexpr uint32_t off_p = off_v + 2 * kTile;
  static constexpr uint32_t off_q = off_p + 2 * pt_bytes;        // hi, lo: [N][D] e4m3
  static constexpr uint32_t off_misc = off_q + 2 * q_bytes;
  static constexpr int NH = N / WG;               // columns per warpgroup
  static constexpr int NO = NH / 8;               // column octets per warpgroup
  static constexpr bool HQ = NH % 8 != 0;         // plus one quad
  static constexpr int NU = NO + (HQ ? 1 : 0);
  // columns are taken in two halves where one would need too many registers
  static constexpr int U0 = NH > 24 ? NU / 2 : 0; // units of the first half
  static constexpr int V0 = 8 * U0, V1 = NH - V0;
  static constexpr int VMAX = V0 > V1 ? V0 : V1;
  static_assert(NH % 4 == 0, "columns per warpgroup");
  static constexpr uint32_t off_m = off_misc;                          // float[N] running max
  static constexpr uint32_t off_alpha = off_m + 4 * N;                 // float[N]
  static constexpr uint32_t off_negm = off_alpha + 4 * N;              // float[N] -m (0 if -inf)
  static constexpr uint32_t off_shift = off_negm + 4 * N;              // float[N]
  static constexpr uint32_t off_c2 = off_shift + 4 * N;                // float[N] column scales
  static constexpr uint32_t off_red = off_c2 + 4 * N;                  // float[4 WG][NH]
  static constexpr uint32_t off_rmask = off_red + 4 * soft_warps * NH; // u64[N]
  static constexpr uint32_t off_ooff = off_rmask + 8 * N;              // i64[N]
  static constexpr uint32_t off_rows = off_ooff + 8 * N;               // i64[kMaxTiles]
  static constexpr uint32_t off_tree = off_rows + 8 * kMaxTiles;       // 4 x 32 bits [128]
  static constexpr uint32_t off_kex = off_tree + 16 * kKeys;           // u8[2 kMaxTiles]
  static constexpr uint32_t off_vex = off_kex + 2 * kMaxTiles;
  static constexpr uint32_t off_bar = off_vex + 2 * kMaxTiles;
  static constexpr int nbar = 19;
  static constexpr uint32_t off_flags = off_bar + 8 * nbar;            // tmem, abort, U
  static constexpr uint32_t total = off_flags + 16;
  static_assert(total + 1024 <= 232448, "shared memory budget");
  __device__ static int col(int lc, int wg) {
    return lc < 8 * NO ? 8 * (WG * (lc >> 3) + wg) + (lc & 7) : 8 * WG * NO + 4 * wg + (lc - 8 * NO);
  }
};

// FULL: the copy landed or the warps wrote; EMPTY: read by the product (V_EMPTY
// is also the end of a tile's O^T product); T_FULL: the scratch rows' keys, which
// take the two K slots behind the last prefix tile (hi, lo).
enum { BAR_K_FULL = 0, BAR_K_EMPTY = 4, BAR_V_FULL = 8, BAR_V_EMPTY = 10, BAR_S_FULL = 12,
       BAR_P_FULL = 14, BAR_FINAL = 16, BAR_O_DONE = 17, BAR_T_FULL = 18 };

template <int N, int D, int WG, int WW, int VD>
__global__ void __launch_bounds__(FewLayout<N, D, WG, WW>::threads, 1)
q8_few_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ Q8AttnArgs a) {
  using L = FewLayout<N, D, WG, WW>;
  constexpr int kSoftWarps = L::soft_warps, kWideWarps = WW, kWideThreads = 32 * WW;
  constexpr int kMmaWarp = kSoftWarps, kTmaWarp = kSoftWarps + 1, kWideWarp0 = kSoftWarps + 2;
  constexpr int NH = L::NH, NO = L::NO, NU = L::NU, U0 = L::U0, VMAX = L::VMAX;
  constexpr int CH = D / 16;                     // 16-code chunks of a row
  constexpr int kChunks = kKeys * CH;
  constexpr int NT = (kChunks + kWideThreads - 1) / kWideThreads;  // of a tile, per widening thread
  if (threadIdx.x == kTmaWarp * 32) tma_desc_prefetch(&kmap);
  grid_dependency_sync();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = su32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  float* m_run = (float*)(smem + L::off_m);
  float* alpha = (float*)(smem + L::off_alpha);
  float* negm = (float*)(smem + L::off_negm);
  float* shiftv = (float*)(smem + L::off_shift);
  float* c2v = (float*)(smem + L::off_c2);
  float* red = (float*)(smem + L::off_red);
  uint64_t* rmask = (uint64_t*)(smem + L::off_rmask);
  long long* ooff = (long long*)(smem + L::off_ooff);
  long long* tile_row = (long long*)(smem + L::off_rows);
  float* kt_in = (float*)(smem + L::off_tree);      // tree rows: factor into fp16 (0: row of zeros)
  float* vt_in = kt_in + kKeys;
  float* kt_out = vt_in + kKeys;                    // factor of the scores (NaN: a row with a NaN or inf)
  int* vt_u = (int*)(kt_out + kKeys);               // exponent of the value row
  uint8_t* kex = smem + L::off_kex;
  uint8_t* vex = smem + L::off_vex;
  volatile uint32_t* flags = (volatile uint32_t*)(smem + L::off_flags);
  int* s_top = (int*)(smem + L::off_flags + 8);     // U
  const uint32_t bar0 = sbase + L::off_bar;
  auto bar = [&](int i) { return bar0 + 8u * i; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x / a.nrg, rg = blockIdx.x % a.nrg, sp = blockIdx.y, b = blockIdx.z;
  const int P = min(max(a.plen[b], 0), a.map.cap);
  const int nsb = q8_splits(a, P);
  if (sp >= nsb) return;
  const int k0 = min(sp * a.split_len, P), k1 = min(P, k0 + a.split_len);
  const int n_pre = (k1 - k0 + kKeys - 1) / kKeys;
  const bool with_tree = sp == nsb - 1;             // R <= 65 < 128: one tile
  const int ntiles = n_pre + (with_tree ? 1 : 0);
  const int row_base = rg * a.rb;
  const int rows_here = min(a.rb, a.M - row_base);

  // ---------------------------------------------------------------- set-up
  if (tid == kMmaWarp * 32) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(bar(BAR_K_FULL + i), 1);
      mbar_init(bar(BAR_K_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(BAR_V_FULL + i), kWideWarps);
      mbar_init(bar(BAR_V_EMPTY + i), 1);
      mbar_init(bar(BAR_S_FULL + i), 1);
      mbar_init(bar(BAR_P_FULL + i), kSoftWarps);
    }
    mbar_init(bar(BAR_FINAL), 1);
    mbar_init(bar(BAR_O_DONE), 1);
    mbar_init(bar(BAR_T_FULL), kWideWarps);
    flags[1] = 0;
    *s_top = -1000;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
        sbase + L::off_flags));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  __syncthreads();

  // widening threads: chunk i of this thread is (row, 16-code chunk); eight
  // lanes that store together take chunks 0-3 of an even and an odd row (D =
  // 128), or of two rows (D = 64): eight different 16-byte columns of a
  // swizzled row pair, so the stores do not conflict
  const int wt = tid - kWideWarp0 * 32;
  auto chunk_row = [&](int i) {
    const int x = wt + kWideThreads * i;
    return D == 128 ? 2 * (x >> 4) + ((x >> 2) & 1) : x >> 2;
  };
  auto chunk_col = [&](int i) {
    const int x = wt + kWideThreads * i;
    return D == 128 ? (x & 3) + 4 * ((x >> 3) & 1) : x & 3;
  };
  uint4 vreg[VD][NT];
  auto load_v = [&](uint4 (&r)[NT], long row, int nvalid) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      r[i] = make_uint4(0u, 0u, 0u, 0u);
      // (the last round may be short; a row past the tile is never valid)
      if (row >= 0 && chunk_row(i) < nvalid)
        r[i] = ld_stream(a.vc + (row + chunk_row(i)) * D + chunk_col(i) * 16);
    }
  };
  auto valid_of = [&](int t) { return min(kKeys, k1 - (k0 + t * kKeys)); };

  if (warp >= kWideWarp0) {
    // the first tile's loads go out before anything else
#pragma unroll
    for (int i = 0; i < VD; ++i)
      if (i < n_pre) load_v(vreg[i], a.map.row(b, hk, k0 + i * kKeys), valid_of(i));
    int top = -1000;
    for (int t = wt; t < n_pre; t += kWideThreads) {
      const int pos = k0 + t * kKeys;
      const long r = a.map.row(b, hk, pos);
      tile_row[t] = r;
      if (r < 0) report_error(a.err, TSD_DEV_ERR_BAD_PAGE, b);
      const long e = a.map.block(b, hk, pos);
      const bool second = pos + kQ8Block < k1;      // (the last block of a tile may not exist)
      const int ka = r < 0 ? 127 : a.ke[e], va = r < 0 ? 127 : a.ve[e];
      const int kb = r < 0 || !second ? 127 : a.ke[e + 1];
      const int vb = r < 0 || !second ? va : a.ve[e + 1];
      kex[2 * t] = (uint8_t)ka;
      kex[2 * t + 1] = (uint8_t)kb;
      vex[2 * t] = (uint8_t)va;
      vex[2 * t + 1] = (uint8_t)vb;
      top = max(top, max(va, vb) - 127);
    }
    if (with_tree) top = max(top, scan_tree<D>(a, b, hk, wt, kWideThreads, kt_in, vt_in, kt_out, vt_u));
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) atomicMax(s_top, top);
    if (D == 64) {       // the upper 64 dims of the value tiles stay zero
      for (int x = wt; x < 2 * (int)(kHalf / 16); x += kWideThreads)
        *(uint4*)(smem + L::off_v + (x >= (int)(kHalf / 16) ? kTile : 0u) + kHalf +
                  (x % (int)(kHalf / 16)) * 16) = make_uint4(0u, 0u, 0u, 0u);
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    }
  } else if (warp < kSoftWarps) {
    stage_q<D>(a, b, hk, row_base, rows_here, N, tid, kSoftWarps * 32, smem + L::off_q,
               smem + L::off_q + L::q_bytes, c2v);
    for (int n = tid; n < N; n += kSoftWarps * 32) {
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
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = flags[0];
  const int U = *s_top;
  auto tm_s = [&](int i) { return tmem + (uint32_t)(i * N); };
  const uint32_t tm_o = tmem + 2u * N;

  // -------------------------------------------------------------- K tiles
  if (warp == kTmaWarp) {
    if (lane == 0) {
      int loaded = 0;
      for (int t = 0; t < n_pre && !flags[1]; ++t) {
        const int sl = t % kRing;
        if (t >= kRing && !mbar_wait(bar(BAR_K_EMPTY + sl), (t / kRing - 1) & 1)) {
          flags[1] = 1;
          break;
        }
        load_keys(a, kmap, b, hk, k0 + t * kKeys, tile_row[t], sbase + L::off_k + sl * L::k_bytes,
                  L::k_bytes, bar(BAR_K_FULL + sl));
        ++loaded;
        if (t == 0)
          for (int i = VD; i < kPrefetch; ++i)
            if (i < n_pre && tile_row[i] >= 0) prefetch_l2(a.vc + tile_row[i] * D, (long)valid_of(i) * D);
        const int i = t + kPrefetch;
        if (i < n_pre && tile_row[i] >= 0) prefetch_l2(a.vc + tile_row[i] * D, (long)valid_of(i) * D);
      }
      // no copy may be in flight when the CTA leaves
      for (int sl = 0; sl < kRing && sl < loaded; ++sl)
        mbar_wait(bar(BAR_K_FULL + sl), ((loaded - 1 - sl) / kRing) & 1);
    }
    __syncwarp();
  }

  // -------------------------------------------------------------- widening
  else if (warp >= kWideWarp0) {
    auto widen = [&](const uint4 (&r)[NT], uint32_t stage) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (kChunks % kWideThreads != 0 && wt + kWideThreads * i >= kChunks) break;
        const int row = chunk_row(i), c = chunk_col(i);
        const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) q8_half4(w[j], h[2 * j], h[2 * j + 1]);
        uint8_t* dst = smem + stage + (c >> 2) * kHalf + row * 128;
        const int u = 2 * (c & 3);
        *(uint4*)(dst + (((u + 0) ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        *(uint4*)(dst + (((u + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
      }
    };
    const int tree_at = max(n_pre - 2, 0);     // the tree's keys are made two tiles early
    bool ok = true;
    for (int t0 = 0; ok && t0 < ntiles; t0 += VD) {
#pragma unroll
      for (int i = 0; i < VD; ++i) {           // (constant register indexes)
        const int t = t0 + i, st = t & 1;
        if (t >= ntiles) break;
        if (with_tree && t == tree_at) {
          const int s0 = n_pre, s1 = n_pre + 1;
          if ((s0 >= kRing && !__all_sync(kFull, mbar_wait(bar(BAR_K_EMPTY + s0 % kRing),
                                                           (s0 / kRing - 1) & 1))) ||
              (s1 >= kRing && !__all_sync(kFull, mbar_wait(bar(BAR_K_EMPTY + s1 % kRing),
                                                           (s1 / kRing - 1) & 1)))) {
            flags[1] = 1;
            ok = false;
            break;
          }
          tree_keys<D>(a, b, hk, wt, kWideThreads, kt_in, smem + L::off_k + (s0 % kRing) * L::k_bytes,
                       smem + L::off_k + (s1 % kRing) * L::k_bytes);
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_T_FULL));
        }
        if (t >= 2 && !__all_sync(kFull, mbar_wait(bar(BAR_V_EMPTY + st), ((t >> 1) - 1) & 1))) {
          flags[1] = 1;
          ok = false;
          break;
        }
        if (t < n_pre) widen(vreg[i], L::off_v + st * kTile);
        else tree_values<D>(a, b, hk, wt, kWideThreads, vt_in, smem + L::off_v + st * kTile);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_V_FULL + st));
        if (t + VD < n_pre) load_v(vreg[i], tile_row[t + VD], valid_of(t + VD));
        if (__any_sync(kFull, flags[1] != 0)) {
          ok = false;
          break;
        }
      }
    }
  }

  // ------------------------------------------------------------------ MMA
  else if (warp == kMmaWarp) {
    if (lane == 0) {
      // fp32 accumulators; e4m3 (S^T) and fp16 (O^T) operands are both format 0
      const uint32_t idesc_qk = (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kKeys >> 4) << 24);
      const uint32_t idesc_pv = idesc_qk | (1u << 15) | (1u << 16);
      const uint64_t kd0 = row_desc<D>(sbase + L::off_k);
      const uint64_t qd0 = row_desc<D>(sbase + L::off_q);
      const uint64_t vd0 = smem_desc(sbase + L::off_v, kHalf, 1024);
      // P^T: 8x8 cores, the key groups of 8 columns contiguous (tsd_verify_tc.cu)
      const uint64_t pd0 = smem_desc_interleave(sbase + L::off_p, 128, 2048);
      // S^T (+)= K slot x (Q hi + Q lo)
      auto products = [&](uint32_t ts, int sl, bool first) {
        const uint64_t kd = kd0 + (uint64_t)(sl * (L::k_bytes >> 4));
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma_f8(ts, kd + 2 * kk, qd0 + (uint64_t)(part * (L::q_bytes >> 4)) + 2 * kk, idesc_qk,
                   first && part == 0 && kk == 0 ? 0u : 1u);
      };
      auto issue_qk = [&](int t) -> bool {
        const int st = t & 1, sl = t % kRing;
        if (!(t < n_pre ? mbar_wait(bar(BAR_K_FULL + sl), (t / kRing) & 1)
                        : mbar_wait(bar(BAR_T_FULL), 0)))
          return false;
        fence_after();
        products(tm_s(st), sl, true);
        if (t >= n_pre) products(tm_s(st), (t + 1) % kRing, false);
        mma_commit(bar(BAR_S_FULL + st));
        mma_commit(bar(BAR_K_EMPTY + sl));
        return true;
      };
      bool ok = issue_qk(0);
      for (int t = 0; ok && t < ntiles; ++t) {
        const int st = t & 1;
        if (t + 1 < ntiles && !issue_qk(t + 1)) { ok = false; break; }
        if (!mbar_wait(bar(BAR_P_FULL + st), (t >> 1) & 1) || flags[1] ||
            !mbar_wait(bar(BAR_V_FULL + st), (t >> 1) & 1)) {
          ok = false;
          break;
        }
        fence_after();
        const uint64_t vd = vd0 + (uint64_t)(st * (kTile >> 4));
        const uint64_t pd = pd0 + (uint64_t)(st * (L::pt_bytes >> 4));
        if (t == 0) mma_f16(tm_o, vd, pd, idesc_pv, 0u);
        else mma_f16_acc(tm_o, vd, pd, idesc_pv);
#pragma unroll
        for (int kk = 1; kk < kKeys / 16; ++kk)
          mma_f16_acc(tm_o, vd + 128 * kk, pd + (uint64_t)(16 * kk), idesc_pv);
        mma_commit(bar(BAR_V_EMPTY + st));
        if (t == ntiles - 1) mma_commit(bar(BAR_O_DONE));
      }
      if (!ok) flags[1] = 1;
      // every product has completed once this commit lands
      mma_commit(bar(BAR_FINAL));
      mbar_wait(bar(BAR_FINAL), 0);
    }
    __syncwarp();
  }

  // -------------------------------------------------------------- softmax
  else {
    const int wg = warp >> 2, q = warp & 3;
    const int key = q * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    const int c_oct = 8 * wg, c_quad = 8 * WG * NO + 4 * wg;
    const uint32_t pt_oct = (uint32_t)key * 16u + (uint32_t)wg * 2048u;
    const uint32_t pt_quad =
        (uint32_t)key * 16u + (uint32_t)(c_quad >> 3) * 2048u + (uint32_t)(c_quad & 4) * 2u;
    float2 l2[NH / 2];
#pragma unroll
    for (int i = 0; i < NH / 2; ++i) l2[i] = make_float2(0.f, 0.f);
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
        fv = pow2i((int)vex[2 * t + (key >> 6)] - 127 - U + kHeadroom);
      }
      const float2 ck2 = make_float2(ck, ck), fv2 = make_float2(fv, fv);
      const bool ok = __all_sync(kFull, mbar_wait(bar(BAR_S_FULL + st), (t >> 1) & 1));
      fence_after();
      const uint32_t srow = tm_s(st) + lane_off;
      uint8_t* pt = smem + L::off_p + st * L::pt_bytes;
      bool stop_now = false;
      bool p_free = t < 2;                   // O^T_(t-2) has read this P^T buffer
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int ua = h == 0 ? 0 : U0, ub = h == 0 ? U0 : NU;
        if (ua >= ub) continue;
        const int lc0 = 8 * ua;
        const int ncol = (ub == NU && L::HQ) ? 8 * (ub - 1 - ua) + 4 : 8 * (ub - ua);
        // x = S^T * scale - m, and the largest x
        float v[VMAX];
        if (ok) {
#pragma unroll
          for (int u = ua; u < ub; ++u) {
            float* x = v + 8 * (u - ua);
            if (u < NO) tmem_ld8(srow + (uint32_t)(8 * WG * u + c_oct), x);
            else tmem_ld4(srow + (uint32_t)c_quad, x[0], x[1], x[2], x[3]);
          }
          tmem_wait_ld();
        }
#pragma unroll
        for (int u = ua; u < ub; ++u) {
          float* x = v + 8 * (u - ua);
          const int nq = u < NO ? 2 : 1;
          const int c = u < NO ? 8 * WG * u + c_oct : c_quad;
#pragma unroll
          for (int j = 0; j < nq; ++j) {
            const float4 nm = *(const float4*)(negm + c + 4 * j);
            const float4 c2 = *(const float4*)(c2v + c + 4 * j);
            const float2 x01 = __ffma2_rn(make_float2(x[4 * j], x[4 * j + 1]),
                                          __fmul2_rn(make_float2(c2.x, c2.y), ck2),
                                          make_float2(nm.x, nm.y));
            const float2 x23 = __ffma2_rn(make_float2(x[4 * j + 2], x[4 * j + 3]),
                                          __fmul2_rn(make_float2(c2.z, c2.w), ck2),
                                          make_float2(nm.z, nm.w));
            x[4 * j] = x01.x;
            x[4 * j + 1] = x01.y;
            x[4 * j + 2] = x23.x;
            x[4 * j + 3] = x23.y;
          }
        }
        if (is_tree || nvalid < kKeys) {
          if (key >= nvalid) {
#pragma unroll
            for (int e = 0; e < VMAX; ++e) v[e] = -INFINITY;
          } else if (is_tree && key > 0) {
            uint32_t vis = 0u;
#pragma unroll 1
            for (int e = 0; e < ncol; ++e)
              vis |= (uint32_t)((rmask[L::col(lc0 + e, wg)] >> (key - 1)) & 1ull) << e;
#pragma unroll
            for (int e = 0; e < VMAX; ++e)
              if (!((vis >> e) & 1u)) v[e] = -INFINITY;
          }
        }
        float tmax = -INFINITY;
#pragma unroll
        for (int e = 0; e < VMAX; e += 2)
          if (e < ncol) tmax = max3f(tmax, v[e], v[e + 1]);

        const bool local_stop = ua == 0 && (!ok || failed || flags[1] != 0);
        if (wg_bar_or(wg, local_stop || t == 0 || tmax > kOverflow)) {
          if (ua == 0 && wg_bar_or(wg, local_stop)) {
            stop_now = true;
            break;
          }
#pragma unroll
          for (int e4 = 0; e4 < VMAX / 4; ++e4) {
            if (4 * e4 >= ncol) break;
            float r4[4] = {v[4 * e4], v[4 * e4 + 1], v[4 * e4 + 2], v[4 * e4 + 3]};
            const float r = warp_reduce_scatter<4, true>(r4, lane);
            if (lane < 4) red[warp * NH + lc0 + 4 * e4 + lane] = r;
          }
          wg_bar(wg);
          for (int n = lc0 + (tid & 127); n < lc0 + ncol; n += 128) {
            const int col = L::col(n, wg);
            float X = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) X = fmaxf(X, red[(wg * 4 + w) * NH + n]);
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
          if (t > 0) {
            if (!__all_sync(kFull, mbar_wait(bar(BAR_V_EMPTY + ((t - 1) & 1)), ((t - 1) >> 1) & 1)))
              failed = true;
            fence_after();
          }
#pragma unroll
          for (int u = ua; u < ub; ++u) {
            float* x = v + 8 * (u - ua);
            const int nq = u < NO ? 2 : 1;
            const int c = u < NO ? 8 * WG * u + c_oct : c_quad;
            const int li = u < NO ? 4 * u : 4 * NO;
#pragma unroll
            for (int j = 0; j < nq; ++j) {
              const float4 sh = *(const float4*)(shiftv + c + 4 * j);
              const float4 al = *(const float4*)(alpha + c + 4 * j);
              x[4 * j] -= sh.x;
              x[4 * j + 1] -= sh.y;
              x[4 * j + 2] -= sh.z;
              x[4 * j + 3] -= sh.w;
              l2[li + 2 * j] = __fmul2_rn(l2[li + 2 * j], make_float2(al.x, al.y));
              l2[li + 2 * j + 1] = __fmul2_rn(l2[li + 2 * j + 1], make_float2(al.z, al.w));
            }
            if (t > 0 && !failed) {
              float o[8];
              const uint32_t ta = tm_o + lane_off + (uint32_t)c;
              if (u < NO) tmem_ld8(ta, o);
              else tmem_ld4(ta, o[0], o[1], o[2], o[3]);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < nq; ++j) {
                const float4 al = *(const float4*)(alpha + c + 4 * j);
                o[4 * j] *= al.x;
                o[4 * j + 1] *= al.y;
                o[4 * j + 2] *= al.z;
                o[4 * j + 3] *= al.w;
              }
              if (u < NO) tmem_st8(ta, o);
              else tmem_st4(ta, o[0], o[1], o[2], o[3]);
            }
          }
          tmem_wait_st();
        }
        if (!p_free) {
          if (!__all_sync(kFull, mbar_wait(bar(BAR_V_EMPTY + st), ((t - 2) >> 1) & 1))) failed = true;
          p_free = true;
        }
        // p = 2^x, its sums, and the P^T row of this key
#pragma unroll
        for (int u = ua; u < ub; ++u) {
          const float* x = v + 8 * (u - ua);
          const int li = u < NO ? 4 * u : 4 * NO;
          const int np = u < NO ? 4 : 2;
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < np; ++i) {
            const float2 p = make_float2(ex2(x[2 * i]), ex2(x[2 * i + 1]));
            l2[li + i] = __fadd2_rn(l2[li + i], p);
            const float2 pv = __fmul2_rn(p, fv2);
            w[i] = pack_half2(pv.x, pv.y);
          }
          if (!failed) {
            if (u < NO) *(uint4*)(pt + pt_oct + 2048u * WG * u) = make_uint4(w[0], w[1], w[2], w[3]);
            else *(uint2*)(pt + pt_quad) = make_uint2(w[0], w[1]);
          }
        }
      }
      if (stop_now) {
        failed = true;
        break;
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_P_FULL + st));
    }

    // ---------------------------------------------------------- epilogue
    failed = __any_sync(kFull, failed);
    const bool ok = !failed && __all_sync(kFull, mbar_wait(bar(BAR_O_DONE), 0));
    fence_after();
    const bool stop = wg_bar_or(wg, !ok || flags[1] != 0);
    if (!stop) {
#pragma unroll
      for (int i = 0; i < NH / 4; ++i) {
        float r4[4] = {l2[2 * i].x, l2[2 * i].y, l2[2 * i + 1].x, l2[2 * i + 1].y};
        const float r = warp_reduce_scatter<4, false>(r4, lane);
        if (lane < 4) red[warp * NH + 4 * i + lane] = r;
      }
      wg_bar(wg);
      const float unit = pow2i(U);
      for (int n = tid & 127; n < NH; n += 128) {
        const int col = L::col(n, wg);
        float ls = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) ls += red[(wg * 4 + w) * NH + n];
        alpha[col] = pow2i(-kHeadroom) / ls;
        if (col < rows_here) {
          const int p = row_base + col;
          const int tr = p / a.g, qh = hk * a.g + p % a.g;
          const float lse2 = m_run[col] + log2f(ls);
          if (nsb == 1) {
            const long orow = ((long)b * a.R + tr) * a.Hq + qh;
            ooff[col] = orow * D;
            a.lse[orow] = lse2 * 0.69314718055994531f;
          } else {
            const long prow = (((long)b * a.Hq + qh) * a.R + tr) * a.nsplit + sp;
            ooff[col] = prow * D;
            a.part_meta[prow] = make_float2(lse2, unit);
          }
        }
      }
      wg_bar(wg);
      // O^T lane = dim.  A split's output, over 2^U, is a mean of numbers of
      // magnitude < 512: fp16 holds it to 2^-12.
      const int d = key;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        float o[8];
        const int c = u < NO ? 8 * WG * u + c_oct : c_quad;
        if (u < NO) tmem_ld8(tm_o + lane_off + (uint32_t)c, o);
        else tmem_ld4(tm_o + lane_off + (uint32_t)c, o[0], o[1], o[2], o[3]);
        tmem_wait_ld();
        if (D == 64 && d >= D) continue;     // (whole warps: lanes 64..127)
#pragma unroll
        for (int e = 0; e < (u < NO ? 8 : 4); ++e) {
          const int col = c + e;
          if (col >= rows_here) continue;
          const float res = o[e] * alpha[col];
          if (nsb == 1) ((__nv_bfloat16*)a.out)[ooff[col] + d] = __float2bfloat16_rn(res * unit);
          else ((__half*)a.part_o)[ooff[col] + d] = __float2half_rn(res);
        }
      }
    }
    if (!ok && lane == 0) flags[1] = 1;
  }

  // --------------------------------------------------------------- teardown
  fence_before();
  __syncthreads();
  if (flags[1] && tid == 0) report_error(a.err, TSD_DEV_ERR_TIMEOUT, b);
  fence_after();
  if (warp == kMmaWarp) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
  }
}

template <int N, int D, int WG, int WW, int VD>
void launch_n(const CUtensorMap& kmap, const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  using L = FewLayout<N, D, WG, WW>;
  const uint32_t smem = L::total + 1024;
  const auto kern = q8_few_kernel<N, D, WG, WW, VD>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  launch(kern, dim3(a.map.Hkv * p.nrg, p.nsplit, a.B), dim3(L::threads), smem, st, kmap, a);
}

// Softmax warpgroups: one per 32 columns or so, so that its fixed work per tile
// (waits, one barrier) is shared by many columns and a thread's sums and scores
// stay in registers; widening warps and tiles in flight: what is left of the
// registers.
template <int D>
bool launch_d(const CUtensorMap& m, const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  switch (p.rb) {
    case 16: launch_n<16, D, 1, 8, 2>(m, a, p, st); return true;
    case 32: launch_n<32, D, 1, 8, 2>(m, a, p, st); return true;
    case 48: launch_n<48, D, 2, 6, 1>(m, a, p, st); return true;
    case 64: launch_n<64, D, 2, 6, 1>(m, a, p, st); return true;
    case 80: launch_n<80, D, 4, 6, 1>(m, a, p, st); return true;
    case 96: launch_n<96, D, 4, 6, 1>(m, a, p, st); return true;
    case 112: launch_n<112, D, 4, 6, 1>(m, a, p, st); return true;
  }
  return false;
}

}  // namespace

bool launch_q8_few(const tsd_attn_desc& d, const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  CUtensorMap m;
  if (encode_fn() == nullptr || !encode_keys(&m, a, d.dk, d.dk)) return false;
  return d.dk == 128 ? launch_d<128>(m, a, p, st) : launch_d<64>(m, a, p, st);
}

}  // namespace tsd
