// tcgen05 path of tsd_tree_verify_attn_q8 for bf16 heads of 64 or 128 dims with few
// packed rows (R tree rows x g query heads of a KV head): decoding, small trees.
//
// Products, transposed so that the packed rows are the columns (N = 16; the tensor
// core takes 45 cycles for an instruction of 128 x 16, and 48 to 64 in the layout of
// tsd_q8_tc.cu, 128 rows whether they are there or not):
//   S^T[key][n]  = K_tile . Q^T     M = 128 keys, N = packed rows, K = d
//   O^T[dim][n] += V_tile^T . P^T   M = 128 dims, N = packed rows, K = 128 keys
//
// Numbers as in tsd_q8_tc.cu.  A score is x = S^T * (2^k_key * scale log2(e) 2^q_n) -
// m_n, in fp32.
//
// What bounds it: the cache's bytes (32 KB per 128-key tile, 1410 cycles at the
// measured 6.8 TB/s over 152 SMs).  A tile's way through the scores, the softmax and
// the product with V takes longer than that, so even and odd tiles are two streams
// with a softmax warpgroup, a score buffer, a P^T buffer, a maximum, sums and an
// accumulator each, joined at the end.  One token of 16 requests of 32 heads over 20k
// to 32k keys: 165 us with the launch, 5.2 TB/s, 128 us by the bytes (one stream: 226
// us; with 30% more unrolled code, for the instruction cache: 177 us, so set-up loops
// are rolled and the scratch rows are outside the loop over tiles).
//
// Softmax with keys on lanes: a column's maximum is a reduction over the warpgroup,
// so the running maximum is lazy: while no x of a tile exceeds 8, the tile keeps the
// old maximum (p <= 256); else, and on the stream's first tile, the warpgroup takes
// the tile's column maxima, re-centres x, and scales the sums and the O^T columns.
//
// Roles (608 threads): warps 0-3 and 4-7 softmax and epilogue; warp 8 issues the
// products with Q and owns the tensor memory, warp 9 those with V; one thread of
// warp 10 loads K tiles by TMA into a ring of four; warps 11-18 load V tiles straight
// into registers, two tiles ahead (behind L2 prefetches), and widen them into two fp16
// stages, laid out as the product reads them (rows of 64 elements, 128-byte swizzle).
// mbarriers order K -> S^T -> softmax -> O^T and V -> O^T; every wait is bounded.
#include "tsd_common.cuh"
#include "tsd_host.h"
#include "tsd_q8_tc.cuh"

namespace tsd {
namespace {

constexpr int kQk = 8, kPv = 9, kTma = 10, kWide = 11, kWideWarps = 8;
constexpr int kWideThreads = kWideWarps * 32;
constexpr int kThreads = (kWide + kWideWarps) * 32;
constexpr int kDepth = 2;                        // V tiles in registers
constexpr int N = kQ8FewRows;                    // columns of the products
static_assert(kMaxTiles <= kWideThreads, "a widening thread per tile in the set-up");

template <int D>
struct FewLayout {
  static constexpr uint32_t k_bytes = kKeys * D;                 // a K tile: [128 keys][D] codes
  static constexpr uint32_t q_bytes = N * D;                     // hi or lo of Q
  static constexpr uint32_t pt_bytes = 256u * N;                 // 128 keys x N fp16
  static constexpr uint32_t off_k = 0;
  static constexpr uint32_t off_v = kRing * k_bytes;
  static constexpr uint32_t off_p = off_v + 2 * kTile;
  static constexpr uint32_t off_q = off_p + 2 * pt_bytes;        // hi, lo: [N][D] e4m3
  // by stream
  static constexpr uint32_t off_m = off_q + 2 * q_bytes;         // float[2][N] running max
  static constexpr uint32_t off_l = off_m + 8 * N;               // float[2][N] sums, at the end
  static constexpr uint32_t off_alpha = off_l + 8 * N;           // float[2][N]
  static constexpr uint32_t off_negm = off_alpha + 8 * N;        // float[2][N] -m (0 if -inf)
  static constexpr uint32_t off_shift = off_negm + 8 * N;        // float[2][N]
  static constexpr uint32_t off_red = off_shift + 8 * N;         // float[2][4][N]
  static constexpr uint32_t off_c2 = off_red + 32 * N;           // float[N] column scales
  static constexpr uint32_t off_rmask = off_c2 + 4 * N;          // u64[N]
  static constexpr uint32_t off_rows = off_rmask + 8 * N;        // i64[kMaxTiles]
  static constexpr uint32_t off_tree = off_rows + 8 * kMaxTiles; // 4 x 32 bits [128]
  static constexpr uint32_t off_kex = off_tree + 16 * kKeys;     // u8[2 kMaxTiles]
  static constexpr uint32_t off_vex = off_kex + 2 * kMaxTiles;
  static constexpr uint32_t off_bar = off_vex + 2 * kMaxTiles;
  static constexpr int nbar = 20;
  static constexpr uint32_t off_flags = off_bar + 8 * nbar;      // tmem, abort
  static constexpr uint32_t off_top = off_flags + 8;             // int[kWideWarps]
  static constexpr uint32_t off_req = off_top + 4 * kWideWarps;  // request, its length
  static constexpr uint32_t total = off_req + 8;
  static_assert(total + 1024 <= 232448, "shared memory budget");
  // (at D = 64 the upper half of a value tile is zeroed while other warps still scan)
  static_assert(kTreeBytes<D> <= (D == 64 ? kHalf : kTile), "the scan's rows");
};

// FULL: the copy landed or the warps wrote; EMPTY: read by the product (V_EMPTY
// is also the end of a tile's O^T product); T_FULL: the scratch rows' keys, which
// take the two K slots behind the last prefix tile (hi, lo); FINAL: one per issuing
// warp.
enum { BAR_K_FULL = 0, BAR_K_EMPTY = 4, BAR_V_FULL = 8, BAR_V_EMPTY = 10, BAR_S_FULL = 12,
       BAR_P_FULL = 14, BAR_FINAL = 16, BAR_O_DONE = 18, BAR_T_FULL = 19 };

template <int D, bool kPoll>
__global__ void __launch_bounds__(kThreads, 1)
q8_few_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ Q8AttnArgs a) {
  using L = FewLayout<D>;
  if (threadIdx.x == kTma * 32) tma_desc_prefetch(&kmap);
  grid_dependency_sync();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = su32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  float* c2v = (float*)(smem + L::off_c2);
  uint64_t* rmask = (uint64_t*)(smem + L::off_rmask);
  long long* tile_row = (long long*)(smem + L::off_rows);
  float* kt_in = (float*)(smem + L::off_tree);      // tree rows: factor into e4m3 (0: row of zeros)
  float* vt_in = kt_in + kKeys;                     // and into fp16
  float* kt_out = vt_in + kKeys;                    // factor of the scores (NaN: a row with a NaN or inf)
  int* vt_u = (int*)(kt_out + kKeys);               // exponent of the value row
  uint8_t* kex = smem + L::off_kex;
  uint8_t* vex = smem + L::off_vex;
  volatile uint32_t* flags = (volatile uint32_t*)(smem + L::off_flags);
  int* s_top = (int*)(smem + L::off_top);           // U by widening warp
  const uint32_t bar0 = sbase + L::off_bar;
  auto bar = [&](int i) { return bar0 + 8u * i; };
  auto wait_ready = [&](uint32_t at, uint32_t parity) {
    return phase_ready<kPoll>(at, parity, a.wait_cycles);
  };
  auto wait_timed = [&](uint32_t at, uint32_t parity) {
    return phase_timed<kPoll>(at, parity, a.wait_cycles);
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x, sp = blockIdx.y;
  int P;
  const int b = request_at(a, blockIdx.z, P, (volatile int*)(smem + L::off_req));
  const int nsb = q8_splits(a, P);
  if (sp >= nsb) return;
  const int k0 = q8_first(a, P, sp), k1 = q8_end(a, P, k0);
  const int n_pre = (k1 - k0 + kKeys - 1) / kKeys;
  const bool with_tree = sp == nsb - 1;             // R <= 65 < 128: one tile
  const int ntiles = n_pre + (with_tree ? 1 : 0);
  auto valid_of = [&](int t) { return min(kKeys, k1 - (k0 + t * kKeys)); };

  const int wt = tid - kWide * 32;
  using Share = WideShare<D / 16, kWideThreads>;
  const Share share(wt);
  uint4 vreg[kDepth][Share::kCount];
  // the tile at cache row `row` (a missing page: none)
  auto load_v = [&](uint4 (&r)[Share::kCount], long row, int nvalid) {
    share.template load<D>(r, a.vc + (row < 0 ? 0 : row) * D, row < 0 ? 0 : nvalid);
  };

  // ---------------------------------------------------------------- set-up
  // Everything that the first products need is requested at once, by the warps
  // that will use it; one barrier.
  if (warp >= kWide) {
    if (with_tree) tree_fetch<D, kWideThreads>(a, b, hk, wt, sbase + L::off_v, kTile);
    long r[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth; ++i) r[i] = i < n_pre ? a.map.row(b, hk, k0 + i * kKeys) : -1;
    const long rt = wt < n_pre ? a.map.row(b, hk, k0 + wt * kKeys) : -1;
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
      if (i < n_pre) load_v(vreg[i], r[i], valid_of(i));
    int top = -1000;
    if (wt < n_pre) {                               // (n_pre <= kMaxTiles = the widening threads)
      const int pos = k0 + wt * kKeys;
      tile_row[wt] = rt;
      if (rt < 0) report_error(a.err, TSD_DEV_ERR_BAD_PAGE, b);
      const long e = a.map.block_at(b, hk, pos, rt);
      const bool second = pos + kQ8Block < k1;      // (the last block of a tile may not exist)
      const int ka = rt < 0 ? 127 : a.ke[e], va = rt < 0 ? 127 : a.ve[e];
      const int kb = rt < 0 || !second ? 127 : a.ke[e + 1];
      const int vb = rt < 0 || !second ? va : a.ve[e + 1];
      kex[2 * wt] = (uint8_t)ka;
      kex[2 * wt + 1] = (uint8_t)kb;
      vex[2 * wt] = (uint8_t)va;
      vex[2 * wt + 1] = (uint8_t)vb;
      top = max(va, vb) - 127;
    }
    if (with_tree)
      top = max(top, tree_scan<D, kWideThreads>(a, b, wt, smem + L::off_v, kTile, kt_in, vt_in, kt_out,
                                                vt_u));
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) s_top[warp - kWide] = top;
    if (D == 64) {       // the upper 64 dims of the value tiles stay zero
      for (int x = wt; x < 2 * (int)(kHalf / 16); x += kWideThreads)
        *(uint4*)(smem + L::off_v + (x >= (int)(kHalf / 16) ? kTile : 0u) + kHalf +
                  (x % (int)(kHalf / 16)) * 16) = make_uint4(0u, 0u, 0u, 0u);
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    }
  } else if (warp < 8) {
    stage_q<D>(a, b, hk, 0, a.M, N, tid, 256, smem + L::off_q, smem + L::off_q + L::q_bytes, c2v);
    if (tid < N) {
      const int tr = tid < a.M ? tid / a.g : 0;
      rmask[tid] = tr > 0 ? a.mask[(long)b * a.R + tr] : 0ull;
    }
    if (tid < 2 * N) {
      ((float*)(smem + L::off_m))[tid] = -INFINITY;
      ((float*)(smem + L::off_l))[tid] = 0.f;
      ((float*)(smem + L::off_negm))[tid] = 0.f;
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  } else if (warp == kTma) {
    long row = 0;                                    // of the ring's tiles
    if (a.map.page_size && lane < kRing && lane < n_pre) row = a.map.row(b, hk, k0 + lane * kKeys);
    if (lane == 0) {
      for (int i = 0; i < kRing; ++i) {
        mbar_init(bar(BAR_K_FULL + i), 1);
        mbar_init(bar(BAR_K_EMPTY + i), 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(BAR_V_FULL + i), kWideWarps);
        mbar_init(bar(BAR_V_EMPTY + i), 1);
        mbar_init(bar(BAR_S_FULL + i), 1);
        mbar_init(bar(BAR_P_FULL + i), 4);
        mbar_init(bar(BAR_FINAL + i), 1);
      }
      mbar_init(bar(BAR_O_DONE), 1);
      mbar_init(bar(BAR_T_FULL), kWideWarps);
      flags[1] = 0;
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncwarp();
#pragma unroll 1
    for (int t = 0; t < kRing && t < n_pre; ++t) {
      const long r = __shfl_sync(kFull, row, t);
      if (lane == 0)
        load_keys(a, kmap, b, hk, k0 + t * kKeys, r, sbase + L::off_k + t * L::k_bytes, L::k_bytes,
                  bar(BAR_K_FULL + t));
    }
    __syncwarp();
  } else if (warp == kQk) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;\n" ::"r"(
        sbase + L::off_flags));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = flags[0];
  int U = s_top[0];
#pragma unroll
  for (int i = 1; i < kWideWarps; ++i) U = max(U, s_top[i]);
  auto tm_s = [&](int p) { return tmem + (uint32_t)(p * N); };
  auto tm_o = [&](int p) { return tmem + (uint32_t)((2 + p) * N); };

  // -------------------------------------------------------------- K tiles
  if (warp == kTma) {
    if (lane == 0) {
      for (int i = kDepth; i < kRing; ++i)
        if (i < n_pre && tile_row[i] >= 0) prefetch_l2(a.vc + tile_row[i] * D, (long)valid_of(i) * D);
      int loaded = min(kRing, n_pre);          // by the set-up
      for (int t = loaded; t < n_pre && !flags[1]; ++t) {
        const int sl = t % kRing;
        if (!wait_timed(bar(BAR_K_EMPTY + sl), (t / kRing - 1) & 1)) {
          flags[1] = 1;
          break;
        }
        load_keys(a, kmap, b, hk, k0 + t * kKeys, tile_row[t], sbase + L::off_k + sl * L::k_bytes,
                  L::k_bytes, bar(BAR_K_FULL + sl));
        ++loaded;
        if (tile_row[t] >= 0) prefetch_l2(a.vc + tile_row[t] * D, (long)valid_of(t) * D);
      }
      // no copy may be in flight when the CTA leaves
      for (int sl = 0; sl < kRing && sl < loaded; ++sl)
        mbar_wait(bar(BAR_K_FULL + sl), ((loaded - 1 - sl) / kRing) & 1);
    }
    __syncwarp();
  }

  // -------------------------------------------------------------- widening
  else if (warp >= kWide) {
    const int tree_at = max(n_pre - 2, 0) & ~1; // the tree's keys are made two tiles early
    bool ok = true;
    auto stage_free = [&](int t) {
      return t < 2 || __all_sync(kFull, wait_timed(bar(BAR_V_EMPTY + (t & 1)), ((t >> 1) - 1) & 1));
    };
    auto stage_written = [&](int t) {
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_V_FULL + (t & 1)));
    };
    for (int t0 = 0; ok && t0 < max(n_pre, 1); t0 += kDepth) {
      if (with_tree && t0 == tree_at) {
        const int s0 = n_pre, s1 = n_pre + 1;
        ok = (s0 < kRing || __all_sync(kFull, wait_timed(bar(BAR_K_EMPTY + s0 % kRing),
                                                        (s0 / kRing - 1) & 1))) &&
             (s1 < kRing || __all_sync(kFull, wait_timed(bar(BAR_K_EMPTY + s1 % kRing),
                                                        (s1 / kRing - 1) & 1)));
        if (!ok) break;
        tree_keys<D>(a, b, hk, wt, kWideThreads, kt_in,
                     smem + L::off_k + (s0 % kRing) * L::k_bytes,
                     smem + L::off_k + (s1 % kRing) * L::k_bytes);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_T_FULL));
      }
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {       // (constant register indexes)
        const int t = t0 + i;
        if (t >= n_pre) break;
        ok = stage_free(t);
        if (!ok) break;
        share.widen(vreg[i], smem + L::off_v + (t & 1) * kTile);
        stage_written(t);
        if (t + kDepth < n_pre) load_v(vreg[i], tile_row[t + kDepth], valid_of(t + kDepth));
        ok = !__any_sync(kFull, flags[1] != 0);
        if (!ok) break;
      }
    }
    if (with_tree && ok) {
      ok = stage_free(n_pre);
      if (ok) {
        tree_values<D>(a, b, hk, wt, kWideThreads, vt_in, smem + L::off_v + (n_pre & 1) * kTile);
        stage_written(n_pre);
      }
    }
    if (!ok) flags[1] = 1;
  }

  // ------------------------------------------------------------- scores
  else if (warp == kQk) {
    // fp32 accumulators; e4m3 (S^T) and fp16 (O^T) operands are both format 0
    constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kKeys >> 4) << 24);
    const uint64_t kd0 = row_desc<D>(sbase + L::off_k);
    const uint64_t qd0 = row_desc<D>(sbase + L::off_q);
    const bool one = elect_one();
    bool ok = true;
    for (int t = 0; t < ntiles; ++t) {
      const int p = t & 1, sl = t % kRing;
      // (the stream's scores before have been read once its P^T is there)
      ok = (t < n_pre ? wait_ready(bar(BAR_K_FULL + sl), (t / kRing) & 1) : wait_ready(bar(BAR_T_FULL), 0)) &&
           (t < 2 || wait_ready(bar(BAR_P_FULL + p), ((t - 2) >> 1) & 1));
      if (!__all_sync(kFull, ok)) break;
      fence_after();
      const uint32_t ts = tmem + (uint32_t)(p * N);
      const uint64_t kd = kd0 + (uint64_t)(sl * (L::k_bytes >> 4));
      if (one) {
        // S^T = K slot x (Q hi + Q lo); the scratch rows' second slot adds their lo
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma_f8(ts, kd + 2 * kk, qd0 + (uint64_t)(part * (L::q_bytes >> 4)) + 2 * kk, idesc,
                   part + kk == 0 ? 0u : 1u);
        if (t >= n_pre) {
          const uint64_t k2 = kd0 + (uint64_t)(((t + 1) % kRing) * (L::k_bytes >> 4));
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              mma_f8(ts, k2 + 2 * kk, qd0 + (uint64_t)(part * (L::q_bytes >> 4)) + 2 * kk, idesc, 1u);
        }
        mma_commit(bar(BAR_S_FULL + p));
        mma_commit(bar(BAR_K_EMPTY + sl));
      }
      __syncwarp();
    }
    if (!ok) flags[1] = 1;
  }

  // ------------------------------------------------------------- outputs
  else if (warp == kPv) {
    constexpr uint32_t idesc = (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(N >> 3) << 17) |
                               ((uint32_t)(kKeys >> 4) << 24);
    const uint64_t vd0 = smem_desc(sbase + L::off_v, kHalf, 1024);
    // P^T: 8x8 cores, the key groups of 8 columns contiguous (tsd_verify_tc.cu)
    const uint64_t pd0 = smem_desc_interleave(sbase + L::off_p, 128, 2048);
    const bool one = elect_one();
    bool ok = true;
    for (int t = 0; t < ntiles; ++t) {
      const int p = t & 1;
      const uint32_t par = (t >> 1) & 1;
      ok = wait_ready(bar(BAR_V_FULL + p), par) && wait_ready(bar(BAR_P_FULL + p), par) && !flags[1];
      if (!__all_sync(kFull, ok)) break;
      fence_after();
      const uint64_t vd = vd0 + (uint64_t)(p * (kTile >> 4));
      const uint64_t pd = pd0 + (uint64_t)(p * (L::pt_bytes >> 4));
      const uint32_t to = tmem + (uint32_t)((2 + p) * N);
      if (one) {
        mma_f16(to, vd, pd, idesc, t < 2 ? 0u : 1u);
#pragma unroll
        for (int kk = 1; kk < kKeys / 16; ++kk)
          mma_f16_acc(to, vd + 128 * kk, pd + (uint64_t)(16 * kk), idesc);
        mma_commit(bar(BAR_V_EMPTY + p));
        if (t == ntiles - 1) mma_commit(bar(BAR_O_DONE));
      }
      __syncwarp();
    }
    if (!ok) flags[1] = 1;
  }

  // -------------------------------------------------------------- softmax
  else {
    const int p = warp >> 2, q = warp & 3;       // stream p: tiles of parity p
    const int key = q * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    float* const m_run = (float*)(smem + L::off_m) + p * N;
    float* const alpha = (float*)(smem + L::off_alpha) + p * N;
    float* const negm = (float*)(smem + L::off_negm) + p * N;
    float* const shiftv = (float*)(smem + L::off_shift) + p * N;
    float* const red = (float*)(smem + L::off_red) + p * 4 * N;
    uint8_t* const pt = smem + L::off_p + p * L::pt_bytes + key * 16;
    float2 l2[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) l2[i] = make_float2(0.f, 0.f);
    bool failed = false;

    for (int t = p; t < ntiles; t += 2) {
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
      const bool ok = __all_sync(kFull, wait_ready(bar(BAR_S_FULL + p), (t >> 1) & 1));
      fence_after();
      // x = S^T * scale - m, and the largest x
      float v[N];
      if (ok) {
#pragma unroll
        for (int u = 0; u < N; u += 8) tmem_ld8(tm_s(p) + lane_off + u, v + u);
        tmem_wait_ld();
      }
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 nm = *(const float4*)(negm + i);
        const float4 c2 = *(const float4*)(c2v + i);
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
      if (key >= nvalid) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = -INFINITY;
      } else if (is_tree && key > 0) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (!((rmask[i] >> (key - 1)) & 1ull)) v[i] = -INFINITY;
      }
      float tmax = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; i += 2) tmax = max3f(tmax, v[i], v[i + 1]);

      const bool local_stop = !ok || failed;
      if (wg_bar_or(p, local_stop || t == p || tmax > kOverflow)) {
        if (wg_bar_or(p, local_stop)) {
          failed = true;
          break;
        }
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          float r4[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
          const float r = warp_reduce_scatter<4, true>(r4, lane);
          if (lane < 4) red[q * N + i + lane] = r;
        }
        wg_bar(p);
        if ((tid & 127) < N) {
          const int n = tid & 127;
          float X = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) X = fmaxf(X, red[w * N + n]);
          const float m_old = m_run[n];
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
          m_run[n] = m_new;
          alpha[n] = al;
          shiftv[n] = sh;
          negm[n] = m_new == -INFINITY ? 0.f : -m_new;
        }
        wg_bar(p);
        // the stream's product before must be done before its columns are scaled
        if (t > p && !__all_sync(kFull, wait_ready(bar(BAR_V_EMPTY + p), ((t - 2) >> 1) & 1)))
          failed = true;
        fence_after();
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const float2 sh = *(const float2*)(shiftv + i), al = *(const float2*)(alpha + i);
          v[i] -= sh.x;
          v[i + 1] -= sh.y;
          l2[i / 2] = __fmul2_rn(l2[i / 2], al);
        }
        if (t > p && !failed) {
#pragma unroll 1
          for (int u = 0; u < N; u += 8) {
            float o[8];
            tmem_ld8(tm_o(p) + lane_off + u, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= alpha[u + e];
            tmem_st8(tm_o(p) + lane_off + u, o);
          }
          tmem_wait_st();
        }
      }
      // P^T's buffer was last read by the stream's product before
      if (t > p && !__all_sync(kFull, wait_ready(bar(BAR_V_EMPTY + p), ((t - 2) >> 1) & 1))) failed = true;
#pragma unroll
      for (int u = 0; u < N; u += 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 pr = make_float2(ex2(v[u + 2 * i]), ex2(v[u + 2 * i + 1]));
          l2[u / 2 + i] = __fadd2_rn(l2[u / 2 + i], pr);
          const float2 pv = __fmul2_rn(pr, fv2);
          w[i] = pack_half2(pv.x, pv.y);
        }
        if (!failed) *(uint4*)(pt + 256 * u) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_P_FULL + p));
    }

    // ------------------------------------- epilogue: the two streams joined
    failed = __any_sync(kFull, failed);
    const bool ok = !failed && __all_sync(kFull, wait_timed(bar(BAR_O_DONE), 0));
    fence_after();
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      float r4[4] = {l2[i / 2].x, l2[i / 2].y, l2[i / 2 + 1].x, l2[i / 2 + 1].y};
      const float r = warp_reduce_scatter<4, false>(r4, lane);
      if (lane < 4) red[q * N + i + lane] = r;
    }
    wg_bar(p);
    if ((tid & 127) < N) {
      const int n = tid & 127;
      float ls = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) ls += red[w * N + n];
      ((float*)(smem + L::off_l))[p * N + n] = ls;
    }
    uint32_t stop;
    asm volatile(
        "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n"
        " bar.red.or.pred po, 3, 256, pi;\n selp.u32 %0, 1, 0, po;\n}\n"
        : "=r"(stop)
        : "r"((uint32_t)(!ok || flags[1] != 0))
        : "memory");
    if (stop == 0) {
      // a thread per column: the streams' shares, and where the column goes
      const float unit = pow2i(U);
      float* const share0 = (float*)(smem + L::off_alpha);
      long long* const to = (long long*)rmask;
      if (tid < a.M) {
        const float* const ms = (const float*)(smem + L::off_m);
        const float* const ls = (const float*)(smem + L::off_l);
        const float m0 = ms[tid], m1 = ms[N + tid], top = fmaxf(m0, m1);
        // (a NaN sum stays one)
        const float w0 = m0 == -INFINITY ? (ls[tid] != ls[tid] ? ls[tid] : 0.f) : ex2(m0 - top);
        const float w1 = m1 == -INFINITY ? (ls[N + tid] != ls[N + tid] ? ls[N + tid] : 0.f) : ex2(m1 - top);
        const float total = w0 * ls[tid] + w1 * ls[N + tid];
        const float inv = pow2i(-kHeadroom) / total;
        share0[tid] = w0 * inv;
        share0[N + tid] = w1 * inv;
        const float lse2 = top + log2f(total);
        const int tr = tid / a.g, qh = hk * a.g + tid % a.g;
        const long orow = ((long)b * a.R + tr) * a.Hq + qh;
        const long prow = (((long)b * a.Hq + qh) * a.R + tr) * a.nsplit + sp;
        to[tid] = (nsb == 1 ? orow : prow) * D;
        if (nsb == 1) a.lse[orow] = lse2 * 0.69314718055994531f;
        else a.part_meta[prow] = make_float2(lse2, unit);
      }
      asm volatile("bar.sync 3, 256;\n" ::: "memory");
      // O^T lane = dim; stream p writes the octets of columns of its parity.  A
      // split's output, over 2^U, is a mean of numbers of magnitude < 512: fp16
      // holds it to 2^-12.
#pragma unroll 1
      for (int u = 8 * p; u < min(N, a.M); u += 16) {
        float o0[8], o1[8];
        tmem_ld8(tm_o(0) + lane_off + u, o0);
        if (ntiles > 1) tmem_ld8(tm_o(1) + lane_off + u, o1);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int col = u + e;
          if (col >= a.M || key >= D) break;
          float res = o0[e] * share0[col];
          if (ntiles > 1) res += o1[e] * share0[N + col];
          if (nsb == 1) ((__nv_bfloat16*)a.out)[to[col] + key] = __float2bfloat16_rn(res * unit);
          else ((__half*)a.part_o)[to[col] + key] = __float2half_rn(res);
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
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;\n" ::"r"(tmem));
  }
}

template <int D>
void launch_few(const CUtensorMap& kmap, const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  const uint32_t smem = FewLayout<D>::total + 1024;
  const auto kern = a.wait_cycles < kWaitCycles ? q8_few_kernel<D, true> : q8_few_kernel<D, false>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  launch(kern, dim3(a.map.Hkv, p.nsplit, a.B), dim3(kThreads), smem, st, kmap, a);
}

}  // namespace

bool launch_q8_few(const tsd_attn_desc& d, const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  CUtensorMap m;
  if (encode_fn() == nullptr || !encode_keys(&m, a, d.dk, d.dk)) return false;
  if (d.dk == 128) launch_few<128>(m, a, p, st);
  else launch_few<64>(m, a, p, st);
  return true;
}

}  // namespace tsd
