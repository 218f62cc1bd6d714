// tcgen05 path of tsd_tree_verify_attn_q8 for bf16 heads of 64 or 128 dims with
// more packed rows (R tree rows x g query heads of a KV head) than
// tsd_q8_few.cu takes: up to 128 per CTA, on the lanes of the tensor memory.
//
//   S[n][key]  = Q . K_tile^T      M = 128 packed rows, N = 128 keys, K = d
//   O[n][dim] += P . V_tile        M = 128 packed rows, N = d, K = 128 keys
//
// A thread owns one packed row: its maximum, its sum and its rescaling need no
// other thread (with keys on lanes, as in tsd_verify_tc.cu, each is a reduction
// across a warpgroup, and a probability costs about twice the instructions: the
// 65-row trees over 8 x 32k keys took 555 us that way).  P goes back to the
// tensor memory and is the product's left operand there: no shared memory and no
// barrier among the softmax warps.  Warps whose 32 rows are all behind the last
// one do nothing.
//
// Numbers.
//   S      kind::f8f6f4: the K tile's codes as they are in the cache, and Q as
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
// V is widened by warps and not taken in 8 bits: kind::f8f6f4 would need P in 8
// bits.  Two e4m3 terms as for Q do not do: P spans 2^-32..2^8, and what lies
// below 2^-17 of the largest would be lost from long flat rows.
//
// Two streams.  The two halves of a tile (64 keys each) have scores, a softmax
// warpgroup, P, an accumulator, a maximum and a sum each, joined at the end.  A softmax
// thread first takes its 64 scores into registers, so that the tensor core can
// compute the next tile's over them while the softmax runs, and waits for its
// product before only behind the first 32 exponentials.  (With P over the scores it
// came from, the next scores waited for the product with V; with one product for both
// halves' scores, the streams wait for each other: 329 us instead of 321 for the
// 65-row trees below, although the tensor core then needs 1024 cycles a tile and not
// 1280.)  The running maximum is lazy: a row keeps it until a tile's largest score
// passes it by 8 (in log2), so that its accumulator is rescaled rarely.  Q (hi, lo) is
// in the tensor memory too, which leaves the shared memory's 128 bytes a cycle to K
// and V.
//
// Roles (512 threads: 128 registers each, which the softmax needs; with three more
// widening warps and 96 registers a tile took 10% longer): warps 0-3 and 4-7 softmax
// and epilogue; warp 8 issues the products with V and owns the tensor memory, warp 9
// those with Q; one thread of warp 10 loads K tiles by TMA into a ring of four; warps
// 11-15 load V tiles straight into registers, a tile ahead (behind L2 prefetches), and
// widen them into three fp16 stages (two: 325 us), laid out as the product reads them
// (rows of 64 elements, 128-byte swizzle).  mbarriers order K -> S -> softmax -> O and
// V -> O; every wait is bounded.
//
// What bounds it: the way of a tile through a stream, about 1600 cycles from its scores
// to its P with few warps to hide latencies: an access to shared memory takes 300
// cycles beside the widening's stores and the products' reads, and five roles of
// unrolled code pass through the instruction cache (which is why set-up loops are
// rolled and the scratch rows' tile has code of its own: 341 -> 321 us).  The tensor
// core needs 1280 cycles (8 products with Q of 128 x 64 at 48 cycles for each half, 8
// with V of 128 x 128 at 64), the cache's bytes 1405.  Set-up and epilogue take 13000
// cycles per CTA.  8 x 65 rows of 32 heads over 32k keys: 321 us, 870 TFLOP/s; 32 x 33
// rows over 1k to 4k keys: 104 us; 8 x 8 rows over 32k keys: 121 us, 4.4 TB/s.
#include <type_traits>

#include "tsd_common.cuh"
#include "tsd_host.h"
#include "tsd_q8_tc.cuh"

namespace tsd {
namespace {

constexpr int kPv = 8, kQk = 9, kTma = 10, kWide = 11, kWideWarps = 5;
constexpr int kWideThreads = kWideWarps * 32;
constexpr int kThreads = (kWide + kWideWarps) * 32;
constexpr int kStages = 3;                      // widened V tiles
constexpr int kRows = 128;
// Tensor memory columns: a tile's scores (128), Q (hi, lo: 64), the streams' P (32
// each), the accumulators (d each).
constexpr uint32_t kColQ = 128, kColP = 192, kColO = 256;

template <int D>
struct RowLayout {
  static constexpr uint32_t k_bytes = kKeys * D;
  static constexpr uint32_t v_bytes = kKeys * D * 2;
  static constexpr uint32_t off_k = 0;
  static constexpr uint32_t off_v = kRing * k_bytes;
  static constexpr uint32_t off_ml = off_v + kStages * v_bytes;        // float2[2][128] (m, l)
  static constexpr uint32_t off_rows = off_ml + 16 * kRows;            // i64[kMaxTiles]
  static constexpr uint32_t off_tree = off_rows + 8 * kMaxTiles;       // 4 x 32 bits [128]
  static constexpr uint32_t off_kex = off_tree + 16 * kKeys;           // u8[2 kMaxTiles]
  static constexpr uint32_t off_vex = off_kex + 2 * kMaxTiles;
  static constexpr uint32_t off_bar = off_vex + 2 * kMaxTiles;
  static constexpr int nbar = 26;
  static constexpr uint32_t off_flags = off_bar + 8 * nbar;            // tmem, abort
  static constexpr uint32_t off_top = off_flags + 8;                   // int[kWideWarps]
  static constexpr uint32_t off_req = off_top + 4 * kWideWarps;  // request, its length
  static constexpr uint32_t total = off_req + 8;
  static_assert(total + 1024 <= 232448, "shared memory budget");
  static_assert(kTreeBytes<D> <= v_bytes && kStages > 1, "the scan's rows");
};

// FULL: the copy landed, the warps wrote or the product is done; EMPTY: read by
// the product (S_EMPTY: by the softmax).  S, P_FULL and PV_DONE: one per stream.
// T_FULL: the scratch rows' keys, which take the two K slots behind the last
// prefix tile (hi, lo).  FINAL: one per issuing warp.
enum { BAR_K_FULL = 0, BAR_K_EMPTY = 4, BAR_V_FULL = 8, BAR_V_EMPTY = 11, BAR_S_FULL = 14,
       BAR_S_EMPTY = 16, BAR_P_FULL = 18, BAR_PV_DONE = 20, BAR_O_DONE = 22, BAR_T_FULL = 23,
       BAR_FINAL = 24 };

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// D (+)= A.B with A in tensor memory: fp16 (two to a column), or e4m3 (four).
__device__ __forceinline__ void mma_f8_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}

template <int D, bool kPoll>
__global__ void __launch_bounds__(kThreads, 1)
q8_rows_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ Q8AttnArgs a) {
  using L = RowLayout<D>;
  if (threadIdx.x == kTma * 32) tma_desc_prefetch(&kmap);
  grid_dependency_sync();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = su32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  float2* s_ml = (float2*)(smem + L::off_ml);
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
  const int hk = blockIdx.x / a.nrg, rg = blockIdx.x % a.nrg, sp = blockIdx.y;
  int P;
  const int b = request_at(a, blockIdx.z, P, (volatile int*)(smem + L::off_req));
  const int nsb = q8_splits(a, P);
  if (sp >= nsb) return;
  const int k0 = min(sp * a.split_len, P), k1 = min(P, k0 + a.split_len);
  const int n_pre = (k1 - k0 + kKeys - 1) / kKeys;
  const bool with_tree = sp == nsb - 1;             // R <= 65 < 128: one tile
  const int ntiles = n_pre + (with_tree ? 1 : 0);
  const int row_base = rg * a.rb;
  const int rows_here = min(a.rb, a.M - row_base);
  const int live_warps = (rows_here + 31) / 32;     // softmax warps of a stream with rows
  auto valid_of = [&](int t) { return min(kKeys, k1 - (k0 + t * kKeys)); };

  // ---------------------------------------------------------------- set-up
  // Everything that the first products need is requested at once, by the warps
  // that will use it, and ready at one barrier.
  const int wt = tid - kWide * 32;
  using Share = WideShare<D / 16, kWideThreads>;
  const Share share(wt);
  uint64_t mask = 0ull;     // softmax threads: the scratch rows that the row sees,
  float c2 = 0.f;           // and the factor of its scores
  uint4 vreg[Share::kCount];
  // the tile at cache row `row` (a missing page: none)
  auto load_v = [&](long row, int nvalid) {
    share.template load<D>(vreg, a.vc + (row < 0 ? 0 : row) * D, row < 0 ? 0 : nvalid);
  };

  if (warp >= kWide) {
    // the first V tile, the exponents and rows of the split's tiles, the scratch rows
    if (with_tree) tree_fetch<D, kWideThreads>(a, b, hk, wt, sbase + L::off_v, L::v_bytes);
    const long r0 = n_pre > 0 ? a.map.row(b, hk, k0) : -1;
    const long rt = wt < n_pre ? a.map.row(b, hk, k0 + wt * kKeys) : -1;
    if (n_pre > 0) load_v(r0, valid_of(0));
    int top = -1000;
#pragma unroll 1
    for (int t = wt; t < n_pre; t += kWideThreads) {
      const int pos = k0 + t * kKeys;
      const long r = t == wt ? rt : a.map.row(b, hk, pos);
      tile_row[t] = r;
      if (r < 0) report_error(a.err, TSD_DEV_ERR_BAD_PAGE, b);
      const long e = a.map.block_at(b, hk, pos, r);
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
    if (with_tree)
      top = max(top, tree_scan<D, kWideThreads>(a, b, wt, smem + L::off_v, L::v_bytes, kt_in, vt_in,
                                                kt_out, vt_u));
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) s_top[warp - kWide] = top;
  } else if (warp < 8) {
    // Q into the tensor memory: a thread takes its packed row, whose largest element
    // scales it, and splits the stream's half of it; and what the row sees
    const int q = warp & 3, p = warp >> 2, row = q * 32 + lane;
    if (q < live_warps) {
      uint4 w[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row < rows_here) {
        const int pr = row_base + row, tr = pr / a.g, qh = hk * a.g + pr % a.g;
        const uint4* src =
            (const uint4*)((const __nv_bfloat16*)a.q + (((long)b * a.R + tr) * a.Hq + qh) * D);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) w[i] = __ldg(src + i);
        mask = tr > 0 ? a.mask[(long)b * a.R + tr] : 0ull;
      }
      uint32_t qtop = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) qtop = top_pairs(qtop, w[i]);
      qtop = top_of(qtop);
      const bool bad = qtop >= 0x7f800000u;
      const int qe = row_exponent(qtop);
      const float f = bad ? 0.f : q8_scale(261 - qe);
      c2 = bad ? __int_as_float(0x7fffffff) : a.qscale * q8_scale(qe - 7);
      __syncwarp();
      asm volatile("bar.sync 2, %0;\n" ::"r"(64 * live_warps + 32) : "memory");   // (allocated)
      const uint32_t tq = flags[0] + kColQ + p * (D / 8) + ((uint32_t)(q * 32) << 16);
      uint4 x[D / 16];                             // the stream's half
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        x[i] = p ? w[D / 16 + i] : w[i];
        if (bad) x[i] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {           // 16 elements: four columns of hi, four of lo
        uint4 hi, lo;
        split16({x[0], x[1]}, f, hi, lo);
        tmem_st4(tq + 4 * c, __uint_as_float(hi.x), __uint_as_float(hi.y), __uint_as_float(hi.z),
                 __uint_as_float(hi.w));
        tmem_st4(tq + D / 4 + 4 * c, __uint_as_float(lo.x), __uint_as_float(lo.y),
                 __uint_as_float(lo.z), __uint_as_float(lo.w));
#pragma unroll
        for (int i = 0; i + 2 < D / 16; ++i) x[i] = x[i + 2];
      }
      tmem_wait_st();
    }
  } else if (warp == kTma) {
    long row = 0;                                    // of the ring's tiles
    if (a.map.page_size && lane < kRing && lane < n_pre) row = a.map.row(b, hk, k0 + lane * kKeys);
    if (lane == 0) {
      for (int i = 0; i < kRing; ++i) {
        mbar_init(bar(BAR_K_FULL + i), 1);
        mbar_init(bar(BAR_K_EMPTY + i), 1);
      }
      for (int i = 0; i < kStages; ++i) {
        mbar_init(bar(BAR_V_FULL + i), kWideWarps);
        mbar_init(bar(BAR_V_EMPTY + i), 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(BAR_P_FULL + i), live_warps);
        mbar_init(bar(BAR_PV_DONE + i), 1);
        mbar_init(bar(BAR_FINAL + i), 1);
        mbar_init(bar(BAR_S_FULL + i), 1);
        mbar_init(bar(BAR_S_EMPTY + i), live_warps);
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
  } else if (warp == kPv) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
        sbase + L::off_flags));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    asm volatile("bar.arrive 2, %0;\n" ::"r"(64 * live_warps + 32) : "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = flags[0];
  int U = s_top[0];
#pragma unroll
  for (int i = 1; i < kWideWarps; ++i) U = max(U, s_top[i]);
  auto tm_o = [&](int p) { return tmem + kColO + (uint32_t)(p * D); };

  // -------------------------------------------------------------- K tiles
  if (warp == kTma) {
    if (lane == 0) {
      for (int i = 1; i < kPrefetch; ++i)
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
    const int tree_at = max(n_pre - 2, 0);     // the tree's keys are made two tiles early
    for (int t = 0; t < ntiles; ++t) {
      const int st = t % kStages;
      if (with_tree && t == tree_at) {
        const int s0 = n_pre, s1 = n_pre + 1;
        if ((s0 >= kRing && !__all_sync(kFull, wait_timed(bar(BAR_K_EMPTY + s0 % kRing),
                                                         (s0 / kRing - 1) & 1))) ||
            (s1 >= kRing && !__all_sync(kFull, wait_timed(bar(BAR_K_EMPTY + s1 % kRing),
                                                         (s1 / kRing - 1) & 1)))) {
          flags[1] = 1;
          break;
        }
        tree_keys<D>(a, b, hk, wt, kWideThreads, kt_in,
                     smem + L::off_k + (s0 % kRing) * L::k_bytes,
                     smem + L::off_k + (s1 % kRing) * L::k_bytes);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_T_FULL));
      }
      if (t >= kStages &&
          !__all_sync(kFull, wait_ready(bar(BAR_V_EMPTY + st), (t / kStages - 1) & 1))) {
        flags[1] = 1;
        break;
      }
      uint8_t* const stage = smem + L::off_v + st * L::v_bytes;
      if (t < n_pre) {
        share.widen(vreg, stage);
      } else {
        tree_values<D>(a, b, hk, wt, kWideThreads, vt_in, stage);
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_V_FULL + st));
      if (t + 1 < n_pre) load_v(tile_row[t + 1], valid_of(t + 1));
      if (__any_sync(kFull, flags[1] != 0)) break;
    }
  }

  // ------------------------------------------------------------- scores
  else if (warp == kQk) {
    // fp32 accumulator; e4m3 operands are format 0
    constexpr uint32_t idesc =
        (1u << 4) | ((uint32_t)(kKeys / 2 >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
    constexpr uint32_t kHalfTile = L::k_bytes / 2 >> 4;
    const uint64_t kd0 = row_desc<D>(sbase + L::off_k);
    const uint32_t tq = tmem + kColQ;
    const bool one = elect_one();
    bool ok = true;
    for (int t = 0; ok && t < ntiles; ++t) {
      const int sl = t % kRing;
      ok = t < n_pre ? wait_ready(bar(BAR_K_FULL + sl), (t / kRing) & 1)
                     : wait_ready(bar(BAR_T_FULL), 0);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        ok = ok && (t == 0 || wait_ready(bar(BAR_S_EMPTY + p), (t - 1) & 1));
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        fence_after();
        const uint64_t kd = kd0 + (uint64_t)(sl * (L::k_bytes >> 4) + p * kHalfTile);
        const uint32_t ts = tmem + 64u * p;
        if (one) {
          // S = (Q hi + Q lo) x K slot; the scratch rows' second slot adds their lo
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              mma_f8_ta(ts, tq + part * (D / 4) + 8 * kk, kd + 2 * kk, idesc, part + kk == 0 ? 0u : 1u);
          if (t >= n_pre) {
            const uint64_t k2 = kd0 + (uint64_t)(((t + 1) % kRing) * (L::k_bytes >> 4) + p * kHalfTile);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_f8_ta(ts, tq + part * (D / 4) + 8 * kk, k2 + 2 * kk, idesc, 1u);
          }
          mma_commit(bar(BAR_S_FULL + p));
          if (p == 1) mma_commit(bar(BAR_K_EMPTY + sl));
        }
        __syncwarp();
      }
    }
    if (!ok) flags[1] = 1;
  }

  // ------------------------------------------------------------- outputs
  else if (warp == kPv) {
    // fp16 operands are format 0; B (V) is N-major
    constexpr uint32_t idesc =
        (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
    const uint64_t vd0 = smem_desc(sbase + L::off_v, kHalf, 1024);
    const bool one = elect_one();
    bool ok = true;
    for (int t = 0; ok && t < ntiles; ++t) {
      const int st = t % kStages;
      const uint64_t vd = vd0 + (uint64_t)(st * (L::v_bytes >> 4));
      ok = wait_ready(bar(BAR_V_FULL + st), (t / kStages) & 1) && !flags[1];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        ok = ok && wait_ready(bar(BAR_P_FULL + p), t & 1);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        fence_after();
        if (one) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_ta(tm_o(p), tmem + kColP + 32 * p + 8 * kk, vd + 128 * (4 * p + kk), idesc,
                       t == 0 && kk == 0 ? 0u : 1u);
          mma_commit(bar(BAR_PV_DONE + p));
          if (p == 1) {
            mma_commit(bar(BAR_V_EMPTY + st));
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
    const int p = warp >> 2, q = warp & 3, row = q * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    float m = -INFINITY, l = 0.f;
    bool failed = false;
    if (q < live_warps) {
      // The stream's product of the tile before: done before its P is written over
      // or its accumulator is rescaled.
      bool done = true;
      auto product_done = [&](int t) -> bool {
        return __all_sync(kFull, done || wait_ready(bar(BAR_PV_DONE + p), (t - 1) & 1));
      };
      // The maximum is raised to X where X passes m by the headroom (or m is none),
      // the sum and the accumulator are rescaled.
      auto raise = [&](float X, int t) -> bool {
        const bool need = !(X <= m + kOverflow);
        if (__builtin_expect(!__any_sync(kFull, need), 1)) return true;
        if (!product_done(t)) return false;
        const float m_new = need ? fmaxf(m, X) : m;
        const float al = m_new == m ? 1.f : m == -INFINITY ? 0.f : ex2(m - m_new);
        m = m_new;
        l *= al;
        if (t == 0) return true;
        fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          uint32_t w[16];
          tmem_ld8(tm_o(p) + lane_off + c, o);
          tmem_ld8(tm_o(p) + lane_off + c + 8, o + 8);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * al);
          tmem_st16(tm_o(p) + lane_off + c, w);
        }
        tmem_wait_st();
        return true;
      };
      // the scores have been read: their columns may take the next tile's
      auto scores_read = [&] {
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_S_EMPTY + p));
      };

      const int h = p;                           // a stream takes one half of every tile
      const uint32_t ts = tmem + lane_off + 64u * h, tp = tmem + lane_off + kColP + 32u * p;
      // what the next tile needs from shared memory is asked for a tile early
      bool ready = false;                        // its scores
      int ke = kex[h], ve = vex[h];              // its exponents
      // (the scratch rows' tile has code of its own: the loop over the prefix stays small)
      auto tile = [&](int t, auto tree) -> bool {
        constexpr bool is_tree = decltype(tree)::value;
        const int nvalid = is_tree ? a.R : valid_of(t);
        if (t > 0) done = complete(bar(BAR_PV_DONE + p), (t - 1) & 1);
        if (!__all_sync(kFull, ready || wait_ready(bar(BAR_S_FULL + p), t & 1))) return false;
        fence_after();
        const int nv = min(nvalid - 64 * h, 64);   // keys of this half
        float v[64];
        tmem_ld32(ts, *(float(*)[32])v);
        tmem_ld32(ts + 32, *(float(*)[32])(v + 32));
        tmem_wait_ld();
        scores_read();
        // x = f v + off.  A prefix block has one factor and one offset.  (Not 0, so
        // that -inf stays -inf; an offset below -60 puts P under fp16's range: its
        // exact value does not matter, and the sum stays within fp32.)
        float f = 1.f;
        int d = 0;
        if constexpr (!is_tree) {
          f = c2 * q8_scale(ke);
          f = f == 0.f ? 1.17549435e-38f : f;
          d = max(ve - 127 - U + kHeadroom, -60);
          const int next = 2 * min(t + 1, kMaxTiles - 1) + h;
          ke = kex[next];
          ve = vex[next];
          if (__builtin_expect(nv < 64, 0)) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= nv) v[i] = -INFINITY;
          }
        } else {
          // scratch rows: a factor per key, and what this row sees (key 0: the root)
          const uint64_t vis = nv <= 0 ? 0ull
                               : (h == 0 ? (mask << 1) | 1ull : mask >> 63) & (~0ull >> (64 - nv));
          const uint32_t vlo = (uint32_t)vis, vhi = (uint32_t)(vis >> 32);
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const float4 k4 = *(const float4*)(kt_out + 64 * h + i);
            const float kf[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t word = i + j < 32 ? vlo : vhi;
              const bool sees = (word >> ((i + j) & 31)) & 1u;
              v[i + j] = sees ? v[i + j] * (c2 * kf[j]) : -INFINITY;
            }
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 64; i += 8)
#pragma unroll
          for (int j = 0; j < 4; ++j) top[j] = max3f(top[j], v[i + 2 * j], v[i + 2 * j + 1]);
        if (!raise(f * fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), t)) return false;
        const float off = (float)d - (m == -INFINITY ? 0.f : m);
        const float2 f2 = make_float2(f, f), o2 = make_float2(off, off);
        float2 sa = make_float2(0.f, 0.f), sb = sa;
        auto weights = [&](auto scaled) {          // scaled: a factor per value row
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t w[16];                        // (32 exponentials hide the product's wait)
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float2 xa = __ffma2_rn(make_float2(v[c + i], v[c + i + 1]), f2, o2);
              const float2 xb = __ffma2_rn(make_float2(v[c + i + 2], v[c + i + 3]), f2, o2);
              float2 pa = make_float2(ex2(xa.x), ex2(xa.y));
              float2 pb = make_float2(ex2(xb.x), ex2(xb.y));
              sa = __fadd2_rn(sa, pa);
              sb = __fadd2_rn(sb, pb);
              if constexpr (decltype(scaled)::value) {
                const int4 u = *(const int4*)(vt_u + 64 * h + c + i);
                pa.x *= pow2i(u.x - U + kHeadroom);
                pa.y *= pow2i(u.y - U + kHeadroom);
                pb.x *= pow2i(u.z - U + kHeadroom);
                pb.y *= pow2i(u.w - U + kHeadroom);
              }
              w[i / 2] = pack_half2(pa.x, pa.y);
              w[i / 2 + 1] = pack_half2(pb.x, pb.y);
            }
            if (c == 0) {
              if (!product_done(t)) return false;
              fence_after();
            }
            tmem_st16(tp + c / 2, w);
            if (c == 0) ready = complete(bar(BAR_S_FULL + p), (t + 1) & 1);
          }
          return true;
        };
        if (!weights(tree)) return false;
        l = fmaf((sa.x + sa.y) + (sb.x + sb.y), pow2i(-d), l);
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_P_FULL + p));
        return true;
      };
      for (int t = 0; t < n_pre && !failed; ++t) failed = !tile(t, std::false_type{});
      if (with_tree && !failed) failed = !tile(n_pre, std::true_type{});
    }

    // ------------------------------------- epilogue: the two streams joined
    const bool ok = !failed && __all_sync(kFull, wait_timed(bar(BAR_O_DONE), 0));
    fence_after();
    s_ml[p * kRows + row] = make_float2(m, l);
    uint32_t stop;
    asm volatile(
        "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n"
        " bar.red.or.pred po, 1, 256, pi;\n selp.u32 %0, 1, 0, po;\n}\n"
        : "=r"(stop)
        : "r"((uint32_t)(!ok || flags[1] != 0))
        : "memory");
    if (stop == 0 && q < live_warps) {
      const float2 s0 = s_ml[row], s1 = s_ml[kRows + row];
      const float top = fmaxf(s0.x, s1.x);
      const float w0 = s0.x == -INFINITY ? (s0.y != s0.y ? s0.y : 0.f) : ex2(s0.x - top);
      const float w1 = s1.x == -INFINITY ? (s1.y != s1.y ? s1.y : 0.f) : ex2(s1.x - top);
      const float total = w0 * s0.y + w1 * s1.y;
      const float unit = pow2i(U), inv = pow2i(-kHeadroom) / total;
      const float g0 = w0 * inv, g1 = w1 * inv;
      const float lse2 = top + log2f(total);
      const int pr = row_base + min(row, rows_here - 1);
      const int tr = pr / a.g, qh = hk * a.g + pr % a.g;
      const long orow = ((long)b * a.R + tr) * a.Hq + qh;
      const long prow = (((long)b * a.Hq + qh) * a.R + tr) * a.nsplit + sp;
      const bool mine = row < rows_here;
      if (mine && p == 0) {
        if (nsb == 1) a.lse[orow] = lse2 * 0.69314718055994531f;
        else a.part_meta[prow] = make_float2(lse2, unit);
      }
      // stream p writes the dims [p D/2, (p + 1) D/2).  A split's output, over
      // 2^U, is a mean of numbers of magnitude < 512: fp16 holds it to 2^-12.
#pragma unroll 1
      for (int c = p * (D / 2); c < (p + 1) * (D / 2); c += 32) {
        float o0[32], o1[32];
        tmem_ld32(tm_o(0) + lane_off + c, o0);
        tmem_ld32(tm_o(1) + lane_off + c, o1);
        tmem_wait_ld();
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float x = o0[i] * g0 + o1[i] * g1, y = o0[i + 1] * g0 + o1[i + 1] * g1;
          w[i / 2] = nsb == 1 ? pack_bf16x2(x * unit, y * unit) : pack_half2(x, y);
        }
        if (mine) {
          uint4* dst = nsb == 1 ? (uint4*)((__nv_bfloat16*)a.out + orow * D + c)
                                : (uint4*)((__half*)a.part_o + prow * D + c);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      }
    }
    if (!ok && lane == 0) flags[1] = 1;
  }

  // --------------------------------------------------------------- teardown
  // Products in flight: the issuing warps wait for a commit of their own.
  if (warp == kPv || warp == kQk) {
    if (elect_one()) mma_commit(bar(BAR_FINAL + warp - kPv));
    __syncwarp();
    mbar_wait(bar(BAR_FINAL + warp - kPv), 0);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (flags[1] && tid == 0) report_error(a.err, TSD_DEV_ERR_TIMEOUT, b);
  fence_after();
  if (warp == kPv) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
  }
}

template <int D>
void launch_rows(const CUtensorMap& kmap, const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  const uint32_t smem = RowLayout<D>::total + 1024;
  const auto kern = a.wait_cycles < kWaitCycles ? q8_rows_kernel<D, true> : q8_rows_kernel<D, false>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  launch(kern, dim3(a.map.Hkv * p.nrg, p.nsplit, a.B), dim3(kThreads), smem, st, kmap, a);
}

}  // namespace

bool launch_q8_rows(const tsd_attn_desc& d, const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  CUtensorMap m;
  if (encode_fn() == nullptr || !encode_keys(&m, a, d.dk, d.dk)) return false;
  if (d.dk == 128) launch_rows<128>(m, a, p, st);
  else launch_rows<64>(m, a, p, st);
  return true;
}

}  // namespace tsd
