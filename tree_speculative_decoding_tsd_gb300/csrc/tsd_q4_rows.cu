// tcgen05 path of tsd_tree_verify_attn_q4 for bf16 heads of 64 or 128 dims with more packed
// rows (R tree rows x g query heads of a KV head) than tsd_q4_few.cu takes: up to 128 per
// CTA, on the lanes of the tensor memory.
//
//   S[n][key]  = Q . K_tile^T      M = 128 packed rows, N = 128 keys, K = d
//   O[n][dim] += P . V_tile        M = 128 packed rows, N = d, K = 128 keys
//
// The layout, the two streams (the halves of a tile have a softmax warpgroup, scores, P, an
// accumulator, a bound and a sum each) and the lazy bound are those of tsd_q8_tc.cu.  Here
// both K and V are widened to fp16 by warps, straight from global memory through
// registers into shared memory (rows of 64 elements, 128-byte swizzle: the same layout
// serves K, whose rows are the product's columns, and V, whose rows are summed over).
//
// Numbers.
//   K, V   fp16: (c - 8) s 2^(-E - 9), E the exponent above the tile's largest scale (K and V
//          apart), by one fused multiply-add of a masked word (tsd_q4.cuh): 2^-12, or 2^-25
//          (2^-18 of the tile's largest value) where that is more.
//   Q      fp16 times a power of two of its row (largest element into [2^14, 2^15)): exact
//          down to 2^-29 of it
//   tree   scratch rows of K and V in fp16, each times a power of two of its own
//   P      fp16: 2^(x + E - m + 7), m a running bound of x + E: 2^-12, and steps of 2^-24, 2^-39
//          of the largest.  Its sum has a bound of its own (kQ4Near).
// A score's factor takes the tile's and the row's power of two in fp32.
//
// Roles (640 threads): warps 0-3 and 4-7 softmax and epilogue; warp 8 issues the products
// with V and owns the tensor memory, warp 9 those with Q; warps 10 and 11 read the tiles'
// scales of K and V ahead, find E and leave fp16 factors in a ring; warps 12-15 widen K,
// 16-19 V.  Registers are dealt out anew at the start: the softmax needs 120.  mbarriers
// order scales -> K -> S -> softmax -> O and V -> O; every wait is bounded.  Of four widening
// warps two take the even tiles and two the odd ones: a tile's way through them is mostly
// latency (all four on each tile: 421 instead of 390 us for the trees below; one group of five
// warps for K and V in turn: 589).
//
// What bounds it: the way of a tile through a softmax warp, about 2000 cycles; K and V lie
// widened 2500 cycles before they are used.  Left out one at a time, 392 us become 331 without
// the widening, 380 without the scales, 373 without the maxima, 374 without the exponentials, 300
// without all of it: instructions and shared memory (64 KB stored and 64 KB read by products per
// tile, half of its rate) are shared by all roles.  The tensor core needs 1280 cycles a tile.
// 8 x 64 rows of 32 heads over 32k keys: 299 us, 920 TFLOP/s; 32 x 32 rows over 1k to 4k: 71 us;
// 8 x 32 rows over 32k: 153 us.  (292, 68, 149 with one bound for both sums and one power of two for
// all rows of a split.  The figures above: 8 x 65 rows in three groups of 87.)
// Tried and dropped: more of the widening on the scheduler that has no softmax warp (three of
// four have rows: 472 us), the next tile's scores asked for during a tile's exponentials (403).
#include <algorithm>
#include <type_traits>

#include "tsd_common.cuh"
#include "tsd_host.h"
#include "tsd_q4.cuh"
#include "tsd_q4_attn.cuh"
#include "tsd_q8_tc.cuh"

namespace tsd {
namespace {

constexpr int kPv = 8, kQk = 9, kScaleK = 10, kScaleV = 11, kWideK = 12, kWideV = 16;
constexpr int kWideWarps = 4;                   // of K, and of V
constexpr int kPair = 2;                        // of them work on one tile, the others on the next
constexpr int kWideThreads = kWideWarps * 32;
constexpr int kThreads = (kWideV + kWideWarps) * 32;
// Registers of a thread: as launched, and then of the softmax, of warps 8-11, of those that
// widen.  (136, 64, 72: 399 us instead of 390 for the 65-row trees.)
constexpr int kLaunchRegs = 96, kSoftRegs = 120, kMidRegs = 80, kWideRegs = 80;
static_assert(2 * kSoftRegs + kMidRegs + 2 * kWideRegs <= 5 * kLaunchRegs, "registers of the launch");
template <int N, bool kMore> __device__ __forceinline__ void set_registers() {
  if (kMore) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
constexpr int kStages = 3;                      // widened tiles of K, and of V
constexpr int kScaleRing = 4;                   // tiles of factors
constexpr int kRows = 128;
// Tensor memory columns: a tile's scores (128), Q (64), the streams' P (32 each), the
// accumulators (d each).
constexpr uint32_t kColQ = 128, kColP = 192, kColO = 256;

template <int D>
struct RowLayout {
  static constexpr int NG = D / kQ4Group;
  static constexpr uint32_t t_bytes = kKeys * D * 2;                   // a widened tile
  static constexpr uint32_t f_bytes = kKeys * NG * 2;                  // a tile's factors of K, or of V
  static constexpr uint32_t off_k = 0;
  static constexpr uint32_t off_v = kStages * t_bytes;
  static constexpr uint32_t off_f = off_v + kStages * t_bytes;         // fp16 [ring][K, V][128][NG]
  static constexpr uint32_t off_ml = off_f + kScaleRing * 2 * f_bytes; // float4[2][128] (m, l, u)
  static constexpr uint32_t off_eu = off_ml + 32 * kRows;              // float[2][128] (kQ4Near)
  static constexpr uint32_t off_rows = off_eu + 8 * kRows;             // i64[kMaxTiles]
  static constexpr uint32_t off_tree = off_rows + 8 * kMaxTiles;       // 4 x 32 bits [128]
  static constexpr uint32_t off_ek = off_tree + 16 * kKeys;            // i8[kMaxTiles]: E of K
  static constexpr uint32_t off_ev = off_ek + kMaxTiles;               // and of V
  static constexpr uint32_t off_near = off_ev + kMaxTiles;             // float[kMaxTiles]: E of V, or NaN
  static constexpr uint32_t off_bar = off_near + 4 * kMaxTiles;
  static constexpr int nbar = 32;
  static constexpr uint32_t off_flags = off_bar + 8 * nbar;            // tmem, abort
  static constexpr uint32_t off_top = off_flags + 8;                   // int[2 kWideWarps]
  static constexpr uint32_t off_req = off_top + 8 * kWideWarps;        // request, its length
  static constexpr uint32_t total = off_req + 8;
  static_assert(total + 1024 <= 232448, "shared memory budget");
  static_assert(kTreeBytes<D> <= t_bytes && kStages > 1, "the scan's rows");
};

// FULL: written, or the product is done; EMPTY: read (F_EMPTY: by the widening warps,
// S_EMPTY: by the softmax, the others: by the product).  S, P_FULL and PV_DONE: one per
// stream.  FINAL: one per issuing warp.
enum { BAR_K_FULL = 0, BAR_K_EMPTY = 3, BAR_V_FULL = 6, BAR_V_EMPTY = 9, BAR_F_FULL = 12,
       BAR_F_EMPTY = 16, BAR_S_FULL = 20, BAR_S_EMPTY = 22, BAR_P_FULL = 24, BAR_PV_DONE = 26,
       BAR_O_DONE = 28, BAR_FINAL = 29 };

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
// D (+)= A.B, fp16, with A in tensor memory (two elements to a column).
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
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

// A widening warp's share of a tile: 16-byte chunks (the 32 codes of a group) of eight (D =
// 128) or sixteen rows at a time, every kPair-th such block.  Eight lanes that store
// together hold two groups of a half row and four rows: their 16-byte units, permuted by
// the swizzle, fall on eight different columns.
template <int D>
struct Share4 {
  static constexpr int NG = D / kQ4Group;
  static constexpr int kBlockRows = 32 / NG, kBlocks = kKeys / kBlockRows;
  static constexpr int kCount = kBlocks / kPair;
  int row, grp, first;                             // within a block; the warp's first block
  uint32_t dst;                                    // the chunk's place in a stage, but for the units
  __device__ __forceinline__ Share4(int warp, int lane) {
    const int r = (lane >> 1) & 3, h = lane >> 3;
    grp = NG == 4 ? (lane & 1) + 2 * (h & 1) : lane & 1;
    row = NG == 4 ? 4 * (h >> 1) + r : 4 * h + r;
    first = warp;
    dst = (uint32_t)((grp >> 1) * kHalf + row * 128);
  }
  // chunks of the rows below nvalid of the tile whose codes start at `src`
  __device__ __forceinline__ void load(uint4 (&w)[kCount], const uint8_t* src, int nvalid) const {
    const uint8_t* const p = src + (first * kBlockRows + row) * (D / 2) + grp * 16;
    if (nvalid >= kKeys) {
#pragma unroll
      for (int i = 0; i < kCount; ++i) w[i] = ld_stream(p + i * (kPair * kBlockRows * (D / 2)));
      return;
    }
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const int r = (first + i * kPair) * kBlockRows + row;
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < nvalid) w[i] = ld_stream(p + i * (kPair * kBlockRows * (D / 2)));
    }
  }
  // factors: fp16 s 2^(15 - E) [128][NG], 0 for rows that are not there
  __device__ __forceinline__ void widen(const uint4 (&w)[kCount], const uint8_t* factors,
                                        uint8_t* stage) const {
    const uint8_t* const fp = factors + ((first * kBlockRows + row) * NG + grp) * 2;
    uint8_t* const base = stage + first * (kBlockRows * 128) + dst;
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const uint32_t f = *(const uint16_t*)(fp + i * (kPair * kBlockRows * NG * 2));
      const uint32_t f0 = f | f << 16, f1 = hmul2(f0, 0x2c002c00u), z = hmul2(f0, 0x80088008u);
      uint8_t* const d = base + i * (kPair * kBlockRows * 128);
      const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t a = in[u], b = a >> 8;
        const uint4 h = make_uint4(hfma2(a & 0x000f000fu, f0, z), hfma2(a & 0x00f000f0u, f1, z),
                                   hfma2(b & 0x000f000fu, f0, z), hfma2(b & 0x00f000f0u, f1, z));
        // (the block's rows start at a multiple of eight: the swizzle is that of `row`)
        *(uint4*)(d + (((4 * (grp & 1) + u) ^ (row & 7)) << 4)) = h;
      }
    }
  }
};

// The scratch rows' keys as fp16, where a K tile would be.
template <int D>
__device__ __forceinline__ void tree_rows(const Q8AttnArgs& a, const void* src, int b, int hk, int wt,
                                          const float* in, uint8_t* stage) {
#pragma unroll 2
  for (int x = wt; x < kKeys * (D / 8); x += kWideThreads) {
    const int row = x / (D / 8), u = x % (D / 8);
    const float f = in[row];
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (f != 0.f)
      v = scale8(__ldg((const uint4*)((const __nv_bfloat16*)src +
                                      (((long)b * a.R + row) * a.map.Hkv + hk) * D) + u), f);
    *(uint4*)(stage + (u >> 3) * kHalf + row * 128 + (((u & 7) ^ (row & 7)) << 4)) = v;
  }
}

// A lane's four rows of a tile's scales: a word or two each.
template <int D>
struct Scales {
  static constexpr int NW = D / 64;                // words of a row
  uint32_t w[4][NW];
  __device__ __forceinline__ void load(const uint8_t* src, int nvalid, int lane) {
    if (nvalid >= kKeys) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (NW == 2) {
          const uint2 v = __ldg((const uint2*)src + lane + 32 * i);
          w[i][0] = v.x;
          w[i][NW - 1] = v.y;
        } else {
          w[i][0] = __ldg((const uint32_t*)src + lane + 32 * i);
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = lane + 32 * i;
#pragma unroll
      for (int x = 0; x < NW; ++x) w[i][x] = 0u;
      if (r < nvalid) {
        if constexpr (NW == 2) {
          const uint2 v = __ldg((const uint2*)src + r);
          w[i][0] = v.x;
          w[i][NW - 1] = v.y;
        } else {
          w[i][0] = __ldg((const uint32_t*)src + r);
        }
      }
    }
  }
  // the exponent above the largest finite one (of the whole warp's)
  __device__ __forceinline__ int exponent() const {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < NW; ++x) top = __vmaxu2(top, w[i][x] & 0x7fff7fffu);
    top = __reduce_max_sync(kFull, max(top & 0xffffu, top >> 16));
    if (top >= 0x7f80u) {                          // (not the scales that are not finite)
      top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < NW; ++x) {
          const uint32_t lo = w[i][x] & 0x7fffu, hi = w[i][x] >> 16 & 0x7fffu;
          top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
      top = __reduce_max_sync(kFull, top);
    }
    return top == 0u ? 0 : min(max((int)(top >> 7) - 126, kQ4MinExp), kQ4MaxExp);   // (zeros: at any)
  }
  // s 2^(15 - E) in fp16: exact down to 2^-29 2^E
  __device__ __forceinline__ void store(uint8_t* dst, int E, int lane) const {
    const float up = q8_scale(127 + 15 - E);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < NW; ++x)
        ((uint32_t*)dst)[(lane + 32 * i) * NW + x] =
            pack_half2(__uint_as_float(w[i][x] << 16) * up, __uint_as_float(w[i][x] & 0xffff0000u) * up);
  }
};

template <int D, bool kPoll>
__global__ void __launch_bounds__(kThreads, 1) q4_rows_kernel(const __grid_constant__ Q8AttnArgs a) {
  using L = RowLayout<D>;
  constexpr int NG = L::NG;
  grid_dependency_sync();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = su32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  float4* s_ml = (float4*)(smem + L::off_ml);
  long long* tile_row = (long long*)(smem + L::off_rows);
  float* kt_in = (float*)(smem + L::off_tree);      // tree rows: factors into fp16 (0: row of zeros)
  float* vt_in = kt_in + kKeys;
  float* kt_out = vt_in + kKeys;                    // factor of the scores (NaN: a row with a NaN or inf)
  int* vt_u = (int*)(kt_out + kKeys);               // exponent of the value row
  volatile int8_t* ek = (volatile int8_t*)(smem + L::off_ek);
  volatile int8_t* ev = (volatile int8_t*)(smem + L::off_ev);
  // E of V; NaN from the first tile on whose E is far from 0 (kQ4Near), so that the softmax meets those
  // tiles where it raises its bounds
  volatile float* e_near = (volatile float*)(smem + L::off_near);
  volatile uint32_t* flags = (volatile uint32_t*)(smem + L::off_flags);
  int* s_top = (int*)(smem + L::off_top);           // largest exponent of a scratch value row, by warp
  const uint32_t bar0 = sbase + L::off_bar;
  auto bar = [&](int i) { return bar0 + 8u * i; };
  auto wait_ready = [&](uint32_t at, uint32_t parity) {
    return phase_ready<kPoll>(at, parity, a.wait_cycles);
  };
  auto wait_timed = [&](uint32_t at, uint32_t parity) {
    return phase_timed<kPoll>(at, parity, a.wait_cycles);
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x / a.nrg, rg = blockIdx.x % a.nrg, sp = a.split0 + blockIdx.y;
  int P;
  const int b = request_at(a, blockIdx.z, P, (volatile int*)(smem + L::off_req));
  const int nsb = q8_splits(a, P);
  if (sp >= nsb) return;
  const int k0 = q8_first(a, P, sp), k1 = q8_end(a, P, k0);
  const int n_pre = (k1 - k0 + kKeys - 1) / kKeys;
  const bool with_tree = sp == nsb - 1;             // R <= 65 < 128: one tile
  const int ntiles = n_pre + (with_tree ? 1 : 0);
  const int row_base = rg * a.rb;
  const int rows_here = min(a.rb, a.M - row_base);
  const int live_warps = (rows_here + 31) / 32;     // softmax warps of a stream with rows
  auto valid_of = [&](int t) { return min(kKeys, k1 - k0 - t * kKeys); };

  // ---------------------------------------------------------------- set-up
  const int wt = tid - kWideK * 32;
  static_assert(2 * kWideThreads >= kMaxTiles, "a thread per tile");
  using Share = Share4<D>;
  const Share share(warp & (kPair - 1), lane);
  const int pair = (warp & 3) / kPair;             // widening: of the even tiles, or of the odd ones
  uint64_t mask = 0ull;     // softmax threads: the scratch rows that the row sees,
  float c2 = 0.f;           // and the factor of its scores
  uint4 reg[Share::kCount];                        // widening: the pair's next tile
  // the tile at cache row `row` (a missing page: none)
  auto load_codes = [&](uint4 (&w)[Share::kCount], const uint8_t* codes, long row, int nvalid) {
    share.load(w, codes + (row < 0 ? 0 : row) * (D / 2), row < 0 ? 0 : nvalid);
  };
  Scales<D> sc[2];          // of this tile and the next
  const bool of_v = warp >= kWideV || warp == kScaleV;
  const uint8_t* const my_codes = of_v ? a.vc : a.kc;
  const uint8_t* const my_scales = of_v ? a.ve : a.ke;
  auto load_scales = [&](Scales<D>& s, long row, int nvalid) {
    s.load(my_scales + (row < 0 ? 0 : row) * (NG * 2), row < 0 ? 0 : nvalid, lane);
  };

  if (warp >= kWideK) {
    // the first tiles, the rows of the split's tiles, the scratch rows
    if (with_tree) tree_fetch<D, 2 * kWideThreads>(a, b, hk, wt, sbase + L::off_v, L::t_bytes);
    const long r0 = pair < n_pre ? a.map.row(b, hk, k0 + pair * kKeys) : -1;
    const long rt = wt < n_pre ? a.map.row(b, hk, k0 + wt * kKeys) : -1;
    if (pair < n_pre) load_codes(reg, my_codes, r0, valid_of(pair));
    if (wt < n_pre) {
      tile_row[wt] = rt;
      if (rt < 0) report_error(a.err, TSD_DEV_ERR_BAD_PAGE, b);
    }
    int top = -1000;
    if (with_tree)
      top = tree_scan<D, 2 * kWideThreads>(a, b, wt, smem + L::off_v, L::t_bytes, kt_in, vt_in, kt_out, vt_u);
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) s_top[warp - kWideK] = top;
  } else if (warp < 8) {
    // Q into the tensor memory: a thread takes its packed row, whose largest element
    // scales it, and converts the stream's half of it; and what the row sees
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
      const float f = bad ? 0.f : q8_scale(268 - qe);
      c2 = bad ? __int_as_float(0x7fffffff) : a.qscale * q8_scale(qe - 14);
      __syncwarp();
      asm volatile("bar.sync 2, %0;\n" ::"r"(64 * live_warps + 32) : "memory");   // (allocated)
      const uint32_t tq = flags[0] + kColQ + p * (D / 4) + ((uint32_t)(q * 32) << 16);
      uint4 x[D / 16];                             // the stream's half
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        x[i] = p ? w[D / 16 + i] : w[i];
        if (bad) x[i] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {           // eight elements: four columns
        const uint4 h = scale8(x[0], f);
        tmem_st4(tq + 4 * c, __uint_as_float(h.x), __uint_as_float(h.y), __uint_as_float(h.z),
                 __uint_as_float(h.w));
#pragma unroll
        for (int i = 0; i + 1 < D / 16; ++i) x[i] = x[i + 1];
      }
      tmem_wait_st();
    }
  } else {
    if (warp >= kScaleK) {
      if (n_pre > 0) load_scales(sc[0], a.map.row(b, hk, k0), valid_of(0));
      if (n_pre > 1) load_scales(sc[1], a.map.row(b, hk, k0 + kKeys), valid_of(1));
    }
    if (warp == kScaleK && lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        mbar_init(bar(BAR_K_FULL + i), kPair);
        mbar_init(bar(BAR_K_EMPTY + i), 1);
        mbar_init(bar(BAR_V_FULL + i), kPair);
        mbar_init(bar(BAR_V_EMPTY + i), 1);
      }
      for (int i = 0; i < kScaleRing; ++i) {
        mbar_init(bar(BAR_F_FULL + i), 2);
        mbar_init(bar(BAR_F_EMPTY + i), 2 * kPair);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(BAR_P_FULL + i), live_warps);
        mbar_init(bar(BAR_PV_DONE + i), 1);
        mbar_init(bar(BAR_FINAL + i), 1);
        mbar_init(bar(BAR_S_FULL + i), 1);
        mbar_init(bar(BAR_S_EMPTY + i), live_warps);
      }
      mbar_init(bar(BAR_O_DONE), 1);
      flags[1] = 0;
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncwarp();
    if (warp == kPv) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
          sbase + L::off_flags));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
      asm volatile("bar.arrive 2, %0;\n" ::"r"(64 * live_warps + 32) : "memory");
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = flags[0];
  auto tm_o = [&](int p) { return tmem + kColO + (uint32_t)(p * D); };
  auto factors = [&](int t, int part) {
    return smem + L::off_f + (uint32_t)((t % kScaleRing) * 2 + part) * L::f_bytes;
  };

  // -------------------------------------------------------------- widening
  if (warp >= kWideK) {
    set_registers<kWideRegs, false>();
    const int full = of_v ? BAR_V_FULL : BAR_K_FULL, empty = of_v ? BAR_V_EMPTY : BAR_K_EMPTY;
    uint8_t* const stages = smem + (of_v ? L::off_v : L::off_k);
    bool ok = true;
#pragma unroll 1
    for (int t = pair; ok && t < n_pre; t += kWideWarps / kPair) {
      const int st = t % kStages;
      ok = t < kStages || wait_ready(bar(empty + st), (t / kStages - 1) & 1);
      ok = ok && wait_ready(bar(BAR_F_FULL + t % kScaleRing), (t / kScaleRing) & 1);
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      share.widen(reg, factors(t, of_v), stages + st * L::t_bytes);
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(full + st));
        mbar_arrive(bar(BAR_F_EMPTY + t % kScaleRing));
      }
      const int next = t + kWideWarps / kPair;
      if (next < n_pre) load_codes(reg, my_codes, tile_row[next], valid_of(next));
      ok = !__any_sync(kFull, flags[1] != 0);
    }
    if (with_tree) {                               // by all four warps (which meet whatever failed)
      const int st = n_pre % kStages;
      ok = ok && (n_pre < kStages || wait_ready(bar(empty + st), (n_pre / kStages - 1) & 1));
      ok = __all_sync(kFull, ok);
      if (ok)
        tree_rows<D>(a, of_v ? a.vt : a.kt, b, hk, wt & (kWideThreads - 1), of_v ? vt_in : kt_in,
                     stages + st * L::t_bytes);
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      if (of_v) asm volatile("bar.sync 3, %0;\n" ::"n"(kWideThreads) : "memory");
      else asm volatile("bar.sync 4, %0;\n" ::"n"(kWideThreads) : "memory");
      if (ok && pair == 0 && lane == 0) mbar_arrive(bar(full + st));
    }
    if (!ok) flags[1] = 1;
  }

  else if (warp >= kPv) {
    set_registers<kMidRegs, false>();   // (one instruction for the four warps)
    // --------------------------------------------------------------- scales
    if (warp == kScaleK || warp == kScaleV) {
      volatile int8_t* const e_of = of_v ? ev : ek;
      bool far_off = false;
      auto one_tile = [&](int t, Scales<D>& s) -> bool {
        if (lane == 0) {                             // codes and scales of the tiles to come
          for (int i = t == 0 ? 2 : t + kPrefetch - 1; i < t + kPrefetch && i < n_pre; ++i)
            if (tile_row[i] >= 0) {
              prefetch_l2(my_codes + tile_row[i] * (D / 2), (long)valid_of(i) * (D / 2));
              prefetch_l2(my_scales + tile_row[i] * (NG * 2), (long)valid_of(i) * (NG * 2));
            }
        }
        __syncwarp();
        const int E = s.exponent();
        if (t >= kScaleRing &&
            !__all_sync(kFull, wait_ready(bar(BAR_F_EMPTY + t % kScaleRing), (t / kScaleRing - 1) & 1)))
          return false;
        s.store(factors(t, of_v), E, lane);
        far_off |= abs(E) > kQ4Near;
        if (lane == 0) {
          e_of[t] = (int8_t)E;
          if (of_v) e_near[t] = far_off ? __int_as_float(0x7fffffff) : (float)E;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_F_FULL + t % kScaleRing));
        if (t + 2 < n_pre) load_scales(s, tile_row[t + 2], valid_of(t + 2));
        return !__any_sync(kFull, flags[1] != 0);
      };
      bool ok = true;
  #pragma unroll 1
      for (int t = 0; ok && t < n_pre; t += 2) {
        ok = one_tile(t, sc[0]);
        if (ok && t + 1 < n_pre) ok = one_tile(t + 1, sc[1]);
      }
      if (!ok) flags[1] = 1;
    }

    // ------------------------------------------------------------- scores
    else if (warp == kQk) {
      // fp16 operands are format 0, fp32 accumulator; B (K) is K-major
      constexpr uint32_t idesc =
          (1u << 4) | ((uint32_t)(kKeys / 2 >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
      const uint64_t kd0 = smem_desc(sbase + L::off_k, 16, 1024);
      const uint32_t tq = tmem + kColQ;
      const bool one = elect_one();
      bool ok = true;
      for (int t = 0; ok && t < ntiles; ++t) {
        const int st = t % kStages;
        ok = wait_ready(bar(BAR_K_FULL + st), (t / kStages) & 1);
  #pragma unroll
        for (int p = 0; p < 2; ++p) {
          ok = ok && (t == 0 || wait_ready(bar(BAR_S_EMPTY + p), (t - 1) & 1));
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          fence_after();
          const uint64_t kd = kd0 + (uint64_t)(st * (L::t_bytes >> 4) + p * (kHalf / 2 >> 4));
          if (one) {
  #pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_f16_ta(tmem + 64u * p, tq + 8 * kk, kd + (kk >> 2) * (kHalf >> 4) + 2 * (kk & 3), idesc,
                         kk == 0 ? 0u : 1u);
            mma_commit(bar(BAR_S_FULL + p));
            if (p == 1) mma_commit(bar(BAR_K_EMPTY + st));
          }
          __syncwarp();
        }
      }
      if (!ok) flags[1] = 1;
    }

    // ------------------------------------------------------------- outputs
    else {
      // B (V) is N-major
      constexpr uint32_t idesc =
          (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
      const uint64_t vd0 = smem_desc(sbase + L::off_v, kHalf, 1024);
      const bool one = elect_one();
      bool ok = true;
      for (int t = 0; ok && t < ntiles; ++t) {
        const int st = t % kStages;
        const uint64_t vd = vd0 + (uint64_t)(st * (L::t_bytes >> 4));
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
  }

  // -------------------------------------------------------------- softmax
  else {
    set_registers<kSoftRegs, true>();
    const int p = warp >> 2, q = warp & 3, row = q * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    float m = -INFINITY, l = 0.f;                  // l: over 2^(m - eu)
    float* const eu = (float*)(smem + L::off_eu) + p * kRows + row;
    *eu = 0.f;
    bool failed = false;
    if (q < live_warps) {
      // The stream's product of the tile before: done before its P is written over
      // or its accumulator is rescaled.
      bool done = true, far = false;             // far: a bound whose last bit is worth something
      float own = -(float)kHeadroom;             // -inf: tiles' sums are computed on their own (kQ4Near)
      auto product_done = [&](int t) -> bool {
        return __all_sync(kFull, done || wait_ready(bar(BAR_PV_DONE + p), (t - 1) & 1));
      };
      // The bound is raised to X = f top + E, top the largest of v, where X passes m by the headroom (or
      // m is none), the sum and the accumulator are rescaled.  E is NaN where it is far from 0, and
      // becomes far_E.
      auto raise = [&](const float (&v)[64], float f, float top, float& fE, int t, auto far_E) -> bool {
        if (__builtin_expect(!__any_sync(kFull, !(fmaf(f, top, fE) <= m + kOverflow)), 1)) return true;
        if (!product_done(t)) return false;
        if (fE != fE) {
          own = -INFINITY;
          fE = far_E();
        }
        const float X = fmaf(f, top, fE);
        const bool need = !(X <= m + kOverflow);
        const float m_new = need ? fmaxf(m, X) : m;
        const float al = m_new == m ? 1.f : m == -INFINITY ? 0.f : ex2(m - m_new);
        if (own == -INFINITY) {
          const float e0 = *eu, e = q4_near(m, e0, m_new, X - fE), base = m_new == -INFINITY ? 0.f : m_new;
          l *= m == -INFINITY ? 0.f : ex2((m - m_new) + (e - e0));
#pragma unroll
          for (int i = 0; i < 64; ++i) l += ex2((fmaf(v[i], f, fE) - base) + (e - fE));
          *eu = e;
        } else {
          l *= al;
        }
        m = m_new;
        far = __any_sync(kFull, fabsf(m) > 1048576.f && m != -INFINITY);
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
      bool ready = false;                        // the next tile's scores
      // (the scratch rows' tile has code of its own: the loop over the prefix stays small)
      auto tile = [&](int t, auto tree) -> bool {
        constexpr bool is_tree = decltype(tree)::value;
        const int nvalid = is_tree ? a.R : valid_of(t);
        done = t == 0;
        if (!__all_sync(kFull, ready || wait_ready(bar(BAR_S_FULL + p), t & 1))) return false;
        fence_after();
        const int nv = min(nvalid - 64 * h, 64);   // keys of this half
        float v[64];
        tmem_ld32(ts, *(float(*)[32])v);
        tmem_ld32(ts + 32, *(float(*)[32])(v + 32));
        int tree_E = 0, eK = 0;
        float fE;
        if constexpr (is_tree) {
          tree_E = s_top[0];
#pragma unroll
          for (int i = 1; i < 2 * kWideWarps; ++i) tree_E = max(tree_E, s_top[i]);
          tree_E = min(max(tree_E - 9, kQ4MinExp), kQ4MaxExp);
          fE = own == -INFINITY || abs(tree_E) > kQ4Near ? __int_as_float(0x7fffffff) : (float)tree_E;
        } else {
          fE = e_near[t];
          eK = ek[t];
        }
        tmem_wait_ld();
        scores_read();
        // x + E = f v + E.  (f not 0, so that -inf stays -inf.)
        float f = 1.f;
        if constexpr (!is_tree) {
          f = c2 * q8_scale(eK + 9 + 127);
          f = f == 0.f ? 1.17549435e-38f : f;
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
        if (!raise(v, f, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), fE, t,
                   [&] { return (float)(is_tree ? tree_E : ev[t]); }))
          return false;
        float off = fE + (float)kHeadroom - (m == -INFINITY ? 0.f : m);
        if (t > 0) done = complete(bar(BAR_PV_DONE + p), (t - 1) & 1);   // (looked at a while before it is needed)
        if (__builtin_expect(far, 0)) {            // rounded as the bound was, not fused with it
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] = fmaf(v[i], f, fE);
          f = 1.f;
          off -= fE;
        }
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
                pa.x *= pow2i(u.x - 9 - tree_E);
                pa.y *= pow2i(u.y - 9 - tree_E);
                pb.x *= pow2i(u.z - 9 - tree_E);
                pb.y *= pow2i(u.w - 9 - tree_E);
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
        l = fmaf((sa.x + sa.y) + (sb.x + sb.y), ex2(own - fE), l);
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
    s_ml[p * kRows + row] = make_float4(m, l, m - *eu, 0.f);
    uint32_t stop;
    asm volatile(
        "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n"
        " bar.red.or.pred po, 1, 256, pi;\n selp.u32 %0, 1, 0, po;\n}\n"
        : "=r"(stop)
        : "r"((uint32_t)(!ok || flags[1] != 0))
        : "memory");
    if (stop == 0 && q < live_warps) {
      const float4 s0 = s_ml[row], s1 = s_ml[kRows + row];
      const float top = fmaxf(s0.x, s1.x), near = fmaxf(s0.z, s1.z);   // of the products, of the sums
      const bool none0 = s0.x == -INFINITY, none1 = s1.x == -INFINITY;
      const float w0 = none0 ? (s0.y != s0.y ? s0.y : 0.f) : ex2(s0.x - top);
      const float w1 = none1 ? (s1.y != s1.y ? s1.y : 0.f) : ex2(s1.x - top);
      const float total = (none0 ? w0 : ex2(s0.z - near)) * s0.y + (none1 ? w1 : ex2(s1.z - near)) * s1.y;
      const float inv = q4_over((float)(9 - kHeadroom) + (top - near), total);
      const float g0 = w0 * inv, g1 = w1 * inv;
      const float lse2 = near + log2f(total);
      const int pr = row_base + min(row, rows_here - 1);
      const int tr = pr / a.g, qh = hk * a.g + pr % a.g;
      const long orow = ((long)b * a.R + tr) * a.Hq + qh;
      const long prow = (((long)b * a.Hq + qh) * a.nr + tr) * a.nsplit + sp;
      const bool mine = row < rows_here;
      // stream p writes the dims [p D/2, (p + 1) D/2)
      float x[D / 2];
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) {
        float o0[32], o1[32];
        tmem_ld32(tm_o(0) + lane_off + p * (D / 2) + c, o0);
        tmem_ld32(tm_o(1) + lane_off + p * (D / 2) + c, o1);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) x[c + i] = o0[i] * g0 + o1[i] * g1;
      }
      // A split's outputs go to fp16 over a power of two of their row, whose largest then lies in
      // [2^14, 2^15): off by 2^-12 of each, and 2^-39 of the largest.  (In fp32: 8 x 64 rows over 32k keys
      // 319 instead of 305 us.  One power of two for all rows, from the values' scales, loses rows that
      // give the largest values no weight.)
      float unit = 1.f, down = 1.f;
      if (nsb > 1) {
        float top2[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 2; i += 4)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            top2[j] = max3f(top2[j], fabsf(x[i + 2 * j]), fabsf(x[i + 2 * j + 1]));
        float big = fmaxf(top2[0], top2[1]);
        if (!(big < INFINITY)) {                   // (of the finite ones)
          big = 0.f;
#pragma unroll
          for (int i = 0; i < D / 2; ++i) big = fmaxf(big, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
        }
        s_ml[p * kRows + row].w = big;
        asm volatile("bar.sync 5, %0;\n" ::"r"(64 * live_warps) : "memory");
        big = fmaxf(big, s_ml[(1 - p) * kRows + row].w);
        const int e = big == 0.f ? 0 : max((int)(__float_as_uint(big) >> 23) - 127, -100) - 14;
        unit = pow2i(e);
        down = pow2i(-e);
      }
      if (mine && p == 0) {
        if (nsb == 1) a.lse[orow] = lse2 * 0.69314718055994531f;
        else a.part_meta[prow] = make_float2(lse2, unit);
      }
      if (mine) {
        uint4* const dst = nsb == 1 ? (uint4*)((__nv_bfloat16*)a.out + orow * D + p * (D / 2))
                                    : (uint4*)((__half*)a.part_o + prow * D + p * (D / 2));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float y = x[8 * i + 2 * j], z = x[8 * i + 2 * j + 1];
            w[j] = nsb == 1 ? pack_bf16x2(y, z) : pack_half2(y * down, z * down);
          }
          dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
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
void launch_rows(const Q8AttnArgs& a, const Q8Plan& p, cudaStream_t st) {
  const uint32_t smem = RowLayout<D>::total + 1024;
  const auto kern = a.wait_cycles < kWaitCycles ? q4_rows_kernel<D, true> : q4_rows_kernel<D, false>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  for (Q8AttnArgs part = a; part.split0 < p.nsplit; part.split0 += kMaxGrid)
    launch(kern, dim3(a.map.Hkv * p.nrg, std::min(p.nsplit - part.split0, kMaxGrid), a.B), dim3(kThreads), smem, st,
           part);
}

}  // namespace

void launch_q4_rows(const Q8AttnArgs& a, const Q8Plan& p, int D, cudaStream_t st) {
  if (D == 128) launch_rows<128>(a, p, st);
  else launch_rows<64>(a, p, st);
}

}  // namespace tsd
