// tsd_cache_evict, tsd_cache_evict_q8: the cache of every head cut to `keep`
// rows by the attention weight each cached token has received.
//
// For a request with more than `keep` rows, each KV head ranks its rows, the
// protected ones first and by index, the others by (weight desc, index asc), and
// keeps the first `keep`; NaN, of either sign, counts as more than infinity.  A row is protected if its token is
// one of the first `sink` or the last `recent` ones.  The kept rows that lie at or
// behind `keep` move, in order, into the places (in order) of the dropped rows
// below it: no row that is read is also written, no row that stays is touched, and
// in the steady state (a few new rows a round) only as many rows move as arrived.
// Attention does not depend on the order of the cached rows; `pos` carries each
// row's token position.
//
// select_kernel, a cluster of 1 to 8 CTAs per (head, request): the keep-th largest
// 32-bit key by four 8-bit histogram rounds.  The histograms are private to 16 lanes
// of a warp (bin x lane, so that equal exponents, the usual case for weights, meet
// in pairs only); the CTAs of a cluster exchange their 256 totals through distributed
// shared memory.  Then ties, holes and movers are numbered by ballots and sums over
// warps and CTAs.  A warp takes consecutive rows and keeps their keys in registers
// (up to 16 per thread; longer caches are read again by each round).  Bounded by
// latency: four rounds over 8 bytes a row.
//
// move_kernel: a warp takes 32 moves, eight of them (K and V, 4 KB) in flight.
// move_q8_kernel: one CTA per block of 64 places, because an incoming row with a
// larger exponent raises the block's:
//   e' = max of the exponents that the block's rows had before the call,
// and every code c becomes e4m3(c * 2^(e - e')).  Both are bounded by memory: each
// moved row is read and written once.
//
// 4 requests of 8 heads, 32k bf16 rows cut to half: selection 19 us, moves 57 us (4
// TB/s: rows of 256 bytes here and there; 4 or 16 moves in flight and twice the CTAs
// measured the same, fewer CTAs 70 us).  32 requests of 4k 8-bit rows, 5 dropped each:
// 16 us and 12 us.
#include <cuda_bf16.h>

#include "tsd_host.h"
#include "tsd_q8.cuh"

namespace tsd {
namespace {

constexpr int kSelThreads = 512, kSelWarps = 16, kSelLanes = 16, kMaxCluster = 8;

struct EvictArgs {
  float* acc;
  int32_t* pos;
  const int32_t* seen;
  char* k;
  char* v;
  uint8_t* kexp;
  uint8_t* vexp;
  int32_t* prefix_len;
  int32_t* err;
  CacheMap map;
  int keep, sink, recent;
  long krow, vrow;          // bytes per K and V row (vrow 0: latent)
  // workspace, per (request, head)
  int32_t* count;           // rows that move; -1: the request keeps all its rows
  int32_t* holes;           // [list] places below keep that fall free, ascending
  int32_t* movers;          // [list] kept rows at or behind keep, ascending
  int32_t* starts;          // [nblk + 1] holes before block j (8-bit cache)
  uint8_t* kexp_old;        // [nblk] exponents of before the call (8-bit cache)
  uint8_t* vexp_old;
  int list, nblk;
};

// Shared memory of a CTA, and of the others of its cluster by rank.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void store_at(const void* local, int rank, uint32_t v) {
  const uint32_t a = (uint32_t)__cvta_generic_to_shared(local);
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(r), "r"(v) : "memory");
}

struct SelectSmem {
  uint32_t hist[256 * kSelLanes];
  uint32_t totals[2][kMaxCluster][256];       // by rank, two sets in turn
  uint32_t counts[3][kMaxCluster];            // ties, holes, movers by rank
  uint32_t bins[256];
  int warps[2][kSelWarps];
  uint32_t prefix, need;
  int bad, split;          // split: not all rows that equal the cut stay
};

// Exclusive sums over the warps of two values per warp (the same on all lanes).
__device__ __forceinline__ void warps_before(SelectSmem& s, int warp, int lane, int x, int y,
                                             int& bx, int& by, int& tx, int& ty) {
  __syncthreads();
  if (lane == 0) {
    s.warps[0][warp] = x;
    s.warps[1][warp] = y;
  }
  __syncthreads();
  const int u = lane < kSelWarps ? s.warps[0][lane] : 0, v = lane < kSelWarps ? s.warps[1][lane] : 0;
  tx = __reduce_add_sync(kFull, u);
  ty = __reduce_add_sync(kFull, v);
  bx = __reduce_add_sync(kFull, lane < warp ? u : 0);
  by = __reduce_add_sync(kFull, lane < warp ? v : 0);
}

template <int ITEMS, bool kQ8>
__global__ void __launch_bounds__(kSelThreads, 2)
select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ SelectSmem s;
  constexpr int kSpan = kSelThreads * ITEMS;
  grid_dependency_sync();
  const int ranks = gridDim.x, rank = blockIdx.x;           // the cluster spans grid x
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long bh = (long)b * a.map.Hkv + h;
  const float* acc = a.acc + bh * a.map.cap;
  const int32_t* pos = a.pos + bh * a.map.cap;
  const int P = a.prefix_len[b];
  const long recent0 = (long)a.seen[bh] - a.recent;
  if (tid == 0) s.bad = 0;
  __syncthreads();
  if (P < 0 || P > a.map.cap) {
    if (tid == 0) s.bad = TSD_DEV_ERR_CAPACITY;
  } else if (a.map.page_size && P > a.keep) {
    for (int p = tid; p < (P + a.map.page_size - 1) / a.map.page_size; p += kSelThreads) {
      const int pg = a.map.page_table[(long)b * a.map.max_pages + p];
      if (pg < 0 || pg >= a.map.num_pages) s.bad = TSD_DEV_ERR_BAD_PAGE;
    }
  }
  __syncthreads();
  if (s.bad != 0 || P <= a.keep) {                          // (the same in every CTA of the cluster)
    if (tid == 0 && rank == 0) {
      a.count[bh] = -1;
      if (s.bad != 0) report_error(a.err, s.bad, b);
    }
    return;
  }
  // this CTA's rows: `rounds` spans from `begin`
  const int rounds = (P + ranks * kSpan - 1) / (ranks * kSpan);
  const int begin = rank * rounds * kSpan;

  // keys of the rows base + 32 it + lane of span r (0 past the end)
  uint32_t key[ITEMS];
  auto load = [&](int r) {
    const int base = begin + r * kSpan + warp * 32 * ITEMS + lane;
    constexpr int kBatch = ITEMS == 12 ? 6 : ITEMS < 8 ? ITEMS : 8;   // loads in flight per thread and array
#pragma unroll
    for (int i0 = 0; i0 < ITEMS; i0 += kBatch) {
      float w[kBatch];
      int p[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = base + 32 * (i0 + j);
        w[j] = i < P ? acc[i] : 0.f;
        p[j] = i < P ? pos[i] : 0;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const bool safe = p[j] < a.sink || p[j] >= recent0;
        // (every NaN, of either sign, has one key, below the protected rows' and above
        // infinity's; keys of rows are above 0: the smallest is that of -infinity)
        key[i0 + j] = base + 32 * (i0 + j) >= P ? 0u
                      : safe                    ? 0xffffffffu
                      : w[j] != w[j]            ? 0xfffffffeu
                                                : f32_order_key(w[j]);
      }
    }
  };
  load(0);

  if constexpr (kQ8) {   // the exponents of before, which the moves read while others write
    for (int j = rank * kSelThreads + tid; j * (long)kQ8Block < P; j += ranks * kSelThreads) {
      const long e = a.map.block(b, h, j * kQ8Block);
      a.kexp_old[bh * a.nblk + j] = a.kexp[e];
      if (a.vrow) a.vexp_old[bh * a.nblk + j] = a.vexp[e];
    }
  }

  cluster_sync();        // (every CTA of the cluster runs: its shared memory may be written)

  // ---- the keep-th largest key: prefix holds its digits found so far, need
  // the rank of the key among those that share them
  uint32_t prefix = 0, need = (uint32_t)a.keep;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    const int set = (shift >> 3) & 1;
    for (int i = tid; i < 64 * kSelLanes; i += kSelThreads) ((uint4*)s.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    for (int r = 0; r < rounds; ++r) {
      if (rounds > 1) load(r);
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) {
        // (rows past the end have key 0 and are left out: a row's is at least 1)
        const bool in = key[it] != 0 && (shift == 24 || (key[it] >> (shift + 8)) == prefix);
        if (in) atomicAdd(&s.hist[((key[it] >> shift) & 255u) * kSelLanes + (lane & (kSelLanes - 1))], 1u);
      }
    }
    __syncthreads();
    if (tid < 256) {
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < kSelLanes / 4; ++i) {
        const uint4 v = ((const uint4*)s.hist)[tid * (kSelLanes / 4) + ((i + tid) & (kSelLanes / 4 - 1))];
        t += v.x + v.y + v.z + v.w;
      }
      for (int k = 0; k < ranks; ++k) store_at(&s.totals[set][rank][tid], k, t);
    }
    cluster_sync();
    if (tid < 256) {
      uint32_t t = 0;
      for (int k = 0; k < ranks; ++k) t += s.totals[set][k][tid];
      s.bins[tid] = t;
    }
    __syncthreads();
    if (warp == 0) {       // lane l takes the bins 255 - 8l .. 248 - 8l, from the largest digit down
      uint32_t c[8], mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = s.bins[255 - (8 * lane + i)];
        mine += c[i];
      }
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += up;
      }
      uint32_t before = incl - mine;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (before < need && need <= before + c[i]) {
          s.prefix = (prefix << 8) | (uint32_t)(255 - (8 * lane + i));
          s.need = need - before;
          s.split = need - before != c[i];
        }
        before += c[i];
      }
    }
    __syncthreads();
    prefix = s.prefix;
    need = s.need;
  }
  const uint32_t cut = prefix;   // the smallest kept key; `need` rows that equal it stay
  const bool split = s.split != 0;

  // ---- number the ties, then the holes and the movers, in index order: counts of
  // the CTA, then (of the cluster) what lies before it
  int ties = 0, holes = 0, movers = 0;           // before the current span
  auto share = [&](int which, uint32_t mine) {   // the CTA's count to every CTA
    if (tid < ranks) store_at(&s.counts[which][rank], tid, mine);
  };
  auto before_rank = [&](int which, uint32_t& total) {
    uint32_t x = 0, t = 0;
    for (int k = 0; k < ranks; ++k) {
      const uint32_t v = s.counts[which][k];
      t += v;
      if (k < rank) x += v;
    }
    total = t;
    return (int)x;
  };
  uint32_t mine = 0;             // bit it: this lane's row of group it stays
  int bx, by, tx, ty;
  uint32_t total;
  // what stays of span r (ties numbered from `tie`), and its holes and movers
  auto keep_span = [&](int r, int tie, int& nh, int& nm) {
    const int base = begin + r * kSpan + warp * 32 * ITEMS;
    mine = 0;
    nh = nm = 0;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      bool k = key[it] >= cut;
      if (split) {
        const uint32_t eq = __ballot_sync(kFull, key[it] == cut);
        k = key[it] > cut || (key[it] == cut && tie + __popc(eq & ((1u << lane) - 1u)) < (int)need);
        tie += __popc(eq);
      }
      const uint32_t kept = __ballot_sync(kFull, k);
      mine |= (uint32_t)k << it;
      const int below = min(max(a.keep - (base + 32 * it), 0), 32);   // positions of the 32 below keep
      const uint32_t lo = below == 32 ? 0xffffffffu : (1u << below) - 1u;
      nh += __popc(~kept & lo);
      nm += __popc(kept & ~lo);
    }
  };
  auto span_ties = [&] {
    int t = 0;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) t += __popc(__ballot_sync(kFull, key[it] == cut));
    return t;
  };
  // the ties before this warp's rows of a span (only where they decide)
  auto ties_before = [&] {
    if (!split) return 0;
    warps_before(s, warp, lane, span_ties(), 0, bx, by, tx, ty);
    const int t = ties + bx;
    ties += tx;
    return t;
  };
  int ties0 = 0;
  if (split) {                   // (the same in every CTA of the cluster)
    for (int r = 0; r < rounds; ++r) {
      if (rounds > 1) load(r);
      ties_before();
    }
    share(0, ties);
    cluster_sync();
    ties0 = before_rank(0, total);
  }
  int nh = 0, nm = 0;
  ties = ties0;
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) load(r);
    keep_span(r, ties_before(), nh, nm);
    warps_before(s, warp, lane, nh, nm, bx, by, tx, ty);
    holes += tx;
    movers += ty;
  }
  share(1, holes);
  share(2, movers);
  cluster_sync();
  holes = before_rank(1, total);
  const uint32_t moved = total;
  movers = before_rank(2, total);
  ties = ties0;
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) {
      load(r);
      keep_span(r, ties_before(), nh, nm);
      warps_before(s, warp, lane, nh, nm, bx, by, tx, ty);
    }
    const int base = begin + r * kSpan + warp * 32 * ITEMS;
    int hole = holes + bx, mover = movers + by;
    holes += tx;
    movers += ty;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const uint32_t kept = __ballot_sync(kFull, (mine >> it) & 1u);
      const int i0 = base + 32 * it, i = i0 + lane;
      const int below = min(max(a.keep - i0, 0), 32);
      const uint32_t lo = below == 32 ? 0xffffffffu : (1u << below) - 1u;
      const uint32_t hm = ~kept & lo, mm = kept & ~lo;
      const uint32_t lt = (1u << lane) - 1u;
      if (kQ8 && lane == 0 && i0 % kQ8Block == 0 && i0 / kQ8Block <= a.nblk)
        a.starts[bh * (a.nblk + 1) + i0 / kQ8Block] = hole;
      if ((hm >> lane) & 1u) a.holes[bh * a.list + hole + __popc(hm & lt)] = i;
      if ((mm >> lane) & 1u) a.movers[bh * a.list + mover + __popc(mm & lt)] = i;
      hole += __popc(hm);
      mover += __popc(mm);
    }
  }
  if (tid == 0 && rank == 0) {
    a.count[bh] = (int)moved;
    if (kQ8) {      // the entry behind the last block of places (a span may end below it)
      const int j = (a.keep + kQ8Block - 1) / kQ8Block;
      a.starts[bh * (a.nblk + 1) + j] = (int)moved;
    }
  }
}

// The rest of a moved row, and the new length (by the first CTA of a request).
__device__ __forceinline__ void move_meta(const EvictArgs& a, long bh, int from, int to) {
  a.acc[bh * a.map.cap + to] = a.acc[bh * a.map.cap + from];
  a.pos[bh * a.map.cap + to] = a.pos[bh * a.map.cap + from];
}

constexpr int kMoveThreads = 256, kMoveUnroll = 8;

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictArgs a) {
  grid_dependency_sync();
  const int h = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long bh = (long)b * a.map.Hkv + h;
  const int n = a.count[bh];
  if (n < 0) return;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) a.prefix_len[b] = a.keep;
  const int kv = (int)(a.krow / 16), vv = (int)(a.vrow / 16);
  const int step = gridDim.x * kMoveThreads;
  // lane l holds move m0 + l
  for (int m0 = (blockIdx.x * (kMoveThreads / 32) + warp) * 32; m0 < n; m0 += step) {
    const int moves = min(32, n - m0);
    long from = -1, to = 0;
    if (lane < moves) {
      const int f = a.movers[bh * a.list + m0 + lane], t = a.holes[bh * a.list + m0 + lane];
      from = a.map.row(b, h, f);
      to = a.map.row(b, h, t);
      move_meta(a, bh, f, t);
    }
    for (int u0 = 0; u0 < moves; u0 += kMoveUnroll) {
      for (int c = lane; c - lane < kv + vv; c += 32) {     // (whole warps, for the shuffles)
        const bool is_k = c < kv, in = c < kv + vv;
        char* const p = is_k ? a.k : a.v;
        const long row = is_k ? a.krow : a.vrow;
        const long off = (long)(is_k ? c : c - kv) * 16;
        int4 x[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
          const long f = __shfl_sync(kFull, from, u0 + u);  // (u0 + u < 32; -1 past the end)
          if (in && f >= 0) x[u] = *(const int4*)(p + f * row + off);
        }
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
          const long f = __shfl_sync(kFull, from, u0 + u), t = __shfl_sync(kFull, to, u0 + u);
          if (in && f >= 0) *(int4*)(p + t * row + off) = x[u];
        }
      }
    }
  }
}

constexpr int kMoveQ8Threads = 128;

__global__ void __launch_bounds__(kMoveQ8Threads)
move_q8_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ long s_from[kQ8Block];
  __shared__ int s_to[kQ8Block];       // place within the block
  __shared__ uint8_t s_e[2][kQ8Block];
  __shared__ uint8_t s_hole[kQ8Block];
  __shared__ int s_max[2];
  grid_dependency_sync();
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const long bh = (long)b * a.map.Hkv + h;
  if (a.count[bh] < 0) return;
  if (blockIdx.x == 0 && h == 0 && tid == 0) a.prefix_len[b] = a.keep;
  uint32_t todo = 0;
  const int parts = a.vrow ? 2 : 1;
  const int32_t* const starts = a.starts + bh * (a.nblk + 1);
  const int blocks = (a.keep + kQ8Block - 1) / kQ8Block;
  for (int j = blockIdx.x; j < blocks; j += gridDim.x) {
    // 32 of this CTA's blocks at a time: which ones have holes (a block has 64 at
    // most; the same answer in every warp)
    if ((j - (int)blockIdx.x) / (int)gridDim.x % 32 == 0) {
      const long l = j + (long)(tid & 31) * gridDim.x;
      todo = __ballot_sync(kFull, l < blocks && starts[l] != starts[l + 1]);
    }
    const bool has = (todo >> ((j - (int)blockIdx.x) / (int)gridDim.x % 32)) & 1u;
    if (!has) continue;                // (the same for the whole CTA)
    const int h0 = starts[j], n = starts[j + 1] - h0;
    const int rows = min(kQ8Block, a.keep - j * kQ8Block);
    __syncthreads();                   // the block before is done with the shared arrays
    if (tid < 2) s_max[tid] = 0;
    if (tid < kQ8Block) s_hole[tid] = 0;
    __syncthreads();
    if (tid < n) {
      const int f = a.movers[bh * a.list + h0 + tid], t = a.holes[bh * a.list + h0 + tid];
      s_from[tid] = a.map.row(b, h, f);
      s_to[tid] = t - j * kQ8Block;
      s_hole[t - j * kQ8Block] = 1;
      const int ek = a.kexp_old[bh * a.nblk + f / kQ8Block];
      const int ev = a.vrow ? a.vexp_old[bh * a.nblk + f / kQ8Block] : 0;
      s_e[0][tid] = (uint8_t)ek;
      s_e[1][tid] = (uint8_t)ev;
      atomicMax(&s_max[0], ek);
      atomicMax(&s_max[1], ev);
      move_meta(a, bh, f, t);
    }
    __syncthreads();
    const long row0 = a.map.row(b, h, j * kQ8Block);
    for (int part = 0; part < parts; ++part) {
      const long rb = part == 0 ? a.krow : a.vrow;
      uint8_t* const base = (uint8_t*)(part == 0 ? a.k : a.v);
      const int own = (part == 0 ? a.kexp_old : a.vexp_old)[bh * a.nblk + j];
      const int e = n < rows ? max(s_max[part], own) : s_max[part];
      const int vr = (int)(rb / 16);
      for (int w = tid; w < n * vr; w += kMoveQ8Threads) {
        const int i = w / vr, c = w - i * vr;
        uint4 x = *(const uint4*)(base + s_from[i] * rb + c * 16);
        if (s_e[part][i] != e) {
          const float f = pow2i((int)s_e[part][i] - e);
          x.x = q8_rescale4(x.x, f);
          x.y = q8_rescale4(x.y, f);
          x.z = q8_rescale4(x.z, f);
          x.w = q8_rescale4(x.w, f);
        }
        *(uint4*)(base + (row0 + s_to[i]) * rb + c * 16) = x;
      }
      if (e != own) {
        const float f = pow2i(own - e);
        for (int w = tid; w < rows * vr; w += kMoveQ8Threads) {
          const int r = w / vr;
          if (s_hole[r]) continue;
          uint4* const p = (uint4*)(base + row0 * rb + (long)w * 16);
          uint4 x = *p;
          x.x = q8_rescale4(x.x, f);
          x.y = q8_rescale4(x.y, f);
          x.z = q8_rescale4(x.z, f);
          x.w = q8_rescale4(x.w, f);
          *p = x;
        }
        if (tid == 0) (part == 0 ? a.kexp : a.vexp)[a.map.block(b, h, j * kQ8Block)] = (uint8_t)e;
      }
    }
  }
}

struct EvictPlan {
  size_t count, holes, movers, starts, kexp, vexp, bytes;
  int list, nblk;
};

EvictPlan plan_evict(const tsd_attn_desc& d) {
  EvictPlan p{};
  const size_t heads = (size_t)d.B * d.Hkv;
  // at most min(keep, P - keep) rows move
  p.list = d.cap / 2 + 1;
  p.nblk = (d.cap + kQ8Block - 1) / kQ8Block;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at = (at + n + 15) / 16 * 16;
    return o;
  };
  p.count = take(heads * 4);
  p.holes = take(heads * p.list * 4);
  p.movers = take(heads * p.list * 4);
  p.starts = take(heads * (p.nblk + 1) * 4);
  p.kexp = take(heads * p.nblk);
  p.vexp = take(heads * p.nblk);
  p.bytes = at;
  return p;
}

template <int ITEMS, bool kQ8>
void launch_cluster(const EvictArgs& a, int B, int ranks, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks, a.map.Hkv, B);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, select_kernel<ITEMS, kQ8>, a);
}

template <bool kQ8>
void launch_select(const EvictArgs& a, int B, cudaStream_t st) {
  // CTAs of a cluster: more while a CTA keeps at least 2048 rows and all of them
  // are resident at once (two per SM)
  int ranks = 1;
  while (ranks < kMaxCluster && a.map.cap > ranks * 2048 && (long)a.map.Hkv * B * ranks * 2 <= 304)
    ranks *= 2;
  const long rows = ceil_div(a.map.cap, ranks);
  if (rows <= 4 * kSelThreads) launch_cluster<4, kQ8>(a, B, ranks, st);
  else if (rows <= 8 * kSelThreads) launch_cluster<8, kQ8>(a, B, ranks, st);
  else if (rows <= 12 * kSelThreads) launch_cluster<12, kQ8>(a, B, ranks, st);
  else launch_cluster<16, kQ8>(a, B, ranks, st);
}

tsd_status evict_impl(const tsd_attn_desc* d, int keep, int sink, int recent, float* acc,
                      int32_t* pos, const int32_t* seen, void* k, void* v, void* kexp, void* vexp,
                      bool q8, const int32_t* page_table, int max_pages, int page_size,
                      int num_pages, int32_t* prefix_len, void* ws, size_t ws_bytes, int32_t* err,
                      tsd_stream_t stream) {
  if (!q8_desc_ok(d) || (((uintptr_t)err) & 3u) != 0) return TSD_ERR_INVALID_ARG;
  const bool alias = d->v_aliases_k != 0;
  if (keep < 1 || sink < 0 || recent < 0 || (long)sink + recent > keep) return TSD_ERR_INVALID_ARG;
  if (!ok_ptr(acc) || !ok_ptr(pos) || !ok_ptr(seen) || !ok_ptr(k) || !ok_ptr(prefix_len))
    return TSD_ERR_INVALID_ARG;
  if (!alias && !ok_ptr(v)) return TSD_ERR_INVALID_ARG;
  if (q8 && (!ok_ptr(kexp) || (!alias && !ok_ptr(vexp)))) return TSD_ERR_INVALID_ARG;
  if (!paging_ok(d, page_table, max_pages, page_size, num_pages)) return TSD_ERR_INVALID_ARG;
  const EvictPlan p = plan_evict(*d);
  if (!ok_ptr(ws) || ws_bytes < p.bytes) return TSD_ERR_INVALID_ARG;
  if (d->Hkv > 65535) return TSD_ERR_INVALID_ARG;

  const int es = q8 ? 1 : d->dtype == TSD_F32 ? 4 : 2;
  EvictArgs a{};
  a.acc = acc;
  a.pos = pos;
  a.seen = seen;
  a.k = (char*)k;
  a.v = alias ? nullptr : (char*)v;
  a.kexp = q8 ? (uint8_t*)kexp : nullptr;
  a.vexp = q8 && !alias ? (uint8_t*)vexp : nullptr;
  a.prefix_len = prefix_len;
  a.err = err;
  a.map = cache_map(d, page_table, max_pages, page_size, num_pages);
  a.keep = keep;
  a.sink = sink;
  a.recent = recent;
  a.krow = (long)d->dk * es;
  a.vrow = alias ? 0 : (long)d->dv * es;
  char* w = (char*)ws;
  a.count = (int32_t*)(w + p.count);
  a.holes = (int32_t*)(w + p.holes);
  a.movers = (int32_t*)(w + p.movers);
  a.starts = (int32_t*)(w + p.starts);
  a.kexp_old = (uint8_t*)(w + p.kexp);
  a.vexp_old = (uint8_t*)(w + p.vexp);
  a.list = p.list;
  a.nblk = p.nblk;
  const cudaStream_t st = (cudaStream_t)stream;
  if (keep >= d->cap) return TSD_OK;   // no request can hold more
  const long heads = (long)d->B * d->Hkv;
  // about eight CTAs per SM over all heads, no more than there can be work for
  if (q8) {
    launch_select<true>(a, d->B, st);
    // (more than are resident: most CTAs of a small cut find no hole)
    long x = ceil_div(152L * 32, heads);
    const long most = ceil_div(keep, kQ8Block);
    if (x > most) x = most;
    launch(move_q8_kernel, dim3((unsigned)x, d->Hkv, d->B), dim3(kMoveQ8Threads), 0, st, a);
  } else {
    launch_select<false>(a, d->B, st);
    long x = ceil_div(152L * 8, heads);
    const long most = ceil_div(p.list, kMoveThreads);
    if (x > most) x = most;
    launch(move_kernel, dim3((unsigned)x, d->Hkv, d->B), dim3(kMoveThreads), 0, st, a);
  }
  return cuda_status();
}

}  // namespace
}  // namespace tsd

using namespace tsd;

extern "C" size_t tsd_cache_evict_workspace_size(const tsd_attn_desc* d) {
  if (!q8_desc_ok(d)) return 0;
  return plan_evict(*d).bytes;
}

extern "C" tsd_status tsd_cache_evict(const tsd_attn_desc* d, int keep, int sink, int recent,
                                      float* acc, int32_t* pos, const int32_t* seen, void* kcache,
                                      void* vcache, const int32_t* page_table, int max_pages,
                                      int page_size, int num_pages, int32_t* prefix_len, void* ws,
                                      size_t ws_bytes, int32_t* err, tsd_stream_t stream) {
  return evict_impl(d, keep, sink, recent, acc, pos, seen, kcache, vcache, nullptr, nullptr, false,
                    page_table, max_pages, page_size, num_pages, prefix_len, ws, ws_bytes, err,
                    stream);
}

extern "C" tsd_status tsd_cache_evict_q8(const tsd_attn_desc* d, int keep, int sink, int recent,
                                         float* acc, int32_t* pos, const int32_t* seen, void* kq,
                                         void* vq, void* kexp, void* vexp,
                                         const int32_t* page_table, int max_pages, int page_size,
                                         int num_pages, int32_t* prefix_len, void* ws,
                                         size_t ws_bytes, int32_t* err, tsd_stream_t stream) {
  return evict_impl(d, keep, sink, recent, acc, pos, seen, kq, vq, kexp, vexp, true, page_table,
                    max_pages, page_size, num_pages, prefix_len, ws, ws_bytes, err, stream);
}
