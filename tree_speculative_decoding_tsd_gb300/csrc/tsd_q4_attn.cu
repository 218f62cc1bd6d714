// tsd_tree_verify_attn_q4: branch-aware tree attention over a 4-bit prefix cache
// (tsd_q4.cuh) plus the scratch pad's rows in the element type of q.
//
// Source: "Adapting Tree-Structured Speculative Decoding to DeepSeek-V4"
// (review), research gap item 1 and "How it works" steps 3 and 5, as for
// tsd_tree_verify_attn.  With s = scale q . k, p = exp(s - m), m the running
// maximum: out = sum p v / sum p, lse = m + log sum p, in one pass over the
// keys; splits of the prefix are merged by combine_kernel.
#include "tsd_q4_attn.cuh"
#include "tsd_simt_attn.cuh"

namespace tsd {
namespace {

// Modelled time of a tensor-core path with splits of `per` tiles (128 keys); the unit is an SM's
// time for a tile.  An SM holds `room` CTAs: one of the rows path; one of twelve warps or three of
// four for nine to sixteen packed rows; two of eight or four of four for fewer.  A CTA's set-up
// and end cost `ends` tiles (twice that of 64 dims); CTAs of four warps start later, and one that
// is alone on its SM takes `alone` times as long.  It is the sum for caches that are full and for
// caches three quarters full on average, whose CTAs fill one another's gaps, the longest requests
// first where each has one split.
// (Measured with larger / smaller CTAs, us.  Four rows of 4 heads each: 1 request over 32k keys 27
// and 30, 32 over 1k to 4k 49 and 61, 8 over 32k 107 and 91, 200 below 900 125 and 87.  One row:
// 1 over 2k 13 and 14, 64 over 1k to 8k 83 and 89, 200 below 900 54 and 44.)
struct CtaShape {
  int room;
  double ends, alone, start;
};
constexpr CtaShape kFewShapes[2][2] = {{{2, 5, 1.1, 0}, {4, 3, 1.35, 4}}, {{1, 6, 1, 0}, {3, 3, 1.4, 4}}};
constexpr CtaShape kRowsShape{1, 5, 1, 0};

double split_cost(long units, long tiles, long per, int D, const CtaShape& s) {
  constexpr double kSms = 152, kFill = 0.75;
  const long n = ceil_div(tiles, per), full = units * n, slots = 152L * s.room;
  const double ends = s.ends * (128 / D), whole = per + ends;
  // CTAs that start together, so many per SM
  auto round = [&](double deep) { return (deep > s.alone ? deep : s.alone) * whole + s.start; };
  double cost = full / slots * s.room * whole;
  if (full % slots) cost += round((double)ceil_div(full % slots, 152));
  const double some = n == 1 ? units : units * (kFill * n + 1 - kFill);
  if (full <= slots || some * 1.1 <= slots) {
    const double deep = n == 1 ? (double)ceil_div(full, 152) : 1.15 * some / kSms;
    cost += round(deep > s.room ? s.room : deep);
  } else {
    cost += (units * tiles * kFill + some * ends) / kSms + (n == 1 ? 0.1 : 0.5) * whole;
  }
  return cost + (n > 1 ? 12 : 0);                  // (the merge, in both)
}

// Plan of a launch for R of the tree's rows.
Q8Plan plan_rows(const tsd_attn_desc& d, int R) {
  Q8Plan p{};
  const int M = R * (d.Hq / d.Hkv);
  const long heads = (long)d.B * d.Hkv;
  if (d.dtype == TSD_BF16) {
    const bool few = M <= kQ4FewRows;
    p.path = few ? kQ8Few : kQ8Rows;
    p.part_bytes = few ? 4 : 2;
    p.nrg = few ? 1 : (int)ceil_div(M, 128);
    p.rb = (int)ceil_div(M, p.nrg);
    // The split count minimises a modelled time: that above, and for up to eight rows that of
    // requests that fill the cache, waves of CTAs times (tiles + 6), and the merge.
    const bool eight = few && M <= 8;
    const long units = heads * p.nrg, tiles = ceil_div(d.cap, 128);
    const long lo = ceil_div(tiles, 256), hi = lo > 64 ? lo : tiles < 64 ? tiles : 64;
    const CtaShape* const shapes = few ? kFewShapes[eight ? 0 : 1] : &kRowsShape;
    double best = -1;
    long best_per = tiles;
    for (long n = lo; n <= hi; ++n) {
      const long per = ceil_div(tiles, n);
      for (int small = 0; small < (few && !eight ? 2 : 1); ++small) {
        const double cost = eight ? ceil_div(units * ceil_div(tiles, per), 304) * (per + 6) + (per < tiles ? 6 : 0)
                                  : split_cost(units, tiles, per, d.dk, shapes[small]);
        if (best < 0 || cost < best) { best = cost; best_per = per; p.small_ctas = small; }
      }
    }
    // Up to eight rows: the smaller CTAs for many short caches.
    if (eight && best_per == tiles)
      p.small_ctas = split_cost(units, tiles, tiles, d.dk, shapes[1]) < split_cost(units, tiles, tiles, d.dk, shapes[0]);
    p.split_len = (int)best_per * 128;
    p.nsplit = (int)ceil_div(d.cap, p.split_len);
    p.tree_split = !few && p.nsplit > 1 && best_per <= 8 ? 1 : 0;
    p.nsplit += p.tree_split;
    // More CTAs than run at once and a request's keys in one: the longest requests first.
    p.by_length = p.nsplit == 1 && d.B > 1 && d.B <= 64 && units > 152L * shapes[p.small_ctas].room;
  } else {
    p.path = kQ4F32;
    p.part_bytes = 4;
    p.nrg = (int)ceil_div(M, 64);
    p.rb = (int)ceil_div(M, p.nrg);
    // As many splits of whole tiles (64 keys), up to 64, as give an SM two CTAs; the scratch rows
    // are a split of their own where they are much of one.  (4 rows of 4 requests over 1k to 4k
    // keys, 3, 6, 12, 24 splits: 69, 48, 34, 40 us; 17 rows of one over 2k: 63, 42, 39, 40, and
    // with the scratch rows in the last split 81, 48, 46, 49.)
    const long tiles = ceil_div(d.cap, 64), most = 304 / (heads * p.nrg);
    const long n = most < 1 ? 1 : most > 64 ? 64 : most, even = ceil_div(tiles, n);
    const long per = even < 32768 ? even : 32768;  // (positions of a split: 2^21)
    p.split_len = (int)per * 64;
    p.nsplit = (int)ceil_div(d.cap, p.split_len);
    p.tree_split = p.nsplit > 1 && per <= 12 ? 1 : 0;
    p.nsplit += p.tree_split;
  }
  p.ws_bytes = p.nsplit > 1 ? (size_t)d.B * d.Hq * R * p.nsplit *
                                  (d.dv * (size_t)p.part_bytes + sizeof(float2))
                            : 0;
  return p;
}

// Trees of 1 + 32 n rows (the root and 32 n nodes) times 4 or 8 heads leave 4 or 8 packed rows behind
// groups of 128.  With much to do the last tree rows then have a launch of their own, on the path for
// few rows and behind the groups', instead of being one more group: where a cache is one split and the
// groups' CTAs are several waves, or where it is several splits and long.  (Rows of 32 heads, us, so
// and in equal groups.  One split: 16, 24, 32, 40, 64 x 33 rows over 1k to 4k keys 83, 114, 120, 151,
// 208 and 78, 100, 124, 157, 231; 32 x 34 122 and 125; 24 x 65 163 and 142; 128 x 33 below 1k 188 and
// 231.  Several: 8 x 33 over 32k 230 and 288, 8 x 34 232 and 288, 8 x 65 384 and 400, 2 x 33 over 20k
// to 32k 79 and 89; 4 x 33 over 4k to 8k, which therefore stay together, 61 and 54.)
constexpr long kQ4RestWork = 4096;                 // heads times tiles
constexpr long kQ4RestHeads = 256, kQ4RestTiles = 128;   // of one split; of several

struct Q4Plan {
  Q8Plan main, rest;
  int rest_rows;                                   // tree rows of `rest`; 0: none
  size_t rest_at, ws_bytes;
};
Q4Plan plan_q4(const tsd_attn_desc& d) {
  Q4Plan p{};
  const int g = d.Hq / d.Hkv, M = d.R * g, behind = M % 128;
  const long tiles = ceil_div(d.cap, 128), heads = (long)d.B * d.Hkv;
  if (d.dtype == TSD_BF16 && M > 128 && behind > 0 && behind <= 8 && behind % g == 0 &&
      heads * tiles >= kQ4RestWork) {
    p.rest_rows = behind / g;
    p.main = plan_rows(d, d.R - p.rest_rows);
    if (p.main.nsplit > 1 ? tiles < kQ4RestTiles : heads < kQ4RestHeads) p.rest_rows = 0;
  }
  if (p.rest_rows == 0) p.main = plan_rows(d, d.R);
  p.ws_bytes = p.main.ws_bytes;
  if (p.rest_rows > 0) {
    p.rest = plan_rows(d, p.rest_rows);
    p.rest_at = (p.ws_bytes + 255) / 256 * 256;
    p.ws_bytes = p.rest_at + p.rest.ws_bytes;
  }
  return p;
}

bool grid_ok(const tsd_attn_desc& d, const Q4Plan& p) { return (long)d.Hkv * p.main.nrg <= kMaxGrid; }

// A launch for tree rows r0 .. r0 + nr - 1, and the merge of its splits.
void run_q4(Q8AttnArgs a, const Q8Plan& p, int r0, int nr, int D, void* ws, cudaStream_t st) {
  a.r0 = r0;
  a.nr = nr;
  a.M = nr * a.g;
  if (p.nsplit > 1) {
    const size_t parts = (size_t)a.B * a.Hq * nr * p.nsplit;
    a.part_o = ws;
    a.part_meta = (float2*)((char*)ws + parts * D * p.part_bytes);
  }
  a.nsplit = p.nsplit;
  a.split_len = p.split_len;
  a.nrg = p.nrg;
  a.rb = p.rb;
  a.tree_split = p.tree_split;
  a.by_length = p.by_length;
  if (p.path == kQ8Few) {
    launch_q4_few(a, p, D, st);
    if (D == 128) launch_combine<__nv_bfloat16, 128, float>(a, p, st);
    else launch_combine<__nv_bfloat16, 64, float>(a, p, st);
  } else if (p.path == kQ8Rows) {
    launch_q4_rows(a, p, D, st);
    if (D == 128) launch_combine<__nv_bfloat16, 128, __half>(a, p, st);
    else launch_combine<__nv_bfloat16, 64, __half>(a, p, st);
  } else {
    launch_q4_f32(a, p, D, st);
    if (D == 128) launch_combine<float, 128, float>(a, p, st);
    else launch_combine<float, 64, float>(a, p, st);
  }
}

}  // namespace
}  // namespace tsd

using namespace tsd;

extern "C" size_t tsd_verify_q4_workspace_size(const tsd_attn_desc* d) {
  if (q4_desc_status(d, true) != TSD_OK) return 0;
  const Q4Plan p = plan_q4(*d);
  return grid_ok(*d, p) ? p.ws_bytes : 0;
}

extern "C" tsd_status tsd_tree_verify_attn_q4(const tsd_attn_desc* d, const void* q,
                                              const void* kq, const void* vq, const void* kscale,
                                              const void* vscale, const int32_t* page_table,
                                              int max_pages, int page_size, int num_pages,
                                              const int32_t* prefix_len, const void* ktree,
                                              const void* vtree, const uint64_t* mask, void* out,
                                              float* lse, void* ws, size_t ws_bytes, int32_t* err,
                                              tsd_stream_t stream) {
  const tsd_status ok = q4_desc_status(d, true);
  if (ok != TSD_OK) return ok;
  if ((((uintptr_t)err) & 3u) != 0 || !ok_ptr(q) || !ok_ptr(kq) || !ok_ptr(vq) || !ok_ptr(kscale) ||
      !ok_ptr(vscale) || !ok_ptr(prefix_len) || !ok_ptr(ktree) || !ok_ptr(vtree) || !ok_ptr(mask) ||
      !ok_ptr(out) || !ok_ptr(lse) || !paging_ok(d, page_table, max_pages, page_size, num_pages))
    return TSD_ERR_INVALID_ARG;
  const Q4Plan p = plan_q4(*d);
  if (!grid_ok(*d, p)) return TSD_ERR_INVALID_ARG;
  if (ws_bytes < p.ws_bytes || (p.ws_bytes > 0 && !ok_ptr(ws))) return TSD_ERR_INVALID_ARG;
  Q8AttnArgs a{};
  a.q = q;
  a.kc = (const uint8_t*)kq;
  a.vc = (const uint8_t*)vq;
  a.ke = (const uint8_t*)kscale;
  a.ve = (const uint8_t*)vscale;
  a.plen = prefix_len;
  a.kt = ktree;
  a.vt = vtree;
  a.mask = mask;
  a.out = out;
  a.lse = lse;
  a.err = err;
  a.map = cache_map(d, page_table, max_pages, page_size, num_pages);
  a.B = d->B;
  a.R = d->R;
  a.Hq = d->Hq;
  a.g = d->Hq / d->Hkv;
  a.qscale = d->scale * 1.4426950408889634f;
  a.wait_cycles = wait_budget();
  const cudaStream_t st = (cudaStream_t)stream;
  const int together = d->R - p.rest_rows;
  run_q4(a, p.main, 0, together, d->dk, ws, st);
  if (p.rest_rows > 0)
    run_q4(a, p.rest, together, p.rest_rows, d->dk, (char*)ws + p.rest_at, st);
  return cuda_status();
}
