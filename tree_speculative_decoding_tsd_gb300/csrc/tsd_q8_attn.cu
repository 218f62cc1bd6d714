// tsd_tree_verify_attn_q8: branch-aware tree attention over an 8-bit prefix
// cache (codes and block exponents of tsd_q8.cuh) plus the scratch pad's rows
// in the element type of q.
//
// Source: "Adapting Tree-Structured Speculative Decoding to DeepSeek-V4"
// (review), research gap item 1 and "How it works" steps 3 and 5, as for
// tsd_tree_verify_attn.  With s = scale q . k, p = exp(s - m), m the running
// maximum: out = sum p v / sum p, lse = m + log sum p, in one pass over the
// keys; splits of the prefix are merged by combine_kernel.
//
// Paths: tcgen05 for bf16 inputs (tsd_q8_few.cu and tsd_q8_tc.cu, heads of 64 or 128
// dims with few or more packed rows; tsd_q8_latent.cu, 576/512), and the CUDA cores
// (tsd_simt_attn.cuh) for fp32 inputs, computed in fp32.  33-row trees of 4 requests of
// 32 heads over 1k to 4k keys: 581 us, 9.7 TFLOP/s of fp32.
#include "tsd_simt_attn.cuh"

namespace tsd {
namespace {

// Four keys of the 8-bit cache from position j, cache row row0, `live` of them there (the
// others are zeros), and their values: words of four dims, lane + 32 t.
template <int DK, int DV, bool ALIAS>
struct Q8Keys {
  static constexpr int WK = (DK / 4 + 31) / 32, WV = (DV / 4 + 31) / 32;
  static constexpr int kDk = DK, kDv = DV;
  static constexpr bool kAlias = ALIAS;
  static __device__ __forceinline__ void read(const Q8AttnArgs& a, int b, int hk, int j, long row0,
                                              int live, int lane, float (&k)[kSimtKeys][WK][4],
                                              float (&v)[kSimtKeys][WV][4]) {
    uint32_t kw[kSimtKeys][WK], vw[kSimtKeys][WV];
    const long blk = row0 < 0 ? 0 : a.map.block_at(b, hk, j, row0);
    const float fk = q8_scale(a.ke[blk]), fv = ALIAS ? fk : q8_scale(a.ve[blk]);
#pragma unroll
    for (int u = 0; u < kSimtKeys; ++u) {
      const long row = row0 + u;
#pragma unroll
      for (int t = 0; t < WK; ++t) {
        const int w = lane + 32 * t;
        kw[u][t] = u < live && w < DK / 4 ? __ldg((const uint32_t*)(a.kc + row * DK) + w) : 0u;
      }
#pragma unroll
      for (int t = 0; t < WV; ++t) {
        const int w = lane + 32 * t;
        vw[u][t] = ALIAS ? kw[u][t]
                         : u < live && w < DV / 4 ? __ldg((const uint32_t*)(a.vc + row * DV) + w) : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < kSimtKeys; ++u) {
#pragma unroll
      for (int t = 0; t < WK; ++t) {
        q8_unpack4(kw[u][t], k[u][t]);
#pragma unroll
        for (int x = 0; x < 4; ++x) k[u][t][x] *= fk;
      }
#pragma unroll
      for (int t = 0; t < WV; ++t) {
        q8_unpack4(vw[u][t], v[u][t]);
#pragma unroll
        for (int x = 0; x < 4; ++x) v[u][t][x] *= fv;
      }
    }
  }
};

Q8Plan plan_q8(const tsd_attn_desc& d) {
  Q8Plan p{};
  const int M = d.R * (d.Hq / d.Hkv);
  if (d.dtype == TSD_BF16) {
    // tcgen05: few packed rows on the columns, more on the lanes, in equal
    // groups of at most 128 per CTA; latent heads 64 per CTA
    p.part_bytes = 2;
    if (d.v_aliases_k) {
      p.path = kQ8Latent;
      p.rb = 64;
      p.nrg = (int)ceil_div(M, 64);
    } else if (M <= kQ8FewRows) {
      p.path = kQ8Few;
      p.nrg = 1;
      p.rb = M;
    } else {
      p.path = kQ8Rows;
      p.nrg = (int)ceil_div(M, 128);
      p.rb = (int)ceil_div(M, p.nrg);
    }
    // One CTA per SM.  The split count minimises the modelled time of requests
    // that fill the cache: waves of CTAs times (tiles of a CTA + 4 for its
    // set-up and epilogue), and 5 tiles' time for the merge.
    const long units = (long)d.B * d.Hkv * p.nrg, tiles = ceil_div(d.cap, 128);
    const long lo = ceil_div(tiles, 256), hi = lo > 64 ? lo : tiles < 64 ? tiles : 64;
    long best = -1, best_per = tiles;
    for (long n = lo; n <= hi; ++n) {
      const long per = ceil_div(tiles, n);
      const long cost = ceil_div(units * ceil_div(tiles, per), 152L) * (per + 4) + (per < tiles ? 5 : 0);
      if (best < 0 || cost < best) { best = cost; best_per = per; }
    }
    p.split_len = (int)best_per * 128;
    p.nsplit = (int)ceil_div(d.cap, p.split_len);
    // short splits: the scratch rows are a split of their own, not a longer last one
    p.tree_split = p.nsplit > 1 && best_per <= 8 ? 1 : 0;
    p.nsplit += p.tree_split;
    // More CTAs than SMs and a request's keys in one: the longest requests first, so
    // that the last wave holds the shortest ones.  (32 requests over 1k to 4k keys, 16
    // rows: 57 us in the batch's order, 50 by length; 132 rows: 105 and 104 us; 16 latent
    // requests over 1k to 8k keys: 372 and 278 us; in seven splits, 16 requests over 20k
    // to 32k keys: 165 and 169 us.)
    p.by_length = p.nsplit == 1 && d.B > 1 && d.B <= 64 && units > 152;
  } else {
    p.path = kQ8Simt;
    p.part_bytes = 4;
    // packed rows of a CTA.  (Four or eight, in a graph: 52-row trees of 24 requests over
    // 60 to 88 keys 271 and 245 us, 2-row trees of 32 requests over 1k to 4k keys 372 and
    // 315 us, one 17-row tree over 2k keys 79 and 82 us; latent rows, two or four: 9-row
    // trees of 2 requests over 1000 keys 325 and 284 us.)
    p.rb = d.dk > 128 || M <= 4 ? 4 : 8;
    p.nrg = (int)ceil_div(M, p.rb);
    // about four CTAs per SM over the whole batch, splits of at least 64 keys
    long ns = ceil_div(152L * 4, (long)d.B * d.Hkv * p.nrg);
    const long most = ceil_div(d.cap, 64);
    if (ns > most) ns = most;
    p.split_len = (int)ceil_div(ceil_div(d.cap, ns), 64) * 64;        // (whole blocks)
    p.nsplit = (int)ceil_div(d.cap, p.split_len);
  }
  p.ws_bytes = p.nsplit > 1 ? (size_t)d.B * d.Hq * d.R * p.nsplit *
                                  (d.dv * (size_t)p.part_bytes + sizeof(float2))
                            : 0;
  return p;
}

}  // namespace
}  // namespace tsd

using namespace tsd;

extern "C" size_t tsd_verify_q8_workspace_size(const tsd_attn_desc* d) {
  if (!q8_desc_ok(d, true)) return 0;
  return plan_q8(*d).ws_bytes;
}

extern "C" tsd_status tsd_tree_verify_attn_q8(const tsd_attn_desc* d, const void* q,
                                              const void* kq, const void* vq, const void* kexp,
                                              const void* vexp, const int32_t* page_table,
                                              int max_pages, int page_size, int num_pages,
                                              const int32_t* prefix_len, const void* ktree,
                                              const void* vtree, const uint64_t* mask, void* out,
                                              float* lse, void* ws, size_t ws_bytes, int32_t* err,
                                              tsd_stream_t stream) {
  if (!q8_desc_ok(d, true) || (((uintptr_t)err) & 3u) != 0) return TSD_ERR_INVALID_ARG;
  const bool alias = d->v_aliases_k != 0;
  if (!ok_ptr(q) || !ok_ptr(kq) || !ok_ptr(kexp) || !ok_ptr(prefix_len) || !ok_ptr(ktree) ||
      !ok_ptr(mask) || !ok_ptr(out) || !ok_ptr(lse))
    return TSD_ERR_INVALID_ARG;
  if (!alias && (!ok_ptr(vq) || !ok_ptr(vexp) || !ok_ptr(vtree))) return TSD_ERR_INVALID_ARG;
  if (!paging_ok(d, page_table, max_pages, page_size, num_pages)) return TSD_ERR_INVALID_ARG;
  const Q8Plan p = plan_q8(*d);
  if ((long)d->Hkv * p.nrg > 65535 || p.nsplit > 65535) return TSD_ERR_INVALID_ARG;
  if (ws_bytes < p.ws_bytes || (p.ws_bytes > 0 && !ok_ptr(ws))) return TSD_ERR_INVALID_ARG;
  Q8AttnArgs a{};
  a.q = q;
  a.kc = (const uint8_t*)kq;
  a.vc = alias ? nullptr : (const uint8_t*)vq;
  a.ke = (const uint8_t*)kexp;
  a.ve = alias ? nullptr : (const uint8_t*)vexp;
  a.plen = prefix_len;
  a.kt = ktree;
  a.vt = alias ? nullptr : vtree;
  a.mask = mask;
  a.out = out;
  a.lse = lse;
  if (p.nsplit > 1) {
    const size_t parts = (size_t)d->B * d->Hq * d->R * p.nsplit;
    a.part_o = ws;
    a.part_meta = (float2*)((char*)ws + parts * d->dv * p.part_bytes);
  }
  a.err = err;
  a.map = cache_map(d, page_table, max_pages, page_size, num_pages);
  a.B = d->B;
  a.R = d->R;
  a.nr = d->R;
  a.Hq = d->Hq;
  a.g = d->Hq / d->Hkv;
  a.M = d->R * a.g;
  a.nsplit = p.nsplit;
  a.split_len = p.split_len;
  a.nrg = p.nrg;
  a.rb = p.rb;
  a.tree_split = p.tree_split;
  a.by_length = p.by_length;
  a.qscale = d->scale * 1.4426950408889634f;
  a.wait_cycles = wait_budget();
  const cudaStream_t st = (cudaStream_t)stream;
  if (p.path != kQ8Simt) {
    const bool launched = p.path == kQ8Latent ? launch_q8_latent(*d, a, p, st)
                          : p.path == kQ8Few  ? launch_q8_few(*d, a, p, st)
                                              : launch_q8_rows(*d, a, p, st);
    if (!launched) return TSD_ERR_UNSUPPORTED;
    if (alias) launch_combine<__nv_bfloat16, 512, __half>(a, p, st);
    else if (d->dv == 128) launch_combine<__nv_bfloat16, 128, __half>(a, p, st);
    else launch_combine<__nv_bfloat16, 64, __half>(a, p, st);
  } else if (alias) {
    launch_simt<float, 4, Q8Keys<576, 512, true>>(a, p, st);
  } else if (d->dk == 128) {
    if (p.rb == 8) launch_simt<float, 8, Q8Keys<128, 128, false>>(a, p, st);
    else launch_simt<float, 4, Q8Keys<128, 128, false>>(a, p, st);
  } else {
    if (p.rb == 8) launch_simt<float, 8, Q8Keys<64, 64, false>>(a, p, st);
    else launch_simt<float, 4, Q8Keys<64, 64, false>>(a, p, st);
  }
  return cuda_status();
}
