// tsd_qk_norm_rope: RMS norm of every head's query and key and the position rotation, one
// pass from a layer's projections to the rows that the attention and the cache take.
//
// Source: "Adapting Tree-Structured Speculative Decoding to DeepSeek-V4" (review),
// research gap item 1: a tree's rows keep the position of their depth behind the prefix,
// whatever their place in the tree; "How it works" step 3 (layout and metadata of the
// tree are what the target's layers are fed).
//
// Per row x of d dims:  y = x / sqrt(mean(x^2) + eps) * w, then for pair i of the rotated
// dims (a, b) -> (a cos t - b sin t, a sin t + b cos t), t = sum over axes of position *
// frequency[axis][i].  All in fp32, rounded once.
//
// An angle is kept in turns, as a fraction of 2^64: position times frequency is a 64-bit
// integer product whose overflow is the whole turns, so far positions lose nothing
// (an fp32 product is off by 0.06 radians at position 10^6, a double's reduction costs
// a division).
//
// A row's 8-element pieces lie on d / 8 lanes, both elements of a pair on one lane: the
// rotation needs no other lane, the mean four (three) shuffles.  A warp takes a token and a run
// of its heads, whose sines it computes once; a grid of few tokens cuts the heads into more
// runs.  Bounded by memory: each element is read and written once (prompts of 4 x up to 8192
// rows of 32 + 16 heads: 91 us on the device, 89 by the bytes; with a head's weights loaded for
// each row instead of kept for all queries or keys 108).  Small trees: the host's side of the
// call.
#include <cuda_bf16.h>
#include <math.h>

#include "tsd_common.cuh"
#include "tsd_host.h"
#include "tsd_q8.cuh"

namespace tsd {
namespace {

struct RopeArgs {
  const void* in[3];        // Q, K, V rows (V may be null)
  void* out[3];
  long stride[3];           // elements between the rows of two tokens
  const void* weight[2];    // of Q, K; null: 1
  const uint64_t* turns;    // [axes][rot / 2]
  const int32_t* start;     // [B] or null
  const int32_t* offset;    // [axes][B][T], or [B][T] for all axes (offset_step 0), or null: 0..T-1
  long offset_step;         // elements between two axes' offsets
  const int32_t* count;     // [B] or null: T
  int B, T, Hq, Hkv, rot, axes, norm, parts;
  float eps, amplitude;
};

constexpr int kRopeThreads = 128;
constexpr int kRopeUnroll = 4;                     // (two: 106 instead of 97 us in a graph, eight: 108)

// Four consecutive elements as they are in memory.
struct Four32 {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *(const float4*)p; }
  __device__ __forceinline__ void store(float* p) const { *(float4*)p = v; }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  __device__ __forceinline__ void set(const float* x) { v = make_float4(x[0], x[1], x[2], x[3]); }
};
struct Four16 {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *(const uint2*)p; }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *(uint2*)p = v; }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  __device__ __forceinline__ void set(const float* x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    v = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};
template <typename T> struct FourOf { using type = Four32; };
template <> struct FourOf<__nv_bfloat16> { using type = Four16; };

// kNear: pairs of neighbours (2i, 2i + 1), else of halves (i, i + rot / 2).
template <typename T, int D, bool kNear>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  using Four = typename FourOf<T>::type;
  constexpr int VR = D / 8, kRows = 32 / VR;       // lanes of a row, rows of a warp
  grid_dependency_sync();
  const int lane = threadIdx.x & 31, c = lane % VR, sub = lane / VR;
  const long unit = (long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const long tok = unit / a.parts;
  const int part = (int)(unit % a.parts);
  if (tok >= (long)a.B * a.T) return;
  const int b = (int)(tok / a.T), t = (int)(tok % a.T);
  if (a.count != nullptr && t >= a.count[b]) return;

  // this lane's two runs of four elements: pairs 4c .. 4c + 3, of the rotated dims or of
  // those behind them
  const int half = a.rot / 2, p0 = 4 * c;
  const bool turned = p0 < half;
  int o0, o1;
  if (kNear) {
    o0 = 8 * c;
    o1 = o0 + 4;
  } else if (turned) {
    o0 = p0;
    o1 = p0 + half;
  } else {
    o0 = a.rot + p0 - half;
    o1 = o0 + (D - a.rot) / 2;
  }
  float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  if (turned) {
    uint64_t angle[4] = {0, 0, 0, 0};
    const long long first = a.start != nullptr ? a.start[b] : 0;
    for (int x = 0; x < a.axes; ++x) {
      const long long pos =
          first + (a.offset != nullptr ? a.offset[x * a.offset_step + tok] : t);
      const ulonglong2* f = (const ulonglong2*)(a.turns + (long)x * half + p0);
      const ulonglong2 f0 = __ldg(f), f1 = __ldg(f + 1);
      angle[0] += (uint64_t)pos * f0.x;
      angle[1] += (uint64_t)pos * f0.y;
      angle[2] += (uint64_t)pos * f1.x;
      angle[3] += (uint64_t)pos * f1.y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // the top 32 bits as half turns in [-1, 1)
      sincospif((float)(int32_t)(angle[i] >> 32) * 4.656612873077393e-10f, &sn[i], &cs[i]);
      cs[i] *= a.amplitude;
      sn[i] *= a.amplitude;
    }
  }

  // Steps of kRows heads: those of the queries, of the keys, of the values; this warp's run of
  // them.  The weights stay in registers through a kind's heads.
  const int steps_q = (a.Hq + kRows - 1) / kRows, steps_k = (a.Hkv + kRows - 1) / kRows;
  const int steps = steps_q + steps_k + (a.in[2] != nullptr ? steps_k : 0);
  const int per = (steps + a.parts - 1) / a.parts;
  const int s0 = part * per, s1 = min(steps, s0 + per);

  auto turn_heads = [&](int kind, int H, int first, int last) {
    if (first >= last) return;
    const T* const src = (const T*)a.in[kind] + tok * a.stride[kind];
    T* const dst = (T*)a.out[kind] + tok * H * D;
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (a.weight[kind] != nullptr) {
      Four w0, w1;
      w0.load((const T*)a.weight[kind] + o0);
      w1.load((const T*)a.weight[kind] + o1);
      w0.get(w);
      w1.get(w + 4);
    }
    for (int s = first; s < last; s += kRopeUnroll) {
      Four x0[kRopeUnroll], x1[kRopeUnroll];
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const int h = min((s + u) * kRows + sub, H - 1);
        x0[u].load(src + h * D + o0);
        x1[u].load(src + h * D + o1);
      }
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const int h = (s + u) * kRows + sub;
        float x[8], f = 1.f;
        x0[u].get(x);
        x1[u].get(x + 4);
        if (a.norm) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
          for (int o = VR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
          f = rsqrtf(sum * (1.f / D) + a.eps);
        }
        if (s + u >= last || h >= H) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= f * w[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float& p = kNear ? x[2 * i] : x[i];
          float& q = kNear ? x[2 * i + 1] : x[4 + i];
          const float y = p * cs[i] - q * sn[i];
          q = p * sn[i] + q * cs[i];
          p = y;
        }
        x0[u].set(x);
        x1[u].set(x + 4);
        x0[u].store(dst + h * D + o0);
        x1[u].store(dst + h * D + o1);
      }
    }
  };
  turn_heads(0, a.Hq, s0, min(s1, steps_q));
  turn_heads(1, a.Hkv, max(s0 - steps_q, 0), min(s1 - steps_q, steps_k));
  if (a.in[2] != nullptr) {
    const T* const src = (const T*)a.in[2] + tok * a.stride[2];
    T* const dst = (T*)a.out[2] + tok * a.Hkv * D;
    const int first = max(s0 - steps_q - steps_k, 0), last = s1 - steps_q - steps_k;
    for (int s = first; s < last; s += kRopeUnroll) {
      Four x0[kRopeUnroll], x1[kRopeUnroll];
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const int h = min((s + u) * kRows + sub, a.Hkv - 1);
        x0[u].load(src + h * D + 8 * c);
        x1[u].load(src + h * D + 8 * c + 4);
      }
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) {
        const int h = (s + u) * kRows + sub;
        if (s + u >= last || h >= a.Hkv) continue;
        x0[u].store(dst + h * D + 8 * c);
        x1[u].store(dst + h * D + 8 * c + 4);
      }
    }
  }
}

template <typename T, int D>
void launch_rope(const RopeArgs& a, bool near, cudaStream_t st) {
  const long units = (long)a.B * a.T * a.parts;
  const dim3 grid((unsigned)ceil_div(units, kRopeThreads / 32));
  if (near) launch(rope_kernel<T, D, true>, grid, dim3(kRopeThreads), 0, st, a);
  else launch(rope_kernel<T, D, false>, grid, dim3(kRopeThreads), 0, st, a);
}

}  // namespace
}  // namespace tsd

using namespace tsd;

extern "C" tsd_status tsd_qk_norm_rope(const tsd_rope_desc* d, const void* q, int64_t q_stride,
                                       const void* k, int64_t k_stride, const void* v,
                                       int64_t v_stride, const void* q_weight,
                                       const void* k_weight, const uint64_t* turns,
                                       const int32_t* start, const int32_t* offset,
                                       int offset_axes, const int32_t* count, void* q_out, void* k_out, void* v_out,
                                       tsd_stream_t stream) {
  if (d == nullptr || d->B < 1 || d->T < 1 || d->Hq < 1 || d->Hkv < 1 || d->Hq > 65535 ||
      d->Hkv > 65535)
    return TSD_ERR_INVALID_ARG;
  if (d->dtype != TSD_F32 && d->dtype != TSD_BF16) return TSD_ERR_INVALID_ARG;
  if (d->d != 64 && d->d != 128) return TSD_ERR_INVALID_ARG;
  if (d->rot < 0 || d->rot > d->d || d->rot % 8 != 0 || d->axes < 1 || d->axes > 4)
    return TSD_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f) || !(d->eps < 1e30f) || !(fabsf(d->amplitude) < 1e30f)) return TSD_ERR_INVALID_ARG;
  if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(q_out) || !ok_ptr(k_out) || !ok_opt_ptr(v) ||
      !ok_opt_ptr(v_out) || (v == nullptr) != (v_out == nullptr) || !ok_opt_ptr(q_weight) ||
      !ok_opt_ptr(k_weight) || !ok_opt_ptr(start) || !ok_opt_ptr(offset) || !ok_opt_ptr(count))
    return TSD_ERR_INVALID_ARG;
  if (d->rot > 0 && !ok_ptr(turns)) return TSD_ERR_INVALID_ARG;
  if (offset != nullptr && offset_axes != 1 && offset_axes != d->axes) return TSD_ERR_INVALID_ARG;
  if (!d->norm && (q_weight != nullptr || k_weight != nullptr)) return TSD_ERR_INVALID_ARG;
  const int vec = d->dtype == TSD_BF16 ? 8 : 4;        // elements of 16 bytes
  const int64_t s[3] = {q_stride, k_stride, v == nullptr ? (int64_t)d->Hkv * d->d : v_stride};
  for (int i = 0; i < 3; ++i)
    if (s[i] < (int64_t)(i == 0 ? d->Hq : d->Hkv) * d->d || s[i] % vec != 0 || s[i] > (1ll << 40))
      return TSD_ERR_INVALID_ARG;
  RopeArgs a{};
  a.in[0] = q; a.in[1] = k; a.in[2] = v;
  a.out[0] = q_out; a.out[1] = k_out; a.out[2] = v_out;
  a.weight[0] = q_weight; a.weight[1] = k_weight;
  a.turns = turns;
  a.start = start;
  a.offset = offset;
  a.offset_step = offset_axes == 1 ? 0 : (long)d->B * d->T;
  a.count = count;
  a.B = d->B; a.T = d->T; a.Hq = d->Hq; a.Hkv = d->Hkv;
  a.rot = d->rot; a.axes = d->axes; a.norm = d->norm != 0;
  a.eps = d->eps;
  a.amplitude = d->amplitude;
  for (int i = 0; i < 3; ++i) a.stride[i] = s[i];
  // runs of a token's heads: as many warps as the GPU holds, or one per batch of loads
  const int rows = 32 / (d->d / 8);
  const long steps = ceil_div(d->Hq, rows) + ceil_div(d->Hkv, rows) * (v != nullptr ? 2 : 1);
  const long most = ceil_div(steps, kRopeUnroll), tokens = (long)d->B * d->T;
  const long want = ceil_div(152L * 48, tokens);
  a.parts = (int)(want < 1 ? 1 : want > most ? most : want);
  if (ceil_div(tokens * a.parts, kRopeThreads / 32) > 0x7fffffffl) return TSD_ERR_INVALID_ARG;
  const cudaStream_t st = (cudaStream_t)stream;
  const bool near = d->neighbours != 0;
  if (d->dtype == TSD_F32) {
    if (d->d == 128) launch_rope<float, 128>(a, near, st);
    else launch_rope<float, 64>(a, near, st);
  } else {
    if (d->d == 128) launch_rope<__nv_bfloat16, 128>(a, near, st);
    else launch_rope<__nv_bfloat16, 64>(a, near, st);
  }
  return cuda_status();
}
