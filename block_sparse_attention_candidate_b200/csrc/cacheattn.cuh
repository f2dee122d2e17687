// Attention of new tokens over the paged K / V cache.
//
// For query head h of token i (of the n that sequence s has in this call, at
// position x = kv_len - n + i) with K / V head h / (heads / kv heads):
//   seen  = [lo, hi): all cached positions (frame = 0), or those of frames
//           floor(x / frame) - window + 1 .. floor(x / frame) (window = 0: 0 ..)
//   o     = sum_seen softmax(scale q.k) v,   lse = ln sum_seen exp(scale q.k)
// A row that sees nothing gives o = 0, lse = -inf.
//
// One warp a row: a lane holds D / 32 channels, each key is a shuffle sum.
#pragma once

#include "kvcache.cuh"

namespace dynrad {

struct CacheAttnParams {
  CacheDev c;
  SeqsDev s;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;                                   // [heads, num_tokens]
  int64_t q_token, q_head, o_token, o_head;     // strides in elements
  int32_t heads, group, frame, window;
  float scale_log2;
};

// Positions that position x of a sequence of length len sees.
__device__ __forceinline__ void seen_range(int frame, int window, int32_t x, int32_t len, int32_t& lo, int32_t& hi) {
  lo = 0;
  hi = len;
  if (frame > 0) {
    if (x < 0) {
      hi = 0;
      return;
    }
    const int64_t f = x / frame;
    hi = static_cast<int32_t>(min(static_cast<int64_t>(len), (f + 1) * frame));
    if (window > 0) lo = static_cast<int32_t>(max(static_cast<int64_t>(0), (f - window + 1) * frame));
  }
}

template <int D, int FMT>
__device__ __forceinline__ float cache_channel(const uint8_t* base, const uint8_t* scale, int64_t at, int c) {
  if (FMT == kCacheBf16)
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[at * D + c]);
  uint32_t f1, f2, lo, hi;
  scale_factors<FMT>(scale[at * (D / kCacheGroup) + c / kCacheGroup], f1, f2);
  unpack4<FMT>(base[at * D + c], lo, hi);
  return __uint_as_float(mul_bf16x2(mul_bf16x2(lo, f1), f2) << 16);
}

template <int D, int FMT>
__global__ void __launch_bounds__(128) cache_attn_kernel(const CacheAttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int t = static_cast<int>(row / p.heads), h = static_cast<int>(row % p.heads);
  if (t >= p.s.num_tokens) return;
  const int seq = seq_of_token(p.s, t);
  if (seq < 0) return;
  const SeqSpan sp = seq_span(p.s, seq, p.c.page_shift);
  int32_t lo, hi;
  seen_range(p.frame, p.window, sp.len - (sp.end - t), sp.len, lo, hi);
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) q[i] = __bfloat162float(p.q[t * p.q_token + h * p.q_head + lane + 32 * i]);
  for (int32_t j = lo; j < hi; ++j) {
    const int64_t r = cache_row(p.c, p.s, seq, j);
    const int64_t at = r + (static_cast<int64_t>(h / p.group) << p.c.page_shift);
    float s = 0.f, v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      s += q[i] * (r < 0 ? 0.f : cache_channel<D, FMT>(p.c.k, p.c.k_scale, at, lane + 32 * i));
      v[i] = r < 0 ? 0.f : cache_channel<D, FMT>(p.c.v, p.c.v_scale, at, lane + 32 * i);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= p.scale_log2;
    const float mn = s > m ? s : m;
    const float a = m == -INFINITY ? 0.f : ex2_approx(m - mn), w = s == -INFINITY ? 0.f : ex2_approx(s - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * a + w * v[i];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < E; ++i) p.o[t * p.o_token + h * p.o_head + lane + 32 * i] = __float2bfloat16(o[i] * inv);
  if (lane == 0)
    p.lse[static_cast<int64_t>(h) * p.s.num_tokens + t] =
        l == 0.f ? -INFINITY : m * 0.69314718055994531f + __logf(l);
}

}  // namespace dynrad
