// Attention of single tokens (16 rows at most of a sequence and K / V head): the same
// mathematics and schedule as cacheattn.cuh, for calls whose time is the reading of the
// cache, or a call's latency.
//
// The tensor-core tiles of cacheattn.cuh are 128 rows high whatever the rows, and want
// bf16 operands in shared memory.  For 8-bit pages and few rows that detour is the
// bound: 64 KB written and 96 KB read again by the products for every 33 KB of 128
// keys; and one row's softmax over 128 keys takes one thread some 2,900 clocks.  Here
// a warp turns the stored bytes into register fragments of 16 x 8 x 16 products
// (warp_mma.cuh) and nothing goes back: shared memory holds the bytes alone, once
// written and once read, and 128 keys are eight warps' work.
//
// The keys are the products' 16 rows, since there are more of them than query rows:
// S^T = K Q^T and O^T = V^T P^T, with 8 query rows a column tile (NT = 1 or 2 of
// them).  Eight rows then cost half the products and accumulators of the other way
// round, and the registers so freed hold more warps, which hide the unpacking.
//
// Fragments without a shuffle.  The products sum over channels (K Q^T) or keys
// (V^T P^T) in any order and their rows may be any keys or channels, so they are
// named to suit 16-byte reads (thread 4 g + t of the warp):
//   K Q^T    rows g and g + 8 are the keys k = 4 (g & 1) + g / 2 and k + 8; thread t
//            has the 16 channels of chunk t (and t + 4): word u of it is step u's
//            operand;
//   V^T P^T  P^T, transposed by movmatrix, sums over the keys t, 4 + t, 8 + t,
//            12 + t; rows g and g + 8 of channel tile j are the channels
//            16 c(g) + 2 j and + 1 (8 c(g) + .. at D = 64), bytes 2 j and 2 j + 1 of
//            what the thread read.
// The bytes lie in shared memory so that the threads served together meet
// different banks: 16-byte chunk c of row r at c ^ (r & 7) (D = 128).  At D = 64, K's
// row r takes place 2 (r & 3) + r / 4 of its eight and V's chunk c is at
// c ^ ((r / 2) & 3).
//
// A segment's 16-key blocks (8-bit: pairs of them) go to the warps in turn, each warp
// with a ring of its own, filled by cp.async, and its own max, sum and O.  At the end of
// a segment they are joined in shared memory while the SM's other CTAs read on.  An SM
// runs twelve warps: two CTAs of six, or three of four (8-bit, NT = 1).
//
// Measured on 8 K / V heads of D 128 (the launch and its join, cold caches / the same call
// again):
//   3 x 131072 keys, 64 heads: e4m3 183 / 167 us (4.6 / 5.0 TB/s), int8 174 / 155 (4.8 / 5.4),
//     bf16 262 / 242 (6.1 / 6.6);
//   64 sequences of up to 16000 keys, 32 heads: int8 203 / 187 us (4.8 / 5.3), e4m3 215 / 202
//     (4.6 / 4.9), bf16 334 / 289 (5.7 / 6.6).
// 8-bit pages are bound by issue (unpacking a byte and scaling it), not by HBM.  Pairs
// of blocks share the softmax step's shuffles and votes: with single blocks and eight
// warps in each of three CTAs (80 registers) the 8-bit times were 182, 170 and 212 us;
// with twelve warps in one CTA 160 and 213 (joined less often, but nothing reads on
// meanwhile); in fours, 195 and 226 (one group in flight).
#pragma once

#include "cacheattn.cuh"
#include "warp_mma.cuh"

namespace dynrad {

constexpr int kTokenKeys = 16;       // keys of a block, the unit of loads and products

template <int D, int FMT, int NT>
struct CacheTokenCfg {
  static constexpr bool kRaw = FMT != kCacheBf16;
  static constexpr int kRows = 8 * NT;                          // rows of an item
  static constexpr int kWarps = kRaw && NT == 1 ? 4 : 6;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCtasPerSm = kRaw && NT == 1 ? 3 : 2;
  // blocks a warp takes at a time: two neighbours of 8-bit pages share one softmax step,
  // whose fixed costs weigh as much as a block's unpacking
  static constexpr int kSub = kRaw ? 2 : 1;
  static constexpr int kRowBytes = kRaw ? D : 2 * D;            // a key's K or V as stored
  static constexpr int kCodes = kTokenKeys * kRowBytes;
  static constexpr int kScales = kRaw ? kTokenKeys * (D / kCacheGroup) : 0;
  static constexpr int kStageBytes = 2 * (kCodes + kScales);    // K, V, K's scales, V's scales
  static constexpr int kStages = (kRaw ? 4 : 2) * (128 / D);
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kQ = NT * (D / 16) * 256;                // Q's operands, 8 bytes a step and lane
  static constexpr int kCtrl = 256 + kWarps * kRows * 8;
  static constexpr int kSmem = kWarps * kRingBytes + kQ + kCtrl;
  static_assert(kStages % kSub == 0, "whole groups of blocks");
  static_assert(kRows * D * 4 <= kRingBytes, "a warp's O over its ring");
  static_assert(kCtasPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

// CTAs of a split launch on an SM
constexpr int token_ctas_per_sm(bool raw, int nt) {
  return raw ? (nt == 1 ? CacheTokenCfg<128, kCacheInt8, 1>::kCtasPerSm : CacheTokenCfg<128, kCacheInt8, 2>::kCtasPerSm)
             : (nt == 1 ? CacheTokenCfg<128, kCacheBf16, 1>::kCtasPerSm : CacheTokenCfg<128, kCacheBf16, 2>::kCtasPerSm);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool fill) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool fill) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(fill ? 4 : 0) : "memory");
}

// 8 x 8 matrix of 16-bit values, a row of pairs in threads 4 r .. 4 r + 3: transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Byte K of a (in the low half) and of b -> a bf16 pair, before their scales: unpack4
// with the bytes of two words.  flip: 0x00800080, kept in a register.
template <int FMT, int K>
__device__ __forceinline__ uint32_t unpack_pair(uint32_t a, uint32_t b, uint32_t flip) {
  if (FMT == kCacheE4m3) {
    constexpr uint32_t kSel = ((4u + K) << 12) | ((8u | K) << 8) | (K << 4) | K;
    return static_cast<uint32_t>(static_cast<int32_t>(prmt<kSel>(a, b)) >> 4) & 0x87f087f0u;
  }
  constexpr uint32_t kSel = ((4u + K) << 12) | ((4u + K) << 8) | (K << 4) | K;
  return bytes_to_bf16x2((prmt<kSel>(a, b) & 0x00ff00ffu) ^ flip);
}

// What a thread carries through its warp's blocks of a segment.
template <int D, int NT>
struct TokenState {
  float o[NT][D / 16][4];     // O^T: of channel tile j rows g, g + 8; query rows 2 t, 2 t + 1
  float m[NT][2], l[NT][2];   // of query rows 2 t, 2 t + 1: max (log2 units), this thread's part of the sum
  int32_t rlo[NT][2], rhi[NT][2];   // what those rows see
  int k_off, v_off0, v_off1, ks_off, vs_off;  // where the thread reads (see the kernel)
  uint32_t flip;              // unpack_pair's constant
};

// From S^T of NB neighbouring blocks to P^T as the second products' operands, in bf16;
// updates max, sum and, when a max grew by more than 2^8, O.
// s[b][n][2 i + e]: key 16 b + 8 i + 4 (g & 1) + g / 2, query row 8 n + 2 t + e
template <int D, int NT, int NB>
__device__ __forceinline__ void token_softmax(TokenState<D, NT>& me, float (&s)[NB][NT][4], int key0, bool partial,
                                              float scale_log2, uint32_t (&pf)[NB][NT][2]) {
  constexpr int NJ = D / 16;
  const int g = (threadIdx.x & 31) >> 2;
  if (partial) {
    const int key = key0 + 4 * (g & 1) + (g >> 1);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int k = key + 16 * b + 8 * (u >> 1);
          if (k < me.rlo[n][u & 1] || k >= me.rhi[n][u & 1]) s[b][n][u] = -INFINITY;
        }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float mx[2], m_new[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[e] = fmaxf(s[0][n][e], s[0][n][2 + e]);
#pragma unroll
      for (int b = 1; b < NB; ++b) mx[e] = fmax3(mx[e], s[b][n][e], s[b][n][2 + e]);
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1)
#pragma unroll
      for (int e = 0; e < 2; ++e) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], x));
#pragma unroll
    for (int e = 0; e < 2; ++e) m_new[e] = fmaxf(me.m[n][e], mx[e] * scale_log2);
    // rescale when a max grew by more than 2^8, the first seen key's block included (m = -inf)
    if (__any_sync(0xffffffffu, m_new[0] > me.m[n][0] + 8.0f || m_new[1] > me.m[n][1] + 8.0f)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool need = m_new[e] > me.m[n][e] + 8.0f;
        const float alpha = need ? ex2_approx(me.m[n][e] - m_new[e]) : 1.0f;
        if (need) me.m[n][e] = m_new[e];
        me.l[n][e] *= alpha;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          me.o[n][j][e] *= alpha;
          me.o[n][j][2 + e] *= alpha;
        }
      }
    }
    const float ref[2] = {me.m[n][0] == -INFINITY ? 0.f : me.m[n][0], me.m[n][1] == -INFINITY ? 0.f : me.m[n][1]};
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) p[u] = ex2_approx(fmaf(s[b][n][u], scale_log2, -ref[u & 1]));
      me.l[n][0] += p[0] + p[2];
      me.l[n][1] += p[1] + p[3];
      pf[b][n][0] = transpose8x8(pack_bf16x2(p[0], p[1]));
      pf[b][n][1] = transpose8x8(pack_bf16x2(p[2], p[3]));
    }
  }
}

// Two blocks, 32 keys from key0 on, their bytes at st one after the other.  partial:
// some row of the item, which sees [lo, hi) and every row of it [lo_max, hi_min), does
// not see all of them.
template <int D, int FMT, int NT>
__device__ __forceinline__ void token_blocks(TokenState<D, NT>& me, const uint8_t* st, int key0, bool partial, int32_t lo,
                                             int32_t hi, int32_t lo_max, int32_t hi_min, float scale_log2,
                                             const uint2* qs, volatile int* poison) {
  using C = CacheTokenCfg<D, FMT, NT>;
  constexpr int KW = D / 64, VB = D / 8, NJ = D / 16, NB = C::kSub, SW = D / kCacheGroup;
  const int t = threadIdx.x & 3;
  // odd: some scale's factor takes more than a shift of its byte (odd_scale); rare
  uint32_t kbyte[NB][2][KW], vbyte[NB][4];
  bool odd_here = false;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        kbyte[b][i][w] = st[b * C::kStageBytes + me.ks_off + i * 8 * SW + w * 2];
        odd_here = odd_here || odd_scale<FMT>(kbyte[b][i][w]);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      vbyte[b][i] = st[b * C::kStageBytes + me.vs_off + i * 4 * SW];
      odd_here = odd_here || odd_scale<FMT>(vbyte[b][i]);
    }
  }
  const bool odd = __any_sync(0xffffffffu, odd_here);
  // S^T = K Q^T
  float s[NB][NT][4] = {};
  uint32_t pf[NB][NT][2];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      uint32_t kf[2][2][4];     // [key row][operand register][step]
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(st + b * C::kStageBytes + i * 8 * D +
                                                        (w == 0 ? me.k_off : me.k_off ^ 64));
        unpack4<FMT>(x.x, kf[i][0][0], kf[i][1][0]);
        unpack4<FMT>(x.y, kf[i][0][1], kf[i][1][1]);
        unpack4<FMT>(x.z, kf[i][0][2], kf[i][1][2]);
        unpack4<FMT>(x.w, kf[i][0][3], kf[i][1][3]);
      }
      if (!odd) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t f = kbyte[b][i][w] * 0x00800080u + kUnpackBias<FMT> * 0x00800080u;
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) kf[i][e][u] = mul_bf16x2(kf[i][e][u], f);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t f1, f2;
          scale_factors<FMT>(kbyte[b][i][w], f1, f2);
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) kf[i][e][u] = mul_bf16x2(mul_bf16x2(kf[i][e][u], f1), f2);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint2 q = qs[(n * NJ + w * 4 + u) * 32];
          mma_16816(s[b][n], kf[0][0][u], kf[1][0][u], kf[0][1][u], kf[1][1][u], q.x, q.y);
        }
    }
  token_softmax<D, NT, NB>(me, s, key0, partial, scale_log2, pf);
  // O^T += V^T P^T: V rows t, 4 + t (first keys of the sum), 8 + t, 12 + t
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    uint32_t x[4][VB / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* src = st + b * C::kStageBytes + ((i & 1) ? me.v_off1 : me.v_off0) + (i >> 1) * 8 * D;
      if constexpr (D == 128) {
        const uint4 v = *reinterpret_cast<const uint4*>(src);
        x[i][0] = v.x;
        x[i][1] = v.y;
        x[i][2] = v.z;
        x[i][3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        x[i][0] = v.x;
        x[i][1] = v.y;
      }
    }
    if (partial) {     // what no row sees, and NaN that some see, stay out of the product (cacheattn.cuh)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + 16 * b + t + 4 * i;
        const bool seen = key >= lo && key < hi;
        if (!seen || (vbyte[b][i] == kCacheNanScale && (key < lo_max || key >= hi_min))) {
          if (seen) *poison = 1;
          vbyte[b][i] = 127;
#pragma unroll
          for (int w = 0; w < VB / 4; ++w) x[i][w] = 0u;
        }
      }
    }
    uint32_t f1[4], f2[4] = {kBf16One, kBf16One, kBf16One, kBf16One};
#pragma unroll
    for (int i = 0; i < 4; ++i) f1[i] = vbyte[b][i] * 0x00800080u + kUnpackBias<FMT> * 0x00800080u;
    if (odd) {
#pragma unroll
      for (int i = 0; i < 4; ++i) scale_factors<FMT>(vbyte[b][i], f1[i], f2[i]);
    }
    const uint32_t fa = prmt<0x5410>(f1[0], f1[1]), fb = prmt<0x5410>(f1[2], f1[3]);
#pragma unroll
    for (int w = 0; w < VB / 4; ++w) {
      uint32_t a[4] = {unpack_pair<FMT, 0>(x[0][w], x[1][w], me.flip), unpack_pair<FMT, 1>(x[0][w], x[1][w], me.flip),
                       unpack_pair<FMT, 2>(x[0][w], x[1][w], me.flip), unpack_pair<FMT, 3>(x[0][w], x[1][w], me.flip)};
      uint32_t c[4] = {unpack_pair<FMT, 0>(x[2][w], x[3][w], me.flip), unpack_pair<FMT, 1>(x[2][w], x[3][w], me.flip),
                       unpack_pair<FMT, 2>(x[2][w], x[3][w], me.flip), unpack_pair<FMT, 3>(x[2][w], x[3][w], me.flip)};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        a[u] = mul_bf16x2(a[u], fa);
        c[u] = mul_bf16x2(c[u], fb);
      }
      if (odd) {
        const uint32_t ga = prmt<0x5410>(f2[0], f2[1]), gb = prmt<0x5410>(f2[2], f2[3]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          a[u] = mul_bf16x2(a[u], ga);
          c[u] = mul_bf16x2(c[u], gb);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_16816(me.o[n][2 * w], a[0], a[1], c[0], c[1], pf[b][n][0], pf[b][n][1]);
        mma_16816(me.o[n][2 * w + 1], a[2], a[3], c[2], c[3], pf[b][n][0], pf[b][n][1]);
      }
    }
  }
}

// One block of bf16 pages: ldmatrix brings both operands as the products want them, K's
// and V's rows named as above (row i of eight is key 4 (i & 1) + i / 2), channels in
// order.  Chunk c of a row lies at c ^ (row & 7).
template <int D, int NT>
__device__ __forceinline__ void token_block_bf16(TokenState<D, NT>& me, const uint8_t* st, int key0, bool partial,
                                                 int32_t lo, int32_t hi, int32_t lo_max, int32_t hi_min,
                                                 float scale_log2, const uint2* qs, volatile int* poison) {
  constexpr int NJ = D / 16, RB = 2 * D;
  const int lane = threadIdx.x & 31, i = lane & 7;
  const int key = 4 * (i & 1) + (i >> 1);
  const uint32_t base = smem_u32(st);
  // lane's row of the four 8 x 8 matrices: K: keys, keys + 8, then the next eight
  // channels; V: keys, the next channels, then keys + 8
  const int krow = key + ((lane >> 3) & 1) * 8, kc = lane >> 4;
  const int vrow = key + (lane >> 4) * 8, vc = (lane >> 3) & 1;
  float s[1][NT][4] = {};
  uint32_t pf[1][NT][2];
#pragma unroll
  for (int u = 0; u < NJ; ++u) {
    uint32_t a0, a1, a2, a3;
    ldsm_x4(base + krow * RB + (((2 * u + kc) ^ key) << 4), a0, a1, a2, a3);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint2 q = qs[(n * NJ + u) * 32];
      mma_16816(s[0][n], a0, a1, a2, a3, q.x, q.y);
    }
  }
  token_softmax<D, NT, 1>(me, s, key0, partial, scale_log2, pf);
  if (partial) {     // what no row sees, and what is not finite of what some see, stay out (cacheattn.cuh)
#pragma unroll 1
    for (int u = lane; u < kTokenKeys * (D / 8); u += 32) {
      const int r = u / (D / 8), k = key0 + r;
      if (k >= lo_max && k < hi_min) continue;
      uint4* at = reinterpret_cast<uint4*>(const_cast<uint8_t*>(st) + kTokenKeys * RB) + u;
      const uint4 x = *at;
      uint4 y = make_uint4(0u, 0u, 0u, 0u);
      if (k >= lo && k < hi) {
        y = make_uint4(finite_bf16x2(x.x), finite_bf16x2(x.y), finite_bf16x2(x.z), finite_bf16x2(x.w));
        if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) *poison = 1;
      }
      *at = y;
    }
    __syncwarp();
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    uint32_t a0, a1, a2, a3;
    ldsm_x4_trans(base + kTokenKeys * RB + vrow * RB + (((2 * j + vc) ^ key) << 4), a0, a1, a2, a3);
#pragma unroll
    for (int n = 0; n < NT; ++n) mma_16816(me.o[n][j], a0, a1, a2, a3, pf[0][n][0], pf[0][n][1]);
  }
}

template <int D, int FMT, int NT>
__global__ void __launch_bounds__(CacheTokenCfg<D, FMT, NT>::kThreads, CacheTokenCfg<D, FMT, NT>::kCtasPerSm)
    cache_token_kernel(const CacheAttnParams p) {
  using C = CacheTokenCfg<D, FMT, NT>;
  constexpr int KW = D / 64;                 // 16-byte chunks of a key that a thread reads
  constexpr int VB = D / 8;                  // bytes of a V row that a thread reads: 16 or 8
  constexpr int NJ = D / 16;                 // channel tiles, and steps of K Q^T
  extern __shared__ __align__(128) uint8_t token_smem[];
  uint2* q_s = reinterpret_cast<uint2*>(token_smem + C::kWarps * C::kRingBytes);   // [row tile][step][lane]
  uint8_t* ctrl = token_smem + C::kWarps * C::kRingBytes + C::kQ;
  CacheRun* run = reinterpret_cast<CacheRun*>(ctrl);
  volatile int* poison = reinterpret_cast<volatile int*>(ctrl + 32);
  CacheSeg* seg_s = reinterpret_cast<CacheSeg*>(ctrl + 64);
  float2* ml = reinterpret_cast<float2*>(ctrl + 256);                                // [warp][row]
  static_assert(sizeof(CacheRun) <= 32 && 64 + sizeof(CacheSeg) <= 256, "control block");

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int item_tokens = p.tile_tokens;
  const int ps = p.c.page_shift;
  int place, head;
  int64_t off = 0, left = 1;
  if (p.split) {
    plan_run<C::kThreads>(p, item_tokens, reinterpret_cast<int32_t*>(token_smem), reinterpret_cast<int64_t*>(ml), run);
    left = run->left;
    off = left > 0 ? run->off : 0;
    head = left > 0 ? run->head : 0;
    place = left > 0 ? run->place : 0;
    if (threadIdx.x == 0)
      p.part_desc[2 * blockIdx.x] = p.part_desc[2 * blockIdx.x + 1] = make_int4(0, 0, kPartNone, 0);
  } else {
    head = blockIdx.y;
    place = p.slots - 1 - static_cast<int>(blockIdx.x);
  }

  uint8_t* ring = token_smem + warp * C::kRingBytes;
  const uint32_t ring_u = smem_u32(ring);
  TokenState<D, NT> me;
  // where this thread reads: chunk t of its first key; its part of V rows t and t + 4
  // (rows t + 8 and t + 12 lie eight rows further on)
  const int krow = (g & 1) * 4 + (g >> 1);
  me.k_off = D == 128 ? krow * 128 + ((t ^ krow) << 4) : g * 64 + (t << 4);
  const int vc = D == 128 ? krow : (g & 1) | ((g & 2) << 1) | ((g & 4) >> 1);   // c(g)
  auto v_place = [&](int r) -> int {
    return C::kCodes + (D == 128 ? r * 128 + ((vc ^ r) << 4) : r * 64 + (((vc >> 1) ^ (r >> 1)) << 4) + (vc & 1) * 8);
  };
  me.v_off0 = v_place(t);
  me.v_off1 = v_place(t + 4);
  me.flip = 0x00800080u ^ (gridDim.z - 1u);   // gridDim.z is 1: a constant that stays in a register
  // scale bytes: of this thread's key and chunk, and of V row t and its channels
  me.ks_off = 2 * C::kCodes + krow * (D / kCacheGroup) + (t >> 1);
  me.vs_off = 2 * C::kCodes + C::kScales + t * (D / kCacheGroup) + vc * VB / kCacheGroup;
  // where this lane's 16-byte chunks of a block go: chunk u = lane + 32 i is row
  // u / (D / 16); i = 2, 3 (D = 128) lie eight rows further on
  [[maybe_unused]] int k_dst[2], v_dst[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = lane + 32 * i, r = u / (D / 16), c = u % (D / 16);
    k_dst[i] = D == 128 ? r * 128 + ((c ^ r) << 4) : ((r & 8) + (r & 3) * 2 + ((r >> 2) & 1)) * 64 + (c << 4);
    v_dst[i] = C::kCodes + (D == 128 ? r * 128 + ((c ^ r) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  }

  while (left > 0) {
    // the next segment, found by one warp
    __syncthreads();
    if (warp == 0) {
      CacheSeg sg;
      for (;;) {
        sg.it = find_item(p, item_tokens, place);
        const int32_t units = item_units(p, item_tokens, sg.it);
        sg.head = head;
        sg.sa = 0;
        sg.sb = sg.it.steps;
        sg.part = -1;
        if (p.split) {
          const int64_t take = min(left, static_cast<int64_t>(units) - off);
          if (units > 0) {
            sg.sa = unit_step(p, item_tokens, sg.it, off);
            sg.sb = unit_step(p, item_tokens, sg.it, off + take);
            left -= take;
          }
          off = 0;
        } else {
          left = 0;
        }
        if (++place == p.slots) {
          place = 0;
          if (++head == p.c.heads) left = 0;
        }
        const bool use = units > 0 && (sg.sb > sg.sa || sg.it.steps == 0);
        if (use && !(sg.sa == 0 && sg.sb == sg.it.steps)) {
          sg.part = sg.sa > 0 ? 0 : 1;
          if (lane == 0)
            p.part_desc[2 * blockIdx.x + sg.part] =
                make_int4(sg.it.tok0, sg.head, sg.sb == sg.it.steps ? kPartLast : kPartOpen, sg.it.ntok);
        }
        sg.end = use ? 0 : 1;
        if (use || left <= 0) break;
      }
      if (lane == 0) {
        sg.narrow = left > 0;        // more segments follow
        *seg_s = sg;
        *poison = 0;
      }
    }
    __syncthreads();
    const CacheItem it = seg_s->it;
    const int sa = seg_s->sa, sb = seg_s->sb, part = seg_s->part, kvh = seg_s->head;
    if (seg_s->end) break;
    left = seg_s->narrow ? max(left, static_cast<int64_t>(1)) : 0;   // warp 0 keeps the count

    const int rows = it.ntok * p.group;
    // 16-key blocks [b0, b1) of the segment, in groups of kSub (blocks of a group that
    // nobody sees are not loaded: whatever lies there is masked); the groups go to the
    // warps in turn
    const int64_t ka = max(static_cast<int64_t>(it.lo), static_cast<int64_t>(it.step0 + sa) << 7);
    const int64_t kb = min(static_cast<int64_t>(it.hi), static_cast<int64_t>(it.step0 + sb) << 7);
    const int b0 = static_cast<int>(ka >> 4), b1 = sb > sa ? static_cast<int>((kb + 15) >> 4) : b0;
    const int32_t* table = p.s.page_table + static_cast<int64_t>(it.seq) * p.s.table_stride;
    auto page_of = [&](int b) -> int32_t { return b >= b0 && b < b1 ? table[b >> (ps - 4)] : 0; };
    auto load = [&](int b, int32_t pg, int stage) {
      if (b >= b0 && b < b1) {
        const bool good = pg >= 0 && pg < p.c.num_pages;
        if (!good && lane == 0) record_error(DYNRAD_ERR_DEVICE);
        // a page outside the pool is filled with zeros
        const int64_t row = good ? (((static_cast<int64_t>(pg) * p.c.heads + kvh) << ps) + ((b << 4) & ((1 << ps) - 1))) : 0;
        const uint8_t* kc = p.c.k + row * C::kRowBytes + lane * 16;
        const uint8_t* vcodes = p.c.v + row * C::kRowBytes + lane * 16;
        const uint32_t dst = ring_u + stage * C::kStageBytes;
        if constexpr (C::kRaw) {
#pragma unroll
          for (int i = 0; i < C::kCodes / 512; ++i) {
            cp_async16(dst + k_dst[i & 1] + (i >> 1) * 1024, kc + i * 512, good);
            cp_async16(dst + v_dst[i & 1] + (i >> 1) * 1024, vcodes + i * 512, good);
          }
          constexpr int W = C::kScales / 4;     // 16 or 8 words each
          if (lane < 2 * W) {
            const uint8_t* sc = (lane < W ? p.c.k_scale : p.c.v_scale) + row * (D / kCacheGroup) + (lane % W) * 4;
            cp_async4(dst + 2 * C::kCodes + lane * 4, sc, good);
          }
        } else {
#pragma unroll
          for (int i = 0; i < C::kCodes / 512; ++i) {
            const int u = lane + 32 * i, r = u / (D / 8), to = r * C::kRowBytes + (((u % (D / 8)) ^ (r & 7)) << 4);
            cp_async16(dst + to, kc + i * 512, good);
            cp_async16(dst + C::kCodes + to, vcodes + i * 512, good);
          }
        }
      }
    };
    constexpr int SUB = C::kSub, GROUPS = C::kStages / SUB;   // groups in the ring
    int b = b0 / SUB * SUB + warp * SUB;
    {
      int32_t pg[C::kStages];
#pragma unroll
      for (int s = 0; s < C::kStages; ++s) pg[s] = page_of(b + s / SUB * C::kWarps * SUB + s % SUB);
#pragma unroll
      for (int s = 0; s < C::kStages; ++s) {
        load(b + s / SUB * C::kWarps * SUB + s % SUB, pg[s], s);
        if (s % SUB == SUB - 1) asm volatile("cp.async.commit_group;" ::: "memory");
      }
    }
    int32_t next_page[SUB];
#pragma unroll
    for (int u = 0; u < SUB; ++u) next_page[u] = page_of(b + GROUPS * C::kWarps * SUB + u);

    // Q's operands: query row 8 n + g, step u.  8-bit: of chunk t + 4 (u / 4) the channels
    // of word u % 4; bf16: channels 16 u + 2 t and 16 u + 8 + 2 t
    for (int x = warp; x < NT * NJ; x += C::kWarps) {
      const int u = x % NJ, r = 8 * (x / NJ) + g, tok = r / p.group;
      uint2 q = make_uint2(0u, 0u);
      if (r < rows) {
        const __nv_bfloat16* src = p.q + (it.tok0 + tok) * p.q_token + (kvh * p.group + r - tok * p.group) * p.q_head;
        if constexpr (C::kRaw) {
          q = *reinterpret_cast<const uint2*>(src + (t + 4 * (u >> 2)) * 16 + (u & 3) * 4);
        } else {
          q.x = *reinterpret_cast<const uint32_t*>(src + 16 * u + 2 * t);
          q.y = *reinterpret_cast<const uint32_t*>(src + 16 * u + 8 + 2 * t);
        }
      }
      q_s[x * 32 + lane] = q;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
        me.rlo[n][e] = 0;
        me.rhi[n][e] = INT32_MAX;     // rows that are not there count as seeing all
        if (r < rows) seen_range(p.frame, p.window, it.pos0 + r / p.group, it.len, me.rlo[n][e], me.rhi[n][e]);
        me.m[n][e] = -INFINITY;
        me.l[n][e] = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) me.o[n][j][e] = me.o[n][j][2 + e] = 0.f;
      }
    __syncthreads();

    int stage = 0;
#pragma unroll 1
    for (; b < b1; b += C::kWarps * SUB) {
      asm volatile("cp.async.wait_group %0;" ::"n"(GROUPS - 1) : "memory");
      __syncwarp();
      const uint8_t* st = ring + stage * C::kStageBytes;
      const int key0 = b << 4;
      const bool partial = key0 < it.lo_max || key0 > it.hi_min - kTokenKeys * SUB;
      if constexpr (C::kRaw)
        token_blocks<D, FMT, NT>(me, st, key0, partial, it.lo, it.hi, it.lo_max, it.hi_min, p.scale_log2, q_s + lane,
                                 poison);
      else
        token_block_bf16<D, NT>(me, st, key0, partial, it.lo, it.hi, it.lo_max, it.hi_min, p.scale_log2, q_s + lane,
                                poison);
      __syncwarp();      // every lane has read the stage
#pragma unroll
      for (int u = 0; u < SUB; ++u) load(b + GROUPS * C::kWarps * SUB + u, next_page[u], stage + u);
      asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
      for (int u = 0; u < SUB; ++u) next_page[u] = page_of(b + (GROUPS + 1) * C::kWarps * SUB + u);
      stage = stage + SUB == C::kStages ? 0 : stage + SUB;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();

    // join the warps: O over their rings
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) me.l[n][e] += __shfl_xor_sync(0xffffffffu, me.l[n][e], x);
        const int r = 8 * n + 2 * t + e;
        if (g == 0) ml[warp * C::kRows + r] = make_float2(me.m[n][e], me.l[n][e]);
        float* dst = reinterpret_cast<float*>(ring) + r * D;
        if constexpr (C::kRaw) {      // the thread's run of channels
#pragma unroll
          for (int j = 0; j < NJ; j += 2)
            *reinterpret_cast<float4*>(dst + vc * VB + 2 * j) =
                make_float4(me.o[n][j][e], me.o[n][j][2 + e], me.o[n][j + 1][e], me.o[n][j + 1][2 + e]);
        } else {
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            dst[16 * j + g] = me.o[n][j][e];
            dst[16 * j + 8 + g] = me.o[n][j][2 + e];
          }
        }
      }
    __syncthreads();
    const bool poisoned = *poison != 0;
    for (int u = threadIdx.x; u < rows * (D / 4); u += C::kThreads) {
      const int r = u / (D / 4), c = u % (D / 4);
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) mm = fmaxf(mm, ml[w * C::kRows + r].x);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        const float2 x = ml[w * C::kRows + r];
        const float f = join_weight(x.x, mm);
        const float4 v = reinterpret_cast<const float4*>(token_smem + w * C::kRingBytes + r * (D * 4))[c];
        ll = fmaf(x.y, f, ll);
        a.x = fmaf(v.x, f, a.x);
        a.y = fmaf(v.y, f, a.y);
        a.z = fmaf(v.z, f, a.z);
        a.w = fmaf(v.w, f, a.w);
      }
      const int tok = r / p.group, qhead = kvh * p.group + r - tok * p.group;
      if (poisoned) {
        int32_t lo, hi;
        seen_range(p.frame, p.window, it.pos0 + tok, it.len, lo, hi);
        const int first = max(lo, static_cast<int>(ka)), last = min(static_cast<int64_t>(hi), kb);
        for (int key = first; key < last; ++key) {
          if (key >= it.lo_max && key < it.hi_min) continue;
          const int64_t at = cache_row(p.c, p.s, it.seq, key);
          if (at < 0) continue;
          const int64_t row = at + (static_cast<int64_t>(kvh) << ps);
          if constexpr (C::kRaw) {
            if (p.c.v_scale[row * (D / kCacheGroup) + c * 4 / kCacheGroup] == kCacheNanScale)
              a.x = a.y = a.z = a.w = __int_as_float(0x7fffffff);
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p.c.v + row * C::kRowBytes + c * 8);
            auto add = [](float& to, uint32_t bits) {
              if ((bits & 0x7f800000u) == 0x7f800000u) to += __uint_as_float(bits);
            };
            add(a.x, v.x << 16);
            add(a.y, v.x & 0xffff0000u);
            add(a.z, v.y << 16);
            add(a.w, v.y & 0xffff0000u);
          }
        }
      }
      const int64_t token = it.tok0 + tok;
      if (part >= 0) {
        const int64_t prow = (2 * static_cast<int64_t>(blockIdx.x) + part) * C::kRows + r;
        reinterpret_cast<float4*>(p.part_o + prow * D)[c] = a;
        if (c == 0) p.part_ml[prow] = make_float2(mm, ll);
      } else {
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        *reinterpret_cast<uint2*>(p.o + token * p.o_token + qhead * p.o_head + c * 4) =
            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        if (c == 0)
          p.lse[static_cast<int64_t>(qhead) * p.s.num_tokens + token] =
              ll == 0.f ? -INFINITY : mm * 0.69314718055994531f + __logf(ll);
      }
    }
  }
}

}  // namespace dynrad
