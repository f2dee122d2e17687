// Paged K / V cache: where a token stands, and the kernels that write new
// tokens into the pages and read them back.
//
// Layout.  A page holds `page` tokens of every K / V head, head-major
// ([num_pages][heads][page][D]), so the tokens of one head of one page are one
// contiguous tile: the unit the attention kernel loads.  Formats: bf16, or 8
// bits a channel (e4m3 / int8) with one scale for every 32 channels of a token,
// kept as the biased exponent byte of a power of two
// ([num_pages][heads][page][D / 32]).  A power of two makes what is stored an
// exact bf16 number (4 or 8 significant bits), so reading back and the
// attention's operands round nothing: the one rounding is the write's.
//
// Quantisation of 32 channels x with a = max |x|:  s = 2^e with the least e
// such that a <= c_max s (c_max = 448 for e4m3, 127 for int8), e >= -117 (then
// the smallest e4m3 step 2^-9 s is still a normal bf16 number); code =
// round-to-nearest-even(x / s); magnitudes over 240 * 2^120 (e4m3) or 127 * 2^121
// (int8), whose code would stand for 2^128, are stored as those.  An infinity or NaN among the 32 gives the
// exponent byte 255, and all 32 read back as NaN.
//
// Both kernels are one pass over the data and bound by HBM: per (token, head)
// they move 2 * D * 2 bytes of bf16 and 2 * (D + D / 32) of the 8-bit pages
// (2 * D * 2 again for bf16 pages).  Small calls are bound by the chain of loads that
// finds a token's place (sequence, its bounds, its page): 5-6 us a launch.
#pragma once

#include "common.cuh"

namespace dynrad {

constexpr int kCacheBf16 = 0, kCacheE4m3 = 1, kCacheInt8 = 2;
constexpr int kCacheGroup = 32;          // channels under one scale
constexpr int kCacheLeastExp = -117;     // least exponent of a scale
constexpr uint32_t kCacheNanScale = 255;

struct CacheDev {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  int64_t num_pages;
  int32_t heads;
  int32_t page_shift;   // log2(tokens a page)
};

struct SeqsDev {
  const int32_t* page_table;
  const int32_t* cu_seq;
  const int32_t* kv_len;
  int64_t table_stride;
  int32_t num_seqs;
  int32_t max_pages;
  int32_t num_tokens;
};

// Tokens [begin, end) and cached length of a sequence, held inside the caller's
// arrays whatever the device arrays say (a bad value is recorded).
struct SeqSpan {
  int32_t begin, end, len;
};

__device__ __forceinline__ SeqSpan seq_span(const SeqsDev& s, int i, int page_shift) {
  SeqSpan r;
  const int32_t a = s.cu_seq[i], b = s.cu_seq[i + 1], n = s.kv_len[i];
  r.begin = min(max(a, 0), s.num_tokens);
  r.end = min(max(b, r.begin), s.num_tokens);
  const int64_t cap = static_cast<int64_t>(s.max_pages) << page_shift;
  r.len = static_cast<int32_t>(min(static_cast<int64_t>(max(n, 0)), cap));
  if (r.begin != a || r.end != b || r.len != n) record_error(DYNRAD_ERR_DEVICE);
  return r;
}

// The sequence that token t belongs to, -1 if none (t lies behind the last one).  A
// warp's search, 32 entries at a time: one round trip for 32 sequences, two for 1024.
__device__ __forceinline__ int seq_of_token(const SeqsDev& s, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = s.num_seqs;   // last i with cu_seq[i] <= t
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, i = lo + lane * step;
    const int n = __popc(__ballot_sync(0xffffffffu, i < hi && s.cu_seq[i] <= t));
    lo += max(n - 1, 0) * step;
    hi = min(lo + step, hi);
  }
  return s.cu_seq[lo] <= t && t < s.cu_seq[lo + 1] ? lo : -1;
}

// Row (page * heads) << page_shift | slot of a cached position; a page outside the
// pool is recorded and gives -1.  A row's head h is page tokens further on.
__device__ __forceinline__ int64_t cache_row(const CacheDev& c, const SeqsDev& s, int seq, int32_t pos) {
  const int32_t pg = s.page_table[static_cast<int64_t>(seq) * s.table_stride + (pos >> c.page_shift)];
  if (pg < 0 || pg >= c.num_pages) {
    record_error(DYNRAD_ERR_DEVICE);
    return -1;
  }
  return ((static_cast<int64_t>(pg) * c.heads) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// 2^e as a bf16 pair, -126 <= e <= 127
__device__ __forceinline__ uint32_t pow2_bf16x2(int e) {
  const uint32_t b = static_cast<uint32_t>(e + 127) << 7;
  return b | (b << 16);
}

// Bytes of a (0 .. 3) and b (4 .. 7) by the selector's four-bit fields; bit 3 of a
// field spreads the byte's sign instead.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "n"(SEL));
  return r;
}

// A pair of bytes u in 0 .. 255, alone in the halves of `w`, -> (u - 128) / 128: as
// bf16 bits u is the number u 2^-133 (the subnormals run into the normals), so one
// exact multiply-add makes it u / 128 - 1.
__device__ __forceinline__ uint32_t bytes_to_bf16x2(uint32_t w) { return fma_bf16x2(w, 0x7e807e80u, 0xbf80bf80u); }

// Four stored bytes -> four bf16 numbers, before their scale: the value times
// 2^-kUnpackBias.  e4m3: the seven low bits moved to bf16's exponent and mantissa
// are the value times 2^-120 (subnormals included); one permute puts each byte in a
// high half, with the first one's sign spread over the byte above it (selector bit
// 3), so that one arithmetic shift by 4 carries both signs along and a mask clears
// the rest.  int8: with the sign bit flipped the byte is the value + 128.
template <int FMT>
constexpr uint32_t kUnpackBias = FMT == kCacheE4m3 ? 120u : 7u;

template <int FMT>
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == kCacheE4m3) {
    lo = static_cast<uint32_t>(static_cast<int32_t>(prmt<0x1804u>(w, 0u)) >> 4) & 0x87f087f0u;
    hi = static_cast<uint32_t>(static_cast<int32_t>(prmt<0x3a24u>(w, 0u)) >> 4) & 0x87f087f0u;
  } else {
    w ^= 0x80808080u;
    lo = bytes_to_bf16x2(prmt<0x4140u>(w, 0u));
    hi = bytes_to_bf16x2(prmt<0x4342u>(w, 0u));
  }
}

// Factors of a scale byte for what unpack4 gives.  The first alone does (and the
// second is 1) but for the NaN byte and scales whose factor would leave bf16's
// range (over 2^7 for e4m3, 2^120 for int8).
constexpr uint32_t kBf16One = 0x3f803f80u;

template <int FMT>
__device__ __forceinline__ bool odd_scale(uint32_t byte) {
  return byte > 254u - kUnpackBias<FMT>;
}

template <int FMT>
__device__ __forceinline__ void scale_factors(uint32_t byte, uint32_t& f1, uint32_t& f2) {
  f1 = byte * 0x00800080u + kUnpackBias<FMT> * 0x00800080u;   // the exponent field, twice
  f2 = kBf16One;
  if (odd_scale<FMT>(byte)) {
    if (byte == kCacheNanScale) {
      f1 = 0x7fc07fc0u;
    } else {
      f1 = 0x7f007f00u;            // 2^127
      f2 = pow2_bf16x2(static_cast<int>(byte + kUnpackBias<FMT>) - 254);
    }
  }
}

// 16 stored bytes under one scale -> 16 bf16 numbers.
template <int FMT>
__device__ __forceinline__ void dequant16(const uint4& w, uint32_t byte, uint4& o0, uint4& o1) {
  uint32_t f1, f2;
  scale_factors<FMT>(byte, f1, f2);
  unpack4<FMT>(w.x, o0.x, o0.y);
  unpack4<FMT>(w.y, o0.z, o0.w);
  unpack4<FMT>(w.z, o1.x, o1.y);
  unpack4<FMT>(w.w, o1.z, o1.w);
  o0.x = mul_bf16x2(o0.x, f1); o0.y = mul_bf16x2(o0.y, f1); o0.z = mul_bf16x2(o0.z, f1); o0.w = mul_bf16x2(o0.w, f1);
  o1.x = mul_bf16x2(o1.x, f1); o1.y = mul_bf16x2(o1.y, f1); o1.z = mul_bf16x2(o1.z, f1); o1.w = mul_bf16x2(o1.w, f1);
  if (f2 != kBf16One) {
    o0.x = mul_bf16x2(o0.x, f2); o0.y = mul_bf16x2(o0.y, f2); o0.z = mul_bf16x2(o0.z, f2); o0.w = mul_bf16x2(o0.w, f2);
    o1.x = mul_bf16x2(o1.x, f2); o1.y = mul_bf16x2(o1.y, f2); o1.z = mul_bf16x2(o1.z, f2); o1.w = mul_bf16x2(o1.w, f2);
  }
}

__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four bf16 numbers (two pairs), already divided by their scale -> four codes.
template <int FMT>
__device__ __forceinline__ uint32_t pack4(uint32_t p0, uint32_t p1) {
  const float a = __uint_as_float(p0 << 16), b = __uint_as_float(p0 & 0xffff0000u);
  const float c = __uint_as_float(p1 << 16), d = __uint_as_float(p1 & 0xffff0000u);
  if (FMT == kCacheE4m3) return cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
  const uint32_t i0 = __float2int_rn(a), i1 = __float2int_rn(b), i2 = __float2int_rn(c), i3 = __float2int_rn(d);
  return __byte_perm(__byte_perm(i0, i1, 0x0040), __byte_perm(i2, i3, 0x0040), 0x5410);
}

// Exponent of the scale for 32 channels whose largest |x| has the bf16 bits `a`
// (finite).  448 = 1.75 * 2^8 and 127 = (1 + 126 / 128) * 2^6, so the mantissa
// field decides between two exponents.
template <int FMT>
__device__ __forceinline__ int scale_exponent(uint32_t a) {
  const int ex = static_cast<int>(a >> 7) - 127;   // subnormals give -127: below the least exponent either way
  const uint32_t man = a & 127u;
  const int e = FMT == kCacheE4m3 ? ex - 8 + (man > 96u ? 1 : 0) : ex - 6 + (man > 126u ? 1 : 0);
  return max(e, kCacheLeastExp);
}

constexpr int kCacheThreads = 256;
// A CTA takes up to 8 tokens (one for each warp to look up) and goes through them head
// by head, tokens inside: runs of 8 rows in the pages, which are head-major.  Measured
// over 32,760 tokens of 40 heads (write e4m3 / write bf16 / read e4m3, us): heads
// inside 216 / 252 / 212; tokens inside, 32 tokens 189 / 268 / 212, 16 tokens 183 /
// 228 / 189, 8 tokens 183 / 216 / 171; with four units' loads in flight (here) 173 /
// 220 / 169, which is 5.9-6.1 TB/s.  Few heads leave threads without a unit and the time
// to the look-ups of 4,096 CTAs (32,760 tokens at D = 128, write bf16 / write e4m3 / read
// e4m3): 8 heads 49 / 45 / 43 us (5.5 / 4.5 / 4.7 TB/s), 5 heads 35 / 37 / 33, 2 heads 23 /
// 29 / 25, one head 18 / 25 / 20 (1.8 / 1.0 / 1.2 TB/s).
constexpr int kCacheTokens = 8;
constexpr int kCacheCtasPerSm = 4;
constexpr int kCacheUnroll = 4;    // units whose loads a thread has in flight

struct CacheMoveParams {
  CacheDev c;
  SeqsDev s;
  const __nv_bfloat16* k_in;       // writing: from the tokens' rows
  const __nv_bfloat16* v_in;
  __nv_bfloat16* k_out;            // reading back: to them
  __nv_bfloat16* v_out;
  int64_t k_token, k_head, v_token, v_head;   // strides in elements
  int32_t tokens;                  // tokens a CTA takes
};

constexpr int64_t kRowNone = -1;     // nothing to do for this token
constexpr int64_t kRowZero = -2;     // read back as zeros

// Cache rows of the CTA's n tokens from t0 on, a warp a token.
__device__ __forceinline__ void place_tokens(const CacheDev& c, const SeqsDev& s, int t0, int n, int64_t* rows) {
  static_assert(kCacheTokens <= kCacheThreads / 32, "a warp a token");
  const int i = threadIdx.x >> 5;
  if (i < n) {
    const int t = t0 + i, seq = seq_of_token(s, t);
    int64_t row = kRowNone;
    if (seq >= 0) {
      const SeqSpan sp = seq_span(s, seq, c.page_shift);
      const int32_t pos = sp.len - (sp.end - t);
      row = pos < 0 || t >= sp.end ? kRowZero : cache_row(c, s, seq, pos);
      if (row < 0) row = kRowZero;
    }
    if ((threadIdx.x & 31) == 0) rows[i] = row;
  }
}

// Unit u of a CTA's n tokens: 16 channels (chunk c of C) of K (kv = 0) or V of one
// (token, head), the tokens of a head together.
struct CacheUnit {
  int tk, kv, h, c;
};

template <int C>
__device__ __forceinline__ CacheUnit cache_unit(uint32_t u, int heads, uint32_t n) {
  CacheUnit x;
  const uint32_t r = u / C, q = r / n;
  x.c = u % C;
  x.tk = r - q * n;
  x.kv = q >= static_cast<uint32_t>(heads) ? 1 : 0;
  x.h = static_cast<int>(q) - x.kv * heads;
  return x;
}

// A thread quantises (or copies) a unit: two 16-byte loads, one 16-byte store (two
// for bf16); its neighbour has the other half of the 32 channels under the scale.
template <int D, int FMT>
__global__ void __launch_bounds__(kCacheThreads, kCacheCtasPerSm) cache_write_kernel(const CacheMoveParams p) {
  constexpr int C = D / 16;
  __shared__ int64_t rows[kCacheTokens];
  const int heads = p.c.heads;
  const int t0 = blockIdx.x * p.tokens;
  const int n = min(p.tokens, p.s.num_tokens - t0), units = n * heads * 2 * C;   // even
  place_tokens(p.c, p.s, t0, n, rows);
  __syncthreads();
  for (int u0 = threadIdx.x; u0 < ((units + 31) & ~31); u0 += kCacheThreads * kCacheUnroll) {
    CacheUnit un[kCacheUnroll];
    int64_t row[kCacheUnroll];
    uint4 a[kCacheUnroll], b[kCacheUnroll];
#pragma unroll
    for (int i = 0; i < kCacheUnroll; ++i) {
      const int u = u0 + i * kCacheThreads;
      un[i] = cache_unit<C>(min(u, units - 1), heads, n);
      row[i] = u < units ? rows[un[i].tk] : kRowNone;
      a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row[i] >= 0) {
        const uint4* src = reinterpret_cast<const uint4*>(
            (un[i].kv == 0 ? p.k_in + (t0 + un[i].tk) * p.k_token + un[i].h * p.k_head
                           : p.v_in + (t0 + un[i].tk) * p.v_token + un[i].h * p.v_head) + un[i].c * 16);
        a[i] = __ldcs(src);
        b[i] = __ldcs(src + 1);
      }
    }
#pragma unroll
    for (int i = 0; i < kCacheUnroll; ++i) {
      const int64_t at = row[i] + (static_cast<int64_t>(un[i].h) << p.c.page_shift);
      uint8_t* base = un[i].kv == 0 ? p.c.k : p.c.v;
      if (FMT == kCacheBf16) {
        if (row[i] >= 0) {
          uint4* dst = reinterpret_cast<uint4*>(base + at * (D * 2) + un[i].c * 32);
          dst[0] = a[i];
          dst[1] = b[i];
        }
      } else {
        uint32_t x[8] = {a[i].x, a[i].y, a[i].z, a[i].w, b[i].x, b[i].y, b[i].z, b[i].w};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = __vmaxu2(m, x[j] & 0x7fff7fffu);
        uint32_t most = max(m & 0xffffu, m >> 16);
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        const bool nan = most >= 0x7f80u;
        // magnitudes that would round to 2^128, past bf16, are held at the largest that does not
        constexpr uint32_t kMost = FMT == kCacheE4m3 ? 0x7f707f70u : 0x7f7e7f7eu;   // 240 * 2^120, 127 * 2^121
        if (!nan && most > (kMost & 0xffffu)) {
          most = kMost & 0xffffu;
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = __vminu2(x[j] & 0x7fff7fffu, kMost) | (x[j] & 0x80008000u);
        }
        const int e = nan ? 0 : scale_exponent<FMT>(most);
        const uint32_t f = pow2_bf16x2(-e);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t y0 = mul_bf16x2(x[2 * j], f), y1 = mul_bf16x2(x[2 * j + 1], f);
          w[j] = nan ? 0u : pack4<FMT>(y0, y1);
        }
        if (row[i] >= 0) {
          *reinterpret_cast<uint4*>(base + at * D + un[i].c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
          if ((un[i].c & 1) == 0) {
            uint8_t* sc = un[i].kv == 0 ? p.c.k_scale : p.c.v_scale;
            sc[at * (D / kCacheGroup) + (un[i].c >> 1)] = nan ? kCacheNanScale : static_cast<uint8_t>(e + 127);
          }
        }
      }
    }
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(kCacheThreads, kCacheCtasPerSm) cache_read_kernel(const CacheMoveParams p) {
  constexpr int C = D / 16;
  __shared__ int64_t rows[kCacheTokens];
  const int heads = p.c.heads;
  const int t0 = blockIdx.x * p.tokens;
  const int n = min(p.tokens, p.s.num_tokens - t0), units = n * heads * 2 * C;
  place_tokens(p.c, p.s, t0, n, rows);
  __syncthreads();
  for (int u0 = threadIdx.x; u0 < units; u0 += kCacheThreads * kCacheUnroll) {
    CacheUnit un[kCacheUnroll];
    int64_t row[kCacheUnroll];
    uint4 a[kCacheUnroll], b[kCacheUnroll];
    uint32_t byte[kCacheUnroll];
#pragma unroll
    for (int i = 0; i < kCacheUnroll; ++i) {
      const int u = u0 + i * kCacheThreads;
      un[i] = cache_unit<C>(min(u, units - 1), heads, n);
      row[i] = u < units ? rows[un[i].tk] : kRowNone;
      a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
      byte[i] = 127u;
      if (row[i] >= 0) {
        const int64_t at = row[i] + (static_cast<int64_t>(un[i].h) << p.c.page_shift);
        const uint8_t* base = un[i].kv == 0 ? p.c.k : p.c.v;
        if (FMT == kCacheBf16) {
          const uint4* src = reinterpret_cast<const uint4*>(base + at * (D * 2) + un[i].c * 32);
          a[i] = __ldcs(src);
          b[i] = __ldcs(src + 1);
        } else {
          const uint8_t* sc = un[i].kv == 0 ? p.c.k_scale : p.c.v_scale;
          a[i] = __ldcs(reinterpret_cast<const uint4*>(base + at * D + un[i].c * 16));
          byte[i] = sc[at * (D / kCacheGroup) + (un[i].c >> 1)];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kCacheUnroll; ++i) {
      if (row[i] == kRowNone) continue;
      if (FMT != kCacheBf16) {
        uint4 o0, o1;
        dequant16<FMT>(a[i], byte[i], o0, o1);
        a[i] = row[i] >= 0 ? o0 : make_uint4(0u, 0u, 0u, 0u);
        b[i] = row[i] >= 0 ? o1 : make_uint4(0u, 0u, 0u, 0u);
      }
      uint4* dst = reinterpret_cast<uint4*>(
          (un[i].kv == 0 ? p.k_out + (t0 + un[i].tk) * p.k_token + un[i].h * p.k_head
                         : p.v_out + (t0 + un[i].tk) * p.v_token + un[i].h * p.v_head) + un[i].c * 16);
      dst[0] = a[i];
      dst[1] = b[i];
    }
  }
}

}  // namespace dynrad
