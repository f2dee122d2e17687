// Attention of new tokens over the paged K / V cache, on the 5th-generation
// tensor cores.
//
// For query head h of token i (of the n that sequence s has in this call, at
// position x = kv_len - n + i) with K / V head h / G, G = heads / kv heads:
//   seen  = [lo, hi): all cached positions (frame = 0), or those of frames
//           floor(x / frame) - window + 1 .. floor(x / frame) (window = 0: 0 ..)
//   o     = sum_seen softmax(scale q.k) v,   lse = ln sum_seen exp(scale q.k)
// A row that sees nothing gives o = 0, lse = -inf.
//
// Rows.  The G query heads of a K / V head and 128 / G consecutive tokens make
// one 128-row tile (row = token * G + head), so every key read serves all of
// them.  An item is QT tiles of one (sequence, K / V head): QT = 2 for chunks,
// whose two tiles share each K / V tile; QT = 1 for few tokens, where the
// freed shared memory deepens the pipeline of loads.  In an item with rows for
// one tile only, that tile's keys are dealt out in turn to two accumulators
// ("narrow"), so that the softmax of one step runs under the products of the
// next; the two are joined in the epilogue.
//
// Schedule.  Keys go by in steps of 128.  With few items the steps of all of
// them are laid end to end and cut into equal runs, one for each CTA (split =
// true): a CTA then works on the end of one item, whole items, and the start of
// another.  What a CTA has of an item it does not hold whole (O unnormalised,
// max and sum, fp32) goes to the workspace, and cache_join_kernel joins the parts
// in order of their keys, so results repeat bit for bit.  Lengths are known on the device only,
// so each CTA finds its run by itself: a scan over the items at its start.
// With many items (split = false) a CTA takes one, from the last place on: of a
// sequence the items that see most come first, between sequences the order says nothing.
//
// Warp roles:
//   warps 0-3, 4-7  softmax of tile 0 / 1: thread = row = TMEM lane; as in the
//              block-sparse kernel: row max, then exponentials, 64 columns at a
//              time, lazy rescale of O (only when the max grows by 2^8), P as bf16
//              over the first half of S.
//   warp 8     producer: publishes the segments (an item or a part of it), loads
//              Q by TMA (a [D, heads, tokens] map: any strides) and each step's K
//              pages, one lane a page;
//   warp 10    the same for V's pages.
//   warp 9     MMA issuer: O_t += P_t V(j), then S_t = Q_t K(j+1)^T.
//   warps 12-19 (8-bit pages) turn what was loaded into bf16 operand tiles.
//              Scales are powers of two, so those tiles are exact and everything
//              behind them is the same for all formats.
//
// P is rounded to bf16: the product takes both operands in one type, and V is kept in
// bf16.  That is off by at most 2^-8 of sum p |v|, as in the block-sparse kernel; the sum
// of a row's weights takes them unrounded.
//
// What nobody sees.  A masked logit is replaced, not added to, so K may hold
// anything.  V meets P = 0 in the product, where NaN and infinity would not
// stay away: on steps that some row of the item does not see whole (`partial`),
// V rows that no row sees are zeroed in shared memory, and of those that some but not
// all rows see the channels that are not finite are zeroed too and noted (`poison`);
// the epilogue of a poisoned segment adds those back, in the rows that do see them,
// by plain loads.
//
// Every wait is bounded (common.cuh).
//
// Measured (cold caches / the same call again): 1560 tokens over 18720 keys of 12 heads,
// bf16, 234 / 220 us (768 / 814 TFLOP/s), e4m3 297 / 284, int8 287 / 275; over 32760 keys
// of 40 heads e4m3 1400 / 1392 us (747 / 752), int8 1389 / 1378; 1536 tokens over 132000
// keys of 12 heads, bf16, 1294 us (962).  A step of 128 keys of two tiles takes about 4300
// cycles (tensor pipe 43 % busy, exponentials 41 %), bound by the chain S -> softmax ->
// P V of each tile; e4m3 about 5500, its unpacking sharing issue slots and ALU with the
// softmax.
#pragma once

#include "attention.cuh"
#include "kvcache.cuh"
#include "tma2d.cuh"

namespace dynrad {

constexpr int kCacheMaxCtas = 148;      // CTAs of a split launch, one for each SM
// The even cut counts units: a step of a two-tile item kWideUnits, one of an item with
// rows for one tile only kNarrowUnits where the launch has both (and else 1).  A narrow
// step takes 0.57 of a wide one in bf16, 0.62 in 8 bits, 0.48 at D = 64; counted alike,
// 1560 tokens over 18720 keys took 234 us instead of 220.
constexpr int kWideUnits = 5, kNarrowUnits = 3;
// An item's start and end, in the launch's longest steps.  Tiles (1 / 2 / 3 / 4): 230 / 216 /
// 204 / 206 us for eight ragged sequences at D = 128, 184 / 175 / 177 / 182 at D = 64.
// Single tokens (1 / 2 / 3 / 5): 64 sequences of up to 4000 keys, 32 heads on 8, int8 94 /
// 88 / 84 / 84 us, e4m3 94 / 88 / 86 / 88, bf16 117 / 119 / 119 / 119; long caches within 2 %.
constexpr int kCacheItemCost = 3;
constexpr int kCacheLeastRun = 3;       // what a CTA takes at least, in those steps
constexpr int kSegRing = 4;

template <int D, int FMT, int QT>
struct CacheAttnCfg {
  static constexpr int kTileBytes = 128 * D * 2;      // one bf16 operand tile (Q, K or V)
  static constexpr int kChunkBytes = 128 * 128;       // 64 columns of it
  static constexpr int kChunks = D / 64;
  static constexpr int kRawCodes = 128 * D, kRawBytes = kRawCodes + 128 * (D / kCacheGroup);
  static constexpr int kCtrl = 2048;
  static constexpr int kBudget = 227 * 1024 - 1024 - kCtrl - QT * kTileBytes;   // 1024: manual alignment
  static constexpr bool kRaw = FMT != kCacheBf16;
  // 8-bit: three operand tiles (V(j), K(j+1), and the one being filled), the rest raw
  static constexpr int kSlots = kRaw ? (D == 64 || QT == 1 ? 4 : 3) : (kBudget / kTileBytes < 8 ? kBudget / kTileBytes : 8);
  static constexpr int kRawFit = kRaw ? (kBudget - kSlots * kTileBytes) / kRawBytes : 0;
  static constexpr int kRawSlots = kRawFit < 8 ? kRawFit : 8;
  static constexpr int kDqWarps = kRaw ? 8 : 0;
  static constexpr int kThreads = kRaw ? 640 : 352;
  // 8-bit: registers a thread after the split by warpgroup (two of softmax, one of
  // producer and MMA, two that dequantise); 640 threads start with 96
  static constexpr int kRegsSoftmax = 144, kRegsControl = 64, kRegsUnpack = 64;
  static_assert(256 * kRegsSoftmax + 128 * kRegsControl + 256 * kRegsUnpack <= 640 * 96, "registers at launch");
  static constexpr int kSmem = QT * kTileBytes + kSlots * kTileBytes + kRawSlots * kRawBytes + kCtrl + 1024;
  static constexpr int kRows = 128 * QT;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kSlots >= 3 && (!kRaw || kRawSlots >= 2), "pipeline depth");
};

struct CacheAttnParams {
  CacheDev c;
  SeqsDev s;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;                    // [heads, num_tokens]
  int64_t q_token, q_head, o_token, o_head;   // strides in elements
  int32_t group;                 // query heads of a K / V head
  int32_t tile_tokens;           // tokens of a 128-row tile: 128 / group
  int32_t frame, window;
  int32_t slots;                 // places for items of one K / V head (see find_item)
  int32_t split;
  float scale_log2;
  float* part_o;                 // [2 * CTAs][rows][D]
  float2* part_ml;               // [2 * CTAs][rows]
  int4* part_desc;               // [2 * CTAs]: first token, K / V head, kPart*, tokens
  uint64_t wait_ns;
  int32_t stall_step;            // as in AttnParams
};

constexpr int kPartNone = 0, kPartOpen = 1, kPartLast = 2;

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

// The tokens of one item, what they see, and the steps that takes.  Bounds grow
// with the token, so the first and last one's are the extremes.
struct CacheItem {
  int32_t seq, tok0, ntok;       // first row's token and how many
  int32_t pos0, len;             // its position, the sequence's length
  int32_t lo, hi;                // seen by some row
  int32_t lo_max, hi_min;        // seen by every row: [lo_max, hi_min)
  int32_t step0, steps;          // 128-key steps that cover [lo, hi)
};

// Place i of the slots: sequence s has the places cu_seq[s] / item_tokens + s ..,
// one for each item_tokens of its tokens, which never reach the next sequence's
// (some places stay empty: ntok = 0).
__device__ __forceinline__ CacheItem find_item(const CacheAttnParams& p, int item_tokens, int place) {
  int a = 0, b = p.s.num_seqs;
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (static_cast<int64_t>(max(p.s.cu_seq[mid], 0) / item_tokens) + mid <= place) a = mid; else b = mid;
  }
  const SeqSpan sp = seq_span(p.s, a, p.c.page_shift);
  CacheItem it;
  it.seq = a;
  const int64_t first = sp.begin +
      (place - a - static_cast<int64_t>(max(p.s.cu_seq[a], 0) / item_tokens)) * static_cast<int64_t>(item_tokens);
  it.tok0 = static_cast<int32_t>(min(max(first, static_cast<int64_t>(sp.begin)), static_cast<int64_t>(sp.end)));
  it.ntok = first < sp.begin ? 0 : min(item_tokens, sp.end - it.tok0);
  it.len = sp.len;
  it.pos0 = sp.len - (sp.end - it.tok0);
  it.lo = it.hi = it.lo_max = it.hi_min = it.step0 = it.steps = 0;
  if (it.ntok > 0) {
    seen_range(p.frame, p.window, it.pos0, it.len, it.lo, it.hi_min);
    seen_range(p.frame, p.window, it.pos0 + it.ntok - 1, it.len, it.lo_max, it.hi);
    if (it.hi > it.lo) {
      it.step0 = it.lo >> 7;
      it.steps = ((it.hi + 127) >> 7) - it.step0;
    }
  }
  return it;
}

// A segment: steps [sa, sb) of an item (counted from its step0).
struct CacheSeg {
  CacheItem it;
  int32_t head, sa, sb;
  int32_t part;                  // -1: the whole item; else the CTA's workspace slot
  int32_t end;                   // 1: no more segments
  int32_t narrow;
  int32_t act_a[2], act_b[2];    // steps in which tile t sees something
};

__device__ __forceinline__ bool seg_active(const CacheSeg& s, int t, int j) {
  return s.narrow ? ((j - s.sa) & 1) == t : j >= s.act_a[t] && j < s.act_b[t];
}

// Some row of the item does not see all of step j.
__device__ __forceinline__ bool seg_partial(const CacheSeg& s, int j) {
  const int32_t key0 = (s.it.step0 + j) << 7;
  return key0 < s.it.lo_max || key0 > s.it.hi_min - 128;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Two bf16 numbers with 0 in the place of what is not finite.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t x) {
  return ((x & 0x7f80u) == 0x7f80u ? 0u : x & 0xffffu) | ((x & 0x7f800000u) == 0x7f800000u ? 0u : x & 0xffff0000u);
}

// Weight of what was summed under the maximum m (log2 units) where the largest of all
// is `most`; 1 where nobody met a logit over -inf.  It may underflow to 0, and such a
// share is added like any other: where it is finite that adds nothing, and its NaN or
// infinity (of a key or V that the row sees) comes through as it does when the same keys
// are summed in one.
__device__ __forceinline__ float join_weight(float m, float most) {
  return most == -INFINITY ? 1.f : ex2_approx(m - most);
}

// Units of the launch's longest steps, and of an item's.
__device__ __forceinline__ int32_t longest_step(const CacheAttnParams& p, int item_tokens) {
  return item_tokens > p.tile_tokens ? kWideUnits : 1;
}
__device__ __forceinline__ int32_t step_units(const CacheAttnParams& p, int item_tokens, const CacheItem& it) {
  return item_tokens <= p.tile_tokens ? 1 : it.ntok > p.tile_tokens ? kWideUnits : kNarrowUnits;
}

// Units (steps and the fixed cost) of an item.
__device__ __forceinline__ int32_t item_units(const CacheAttnParams& p, int item_tokens, const CacheItem& it) {
  return it.ntok > 0 ? it.steps * step_units(p, item_tokens, it) + kCacheItemCost * longest_step(p, item_tokens) : 0;
}

// The item's step that unit u falls into (its fixed cost comes first).
__device__ __forceinline__ int32_t unit_step(const CacheAttnParams& p, int item_tokens, const CacheItem& it, int64_t u) {
  const int32_t at = static_cast<int32_t>(u) - kCacheItemCost * longest_step(p, item_tokens);
  return max(at, 0) / step_units(p, item_tokens, it);
}

// Where a CTA's run of a split launch starts.
struct CacheRun {
  int64_t left;                  // units of the run
  int64_t off;                   // units of the first item that other CTAs have
  int32_t head, place;
};

// Finds the CTA's run: units of all places, their sum, and the cut.  scratch:
// p.slots int32; every thread of the CTA takes part.
template <int THREADS>
__device__ __forceinline__ void plan_run(const CacheAttnParams& p, int item_tokens, int32_t* scratch, int64_t* sums,
                                         CacheRun* run) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < p.slots; i += THREADS) scratch[i] = item_units(p, item_tokens, find_item(p, item_tokens, i));
  if (tid == 0) run->left = 0;
  __syncthreads();
  const int per = (p.slots + THREADS - 1) / THREADS;
  const int i0 = min(tid * per, p.slots), i1 = min(i0 + per, p.slots);
  int64_t mine = 0;
  for (int i = i0; i < i1; ++i) mine += scratch[i];
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int64_t v = sums[w];
    if (w < warp) before += v;
    total += v;
  }
  const int64_t all = total * p.c.heads;
  const int64_t n = gridDim.x, c = blockIdx.x;
  const int64_t least = kCacheLeastRun * longest_step(p, item_tokens);
  int64_t a, b;
  if (all < n * least) {
    a = min(all, c * least);
    b = min(all, a + least);
  } else {
    a = c * all / n;
    b = (c + 1) * all / n;
  }
  if (b > a) {
    const int64_t head = a / total, w = a - head * total;
    if (w >= before && w < before + mine) {
      int64_t at = before;
      int i = i0;
      while (at + scratch[i] <= w) at += scratch[i++];
      run->left = b - a;
      run->off = w - at;
      run->head = static_cast<int32_t>(head);
      run->place = i;
    }
  }
  fence_async_shared();   // the scratch is loaded over next
  __syncthreads();
}

template <int D, int FMT, int QT>
__global__ void __launch_bounds__(CacheAttnCfg<D, FMT, QT>::kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const CacheAttnParams p) {
  using C = CacheAttnCfg<D, FMT, QT>;
  constexpr int NS = C::kSlots, NR = C::kRaw ? C::kRawSlots : 1;
  constexpr int TB = C::kTileBytes;
  extern __shared__ uint8_t cache_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(cache_smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* q_smem = smem;
  uint8_t* slot_smem = smem + QT * TB;             // load i (K: even, V: odd) as an operand tile in slot i % NS
  uint8_t* raw_smem = slot_smem + NS * TB;         // load i as stored in slot i % NR
  uint8_t* ctrl = raw_smem + C::kRawSlots * C::kRawBytes;
  uint64_t* bar = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* q_full = bar;
  uint64_t* q_empty = bar + 1;
  uint64_t* slot_full = bar + 2;                   // [8]
  uint64_t* slot_empty = bar + 10;                 // [8]
  uint64_t* raw_full = bar + 18;                   // [8]
  uint64_t* raw_empty = bar + 26;                  // [8]
  uint64_t* s_full = bar + 34;                     // [tile]
  uint64_t* p_full = bar + 36;                     // [tile]
  uint64_t* seg_full = bar + 38;                   // [kSegRing]
  uint64_t* seg_empty = bar + 42;
  uint64_t* ml_full = bar + 46;                    // narrow: tile 1's max and sum are in ml
  uint64_t* ml_done = bar + 47;                    // narrow: tile 1's accumulator has been read
  uint64_t* drain = bar + 48;
  uint64_t* stall = bar + 49;                      // never completed (failure-path tests)
  uint64_t* o_full = bar + 50;                     // [tile]: the segment's last product is in O
  float2* ml = reinterpret_cast<float2*>(bar + 52);                  // [128]
  CacheSeg* segs = reinterpret_cast<CacheSeg*>(ml + 128);            // [kSegRing]
  volatile int* poison = reinterpret_cast<volatile int*>(segs + kSegRing);   // [kSegRing]
  uint32_t* tmem_base_s = const_cast<uint32_t*>(reinterpret_cast<volatile uint32_t*>(poison + kSegRing));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_s + 1);
  CacheRun* run = reinterpret_cast<CacheRun*>(tmem_base_s + 2);
  static_assert(52 * 8 + 128 * 8 + kSegRing * sizeof(CacheSeg) + kSegRing * 4 + 8 + sizeof(CacheRun) <= C::kCtrl,
                "control block");
  static_assert(kSegRing * sizeof(CacheSeg) % 8 == 0 && kSegRing % 2 == 0, "alignment of the control block");

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint64_t wlim = p.wait_ns;
  const int item_tokens = QT * p.tile_tokens;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < 8; ++s) {
      mbar_init(&slot_full[s], C::kRaw ? C::kDqWarps : 1);
      mbar_init(&slot_empty[s], 1);
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], C::kRaw ? C::kDqWarps : 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&o_full[t], 1);
      mbar_init(&p_full[t], 4);
    }
    for (int g = 0; g < kSegRing; ++g) {
      mbar_init(&seg_full[g], 1);
      mbar_init(&seg_empty[g], 10 + C::kDqWarps);   // softmax, MMA, V's producer and dequantising warps
      poison[g] = 0;
    }
    mbar_init(ml_full, 4);
    mbar_init(ml_done, 4);
    mbar_init(drain, 1);
    mbar_init(stall, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_base_s, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = *tmem_base_s;
  if (p.split) plan_run<C::kThreads>(p, item_tokens, reinterpret_cast<int32_t*>(slot_smem),
                                     reinterpret_cast<int64_t*>(ml), run);

  // waits for segment g of the CTA and gives it back when a warp is through with it
  auto seg_wait = [&](int g) -> bool { return mbar_wait(&seg_full[g % kSegRing], (g / kSegRing) & 1, abort_flag, wlim); };

  // The K (kv = 0) or V tiles of the sequence's steps [step_a, step_b), as loads li, li + 2, ..; lane b has page b
  // of a step.  A producer's pages go out one lane after the other (some 60 clocks a
  // copy), so K and V have a warp each.
  const int ps = p.c.page_shift, page = 1 << ps, npg = 128 >> ps;
  auto load_tiles = [&](int kv, int seq, int head, int step_a, int step_b, int32_t lo, int32_t hi, int& li) -> bool {
    const int32_t* row = p.s.page_table + static_cast<int64_t>(seq) * p.s.table_stride;
    // page of lane's positions of step j: -1 not needed, -2 outside the pool
    auto page_of = [&](int j) -> int32_t {
      const int64_t key = (static_cast<int64_t>(j) << 7) + (lane << ps);
      if (lane >= npg || key >= hi || key + page <= lo) return -1;
      const int32_t pg = row[key >> ps];
      if (pg >= 0 && pg < p.c.num_pages) return pg;
      record_error(DYNRAD_ERR_DEVICE);
      return -2;
    };
    int32_t pg = step_a < step_b ? page_of(step_a) : -1;
    for (int j = step_a; j < step_b; ++j, li += 2) {
      const int32_t next = j + 1 < step_b ? page_of(j + 1) : -1;
      const int pages = __popc(__ballot_sync(0xffffffffu, C::kRaw ? pg >= 0 : pg != -1));
      const int64_t tile = (static_cast<int64_t>(pg) * p.c.heads + head) << ps;   // first row of the page's head
      constexpr int n = C::kRaw ? NR : NS;
      const int sl = li % n;
      uint64_t* full = C::kRaw ? &raw_full[sl] : &slot_full[sl];
      uint64_t* empty = C::kRaw ? &raw_empty[sl] : &slot_empty[sl];
      bool w = true;
      if (li >= n && lane == 0) w = mbar_wait(empty, ((li / n) - 1) & 1, abort_flag, wlim);
      if (!__shfl_sync(0xffffffffu, w, 0)) return false;
      if constexpr (C::kRaw) {
        uint8_t* dst = raw_smem + sl * C::kRawBytes;
        if (pg == -2) {   // reads as zeros
          for (int i = 0; i < page * D / 16; ++i)
            reinterpret_cast<uint4*>(dst + (lane << ps) * D)[i] = make_uint4(0u, 0u, 0u, 0u);
          for (int i = 0; i < page * (D / kCacheGroup); ++i)
            dst[C::kRawCodes + (lane << ps) * (D / kCacheGroup) + i] = 127;
          fence_async_shared();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full, pages * page * (D + D / kCacheGroup));
        __syncwarp();
        if (pg >= 0) {
          const uint8_t* codes = kv == 0 ? p.c.k : p.c.v;
          const uint8_t* scales = kv == 0 ? p.c.k_scale : p.c.v_scale;
          bulk_load(dst + (lane << ps) * D, codes + tile * D, page * D, full);
          bulk_load(dst + C::kRawCodes + (lane << ps) * (D / kCacheGroup), scales + tile * (D / kCacheGroup),
                    page * (D / kCacheGroup), full);
        }
      } else {
        uint8_t* dst = slot_smem + sl * TB;
        if (lane == 0) mbar_arrive_expect_tx(full, pages * page * D * 2);
        __syncwarp();
        if (pg != -1) {
          // a row past the tensor (a page outside the pool) is filled with zeros
          const int32_t r = static_cast<int32_t>(pg >= 0 ? tile : (p.c.num_pages * p.c.heads) << ps);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_2d(dst + c * C::kChunkBytes + (lane << ps) * 128, kv == 0 ? &tm_k : &tm_v, full, c * 64, r);
        }
      }
      __syncwarp();
      pg = next;
    }
    return true;
  };
  // unwinding: lets the copies of loads li - 2, li - 4, .. land before shared memory is
  // given back
  auto drain_loads = [&](int li) {
    constexpr int n = C::kRaw ? NR : NS;
    if (lane == 0)
      for (int i = li - 2; i >= 0 && i > li - 2 - n; i -= 2)
        mbar_wait(C::kRaw ? &raw_full[i % n] : &slot_full[i % n], (i / n) & 1, nullptr);
  };

  if (warp < 8) {
    if constexpr (C::kRaw) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    // -------------------------------------------------------------- softmax
    // Both 64-column halves unrolled for bf16 pages; looped over beside the
    // dequantising warps, whose code shares the instruction cache (one 480p frame of
    // 40 heads over 32,760 keys: e4m3 1.46 -> 1.43 ms looped, bf16 1.26 -> 1.32).
    constexpr int kHalves = C::kRaw ? 1 : 2;
    const int tile = warp >> 2;
    const int t = threadIdx.x - tile * 128;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t col_s = 256u + 128u * tile, col_o = 128u * tile;
    const float c2 = p.scale_log2;
    const int rtok = t / p.group, rhead = t - rtok * p.group;
    int ns = 0, no = 0, nml = 0, li = 0;      // s_full and o_full phases, narrow joins, K / V tiles
    bool ok = true;
    for (int g = 0; ok; ++g) {
      if (!__all_sync(0xffffffffu, seg_wait(g))) break;
      const CacheSeg& sg = segs[g % kSegRing];
      if (sg.end) break;
      // this thread's row: in a narrow segment both warpgroups have the same rows
      const int tok = rtok + (sg.narrow ? 0 : tile * p.tile_tokens);
      const bool valid = rtok < p.tile_tokens && tok < sg.it.ntok;
      int32_t lo = 0, hi = INT32_MAX;    // rows that are not there count as seeing all: nothing to mask
      if (valid) seen_range(p.frame, p.window, sg.it.pos0 + tok, sg.it.len, lo, hi);
      const bool warp_rows = __any_sync(0xffffffffu, valid);
      const int sa = sg.sa, sb = sg.sb, step0 = sg.it.step0;
      float m_used = -INFINITY, l = 0.f;
      for (int j = sa; j < sb; ++j, li += 2) {
        const int32_t key0 = (step0 + j) << 7;
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[tile], ns & 1, abort_flag, wlim))) { ok = false; break; }
        ++ns;
        tc_fence_after();
        if (!C::kRaw && tile == 0 && seg_partial(sg, j)) {
          if (!__all_sync(0xffffffffu,
                          mbar_wait(&slot_full[(li + 1) % NS], ((li + 1) / NS) & 1, abort_flag, wlim))) {
            ok = false;
            break;
          }
          // eight lanes a row: V rows that nobody sees, and of those that some rows see
          // what is not finite
          bool bad = false;
#pragma unroll 1
          for (int r = warp * 32 + (lane >> 3); r < warp * 32 + 32; r += 4) {
            const int32_t key = key0 + r;
            if (key >= sg.it.lo_max && key < sg.it.hi_min) continue;     // seen by all
            const bool seen = key >= sg.it.lo && key < sg.it.hi;
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
              uint4* at = reinterpret_cast<uint4*>(slot_smem + ((li + 1) % NS) * TB + c * C::kChunkBytes + r * 128 +
                                                   (lane & 7) * 16);
              uint4 y = make_uint4(0u, 0u, 0u, 0u);
              if (seen) {
                const uint4 x = *at;
                y = make_uint4(finite_bf16x2(x.x), finite_bf16x2(x.y), finite_bf16x2(x.z), finite_bf16x2(x.w));
                if (x.x == y.x && x.y == y.y && x.z == y.z && x.w == y.w) continue;
                bad = true;
              }
              *at = y;
            }
          }
          if (bad) poison[g % kSegRing] = g + 1;
          fence_async_shared();
        }
        if (warp_rows && seg_active(sg, tile, j)) {
          const int32_t rl = max(lo - key0, 0), rh = min(hi - key0, 128);   // columns [rl, rh) count
          // of each 64-column half: all lanes see all of it, or none any
          uint32_t half_full = 0, half_none = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (__all_sync(0xffffffffu, rl <= 64 * h && rh >= 64 * h + 64)) half_full |= 1u << h;
            if (__all_sync(0xffffffffu, rl >= 64 * h + 64 || rh <= 64 * h)) half_none |= 1u << h;
          }
          float mx = -INFINITY;
#pragma unroll kHalves
          for (int h = 0; h < 2; ++h) {
            if ((half_none >> h) & 1u) continue;
            float m4[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
            if ((half_full >> h) & 1u) {
              float sv[64];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t r[32];
                tmem_ld32(taddr + lane_base + col_s + h * 64 + c * 32, r);
#pragma unroll
                for (int i = 0; i < 32; ++i) sv[c * 32 + i] = __uint_as_float(r[i]);
              }
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 64; i += 8) {
#pragma unroll
                for (int u = 0; u < 4; ++u) m4[u] = fmax3(m4[u], sv[i + 2 * u], sv[i + 2 * u + 1]);
              }
            } else {
              // columns that do not count become -inf, in tensor memory too: the second
              // pass takes all it reads
#pragma unroll kHalves
              for (int c = h * 64; c < h * 64 + 64; c += 32) {
                uint32_t r[32];
                tmem_ld32(taddr + lane_base + col_s + c, r);
                tmem_wait_ld();
                const int from = rl - c, to = rh - c;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  if (i < from || i >= to) r[i] = 0xff800000u;
                  m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(r[i]));
                }
                tmem_st32(taddr + lane_base + col_s + c, r);
              }
              tmem_wait_st();
            }
            mx = fmax3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
          }
          const float m_new = fmaxf(m_used, mx * c2);
          const bool need = valid && m_used != -INFINITY && m_new > m_used + 8.0f;
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = need ? ex2_approx(m_used - m_new) : 1.0f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t r[32];
              tmem_ld32(taddr + lane_base + col_o + c * 32, r);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
              tmem_st32(taddr + lane_base + col_o + c * 32, r);
            }
            if (need) {
              l *= alpha;
              m_used = m_new;
            }
          }
          if (m_used == -INFINITY) m_used = m_new;
          // a row whose logits so far are all -inf keeps 0 as its reference: every P is 0
          const float ref = m_used == -INFINITY ? 0.f : m_used;
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 cc = make_float2(c2, c2), mm = make_float2(-ref, -ref);
#pragma unroll kHalves
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
            if ((half_none >> h) & 1u) {
#pragma unroll
              for (int i = 0; i < 32; ++i) pk[i] = 0u;
            } else {
              float sv[64];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t r[32];
                tmem_ld32(taddr + lane_base + col_s + h * 64 + c * 32, r);
#pragma unroll
                for (int i = 0; i < 32; ++i) sv[c * 32 + i] = __uint_as_float(r[i]);
              }
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float2 x = __ffma2_rn(make_float2(sv[2 * i], sv[2 * i + 1]), cc, mm);
                const float2 pe = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                acc[i & 3] = __fadd2_rn(acc[i & 3], pe);
                pk[i] = pack_bf16x2(pe.x, pe.y);
              }
            }
            tmem_st32(taddr + lane_base + col_s + h * 32, pk);
          }
          const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
          l += a.x + a.y;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[tile]);
      }
      if (!ok) break;
      // the last product into this tile's O
      bool have = false, have1 = false;
      if (sb > sa) {
        if (!__all_sync(0xffffffffu, mbar_wait(&o_full[tile], no & 1, abort_flag, wlim))) { ok = false; break; }
        ++no;
        tc_fence_after();
        have = sg.narrow ? sb - sa > tile : max(sa, sg.act_a[tile]) < min(sb, sg.act_b[tile]);
      }
      float w0 = 1.f, w1 = 0.f;
      if (sg.narrow && sb > sa) {
        if (tile == 1) {
          ml[t] = make_float2(m_used, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ml_full);
          if (!__all_sync(0xffffffffu, mbar_wait(ml_done, nml & 1, abort_flag, wlim))) { ok = false; break; }
        } else {
          if (!__all_sync(0xffffffffu, mbar_wait(ml_full, nml & 1, abort_flag, wlim))) { ok = false; break; }
          tc_fence_after();
          if (sb - sa > 1) {
            have1 = true;
            const float2 b = ml[t];
            const float m = fmaxf(m_used, b.x);
            w0 = join_weight(m_used, m);
            w1 = join_weight(b.x, m);
            l = l * w0 + b.y * w1;
            m_used = m;
          }
        }
        ++nml;
      }
      if (warp_rows && !(sg.narrow && tile == 1)) {
        const bool poisoned = poison[g % kSegRing] == g + 1;
        const bool part = sg.part >= 0;
        const float inv = part ? 1.f : (l == 0.f ? 0.f : 1.f / l);
        const int64_t token = sg.it.tok0 + tok;
        const int qhead = sg.head * p.group + rhead;
        __nv_bfloat16* orow = p.o + token * p.o_token + qhead * p.o_head;
        const int64_t prow = part ? (2 * static_cast<int64_t>(blockIdx.x) + sg.part) * C::kRows +
                                        (sg.narrow ? 0 : tile * 128) + t
                                  : 0;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float x[32];
          {
            uint32_t r[32];
            if (have) {
              tmem_ld32(taddr + lane_base + col_o + c * 32, r);
              tmem_wait_ld();
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = have ? __uint_as_float(r[i]) * w0 : 0.f;
            if (have1) {
              tmem_ld32(taddr + lane_base + 128u + c * 32, r);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = fmaf(__uint_as_float(r[i]), w1, x[i]);
            }
          }
          if (poisoned && valid) {
            for (int j = sa; j < sb; ++j) {
              if (!seg_partial(sg, j)) continue;
              const int32_t key0 = (step0 + j) << 7;
              for (int32_t key = max(lo, key0); key < min(hi, key0 + 128); ++key) {
                if (key >= sg.it.lo_max && key < sg.it.hi_min) continue;
                const int64_t at = cache_row(p.c, p.s, sg.it.seq, key);
                if (at < 0) continue;
                const int64_t row = at + (static_cast<int64_t>(sg.head) << p.c.page_shift);
                if (C::kRaw) {
                  if (p.c.v_scale[row * (D / kCacheGroup) + c] == kCacheNanScale) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = __int_as_float(0x7fffffff);
                  }
                } else {
                  const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.c.v) + row * D;
#pragma unroll
                  for (int i = 0; i < 32; ++i) {
                    const float f = __bfloat162float(v[c * 32 + i]);
                    if (!isfinite(f)) x[i] += f;
                  }
                }
              }
            }
          }
          if (valid) {
            if (part) {
              float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + c * 32);
#pragma unroll
              for (int i = 0; i < 8; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dst[i] = make_uint4(pack_bf16x2(x[8 * i] * inv, x[8 * i + 1] * inv),
                                    pack_bf16x2(x[8 * i + 2] * inv, x[8 * i + 3] * inv),
                                    pack_bf16x2(x[8 * i + 4] * inv, x[8 * i + 5] * inv),
                                    pack_bf16x2(x[8 * i + 6] * inv, x[8 * i + 7] * inv));
            }
          }
        }
        if (valid) {
          if (part)
            p.part_ml[prow] = make_float2(m_used, l);
          else
            p.lse[static_cast<int64_t>(qhead) * p.s.num_tokens + token] =
                l == 0.f ? -INFINITY : m_used * 0.69314718055994531f + __logf(l);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (sg.narrow && sb > sa && tile == 0) mbar_arrive(ml_done);
        mbar_arrive(&seg_empty[g % kSegRing]);
      }
    }
  } else if (warp < 12) {   // 11 only fills up the warpgroup
    if constexpr (C::kRaw) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsControl));
  if (warp == 8) {
    // ------------------------------------------------------------- producer
    int head = 0, place = 0;
    int64_t off = 0, left = 0;
    if (p.split) {
      left = run->left;
      if (left > 0) {
        off = run->off;
        head = run->head;
        place = run->place;
      }
      if (lane == 0)
        p.part_desc[2 * blockIdx.x] = p.part_desc[2 * blockIdx.x + 1] = make_int4(0, 0, kPartNone, 0);
    } else {
      head = blockIdx.y;
      place = p.slots - 1 - static_cast<int>(blockIdx.x);   // a sequence's later tokens see more: they first
      left = 1;
    }
    if (lane == 0) {
      prefetch_tensormap(&tm_q);
      if (!C::kRaw) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
      }
    }
    bool ok = true;
    int g = 0, nq = 0, li = 0;   // segments, Q loads, K tile loads (even numbers)
    auto publish = [&](const CacheSeg& sg) -> bool {
      bool w = true;
      if (g >= kSegRing && lane == 0)
        w = mbar_wait(&seg_empty[g % kSegRing], ((g / kSegRing) - 1) & 1, abort_flag, wlim);
      if (!__shfl_sync(0xffffffffu, w, 0)) return false;
      if (lane == 0) {
        segs[g % kSegRing] = sg;
        mbar_arrive(&seg_full[g % kSegRing]);
      }
      __syncwarp();
      ++g;
      return true;
    };
    CacheSeg sg;
    sg.end = 0;
    while (ok && left > 0) {
      sg.it = find_item(p, item_tokens, place);
      sg.head = head;
      const int32_t units = item_units(p, item_tokens, sg.it);
      sg.sa = 0;
      sg.sb = sg.it.steps;
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
      if (units > 0 && (sg.sb > sg.sa || sg.it.steps == 0)) {
        const bool whole = sg.sa == 0 && sg.sb == sg.it.steps;
        sg.part = whole ? -1 : (sg.sa > 0 ? 0 : 1);
        if (!whole && lane == 0)
          p.part_desc[2 * blockIdx.x + sg.part] =
              make_int4(sg.it.tok0, head, sg.sb == sg.it.steps ? kPartLast : kPartOpen, sg.it.ntok);
        sg.narrow = QT == 1 || sg.it.ntok <= p.tile_tokens;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          sg.act_a[t] = sg.act_b[t] = 0;
          const int i0 = t * p.tile_tokens, i1 = min(sg.it.ntok, (t + 1) * p.tile_tokens) - 1;
          if (i0 <= i1) {
            int32_t lo, hi, x;
            seen_range(p.frame, p.window, sg.it.pos0 + i0, sg.it.len, lo, x);
            seen_range(p.frame, p.window, sg.it.pos0 + i1, sg.it.len, x, hi);
            if (hi > lo) {
              sg.act_a[t] = (lo >> 7) - sg.it.step0;
              sg.act_b[t] = ((hi + 127) >> 7) - sg.it.step0;
            }
          }
        }
        if (!publish(sg)) { ok = false; break; }
        if (sg.sb > sg.sa) {
          // Q
          bool w = true;
          if (nq > 0 && lane == 0) w = mbar_wait(q_empty, (nq - 1) & 1, abort_flag, wlim);
          if (!__shfl_sync(0xffffffffu, w, 0)) { ok = false; break; }
          if (lane == 0) {
            const int rows = p.tile_tokens * p.group;
            const int tiles = sg.narrow ? 1 : QT;
            mbar_arrive_expect_tx(q_full, tiles * C::kChunks * rows * 128);
            for (int t = 0; t < tiles; ++t)
#pragma unroll
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_3d(q_smem + t * TB + c * C::kChunkBytes, &tm_q, q_full, c * 64, head * p.group,
                            sg.it.tok0 + t * p.tile_tokens);
          }
          ++nq;
          ok = load_tiles(0, sg.it.seq, head, sg.it.step0 + sg.sa, sg.it.step0 + sg.sb, sg.it.lo, sg.it.hi, li);
        }
      }
      ++place;
      if (place == p.slots) {
        place = 0;
        if (++head == p.c.heads) break;
      }
    }
    if (ok) {
      sg.end = 1;
      ok = publish(sg);
    }
    if (!ok) {
      if (nq > 0 && lane == 0) mbar_wait(q_full, (nq - 1) & 1, nullptr);
      drain_loads(li);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------------ MMA
    // The whole warp runs the loop and one lane issues: what the products' operands
    // are made from stays the same in all lanes, so it lives in uniform registers
    // and an issue costs little beside the product itself.
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, false, true);
    const uint64_t qdesc0 = smem_desc_sw128(smem_u32(q_smem), 16, 1024);
    const uint64_t kdesc0 = smem_desc_sw128(smem_u32(slot_smem), 16, 1024);
    const uint64_t vdesc0 = smem_desc_sw128(smem_u32(slot_smem), C::kChunkBytes, 1024);
    auto desc_add = [](uint64_t d, uint32_t bytes) -> uint64_t { return d + (bytes >> 4); };
    auto uniform = [](int x) -> int { return __shfl_sync(0xffffffffu, x, 0); };
    const bool leader = elect_one();
    bool ok = true;
    int nq = 0, li = 0, np = 0, nsteps = 0;
    auto wait = [&](uint64_t* b, int phase) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(b, phase & 1, abort_flag, wlim));
    };
    auto full = [&](int i) -> bool { return wait(&slot_full[i % NS], i / NS); };
    auto commit = [&](uint64_t* b) {
      if (leader) mma_commit(b);
    };
    // S_t = Q_t K^T (a narrow segment's tiles share Q_0); O_t += P_t V, or = for the
    // tile's first product of a segment
    auto issue_qk = [&](uint32_t d, uint64_t ad, int i) {
      const uint64_t bd = desc_add(kdesc0, (i % NS) * TB);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int c = kk >> 2, off = (kk & 3) * 32;
          mma_ss(d, desc_add(ad, c * C::kChunkBytes + off), desc_add(bd, c * C::kChunkBytes + off), idesc_qk,
                 kk > 0 ? 1u : 0u);
        }
      }
    };
    auto issue_pv = [&](uint32_t d, uint32_t a, int i, uint32_t acc0) {
      const uint64_t bd = desc_add(vdesc0, (i % NS) * TB);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mma_ts(d, a + kk * 8, desc_add(bd, kk * 2048), idesc_pv, kk > 0 ? 1u : acc0);
      }
    };
    const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(taddr)));
    const uint32_t s0 = tm + 256u, s1 = tm + 384u, o0 = tm, o1 = tm + 128u;
    for (int g = 0; ok; ++g) {
      if (!wait(&seg_full[g % kSegRing], g / kSegRing)) break;
      const CacheSeg& sr = segs[g % kSegRing];
      const int n = uniform(sr.sb - sr.sa);
      const bool end = uniform(sr.end), narrow = uniform(sr.narrow);
      // steps, counted from the segment's first, in which the tiles see something
      const int a0 = uniform(sr.act_a[0] - sr.sa), b0 = uniform(sr.act_b[0] - sr.sa);
      const int a1 = uniform(sr.act_a[1] - sr.sa), b1 = uniform(sr.act_b[1] - sr.sa);
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[g % kSegRing]);
      if (end) break;
      if (n <= 0) continue;
      if (!wait(q_full, nq) || !full(li)) break;
      ++nq;
      tc_fence_after();
      const uint64_t q0 = qdesc0, q1 = desc_add(qdesc0, TB);
      uint32_t acc0 = 0u, acc1 = 0u;
      if (narrow || (a0 <= 0 && b0 > 0)) issue_qk(s0, q0, li);
      commit(&s_full[0]);
      if (!narrow && a1 <= 0 && b1 > 0) issue_qk(s1, q1, li);
      commit(&s_full[1]);
      commit(&slot_empty[li % NS]);
      if (n == 1) commit(q_empty);
      // At a segment's last step the next one's first S may follow before the softmax
      // has seen this one's last product, so that one has a barrier of its own.
      for (int j = 0; ok && j < n; ++j, ++np, li += 2) {
        const int iv = li + 1, ik = li + 2;
        const bool more = j + 1 < n;
        ok = false;
        if (nsteps++ == p.stall_step && !wait(stall, 0)) break;
        if (more && !full(ik)) break;
        if (!narrow) {
          // both tiles' waits but the softmax's come first: each tile's products go
          // out back to back
          const bool v0 = j >= a0 && j < b0, v1 = j >= a1 && j < b1;
          const bool k0 = more && j + 1 >= a0 && j + 1 < b0, k1 = more && j + 1 >= a1 && j + 1 < b1;
          if (!full(iv) || !wait(&p_full[0], np)) break;
          tc_fence_after();
          if (v0) issue_pv(o0, s0, iv, acc0), acc0 = 1u;
          if (k0) issue_qk(s0, q0, ik);
          commit(more ? &s_full[0] : &o_full[0]);
          if (!wait(&p_full[1], np)) break;
          tc_fence_after();
          if (v1) issue_pv(o1, s1, iv, acc1), acc1 = 1u;
          if (k1) issue_qk(s1, q1, ik);
          commit(&slot_empty[iv % NS]);
          if (more) commit(&slot_empty[ik % NS]);
          if (j + 2 == n) commit(q_empty);
          commit(more ? &s_full[1] : &o_full[1]);
        } else {
          // the idle tile's next S first: it does not wait for this step's softmax
          const int t = j & 1;
          const uint32_t s_t = t ? s1 : s0, s_i = t ? s0 : s1;
          if (!wait(&p_full[t ^ 1], np)) break;
          tc_fence_after();
          if (more) {
            issue_qk(s_i, q0, ik);
            commit(&slot_empty[ik % NS]);
            if (j + 2 == n) commit(q_empty);
          }
          commit(more ? &s_full[t ^ 1] : &o_full[t ^ 1]);
          if (!full(iv) || !wait(&p_full[t], np)) break;
          tc_fence_after();
          issue_pv(t ? o1 : o0, s_t, iv, j > 1 ? 1u : 0u);
          commit(&slot_empty[iv % NS]);
          commit(more ? &s_full[t] : &o_full[t]);
        }
        ok = true;
      }
    }
    // all issued tensor-core work finished before tensor memory is released
    commit(drain);
    mbar_wait(drain, 0, nullptr);
    __syncwarp();
  } else if (warp == 10) {
    // ----------------------------------------------------------- V's producer
    int li = 1;
    bool ok = true;
    for (int g = 0; ok; ++g) {
      if (!__all_sync(0xffffffffu, seg_wait(g))) { ok = false; break; }
      const CacheSeg& sr = segs[g % kSegRing];
      const int seq = sr.it.seq, head = sr.head, a = sr.it.step0 + sr.sa, b = sr.it.step0 + sr.sb;
      const int32_t lo = sr.it.lo, hi = sr.it.hi;
      const bool end = sr.end;
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[g % kSegRing]);
      if (end) break;
      ok = load_tiles(1, seq, head, a, b, lo, hi, li);
    }
    if (!ok) drain_loads(li);
    __syncwarp();
  }
  } else {
    // -------------------------------------------------- 8-bit pages to bf16 tiles
    if constexpr (C::kRaw) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsUnpack));
      constexpr int U = D / 16;                          // 16-channel units a row
      constexpr int RP = C::kDqWarps * 32 / U;           // rows a pass, a multiple of 8
      constexpr int NP = 128 / RP;
      static_assert(RP % 8 == 0 && 128 % RP == 0, "rows a pass");
      const int tid = threadIdx.x - 384;
      // 128-byte swizzle: 16-byte unit v of row r at v ^ (r & 7).  At D = 128 the eight
      // threads that share a store meet both 64-column chunks, whose same units share
      // banks: the second chunk's take the neighbouring row, which flips the unit.
      const int c = tid % U, r0 = (tid / U) ^ (c >> 2), v = (c & 3) * 2;
      const int src_off = r0 * D + c * 16, scale_off = C::kRawCodes + r0 * (D / kCacheGroup) + (c >> 1);
      const int row_off = (c >> 2) * C::kChunkBytes + r0 * 128;
      const int dst_a = row_off + ((v ^ (r0 & 7)) << 4), dst_b = row_off + (((v + 1) ^ (r0 & 7)) << 4);
      int li = 0;
      bool ok = true;
      for (int g = 0; ok; ++g) {
        if (!__all_sync(0xffffffffu, seg_wait(g))) break;
        const CacheSeg& sr = segs[g % kSegRing];
        const bool end = sr.end;
        const int sa = sr.sa, sb = sr.sb, step0 = sr.it.step0, lo = sr.it.lo, hi = sr.it.hi;
        const int lo_max = sr.it.lo_max, hi_min = sr.it.hi_min;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[g % kSegRing]);
        if (end) break;
        for (int j = sa; ok && j < sb; ++j) {
          const int key0 = (step0 + j) << 7;
          const bool partial = key0 < lo_max || key0 > hi_min - 128;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++li) {
            if (!__all_sync(0xffffffffu, mbar_wait(&raw_full[li % NR], (li / NR) & 1, abort_flag, wlim))) {
              ok = false;
              break;
            }
            const uint8_t* src = raw_smem + (li % NR) * C::kRawBytes;
            uint8_t* dst = slot_smem + (li % NS) * TB;
            uint4 x[NP];
            uint32_t byte[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              x[i] = *reinterpret_cast<const uint4*>(src + src_off + i * RP * D);
              byte[i] = src[scale_off + i * RP * (D / kCacheGroup)];
            }
            if (kv == 1 && partial) {
              bool bad = false;
#pragma unroll
              for (int i = 0; i < NP; ++i) {
                const int key = key0 + r0 + i * RP;
                const bool seen = key >= lo && key < hi;
                const bool all = key >= lo_max && key < hi_min;
                if (!seen || (byte[i] == kCacheNanScale && !all)) {
                  bad = bad || seen;
                  x[i] = make_uint4(0u, 0u, 0u, 0u);
                  byte[i] = 127;
                }
              }
              if (bad) poison[g % kSegRing] = g + 1;
            }
            if (li >= NS && !__all_sync(0xffffffffu, mbar_wait(&slot_empty[li % NS], ((li / NS) - 1) & 1, abort_flag,
                                                               wlim))) {
              ok = false;
              break;
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              uint4 o0, o1;
              dequant16<FMT>(x[i], byte[i], o0, o1);
              *reinterpret_cast<uint4*>(dst + dst_a + i * RP * 128) = o0;
              *reinterpret_cast<uint4*>(dst + dst_b + i * RP * 128) = o1;
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&slot_full[li % NS]);
              mbar_arrive(&raw_empty[li % NR]);
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(taddr, 512);
}

// Joins the parts of the items that a split launch cut: CTA x has the item whose
// first part CTA x of that launch wrote (slot 1), followed by slot 0 of the CTAs
// after it up to the last part.  Weights 2^(m_i - max m), sums in order of the parts.
// A row belongs to D / 4 lanes: they weigh its parts side by side, then each adds up
// its four channels, N parts' loads in flight.  Chains of loads bound it: descriptors
// (32 at a look, with all that is needed of the item), then parts.  N = 8 for few rows
// (74 parts of 8 rows: 21 us with one load at a time, 6 so); chunks' items have many
// rows of few parts and take N = 4, whose registers let five CTAs on an SM.
constexpr int kJoinThreads = 256;
constexpr int kJoinMost = 3 * kCacheMaxCtas;     // parts of an item, at most one for each CTA

template <int D, int N>
__global__ void __launch_bounds__(kJoinThreads, N == 8 ? 3 : 5) cache_join_kernel(const CacheAttnParams p,
                                                                                  int rows_per_part, int ctas) {
  constexpr int L = D / 4;        // lanes a row
  constexpr int R = kJoinThreads / L;
  __shared__ float weights[R][kJoinMost];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int x = blockIdx.x, lane = threadIdx.x & 31;
  int4 d = make_int4(0, 0, kPartNone, 0);
  if (x + lane < ctas) d = p.part_desc[2 * (x + lane) + (lane == 0 ? 1 : 0)];
  if (__shfl_sync(0xffffffffu, d.z, 0) != kPartOpen) return;
  const int tok0 = __shfl_sync(0xffffffffu, d.x, 0), kv_head = __shfl_sync(0xffffffffu, d.y, 0);
  const int ntok = __shfl_sync(0xffffffffu, d.w, 0);
  // the first later part that is not open ends the item
  int parts = 0;
  while (true) {
    const uint32_t stop = __ballot_sync(0xffffffffu, d.z != kPartOpen);
    if (stop != 0u) {
      const int first = __ffs(stop) - 1;
      if (__shfl_sync(0xffffffffu, d.z, first) == kPartNone) return;   // a launch that gave up (recorded)
      parts += first + 1;
      break;
    }
    parts += 32;
    d.z = x + parts + lane < ctas ? p.part_desc[2 * (x + parts + lane)].z : kPartNone;
  }
  // row = tile * 128 + token of the tile * group + head of the group
  const int tile_rows = p.tile_tokens * p.group, rows = ntok * p.group;
  const int c = threadIdx.x % L, slot = threadIdx.x / L;
  const uint32_t lanes = L == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);
  float* w = weights[slot];
  for (int i = blockIdx.y * R + slot; i < rows; i += gridDim.y * R) {
    const int tile = i / tile_rows, row = tile * 128 + (i - tile * tile_rows);
    auto at = [&](int k) { return static_cast<int64_t>(k == 0 ? 2 * x + 1 : 2 * (x + k)) * rows_per_part + row; };
    // the first parts' channels do not wait for the weights
    float4 v[N];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int u = 0; u < N; ++u)
        if (k0 + u < parts) v[u] = __ldcs(reinterpret_cast<const float4*>(p.part_o + at(k0 + u) * D) + c);
    };
    fetch(0);
    float m = -INFINITY, l = 0.f;
    for (int k = c; k < parts; k += L) m = fmaxf(m, p.part_ml[at(k)].x);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, o));
    for (int k = c; k < parts; k += L) {
      const float2 b = p.part_ml[at(k)];
      const float f = join_weight(b.x, m);
      w[k] = f;
      l = fmaf(b.y, f, l);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) l += __shfl_xor_sync(lanes, l, o);
    __syncwarp(lanes);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < parts; k0 += N) {
      if (k0 > 0) fetch(k0);
#pragma unroll
      for (int u = 0; u < N; ++u) {
        if (k0 + u >= parts) continue;
        const float f = w[k0 + u];
        o.x = fmaf(v[u].x, f, o.x);
        o.y = fmaf(v[u].y, f, o.y);
        o.z = fmaf(v[u].z, f, o.z);
        o.w = fmaf(v[u].w, f, o.w);
      }
    }
    __syncwarp(lanes);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t token = tok0 + i / p.group;
    const int head = kv_head * p.group + i % p.group;
    *reinterpret_cast<uint2*>(p.o + token * p.o_token + head * p.o_head + c * 4) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (c == 0)
      p.lse[static_cast<int64_t>(head) * p.s.num_tokens + token] =
          l == 0.f ? -INFINITY : m * 0.69314718055994531f + __logf(l);
  }
}

}  // namespace dynrad
