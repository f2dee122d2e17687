// Host test of the overlap checks (block_sparse_attention_candidate_b200/csrc/rows.h)
// against every pair of rows.  Prints "ok" and exits 0 when every check holds.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "rows.h"

#define CHECK(c)                                                   \
  do {                                                             \
    if (!(c)) {                                                    \
      std::printf("FAILED line %d: %s\n", __LINE__, #c);           \
      return 1;                                                    \
    }                                                              \
  } while (0)

using dynrad::rows_meet;
using dynrad::rows_meet_own;

static std::vector<int64_t> starts(int64_t at, int64_t ts, int64_t hs, int64_t tokens, int64_t heads) {
  std::vector<int64_t> r;
  for (int64_t t = 0; t < tokens; ++t)
    for (int64_t h = 0; h < heads; ++h) r.push_back(at + t * ts + h * hs);
  return r;
}

static const void* at(int64_t element) { return reinterpret_cast<const void*>(static_cast<uintptr_t>(2 * element)); }

int main() {
  std::mt19937 rng(1);
  auto pick = [&](int lo, int hi) { return static_cast<int64_t>(std::uniform_int_distribution<int>(lo, hi)(rng)); };
  int64_t own[2] = {0, 0}, two[2] = {0, 0}, other[2] = {0, 0};
  for (int n = 0; n < 300000; ++n) {
    const int64_t D = pick(0, 1) ? 64 : 128, tokens = pick(1, 7), heads = pick(1, 6);
    int64_t ts, hs;
    switch (pick(0, 3)) {
      case 0: ts = (heads + pick(0, heads + 2)) * D, hs = D; break;       // a slice of wider tokens
      case 1: ts = D, hs = (tokens + pick(0, tokens + 2)) * D; break;     // of heads with more tokens
      case 2: ts = pick(1, 4) * D, hs = pick(1, 4) * D; break;
      default: ts = 8 * pick(0, 60), hs = 8 * pick(0, 60);
    }
    const int64_t base = 1 << 20, to = base + 8 * pick(-300, 300);
    const auto a = starts(base, ts, hs, tokens, heads), b = starts(to, ts, hs, tokens, heads);
    bool self = false, meet = false;
    for (size_t i = 0; i < a.size(); ++i)
      for (size_t j = 0; j < b.size(); ++j) {
        self = self || (i < j && std::llabs(a[i] - a[j]) < D);
        meet = meet || std::llabs(a[i] - b[j]) < D;
      }
    CHECK(rows_meet_own(ts, hs, tokens, heads, D) == self);
    ++own[self];
    if (self) continue;     // rows_meet is asked about operands whose own rows are apart
    CHECK(rows_meet(at(base), ts, hs, at(to), ts, hs, tokens, heads, D) == meet);
    ++two[meet];
    // other strides: never apart where a row is shared, apart where the spans are
    const int64_t ts2 = 8 * pick(0, 60), hs2 = 8 * pick(0, 60);
    const auto c = starts(to, ts2, hs2, tokens, heads);
    bool meet2 = false;
    for (int64_t x : a)
      for (int64_t y : c) meet2 = meet2 || std::llabs(x - y) < D;
    const bool spans = a.back() + D > c.front() && c.back() + D > a.front();
    const bool got = rows_meet(at(base), ts, hs, at(to), ts2, hs2, tokens, heads, D);
    CHECK(got || !meet2);
    CHECK(!got || spans);
    ++other[got];
  }
  CHECK(own[0] > 10000 && own[1] > 10000 && two[0] > 10000 && two[1] > 10000 && other[0] > 10000 && other[1] > 10000);
  // large strides do not wrap
  const int64_t big = (int64_t{1} << 62) + (int64_t{1} << 61);
  CHECK(rows_meet(at(1 << 20), big, 128, at(1 << 24), 512, 128, 7, 4, 128));
  CHECK(!rows_meet(at(1 << 20), 512, 128, at((1 << 20) + 7 * 512), 512, 128, 7, 4, 128));
  CHECK(!rows_meet(at(1 << 20), 512, 128, at((1 << 20) + 128), big, big, 1, 1, 128));
  CHECK(!rows_meet_own(big, 128, 7, 4, 128) && !rows_meet_own(big, big - 128, 2, 1, 128));
  std::printf("ok\n");
  return 0;
}
