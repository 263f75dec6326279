// The walk from packed rows to cache slots (csrc/cache_places.h) on the host, over index arrays that
// keep the preconditions and arrays that break them: sorted and unsorted, negative, past every end.
// Every index that the walk reads is checked against its array, and every place that it gives against
// the arrays themselves.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>
#include <vector>

static void fail(const char* what, long long a, long long b) {
  printf("%s: %lld %lld\n", what, a, b);
  exit(1);
}

// An index array whose reads are checked.
struct Checked {
  const std::vector<int>* v;
  long long at;
  template <typename I>
  Checked operator+(I i) const {
    return Checked{v, at + (long long)i};
  }
};

static bool g_bad;
namespace gcs {
struct Warp {
  template <typename F>
  static int count(F f) {
    int n = 0;
    for (int lane = 0; lane < 32; ++lane) n += f(lane) ? 1 : 0;
    return n;
  }
  static int load(const Checked& p) {
    if (p.at < 0 || p.at >= (long long)p.v->size()) fail("an index outside its array", p.at, (long long)p.v->size());
    return (*p.v)[(size_t)p.at];
  }
  template <typename P>
  static void bad(const P&) {
    g_bad = true;
  }
};
}  // namespace gcs
#include "../../gated_causal_softmax_gb300/csrc/cache_places.h"
using namespace gcs;

struct Params {
  int num_reqs, total;
  Checked cu, seq_lens, block_table;
  int max_blocks, num_blocks, block_size, log2_block;
  long long capacity;
};

// What the row's own look at the arrays allows: some request whose rows hold t, at its position.
static bool allowed(const Params& p, const std::vector<int>& cu, const std::vector<int>& lens, const std::vector<int>& table,
                    int t, const Place& w) {
  for (int r = 0; r < p.num_reqs; ++r) {
    if (t < cu[r] || t >= cu[r + 1]) continue;
    const long long pos = (long long)lens[r] - cu[r + 1] + t;
    if (pos < 0 || pos >= p.capacity || pos != w.pos || (pos & (p.block_size - 1)) != w.slot) continue;
    if (table[(size_t)r * p.max_blocks + (size_t)(pos >> p.log2_block)] == w.blk) return true;
  }
  return false;
}

// All runs of a call, with steps of `tokens` rows; returns the rows that have a place.
static int walk(const Params& p, const std::vector<int>& cu, const std::vector<int>& lens, const std::vector<int>& table,
                int runs, int tokens) {
  int placed = 0;
  for (int i = 0; i < runs; ++i) {
    const int t0 = (int)((long long)p.total * i / runs), t1 = (int)((long long)p.total * (i + 1) / runs);
    for (int off = 0; off < tokens; ++off) {  // the lanes of a warp one by one
      const Step s{tokens, off, 0, 32 / tokens};
      Cursor c;
      for (int t = t0; t < t1; t += tokens) {
        const Place w = place_of(p, t, t1, s, c);
        if (w.blk < 0) continue;
        if (t + off >= t1) fail("a place behind the run", t + off, t1);
        if (w.blk >= p.num_blocks || w.slot < 0 || w.slot >= p.block_size) fail("a place outside the cache", w.blk, w.slot);
        if (!allowed(p, cu, lens, table, t + off, w)) fail("a place of no request of the row", t + off, w.pos);
        ++placed;
      }
    }
  }
  return placed;
}

int main() {
  std::mt19937 rng(1);
  auto in = [&](int lo, int hi) { return (int)(lo + (long long)(rng() % (uint32_t)(hi - lo + 1))); };
  for (int round = 0; round < 6000; ++round) {
    const bool valid = round % 4 == 0;
    Params p{};
    // enough requests for two and three rounds of the search now and then
    p.num_reqs = round % 50 == 49 ? in(1000, 1200) : round % 10 == 9 ? in(30, 70) : in(1, 6);
    p.log2_block = in(4, 6);
    p.block_size = 1 << p.log2_block;
    p.max_blocks = in(1, 8);
    p.num_blocks = in(1, 40);
    p.capacity = (long long)p.max_blocks * p.block_size;
    std::vector<int> cu(p.num_reqs + 1), lens(p.num_reqs), table((size_t)p.num_reqs * p.max_blocks);
    for (int& x : table) x = in(0, p.num_blocks - 1);
    for (int r = 0; r < p.num_reqs; ++r) {
      const int most = p.num_reqs > 100 ? 3 : (int)p.capacity;
      const int n = in(0, 2) ? in(0, most) : 0;
      cu[r + 1] = cu[r] + n;
      lens[r] = n + in(0, (int)p.capacity - n);
    }
    p.total = cu[p.num_reqs] + in(0, 3);
    if (p.total == 0) p.total = 1;
    if (!valid) {
      const int odd[] = {-1, 0, 1, 3, -100, 60, p.total - 1, p.total, p.total + 1, 2 * p.total, INT32_MAX, INT32_MIN, -(1 << 30)};
      const int n_odd = (int)(sizeof(odd) / sizeof(odd[0]));
      for (int n = in(1, 4); n; --n) switch (in(0, 4)) {
          case 0: cu[in(0, p.num_reqs)] = odd[in(0, n_odd - 1)]; break;
          case 1: cu[in(0, p.num_reqs)] = in(0, p.total); break;
          case 2: std::swap(cu[in(0, p.num_reqs)], cu[in(0, p.num_reqs)]); break;
          case 3: lens[in(0, p.num_reqs - 1)] = odd[in(0, n_odd - 1)]; break;
          default: table[(size_t)in(0, (int)table.size() - 1)] = in(0, 1) ? -1 - in(0, 5) : p.num_blocks + in(0, 5);
        }
    }
    p.cu = Checked{&cu, 0};
    p.seq_lens = Checked{&lens, 0};
    p.block_table = Checked{&table, 0};
    for (int tokens = 1; tokens <= 8; tokens *= 2) {
      const int runs = in(1, p.total < 40 ? p.total : 40);
      g_bad = false;
      const int placed = walk(p, cu, lens, table, runs, tokens);
      if (valid && (g_bad || placed != cu[p.num_reqs])) fail("rows of valid arrays left out", placed, cu[p.num_reqs]);
      if (std::is_sorted(cu.begin(), cu.end()) && cu[0] > 0 && !g_bad) fail("a row before the first request, and no record", cu[0], p.total);
    }
  }
  // an array that leads row 99 to the request of the rows from 100 on, and row 100 to none: what row 99
  // finds must not serve row 100
  {
    std::vector<int> cu{0, 100, 200, 3}, lens{100, 100, 100}, table(3 * 7, 5);
    Params p{3, 200, Checked{&cu, 0}, Checked{&lens, 0}, Checked{&table, 0}, 7, 9, 16, 4, 7 * 16};
    for (int runs = 1; runs <= 200; ++runs)
      for (int tokens = 1; tokens <= 8; tokens *= 2) walk(p, cu, lens, table, runs, tokens);
  }
  puts("ok");
  return 0;
}
