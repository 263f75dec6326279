// Where the packed rows of a cache call are cached: the request of a row, its position, and the block
// and slot of the paged cache.  Every index that comes from a device array is checked against its
// buffer before it is used, whatever the arrays hold: that walk is this file, apart from the kernels,
// so that it also compiles for the host, where a test takes it over arrays that break every
// precondition and looks at each index.
//
// P has the index arrays and sizes of CacheParams.  Warp is what a warp does (on the host the
// includer's): count(f), for how many lanes f(lane) holds; load(p), an element of an index array;
// bad(p), a record that an index lies outside, once for the warp.
#pragma once

#include <stddef.h>

#ifdef __CUDACC__
#include "kernels.h"
#include "sm103_ptx.cuh"
#define GCS_WALK __device__ __forceinline__
#else
#define GCS_WALK inline
#endif

namespace gcs {

#ifdef __CUDACC__
struct Warp {
  template <typename F>
  static GCS_WALK int count(F f) {
    return __popc(__ballot_sync(0xffffffffu, f(threadIdx.x & 31)));
  }
  static GCS_WALK int load(const int32_t* p) { return __ldg(p); }
  template <typename P>
  static GCS_WALK void bad(const P& p) {
    if ((threadIdx.x & 31) == 0) atomicCAS(p.status, kDevOk, kDevInvalidArg);
  }
};
#endif

// The last i in [0, n) with f(i) <= t, by the whole warp, for f that does not decrease; -1 if
// there is none.  Whatever f returns, i stays in [-1, n).
template <typename F>
GCS_WALK int warp_last_le(int n, int t, F f) {
  int lo = 0, left = n;
  while (true) {
    const int stride = (left + 31) / 32;
    const int c = Warp::count([&](int lane) { return lane * stride < left && f(lo + lane * stride) <= t; });
    if (c == 0) return lo - 1;
    if (stride == 1) return lo + c - 1;
    lo += (c - 1) * stride;
    const int rest = left - (c - 1) * stride;
    left = stride < rest ? stride : rest;
  }
}

// The table's entry for position pos of request r in [0, num_reqs), -1 for a position outside the
// table: to be checked before its use.
template <typename P>
GCS_WALK int table_entry(const P& p, int r, long long pos) {
  return pos >= 0 && pos < p.capacity ? Warp::load(p.block_table + ((size_t)r * p.max_blocks + (pos >> p.log2_block))) : -1;
}
// The entry if it is a block of the cache; -1, and a record, if not.
template <typename P>
GCS_WALK int checked_block(const P& p, int entry) {
  if (entry >= 0 && entry < p.num_blocks) return entry;
  Warp::bad(p);
  return -1;
}
template <typename P>
GCS_WALK int block_of(const P& p, int r, long long pos) {
  return checked_block(p, table_entry(p, r, pos));
}

// Where packed row t is cached: blk < 0: left out.
struct Place {
  int blk, slot, pos;
};
// A warp goes through neighbouring rows, so it looks the request up again only past its end, and
// the block only past the block's.
struct Cursor {
  int r = -1, a = 0, b = 0;  // the request of the rows [a, b): none of a cursor that has found none
  int shift = 0;             // position - row
  int page = -1, blk = -1;
};
// The cursor takes a request's rows on only when row t is one of them: the rows after a row that
// belongs to none (or to a request that cu, not sorted, does not lead to) are looked up again.
template <typename P>
GCS_WALK bool find_request(const P& p, int t, Cursor& c) {
  c.a = c.b = 0;
  const int r = warp_last_le(p.num_reqs + 1, t, [&](int i) { return Warp::load(p.cu + i); });
  if (r >= p.num_reqs) return false;  // behind the last request
  const int a = r >= 0 ? Warp::load(p.cu + r) : 0, b = r >= 0 ? Warp::load(p.cu + (r + 1)) : 0;
  if (t < a || t >= b) {  // cu does not start at 0 or is not sorted
    Warp::bad(p);
    return false;
  }
  c.r = r;
  c.a = a;
  c.b = b;
  // rows stay below 2^30: a position below that is negative with either shift
  const long long shift = (long long)Warp::load(p.seq_lens + r) - b, least = -(1LL << 30) - 1;
  c.shift = (int)(shift > least ? shift : least);
  c.page = -1;
  c.blk = -1;
  return true;
}
template <typename P>
GCS_WALK Place place_of(const P& p, int t, Cursor& c) {
  Place w{-1, 0, 0};
  if ((t < c.a || t >= c.b) && !find_request(p, t, c)) return w;
  w.pos = t + c.shift;
  const int page = w.pos >> p.log2_block;
  if (page != c.page || w.pos < 0) {
    c.page = page;
    c.blk = block_of(p, c.r, w.pos);
  }
  w.blk = c.blk;
  w.slot = w.pos & (p.block_size - 1);
  return w;
}

// A step of a warp takes `tokens` rows of the packed tensors: one, or with few kv heads as many as
// its lane groups have room for (powers of two).  This lane's group works on row t + off.
struct Step {
  int tokens, off, head;  // head: of the group, from the share's first on
  int lanes;              // of one row's heads
};
// This lane's place; the same block for all rows of the step in the middle of a block, and one by
// one over the ends.
template <typename P>
GCS_WALK Place place_of(const P& p, int t, int t1, const Step& s, Cursor& c) {
  if (s.tokens == 1) return place_of(p, t, c);
  const int n = s.tokens < t1 - t ? s.tokens : t1 - t;
  if (n > 1 && t >= c.a && t + n <= c.b && t + c.shift >= 0 && (t + c.shift) >> p.log2_block == c.page &&
      (t + n - 1 + c.shift) >> p.log2_block == c.page) {
    Place w{s.off < n ? c.blk : -1, 0, t + c.shift + (s.off < n ? s.off : 0)};
    w.slot = w.pos & (p.block_size - 1);
    return w;
  }
  Place w = place_of(p, t, c);
  for (int i = 1; i < n; ++i) {
    const Place x = place_of(p, t + i, c);
    if (s.off == i) w = x;
  }
  if (s.off >= n) w.blk = -1;
  return w;
}

}  // namespace gcs
