// Write of new keys, values and log gates into the paged cache, and the read of cached rows back
// into packed tensors.  Row t of the packed tensors belongs to the request r with cu[r] <= t <
// cu[r + 1]; with len = cu[r + 1] - cu[r] it is cached position seq_lens[r] - len + t - cu[r], in
// slot position % block_size of block block_table[r][position / block_size].  (The paged calls
// place a request's query rows in the same way.)
//
//   fp8, per token   scale = max|x| / 448 over the row's d elements (stored), code = e4m3(x / scale)
//   fp8, per tensor  code = e4m3(x / scale) with the caller's scale
//   bf16             the elements as they are
//   gates            G_p = G_{p-1} + log_gate_p per query head, G_{-1} = 0
//   read             bf16(code * scale); log_gate_p = G_p - G_{p-1}
//
// e4m3() rounds to nearest even and saturates at +-448.  A row of zeros has scale 0 and codes 0;
// a row with an infinity or a NaN has that for its scale, and reads back as NaN wherever the
// products say so.
//
// All of it is bound by HBM, or by latency when there are few rows.  Every index that comes from
// a device array is checked against its buffer before it is used: a row whose place is not in
// the cache is left out and recorded in the status word.
#include <algorithm>

#include "kernels.h"
#include "rows.cuh"

namespace gcs {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Blocks of an SM: beyond 152 SMs full, warps take longer runs of tokens.
constexpr int kAppendBlocks = 4, kGatherBlocks = 8;
constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ void record_bad(int* status) { atomicCAS(status, kDevOk, kDevInvalidArg); }

// The last i in [0, n) with f(i) <= t, by the whole warp, for f that does not decrease; -1 if
// there is none.  Whatever f returns, i stays in [-1, n).
template <typename F>
__device__ __forceinline__ int warp_last_le(int n, int t, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, left = n;
  while (true) {
    const int stride = (left + 31) / 32;
    const int i = lane * stride;
    const int c = __popc(__ballot_sync(kFullMask, i < left && f(lo + i) <= t));
    if (c == 0) return lo - 1;
    if (stride == 1) return lo + c - 1;
    lo += (c - 1) * stride;
    left = min(stride, left - (c - 1) * stride);
  }
}

// The block that holds position pos of request r; -1 (and a record) when it is not in the cache.
__device__ __forceinline__ int block_of(const CacheParams& p, int r, long long pos) {
  if (pos >= 0 && pos < p.capacity) {
    const int blk = __ldg(p.block_table + (size_t)r * p.max_blocks + (pos >> p.log2_block));
    if (blk >= 0 && blk < p.num_blocks) return blk;
  }
  if ((threadIdx.x & 31) == 0) record_bad(p.status);
  return -1;
}

// Where packed row t is cached: blk < 0: left out.
struct Place {
  int blk, slot;
  long long pos;
};
// A warp goes through neighbouring rows, so it looks the request up again only past its end, and
// the block only past the block's.
struct Cursor {
  int r = -1, a = 0, b = 0;  // the request of the rows [a, b)
  long long shift = 0;       // position - row
  long long page = -1;
  int blk = -1;
};
__device__ __forceinline__ Place place_of(const CacheParams& p, int t, Cursor& c) {
  Place w{-1, 0, 0};
  if (t < c.a || t >= c.b) {
    c.a = c.b = 0;
    const int r = warp_last_le(p.num_reqs + 1, t, [&](int i) { return __ldg(p.cu + i); });
    if (r >= p.num_reqs) return w;  // behind the last request
    if (r >= 0) {
      c.a = __ldg(p.cu + r);
      c.b = __ldg(p.cu + r + 1);
    }
    if (t < c.a || t >= c.b) {  // cu does not start at 0 or is not sorted
      if ((threadIdx.x & 31) == 0) record_bad(p.status);
      return w;
    }
    c.r = r;
    c.shift = (long long)__ldg(p.seq_lens + r) - c.b;
    c.page = -1;
    c.blk = -1;
  }
  w.pos = t + c.shift;
  const long long page = w.pos >> p.log2_block;
  if (page != c.page || w.pos < 0) {
    c.page = page;
    c.blk = block_of(p, c.r, w.pos);
  }
  w.blk = c.blk;
  w.slot = (int)(w.pos & (p.block_size - 1));
  return w;
}

// A warp's share of the rows: one of `segs` groups of heads, and a run of tokens [t, t1).
struct Run {
  int seg, t, t1;
};
__device__ __forceinline__ Run warp_run(const CacheParams& p, int segs) {
  const long long w = (long long)(blockIdx.x - p.n_gate) * kWarps + (threadIdx.x >> 5);
  const long long runs = (long long)(gridDim.x - p.n_gate) * kWarps / segs;  // of a group of heads
  Run x{(int)(w % segs), 0, 0};
  const long long i = w / segs;
  if (i < runs) {
    x.t = (int)(p.total * i / runs);
    x.t1 = (int)(p.total * (i + 1) / runs);
  }
  return x;
}

// ------------------------------------------------------------------------- e4m3
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

// Codes of x / scale.  The quotient is the rounded product with 1 / scale, corrected once by its
// exact remainder (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990), three multiply-adds an element in place of a division; scales near the ends
// of the exponent range, where the remainder could underflow, divide.  With a caller's scale the
// product can be far beyond +-448 (CUT), up to infinity: it saturates without the correction.
template <bool CUT>
__device__ __forceinline__ void quantise_row(const float* x, float scale, uint32_t* code) {
  float q[16];
  if (scale >= 0x1p-90f && scale <= 0x1p90f) {
    const float inv = 1.f / scale;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float y = x[i] * inv;
      q[i] = CUT && fabsf(y) > 512.f ? y : fmaf(fmaf(-y, scale, x[i]), inv, y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = scale > 0.f ? x[i] / scale : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) code[i] = to_e4m3x4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
}

// max|x| over the row.  Magnitudes compare as integers, and a NaN is above every number.
template <int L>
__device__ __forceinline__ float row_amax(const float* x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
  for (int off = L / 2; off; off >>= 1) m = max(m, __shfl_xor_sync(kFullMask, m, off));
  return __uint_as_float(m);
}

// Writes one row's 16 elements of a lane (row_runs order) to its slot of a cache.
template <int D, int FMT>
__device__ __forceinline__ void write_cache_row(const CacheParams& p, uint8_t* cache, float* scales, const Place& w,
                                                int h, bool valid, int sub, const RowRuns& runs, const float* x) {
  uint8_t* row = cache + (long long)w.blk * p.kv_bs + (long long)h * p.kv_hs + (long long)w.slot * p.kv_ss;
  if (FMT == kCacheBf16) {
    if (valid) store_row(reinterpret_cast<uint16_t*>(row), runs, x);
    return;
  }
  float scale;
  if (FMT == kCachePerToken) {
    scale = row_amax<RowLanes<D>::kLanes>(x) / kE4m3Max;
    if (valid && sub == 0) scales[((size_t)w.blk * p.hkv + h) * p.block_size + w.slot] = scale;
  } else {
    scale = __ldg(scales);
  }
  uint32_t code[4];
  quantise_row<FMT == kCachePerTensor>(x, scale, code);
  if (valid) {
    *reinterpret_cast<uint2*>(row + runs.a) = make_uint2(code[0], code[1]);
    *reinterpret_cast<uint2*>(row + runs.b) = make_uint2(code[2], code[3]);
  }
}

// ------------------------------------------------------------------------- gates
// A tile is 64 positions of one request x 32 query heads: a warp holds 16 positions (aligned, so
// they lie in one block and their cached values are 64 contiguous bytes of a head), a lane one
// head.  Tile slots of request r start at cu[r] / 64 + 2 r; at most floor(len / 64) + 2 are used.
constexpr int kStrip = 16;
constexpr int kTile = kStrip * kWarps;
// Up to this many positions a tile adds up the log gates before it by itself; for longer
// appends gate_sums_kernel adds up every tile first.
constexpr int kDirectRows = 512;

struct GateStrip {
  int r, a, tile;          // request, its first row, tile index within it
  long long p0, p1, s0;    // positions [p0, p1) of its rows; the strip's first position
  int h;                   // this lane's head
  bool any;                // the strip has rows
};
__device__ __forceinline__ bool gate_strip(const CacheParams& p, int slot, int hgroup, GateStrip& g) {
  g.r = warp_last_le(p.num_reqs, slot, [&](int i) { return __ldg(p.cu + i) / kTile + 2 * i; });
  if (g.r < 0) return false;
  g.a = __ldg(p.cu + g.r);
  const int b = __ldg(p.cu + g.r + 1);
  if (b <= g.a) return false;
  g.p1 = __ldg(p.seq_lens + g.r);
  g.p0 = g.p1 - ((long long)b - g.a);
  if (g.a < 0 || b > p.total || g.p0 < 0 || g.p1 > p.capacity) {
    if (threadIdx.x == 0) record_bad(p.status);
    return false;
  }
  g.tile = slot - (g.a / kTile + 2 * g.r);
  const long long first = (g.p0 & ~(long long)(kStrip - 1)) + (long long)g.tile * kTile;
  if (g.tile < 0 || first >= g.p1) return false;
  g.s0 = first + (threadIdx.x >> 5) * kStrip;
  g.h = hgroup * 32 + (threadIdx.x & 31);
  g.any = g.s0 < g.p1;
  return true;
}
// This lane's 16 log gates (0 outside the request's rows).
__device__ __forceinline__ void load_log_gates(const CacheParams& p, const GateStrip& g, float* v) {
#pragma unroll
  for (int i = 0; i < kStrip; ++i) {
    const long long pos = g.s0 + i;
    const bool in = pos >= g.p0 && pos < g.p1 && g.h < p.hq;
    v[i] = in ? __ldg(p.log_gate + (size_t)(g.a + (pos - g.p0)) * p.hq + g.h) : 0.f;
  }
}

// Sum of every tile's log gates, [tile slot][hq].
__global__ void __launch_bounds__(kThreads) gate_sums_kernel(const CacheParams p) {
  __shared__ float sums[kWarps][32];
  GateStrip g;
  if (!gate_strip(p, blockIdx.x, blockIdx.y, g)) return;
  float v[kStrip], sum = 0.f;
  load_log_gates(p, g, v);
#pragma unroll
  for (int i = 0; i < kStrip; ++i) sum += v[i];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && g.h < p.hq) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) sum += sums[i][lane];
    p.tile_sums[(size_t)blockIdx.x * p.hq + g.h] = sum;
  }
}

__device__ __forceinline__ void write_gates(const CacheParams& p, int slot, int hgroup, float (*sums)[kWarps][32]) {
  GateStrip g;
  if (!gate_strip(p, slot, hgroup, g)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool head = g.h < p.hq;
  float v[kStrip];
  load_log_gates(p, g, v);
  // the rows of the request before this tile, split over the warps
  float before = 0.f;
  if (p.tile_sums) {
    const float* ts = p.tile_sums + (size_t)(slot - g.tile) * p.hq + g.h;
    for (int j = warp; j < g.tile; j += kWarps)
      if (head) before += __ldg(ts + (size_t)j * p.hq);
  } else if (g.tile > 0) {
    const int n = (int)(g.s0 - warp * kStrip - g.p0);
    const float* lg = p.log_gate + (size_t)g.a * p.hq + g.h;
    for (int j = warp; j < n; j += kWarps)
      if (head) before += __ldg(lg + (size_t)j * p.hq);
  }
  float prev = 0.f;
  bool known = true;  // the cached gate to continue from
  if (g.p0 > 0) {
    const long long q = g.p0 - 1;
    const int blk = block_of(p, g.r, q);
    known = blk >= 0;
    if (known && head)
      prev = __ldcg(p.g_cache + ((size_t)blk * p.hq + g.h) * p.block_size + (q & (p.block_size - 1)));
  }
#pragma unroll
  for (int i = 1; i < kStrip; ++i) v[i] += v[i - 1];
  sums[0][warp][lane] = before;
  sums[1][warp][lane] = v[kStrip - 1];
  __syncthreads();
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) sum += sums[0][i][lane];
#pragma unroll
  for (int i = 0; i < kWarps; ++i)
    if (i < warp) sum += sums[1][i][lane];
  if (!g.any || !known) return;
  const int blk = block_of(p, g.r, g.s0);
  if (blk < 0 || !head) return;
  float* dst = p.g_cache + ((size_t)blk * p.hq + g.h) * p.block_size + (g.s0 & (p.block_size - 1));
#pragma unroll
  for (int i = 0; i < kStrip; ++i) v[i] = prev + (sum + v[i]);
  if (g.s0 >= g.p0 && g.s0 + kStrip <= g.p1) {
#pragma unroll
    for (int i = 0; i < kStrip; i += 4)
      *reinterpret_cast<float4*>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < kStrip; ++i)
      if (g.s0 + i >= g.p0 && g.s0 + i < g.p1) dst[i] = v[i];
  }
}

__device__ __forceinline__ void read_gates(const CacheParams& p, int slot, int hgroup) {
  GateStrip g;
  if (!gate_strip(p, slot, hgroup, g) || !g.any) return;
  const bool head = g.h < p.hq;
  const int blk = block_of(p, g.r, g.s0);
  if (blk < 0) return;
  const size_t row = ((size_t)blk * p.hq + g.h) * p.block_size;
  const int s = (int)(g.s0 & (p.block_size - 1));
  float prev = 0.f;
  if (s > 0) {
    if (head) prev = __ldg(p.g_cache + row + s - 1);
  } else if (g.s0 > 0) {
    const int b1 = block_of(p, g.r, g.s0 - 1);
    if (b1 >= 0 && head) prev = __ldg(p.g_cache + ((size_t)b1 * p.hq + g.h) * p.block_size + p.block_size - 1);
  }
  if (!head) return;
  float v[kStrip];
#pragma unroll
  for (int i = 0; i < kStrip; i += 4) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(p.g_cache + row + s + i));
    v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
  }
#pragma unroll
  for (int i = 0; i < kStrip; ++i) {
    const long long pos = g.s0 + i;
    if (pos >= g.p0 && pos < g.p1) p.log_gate_out[(size_t)(g.a + (pos - g.p0)) * p.hq + g.h] = v[i] - (i ? v[i - 1] : prev);
  }
}

// ------------------------------------------------------------------------- append
// Blocks [0, n_gate): a gate tile each; the rest: rows.  A warp takes either the queries of 2 R
// heads or the keys and values of R heads (R rows to a warp), of one token a step, with the copies
// of the next token under way.
template <int D, int FMT, bool ROPE>
__global__ void __launch_bounds__(kThreads, kAppendBlocks) cache_append_kernel(const CacheParams p, const RopeParams q) {
  constexpr int L = RowLanes<D>::kLanes, R = RowLanes<D>::kRows;
  __shared__ union {
    WarpStage<D, 2> ring[kWarps][2];
    float sums[2][kWarps][32];
  } sm;
  if ((int)blockIdx.x < p.n_gate) {
    write_gates(p, blockIdx.x / p.gate_groups, blockIdx.x % p.gate_groups, sm.sums);
    return;
  }
  const int q_segs = ROPE ? (p.hq + 2 * R - 1) / (2 * R) : 0;
  const Run run = warp_run(p, q_segs + (p.hkv + R - 1) / R);
  if (run.t >= run.t1) return;
  WarpStage<D, 2>* ring = sm.ring[threadIdx.x >> 5];
  const bool is_q = run.seg < q_segs;
  const int sub = threadIdx.x & (L - 1), grp = (threadIdx.x & 31) / L;
  const RowRuns plain = row_runs<D>(sub, 0, false);
  const RowRuns turned = ROPE ? row_runs<D>(sub, q.rotary_dim, q.interleaved) : plain;
  // the lane's two rows of a token: two query heads, or the key and the value of one head
  const int h = is_q ? run.seg * 2 * R + grp : (run.seg - q_segs) * R + grp;
  const int heads = is_q ? p.hq : p.hkv;
  const bool valid0 = h < heads, valid1 = is_q ? h + R < heads : valid0;
  const uint16_t* row0 = is_q ? q.q + (valid0 ? h : 0) * q.q_hs : p.k + (valid0 ? h : 0) * p.k_hs;
  const uint16_t* row1 = is_q ? q.q + (valid1 ? h + R : 0) * q.q_hs : p.v + (valid1 ? h : 0) * p.v_hs;
  const long long ts0 = is_q ? q.q_ts : p.k_ts, ts1 = is_q ? q.q_ts : p.v_ts;
  const RowRuns runs1 = is_q ? turned : plain;
  float wt[16];
  if (ROPE) load_weights(is_q ? q.q_weight : q.k_weight, turned, wt);

  Cursor cursor;
  // starts the copies of row t; its place (left out: blk < 0)
  auto fetch = [&](WarpStage<D, 2>& st, int t) {
    fetch_row(st, 0, row0 + t * ts0, turned, valid0);
    fetch_row(st, 1, row1 + t * ts1, runs1, valid1);
    Place w = place_of(p, t, cursor);
    if (ROPE && w.blk >= 0) {
      const long long pos = q.positions ? __ldg(q.positions + t) : w.pos;
      if (pos < 0) {
        w.blk = -1;
      } else if (q.cos_sin) {
        if (pos < q.max_pos) {
          fetch_angles(st, q.cos_sin, pos, q.rotary_dim);
        } else {
          if ((threadIdx.x & 31) == 0) record_bad(p.status);
          w.blk = -1;
        }
      }
    }
    return w;
  };
  auto norm_turn = [&](float* x, const Angles& ang) {
    if (q.norm) {
      const float r = row_rstd<D>(x, q.eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = x[i] * r * wt[i];
    }
    rotate_row<false>(x, turned, ang, q.interleaved);
  };
  auto use = [&](const WarpStage<D, 2>& st, int t, const Place& w) {
    if (w.blk < 0) return;
    float x[16];
    Angles ang;
    if (ROPE) read_angles(st.angles, q.rotary_dim, turned, ang);
    unpack_row(fetched_row(st, 0), x);
    if (ROPE) norm_turn(x, ang);
    if (ROPE && is_q) {
      uint16_t* out = q.q_out + t * q.qo_ts;
      if (valid0) store_row(out + h * q.qo_hs, turned, x);
      unpack_row(fetched_row(st, 1), x);
      norm_turn(x, ang);
      if (valid1) store_row(out + (h + R) * q.qo_hs, turned, x);
    } else {
      write_cache_row<D, FMT>(p, p.k_cache, p.k_scale, w, h, valid0, sub, turned, x);
      unpack_row(fetched_row(st, 1), x);
      write_cache_row<D, FMT>(p, p.v_cache, p.v_scale, w, h, valid0, sub, plain, x);
    }
  };

  Place now = fetch(ring[0], run.t), next = now;
  copy_commit();
  for (int t = run.t, slot = 0; t < run.t1; ++t, slot ^= 1) {
    if (t + 1 < run.t1) next = fetch(ring[slot ^ 1], t + 1);
    copy_commit();
    copy_wait<1>();
    __syncwarp();
    use(ring[slot], t, now);
    __syncwarp();
    now = next;
  }
}

// ------------------------------------------------------------------------- gather
// Values of 4 codes times the scale, rounded to bf16.
__device__ __forceinline__ uint2 from_e4m3x4(uint32_t code, float scale) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)code));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(code >> 16)));
  float x[4];
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
      : "=f"(x[0]), "=f"(x[1])
      : "r"(lo));
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
      : "=f"(x[2]), "=f"(x[3])
      : "r"(hi));
  return make_uint2(pack_bf16x2(x[0] * scale, x[1] * scale), pack_bf16x2(x[2] * scale, x[3] * scale));
}

// The codes (or bf16 elements) and scales of a warp's steps ahead; codes and scales are copied and
// read by the same lane.
constexpr int kGatherStages = 4;
template <int FMT>
struct alignas(16) GatherStage {
  static constexpr int kRun = FMT == kCacheBf16 ? 16 : 8;  // bytes of a run of 8 elements
  uint8_t raw[2][2][32][kRun];                             // keys, values; the lane's two runs
  float scale[2][32];
};

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, kGatherBlocks) cache_gather_kernel(const CacheParams p) {
  constexpr int L = RowLanes<D>::kLanes, R = RowLanes<D>::kRows;
  using Stage = GatherStage<FMT>;
  __shared__ Stage rings[kWarps][kGatherStages];
  if ((int)blockIdx.x < p.n_gate) {
    read_gates(p, blockIdx.x / p.gate_groups, blockIdx.x % p.gate_groups);
    return;
  }
  const Run run = warp_run(p, (p.hkv + R - 1) / R);
  if (run.t >= run.t1) return;
  Stage* ring = rings[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31, sub = lane & (L - 1), h = run.seg * R + lane / L;
  const bool valid = h < p.hkv;
  const RowRuns runs = row_runs<D>(sub, 0, false);
  const float ks = FMT == kCachePerTensor ? __ldg(p.k_scale) : 1.f, vs = FMT == kCachePerTensor ? __ldg(p.v_scale) : 1.f;
  Cursor cursor;
  uint32_t there = 0;  // bit i: the row i steps back from the last fetched one is in the cache
  auto fetch = [&](Stage& st, int t) {
    there <<= 1;
    const Place w = place_of(p, t, cursor);
    if (w.blk < 0) return;
    there |= 1;
    if (!valid) return;
    const long long row = (long long)w.blk * p.kv_bs + h * p.kv_hs + (long long)w.slot * p.kv_ss;
    constexpr int B = Stage::kRun;
    copy_async<B>(st.raw[0][0][lane], p.k_cache + row + runs.a * (B / 8));
    copy_async<B>(st.raw[0][1][lane], p.k_cache + row + runs.b * (B / 8));
    copy_async<B>(st.raw[1][0][lane], p.v_cache + row + runs.a * (B / 8));
    copy_async<B>(st.raw[1][1][lane], p.v_cache + row + runs.b * (B / 8));
    if (FMT == kCachePerToken) {
      const size_t s = ((size_t)w.blk * p.hkv + h) * p.block_size + w.slot;
      copy_async<4>(&st.scale[0][lane], p.k_scale + s);
      copy_async<4>(&st.scale[1][lane], p.v_scale + s);
    }
  };
  auto write = [&](const Stage& st, int i, float scale, uint16_t* row) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint4* dst = reinterpret_cast<uint4*>(row + (r ? runs.b : runs.a));
      if (FMT == kCacheBf16) {
        *dst = *reinterpret_cast<const uint4*>(st.raw[i][r][lane]);
      } else {
        const uint2 c = *reinterpret_cast<const uint2*>(st.raw[i][r][lane]);
        const uint2 u = from_e4m3x4(c.x, scale), v = from_e4m3x4(c.y, scale);
        *dst = make_uint4(u.x, u.y, v.x, v.y);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kGatherStages - 1; ++i) {
    if (run.t + i < run.t1) fetch(ring[i], run.t + i);
    else there <<= 1;
    copy_commit();
  }
  int slot = 0;
  for (int t = run.t; t < run.t1; ++t) {
    if (t + kGatherStages - 1 < run.t1) fetch(ring[(slot + kGatherStages - 1) % kGatherStages], t + kGatherStages - 1);
    else there <<= 1;
    copy_commit();
    copy_wait<kGatherStages - 1>();
    if ((there >> (kGatherStages - 1) & 1) && valid) {
      const Stage& st = ring[slot];
      const bool per_token = FMT == kCachePerToken;
      write(st, 0, per_token ? st.scale[0][lane] : ks, p.k_out + t * p.k_ts + h * p.k_hs);
      write(st, 1, per_token ? st.scale[1][lane] : vs, p.v_out + t * p.v_ts + h * p.v_hs);
    }
    slot = (slot + 1) % kGatherStages;
  }
}

int row_blocks(int total, int segs, int most) {
  const long long blocks = ((long long)total * segs + kWarps - 1) / kWarps;
  // at least one warp for each group of heads
  return (int)std::max<long long>(std::min<long long>(blocks, most), (segs + kWarps - 1) / kWarps);
}

void plan_gates(CacheParams& p, bool gates) {
  p.gate_groups = (p.hq + 31) / 32;
  p.n_gate = gates ? cache_gate_slots(p.total, p.num_reqs) * p.gate_groups : 0;
}

template <int D, int FMT, bool ROPE>
cudaError_t append(const CacheParams& p, const RopeParams& q, cudaStream_t s) {
  constexpr int R = RowLanes<D>::kRows;
  const int segs = (ROPE ? (p.hq + 2 * R - 1) / (2 * R) : 0) + (p.hkv + R - 1) / R;
  cache_append_kernel<D, FMT, ROPE>
      <<<p.n_gate + row_blocks(p.total, segs, 152 * kAppendBlocks), kThreads, 0, s>>>(p, q);
  return cudaGetLastError();
}
template <int D, int FMT>
cudaError_t append(const CacheParams& p, const RopeParams* q, cudaStream_t s) {
  return q ? append<D, FMT, true>(p, *q, s) : append<D, FMT, false>(p, RopeParams{}, s);
}
template <int D>
cudaError_t append(const CacheParams& p, const RopeParams* q, cudaStream_t s) {
  return p.format == kCachePerToken    ? append<D, kCachePerToken>(p, q, s)
         : p.format == kCachePerTensor ? append<D, kCachePerTensor>(p, q, s)
                                       : append<D, kCacheBf16>(p, q, s);
}

template <int D, int FMT>
cudaError_t gather(const CacheParams& p, cudaStream_t s) {
  constexpr int R = RowLanes<D>::kRows;
  cache_gather_kernel<D, FMT>
      <<<p.n_gate + row_blocks(p.total, (p.hkv + R - 1) / R, 152 * kGatherBlocks), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}
template <int D>
cudaError_t gather(const CacheParams& p, cudaStream_t s) {
  return p.format == kCachePerToken    ? gather<D, kCachePerToken>(p, s)
         : p.format == kCachePerTensor ? gather<D, kCachePerTensor>(p, s)
                                       : gather<D, kCacheBf16>(p, s);
}

}  // namespace

int cache_gate_slots(int total, int num_reqs) { return total / kTile + 2 * num_reqs; }

bool cache_gates_need_sums(int max_rows) { return max_rows > kDirectRows; }

cudaError_t launch_cache_append(const CacheParams& args, const RopeParams* rope, cudaStream_t s) {
  CacheParams p = args;
  plan_gates(p, p.log_gate != nullptr);
  if (p.tile_sums) {
    gate_sums_kernel<<<dim3(p.n_gate / p.gate_groups, p.gate_groups), kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  switch (p.d) {
    case 64: return append<64>(p, rope, s);
    case 128: return append<128>(p, rope, s);
    case 256: return append<256>(p, rope, s);
    default: return append<512>(p, rope, s);
  }
}

cudaError_t launch_cache_gather(const CacheParams& args, cudaStream_t s) {
  CacheParams p = args;
  plan_gates(p, p.log_gate_out != nullptr);
  switch (p.d) {
    case 64: return gather<64>(p, s);
    case 128: return gather<128>(p, s);
    case 256: return gather<256>(p, s);
    default: return gather<512>(p, s);
  }
}

}  // namespace gcs
