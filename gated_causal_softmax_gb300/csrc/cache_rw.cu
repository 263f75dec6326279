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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks = 152 * 8;
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

// The place of packed row t; blk < 0: left out.
struct Place {
  int blk, slot;
  long long pos;
};
__device__ __forceinline__ Place place_of(const CacheParams& p, int t) {
  Place w{-1, 0, 0};
  const int r = warp_last_le(p.num_reqs + 1, t, [&](int i) { return __ldg(p.cu + i); });
  if (r >= p.num_reqs) return w;  // behind the last request
  long long a = 0, b = 0;
  if (r >= 0) {
    a = __ldg(p.cu + r);
    b = __ldg(p.cu + r + 1);
  }
  if (!(r >= 0 && a <= t && t < b)) {  // cu does not start at 0 or is not sorted
    if ((threadIdx.x & 31) == 0) record_bad(p.status);
    return w;
  }
  w.pos = __ldg(p.seq_lens + r) - (b - a) + (t - a);
  w.blk = block_of(p, r, w.pos);
  w.slot = (int)(w.pos & (p.block_size - 1));
  return w;
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
// A tile is 128 positions of one request x 32 query heads: a warp holds 16 positions (aligned, so
// they lie in one block and their cached values are 64 contiguous bytes of a head), a lane one
// head.  Tile slots of request r start at cu[r] / 128 + 2 r; at most floor(len / 128) + 2 are used.
constexpr int kTile = 128;
constexpr int kStrip = 16;
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
// Blocks [0, n_gate): a gate tile each; the rest: rows.  A warp takes one row of all heads of a
// share (queries, keys or values) of every step-th token.
template <int D, int FMT, bool ROPE>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const CacheParams p, const RopeParams q) {
  constexpr int L = RowLanes<D>::kLanes, R = RowLanes<D>::kRows;
  __shared__ float sums[2][kWarps][32];
  if ((int)blockIdx.x < p.n_gate) {
    write_gates(p, blockIdx.x / p.gate_groups, blockIdx.x % p.gate_groups, sums);
    return;
  }
  const int q_segs = ROPE ? (p.hq + R - 1) / R : 0, kv_segs = (p.hkv + R - 1) / R, segs = q_segs + 2 * kv_segs;
  const uint32_t w = (blockIdx.x - p.n_gate) * kWarps + (threadIdx.x >> 5);
  const uint32_t step = (gridDim.x - p.n_gate) * kWarps / segs;
  if (w >= step * segs) return;
  const int seg = w % segs;
  const bool is_q = seg < q_segs, is_v = seg >= q_segs + kv_segs;
  const int sub = threadIdx.x & (L - 1), grp = (threadIdx.x & 31) / L;
  const int h = (is_q ? seg : is_v ? seg - q_segs - kv_segs : seg - q_segs) * R + grp;
  const bool valid = h < (is_q ? p.hq : p.hkv);
  const bool turns = ROPE && !is_v;
  const RowRuns runs = row_runs(sub, turns ? q.rotary_dim : 0, turns && q.interleaved);
  const uint16_t* in = is_q ? q.q : is_v ? p.v : p.k;
  const long long ts = is_q ? q.q_ts : is_v ? p.v_ts : p.k_ts, hs = is_q ? q.q_hs : is_v ? p.v_hs : p.k_hs;
  float wt[16];
  if (turns) load_weights(is_q ? q.q_weight : q.k_weight, runs, wt);
  for (uint32_t t = w / segs; t < (uint32_t)p.total; t += step) {
    const RawRow raw = valid ? load_row(in + t * ts + h * hs, runs) : zero_row();
    const Place pl = place_of(p, t);
    if (pl.blk < 0) continue;
    float x[16];
    unpack_row(raw, x);
    if (ROPE) {
      long long pos = pl.pos;
      if (q.positions) pos = __ldg(q.positions + t);
      if (pos < 0) continue;
      if (q.cos_sin && pos >= q.max_pos) {
        if ((threadIdx.x & 31) == 0) record_bad(p.status);
        continue;
      }
      if (turns) {
        Angles ang;
        load_angles(q.cos_sin, pos, q.rotary_dim, sub, runs, ang);
        if (q.norm) {
          const float r = row_rstd<D>(x, q.eps);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = x[i] * r * wt[i];
        }
        rotate_row<false>(x, runs, ang, q.interleaved);
        if (is_q) {
          if (valid) store_row(q.q_out + t * q.qo_ts + h * q.qo_hs, runs, x);
          continue;
        }
      }
    }
    write_cache_row<D, FMT>(p, is_v ? p.v_cache : p.k_cache, is_v ? p.v_scale : p.k_scale, pl, h, valid, sub, runs, x);
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

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) cache_gather_kernel(const CacheParams p) {
  constexpr int L = RowLanes<D>::kLanes, R = RowLanes<D>::kRows;
  if ((int)blockIdx.x < p.n_gate) {
    read_gates(p, blockIdx.x / p.gate_groups, blockIdx.x % p.gate_groups);
    return;
  }
  const int kv_segs = (p.hkv + R - 1) / R, segs = 2 * kv_segs;
  const uint32_t w = (blockIdx.x - p.n_gate) * kWarps + (threadIdx.x >> 5);
  const uint32_t step = (gridDim.x - p.n_gate) * kWarps / segs;
  if (w >= step * segs) return;
  const int seg = w % segs;
  const bool is_v = seg >= kv_segs;
  const int sub = threadIdx.x & (L - 1), grp = (threadIdx.x & 31) / L;
  const int h = (is_v ? seg - kv_segs : seg) * R + grp;
  const bool valid = h < p.hkv;
  const uint8_t* cache = is_v ? p.v_cache : p.k_cache;
  const float* scales = is_v ? p.v_scale : p.k_scale;
  uint16_t* out = is_v ? p.v_out : p.k_out;
  const long long ts = is_v ? p.v_ts : p.k_ts, hs = is_v ? p.v_hs : p.k_hs;
  for (uint32_t t = w / segs; t < (uint32_t)p.total; t += step) {
    const Place pl = place_of(p, t);
    if (pl.blk < 0 || !valid) continue;
    const uint8_t* row = cache + (long long)pl.blk * p.kv_bs + (long long)h * p.kv_hs + (long long)pl.slot * p.kv_ss;
    uint4* dst = reinterpret_cast<uint4*>(out + t * ts + h * hs + 16 * sub);
    if (FMT == kCacheBf16) {
      const uint4* src = reinterpret_cast<const uint4*>(row) + 2 * sub;
      const uint4 u = __ldg(src), v = __ldg(src + 1);
      dst[0] = u;
      dst[1] = v;
    } else {
      const uint4 c = __ldg(reinterpret_cast<const uint4*>(row) + sub);
      const float sc =
          __ldg(FMT == kCachePerToken ? scales + ((size_t)pl.blk * p.hkv + h) * p.block_size + pl.slot : scales);
      const uint2 u0 = from_e4m3x4(c.x, sc), u1 = from_e4m3x4(c.y, sc), u2 = from_e4m3x4(c.z, sc),
                  u3 = from_e4m3x4(c.w, sc);
      dst[0] = make_uint4(u0.x, u0.y, u1.x, u1.y);
      dst[1] = make_uint4(u2.x, u2.y, u3.x, u3.y);
    }
  }
}

int row_blocks(int total, int segs) {
  const long long blocks = ((long long)total * segs + kWarps - 1) / kWarps;
  return (int)std::max<long long>(std::min<long long>(blocks, kMaxBlocks), (segs + kWarps - 1) / kWarps);
}

void plan_gates(CacheParams& p, bool gates) {
  p.gate_groups = (p.hq + 31) / 32;
  p.n_gate = gates ? cache_gate_slots(p.total, p.num_reqs) * p.gate_groups : 0;
}

template <int D, int FMT, bool ROPE>
cudaError_t append(const CacheParams& p, const RopeParams& q, cudaStream_t s) {
  constexpr int R = RowLanes<D>::kRows;
  const int segs = (ROPE ? (p.hq + R - 1) / R : 0) + 2 * ((p.hkv + R - 1) / R);
  cache_append_kernel<D, FMT, ROPE><<<p.n_gate + row_blocks(p.total, segs), kThreads, 0, s>>>(p, q);
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
  cache_gather_kernel<D, FMT><<<p.n_gate + row_blocks(p.total, 2 * ((p.hkv + R - 1) / R)), kThreads, 0, s>>>(p);
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
