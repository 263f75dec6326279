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
// e4m3() rounds to nearest even and saturates at +-448.  A scale that is not above 0 (a row of zeros,
// or a NaN in the row) has codes 0; a row with an infinity has scale inf.  Both read back as the
// products say.
//
// All of it is bound by HBM, or by latency when there are few rows.  Every index that comes from
// a device array is checked against its buffer before it is used (cache_places.h): a row whose place
// is not in the cache is left out and recorded in the status word.
#include <algorithm>

#include "cache_places.h"
#include "kernels.h"
#include "rows.cuh"

namespace gcs {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kGatherBlocks = 8;  // of an SM
constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ void record_bad(int* status) { atomicCAS(status, kDevOk, kDevInvalidArg); }

template <int D>
__device__ __forceinline__ Step narrow_step(int log2_tokens) {
  const int lane = threadIdx.x & 31, lanes = 32 >> log2_tokens;
  return Step{1 << log2_tokens, lane >> (5 - log2_tokens), (lane & (lanes - 1)) / RowLanes<D>::kLanes, lanes};
}

// A warp's share of the rows, which the last row_blocks blocks take: one of `segs` groups of heads,
// and a run of tokens [t, t1).
struct Run {
  int seg, t, t1;
};
__device__ __forceinline__ Run warp_run(const CacheParams& p, int segs) {
  const long long w = ((long long)blockIdx.x - (gridDim.x - p.row_blocks)) * kWarps + (threadIdx.x >> 5);
  const long long runs = (long long)p.row_blocks * kWarps / segs;  // of a group of heads
  if (w < 0) return Run{0, 0, 0};
  Run x{(int)(w % segs), 0, 0};
  const long long i = w / segs;
  if (i < runs) {
    x.t = (int)(p.total * i / runs);
    x.t1 = (int)(p.total * (i + 1) / runs);
  }
  return x;
}

// ------------------------------------------------------------------------- e4m3
__device__ __forceinline__ uint32_t to_e4m3x4(const float2& a, const float2& b) {
  uint32_t r;
  asm("{.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {  // within an ulp
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// x / y for quotients away from the ends of the exponent range: the product with 1 / y corrected once by
// its exact remainder (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990), three multiply-adds in place of a division.  It is x / y rounded to
// fp32 where inv is the rounded reciprocal, as in scale_of; with reciprocal(), which may be an ulp off,
// that is not proven for every quotient.  Only codes are made of those: a quotient that is an e4m3 value or
// the middle of two comes out exactly (its remainder corrects the product to it), and the codes are
// tested bit by bit against those of the rounded quotients.
__device__ __forceinline__ float2 quotient2(const float2& x, const float2& y, const float2& inv) {
  const float2 q = mul2(x, inv);
  return fma2(fma2(neg2(q), y, x), inv, q);
}
constexpr float kSafeLo = 0x1p-80f, kSafeHi = 0x1p80f;  // of divisors whose remainders stay normal

__device__ __forceinline__ bool safe(float x) { return x >= kSafeLo && x <= kSafeHi; }

// max|x| / 448: the scale of a row from the largest magnitude.
__device__ __forceinline__ float scale_of(float amax) {
  const float q = quotient2(both(amax), both(kE4m3Max), both(1.f / kE4m3Max)).x;  // 0 of 0
  return safe(amax) || amax == 0.f ? q : amax / kE4m3Max;
}

__device__ __forceinline__ void pack_codes(const Row& q, uint32_t* code) {
#pragma unroll
  for (int i = 0; i < 4; ++i) code[i] = to_e4m3x4(q.e[2 * i], q.e[2 * i + 1]);
}
// Codes of x / scale; all bits 0 where the scale is not above 0 (the products with it would leave NaN, and
// the signs of zeros).  With a caller's scale (CUT) a quotient
// can be far beyond +-448, up to infinity, where the correction has no meaning: it saturates
// without.
template <bool CUT>
__device__ __forceinline__ void quantise_row(const Row& x, float scale, uint32_t* code) {
  const float2 y = both(scale), inv = both(scale > 0.f ? reciprocal(scale) : 0.f);
  Row q;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q.e[i] = quotient2(x.e[i], y, inv);
    if (CUT) {
      const float2 far = mul2(x.e[i], inv);
      if (fabsf(far.x) > 512.f) q.e[i].x = far.x;
      if (fabsf(far.y) > 512.f) q.e[i].y = far.y;
    }
  }
  pack_codes(q, code);
  const uint32_t keep = scale > 0.f ? 0xffffffffu : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) code[i] &= keep;
}
// The same by divisions, for the scales that quantise_row is not for.
__device__ __noinline__ uint4 divide_row(Row x, float scale) {
  if (!(scale > 0.f)) return make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) x.e[i] = make_float2(x.e[i].x / scale, x.e[i].y / scale);
  uint32_t c[4];
  pack_codes(x, c);
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// max|x| of N rows; a NaN anywhere is the maximum.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int L, int N>
__device__ __forceinline__ void row_amax(const Row (&x)[N], float (&m)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    m[n] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m[n] = max3_abs(x[n].e[i].x, x[n].e[i].y, m[n]);
  }
#pragma unroll
  for (int off = L / 2; off; off >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float o = __shfl_xor_sync(kFullMask, m[n], off);
      m[n] = max3_abs(m[n], o, o);
    }
}

// One head's rows of a cache as a lane writes them.
struct CacheRows {
  uint8_t* base;      // block 0, slot 0
  float* scale;       // per token: the same; per tensor: the scale
  float tensor_scale;
};
template <int FMT>
__device__ __forceinline__ CacheRows cache_rows(const CacheParams& p, uint8_t* cache, float* scales, int h) {
  CacheRows c{cache + h * p.kv_hs, scales, 0.f};
  if (FMT == kCachePerToken) c.scale += (size_t)h * p.block_size;
  if (FMT == kCachePerTensor) c.tensor_scale = __ldg(scales);
  return c;
}
// Writes a lane's elements of a head's key and value (x[0], x[1]) to their slots.
template <int D, int FMT>
__device__ __forceinline__ void write_cache_rows(const CacheParams& p, const CacheRows (&c)[2], const Place& w,
                                                 bool valid, int sub, const RowRuns (&runs)[2], const Row (&x)[2]) {
  const long long slot = (long long)w.blk * p.kv_bs + (long long)w.slot * p.kv_ss;
  if (FMT == kCacheBf16) {
    if (!valid) return;
#pragma unroll
    for (int n = 0; n < 2; ++n) store_row(reinterpret_cast<uint16_t*>(c[n].base + slot), runs[n], x[n]);
    return;
  }
  float scale[2];
  if (FMT == kCachePerToken) {
    row_amax<RowLanes<D>::kLanes>(x, scale);
    scale[0] = scale_of(scale[0]);
    scale[1] = scale_of(scale[1]);
  } else {
    scale[0] = c[0].tensor_scale;
    scale[1] = c[1].tensor_scale;
  }
  uint32_t code[2][4];
#pragma unroll
  for (int n = 0; n < 2; ++n) quantise_row<FMT == kCachePerTensor>(x[n], scale[n], code[n]);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    if (!safe(scale[n]) && scale[n] != 0.f) {
      const uint4 u = divide_row(x[n], scale[n]);
      code[n][0] = u.x, code[n][1] = u.y, code[n][2] = u.z, code[n][3] = u.w;
    }
  }
  if (!valid) return;
  const long long at = (long long)w.blk * p.hkv * p.block_size + w.slot;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    *reinterpret_cast<uint2*>(c[n].base + slot + runs[n].a) = make_uint2(code[n][0], code[n][1]);
    *reinterpret_cast<uint2*>(c[n].base + slot + runs[n].b) = make_uint2(code[n][2], code[n][3]);
    if (FMT == kCachePerToken && sub == 0) c[n].scale[at] = scale[n];
  }
}

// ------------------------------------------------------------------------- gates
// A tile is 64 positions of one request x 32 query heads: a warp holds 16 positions (aligned, so
// they lie in one block and their cached values are 64 contiguous bytes of a head), a lane one
// head.  Tile slots of request r start at cu[r] / 64 + 2 r; at most floor(len / 64) + 2 are used.
constexpr int kStrip = 16;
constexpr int kTile = kStrip * kWarps;
// Up to this many positions a tile adds up the log gates before it by itself; for longer appends
// the kernel that writes the rows adds up every tile, and the gates are a kernel behind it.  8
// requests of 256 rows: 7.3 us alone, 5.4 with the sums; of 128: 6.2 and 5.0, but a second launch
// costs the host 5.
constexpr int kDirectRows = 128;

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

// The sum of a tile's log gates, to p.tile_sums [tile slot][hq].
__device__ __forceinline__ void sum_gates(const CacheParams& p, int slot, int hgroup, float (*sums)[32]) {
  GateStrip g;
  if (!gate_strip(p, slot, hgroup, g)) return;
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
    p.tile_sums[(size_t)slot * p.hq + g.h] = sum;
  }
}

// Writes a tile's gates.  It is all latency, so its loads go out together: the table's entries and the
// log gates, then the gate to continue from, and last, behind the wait for the kernel that sums the
// tiles, the sums of the tiles before.
__device__ __forceinline__ void write_gates(const CacheParams& p, int slot, int hgroup, float (*sums)[kWarps][32]) {
  GateStrip g;
  if (!gate_strip(p, slot, hgroup, g)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool head = g.h < p.hq;
  const int h = head ? g.h : 0;
  const bool goes_on = g.p0 > 0;
  const int entry = g.any ? table_entry(p, g.r, g.s0) : -1;
  const int entry_before = goes_on ? table_entry(p, g.r, g.p0 - 1) : -1;
  float v[kStrip];
  load_log_gates(p, g, v);
  const int blk = g.any ? checked_block(p, entry) : -1;
  const int blk_before = goes_on ? checked_block(p, entry_before) : -1;
  float prev = 0.f;
  if (blk_before >= 0)
    prev = __ldcg(p.g_cache + ((size_t)blk_before * p.hq + h) * p.block_size + ((g.p0 - 1) & (p.block_size - 1)));
  // the rows of the request before this tile, split over the warps
  float before = 0.f;
  if (p.tile_sums) {
    grid_wait();
    const float* ts = p.tile_sums + (size_t)(slot - g.tile) * p.hq + h;
#pragma unroll 16
    for (int j = warp; j < g.tile; j += kWarps) before += __ldcg(ts + (size_t)j * p.hq);
  } else if (g.tile > 0) {
    const int n = (int)(g.s0 - warp * kStrip - g.p0);
    const float* lg = p.log_gate + (size_t)g.a * p.hq + h;
#pragma unroll 16
    for (int j = warp; j < n; j += kWarps) before += __ldg(lg + (size_t)j * p.hq);
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
  // nothing to write, or no cached gate to continue from
  if (blk < 0 || (goes_on && blk_before < 0) || !head) return;
  float* dst = p.g_cache + ((size_t)blk * p.hq + h) * p.block_size + (g.s0 & (p.block_size - 1));
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
  // the gate before the strip, where the strip's first position is a row: the other rows have theirs
  // inside.  Without it (its page is not in the cache) that row's log gate is left out.
  const bool reaches_back = g.s0 >= g.p0 && g.s0 > 0;
  bool has_first = true;
  float prev = 0.f;
  if (reaches_back && s > 0) {
    if (head) prev = __ldg(p.g_cache + row + s - 1);
  } else if (reaches_back) {
    const int b1 = block_of(p, g.r, g.s0 - 1);
    has_first = b1 >= 0;
    if (has_first && head) prev = __ldg(p.g_cache + ((size_t)b1 * p.hq + g.h) * p.block_size + p.block_size - 1);
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
    if (pos >= g.p0 && pos < g.p1 && (i || has_first))
      p.log_gate_out[(size_t)(g.a + (pos - g.p0)) * p.hq + g.h] = v[i] - (i ? v[i - 1] : prev);
  }
}

// ------------------------------------------------------------------------- append
template <int D>
using AppendStage = WarpStage<D, 2, RowLanes<D>::kRows>;

// Starts the copies of the angles of a step's rows, by their positions (the cached ones unless the
// caller gives others), and takes those out that have none.
template <int D>
__device__ __forceinline__ void start_angles(const RopeParams& q, int t, const Step& s, Place& w, AppendStage<D>& st) {
  int pos = w.pos;
  if (q.positions && w.blk >= 0) pos = __ldg(q.positions + t + s.off);
  if (pos < 0) w.blk = -1;
  if (!q.cos_sin) return;
  if (w.blk >= 0 && pos >= q.max_pos) {
    record_bad(q.status);
    w.blk = -1;
  }
  if (s.tokens == 1) {
    if (w.blk >= 0) fetch_angles(st.angles[0], q.cos_sin, pos, q.rotary_dim);
    return;
  }
  for (int i = 0; i < s.tokens; ++i) {
    const int at = __shfl_sync(kFullMask, pos, i * s.lanes), blk = __shfl_sync(kFullMask, w.blk, i * s.lanes);
    if (blk >= 0) fetch_angles(st.angles[i], q.cos_sin, at, q.rotary_dim);
  }
}

// Runs through a warp's rows with the copies of the next step under way: fetch(stage, t) starts the
// copies of a step's rows, use(stage, t, place) works on them.
template <int D, bool ROPE, typename Fetch, typename Use>
__device__ __forceinline__ void for_rows(const CacheParams& p, const RopeParams& q, const Run& run, const Step& s,
                                         AppendStage<D>* ring, Fetch fetch, Use use) {
  Cursor cursor;
  auto start = [&](AppendStage<D>& st, int t) {
    fetch(st, t);
    Place w = place_of(p, t, run.t1, s, cursor);
    if (ROPE) start_angles<D>(q, t, s, w, st);
    return w;
  };
  Place now = start(ring[0], run.t), next = now;
  copy_commit();
  int slot = 0;
  for (int t = run.t; t < run.t1; t += s.tokens, slot ^= 1) {
    if (t + s.tokens < run.t1) next = start(ring[slot ^ 1], t + s.tokens);
    copy_commit();
    copy_wait<1>();
    __syncwarp();
    use(ring[slot], t, now);
    __syncwarp();
    now = next;
  }
}

// A warp takes either the queries of 2 R heads or the keys and values of R heads (R rows to a
// warp), of one token a step, or with few kv heads the keys and values of several.
template <int D>
__device__ __forceinline__ void append_queries(const CacheParams& p, const RopeParams& q, const Run& run,
                                               AppendStage<D>* ring) {
  constexpr int L = RowLanes<D>::kLanes, R = RowLanes<D>::kRows;
  const int sub = threadIdx.x & (L - 1), h = run.seg * 2 * R + (threadIdx.x & 31) / L;
  const RowRuns runs = row_runs<D>(sub, q.rotary_dim, q.interleaved);
  const bool valid[2] = {h < p.hq, h + R < p.hq};
  const uint16_t* in[2] = {q.q + (valid[0] ? h : 0) * q.q_hs, q.q + (valid[1] ? h + R : 0) * q.q_hs};
  uint16_t* out = q.q_out + (valid[0] ? h : 0) * q.qo_hs;
  const Row w = load_weights(q.q_weight, runs);
  auto fetch = [&](AppendStage<D>& st, int t) {
    fetch_row(st, 0, in[0] + t * q.q_ts, runs, valid[0]);
    fetch_row(st, 1, in[1] + t * q.q_ts, runs, valid[1]);
  };
  auto use = [&](const AppendStage<D>& st, int t, const Place& place) {
    if (place.blk < 0) return;
    const Angles ang = read_angles<false>(st.angles[0], q.rotary_dim, runs);
    Row x[2] = {unpack_row(fetched_row(st, 0)), unpack_row(fetched_row(st, 1))};
    norm_rotate_rows<D>(x, w, runs, ang, q.norm, q.eps, q.interleaved);
    uint16_t* row = out + t * q.qo_ts;
    if (valid[0]) store_row(row, runs, x[0]);
    if (valid[1]) store_row(row + R * q.qo_hs, runs, x[1]);
  };
  for_rows<D, true>(p, q, run, Step{1, 0, 0, 32}, ring, fetch, use);
}

template <int D, int FMT, bool ROPE>
__device__ __forceinline__ void append_keys_values(const CacheParams& p, const RopeParams& q, const Run& run, int seg,
                                                   AppendStage<D>* ring) {
  constexpr int L = RowLanes<D>::kLanes, R = RowLanes<D>::kRows;
  const Step s = narrow_step<D>(p.log2_step);
  const int sub = threadIdx.x & (L - 1), head = seg * R + s.head;
  const bool has_head = head < p.hkv;
  const int h = has_head ? head : 0;
  const RowRuns plain = row_runs<D>(sub, 0, false);
  const RowRuns runs[2] = {ROPE ? row_runs<D>(sub, q.rotary_dim, q.interleaved) : plain, plain};
  const CacheRows rows[2] = {cache_rows<FMT>(p, p.k_cache, p.k_scale, h), cache_rows<FMT>(p, p.v_cache, p.v_scale, h)};
  const uint16_t *k = p.k + h * p.k_hs, *v = p.v + h * p.v_hs;
  Row w;
  if (ROPE) w = load_weights(q.k_weight, runs[0]);
  auto fetch = [&](AppendStage<D>& st, int t) {
    const bool valid = has_head && t + s.off < run.t1;
    const int row = valid ? t + s.off : t;
    fetch_row(st, 0, k + row * p.k_ts, runs[0], valid);
    fetch_row(st, 1, v + row * p.v_ts, plain, valid);
  };
  auto use = [&](const AppendStage<D>& st, int t, const Place& place) {
    Row x[2];
    x[0] = unpack_row(fetched_row(st, 0));
    if (ROPE) {
      Row key[1] = {x[0]};
      norm_rotate_rows<D>(key, w, runs[0], read_angles<false>(st.angles[s.off], q.rotary_dim, runs[0]), q.norm, q.eps,
                          q.interleaved);
      x[0] = key[0];
    }
    x[1] = unpack_row(fetched_row(st, 1));
    write_cache_rows<D, FMT>(p, rows, place, has_head && place.blk >= 0, sub, runs, x);
  };
  for_rows<D, ROPE>(p, q, run, s, ring, fetch, use);
}

template <int D, int FMT, bool ROPE>
__device__ __forceinline__ void append_rows(const CacheParams& p, const RopeParams& q, AppendStage<D>* ring) {
  constexpr int R = RowLanes<D>::kRows;
  const int q_segs = ROPE ? (p.hq + 2 * R - 1) / (2 * R) : 0;
  const Run run = warp_run(p, q_segs + (p.hkv + R - 1) / R);
  if (run.t >= run.t1) return;
  if (ROPE && run.seg < q_segs)
    append_queries<D>(p, q, run, ring);
  else
    append_keys_values<D, FMT, ROPE>(p, q, run, run.seg - q_segs, ring);
}

// Blocks of an SM; beyond 152 SMs full, warps take longer runs of tokens.  Four chunks of 1024 with the
// rotation 28 us with 4, 34 with 5 (spills); prompts of 36K tokens without it 42 with 4, 39 with 5.
template <bool ROPE>
constexpr int kAppendBlocks = ROPE ? 4 : 5;

// Rows in the last row_blocks blocks; gate tiles (their sums alone, with p.tile_sums) in all of
// them, from the first on: few of both run side by side.
//
// The rows are bound by HBM and by the latency of a step's chain (row maximum over the lanes, scale,
// quotients, conversion) at the few warps that their registers leave: 16 to 20 an SM, of which one issues
// in 54% of the cycles with the rotation and in 67% without.  A step of 4 keys and 4 values of 128 is 3 KB
// of traffic and about 330 instructions; shares of queries and of keys and values get the same number
// of warps, though theirs is not the same work.  Prompts of 36K tokens and 8 kv heads (231 MB) take
// 39 us, 5.9 TB/s, 87% of the measured copy rate, and 8 us more with the gates of 32 heads (10 MB), which
// are latency: two rounds over the tiles, of which only the first overlaps the rows.  Each tile adds up
// the sums of all before it: one request of 16K rows takes 0.35 ns a row more with 32 gate heads and 0.49
// with 64, one of 128K rows 0.34 and 0.60.
template <int D, int FMT, bool ROPE>
__global__ void __launch_bounds__(kThreads, kAppendBlocks<ROPE>)
    cache_append_kernel(const CacheParams p, const RopeParams q) {
  __shared__ union {
    AppendStage<D> ring[kWarps][2];
    float sums[2][kWarps][32];
  } sm;
  if (p.tile_sums) {
    grid_release();
    for (int i = blockIdx.x; i < p.n_gate; i += gridDim.x) {
      sum_gates(p, i / p.gate_groups, i % p.gate_groups, sm.sums[0]);
      __syncthreads();
    }
  }
  append_rows<D, FMT, ROPE>(p, q, sm.ring[threadIdx.x >> 5]);
  if (!p.tile_sums) {
    for (int i = blockIdx.x; i < p.n_gate; i += gridDim.x) {
      __syncthreads();
      write_gates(p, i / p.gate_groups, i % p.gate_groups, sm.sums);
    }
  }
}

// Behind the kernel with the tile sums.
__global__ void __launch_bounds__(kThreads) gate_tiles_kernel(const CacheParams p) {
  __shared__ float sums[2][kWarps][32];
  write_gates(p, blockIdx.x, blockIdx.y, sums);
  grid_wait();  // the call ends when both of its kernels have
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
//
// Bound by its writes, and by the load / store unit: each of a lane's 8 codes are an 8-byte copy, an
// 8-byte read and a 16-byte store.  60K tokens of 4 kv heads of 128 (188 MB) take 34.5 us, 5.4 TB/s, 80%
// of the measured copy rate; a fill of the 124 MB that it writes takes 32.  (16 neighbouring codes a
// lane with 32-byte stores 36 us, with two 16-byte stores 40; 2, 3 and 6 stages ahead the same.)
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
  for (int i = blockIdx.x; i < p.n_gate; i += gridDim.x) read_gates(p, i / p.gate_groups, i % p.gate_groups);
  const Run run = warp_run(p, (p.hkv + R - 1) / R);
  if (run.t >= run.t1) return;
  Stage* ring = rings[threadIdx.x >> 5];
  const Step s = narrow_step<D>(p.log2_step);
  const int lane = threadIdx.x & 31, sub = lane & (L - 1), h = run.seg * R + s.head;
  const bool has_head = h < p.hkv;
  const RowRuns runs = row_runs<D>(sub, 0, false);
  const float ks = FMT == kCachePerTensor ? __ldg(p.k_scale) : 1.f;
  const float vs = FMT == kCachePerTensor ? __ldg(p.v_scale) : 1.f;
  Cursor cursor;
  uint32_t there = 0;  // bit i: this lane's row i steps back from the last fetched one is in the cache
  auto fetch = [&](Stage& st, int t) {
    there <<= 1;
    const Place w = place_of(p, t, run.t1, s, cursor);
    if (w.blk < 0 || !has_head) return;
    there |= 1;
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
  auto start = [&](int slot, int t) {
    if (t < run.t1)
      fetch(ring[slot], t);
    else
      there <<= 1;
    copy_commit();
  };
  constexpr int S = kGatherStages;
#pragma unroll
  for (int i = 0; i < S - 1; ++i) start(i, run.t + i * s.tokens);
  int slot = 0;
  for (int t = run.t; t < run.t1; t += s.tokens) {
    start((slot + S - 1) % S, t + (S - 1) * s.tokens);
    copy_wait<S - 1>();
    if (there >> (S - 1) & 1) {
      const Stage& st = ring[slot];
      const bool per_token = FMT == kCachePerToken;
      const int row = t + s.off;
      write(st, 0, per_token ? st.scale[0][lane] : ks, p.k_out + row * p.k_ts + h * p.k_hs);
      write(st, 1, per_token ? st.scale[1][lane] : vs, p.v_out + row * p.v_ts + h * p.v_hs);
    }
    slot = (slot + 1) % S;
  }
}

// Rows of a step (its logarithm): as many as the kv heads leave room for among the R lane groups,
// once every warp of a full GPU has a row (before that a step of one row is the shortest way).  36K
// tokens of one head of 128 append in 9.2 us with 4 rows a step and in 24.0 with one.
template <int R>
int log2_step(const CacheParams& p, int most) {
  int n = 0;
  while ((2LL * p.hkv << n) <= R && p.total > (2LL * most * kWarps << n)) ++n;
  return n;
}

// Sets the blocks of the rows and the gate tiles; the grid's blocks: side by side as far as that
// fills the GPU once.
int plan(CacheParams& p, bool gates, int segs, int most) {
  p.gate_groups = (p.hq + 31) / 32;
  p.n_gate = gates ? cache_gate_slots(p.total, p.num_reqs) * p.gate_groups : 0;
  const long long rows = ((long long)p.total * segs + kWarps - 1) / kWarps;
  // at least one warp for each group of heads
  p.row_blocks = (int)std::max<long long>(std::min<long long>(rows, most), (segs + kWarps - 1) / kWarps);
  return std::max(p.row_blocks, (int)std::min<long long>((long long)p.n_gate + p.row_blocks, most));
}

template <int D, int FMT, bool ROPE>
cudaError_t append(CacheParams p, const RopeParams& q, cudaStream_t s) {
  constexpr int R = RowLanes<D>::kRows;
  const int segs = (ROPE ? (p.hq + 2 * R - 1) / (2 * R) : 0) + (p.hkv + R - 1) / R;
  const int blocks = plan(p, p.log_gate != nullptr, segs, 152 * kAppendBlocks<ROPE>);
  p.log2_step = log2_step<R>(p, 152 * kAppendBlocks<ROPE> / segs);
  cache_append_kernel<D, FMT, ROPE><<<blocks, kThreads, 0, s>>>(p, q);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.tile_sums) return e;
  return launch_behind(gate_tiles_kernel, dim3(p.n_gate / p.gate_groups, p.gate_groups), kThreads, s, p);
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
cudaError_t gather(CacheParams p, cudaStream_t s) {
  constexpr int R = RowLanes<D>::kRows;
  const int blocks = plan(p, p.log_gate_out != nullptr, (p.hkv + R - 1) / R, 152 * kGatherBlocks);
  p.log2_step = log2_step<R>(p, 152 * kGatherBlocks);
  cache_gather_kernel<D, FMT><<<blocks, kThreads, 0, s>>>(p);
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

cudaError_t launch_cache_append(const CacheParams& p, const RopeParams* rope, cudaStream_t s) {
  switch (p.d) {
    case 64: return append<64>(p, rope, s);
    case 128: return append<128>(p, rope, s);
    case 256: return append<256>(p, rope, s);
    default: return append<512>(p, rope, s);
  }
}

cudaError_t launch_cache_gather(const CacheParams& p, cudaStream_t s) {
  switch (p.d) {
    case 64: return gather<64>(p, s);
    case 128: return gather<128>(p, s);
    case 256: return gather<256>(p, s);
    default: return gather<512>(p, s);
  }
}

}  // namespace gcs
