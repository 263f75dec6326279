// Gathered attention weights (see cache_weights.cu for what is computed) with many query rows to a key:
// the chunks of a prefill, the last rows of a prompt.  Bound by the exponentials, of which each pair
// of a row and a key takes one in each of two kernels, beside d multiply-adds on the tensor cores.
//
//   sums kernel      S = Q K^T: rows on the accumulator's lanes, so a row's maximum and sum stay in
//                    its thread; K tiles stream by.  One partial (max, sum) a row and segment.
//   rows kernel      joins a row's partials and the sink: b = -lse (log2 units), beside its gate.
//   weights kernel   S^T = K Q^T: keys on the lanes, so a key's weight, the sum over rows of
//                    2^(scale s + b), stays in its thread too; the query tiles stream by.
// Neither kernel moves data between threads until the four groups of lanes that share a row or a key join
// their parts at its end, and nothing but (max, sum) leaves the SM.
//
// Both kernels are one engine: NA resident operand tiles of 128 rows x d (two, one at d 512) in tensor
// memory, streamed tiles of 128 rows x d in a shared-memory ring of 64-dim stages, and accumulators of
// 128 x 128 in turn.  With the resident side out of tensor memory an MMA reads 64 bytes a cycle of shared
// memory; out of shared memory it would be the 128 there are, and the vectors' reads would wait for it.
// A query tile is floor(128 / G) tokens x the G query heads of a kv head; the rows
// left over are zero.  With an fp8 cache the operands are f16 (codes are exact in it; the queries are
// rounded to it by a kernel of their own for the streamed side), with a bf16 one bf16.
//
// Warp roles (640 threads, 768 where codes are converted):
//   warp 0        streamed tiles by tensor copies (bf16 keys, queries)
//   warp 1        tcgen05 issuer
//   warps 2-3     per-column vectors of the streamed tile (scales or b, gates, last visible keys)
//   warps 4-19    sums or weights: four groups of 128 lanes, one accumulator at a time each
//   warps 20-23   sums kernel over an fp8 cache: e4m3 -> f16 stages, straight from memory
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "launch.h"
#include "rows.cuh"
#include "sm103_ptx.cuh"

namespace gcs {
namespace {

// 4 warps, 16 of the accumulators and, where codes are converted, 4 more
constexpr int kEpiWarps = 16;
template <bool CONVERT>
constexpr int kThreadsOf = (4 + kEpiWarps + (CONVERT ? 4 : 0)) * 32;
constexpr int kTile = 128;
constexpr int kStage = 16384;  // 128 rows x 64 dims of 16 bits
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxGates = 16;          // heads of a kv head, with gates
constexpr int kGateRow = kTile + 4;    // floats of a head's gates: rows 16 bytes apart in the banks

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ void record_bad(int* status) { atomicCAS(status, kDevOk, kDevInvalidArg); }
__device__ __forceinline__ float2 add2(const float2& a, const float2& b) { return fma2(a, both(1.f), b); }

__device__ __forceinline__ void e4m3x4_to_f16x2x2(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n"
      " cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  return pack_f16x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// 16 e4m3 codes to the two 16-byte units 2 u and 2 u + 1 of row r of a swizzled stage
__device__ __forceinline__ void put_codes(uint8_t* stage, int r, int u, uint4 v) {
  uint32_t w[8];
  e4m3x4_to_f16x2x2(v.x, w[0], w[1]);
  e4m3x4_to_f16x2x2(v.y, w[2], w[3]);
  e4m3x4_to_f16x2x2(v.z, w[4], w[5]);
  e4m3x4_to_f16x2x2(v.w, w[6], w[7]);
  *reinterpret_cast<uint4*>(stage + sw128_offset(r, 2 * u)) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(stage + sw128_offset(r, 2 * u + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int NCH>
struct Cfg {
  static constexpr int NA = NCH == 8 ? 1 : 2;               // resident tiles
  static constexpr int A_COLS = NCH * 32;                   // tensor memory columns of one
  static constexpr int SLOTS = NCH <= 2 ? 3 : 2;            // accumulators
  static_assert(NA * A_COLS + SLOTS * kTile <= 512, "tensor memory");
  static constexpr int NST = NCH == 1 ? 6 : 8;              // stages of the ring
  static constexpr int OFF_RING = 0;
  static constexpr int NAUX = 4;                            // vectors of as many streamed tiles
  static constexpr int OFF_AUX = OFF_RING + NST * kStage;
  static constexpr int VECS = 3 * kTile * 4;                // 3 x [128]
  static constexpr int AUX = VECS + kMaxGates * kGateRow * 4;
  static constexpr int OFF_BAR = OFF_AUX + NAUX * AUX;
  static constexpr int OFF_MISC = OFF_BAR + (2 * NST + 8 + 2 * NAUX + 2) * 8;
  static constexpr int SMEM = OFF_MISC + 32 + 1024;
  static_assert(SMEM <= 226 * 1024, "shared memory budget");
};

struct Request {
  int q0, ql, L;
  bool ok;
};
__device__ __forceinline__ Request request(const WeightsParams& p, int r) {
  Request x;
  x.q0 = __ldg(p.cu_q + r);
  const int q1 = __ldg(p.cu_q + r + 1);
  x.ql = q1 - x.q0;
  x.L = __ldg(p.seq_lens + r);
  x.ok = !(x.q0 < 0 || q1 < x.q0 || q1 > p.total_q || x.ql > p.max_q_len || x.L < x.ql || x.L > p.max_seq_len);
  return x;
}
// Block of a cached position, -1 (recorded) outside the cache.
__device__ __forceinline__ int block_of(const WeightsParams& p, const int32_t* table, int pos) {
  const int blk = __ldg(table + (pos >> p.log2_block));
  if (blk >= 0 && blk < p.num_blocks) return blk;
  record_bad(p.status);
  return -1;
}

// WRITE false: the sums kernel, true: the weights kernel.  NCH: d / 64.
template <bool BF16, int NCH, bool WRITE>
__global__ void __launch_bounds__(kThreadsOf<!BF16 && !WRITE>, 1)
    weights_long_kernel(const __grid_constant__ CUtensorMap tm, const WeightsParams p) {
  using C = Cfg<NCH>;
  constexpr int NA = C::NA, NST = C::NST, kThreads = kThreadsOf<!BF16 && !WRITE>;
  // Each kernel of a call may run beside the one before it: the sums need nothing of the queries' copy, the
  // weights wait for the rows' constants (behind the sums) once their keys are in place.
  WaitAtEnd at_end;
  grid_release();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align_1k(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.y, r = blockIdx.z;
  const Request rq = request(p, r);
  if (!rq.ok) {
    if (threadIdx.x == 0) record_bad(p.status);
    return;
  }
  const int ql = rq.ql, L = rq.L, G = p.group, W = p.window;
  const int ntok = kTile / G, nrow = ntok * G;  // tokens and rows of a query tile
  const int32_t* table = p.block_table + (size_t)r * p.max_blocks;
  const bool gates = p.g_cache != nullptr;
  const float sl2 = p.scale * kLog2e;
  const float kst = p.format == kCachePerTensor ? __ldg(p.k_scale) : 1.f;

  // resident rows: tokens a0 .. (sums) or keys a0 .. (weights); streamed tiles b_lo .. b_hi, tile i
  // from token i ntok or key key0 + 128 i on
  int a0, b_lo, b_hi, key0 = 0, seg = 0, left = 0;  // left: first key whose weight is written
  if (!WRITE) {
    seg = blockIdx.x % p.segs;
    a0 = blockIdx.x / p.segs * NA * ntok;
    key0 = seg * p.seg_len;
    if (a0 >= ql || key0 >= L) return;
    const int see = L - ql + min(a0 + NA * ntok, ql) - 1;  // last key that any of the rows sees
    const int from = W > 0 ? max(0, L - ql + a0 - W + 1) : 0;
    const int key1 = min(min(key0 + p.seg_len, L), see + 1);
    b_lo = max(0, from - key0) / kTile;
    b_hi = key1 > key0 ? (key1 - key0 - 1) / kTile : -1;
  } else {
    a0 = blockIdx.x * NA * kTile;
    left = p.first_lens ? __ldg(p.first_lens + r) : 0;
    if (a0 >= L || (long long)a0 + NA * kTile <= left) return;
    const int last = min(a0 + NA * kTile, L) - 1;  // last of the keys
    // token t sees key j iff j <= L - ql + t, and L - ql + t < j + W
    b_lo = max(0, a0 - (L - ql)) / ntok;
    b_hi = ql > 0 ? (W > 0 ? (int)min((long long)ql - 1, (long long)last + W - 1 - (L - ql)) : ql - 1) : -1;
    b_hi = b_hi < 0 ? -1 : b_hi / ntok;
  }
  const int nt = max(0, b_hi - b_lo + 1);
  // resident tiles with anything in them
  const int nx = NA == 2 && (WRITE ? a0 + kTile < L : a0 + ntok < ql) ? 2 : 1;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;               // [NST]
  uint64_t* empty = bars + NST;        // [NST]
  uint64_t* s_full = bars + 2 * NST;   // [4 groups] the group's next product (a group sees every phase of its
                                       // barrier, which a barrier of a slot would not give it)
  uint64_t* s_empty = s_full + 4;      // [SLOTS] accumulators
  uint64_t* aux_full = s_full + 8;     // [NAUX]
  uint64_t* aux_empty = aux_full + C::NAUX;
  uint64_t* drain = aux_empty + C::NAUX;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  uint32_t* bad_pages = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 8);  // [NAUX] pages of a key tile that are not there
  const Abort ab{abort_flag, p.status};
  constexpr bool kCopied = BF16 || WRITE;  // the streamed tiles come by tensor copies
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], kCopied ? 1 : 4);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&s_full[i], 1);
    for (int i = 0; i < C::SLOTS; ++i) mbar_init(&s_empty[i], 4);
    for (int i = 0; i < C::NAUX; ++i) {
      mbar_init(&aux_full[i], !WRITE && gates ? 33 : 1);  // with gates each lane's copies, too
      mbar_init(&aux_empty[i], 4 * nx);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t kAccCol = NA * C::A_COLS;  // first column of the accumulators
  if (warp >= 4 && warp < 4 + kEpiWarps) {
    // the resident rows, 16-bit, one row a lane, two dims a column; a row is shared out over the
    // warps of its lanes
    constexpr int kParts = NA == 2 ? 2 : 4;
    const int grp = (warp - 4) >> 2, x = NA == 2 ? grp & 1 : 0, part = NA == 2 ? grp >> 1 : grp;
    const int rr = (warp & 3) * 32 + lane;
    const uint4* src = nullptr;
    if (!WRITE) {
      const int t = a0 + x * ntok + rr / G;
      if (rr < nrow && t < ql)
        src = reinterpret_cast<const uint4*>(p.q + (size_t)(rq.q0 + t) * p.q_ts + (size_t)(kvh * G + rr % G) * p.q_hs);
    } else {
      const int pos = a0 + x * kTile + rr, blk = pos < L ? block_of(p, table, pos) : -1;
      if (blk >= 0)
        src = reinterpret_cast<const uint4*>(p.k_cache + (size_t)blk * p.kv_bs + (size_t)kvh * p.kv_hs +
                                             (size_t)(pos & (p.block_size - 1)) * p.kv_ss);
    }
    const uint32_t col0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + x * C::A_COLS;
    constexpr int kWords = C::A_COLS / kParts;      // columns of a thread's share: 16 .. 64
    constexpr bool kCodes = !BF16 && WRITE;
    constexpr int kLoads = kWords / (kCodes ? 8 : 4);
    // All on their way at once.  Neighbouring lanes read neighbouring pieces of a row and change them in the ring's
    // place (not in use yet; the pieces permuted by the row, so that both ways spread over the banks): with a row a
    // lane each load touches 32 lines (8 x 33 rows of 256 dims 275 us, so 251; two pieces a row: 286, 293).
    uint4 v[kLoads];
    if constexpr (kLoads == 2) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) v[i] = src ? __ldg(src + part * kLoads + i) : make_uint4(0, 0, 0, 0);
    } else {
      static_assert(kEpiWarps * 32 * kLoads * 16 <= NST * kStage, "the ring holds the rows");
      uint8_t* mine = smem + C::OFF_RING + (warp - 4) * 32 * kLoads * 16;
      constexpr int kPerm = kLoads < 8 ? kLoads : 8;
      auto place = [&](int row, int piece) {
        return reinterpret_cast<uint4*>(mine + (row * kLoads + (piece ^ (row * kPerm / 8 & (kPerm - 1)))) * 16);
      };
      const int piece = lane % kLoads;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint4* from = reinterpret_cast<const uint4*>(__shfl_sync(
            0xffffffffu, reinterpret_cast<unsigned long long>(src), i * (32 / kLoads) + lane / kLoads));
        v[i] = from ? __ldg(from + part * kLoads + piece) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) *place(i * (32 / kLoads) + lane / kLoads, piece) = v[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kLoads; ++i) v[i] = *place(lane, i);
    }
#pragma unroll
    for (int c = 0; c < kWords; c += 16) {  // 32 dims
      uint32_t w[16];
      if (!kCodes) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 x4 = v[c / 4 + u];
          w[4 * u] = x4.x, w[4 * u + 1] = x4.y, w[4 * u + 2] = x4.z, w[4 * u + 3] = x4.w;
        }
        if (!BF16) {
#pragma unroll
          for (int u = 0; u < 16; ++u) w[u] = bf16x2_to_f16x2(w[u]);
        }
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint4 x4 = v[c / 8 + u];
          e4m3x4_to_f16x2x2(x4.x, w[8 * u], w[8 * u + 1]);
          e4m3x4_to_f16x2x2(x4.y, w[8 * u + 2], w[8 * u + 3]);
          e4m3x4_to_f16x2x2(x4.z, w[8 * u + 4], w[8 * u + 5]);
          e4m3x4_to_f16x2x2(x4.w, w[8 * u + 6], w[8 * u + 7]);
        }
      }
      tmem_st16(col0 + part * kWords + c, w);
    }
    tmem_st_wait();
    fence_proxy_async_smem();
  }
  if (WRITE && nrow < kTile) {  // rows of the streamed tiles that no copy writes
    __syncthreads();
    for (int i = threadIdx.x; i < NST * (kTile - nrow) * 8; i += kThreads) {
      const int st = i / ((kTile - nrow) * 8), k = i % ((kTile - nrow) * 8);
      *reinterpret_cast<uint4*>(smem + C::OFF_RING + st * kStage + nrow * 128 + k * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  if (WRITE) grid_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  auto ring_next = [&](uint32_t& stage, uint32_t& phase) {
    if (++stage == NST) {
      stage = 0;
      phase ^= 1;
    }
  };

  if (warp == 0) {
    if (kCopied) {
      if (lane == 0) prefetch_tmap(&tm);
      uint32_t stage = 0, phase = 0;
      for (int n = 0; n < nt; ++n) {
        const int b = b_lo + n;
        int blk = -1, cy = 0, cz = 0, tok = 0;
        uint32_t bytes = 64 * 2 * nrow;
        if (WRITE) {
          tok = rq.q0 + b * ntok;
        } else {  // lane = page
          const int pos = key0 + b * kTile + lane * 16;
          if (lane < 8 && pos < L) blk = block_of(p, table, pos);
          const int sub = pos & (p.block_size - 1);
          cy = p.kv_head_inner ? kvh : sub;
          cz = p.kv_head_inner ? sub : kvh;
          bytes = __popc(__ballot_sync(0xffffffffu, blk >= 0)) * 2048;
        }
        bool okl = true;
        for (int c = 0; c < NCH && okl; ++c) {
          okl = wait_bar(&empty[stage], phase ^ 1, ab);
          okl = __all_sync(0xffffffffu, okl);
          if (!okl) break;
          if (lane == 0) mbar_expect_tx(&full[stage], bytes);
          __syncwarp();
          uint8_t* st = smem + C::OFF_RING + stage * kStage;
          if (WRITE) {
            if (lane == 0) tma_load_3d(st, &tm, &full[stage], 64 * c, kvh * G, tok);
          } else if (blk >= 0) {
            tma_load_4d(st + lane * 2048, &tm, &full[stage], 64 * c, cy, cz, blk);
          }
          ring_next(stage, phase);
        }
        if (!okl) break;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t id = BF16 ? idesc_bf16(kTile, kTile, false, false) : idesc_f16(kTile, kTile, false, false);
      const uint64_t dB = sdesc_sw128(smem_u32(smem + C::OFF_RING), 16, 1024);
      constexpr uint32_t kSt16 = kStage >> 4;
      uint32_t stage = 0, phase = 0, slot = 0, slot_phase = 0;
      bool ok = true;
      auto products = [&](auto tiles) {
        constexpr int kX = decltype(tiles)::value;
        for (int n = 0; n < nt && ok; ++n) {
          const uint32_t first = stage;
#pragma unroll
          for (int x = 0; x < kX; ++x) {  // a tile's stages are held until its last product
            if (ok) ok = wait_bar(&s_empty[slot], slot_phase ^ 1, ab);
            uint32_t st = first;
            for (int c = 0; c < NCH && ok; ++c) {
              if (x == 0) {
                ok = wait_bar(&full[stage], phase, ab);
                if (!ok) break;
                ring_next(stage, phase);
              }
              tc_fence_after();
              const uint64_t b = dB + st * kSt16;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts(tmem + kAccCol + slot * kTile, tmem + x * C::A_COLS + c * 32 + k * 8, b + 2 * k, id, (c | k) != 0);
              if (x == kX - 1) mma_commit(&empty[st]);
              st = st + 1 == NST ? 0 : st + 1;
            }
            if (ok) mma_commit(&s_full[(n * kX + x) & 3]);
            if (++slot == C::SLOTS) {
              slot = 0;
              slot_phase ^= 1;
            }
          }
        }
      };
      if (nx == NA) products(std::integral_constant<int, NA>());
      else products(std::integral_constant<int, 1>());
      if (!ok) {
        mma_commit(drain);
        mbar_wait(drain, 0, nullptr);
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------- per-column vectors
    // The two warps take the tiles in turn; what a tile needs from memory is on its way while the one before
    // it is written.
    if constexpr (WRITE) {  // (b, own gate) and the last visible key of a row, a lane rows lane + 32 k
      float2 next[4];
      int next_see[4];
      auto fetch = [&](int n) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = lane + 32 * k, t = (b_lo + n) * ntok + i / G;
          next_see[k] = -1;
          next[k] = make_float2(neg_inf(), 0.f);
          if (n < nt && i < nrow && t < ql) {
            // written while this kernel may already run: not by the read-only path
            next[k] = p.rows[(size_t)(rq.q0 + t) * p.hq + kvh * G + i % G];
            next_see[k] = L - ql + t;
          }
        }
      };
      fetch(warp - 2);
      for (int n = warp - 2; n < nt; n += 2) {
        const int a = n % C::NAUX;
        float2 v[4];
        int see[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = next[k], see[k] = next_see[k];
        fetch(n + 2);
        if (!wait_bar(&aux_empty[a], ((n / C::NAUX) & 1) ^ 1, ab)) break;
        float* ax = reinterpret_cast<float*>(smem + C::OFF_AUX + a * C::AUX);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = lane + 32 * k;
          ax[i] = v[k].x;
          ax[kTile + i] = v[k].y;
          reinterpret_cast<int*>(ax)[2 * kTile + i] = see[k];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&aux_full[a]);
      }
    } else {  // scales and gates of the keys, a lane four in a row (of one block)
      float4 next;
      int next_blk;
      auto fetch = [&](int n) {
        const int pos = key0 + (b_lo + n) * kTile + 4 * lane;
        next_blk = n < nt && pos < L ? block_of(p, table, pos) : -1;
        next = make_float4(kst, kst, kst, kst);
        if (next_blk >= 0 && p.format == kCachePerToken) {
          const float* src = p.k_scale + (((size_t)next_blk * p.hkv + kvh) << p.log2_block) + (pos & (p.block_size - 1));
          next = make_float4(__ldg(src), __ldg(src + 1), __ldg(src + 2), __ldg(src + 3));
        }
      };
      fetch(warp - 2);
      for (int n = warp - 2; n < nt; n += 2) {
        const int a = n % C::NAUX, pos = key0 + (b_lo + n) * kTile + 4 * lane, blk = next_blk;
        const float4 v = next;
        fetch(n + 2);
        if (!wait_bar(&aux_empty[a], ((n / C::NAUX) & 1) ^ 1, ab)) break;
        float* ax = reinterpret_cast<float*>(smem + C::OFF_AUX + a * C::AUX);
        if (gates) {  // no lane waits for its copies: they arrive at the barrier by themselves
          const float* src = p.g_cache + (((size_t)max(blk, 0) * p.hq + kvh * G) << p.log2_block) +
                             (pos & (p.block_size - 1));
          for (int h = 0; h < G; ++h)
            copy_async16(ax + 3 * kTile + h * kGateRow + 4 * lane, src + ((size_t)h << p.log2_block), blk >= 0);
          copies_arrive(&aux_full[a]);
        }
        *reinterpret_cast<float4*>(ax + 4 * lane) = make_float4(v.x * sl2, v.y * sl2, v.z * sl2, v.w * sl2);
        const uint32_t bad = __reduce_or_sync(0xffffffffu, blk < 0 && pos < L ? 1u << (lane >> 2) : 0u);
        if (lane == 0) bad_pages[a] = bad;
        __syncwarp();
        if (lane == 0) mbar_arrive(&aux_full[a]);
      }
      copy_commit();
      copy_wait<0>();
    }
    __syncwarp();
  } else if (warp < 4 + kEpiWarps) {
    // ---------------------------------------------------------- sums or weights
    // Four groups of 128 lanes take the products in turn: while one waits for its product or its registers,
    // others keep the exponentials going.  The code between two waits has no branch: with one for the mask every
    // four columns the weights kernel took 1.48 ms (4 x 1024 rows over up to 32K keys, 64 / 4 heads of 128,
    // bf16), without 1.03; its exponentials alone are 0.55, its products 0.55.
    const int grp = (warp - 4) >> 2, quarter = warp & 3;
    const int rr = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int x = nx == 2 ? grp & 1 : 0;  // its resident tile
    // sums: the row's token and last visible key; weights: the key and its constants
    const int t = a0 + x * ntok + rr / G, head = rr % G;
    const bool row_ok = rr < nrow && t < ql;
    const int pos = WRITE ? a0 + x * kTile + rr : L - ql + min(t, ql - 1);
    float gi = 0.f, ks = 0.f;
    int blk = -1, slot_k = 0;
    if (WRITE) {
      blk = pos < L && pos >= left ? block_of(p, table, pos) : -1;
      if (blk >= 0) {
        slot_k = pos & (p.block_size - 1);
        ks = kst * sl2;
        if (p.format == kCachePerToken)
          ks = __ldg(p.k_scale + (((size_t)blk * p.hkv + kvh) << p.log2_block) + slot_k) * sl2;
      }
    } else if (gates && row_ok) {
      const int b = block_of(p, table, pos);
      if (b >= 0)
        gi = __ldg(p.g_cache + (((size_t)b * p.hq + kvh * G + head) << p.log2_block) + (pos & (p.block_size - 1)));
    }
    float m = neg_inf();
    float2 acc[2];  // sums, or the weight
    acc[0] = acc[1] = make_float2(0.f, 0.f);
    bool ok = true;

    auto columns = [&](auto with_gates) {
      constexpr bool kGates = decltype(with_gates)::value;
      float gk[kGates && WRITE ? kMaxGates : 1];
      [[maybe_unused]] const bool repeat = (kMaxGates % G) == 0;  // column i has head i % 16 % G
      if (kGates && WRITE) {
#pragma unroll
        for (int h = 0; h < kMaxGates; ++h)
          gk[h] = blk >= 0 ? __ldg(p.g_cache + (((size_t)blk * p.hq + kvh * G + h % G) << p.log2_block) + slot_k) : 0.f;
      }
      for (int u = grp; u < nt * nx; u += 4) {  // streamed tile n with resident tile x
        const int n = nx == 2 ? u >> 1 : u, a = n % C::NAUX;
        const int slot = u % C::SLOTS;
        ok = wait_bar(&aux_full[a], (n / C::NAUX) & 1, ab) && wait_bar(&s_full[grp], (u >> 2) & 1, ab);
        if (!ok) break;
        tc_fence_after();
        const float* ax = reinterpret_cast<const float*>(smem + C::OFF_AUX + a * C::AUX);
        const uint32_t tS = tmem + lane_off + kAccCol + slot * kTile;
        if constexpr (!WRITE) {
          const int j0 = key0 + (b_lo + n) * kTile;
          const uint32_t bad = bad_pages[a];
          const int first_t = a0 + x * ntok, last_t = min(first_t + ntok, ql) - 1;
          const bool need_mask = j0 + kTile - 1 > L - ql + first_t || bad != 0 || (W > 0 && j0 <= L - ql + last_t - W);
          const float4* g4 = reinterpret_cast<const float4*>(ax + 3 * kTile + head * kGateRow);
          const float4* ks4 = reinterpret_cast<const float4*>(ax);
          // four scores (log2 units) and `base` at a time of 32 columns into f
          auto scores = [&](auto masked, int cc, float base, auto f) {
            constexpr bool kMask = decltype(masked)::value;
            uint32_t sv[32];
            tmem_ld32(tS + cc * 32, sv);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float4 k4 = ks4[cc * 8 + q];
              float2 va = both(base), vb = both(base);
              if (kGates) {
                const float4 g = g4[cc * 8 + q];
                va = fma2(make_float2(gi - g.x, gi - g.y), both(kLog2e), va);
                vb = fma2(make_float2(gi - g.z, gi - g.w), both(kLog2e), vb);
              }
              va = fma2(make_float2(__uint_as_float(sv[4 * q]), __uint_as_float(sv[4 * q + 1])),
                        make_float2(k4.x, k4.y), va);
              vb = fma2(make_float2(__uint_as_float(sv[4 * q + 2]), __uint_as_float(sv[4 * q + 3])),
                        make_float2(k4.z, k4.w), vb);
              if (kMask) {
                const int j = j0 + cc * 32 + 4 * q;
                const bool off = bad >> (cc * 2 + q / 4) & 1;
                va.x = off || j > pos || (W > 0 && j <= pos - W) ? neg_inf() : va.x;
                va.y = off || j + 1 > pos || (W > 0 && j + 1 <= pos - W) ? neg_inf() : va.y;
                vb.x = off || j + 2 > pos || (W > 0 && j + 2 <= pos - W) ? neg_inf() : vb.x;
                vb.y = off || j + 3 > pos || (W > 0 && j + 3 <= pos - W) ? neg_inf() : vb.y;
              }
              f(va, vb);
            }
          };
          float2 s0 = make_float2(0.f, 0.f), s1 = s0;
          auto add = [&](const float2& va, const float2& vb) {
            s0.x += ex2(va.x);
            s0.y += ex2(va.y);
            s1.x += ex2(vb.x);
            s1.y += ex2(vb.y);
          };
          // One straight run of code for each case: a branch within it would part the exponentials.  The
          // reference m keeps them below 2^60 or so: as long as a tile's sum says that, no maximum is looked for.
          if (need_mask) {
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) scores(std::true_type(), cc, m == neg_inf() ? 0.f : -m, add);
          } else {
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) scores(std::false_type(), cc, m == neg_inf() ? 0.f : -m, add);
          }
          float2 s = add2(s0, s1);
          if (__any_sync(0xffffffffu, m == neg_inf() || !(s.x + s.y < 0x1p60f))) {
            // the first keys, or far larger ones (or a NaN): the reference becomes the maximum
            float mx = m;
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc)
              scores(std::true_type(), cc, 0.f, [&](const float2& va, const float2& vb) {
                mx = fmaxf(fmaxf(mx, fmaxf(va.x, va.y)), fmaxf(vb.x, vb.y));
              });
            const float f = m == neg_inf() ? 0.f : ex2(m - mx);
            acc[0] = mul2(acc[0], both(f));
            acc[1] = mul2(acc[1], both(f));
            m = mx;
            s0 = s1 = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc) scores(std::true_type(), cc, m == neg_inf() ? 0.f : -m, add);
            s = add2(s0, s1);
          }
          acc[0] = add2(acc[0], s);
        } else {
          const int t0 = (b_lo + n) * ntok;
          const int j_lo = a0 + x * kTile, j_hi = j_lo + kTile - 1;
          const bool need_mask = t0 + ntok > ql || j_hi > L - ql + t0 || (W > 0 && j_lo <= L - ql + t0 + ntok - 1 - W);
          const float4* b4 = reinterpret_cast<const float4*>(ax);
          const float4* gi4 = reinterpret_cast<const float4*>(ax + kTile);
          const int* see = reinterpret_cast<const int*>(ax) + 2 * kTile;
          auto tile = [&](auto masked, auto columns32) {
            constexpr bool kMask = decltype(masked)::value;
#pragma unroll
            for (int cc = 0; cc < decltype(columns32)::value; ++cc) {
              uint32_t sv[32];
              tmem_ld32(tS + cc * 32, sv);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                float4 b = b4[cc * 8 + q];
                if (kGates) {
                  const float4 g = gi4[cc * 8 + q];
                  float k4[4];
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    k4[e] = gk[(4 * q + e) % kMaxGates];
                    if (!repeat) {  // groups that 16 is no multiple of
                      const int h = (cc * 32 + 4 * q + e) % G;
#pragma unroll
                      for (int w = 0; w < kMaxGates; ++w) k4[e] = h == w ? gk[w] : k4[e];
                    }
                  }
                  b.x = fmaf(g.x - k4[0], kLog2e, b.x);
                  b.y = fmaf(g.y - k4[1], kLog2e, b.y);
                  b.z = fmaf(g.z - k4[2], kLog2e, b.z);
                  b.w = fmaf(g.w - k4[3], kLog2e, b.w);
                }
                const uint32_t* s4 = sv + 4 * q;
                float2 va = fma2(make_float2(__uint_as_float(s4[0]), __uint_as_float(s4[1])), both(ks),
                                 make_float2(b.x, b.y));
                float2 vb = fma2(make_float2(__uint_as_float(s4[2]), __uint_as_float(s4[3])), both(ks),
                                 make_float2(b.z, b.w));
                if (kMask) {
                  const int4 lk = *reinterpret_cast<const int4*>(see + cc * 32 + 4 * q);
                  va.x = pos > lk.x || (W > 0 && pos <= lk.x - W) ? neg_inf() : va.x;
                  va.y = pos > lk.y || (W > 0 && pos <= lk.y - W) ? neg_inf() : va.y;
                  vb.x = pos > lk.z || (W > 0 && pos <= lk.z - W) ? neg_inf() : vb.x;
                  vb.y = pos > lk.w || (W > 0 && pos <= lk.w - W) ? neg_inf() : vb.y;
                }
                acc[0].x += ex2(va.x);
                acc[0].y += ex2(va.y);
                acc[1].x += ex2(vb.x);
                acc[1].y += ex2(vb.y);
              }
            }
          };
          using All = std::integral_constant<int, 4>;
          if (!need_mask) tile(std::false_type(), All());
          else if ((ql - t0) * G > 32) tile(std::true_type(), All());
          else tile(std::true_type(), std::integral_constant<int, 1>());  // a last tile of few rows: 211 us, so 203
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s_empty[slot]);
          mbar_arrive(&aux_empty[a]);
        }
      }
    };
    if (gates) columns(std::true_type());
    else columns(std::false_type());
    const float2 s2 = add2(acc[0], acc[1]);
    float sum = s2.x + s2.y;
    // the other groups' parts of the same rows, in a fixed order, by shared memory (the ring is done with)
    const int parts = 4 / nx, part = nx == 2 ? grp >> 1 : grp;
    float2* others = reinterpret_cast<float2*>(smem + C::OFF_RING) + x * 2 * kTile;
    asm volatile("bar.sync 1, 512;" ::: "memory");
    if (part > 0) others[part * kTile + rr] = make_float2(m, sum);
    asm volatile("bar.sync 1, 512;" ::: "memory");
    if (part == 0 && !*abort_flag) {
      for (int k = 1; k < parts; ++k) {
        const float2 o = others[k * kTile + rr];
        if (WRITE) {
          sum += o.y;
        } else {
          const float M = fmaxf(m, o.x);
          sum = (m == neg_inf() ? 0.f : sum * ex2(m - M)) + (o.x == neg_inf() ? 0.f : o.y * ex2(o.x - M));
          m = M;
        }
      }
      if (!WRITE) {
        if (row_ok)
          p.part[((size_t)seg * p.total_q + rq.q0 + t) * p.hq + kvh * G + head] = make_float2(m, sum);
      } else if (blk >= 0) {
        float* w = p.w_cache + (((size_t)blk * p.hkv + kvh) << p.log2_block) + slot_k;
        *w = p.decay != 0.f && pos < L - ql ? fmaf(p.decay, *w, sum) : sum;
      }
    }
  } else if (!kCopied) {
    // ---------------------------------------------------------- e4m3 -> f16 stages (warps 20-23)
    // thread c takes the 16-byte piece c & 3 of keys 32 i + c / 4; two chunks are on their way
    // while one is converted
    const int c = threadIdx.x - (4 + kEpiWarps) * 32, piece = c & 3, row = c >> 2;
    const int total = nt * NCH;
    uint4 ring[2][4];
    // this thread's keys of the tile that is fetched, and of the one after it (looked up a tile ahead)
    const uint8_t *src[4], *src_next[4];
    auto look_up = [&](int n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int pos = key0 + (b_lo + n) * kTile + 32 * i + row;
        src_next[i] = nullptr;
        if (n < nt && pos < L) {
          const int blk = __ldg(table + (pos >> p.log2_block));  // the vectors' warps record it
          if (blk >= 0 && blk < p.num_blocks)
            src_next[i] = p.k_cache + (size_t)blk * p.kv_bs + (size_t)kvh * p.kv_hs +
                          (size_t)(pos & (p.block_size - 1)) * p.kv_ss + piece * 16;
        }
      }
    };
    look_up(0);
    auto fetch = [&](int q, uint4 (&d)[4]) {
      if (q % NCH == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) src[i] = src_next[i];
        look_up(q / NCH + 1);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[i] = src[i] ? __ldg(reinterpret_cast<const uint4*>(src[i] + (q % NCH) * 64)) : make_uint4(0, 0, 0, 0);
    };
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    auto store = [&](const uint4 (&d)[4]) {
      ok = wait_bar(&empty[stage], phase ^ 1, ab);
      if (!ok) return;
      uint8_t* st = smem + C::OFF_RING + stage * kStage;
#pragma unroll
      for (int i = 0; i < 4; ++i) put_codes(st, 32 * i + row, piece, d[i]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[stage]);
      ring_next(stage, phase);
    };
    fetch(0, ring[0]);
    fetch(1, ring[1]);
    for (int q = 0; q < total && ok; q += 2) {
      store(ring[0]);
      fetch(q + 2, ring[0]);
      if (!ok || q + 1 >= total) break;
      store(ring[1]);
      fetch(q + 3, ring[1]);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {  // copies in flight land before the shared memory is given back
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// (b, own gate) of every query row: b = -log2 of its sum of exponentials, joined over the segments it
// sees.
__global__ void __launch_bounds__(256) weights_rows_kernel(const WeightsParams p) {
  WaitAtEnd at_end;
  grid_release();
  const int r = blockIdx.y;
  const Request rq = request(p, r);
  if (!rq.ok) return;
  grid_wait();  // the sums
  const long long n = (long long)rq.ql * p.hq;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const int t = (int)(i / p.hq), h = (int)(i % p.hq), pos = rq.L - rq.ql + t;
    const size_t at = (size_t)(rq.q0 + t) * p.hq + h;
    float b = neg_inf();
    if (p.lse) {
      const float lse = __ldg(p.lse + (size_t)h * p.total_q + rq.q0 + t);
      if (lse != neg_inf()) b = -lse * kLog2e;
    } else {
      float m = neg_inf(), l = 0.f;
      auto join = [&](float m2, float l2) {
        const float M = fmaxf(m, m2);
        l = (m == neg_inf() ? 0.f : l * ex2(m - M)) + (m2 == neg_inf() ? 0.f : l2 * ex2(m2 - M));
        m = M;
      };
      const int first = p.window > 0 ? max(0, pos - p.window + 1) / p.seg_len : 0;
      const int last = pos / p.seg_len;
      for (int s = first; s <= last; s += 8) {  // eight on their way at once
        float2 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = s + j <= last ? p.part[(size_t)(s + j) * p.total_q * p.hq + at] : make_float2(neg_inf(), 0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) join(v[j].x, v[j].y);
      }
      if (p.sink) join(__ldg(p.sink + h) * kLog2e, 1.f);
      if (l != 0.f) b = -(m + log2f(l));  // 0: a row whose every key lies outside the cache
    }
    float g = 0.f;
    if (p.g_cache) {
      const int blk = block_of(p, p.block_table + (size_t)r * p.max_blocks, pos);
      if (blk >= 0) g = __ldg(p.g_cache + (((size_t)blk * p.hq + h) << p.log2_block) + (pos & (p.block_size - 1)));
    }
    p.rows[at] = make_float2(b, p.lse && b == neg_inf() ? 0.f : g);
  }
}

// The queries as the weights kernel streams them, [total_q, hq, d]: in f16 for an fp8 cache, and with given sums
// zeros for a row without one (-inf), which adds nothing whatever its elements are.  (Masked by the tile
// instead, over a bf16 cache 4 x 1024 rows took 1864 us and 8 x 33 of 256 dims 286, unmasked 1800 and 266.)
template <bool BF16>
__global__ void __launch_bounds__(256) queries_kernel(const WeightsParams p) {
  grid_release();
  const int units = p.d / 8;
  const long long n = (long long)p.total_q * p.hq * units;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const long long row = i / units, t = row / p.hq, h = row % p.hq;
    uint4 v = __ldg(reinterpret_cast<const uint4*>(p.q + t * p.q_ts + h * p.q_hs) + i % units);
    if (p.lse && __ldg(p.lse + h * p.total_q + t) == neg_inf()) v = make_uint4(0, 0, 0, 0);
    if (!BF16) v = make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
    reinterpret_cast<uint4*>(p.q16)[i] = v;
  }
}

template <bool BF16, int NCH, bool WRITE>
cudaError_t launch_t(const WeightsParams& p, const CUtensorMap& map, bool beside, cudaStream_t s) {
  using C = Cfg<NCH>;
  auto kern = weights_long_kernel<BF16, NCH, WRITE>;
  cudaError_t e = allow_smem<weights_long_kernel<BF16, NCH, WRITE>>(C::SMEM);
  if (e != cudaSuccess) return e;
  const int per = WRITE ? C::NA * kTile : C::NA * (kTile / p.group);
  const int n = WRITE ? (p.max_seq_len + per - 1) / per : (p.max_q_len + per - 1) / per * p.segs;
  const dim3 grid(n, p.hkv, p.num_reqs);
  if (beside) return launch_beside(kern, grid, kThreadsOf<!BF16 && !WRITE>, C::SMEM, s, map, p);
  kern<<<grid, kThreadsOf<!BF16 && !WRITE>, C::SMEM, s>>>(map, p);
  return cudaGetLastError();
}
template <bool BF16, int NCH>
cudaError_t launch_d(const WeightsParams& p, const WeightsMaps& maps, cudaStream_t s) {
  cudaError_t e;
  bool beside = !BF16 || p.lse;  // behind the queries' kernel
  if (!p.lse && (e = launch_t<BF16, NCH, false>(p, maps.k, beside, s)) != cudaSuccess) return e;
  beside = beside || !p.lse;
  const long long rows = (long long)p.max_q_len * p.hq;
  const dim3 grid((unsigned)std::min(1024LL, (rows + 255) / 256), p.num_reqs);
  if (beside) {
    e = launch_beside(weights_rows_kernel, grid, 256, 0, s, p);
  } else {
    weights_rows_kernel<<<grid, 256, 0, s>>>(p);
    e = cudaGetLastError();
  }
  return e != cudaSuccess ? e : launch_t<BF16, NCH, true>(p, maps.q, true, s);
}
template <bool BF16>
cudaError_t launch_f(const WeightsParams& p, const WeightsMaps& maps, cudaStream_t s) {
  return p.d == 64 ? launch_d<BF16, 1>(p, maps, s) : p.d == 128 ? launch_d<BF16, 2>(p, maps, s)
         : p.d == 256 ? launch_d<BF16, 4>(p, maps, s) : launch_d<BF16, 8>(p, maps, s);
}

}  // namespace

// From more than 64 rows a (request, kv head) on, where the tensor cores' tiles are half full.
bool cache_weights_long(int max_q_len, int group, bool gates) {
  return (long long)max_q_len * group > 64 && group <= kTile && (!gates || group <= kMaxGates);
}

// Context segments of the sums kernel: blocks for about three an SM (contexts shorter than max_seq_len leave some
// of them empty; 8 x 33 rows of 256 dims: two 219 us, three 213, four 225), of 128 tokens or more.
int cache_weights_long_segment(int max_seq_len, int max_q_len, int group, int d, long long units, int sms) {
  const long long per = (long long)(d == 512 ? 1 : 2) * (kTile / group);
  const long long blocks = (max_q_len + per - 1) / per * units;
  const long long want = std::max(1LL, 3LL * sms / blocks);
  const long long tiles = (max_seq_len + kTile - 1) / kTile;
  return (int)((tiles + want - 1) / want * kTile);
}

cudaError_t launch_cache_weights_long(const WeightsParams& p, const WeightsMaps& maps, cudaStream_t s) {
  const bool bf16 = p.format == kCacheBf16;
  if (p.q16) {
    const long long units = (long long)p.total_q * p.hq * (p.d / 8);
    const unsigned blocks = (unsigned)std::min(4096LL, (units + 255) / 256);
    if (bf16) queries_kernel<true><<<blocks, 256, 0, s>>>(p);
    else queries_kernel<false><<<blocks, 256, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return bf16 ? launch_f<true>(p, maps, s) : launch_f<false>(p, maps, s);
}

}  // namespace gcs
