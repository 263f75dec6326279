// Decoding of requests that share a prefix of their contexts: the prefix's keys and values are read
// once for all query rows of a group of requests, each request's own tokens behind it by the split-K
// kernel of the paged decode, and a combine joins the two.
//
// softmax over prefix and own tokens = join of the two partial softmaxes (max m, sum l, sum of
// weighted values a):  M = max(m1, m2),  l = l1 e^(m1 - M) + l2 e^(m2 - M),  a likewise.
//
// prefix kernel: the query rows of a group are packed rows cu_q[first] .. cu_q[end], so a 128-row
// tile is 128 / G of them x the G query heads of one kv head, whichever requests they belong
// to; each row carries its own position (causal mask, window) and gate.  One CTA takes two
// tiles and one segment of the prefix, in 128-key tiles.  With R requests of 16 heads a kv head
// serves 16 R rows per key: from about 8 requests on the tensor cores and the exponentials bound it,
// not the cache's bytes.  Operands as in the chunked prefill: f16 from an fp8 cache (converted in
// the CTA), bf16 from a bf16 one (copied straight into the operand tiles).
//
// Warp roles (768 threads):
//   warp 0        tensor copies: fp8: tiles of codes; bf16: the operand tiles, 64 dims x 16 slots each
//   warp 1        tcgen05 issuer: S_x = Q_x K^T and O_x += P_x V (P in TMEM)
//   warps 2-3     per-key vectors of the tiles in turn (scales, gates), up to four tiles ahead (two with gates)
//   warps 4-19    softmax of tiles A and B, two threads a row with half of a tile's keys each (a tile's next
//                 products wait for its softmax, so its length counts; the halves agree on a row's maximum
//                 by shared memory)
//   warps 20-23   fp8: e4m3 -> f16 operand tiles; bf16: zeros over the values of the last tile past the
//                 prefix
#include <type_traits>

#include "decode_split.cuh"
#include "launch.h"
#include "rows.cuh"

namespace gcs {
namespace {

constexpr int kTileKeys = 128;    // 8 pages
constexpr int kPreThreads = 768;
constexpr int kStage = 16384;     // one operand stage: 128 rows x 64 dims or 64 keys x 128 dims
constexpr int kVecs = 4;          // tiles whose vectors are held
constexpr float kPrePScale = 16.f;  // P * vscale carried x 2^4
constexpr float kPreLazy = 4.f;     // lazy rescale threshold (log2 units): P <= 2^4

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 add2(const float2& a, const float2& b) { return fma2(a, both(1.f), b); }

template <bool BF16, bool GATES>
struct PreCfg {
  static constexpr int STAGES = BF16 ? 8 : 6;              // a tile's K dims 0..63, 64..127, V keys 0..63, 64..127
  static constexpr int RAW = BF16 ? 0 : GATES ? 2 : 3;     // K or V tiles of codes, on their way to be converted
  static constexpr int OFF_Q = 0;                          // [2 tiles][2 dim chunks] x 16 KB
  static constexpr int OFF_RING = 4 * kStage;
  static constexpr int OFF_RAW = OFF_RING + STAGES * kStage;   // [RAW] x 16 KB
  static constexpr int OFF_VEC = OFF_RAW + RAW * kStage;   // [HELD] x {ks'[128], vs'[128], G[16][132]}
  static constexpr int GATE_ROW = kTileKeys + 4;           // floats: the heads' rows 16 bytes apart in the banks
  static constexpr int VEC = 1024 + (GATES ? 16 * GATE_ROW * 4 : 0);
  static constexpr int HELD = GATES ? 2 : kVecs;           // tiles whose vectors are held
  static constexpr int OFF_BAR = OFF_VEC + HELD * VEC;
  static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 2 * kVecs + 26) * 8;
  static constexpr int OFF_MAX = OFF_MISC + 32;            // [2] x [2 tiles][2 halves][128 rows]
  static constexpr int SMEM = OFF_MAX + 2 * 512 * 4 + 1024;
  static_assert(SMEM <= 226 * 1024, "shared memory budget");
  static_assert(256 * 528 <= OFF_VEC, "the rows that leave");
};

// 128 x (48 + 4 x 96 + 48) = 61440 = 768 threads x 80 at launch
template <int N>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N) : "memory"); }
template <int N>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N) : "memory"); }

__device__ __forceinline__ void sts128(uint8_t* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }
// 16 e4m3 codes to the units 2 u and 2 u + 1 of row r of a swizzled tile
__device__ __forceinline__ void put_codes(uint8_t* tile, int r, int u, uint4 v) {
  uint32_t w[8];
  e4m3x4_to_f16x2x2(v.x, w[0], w[1]);
  e4m3x4_to_f16x2x2(v.y, w[2], w[3]);
  e4m3x4_to_f16x2x2(v.z, w[4], w[5]);
  e4m3x4_to_f16x2x2(v.w, w[6], w[7]);
  sts128(tile + sw128_offset(r, 2 * u), make_uint4(w[0], w[1], w[2], w[3]));
  sts128(tile + sw128_offset(r, 2 * u + 1), make_uint4(w[4], w[5], w[6], w[7]));
}
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Arrives once this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Plain bulk copy shared -> global: both addresses and the size in 16-byte steps; tracked by this thread's bulk
// group.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

// Tokens that group g shares, as far as the first request's cache and the host's bound go.
__device__ __forceinline__ int group_len(const DecodeParams& p, int g, int first) {
  return max(0, min(min(__ldg(p.prefix_lens + g), p.max_prefix), __ldg(p.seq_lens + first)));
}

template <bool BF16, bool GATES>
__global__ void __launch_bounds__(kPreThreads, 1)
    decode_prefix_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const DecodeParams p) {
  using C = PreCfg<BF16, GATES>;
  constexpr int kStages = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align_1k(smem_raw);

  // This kernel may run beside the one before it, and what comes after it waits for it alone: no block ends
  // before that one has.
  WaitAtEnd at_end;
  grid_release();
  const int seg = blockIdx.x % p.pre_segs, qp = blockIdx.x / p.pre_segs;
  const int kvh = blockIdx.y, grp = blockIdx.z;
  const int r0 = __ldg(p.cu_groups + grp), r1 = __ldg(p.cu_groups + grp + 1);
  if (r1 <= r0) return;
  const int q_begin = __ldg(p.cu_q + r0);
  const int ql = __ldg(p.cu_q + r1) - q_begin;  // query rows of the group
  const int P = group_len(p, grp, r0);
  const int G = p.group, lgG = G == 16 ? 4 : 3;
  const int pos_tile = 128 / G;  // query rows of a 128-row tile
  const int row0 = qp * 2 * pos_tile;
  const int key0 = seg * p.pre_seg_keys;
  if (row0 >= ql || key0 >= P) return;
  const int key1 = min(P, key0 + p.pre_seg_keys);
  const int W = p.window;
  const int32_t* trow = p.block_table + (size_t)r0 * p.max_blocks;
  const int lb = p.log2_block_pages + 4;  // log2 of a cache block's tokens

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;                 // [kStages] operand stages written
  uint64_t* empty = bars + kStages;      // [kStages] consumed
  uint64_t* vec_full = bars + 2 * kStages;   // [HELD]
  uint64_t* vec_empty = vec_full + kVecs;    // [HELD]
  uint64_t* q_full = vec_empty + kVecs;  // [2 tiles]
  uint64_t* s_full = q_full + 2;         // [2 tiles]
  uint64_t* p_full = q_full + 4;         // [2 tiles]
  uint64_t* pv_done = q_full + 6;        // [2 tiles]
  uint64_t* tail_full = q_full + 8;      // bf16: the values of the last tile
  uint64_t* drain = q_full + 9;
  uint64_t* raw_full = q_full + 10;      // [RAW] fp8
  uint64_t* raw_empty = q_full + 13;     // [RAW]
  uint64_t* agreed = q_full + 16;        // [2 tiles][4 quarters] both halves' maxima written
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* see = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);  // [2 tiles] x {least, greatest last key of a row}
  const Abort ab{abort_flag, p.status};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], BF16 ? 1 : 4);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::HELD; ++i) {
      mbar_init(&vec_full[i], GATES ? 64 : 32);
      mbar_init(&vec_empty[i], 16);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 8);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);
      mbar_init(&pv_done[i], 1);
      see[2 * i] = 0x7fffffff;
      see[2 * i + 1] = -1;
    }
    for (int i = 0; i < C::RAW; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&agreed[i], 2);
    mbar_init(tail_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  __syncthreads();
  // the softmax threads' rows: packed row, its request's last visible key
  const bool softmax = warp >= 4 && warp < 20;
  const int x_of = softmax ? (warp - 4) >> 3 : 0, half = (warp - 4) >> 2 & 1;
  const int rr = (warp & 3) * 32 + lane;  // row of the tile
  const int head = rr & (G - 1);
  const int pos = row0 + x_of * pos_tile + (rr >> lgG);
  const bool row_valid = softmax && pos < ql;
  const int tt = q_begin + min(pos, ql - 1);  // packed row
  int lastk = -1, req = r0;
  uint4 qv[8];  // half of this row of Q, on its way
  if (softmax) {
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (size_t)tt * p.q_ts + (size_t)(kvh * G + head) * p.q_hs);
#pragma unroll
    for (int u = 0; u < 8; ++u) qv[u] = row_valid ? __ldg(src + 8 * half + u) : make_uint4(0u, 0u, 0u, 0u);
    // the request whose rows hold tt: where rows of one length would have it, or searched for
    req = r0 + (int)((long long)(tt - q_begin) * (r1 - r0) / ql);
    int from = __ldg(p.cu_q + req), to = __ldg(p.cu_q + req + 1), len = __ldg(p.seq_lens + req);
    if (from > tt || to <= tt) {
      int lo = r0, hi = r1;  // cu_q[lo] <= tt < cu_q[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu_q + mid) <= tt) lo = mid;
        else hi = mid;
      }
      req = lo;
      to = __ldg(p.cu_q + req + 1);
      len = __ldg(p.seq_lens + req);
    }
    lastk = len - (to - tt);
    if (row_valid && half == 0) {
      atomicMin(&see[2 * x_of], lastk);
      atomicMax(&see[2 * x_of + 1], lastk);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // key tiles of the segment (index jt, keys key0 + 128 jt ..) that each query tile sees
  const int ntile_seg = (key1 - key0 + kTileKeys - 1) / kTileKeys;
  int lo[2], hi[2];
  for (int x = 0; x < 2; ++x) {
    const int lk_min = see[2 * x], lk_max = see[2 * x + 1];
    lo[x] = 0;
    hi[x] = -1;
    if (lk_max < key0) continue;  // no rows, or none that sees this far
    hi[x] = min(ntile_seg - 1, (lk_max - key0) / kTileKeys);
    const int fk = W > 0 ? max(0, lk_min - W + 1) : 0;
    if (fk > key0) lo[x] = (fk - key0) / kTileKeys;
  }
  int hi_t = -1, lo_t = 1 << 30;
  for (int x = 0; x < 2; ++x)
    if (lo[x] <= hi[x]) {
      hi_t = max(hi_t, hi[x]);
      lo_t = min(lo_t, lo[x]);
    }
  const int nt = hi_t < 0 ? 0 : hi_t - lo_t + 1;  // processed as jt = lo_t + n, n = 0 .. nt - 1
  int n_first[2], n_last[2];
  for (int x = 0; x < 2; ++x) {
    const bool any = lo[x] <= hi[x];
    n_first[x] = any ? lo[x] - lo_t : nt;
    n_last[x] = any ? hi[x] - lo_t : -1;
  }
  auto part = [&](int x, int n) -> bool { return n >= n_first[x] && n <= n_last[x]; };
  auto ring_next = [&](uint32_t& stage, uint32_t& phase) {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  };

  if (warp < 4) {
    reg_dec<48>();
    if (warp == 0) {
      if (!BF16) {
        // ---------------------------------------------------------- codes: K and V tiles in turn, lane = page
        if (lane == 0) {
          prefetch_tmap(&tmK);
          prefetch_tmap(&tmV);
        }
        const int last_page = (P + kPage - 1) / kPage;
        int i = 0;  // K or V tile
        uint32_t buf = 0, phase = 0;
        for (int n = 0; n < nt; ++n) {
          const int pg0 = key0 / kPage + (lo_t + n) * 8, pg = pg0 + lane;
          const int nv = min(8, last_page - pg0);  // pages of the tile that exist
          const int blk = lane < nv ? __ldg(trow + (pg >> p.log2_block_pages)) : 0;
          const int sub = (pg & ((1 << p.log2_block_pages) - 1)) * kPage;
          const int cy = p.kv_head_inner ? kvh : sub, cz = p.kv_head_inner ? sub : kvh;
          bool okl = true;
          for (int v = 0; v < 2 && okl; ++v, ++i) {
            okl = __all_sync(0xffffffffu, wait_bar(&raw_empty[buf], phase ^ 1, ab));
            if (!okl) break;
            if (lane == 0) mbar_expect_tx(&raw_full[buf], nv * 2048);
            __syncwarp();
            if (lane < nv)
              tma_load_4d(smem + C::OFF_RAW + buf * kStage + lane * 2048, v ? &tmV : &tmK, &raw_full[buf], 0, cy, cz, blk);
            if (++buf == (uint32_t)C::RAW) {
              buf = 0;
              phase ^= 1;
            }
          }
          if (!okl) break;
        }
      } else {
        // ---------------------------------------------------------- operand tiles by tensor copies
        // The values of the prefix's last, partly filled tile go by tail_full to warp 20, which zeroes what
        // lies past the prefix (whatever its bytes hold) before the stages count as written.
        const int pl = lane & 7, c = lane >> 3 & 1;  // page, 64 dims
        if (lane == 0) {
          prefetch_tmap(&tmK);
          prefetch_tmap(&tmV);
        }
        const int last_page = (P + kPage - 1) / kPage;
        uint32_t stage = 0, phase = 0;
        for (int n = 0; n < nt; ++n) {
          const int pg0 = key0 / kPage + (lo_t + n) * 8, pg = pg0 + pl;
          const int nv = min(8, last_page - pg0);  // pages of the tile that exist
          const int blk = pl < nv ? __ldg(trow + (pg >> p.log2_block_pages)) : 0;
          const int sub = (pg & ((1 << p.log2_block_pages) - 1)) * kPage;  // first slot of the page in its block
          const int cy = p.kv_head_inner ? kvh : sub, cz = p.kv_head_inner ? sub : kvh;
          const bool tail = key0 + (lo_t + n + 1) * kTileKeys > P;
          bool okl = true;
          for (int v = 0; v < 2 && okl; ++v) {  // K, V
            const uint32_t s0 = stage;
            okl = wait_bar(&empty[stage], phase ^ 1, ab);
            ring_next(stage, phase);
            const uint32_t s1 = stage;
            if (okl) okl = wait_bar(&empty[stage], phase ^ 1, ab);
            ring_next(stage, phase);
            okl = __all_sync(0xffffffffu, okl);
            if (!okl) break;
            if (lane == 0) {
              if (v == 0) {
                mbar_expect_tx(&full[s0], nv * 2048);
                mbar_expect_tx(&full[s1], nv * 2048);
              } else if (tail) {
                mbar_expect_tx(tail_full, nv * 4096);
              } else {
                mbar_expect_tx(&full[s0], 4 * 4096);
                mbar_expect_tx(&full[s1], 4 * 4096);
              }
            }
            __syncwarp();
            if (lane < 16 && pl < nv) {
              const uint32_t st = (v == 0 ? c : pl >> 2) ? s1 : s0;
              uint8_t* dst = smem + C::OFF_RING + st * kStage + (v == 0 ? pl * 2048 : c * (kStage / 2) + (pl & 3) * 2048);
              tma_load_4d(dst, v == 0 ? &tmK : &tmV, v == 1 && tail ? tail_full : &full[st], 64 * c, cy, cz, blk);
            }
          }
          if (!okl) break;
        }
      }
    } else if (warp == 1) {
      if (lane == 0 && nt > 0) {
        // -------------------------------------------------------- MMA issuer
        const uint32_t idS = BF16 ? idesc_bf16(128, kTileKeys, false, false) : idesc_f16(128, kTileKeys, false, false);
        const uint32_t idPV = BF16 ? idesc_bf16(128, kD, false, true) : idesc_f16(128, kD, false, true);
        const uint64_t dQ0 = sdesc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
        const uint64_t dK0 = sdesc_sw128(smem_u32(smem + C::OFF_RING), 16, 1024);
        const uint64_t dV0 = sdesc_sw128(smem_u32(smem + C::OFF_RING), kStage / 2, 1024);
        constexpr uint32_t kSt16 = kStage >> 4;
        uint32_t stage = 0, phase = 0;  // ring position of the next stage (K0 K1 V0 V1 per tile)
        auto next = [&](uint32_t& st, uint32_t& ph) {
          st = stage;
          ph = phase;
          ring_next(stage, phase);
        };
        auto mma_s = [&](int x, uint32_t k0, uint32_t k1) {  // S_x = Q_x K^T
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint64_t a = dQ0 + (x * 2 + c) * kSt16, b = dK0 + (c ? k1 : k0) * kSt16;
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ss(tmem + 128 * x, a + 2 * k, b + 2 * k, idS, (c | k) != 0);
          }
          mma_commit(&s_full[x]);
        };
        auto mma_pv = [&](int x, uint32_t v0, uint32_t v1, bool acc) {  // O_x += P_x V
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t b = dV0 + (h ? v1 : v0) * kSt16;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(tmem + 256 + 128 * x, tmem + 128 * x + (4 * h + k) * 8, b + 128 * k, idPV,
                     (acc || h || k) ? 1u : 0u);
          }
          mma_commit(&pv_done[x]);
        };
        bool qr[2] = {false, false};
        int kp[2] = {0, 0};
        uint32_t k0, pk0, k1, pk1;
        next(k0, pk0);
        next(k1, pk1);
        bool ok = wait_bars(ab, &full[k0], pk0, &full[k1], pk1);
        for (int x = 0; x < 2 && ok; ++x) {
          if (!part(x, 0)) continue;
          ok = wait_bar(&q_full[x], 0, ab);
          qr[x] = true;
          if (!ok) break;
          tc_fence_after();
          mma_s(x, k0, k1);
        }
        if (ok) {
          mma_commit(&empty[k0]);
          mma_commit(&empty[k1]);
        }
        for (int n = 0; n < nt && ok; ++n) {
          const bool more = n + 1 < nt;
          uint32_t v0, pv0, v1, pv1, n0 = 0, pn0 = 0, n1 = 0, pn1 = 0;
          next(v0, pv0);
          next(v1, pv1);
          if (more) {
            next(n0, pn0);
            next(n1, pn1);
          }
          // a tile's values are waited for before its first PV, the next keys only behind that, and the
          // values' stages go back before the second tile's scores
          bool have_v = false, have_k = !more;
          for (int x = 0; x < 2 && ok; ++x) {
            const bool do_pv = part(x, n), do_s = more && part(x, n + 1);
            if (!have_v && (do_pv || x == 1)) {
              ok = wait_bars(ab, &full[v0], pv0, &full[v1], pv1, do_pv ? &p_full[x] : nullptr, kp[x] & 1);
              have_v = true;
            } else if (do_pv) {
              ok = wait_bar(&p_full[x], kp[x] & 1, ab);
            }
            if (!ok) break;
            tc_fence_after();
            if (do_pv) {
              mma_pv(x, v0, v1, kp[x] > 0);
              ++kp[x];
            }
            if (x == 1) {
              mma_commit(&empty[v0]);
              mma_commit(&empty[v1]);
            }
            if (!have_k && (do_s || x == 1)) {
              ok = wait_bars(ab, &full[n0], pn0, &full[n1], pn1);
              have_k = true;
            }
            if (ok && do_s && !qr[x]) {
              ok = wait_bar(&q_full[x], 0, ab);
              qr[x] = true;
            }
            if (!ok) break;
            tc_fence_after();
            if (do_s) mma_s(x, n0, n1);
          }
          if (!ok) break;
          if (more) {
            mma_commit(&empty[n0]);
            mma_commit(&empty[n1]);
          }
        }
        if (!ok) {
          mma_commit(drain);
          mbar_wait(drain, 0, nullptr);
        }
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- per-key vectors
      // The two warps take the tiles in turn, lane l the keys 4 l .. 4 l + 3 (of one page).  A tile's scales
      // are on their way while the one before is written; the gates go straight into shared memory.
      const bool per_token = !BF16 && p.scale_mode == 0;
      const float kst = BF16 ? 1.f : per_token ? 0.f : __ldg(p.k_scale);
      const float vst = BF16 ? 1.f : per_token ? 0.f : __ldg(p.v_scale);
      const float sl2 = p.scale * kLog2e;
      float4 ks, vs;
      int blk, slot;
      auto fetch = [&](int n) {
        const int k = key0 + (lo_t + n) * kTileKeys + 4 * lane;
        ks = make_float4(kst, kst, kst, kst);
        vs = make_float4(vst, vst, vst, vst);
        blk = -1;
        if (n < nt && k < P) {
          blk = __ldg(trow + (k >> lb));
          slot = k & (p.block_size - 1);
          if (per_token) {
            const size_t at = ((size_t)blk * p.hkv + kvh) * p.block_size + slot;
            ks = __ldg(reinterpret_cast<const float4*>(p.k_scale + at));
            vs = __ldg(reinterpret_cast<const float4*>(p.v_scale + at));
          }
        }
      };
      fetch(warp - 2);
      for (int n = warp - 2; n < nt; n += 2) {
        const int a = n % C::HELD, left = P - (key0 + (lo_t + n) * kTileKeys + 4 * lane);  // of this lane's keys
        float4 k4 = ks, v4 = vs;
        const int b = blk, sl = slot;
        fetch(n + 2);
        if (!wait_bar(&vec_empty[a], ((n / C::HELD) & 1) ^ 1, ab)) break;
        float* vec = reinterpret_cast<float*>(smem + C::OFF_VEC + a * C::VEC);
        if (GATES) {
          if (b >= 0) {
            const float* g = p.g_cache + ((size_t)b * p.hq + kvh * G) * p.block_size + sl;
            for (int h = 0; h < G; ++h) copy16(vec + 2 * kTileKeys + h * C::GATE_ROW + 4 * lane, g + (size_t)h * p.block_size);
          }
          copies_arrive(&vec_full[a]);
        }
        // zeros past the prefix, whatever is there
        k4.x = left > 0 ? k4.x * sl2 : 0.f, v4.x = left > 0 ? v4.x * kPrePScale : 0.f;
        k4.y = left > 1 ? k4.y * sl2 : 0.f, v4.y = left > 1 ? v4.y * kPrePScale : 0.f;
        k4.z = left > 2 ? k4.z * sl2 : 0.f, v4.z = left > 2 ? v4.z * kPrePScale : 0.f;
        k4.w = left > 3 ? k4.w * sl2 : 0.f, v4.w = left > 3 ? v4.w * kPrePScale : 0.f;
        reinterpret_cast<float4*>(vec)[lane] = k4;
        reinterpret_cast<float4*>(vec + kTileKeys)[lane] = v4;
        mbar_arrive(&vec_full[a]);
      }
    }
    __syncwarp();
  } else if (warp >= 20) {
    reg_dec<48>();
    uint32_t stage = 0, phase = 0;
    if (BF16) {
      // ---------------------------------------------------------- zeros past the prefix
      // (the segment's last tile is processed by some query tile only if a row sees it)
      if (warp == 20 && nt > 0 && key0 + (lo_t + nt) * kTileKeys > P) {
        if (wait_bar(tail_full, 0, ab)) {
          const uint32_t s2 = (4 * (nt - 1) + 2) % kStages, s3 = s2 + 1;
          const int kbase = key0 + (lo_t + nt - 1) * kTileKeys;
          for (int i = lane; i < kTileKeys * 16; i += 32) {
            const int k = i >> 4, u = i & 15;  // key, 16 bytes of it
            if (kbase + k >= P)
              sts128(smem + C::OFF_RING + (k >> 6 ? s3 : s2) * kStage + (u >> 3) * (kStage / 2) + (k & 63) * 128 +
                         (u & 7) * 16,
                     make_uint4(0u, 0u, 0u, 0u));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full[s2]);
            mbar_arrive(&full[s3]);
          }
        }
      }
    } else {
      // ---------------------------------------------------------- e4m3 -> f16 operand tiles
      // A tile of codes is 128 keys x 128 B, 128-byte swizzled.  Thread t takes the keys 8 i + (t & 7) of one
      // half of them and the 16-dim group (t / 8) & 7 of each: a quarter warp reads one group of eight
      // neighbouring keys and writes the two 16-B halves of each result to units of their swizzled
      // rows that are all in different bank groups.
      //   K: the first stage holds dims 0..63, the second dims 64..127; row = key (K-major)
      //   V: the first stage holds keys 0..63, the second keys 64..127; inside a stage, dims 0..63 then
      //      64..127 (8 KB apart), row = key (MN-major)
      const int t = threadIdx.x - 640, ck = t & 7, cq = t >> 3 & 7, hf = t >> 6;
      uint32_t buf = 0, raw_phase = 0;
      bool ok = true;
      for (int i = 0; i < 2 * nt && ok; ++i) {
        const bool v = i & 1;
        const int kbase = key0 + (lo_t + (i >> 1)) * kTileKeys + 64 * hf + ck;
        const uint32_t sa = stage, pa = phase;
        ring_next(stage, phase);
        const uint32_t sb = stage, pb = phase;
        ring_next(stage, phase);
        ok = wait_bar(&raw_full[buf], raw_phase, ab) && wait_bar(&empty[sa], pa ^ 1, ab) && wait_bar(&empty[sb], pb ^ 1, ab);
        if (!ok) break;
        const uint8_t* src = smem + C::OFF_RAW + buf * kStage + (64 * hf + ck) * 128 + ((cq ^ ck) << 4);
        uint8_t* dst = smem + C::OFF_RING;
        int row = ck;  // of the operand tile
        if (v) {
          dst += (hf ? sb : sa) * kStage + (cq >> 2) * (kStage / 2);
        } else {
          dst += (cq >> 2 ? sb : sa) * kStage;
          row += 64 * hf;
        }
#pragma unroll 4
        for (int j = 0; j < 8; ++j) {
          uint4 x = make_uint4(0u, 0u, 0u, 0u);  // past the prefix, whatever is there
          if (kbase + 8 * j < P) x = lds128(src + j * 1024);
          put_codes(dst, row + 8 * j, cq & 3, x);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[sa]);
          mbar_arrive(&full[sb]);
          mbar_arrive(&raw_empty[buf]);
        }
        if (++buf == (uint32_t)C::RAW) {
          buf = 0;
          raw_phase ^= 1;
        }
      }
    }
    __syncwarp();
  } else {
    reg_inc<96>();
    // ------------------------------------------------------------ softmax, tile x
    const int x = x_of, quarter = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + 128 * x, tO = tmem + lane_off + 256 + 128 * x;
    const int my_first = x ? n_first[1] : n_first[0], my_last = x ? n_last[1] : n_last[0];
    if (my_first <= my_last) {
      // 64 dims of this row of Q into their 128-B-swizzled K-major tile
      uint8_t* qs = smem + C::OFF_Q + (x * 2 + half) * kStage;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        uint4 f = qv[u];
        if (!BF16)
          f = make_uint4(bf16pair_to_f16x2(f.x), bf16pair_to_f16x2(f.y), bf16pair_to_f16x2(f.z),
                         bf16pair_to_f16x2(f.w));
        sts128(qs + sw128_offset(rr, u), f);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[x]);
    }
    float gi = 0.f;  // the row's own G
    if (GATES && row_valid) {  // a row that stands inside the prefix: like every key there, by the first request's table
      const int32_t* own = lastk < P ? trow : p.block_table + (size_t)req * p.max_blocks;
      const int blk = __ldg(own + lastk / p.block_size);
      gi = __ldg(p.g_cache + ((size_t)blk * p.hq + kvh * G + head) * p.block_size + lastk % p.block_size);
    }
    const float sl2 = p.scale * kLog2e;
    float m = neg_inf(), l = 0.f;
    const int lk_min = see[2 * x], lk_max = see[2 * x + 1];
    bool ok = true;
    int kx = 0;  // key tiles processed by this query tile
    for (int n = 0; n < nt; ++n) {
      const int a = n % C::HELD;
      ok = wait_bar(&vec_full[a], (n / C::HELD) & 1, ab);
      if (!ok) break;
      if (n >= my_first && n <= my_last) {
        const int j0 = key0 + (lo_t + n) * kTileKeys;
        ok = wait_bar(&s_full[x], kx & 1, ab);
        if (!ok) break;
        tc_fence_after();
        uint32_t sv[64];  // this thread's keys: 64 half .. of the tile
        tmem_ld32(tS + 64 * half, sv);
        tmem_ld32(tS + 64 * half + 32, sv + 32);
        tmem_ld_wait();
        const float* vec = reinterpret_cast<const float*>(smem + C::OFF_VEC + a * C::VEC) + 64 * half;
        const float4* ks4 = reinterpret_cast<const float4*>(vec);
        const float4* vs4 = reinterpret_cast<const float4*>(vec + kTileKeys);
        const float4* g4 = reinterpret_cast<const float4*>(vec + 2 * kTileKeys + head * C::GATE_ROW);
        const bool need_mask = j0 + kTileKeys > P || j0 + kTileKeys - 1 > lk_min || (W > 0 && j0 < lk_max - W + 1);
        const int jmax = min(lastk, P - 1) - j0 - 64 * half;
        const int jmin = W > 0 ? lastk - W + 1 - j0 - 64 * half : -(1 << 30);
        float mxp[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
        // one straight run of code for each case: a branch within it would part it
        auto scores = [&](auto masked) {
#pragma unroll
          for (int j4 = 0; j4 < 16; ++j4) {
            float2 ka = both(sl2), kb = both(sl2);
            if (!BF16) {
              const float4 k4 = ks4[j4];
              ka = make_float2(k4.x, k4.y), kb = make_float2(k4.z, k4.w);
            }
            float2 ta = make_float2(__uint_as_float(sv[4 * j4]), __uint_as_float(sv[4 * j4 + 1]));
            float2 tb = make_float2(__uint_as_float(sv[4 * j4 + 2]), __uint_as_float(sv[4 * j4 + 3]));
            if (GATES) {  // G_i - G_j before the change of units: the difference is what is small
              const float4 g = g4[j4];
              ta = fma2(ta, ka, make_float2((gi - g.x) * kLog2e, (gi - g.y) * kLog2e));
              tb = fma2(tb, kb, make_float2((gi - g.z) * kLog2e, (gi - g.w) * kLog2e));
            } else {
              ta = mul2(ta, ka);
              tb = mul2(tb, kb);
            }
            if (decltype(masked)::value) {
              const int j = 4 * j4;
              ta.x = j >= jmin && j <= jmax ? ta.x : neg_inf();
              ta.y = j + 1 >= jmin && j + 1 <= jmax ? ta.y : neg_inf();
              tb.x = j + 2 >= jmin && j + 2 <= jmax ? tb.x : neg_inf();
              tb.y = j + 3 >= jmin && j + 3 <= jmax ? tb.y : neg_inf();
            }
            sv[4 * j4] = __float_as_uint(ta.x), sv[4 * j4 + 1] = __float_as_uint(ta.y);
            sv[4 * j4 + 2] = __float_as_uint(tb.x), sv[4 * j4 + 3] = __float_as_uint(tb.y);
            mxp[(2 * j4) & 3] = fmax3(mxp[(2 * j4) & 3], ta.x, ta.y);
            mxp[(2 * j4 + 1) & 3] = fmax3(mxp[(2 * j4 + 1) & 3], tb.x, tb.y);
          }
        };
        if (need_mask) scores(std::true_type());
        else scores(std::false_type());
        // the halves agree (and both have read their scores: P takes the place of some of them)
        const float mine = fmaxf(fmax3(mxp[0], mxp[1], mxp[2]), mxp[3]);
        float* mx = reinterpret_cast<float*>(smem + C::OFF_MAX) + (kx & 1) * 512 + x * 256 + rr;
        mx[half * 128] = mine;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&agreed[x * 4 + quarter]);
        ok = wait_bar(&agreed[x * 4 + quarter], kx & 1, ab);
        if (!ok) break;
        tc_fence_after();
        const float m_new = fmax3(m, mine, mx[(half ^ 1) * 128]);
        const bool need = m_new > m + kPreLazy;
        if (__any_sync(0xffffffffu, need)) {
          const float alpha = need ? ex2(m - m_new) : 1.f;
          if (kx > 0) {
            // O holds the previous key tiles: wait for their PV before scaling it, half of its columns
            ok = wait_bar(&pv_done[x], (kx - 1) & 1, ab);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t ov[16];
              tmem_ld16(tO + half * 64 + cc * 16, ov);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
              tmem_st16(tO + half * 64 + cc * 16, ov);
            }
            tmem_st_wait();
          }
          l *= alpha;
          if (need) m = m_new;
        }
        const float2 mu = both(m == neg_inf() ? 0.f : -m);
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int qt = 0; qt < 2; ++qt) {
          uint32_t pk[16];
#pragma unroll
          for (int jj = 0; jj < 8; ++jj) {
            const int j = qt * 32 + 4 * jj;
            const float2 za = add2(make_float2(__uint_as_float(sv[j]), __uint_as_float(sv[j + 1])), mu);
            const float2 zb = add2(make_float2(__uint_as_float(sv[j + 2]), __uint_as_float(sv[j + 3])), mu);
            const float2 pa = make_float2(ex2(za.x), ex2(za.y)), pb = make_float2(ex2(zb.x), ex2(zb.y));
            ls[0] = add2(ls[0], pa);
            ls[1] = add2(ls[1], pb);
            if (BF16) {
              pk[2 * jj] = pack_bf16x2(pa.x, pa.y);
              pk[2 * jj + 1] = pack_bf16x2(pb.x, pb.y);
            } else {  // V scales multiply the probabilities after the row sum
              const float4 v4 = vs4[j >> 2];
              const float2 wa = mul2(pa, make_float2(v4.x, v4.y)), wb = mul2(pb, make_float2(v4.z, v4.w));
              pk[2 * jj] = pack_f16x2(wa.x, wa.y);
              pk[2 * jj + 1] = pack_f16x2(wb.x, wb.y);
            }
          }
          tmem_st16(tS + half * 32 + qt * 16, pk);
        }
        l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
        ++kx;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&vec_empty[a]);
    }
    if (ok && kx > 0) ok = wait_bar(&pv_done[x], (kx - 1) & 1, ab);
    // Both tiles are through with the operands: their shared memory takes the rows, 16 bytes apart in the
    // banks, and each thread's half row leaves in one copy of 256 bytes (stores by row would be 32 lanes in 32
    // rows).
    float* sums = reinterpret_cast<float*>(smem + C::OFF_MAX) + (kx & 1) * 512 + x * 256 + rr;
    if (half) *sums = l;
    asm volatile("bar.sync 1, 512;" ::: "memory");
    if (ok && !*abort_flag) {
      const size_t at = ((size_t)seg * p.total_q + tt) * p.hq + kvh * G + head;
      if (kx > 0) {
        tc_fence_after();
        uint8_t* mine = smem + (x * 128 + rr) * 528 + half * 256;
        constexpr float kInv = BF16 ? 1.f : 1.f / kPrePScale;
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t ov[32];
          tmem_ld32(tO + half * 64 + cc * 32, ov);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            reinterpret_cast<float4*>(mine)[cc * 8 + j] =
                make_float4(__uint_as_float(ov[4 * j]) * kInv, __uint_as_float(ov[4 * j + 1]) * kInv,
                            __uint_as_float(ov[4 * j + 2]) * kInv, __uint_as_float(ov[4 * j + 3]) * kInv);
        }
        fence_proxy_async_smem();
        if (row_valid) bulk_store(p.pre_acc + at * kD + half * 64, mine, kD * 2);
        bulk_commit_group();
        bulk_wait_group0();
      }
      // the combine does not use the accumulators of an empty partial
      if (row_valid && !half) p.pre_ml[at] = kx > 0 ? make_float2(m, l + *sums) : make_float2(neg_inf(), 0.f);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partials of the prefix and of the tokens behind it for every (query row, head): 16 dim
// groups x SL segment lanes a head, the lanes adjacent; each joins every SL-th segment, shuffles
// join the lanes.
template <int SL>
__global__ void __launch_bounds__(256) decode_join_kernel(const DecodeParams p) {
  constexpr int kHeads = 16 / SL;  // query heads per CTA
  WaitAtEnd at_end;
  const int r = blockIdx.x / p.max_q_len, t = blockIdx.x % p.max_q_len;
  const int kvh = blockIdx.y;
  const int q_begin = __ldg(p.cu_q + r);
  const int ql = __ldg(p.cu_q + r + 1) - q_begin;
  if (t >= ql) return;
  int group_first;
  const int L = __ldg(p.seq_lens + r), start = shared_len(p, r, group_first);
  const int G = p.group;
  const int sl = threadIdx.x & (SL - 1), d0 = ((threadIdx.x / SL) & 15) * 8;
  const int hh = blockIdx.z * kHeads + threadIdx.x / (16 * SL);
  const int rows = p.max_q_len * kRows;
  // segments of the prefix, then those behind it (the ones wholly before every window were not written)
  const int npre = (start + p.pre_seg_keys - 1) / p.pre_seg_keys;
  const int page0 = start / kPage, npages = (L + kPage - 1) / kPage;
  const int nseg = start < L ? min(p.max_segs, (npages - page0 + p.seg_pages - 1) / p.seg_pages) : 0;
  const int first_page = p.window > 0 ? max(0, L - ql - p.window + 1) / kPage : 0;
  const int s_begin = first_page > page0 ? (first_page - page0) / p.seg_pages : 0;
  const int n = npre + max(0, nseg - s_begin);
  float m = neg_inf(), l = 0.f;
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  grid_wait();  // the partials
  if (hh < G) {
#pragma unroll 4
    for (int i = sl; i < n; i += SL) {
      const size_t pre = ((size_t)i * p.total_q + q_begin + t) * p.hq + kvh * G + hh;
      const size_t own = (((size_t)r * p.max_segs + s_begin + i - npre) * p.hkv + kvh) * rows + t * G + hh;
      const float2 v = i < npre ? p.pre_ml[pre] : reinterpret_cast<const float2*>(p.part_ml)[own];
      const float4* a = reinterpret_cast<const float4*>((i < npre ? p.pre_acc + pre * kD : p.part_acc + own * kD) + d0);
      float4 x0 = a[0], x1 = a[1];
      if (v.x == neg_inf()) x0 = x1 = make_float4(0.f, 0.f, 0.f, 0.f);  // empty: not written
      const float a2[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
      merge_partial(m, l, acc, v.x, v.y, a2);
    }
  }
#pragma unroll
  for (int off = 1; off < SL; off <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, off);
    const float l2 = __shfl_xor_sync(0xffffffffu, l, off);
    float a2[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) a2[j] = __shfl_xor_sync(0xffffffffu, acc[j], off);
    merge_partial(m, l, acc, m2, l2, a2);
  }
  if (sl != 0 || hh >= G) return;
  // the sink logit (log2 units) joins the max and, once, the denominator
  float den = l;
  if (p.sink) {
    const float sg = __ldg(p.sink + kvh * G + hh) * kLog2e;
    const float M = fmaxf(m, sg);
    const float w = (m == neg_inf()) ? 0.f : ex2(m - M);
    den = w * l + ex2(sg - M);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] *= w;
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  uint4 o;
  o.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  o.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
  o.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
  o.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
  *reinterpret_cast<uint4*>(p.out + (size_t)(q_begin + t) * p.out_ts + (size_t)(kvh * G + hh) * p.out_hs + d0) = o;
}

template <bool BF16, bool GATES>
cudaError_t launch_prefix(const DecodeParams& p, const DecodeMaps& maps, bool beside, cudaStream_t s) {
  using C = PreCfg<BF16, GATES>;
  auto kern = decode_prefix_kernel<BF16, GATES>;
  cudaError_t e = allow_smem<decode_prefix_kernel<BF16, GATES>>(C::SMEM);
  if (e != cudaSuccess) return e;
  const int rows = 2 * (128 / p.group);  // query rows of one CTA
  const dim3 grid((p.max_group_q + rows - 1) / rows * p.pre_segs, p.hkv, p.num_groups);
  if (beside) return launch_beside(kern, grid, kPreThreads, C::SMEM, s, maps.k, maps.v, p);
  kern<<<grid, kPreThreads, C::SMEM, s>>>(maps.k, maps.v, p);
  return cudaGetLastError();
}

template <int KVF, bool PT, bool FEAT, int G, bool SQ>
cudaError_t launch_split(const DecodeParams& p, const DecodeMaps& maps, dim3 grid, cudaStream_t s) {
  constexpr int smem = DecCfg<KVF, PT, FEAT, SQ>::SMEM;  // + 4 KB of query fragments a position
  auto kern = decode_split_kernel<KVF, PT, FEAT, G, SQ, false, true>;
  const cudaError_t e = allow_smem<decode_split_kernel<KVF, PT, FEAT, G, SQ, false, true>>(smem + 4096 * 4);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, smem + 4096 * p.max_q_len, s>>>(maps.k, maps.v, p);
  return cudaGetLastError();
}

// The tokens behind the prefixes.
cudaError_t launch_own(const DecodeParams& p, const DecodeMaps& maps, cudaStream_t s) {
  const dim3 grid(p.max_segs, p.hkv, p.num_reqs);
  const bool feat = p.g_cache != nullptr || p.window > 0;
#define GCS_RUN2(KVF, PT, F, SQ) \
  (p.group == 8 ? launch_split<KVF, PT, F, 8, SQ>(p, maps, grid, s) : launch_split<KVF, PT, F, 16, SQ>(p, maps, grid, s))
#define GCS_RUN(KVF, PT, F) (p.max_q_len > 2 ? GCS_RUN2(KVF, PT, F, true) : GCS_RUN2(KVF, PT, F, false))
  if (p.kv_format == 1) return feat ? GCS_RUN(1, false, true) : GCS_RUN(1, false, false);
  if (p.scale_mode == 1) return feat ? GCS_RUN(0, true, true) : GCS_RUN(0, true, false);
  return feat ? GCS_RUN(0, false, true) : GCS_RUN(0, false, false);
#undef GCS_RUN
#undef GCS_RUN2
}

}  // namespace

cudaError_t launch_decode_shared(const DecodeParams& p, const DecodeMaps& maps, cudaStream_t s) {
  // The two kernels need nothing of each other: the prefix's blocks follow as the others' SMs fall free (64 x 1
  // behind 16K: 99.4 -> 93.6 us).
  cudaError_t e = cudaSuccess;
  const bool both = p.max_segs > 0;
  if (both && (e = launch_own(p, maps, s)) != cudaSuccess) return e;
  if (p.pre_segs > 0) {
    const bool gates = p.g_cache != nullptr;
    if (p.kv_format == 1)
      e = gates ? launch_prefix<true, true>(p, maps, both, s) : launch_prefix<true, false>(p, maps, both, s);
    else
      e = gates ? launch_prefix<false, true>(p, maps, both, s) : launch_prefix<false, false>(p, maps, both, s);
    if (e != cudaSuccess) return e;
  }
  const int segs = p.pre_segs + p.max_segs;
  const dim3 grid(p.num_reqs * p.max_q_len, p.hkv, segs >= 32 ? p.group / 2 : (p.group + 3) / 4);
  if (segs == 0) {  // no partials, and no kernel of this call to run beside
    decode_join_kernel<4><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
  }
  // the join finds its places while the kernel before it ends
  if (segs >= 32) return launch_beside(decode_join_kernel<8>, grid, 256, 0, s, p);
  return launch_beside(decode_join_kernel<4>, grid, 256, 0, s, p);
}

}  // namespace gcs
