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
// Warp roles (384 threads):
//   warp 0      producer: per 128-key tile the 8 pages' K and V (fp8: raw pages with their
//               scales; bf16: the operand tiles, 64 dims x 16 slots a copy) and the gates
//   warp 1      tcgen05 issuer: S_x = Q_x K^T and O_x += P_x V (P in TMEM)
//   warps 2-3   fp8: e4m3 -> f16 operand tiles; bf16: zeros over the values past the prefix; both:
//               the per-key vectors for the softmax
//   warps 4-7   softmax of tile A, warps 8-11 of tile B, one thread per row
#include "decode_split.cuh"

namespace gcs {
namespace {

constexpr int kTileKeys = 128;    // 8 pages
constexpr int kPreThreads = 384;
constexpr int kStage = 16384;     // one operand stage: 128 rows x 64 dims or 64 keys x 128 dims
constexpr float kPrePScale = 16.f;  // P * vscale carried x 2^4
constexpr float kPreLazy = 4.f;     // lazy rescale threshold (log2 units): P <= 2^4

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <bool BF16, bool FEAT>
struct PreCfg {
  static constexpr int NST = BF16 ? 8 : FEAT ? 6 : 7;      // operand stages
  static constexpr int OFF_Q = 0;                          // [2 tiles][2 dim chunks] x 16 KB
  static constexpr int OFF_RING = 4 * kStage;
  static constexpr int OFF_KRAW = OFF_RING + NST * kStage; // (fp8: K pages | K scales | V scales |) gates
  static constexpr int KR_KS = BF16 ? 0 : 8 * 2048, KR_VS = KR_KS + (BF16 ? 0 : 512), KR_G = KR_VS + (BF16 ? 0 : 512);
  static constexpr int KRAW = KR_G + (FEAT ? 8 * 1024 : 0);
  static constexpr int OFF_VRAW = OFF_KRAW + KRAW;         // V pages
  static constexpr int OFF_AUX = OFF_VRAW + (BF16 ? 0 : 8 * 2048);  // [2] x {ks'[128], vs'[128], G'[16][128]}
  static constexpr int AUX = 1024 + (FEAT ? 8192 : 0);
  static constexpr int OFF_BAR = OFF_AUX + 2 * AUX;
  static constexpr int OFF_MISC = OFF_BAR + (2 * NST + 24) * 8;
  static constexpr int SMEM = OFF_MISC + 32 + 1024;
  static_assert(SMEM <= 226 * 1024, "shared memory budget");
};

// 128 x 88 + 256 x 208 = 64512 = 384 threads x 168 at launch
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n" ::: "memory"); }
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n" ::: "memory"); }

__device__ __forceinline__ void sts128(uint8_t* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }

// Tokens that group g shares, as far as the first request's cache and the host's bound go.
__device__ __forceinline__ int group_len(const DecodeParams& p, int g, int first) {
  return max(0, min(min(__ldg(p.prefix_lens + g), p.max_prefix), __ldg(p.seq_lens + first)));
}

template <bool BF16, bool FEAT>
__global__ void __launch_bounds__(kPreThreads, 1)
    decode_prefix_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const DecodeParams p) {
  using C = PreCfg<BF16, FEAT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align_1k(smem_raw);

  const int seg = blockIdx.x % p.pre_segs, qp = blockIdx.x / p.pre_segs;
  const int kvh = blockIdx.y, grp = blockIdx.z;
  const int r0 = __ldg(p.cu_groups + grp), r1 = __ldg(p.cu_groups + grp + 1);
  if (r1 <= r0) return;
  const int q_begin = __ldg(p.cu_q + r0);
  const int ql = __ldg(p.cu_q + r1) - q_begin;  // query rows of the group
  const int P = group_len(p, grp, r0);
  const int G = p.group, lgG = G == 16 ? 4 : 3;
  const int pos_tile = 128 / G;  // query rows of a 128-row tile
  const int lbp = p.log2_block_pages;
  const int row0 = qp * 2 * pos_tile;
  const int key0 = seg * p.pre_seg_keys;
  if (row0 >= ql || key0 >= P) return;
  const int key1 = min(P, key0 + p.pre_seg_keys);
  const int W = FEAT ? p.window : 0;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;               // [NST] operand stages written
  uint64_t* empty = bars + C::NST;     // [NST] consumed
  uint64_t* kr_full = bars + 2 * C::NST;
  uint64_t* kr_empty = kr_full + 1;
  uint64_t* vr_full = kr_full + 2;
  uint64_t* vr_empty = kr_full + 3;
  uint64_t* aux_full = kr_full + 4;    // [2]
  uint64_t* aux_empty = kr_full + 6;   // [2]
  uint64_t* q_full = kr_full + 8;      // [2 tiles]
  uint64_t* s_full = kr_full + 10;     // [2 tiles]
  uint64_t* p_full = kr_full + 12;     // [2 tiles]
  uint64_t* pv_done = kr_full + 14;    // [2 tiles]
  uint64_t* drain = kr_full + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* see = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);  // [2 tiles] x {least, greatest last key of a row}
  const Abort ab{abort_flag, p.status};
  uint8_t* kraw = smem + C::OFF_KRAW;
  uint8_t* vraw = smem + C::OFF_VRAW;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&full[i], BF16 ? 1 : 2);
      mbar_init(&empty[i], 1);
    }
    mbar_init(kr_full, 1);
    mbar_init(kr_empty, 2);
    mbar_init(vr_full, 1);
    mbar_init(vr_empty, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&aux_full[i], 2);
      mbar_init(&aux_empty[i], 8);
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
      see[2 * i] = 0x7fffffff;
      see[2 * i + 1] = -1;
    }
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
  const int x_of = warp < 4 ? 0 : (warp - 4) >> 2;
  const int rr = (warp & 3) * 32 + lane;  // row of the tile
  const int head = rr & (G - 1);
  const int pos = row0 + x_of * pos_tile + (rr >> lgG);
  const bool row_valid = warp >= 4 && pos < ql;
  const int tt = q_begin + min(pos, ql - 1);  // packed row
  int lastk = -1, req = r0;
  if (warp >= 4) {
    int lo = r0, hi = r1;  // cu_q[lo] <= tt < cu_q[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu_q + mid) <= tt) lo = mid;
      else hi = mid;
    }
    req = lo;
    lastk = __ldg(p.seq_lens + req) - (__ldg(p.cu_q + req + 1) - tt);
    if (row_valid) {
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

  if (warp < 4) {
    reg_dec();
    if (nt == 0) {
    } else if (warp == 0) {
      // ---------------------------------------------------------- page producer
      const int32_t* trow = p.block_table + (size_t)r0 * p.max_blocks;
      const bool per_token = !BF16 && p.scale_mode == 0;
      const bool has_gate = FEAT && p.g_cache != nullptr;
      const int pl = lane & 7, kind = lane >> 3;
      if (lane == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
      }
      const int last_page = (P + kPage - 1) / kPage;
      uint32_t stage = 0, phase = 0;
      for (int n = 0; n < nt; ++n) {
        const int pg0 = key0 / kPage + (lo_t + n) * 8;
        const int nv = min(8, last_page - pg0);  // pages of the tile that exist
        const uint32_t par = (n & 1) ^ 1;
        const int pg = pg0 + pl;
        const int blk = pl < nv ? __ldg(trow + (pg >> lbp)) : 0;
        const int sub = (pg & ((1 << lbp) - 1)) * kPage;  // first slot of the page in its block
        const int cy = p.kv_head_inner ? kvh : sub, cz = p.kv_head_inner ? sub : kvh;
        auto gates = [&](uint64_t* bar) {
          // the group's G heads x 16 slots: adjacent when a block is one page
          const float* src = p.g_cache + ((size_t)blk * p.hq + kvh * G) * p.block_size + sub;
          if (lbp == 0) {
            bulk_load(kraw + C::KR_G + pl * 1024, src, G * kPage * 4, bar);
          } else {
            for (int hh = 0; hh < G; ++hh)
              bulk_load(kraw + C::KR_G + pl * 1024 + hh * kPage * 4, src + (size_t)hh * p.block_size, kPage * 4, bar);
          }
        };
        if constexpr (!BF16) {
          bool okl = wait_bar(kr_empty, par, ab);
          if (!__all_sync(0xffffffffu, okl)) break;
          if (lane == 0)
            mbar_expect_tx(kr_full, nv * (2048 + (per_token ? 128 : 0) + (has_gate ? G * kPage * 4 : 0)));
          __syncwarp();
          if (pl < nv) {
            const size_t slot0 = ((size_t)blk * p.hkv + kvh) * p.block_size + sub;
            if (kind == 0) tma_load_4d(kraw + pl * 2048, &tmK, kr_full, 0, cy, cz, blk);
            else if (kind == 1 && per_token) bulk_load(kraw + C::KR_KS + pl * 64, p.k_scale + slot0, 64, kr_full);
            else if (kind == 2 && per_token) bulk_load(kraw + C::KR_VS + pl * 64, p.v_scale + slot0, 64, kr_full);
            else if (kind == 3 && has_gate) gates(kr_full);
          }
          okl = wait_bar(vr_empty, par, ab);
          if (!__all_sync(0xffffffffu, okl)) break;
          if (lane == 0) mbar_expect_tx(vr_full, nv * 2048);
          __syncwarp();
          if (kind == 0 && pl < nv) tma_load_4d(vraw + pl * 2048, &tmV, vr_full, 0, cy, cz, blk);
        } else {
          // operand stages of the tile: K dims 0..63, K dims 64..127, V keys 0..63, V keys 64..127.  The
          // values of the prefix's last, partly filled tile go by vr_full to warp 2, which zeroes what
          // lies past the prefix (whatever its bytes hold) before the stages count as written.
          const bool tail = key0 + (lo_t + n + 1) * kTileKeys > P;
          uint8_t* st[4];
          uint64_t* fb[4];
          bool okl = true;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            st[i] = smem + C::OFF_RING + stage * kStage;
            fb[i] = &full[stage];
            if (okl) okl = wait_bar(&empty[stage], phase ^ 1, ab);
            if (++stage == C::NST) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (has_gate && okl) okl = wait_bar(kr_empty, par, ab);
          if (!__all_sync(0xffffffffu, okl)) break;
          if (lane == 0) {
            mbar_expect_tx(fb[0], nv * 2048);
            mbar_expect_tx(fb[1], nv * 2048);
            if (tail) {
              mbar_expect_tx(vr_full, nv * 4096);
            } else {
              mbar_expect_tx(fb[2], 4 * 4096);
              mbar_expect_tx(fb[3], 4 * 4096);
            }
            if (has_gate) mbar_expect_tx(kr_full, nv * G * kPage * 4);
          }
          __syncwarp();
          if (pl < nv) {
            const int c = kind & 1;  // 64 dims
            if (kind < 2) {
              tma_load_4d(st[c] + pl * 2048, &tmK, fb[c], 64 * c, cy, cz, blk);
            } else {
              const int hv = pl >> 2;
              tma_load_4d(st[2 + hv] + c * (kStage / 2) + (pl & 3) * 2048, &tmV, tail ? vr_full : fb[2 + hv], 64 * c, cy,
                          cz, blk);
            }
            if (kind == 0 && has_gate) gates(kr_full);
          }
        }
      }
    } else if (warp == 1) {
      if (lane == 0) {
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
          if (++stage == C::NST) {
            stage = 0;
            phase ^= 1;
          }
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
          bool waited = false;
          for (int x = 0; x < 2 && ok; ++x) {
            const bool do_pv = part(x, n), do_s = more && part(x, n + 1);
            if (!do_pv && !do_s) continue;
            if (!waited) {
              ok = wait_bars(ab, &full[v0], pv0, &full[v1], pv1, do_pv ? &p_full[x] : nullptr, kp[x] & 1);
              if (ok && more) ok = wait_bars(ab, &full[n0], pn0, &full[n1], pn1);
              waited = true;
            } else if (do_pv) {
              ok = wait_bar(&p_full[x], kp[x] & 1, ab);
            }
            if (ok && do_s && !qr[x]) {
              ok = wait_bar(&q_full[x], 0, ab);
              qr[x] = true;
            }
            if (!ok) break;
            tc_fence_after();
            if (do_pv) {
              mma_pv(x, v0, v1, kp[x] > 0);
              ++kp[x];
            }
            if (do_s) mma_s(x, n0, n1);
          }
          // a stage is released only after its data was waited for, so its writer never runs two
          // phases ahead of this thread
          if (ok && !waited) {
            ok = wait_bars(ab, &full[v0], pv0, &full[v1], pv1);
            if (ok && more) ok = wait_bars(ab, &full[n0], pn0, &full[n1], pn1);
          }
          if (!ok) break;
          mma_commit(&empty[v0]);
          mma_commit(&empty[v1]);
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
      // ---------------------------------------------------------- converters (warps 2-3)
      const int c = threadIdx.x - 64;  // 0 .. 63
      const bool per_token = !BF16 && p.scale_mode == 0;
      const bool has_gate = FEAT && p.g_cache != nullptr;
      const float kst = BF16 ? 1.f : per_token ? 0.f : __ldg(p.k_scale);
      const float vst = BF16 ? 1.f : per_token ? 0.f : __ldg(p.v_scale);
      const float sl2 = p.scale * kLog2e;
      uint8_t* ring = smem + C::OFF_RING;
      uint32_t stage = 0, phase = 0;
      auto next = [&](uint32_t& st, uint32_t& ph) {
        st = stage;
        ph = phase;
        if (++stage == C::NST) {
          stage = 0;
          phase ^= 1;
        }
      };
      // 8 pages of fp8 rows (128 B, 128-byte swizzled) -> f16 operand rows.  Thread c takes the
      // keys 8 i + (c & 7), i = 0..15, and the 16-dim group q = c / 8 of each: a quarter warp
      // reads one group of eight consecutive keys and writes the two 16-B halves of each result
      // to units (2 (q & 3), 2 (q & 3) + 1) of their swizzled rows, all in different bank groups.
      //   K (is_v false): stage sa holds dims 0..63, sb dims 64..127; row = key (K-major).
      //   V (is_v true):  stage sa holds keys 0..63, sb keys 64..127; inside a stage, dims
      //                   0..63 then 64..127 (8 KB apart), row = key (MN-major).
      const int cq = c >> 3, ck = c & 7;
      const uint32_t su0 = ((2 * (cq & 3)) ^ ck) << 4, su1 = ((2 * (cq & 3) + 1) ^ ck) << 4;
      auto convert = [&](const uint8_t* raw, int kbase, bool is_v, uint32_t sa, uint32_t sb) {
        const uint8_t* src = raw + ck * 128 + ((cq ^ ck) << 4);
        uint8_t* dst_a;
        uint8_t* dst_b;
        if (!is_v) {
          dst_a = dst_b = ring + ((cq >> 2) ? sb : sa) * kStage + ck * 128;
        } else {
          dst_a = ring + sa * kStage + (cq >> 2) * (kStage / 2) + ck * 128;
          dst_b = ring + sb * kStage + (cq >> 2) * (kStage / 2) + ck * 128;
        }
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          uint4 xv = make_uint4(0u, 0u, 0u, 0u);
          if (kbase + 8 * i + ck < P) xv = lds128(src + i * 1024);
          uint32_t w[8];
          e4m3x4_to_f16x2x2(xv.x, w[0], w[1]);
          e4m3x4_to_f16x2x2(xv.y, w[2], w[3]);
          e4m3x4_to_f16x2x2(xv.z, w[4], w[5]);
          e4m3x4_to_f16x2x2(xv.w, w[6], w[7]);
          uint8_t* row = !is_v ? dst_a + i * 1024 : (i < 8 ? dst_a + i * 1024 : dst_b + (i - 8) * 1024);
          sts128(row + su0, make_uint4(w[0], w[1], w[2], w[3]));
          sts128(row + su1, make_uint4(w[4], w[5], w[6], w[7]));
        }
      };
      for (int n = 0; n < nt; ++n) {
        const int kbase = key0 + (lo_t + n) * kTileKeys;
        const int a = n & 1;
        bool ok = wait_bar(&aux_empty[a], ((n >> 1) & 1) ^ 1, ab);
        if (ok && (!BF16 || has_gate)) ok = wait_bar(kr_full, n & 1, ab);
        if (!ok) break;
        // per-key vectors of this tile (zero past the prefix)
        float* ax = reinterpret_cast<float*>(smem + C::OFF_AUX + a * C::AUX);
        for (int k = c; k < kTileKeys; k += 64) {
          const bool valid = kbase + k < P;
          const float ks = per_token ? reinterpret_cast<const float*>(kraw + C::KR_KS)[k] : kst;
          const float vs = per_token ? reinterpret_cast<const float*>(kraw + C::KR_VS)[k] : vst;
          ax[k] = valid ? ks * sl2 : 0.f;
          ax[kTileKeys + k] = valid ? vs * kPrePScale : 0.f;
        }
        if (FEAT) {
          // G_j for the group's G heads: raw pages hold [head][slot], 1 KB apart
          const float* gr = reinterpret_cast<const float*>(kraw + C::KR_G);
          for (int i = c; i < p.group * kTileKeys; i += 64) {
            const int h = i >> 7, k = i & 127;
            ax[2 * kTileKeys + i] = (has_gate && kbase + k < P) ? gr[(k >> 4) * 256 + h * kPage + (k & 15)] : 0.f;
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&aux_full[a]);
          if (BF16 && has_gate) mbar_arrive(kr_empty);
        }
        uint32_t s0, p0, s1, p1, s2, p2, s3, p3;
        next(s0, p0);
        next(s1, p1);
        next(s2, p2);
        next(s3, p3);
        if constexpr (BF16) {
          if (kbase + kTileKeys > P && warp == 2) {  // the last tile
            ok = wait_bar(vr_full, 0, ab);
            if (!ok) break;
            for (int i = lane; i < kTileKeys * 16; i += 32) {
              const int k = i >> 4, u = i & 15;  // key, 16 bytes of it
              if (kbase + k >= P)
                sts128(ring + (k >> 6 ? s3 : s2) * kStage + (u >> 3) * (kStage / 2) + (k & 63) * 128 + (u & 7) * 16,
                       make_uint4(0u, 0u, 0u, 0u));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&full[s2]);
              mbar_arrive(&full[s3]);
            }
          }
        } else {
          ok = wait_bar(&empty[s0], p0 ^ 1, ab) && wait_bar(&empty[s1], p1 ^ 1, ab);
          if (!ok) break;
          convert(kraw, kbase, false, s0, s1);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full[s0]);
            mbar_arrive(&full[s1]);
            mbar_arrive(kr_empty);
          }
          ok = wait_bar(vr_full, n & 1, ab) && wait_bar(&empty[s2], p2 ^ 1, ab) && wait_bar(&empty[s3], p3 ^ 1, ab);
          if (!ok) break;
          convert(vraw, kbase, true, s2, s3);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full[s2]);
            mbar_arrive(&full[s3]);
            mbar_arrive(vr_empty);
          }
        }
      }
    }
    __syncwarp();
  } else {
    reg_inc();
    // ------------------------------------------------------------ softmax, tile x
    const int x = x_of, quarter = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + 128 * x, tO = tmem + lane_off + 256 + 128 * x;
    const int my_first = x ? n_first[1] : n_first[0], my_last = x ? n_last[1] : n_last[0];
    if (my_first <= my_last) {
      // this row of Q into the 128-B-swizzled K-major tile (two 64-dim chunks)
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (size_t)tt * p.q_ts + (size_t)(kvh * G + head) * p.q_hs);
      uint8_t* qs = smem + C::OFF_Q + x * 2 * kStage;
#pragma unroll 4
      for (int u = 0; u < 16; ++u) {
        uint4 f = row_valid ? __ldg(src + u) : make_uint4(0u, 0u, 0u, 0u);
        if (!BF16)
          f = make_uint4(bf16pair_to_f16x2(f.x), bf16pair_to_f16x2(f.y), bf16pair_to_f16x2(f.z),
                         bf16pair_to_f16x2(f.w));
        sts128(qs + (u >> 3) * kStage + rr * 128 + (((u & 7) ^ (rr & 7)) << 4), f);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[x]);
    }
    const bool has_gate = FEAT && p.g_cache != nullptr;
    float gi = 0.f;  // the row's own G
    if (has_gate && row_valid) {
      const int blk = __ldg(p.block_table + (size_t)req * p.max_blocks + lastk / p.block_size);
      gi = __ldg(p.g_cache + ((size_t)blk * p.hq + kvh * G + head) * p.block_size + lastk % p.block_size);
    }
    float m = neg_inf(), l = 0.f;
    const int lk_min = see[2 * x], lk_max = see[2 * x + 1];
    bool ok = true;
    int kx = 0;  // key tiles processed by this query tile
    for (int n = 0; n < nt; ++n) {
      const int a = n & 1;
      ok = wait_bar(&aux_full[a], (n >> 1) & 1, ab);
      if (!ok) break;
      if (n >= my_first && n <= my_last) {
        const int j0 = key0 + (lo_t + n) * kTileKeys;
        ok = wait_bar(&s_full[x], kx & 1, ab);
        if (!ok) break;
        tc_fence_after();
        uint32_t sv[128];
        tmem_ld32(tS + 0, sv);
        tmem_ld32(tS + 32, sv + 32);
        tmem_ld32(tS + 64, sv + 64);
        tmem_ld32(tS + 96, sv + 96);
        tmem_ld_wait();
        const float* ax = reinterpret_cast<const float*>(smem + C::OFF_AUX + a * C::AUX);
        const float4* ks4 = reinterpret_cast<const float4*>(ax);
        const float4* vs4 = reinterpret_cast<const float4*>(ax + kTileKeys);
        const float4* g4 = reinterpret_cast<const float4*>(ax + 2 * kTileKeys + head * kTileKeys);
        const bool need_mask = j0 + kTileKeys > P || j0 + kTileKeys - 1 > lk_min || (W > 0 && j0 < lk_max - W + 1);
        const int jmax = min(lastk, P - 1) - j0;
        const int jmin = W > 0 ? lastk - W + 1 - j0 : -(1 << 30);
        float mxp[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mxp[e] = neg_inf();
#pragma unroll
        for (int j4 = 0; j4 < 32; ++j4) {
          const float4 k4 = ks4[j4];
          const float ks[4] = {k4.x, k4.y, k4.z, k4.w};
          float gs[4] = {0.f, 0.f, 0.f, 0.f};
          if (FEAT) {  // G_i - G_j before the change of units: the difference is what is small
            const float4 g = g4[j4];
            gs[0] = (gi - g.x) * kLog2e;
            gs[1] = (gi - g.y) * kLog2e;
            gs[2] = (gi - g.z) * kLog2e;
            gs[3] = (gi - g.w) * kLog2e;
          }
          float t[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 4 * j4 + e;
            t[e] = FEAT ? fmaf(__uint_as_float(sv[j]), ks[e], gs[e]) : __uint_as_float(sv[j]) * ks[e];
            if (need_mask) t[e] = (j >= jmin && j <= jmax) ? t[e] : neg_inf();
            sv[j] = __float_as_uint(t[e]);
          }
          mxp[(2 * j4) & 7] = fmax3(mxp[(2 * j4) & 7], t[0], t[1]);
          mxp[(2 * j4 + 1) & 7] = fmax3(mxp[(2 * j4 + 1) & 7], t[2], t[3]);
        }
        const float mx = fmax3(fmax3(mxp[0], mxp[1], mxp[2]), fmax3(mxp[3], mxp[4], mxp[5]), fmaxf(mxp[6], mxp[7]));
        const float m_new = fmaxf(m, mx);
        const bool need = m_new > m + kPreLazy;
        if (__any_sync(0xffffffffu, need)) {
          const float alpha = need ? ex2(m - m_new) : 1.f;
          if (kx > 0) {
            // O holds the previous key tiles: wait for their PV before scaling it
            ok = wait_bar(&pv_done[x], (kx - 1) & 1, ab);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < kD / 32; ++cc) {
              uint32_t ov[32];
              tmem_ld32(tO + cc * 32, ov);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
              tmem_st32(tO + cc * 32, ov);
            }
            tmem_st_wait();
          }
          l *= alpha;
          if (need) m = m_new;
        }
        const float mu = (m == neg_inf()) ? 0.f : m;
        float lsp[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) lsp[e] = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int jj = 0; jj < 16; ++jj) {
            const int j = half * 64 + 4 * jj;
            const float4 v4 = vs4[j >> 2];
            const float p0 = ex2(__uint_as_float(sv[j]) - mu), p1 = ex2(__uint_as_float(sv[j + 1]) - mu);
            const float p2 = ex2(__uint_as_float(sv[j + 2]) - mu), p3 = ex2(__uint_as_float(sv[j + 3]) - mu);
            lsp[(2 * jj) & 7] += p0 + p1;
            lsp[(2 * jj + 1) & 7] += p2 + p3;
            // V scales multiply the probabilities after the row sum
            pk[2 * jj] = BF16 ? pack_bf16x2(p0 * v4.x, p1 * v4.y) : pack_f16x2(p0 * v4.x, p1 * v4.y);
            pk[2 * jj + 1] = BF16 ? pack_bf16x2(p2 * v4.z, p3 * v4.w) : pack_f16x2(p2 * v4.z, p3 * v4.w);
          }
          tmem_st32(tS + half * 32, pk);
        }
        l += ((lsp[0] + lsp[1]) + (lsp[2] + lsp[3])) + ((lsp[4] + lsp[5]) + (lsp[6] + lsp[7]));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
        ++kx;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&aux_empty[a]);
    }
    if (ok && kx > 0) ok = wait_bar(&pv_done[x], (kx - 1) & 1, ab);
    if (ok) {
      const size_t at = ((size_t)seg * p.total_q + tt) * p.hq + kvh * G + head;
      if (kx > 0) {
        tc_fence_after();
        float4* arow = reinterpret_cast<float4*>(p.pre_acc + at * kD);
        constexpr float kInv = 1.f / kPrePScale;
#pragma unroll 1
        for (int cc = 0; cc < kD / 32; ++cc) {
          uint32_t ov[32];
          tmem_ld32(tO + cc * 32, ov);
          tmem_ld_wait();
          if (row_valid) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              arow[cc * 8 + j] = make_float4(__uint_as_float(ov[4 * j]) * kInv, __uint_as_float(ov[4 * j + 1]) * kInv,
                                             __uint_as_float(ov[4 * j + 2]) * kInv,
                                             __uint_as_float(ov[4 * j + 3]) * kInv);
          }
        }
      }
      // the combine does not read the accumulators of an empty partial
      if (row_valid) p.pre_ml[at] = kx > 0 ? make_float2(m, l) : make_float2(neg_inf(), 0.f);
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
  const int r = blockIdx.x / p.max_q_len, t = blockIdx.x % p.max_q_len;
  const int kvh = blockIdx.y;
  const int q_begin = __ldg(p.cu_q + r);
  const int ql = __ldg(p.cu_q + r + 1) - q_begin;
  if (t >= ql) return;
  const int L = __ldg(p.seq_lens + r), start = shared_len(p, r);
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
  if (hh < G) {
#pragma unroll 2
    for (int i = sl; i < n; i += SL) {
      float2 v;
      const float4* a;
      if (i < npre) {
        const size_t at = ((size_t)i * p.total_q + q_begin + t) * p.hq + kvh * G + hh;
        v = p.pre_ml[at];
        a = reinterpret_cast<const float4*>(p.pre_acc + at * kD + d0);
      } else {
        const size_t at = (((size_t)r * p.max_segs + s_begin + i - npre) * p.hkv + kvh) * rows + t * G + hh;
        v = reinterpret_cast<const float2*>(p.part_ml)[at];
        a = reinterpret_cast<const float4*>(p.part_acc + at * kD + d0);
      }
      if (v.x == neg_inf()) continue;
      const float4 x0 = a[0], x1 = a[1];
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

template <bool BF16, bool FEAT>
cudaError_t launch_prefix(const DecodeParams& p, const DecodeMaps& maps, cudaStream_t s) {
  using C = PreCfg<BF16, FEAT>;
  auto kern = decode_prefix_kernel<BF16, FEAT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const int rows = 2 * (128 / p.group);  // query rows of one CTA
  const dim3 grid((p.max_group_q + rows - 1) / rows * p.pre_segs, p.hkv, p.num_groups);
  kern<<<grid, kPreThreads, C::SMEM, s>>>(maps.k, maps.v, p);
  return cudaGetLastError();
}

// The tokens behind the prefixes.
cudaError_t launch_behind(const DecodeParams& p, const DecodeMaps& maps, cudaStream_t s) {
  const dim3 grid(p.max_segs, p.hkv, p.num_reqs);
  auto run = [&](auto kern, int smem) -> cudaError_t {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem + 4096 * 4);
    if (e != cudaSuccess) return e;
    kern<<<grid, kThreads, smem + 4096 * p.max_q_len, s>>>(maps.k, maps.v, p);  // + the query fragments
    return cudaGetLastError();
  };
  const bool feat = p.g_cache != nullptr || p.window > 0;
#define GCS_RUN2(KVF, PT, F, SQ)                                                                                    \
  (p.group == 8 ? run(decode_split_kernel<KVF, PT, F, 8, SQ, false, true>, DecCfg<KVF, PT, F, SQ>::SMEM)            \
                : run(decode_split_kernel<KVF, PT, F, 16, SQ, false, true>, DecCfg<KVF, PT, F, SQ>::SMEM))
#define GCS_RUN(KVF, PT, F) (p.max_q_len > 2 ? GCS_RUN2(KVF, PT, F, true) : GCS_RUN2(KVF, PT, F, false))
  if (p.kv_format == 1) return feat ? GCS_RUN(1, false, true) : GCS_RUN(1, false, false);
  if (p.scale_mode == 1) return feat ? GCS_RUN(0, true, true) : GCS_RUN(0, true, false);
  return feat ? GCS_RUN(0, false, true) : GCS_RUN(0, false, false);
#undef GCS_RUN
#undef GCS_RUN2
}

}  // namespace

cudaError_t launch_decode_shared(const DecodeParams& p, const DecodeMaps& maps, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (p.pre_segs > 0) {
    const bool feat = p.g_cache != nullptr || p.window > 0;
    if (p.kv_format == 1) e = feat ? launch_prefix<true, true>(p, maps, s) : launch_prefix<true, false>(p, maps, s);
    else e = feat ? launch_prefix<false, true>(p, maps, s) : launch_prefix<false, false>(p, maps, s);
    if (e != cudaSuccess) return e;
  }
  if (p.max_segs > 0 && (e = launch_behind(p, maps, s)) != cudaSuccess) return e;
  if (p.pre_segs + p.max_segs >= 32) {
    decode_join_kernel<8><<<dim3(p.num_reqs * p.max_q_len, p.hkv, p.group / 2), 256, 0, s>>>(p);
  } else {
    decode_join_kernel<4><<<dim3(p.num_reqs * p.max_q_len, p.hkv, (p.group + 3) / 4), 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace gcs
