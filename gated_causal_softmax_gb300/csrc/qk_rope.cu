// Norm of every query and key head with the rotation by position in the same pass, and its
// backward.  For a row x of token t (one head), weights w and the angles of position p_t:
//
//   forward    r = (mean(x^2) + eps)^(-1/2),  y = x r w,  out = R(p_t) y
//   backward   g = R(p_t)^T dout,  dw = sum over tokens and heads of g x r,  u = g w,
//              dx = r (u - x r mean(u x r))
//
// R turns the first rotary_dim elements in pairs; both sums of a row's backward (x^2 and u x)
// are reduced side by side, as mean(u x r) = r mean(u x).
//
// Both are bound by HBM: each element is read once (twice in the backward: x and dout) and
// written once, all arithmetic in fp32 between one load and one rounding to bf16.  Forward of 8192
// tokens of 40 heads of 128 (172 MB): 27.6 us, 6.2 TB/s, 92% of the measured copy rate; of 16384 of 36
// heads of 512 (1.2 GB): 179 us, 100%.  Backward of the first (256 MB): 41.5 us, 91%, of which 2.5 are
// the kernel that adds up the weights' gradients.
#include <algorithm>

#include "kernels.h"
#include "rows.cuh"

namespace gcs {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Rows of a lane group in a step, and blocks of an SM: warps take further tokens beyond
// 152 SMs full.  16384 x 36 heads of 512 forward: 179 us with 3, 193 with 4; 8192 x 40 of 128: 28.9 and
// 27.6, 38 with 5 (spills).  Backward of the latter with 1 row: 47.0 with 3 blocks, 45.1 with 4; with 2
// rows 41.5 with 3, 46.4 with 4 (spills).
constexpr int kFwdRows = 2, kBwdRows = 2;
template <int D>
constexpr int kFwdBlocks = D == 512 ? 3 : 4;
constexpr int kBwdBlocks = 3;

// A warp's share: heads [h0, h1) of the queries or of the keys, and every step-th token.
struct Share {
  bool is_k;
  int h0, h1;
  uint32_t t, step;
};
template <int H>  // heads of a share
__device__ __forceinline__ bool warp_share(int hq, int hkv, Share& s) {
  const int q_segs = (hq + H - 1) / H, segs = q_segs + (hkv + H - 1) / H;
  const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5), warps = gridDim.x * kWarps;
  s.step = warps / segs;
  if (w >= s.step * segs) return false;
  const int seg = w % segs;
  s.is_k = seg >= q_segs;
  s.h0 = (s.is_k ? seg - q_segs : seg) * H;
  s.h1 = min(s.h0 + H, s.is_k ? hkv : hq);
  s.t = w / segs;
  return true;
}
int blocks_for(int total, int hq, int hkv, int H, int most) {
  const int segs = (hq + H - 1) / H + (hkv + H - 1) / H;
  const long long blocks = ((long long)total * segs + kWarps - 1) / kWarps;
  // at least one warp for each share of heads
  return (int)std::max<long long>(std::min<long long>(blocks, most), (segs + kWarps - 1) / kWarps);
}

// Positions of the steps ahead.
__device__ __forceinline__ int position_of(const RopeParams& p, uint32_t t) {
  return p.positions && t < (uint32_t)p.total ? __ldg(p.positions + t) : 0;
}
// False for a token to leave out (negative: padding; past the table: an error).
__device__ __forceinline__ bool token_used(const RopeParams& p, int pos) {
  if (pos < 0) return false;
  if (p.cos_sin && pos >= p.max_pos) {
    if ((threadIdx.x & 31) == 0) atomicCAS(p.status, kDevOk, kDevInvalidArg);
    return false;
  }
  return true;
}

// Runs through a warp's tokens with the copies of the next one under way: fetch(stage, t) starts the
// copies of a token's rows, use(stage, t, used) works on them.
template <int D, int ROWS, typename Fetch, typename Use>
__device__ __forceinline__ void for_tokens(const RopeParams& p, const Share& s, WarpStage<D, ROWS>* ring, Fetch fetch,
                                           Use use) {
  const uint32_t total = p.total;
  auto start = [&](int slot, uint32_t t, int pos) {
    if (t < total) {
      fetch(ring[slot], t);
      if (p.cos_sin && pos >= 0 && pos < p.max_pos) fetch_angles(ring[slot].angles[0], p.cos_sin, pos, p.rotary_dim);
    }
    copy_commit();
  };
  int pos = position_of(p, s.t), next = position_of(p, s.t + s.step);
  start(0, s.t, pos);
  int slot = 0;
  for (uint32_t t = s.t; t < total; t += s.step, slot ^= 1) {
    start(slot ^ 1, t + s.step, next);
    const int after = position_of(p, t + 2 * s.step);
    copy_wait<1>();
    __syncwarp();
    use(ring[slot], t, token_used(p, pos));
    __syncwarp();
    pos = next;
    next = after;
  }
}

// BACK: the gradient without the norm, which is the rotation back of dout (p.q_out, p.k_out) into dx.
template <int D, bool BACK>
__global__ void __launch_bounds__(kThreads, kFwdBlocks<D>) norm_rope_fwd_kernel(const RopeParams p) {
  constexpr int L = RowLanes<D>::kLanes, R = RowLanes<D>::kRows, U = kFwdRows;
  __shared__ WarpStage<D, U> ring[kWarps][2];
  Share s;
  if (!warp_share<R * U>(p.hq, p.hkv, s)) return;
  const int sub = threadIdx.x & (L - 1), grp = (threadIdx.x & 31) / L;
  const RowRuns runs = row_runs<D>(sub, p.rotary_dim, p.interleaved);
  const uint16_t* in = BACK ? s.is_k ? p.k_out : p.q_out : s.is_k ? p.k : p.q;
  uint16_t* out = BACK ? s.is_k ? p.dk : p.dq : s.is_k ? p.k_out : p.q_out;
  const long long its = BACK ? s.is_k ? p.ko_ts : p.qo_ts : s.is_k ? p.k_ts : p.q_ts;
  const long long ihs = BACK ? s.is_k ? p.ko_hs : p.qo_hs : s.is_k ? p.k_hs : p.q_hs;
  const long long ots = BACK ? s.is_k ? p.dk_ts : p.dq_ts : s.is_k ? p.ko_ts : p.qo_ts;
  const long long ohs = BACK ? s.is_k ? p.dk_hs : p.dq_hs : s.is_k ? p.ko_hs : p.qo_hs;
  const Row w = load_weights(s.is_k ? p.k_weight : p.q_weight, runs);
  auto fetch = [&](WarpStage<D, U>& st, uint32_t t) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = s.h0 + u * R + grp;
      const bool valid = h < s.h1;
      fetch_row(st, u, in + t * its + (valid ? h : s.h0) * ihs, runs, valid);
    }
  };
  auto use = [&](const WarpStage<D, U>& st, uint32_t t, bool used) {
    if (!used && !BACK) return;
    const Angles ang = read_angles<BACK>(st.angles[0], p.rotary_dim, runs);
    Row x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = BACK && !used ? zero_row() : unpack_row(fetched_row(st, u));
    if (!BACK)
      norm_rotate_rows<D>(x, w, runs, ang, p.norm, p.eps, p.interleaved);
    else if (used)  // else the row's output does not depend on it
      rotate_rows(x, runs, ang, p.interleaved);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = s.h0 + u * R + grp;
      if (h < s.h1) store_row(out + t * ots + h * ohs, runs, x[u]);
    }
  };
  for_tokens(p, s, ring[threadIdx.x >> 5], fetch, use);
}

// The backward with the norm, and the gradients of its weights: every lane sums g x r of its 16
// elements over its rows, the lanes of a block with the same elements are added in a fixed order, and
// the block writes its part of d q_weight and d k_weight to p.partials [blocks][2][D];
// weight_grad_kernel adds those.
template <int D>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) norm_rope_bwd_kernel(const RopeParams p) {
  constexpr int L = RowLanes<D>::kLanes, R = RowLanes<D>::kRows;
  constexpr int U = kBwdRows;
  using Stage = WarpStage<D, 2 * U>;
  __shared__ union {
    Stage ring[kWarps][2];
    struct {
      float dw[kWarps][D];
      int of[kWarps];  // of the queries 0, the keys 1, none 2
    } part;  // after the last step
  } sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = threadIdx.x & (L - 1), grp = lane / L;
  const RowRuns runs = row_runs<D>(sub, p.rotary_dim, p.interleaved);
  Share s;
  Row dw = zero_row();
  const bool works = warp_share<R * U>(p.hq, p.hkv, s);
  if (works) {
    const uint16_t* in = s.is_k ? p.k : p.q;
    const uint16_t* dout = s.is_k ? p.k_out : p.q_out;
    uint16_t* dx = s.is_k ? p.dk : p.dq;
    const long long its = s.is_k ? p.k_ts : p.q_ts, ihs = s.is_k ? p.k_hs : p.q_hs;
    const long long ots = s.is_k ? p.ko_ts : p.qo_ts, ohs = s.is_k ? p.ko_hs : p.qo_hs;
    const long long dts = s.is_k ? p.dk_ts : p.dq_ts, dhs = s.is_k ? p.dk_hs : p.dq_hs;
    const Row w = load_weights(s.is_k ? p.k_weight : p.q_weight, runs);
    auto fetch = [&](Stage& st, uint32_t t) {
#pragma unroll
      for (int n = 0; n < U; ++n) {
        const int head = s.h0 + n * R + grp;
        const bool valid = head < s.h1;
        const int h = valid ? head : s.h0;
        fetch_row(st, 2 * n, dout + t * ots + h * ohs, runs, valid);
        fetch_row(st, 2 * n + 1, in + t * its + h * ihs, runs, valid);
      }
    };
    auto use = [&](const Stage& st, uint32_t t, bool used) {
      const Angles ang = read_angles<true>(st.angles[0], p.rotary_dim, runs);
#pragma unroll
      for (int n = 0; n < U; ++n) {
        const int h = s.h0 + n * R + grp;
        const bool valid = h < s.h1;
        Row gs[1] = {zero_row()}, &g = gs[0];
        if (used) {
          g = unpack_row(fetched_row(st, 2 * n));
          rotate_rows(gs, runs, ang, p.interleaved);
          Row x = unpack_row(fetched_row(st, 2 * n + 1)), u;
          float2 xx = both(0.f), ux = both(0.f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            u.e[i] = mul2(g.e[i], w.e[i]);
            xx = fma2(x.e[i], x.e[i], xx);
            ux = fma2(u.e[i], x.e[i], ux);
          }
          float sums[2] = {xx.x + xx.y, ux.x + ux.y};
          row_sums<L>(sums);
          // the idle lanes' rows of zeros would have r = inf with eps = 0, and be a NaN in the sum
          const float r = valid ? rsqrtf(fmaf(sums[0], 1.f / D, p.eps)) : 0.f;
          const float m = sums[1] * r * (1.f / D);  // mean(u x r)
          const float2 r2 = both(r), m2 = both(-m * r);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x.e[i] = mul2(x.e[i], r2);
            dw.e[i] = fma2(g.e[i], x.e[i], dw.e[i]);
            g.e[i] = fma2(x.e[i], m2, mul2(u.e[i], r2));
          }
        }
        if (valid) store_row(dx + t * dts + h * dhs, runs, g);
      }
    };
    for_tokens(p, s, sm.ring[warp], fetch, use);
  }
  if (!p.partials) return;
  grid_release();
#pragma unroll
  for (int off = L; off < 32; off <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw.e[i].x += __shfl_xor_sync(kFullMask, dw.e[i].x, off);
      dw.e[i].y += __shfl_xor_sync(kFullMask, dw.e[i].y, off);
    }
  __syncthreads();  // the ring is done with
  if (grp == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *reinterpret_cast<float2*>(&sm.part.dw[warp][runs.a + 2 * i]) = dw.e[i];
      *reinterpret_cast<float2*>(&sm.part.dw[warp][runs.b + 2 * i]) = dw.e[4 + i];
    }
  }
  if (lane == 0) sm.part.of[warp] = works ? (s.is_k ? 1 : 0) : 2;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
    const int of = c / D;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i)
      if (sm.part.of[i] == of) sum += sm.part.dw[i][c % D];
    p.partials[(size_t)blockIdx.x * 2 * D + c] = sum;
  }
}

// dw of 16 columns a block: 64 threads a column add every 64th block's part, then their sums.
constexpr int kGradCols = 16, kGradRows = 64;
__global__ void __launch_bounds__(kGradCols * kGradRows) weight_grad_kernel(const float* partials, int blocks, int d,
                                                                             float* dq_weight, float* dk_weight) {
  __shared__ float sm[kGradRows][kGradCols + 1];
  const int x = threadIdx.x % kGradCols, y = threadIdx.x / kGradCols;
  float sum = 0.f;
  grid_wait();
#pragma unroll 5
  for (int b = y; b < blocks; b += kGradRows) sum += __ldcg(partials + (size_t)b * 2 * d + blockIdx.x * kGradCols + x);
  sm[y][x] = sum;
  __syncthreads();
  const int lane = threadIdx.x & 31, c = threadIdx.x >> 5;  // a warp a column
  if (c >= kGradCols) return;
  sum = sm[lane][c] + sm[lane + 32][c];
#pragma unroll
  for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(kFullMask, sum, off);
  if (lane == 0) {
    const int col = blockIdx.x * kGradCols + c;
    float* dst = col < d ? dq_weight : dk_weight;
    if (dst) dst[col < d ? col : col - d] = sum;
  }
}

int bwd_blocks(const RopeParams& p) {
  return blocks_for(p.total, p.hq, p.hkv, 512 / p.d * kBwdRows, 152 * kBwdBlocks);
}

template <int D, bool BACK>
cudaError_t fwd(const RopeParams& p, cudaStream_t s) {
  const int blocks = blocks_for(p.total, p.hq, p.hkv, RowLanes<D>::kRows * kFwdRows, 152 * kFwdBlocks<D>);
  norm_rope_fwd_kernel<D, BACK><<<blocks, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t bwd(const RopeParams& p, float* dq_weight, float* dk_weight, cudaStream_t s) {
  if (!p.norm) return fwd<D, true>(p, s);
  const int blocks = bwd_blocks(p);
  norm_rope_bwd_kernel<D><<<blocks, kThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.partials) return e;
  return launch_behind(weight_grad_kernel, 2 * D / kGradCols, kGradCols * kGradRows, s, p.partials, blocks, D,
                       dq_weight, dk_weight);
}

}  // namespace

size_t norm_rope_bwd_partials(const RopeParams& p) {
  return (size_t)bwd_blocks(p) * 2 * p.d;
}

cudaError_t launch_norm_rope_fwd(const RopeParams& p, cudaStream_t s) {
  switch (p.d) {
    case 64: return fwd<64, false>(p, s);
    case 128: return fwd<128, false>(p, s);
    case 256: return fwd<256, false>(p, s);
    default: return fwd<512, false>(p, s);
  }
}

cudaError_t launch_norm_rope_bwd(const RopeParams& p, float* dq_weight, float* dk_weight, cudaStream_t s) {
  switch (p.d) {
    case 64: return bwd<64>(p, dq_weight, dk_weight, s);
    case 128: return bwd<128>(p, dq_weight, dk_weight, s);
    case 256: return bwd<256>(p, dq_weight, dk_weight, s);
    default: return bwd<512>(p, dq_weight, dk_weight, s);
  }
}

}  // namespace gcs
