// The attention weight that cached tokens gather from a call's query rows:
//     w_j <- decay * w_j + sum over rows t and the query heads h of the kv head of exp(s_thj - lse_th),
// with the scores s, masks and sums of exponentials of the paged attention calls.  w_cache is paged
// like the scales.  The tokens that the rows themselves stand for (the last q_len positions) are
// written without the old value.
//
// Two kernels of one walk over the keys: the first leaves (max, sum) of every row and context
// segment, the second joins them to the row's sum, walks the keys again and adds up the weights; with
// the sums given there is only the second.  A warp takes 32 keys a step as the rows of two m16n8k16
// products, the query rows are the columns: a key's weight is then a sum over a thread's own
// accumulators and four lanes.  Key dims go from memory straight to the product's registers (a lane's
// 16 bytes of each 64 dims, the query's dims in the same order).
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "launch.h"
#include "rows.cuh"
#include "sm103_ptx.cuh"

namespace gcs {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStep = 32;  // keys of a warp's step
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ void record_bad(int* status) { atomicCAS(status, kDevOk, kDevInvalidArg); }

__device__ __forceinline__ void e4m3x4_to_f16x2x2(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n"
      " cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  return pack_f16x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Joins (m2, l2) to (m, l): sums of exponentials relative to their maxima (log2 units).
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2) {
  const float M = fmaxf(m, m2);
  l = (m == neg_inf() ? 0.f : l * ex2(m - M)) + (m2 == neg_inf() ? 0.f : l2 * ex2(m2 - M));
  m = M;
}

// NT: blocks of 8 query rows a walk takes; WRITE: the second kernel.
template <bool BF16, int D, int NT, bool WRITE>
__global__ void __launch_bounds__(kThreads) cache_weights_kernel(const WeightsParams p) {
  constexpr int kRows = NT * 8;
  constexpr int kChunks = D / 64;
  extern __shared__ __align__(16) uint8_t smem[];
  uint2* qf = reinterpret_cast<uint2*>(smem);  // [chunk][k-step][row block][lane]
  float* row_g = reinterpret_cast<float*>(smem + (size_t)kChunks * 4 * NT * 32 * sizeof(uint2));
  float* row_sum = row_g + kRows;   // WRITE: the row's sum (log2 units), +inf: no such row
  int* row_last = reinterpret_cast<int*>(row_sum + kRows);  // last key the row sees; -1: none
  int* row_head = row_last + kRows;
  float2* warp_ml = reinterpret_cast<float2*>(row_head + kRows);   // first kernel: [warp][row]
  float* gathered = reinterpret_cast<float*>(row_head + kRows);    // second: [key of the segment]

  // the second kernel takes the requests in the other order: the last ones' keys are still in L2
  const int seg = blockIdx.x, kvh = blockIdx.y, r = WRITE ? gridDim.z - 1 - blockIdx.z : blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  if (!WRITE) grid_release();
  std::conditional_t<WRITE, WaitAtEnd, int> at_end{};  // the second kernel may run beside the first
  (void)at_end;
  const int q0 = __ldg(p.cu_q + r), q1 = __ldg(p.cu_q + r + 1), L = __ldg(p.seq_lens + r);
  const int ql = q1 - q0;
  if (q0 < 0 || q1 < q0 || q1 > p.total_q || ql > p.max_q_len || L < ql || L > p.max_seq_len) {
    if (tid == 0) record_bad(p.status);
    return;
  }
  const int k_begin = seg * p.seg_len, k_end = min(k_begin + p.seg_len, L);
  if (k_begin >= k_end || (ql == 0 && p.decay == 1.f)) return;
  const int left = WRITE && p.first_lens ? max(0, __ldg(p.first_lens + r)) : 0;  // keys that are not written
  if (WRITE && k_end <= left) return;
  const int G = p.group, nrows = ql * G;
  const int32_t* table = p.block_table + (size_t)r * p.max_blocks;
  const bool gates = p.g_cache != nullptr;
  const float sl2 = p.scale * kLog2e;
  const float kst = p.format == kCachePerTensor ? __ldg(p.k_scale) : 1.f;
  auto block_of = [&](int pos) {
    const int blk = __ldg(table + (pos >> p.log2_block));
    if (blk >= 0 && blk < p.num_blocks) return blk;
    record_bad(p.status);
    return -1;
  };
  if (WRITE)
    for (int i = tid; i < p.seg_len; i += kThreads) gathered[i] = 0.f;

  for (int row0 = 0; row0 < nrows; row0 += kRows) {
    const int rows_here = min(kRows, nrows - row0);
    const int last_max = L - ql + (row0 + rows_here - 1) / G;  // last key any of these rows sees
    const int last_min = L - ql + row0 / G;
    const int key_first = max(left, p.window > 0 ? last_min - p.window + 1 : 0);

    // A step's key dims come in units of 128 codes or 64 bf16 dims, one ahead of the products (across the
    // steps too), its blocks another step ahead.  This lane's keys are 16 u + g and 16 u + g + 8.
    constexpr int kUnitChunks = BF16 || kChunks == 1 ? 1 : 2, kUnits = kChunks / kUnitChunks;
    constexpr int kVecs = kUnitChunks * (BF16 ? 2 : 1);
    struct Unit {
      uint4 v[2][2][kVecs];  // [page][key][chunk, or half of its dims]
    };
    struct Keys {
      int blk[2];
      float ks[2][2];
    };
    const uint8_t* k_lane = p.k_cache + (size_t)kvh * p.kv_hs + (size_t)g * p.kv_ss + tq * 16;
    const int key_lo = max(k_begin, key_first & ~(kStep - 1)), key_hi = min(k_end, last_max + 1);
    auto blocks = [&](int key0, int (&blk)[2]) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int pos = key0 + 16 * u;
        blk[u] = key0 < key_hi && pos < L ? block_of(pos) : -1;
      }
    };
    auto load_unit = [&](int key0, const int (&blk)[2], int unit, Unit& x) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int slot = (key0 + 16 * u) & (p.block_size - 1);
        const uint8_t* at = k_lane + (size_t)max(blk[u], 0) * p.kv_bs + (size_t)slot * p.kv_ss +
                            unit * (BF16 ? 128 : 64 * kUnitChunks);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < kVecs; ++i)
            x.v[u][k][i] = blk[u] >= 0 ? __ldg(reinterpret_cast<const uint4*>(at + k * 8 * p.kv_ss + i * 64))
                                       : make_uint4(0, 0, 0, 0);
      }
    };
    auto load_scales = [&](int key0, Keys& x) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        x.ks[u][0] = x.ks[u][1] = kst;
        if (p.format == kCachePerToken && x.blk[u] >= 0) {
          const float* sc = p.k_scale + (((size_t)x.blk[u] * p.hkv + kvh) << p.log2_block) +
                            ((key0 + 16 * u) & (p.block_size - 1)) + g;
          x.ks[u][0] = __ldg(sc);
          x.ks[u][1] = __ldg(sc + 8);
        }
      }
    };
    Keys next;
    Unit cur;
    int ahead[2];
    {
      const int key0 = key_lo + warp * kStep;
      blocks(key0, next.blk);
      blocks(key0 + kWarps * kStep, ahead);
      load_scales(key0, next);
      load_unit(key0, next.blk, 0, cur);
    }
    if (WRITE) grid_wait();  // the first kernel's parts
    __syncthreads();
    // the rows' constants and, in the second kernel, their sums
    for (int i = tid; i < kRows; i += kThreads) {
      const int row = row0 + i, t = row / G, head = row - t * G;
      const bool valid = row < nrows;
      row_head[i] = head;
      row_last[i] = valid ? L - ql + t : -1;
      float gq = 0.f;
      if (gates && valid) {
        const int pos = L - ql + t, blk = block_of(pos);
        if (blk >= 0)
          gq = __ldg(p.g_cache + (((size_t)blk * p.hq + kvh * G + head) << p.log2_block) + (pos & (p.block_size - 1)));
      }
      row_g[i] = gq;
      if (WRITE) {
        float z = __int_as_float(0x7f800000);
        if (valid) {
          const size_t at = (size_t)(q0 + t) * p.hq + kvh * G + head;
          if (p.lse) {
            const float lse = __ldg(p.lse + (size_t)(kvh * G + head) * p.total_q + q0 + t);
            if (lse != neg_inf()) z = lse * kLog2e;
            else row_g[i] = 0.f;  // adds nothing, whatever its elements and its gate are
          } else {
            float m = neg_inf(), l = 0.f;
            const int first = p.window > 0 ? max(0, L - ql + t - p.window + 1) / p.seg_len : 0;
            const int last = (L - ql + t) / p.seg_len;
            for (int s = first; s <= last; s += 8) {  // eight on their way at once
              float2 v[8];
#pragma unroll
              for (int j = 0; j < 8; ++j)
                v[j] = s + j <= last ? p.part[(size_t)(s + j) * p.total_q * p.hq + at] : make_float2(neg_inf(), 0.f);
#pragma unroll
              for (int j = 0; j < 8; ++j) join(m, l, v[j].x, v[j].y);
            }
            if (p.sink) join(m, l, __ldg(p.sink + kvh * G + head) * kLog2e, 1.f);
            if (l != 0.f) z = m + log2f(l);  // 0: a row whose every key lies outside the cache
          }
        }
        row_sum[i] = z;
      }
    }
    // the query rows, as the product's second operand: k-step s of a chunk holds this lane's dims
    // dim0(s) .. + 3 of it
    for (int i = tid; i < kChunks * 4 * NT * 32; i += kThreads) {
      const int ln = i & 31, nt = (i >> 5) % NT, s = (i >> 5) / NT % 4, c = (i >> 5) / NT / 4;
      const int row = row0 + nt * 8 + (ln >> 2), t = row / G, head = row - t * G;
      const int dim = c * 64 + (BF16 ? (s >> 1) * 32 + (ln & 3) * 8 + (s & 1) * 4 : (ln & 3) * 16 + s * 4);
      uint2 v = make_uint2(0, 0);
      // a row without a sum is one of zeros
      const bool valid = row < nrows && !(WRITE && p.lse &&
                                          __ldg(p.lse + (size_t)(kvh * G + head) * p.total_q + q0 + t) == neg_inf());
      if (valid)
        v = __ldg(reinterpret_cast<const uint2*>(p.q + (size_t)(q0 + t) * p.q_ts + (size_t)(kvh * G + head) * p.q_hs + dim));
      if (!BF16) v = make_uint2(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y));
      qf[i] = v;
    }
    __syncthreads();
    float m[NT][2], l[NT][2];
    if (!WRITE) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = neg_inf(), l[nt][0] = l[nt][1] = 0.f;
    }
    for (int key0 = key_lo + warp * kStep; key0 < key_hi; key0 += kWarps * kStep) {
      const int key1 = key0 + kWarps * kStep;  // the warp's next step
      const Keys here = next;
      next.blk[0] = ahead[0], next.blk[1] = ahead[1];
      blocks(key1 + kWarps * kStep, ahead);
      load_scales(key1, next);
      const int(&blk)[2] = here.blk;
      float ks[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) ks[u][0] = here.ks[u][0] * sl2, ks[u][1] = here.ks[u][1] * sl2;
      float acc[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[u][nt][0] = acc[u][nt][1] = acc[u][nt][2] = acc[u][nt][3] = 0.f;
#pragma unroll
      for (int unit = 0; unit < kUnits; ++unit) {
        Unit soon;
        if (unit + 1 < kUnits) load_unit(key0, here.blk, unit + 1, soon);
        else load_unit(key1, next.blk, 0, soon);
#pragma unroll
        for (int cu = 0; cu < kUnitChunks; ++cu) {
          const int c = unit * kUnitChunks + cu;
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t f[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint4 v = cur.v[u][k][BF16 ? s >> 1 : cu];
                if constexpr (BF16) {
                  f[u][k] = s & 1 ? v.z : v.x;
                  f[u][2 + k] = s & 1 ? v.w : v.y;
                } else {
                  e4m3x4_to_f16x2x2(s == 0 ? v.x : s == 1 ? v.y : s == 2 ? v.z : v.w, f[u][k], f[u][2 + k]);
                }
              }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 b = qf[((c * 4 + s) * NT + nt) * 32 + lane];
              mma<BF16>(acc[0][nt], f[0][0], f[0][1], f[0][2], f[0][3], b);
              mma<BF16>(acc[1][nt], f[1][0], f[1][1], f[1][2], f[1][3], b);
            }
          }
        }
        cur = soon;
      }
      const bool inner = key0 + kStep - 1 <= last_min && rows_here == kRows && blk[0] >= 0 && blk[1] >= 0 &&
                         (p.window == 0 || key0 > last_max - p.window);
      float w[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
      // one straight run of code for each case: a branch within it would part the exponentials
      auto columns = [&](auto with_gates, auto masked) {
        constexpr bool kGates = decltype(with_gates)::value, kMask = decltype(masked)::value;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int col = nt * 8 + 2 * tq;
          float x[2][2][2];  // [page][key][column]
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float v = acc[u][nt][2 * k + e] * ks[u][k];
                if (kGates) {
                  const float gk =
                      __ldg(p.g_cache + (((size_t)max(blk[u], 0) * p.hq + kvh * G + row_head[col + e]) << p.log2_block) +
                            ((key0 + 16 * u) & (p.block_size - 1)) + g + 8 * k);
                  v = fmaf(row_g[col + e] - gk, kLog2e, v);
                }
                if (kMask) {
                  const int key = key0 + 16 * u + g + 8 * k, lk = row_last[col + e];
                  v = key > lk || blk[u] < 0 || (p.window > 0 && key <= lk - p.window) ? neg_inf() : v;
                }
                x[u][k][e] = v;
              }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (WRITE) {
              const float z = row_sum[col + e];
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k) w[u][k] += ex2(x[u][k][e] - z);
            } else {
              const float top = fmaxf(fmaxf(x[0][0][e], x[0][1][e]), fmaxf(x[1][0][e], x[1][1][e]));
              const float mn = fmaxf(m[nt][e], top), ref = mn == neg_inf() ? 0.f : mn;
              l[nt][e] = l[nt][e] * ex2(m[nt][e] - ref) + ((ex2(x[0][0][e] - ref) + ex2(x[0][1][e] - ref)) +
                                                           (ex2(x[1][0][e] - ref) + ex2(x[1][1][e] - ref)));
              m[nt][e] = mn;
            }
          }
        }
      };
      if (gates) {
        if (inner) columns(std::true_type(), std::false_type());
        else columns(std::true_type(), std::true_type());
      } else {
        if (inner) columns(std::false_type(), std::false_type());
        else columns(std::false_type(), std::true_type());
      }
      if (WRITE) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            w[u][k] += __shfl_xor_sync(0xffffffffu, w[u][k], 1);
            w[u][k] += __shfl_xor_sync(0xffffffffu, w[u][k], 2);
            // the key's only owner, in every round of rows
            if (tq == 0) gathered[key0 - k_begin + 16 * u + g + 8 * k] += w[u][k];
          }
      }
    }
    if (!WRITE) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            join(m[nt][e], l[nt][e], __shfl_xor_sync(0xffffffffu, m[nt][e], o),
                 __shfl_xor_sync(0xffffffffu, l[nt][e], o));
          if (g == 0) warp_ml[warp * kRows + nt * 8 + 2 * tq + e] = make_float2(m[nt][e], l[nt][e]);
        }
      __syncthreads();
      for (int i = tid; i < rows_here; i += kThreads) {
        float2 v = warp_ml[i];
        for (int k = 1; k < kWarps; ++k) join(v.x, v.y, warp_ml[k * kRows + i].x, warp_ml[k * kRows + i].y);
        const int row = row0 + i, t = row / G, head = row - t * G;
        p.part[(size_t)seg * p.total_q * p.hq + (size_t)(q0 + t) * p.hq + kvh * G + head] = v;
      }
    }
  }
  if (WRITE) {
    __syncthreads();
    // four neighbouring keys a thread, four of those on their way at once
    const int n = k_end - k_begin, fresh = L - ql - k_begin;  // keys from `fresh` on start from 0
    const int skip = left - k_begin;
    for (int i0 = tid * 4; i0 < n; i0 += 4 * 4 * kThreads) {
      float* at[4];
      float old[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * 4 * kThreads, pos = k_begin + i;
        const int blk = i < n && i + 3 >= skip ? block_of(pos) : -1;
        at[j] = blk < 0 ? nullptr : p.w_cache + (((size_t)blk * p.hkv + kvh) << p.log2_block) + (pos & (p.block_size - 1));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (at[j] && p.decay != 0.f && i < fresh) v = *reinterpret_cast<const float4*>(at[j]);
        old[j][0] = v.x, old[j][1] = v.y, old[j][2] = v.z, old[j][3] = v.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * 4 * kThreads;
        if (!at[j]) continue;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = i + e < n ? (p.decay != 0.f && i + e < fresh ? fmaf(p.decay, old[j][e], gathered[i + e]) : gathered[i + e])
                           : 0.f;
        if (i + 3 < n && i >= skip) {
          *reinterpret_cast<float4*>(at[j]) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < n && i + e >= skip) at[j][e] = v[e];
        }
      }
    }
  }
}

template <bool BF16, int D, int NT>
cudaError_t launch_t(const WeightsParams& p, cudaStream_t s) {
  constexpr size_t kFixed = (size_t)(D / 64) * 4 * NT * 32 * 8 + 4 * NT * 8 * 4;
  const dim3 grid(p.segs, p.hkv, p.num_reqs);
  cudaError_t e = cudaSuccess;
  if (!p.lse) {
    constexpr size_t smem = kFixed + kWarps * NT * 8 * 8;
    auto kern = cache_weights_kernel<BF16, D, NT, false>;
    e = allow_smem<cache_weights_kernel<BF16, D, NT, false>>((int)smem);
    if (e != cudaSuccess) return e;
    kern<<<grid, kThreads, smem, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const size_t smem = kFixed + (size_t)p.seg_len * 4;
  auto kern = cache_weights_kernel<BF16, D, NT, true>;
  e = allow_smem<cache_weights_kernel<BF16, D, NT, true>>((int)(kFixed + 4096 * 4));
  if (e != cudaSuccess) return e;
  if (!p.lse) return launch_beside(kern, grid, kThreads, smem, s, p);  // its first keys are on their way by then
  kern<<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}
// Blocks of 8 rows a walk takes: 2 for up to 16 rows of a kv head, 8 for more.  Eight take so many registers that
// an SM holds one block, and 48 rows cost what 64 do, or more (a walk that is not full is masked throughout).  64
// requests of 16K tokens, 4 kv heads of 128, fp8, with 2 and with 8: 16 rows 215 and 731 us, 32 rows 386 (two
// walks) and 731, 48 rows 562 and 732, 64 rows 738 and 526; bf16 366 and 864, 686 and 863, 1006 and 864, 1327
// and 668.  So the border lies too low for 17 to 48 rows; four blocks have not been built.
template <bool BF16, int D>
cudaError_t launch_d(const WeightsParams& p, cudaStream_t s) {
  return (long long)p.max_q_len * p.group <= 16 ? launch_t<BF16, D, 2>(p, s) : launch_t<BF16, D, 8>(p, s);
}
template <bool BF16>
cudaError_t launch_f(const WeightsParams& p, cudaStream_t s) {
  return p.d == 64 ? launch_d<BF16, 64>(p, s) : p.d == 128 ? launch_d<BF16, 128>(p, s)
         : p.d == 256 ? launch_d<BF16, 256>(p, s) : launch_d<BF16, 512>(p, s);
}

}  // namespace

// Context segments: enough blocks for about eight an SM, of 256 to 4096 keys (a block spends a few microseconds
// before its first products: 64 requests up to 32K with 1024, 2048, 4096: 349, 298, 283 us, since then 237).
int cache_weights_segment(int max_seq_len, long long units, int sms) {
  const long long want = (8LL * sms + units - 1) / units;
  long long len = (max_seq_len + want - 1) / want;
  len = std::min(std::max((len + 255) / 256 * 256, 256LL), 4096LL);
  return (int)len;
}

cudaError_t launch_cache_weights(const WeightsParams& p, cudaStream_t s) {
  return p.format == kCacheBf16 ? launch_f<true>(p, s) : launch_f<false>(p, s);
}

}  // namespace gcs
