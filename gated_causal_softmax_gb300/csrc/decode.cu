// Paged decode / short-query attention over an fp8 e4m3 KV cache with per-token scales.
//
// ROCm/aiter PR #6660 (gfx1250 unified attention), commit messages and "Technical
// details": one fp32 K and V scale per cached token and KV head, laid out [num_blocks,
// num_kv_heads, block_size]; each tile is one page; K scales multiply the QK columns; V
// scales multiply the P columns after the row sum; slots past seq_len get scale 0; the
// context is split into segments (split-K) whose partials are merged by an LSE-weighted
// reduce in which an empty partial (M = -inf) weighs 0.
//
// The split-K kernel is in decode_split.cuh.
// decode_combine_kernel: LSE-weighted merge of the segments of each (query row, head).
#include <mutex>

#include "decode_split.cuh"

namespace gcs {
namespace {

// Fixed scratch for the allocation-free decode entry point: the split-K partials live
// here instead of in a caller-provided workspace.  Every GPU that loads the library
// holds this array until the process exits.
static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];
constexpr int kMaxScratchDevices = 64;
void* g_noalloc_ptr[kMaxScratchDevices] = {nullptr};
std::mutex g_noalloc_mu;

// One CTA per (request x query position, kv head, 16 / SL query heads); 256 threads = 16 / SL
// heads x 16 groups of 8 value dims x SL segment lanes.  The SL lanes of a (head, dims) pair are
// adjacent: each merges every SL-th segment online (their loads are independent), then log2 SL
// shuffle rounds merge them.  SL = 4 for short contexts, 8 from 32 segments on (fewer serial
// merges per lane: 3 x 4 queries at 227K, 114 segments, 20.1 -> 17.5 us per combine; 16 lanes
// measured no better than 4 there, and 16 lanes on 16 segments cost the 64 x 1 call 8 us).
template <int SL>
__global__ void __launch_bounds__(256) decode_combine_kernel(const DecodeParams p) {
  constexpr int kHeads = 16 / SL;  // query heads per CTA
  const int r = blockIdx.x / p.max_q_len, t = blockIdx.x % p.max_q_len;
  const int kvh = blockIdx.y;
  const int q_begin = __ldg(p.cu_q + r);
  const int ql = __ldg(p.cu_q + r + 1) - q_begin;
  if (t >= ql) return;
  const int L = __ldg(p.seq_lens + r);
  const int npages = (L + kPage - 1) / kPage;
  const int nseg = (npages + p.seg_pages - 1) / p.seg_pages;
  const int G = p.group;
  const int sl = threadIdx.x & (SL - 1), dg = (threadIdx.x / SL) & 15;
  const int hh = blockIdx.z * kHeads + threadIdx.x / (16 * SL);
  const int d0 = dg * 8;
  const int rows = p.max_q_len * kRows;
  const int row = t * G + hh;
  auto unit_row = [&](int s) { return ((((size_t)r * p.max_segs + s) * p.hkv + kvh) * rows + row); };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  // segments wholly before every window of the request were not written (see the split kernel)
  const int s_begin = p.window > 0 ? (max(0, L - ql - p.window + 1) / kPage) / p.seg_pages : 0;
  float m = neg_inf(), l = 0.f;
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (hh < G) {
#pragma unroll 2
    for (int s = s_begin + sl; s < nseg; s += SL) {
      const float2 v = ml[unit_row(s)];
      const float4* a = reinterpret_cast<const float4*>(p.part_acc + unit_row(s) * kD + d0);
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
  uint4 outv;
  outv.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  outv.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
  outv.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
  outv.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
  *reinterpret_cast<uint4*>(p.out + (size_t)(q_begin + t) * p.out_ts + (size_t)(kvh * G + hh) * p.out_hs + d0) = outv;
}

}  // namespace

cudaError_t launch_decode(const DecodeParams& p, const DecodeMaps& maps, cudaStream_t s,
                          const cudaEvent_t* ev_before, const cudaEvent_t* ev_after) {
  dim3 g1(p.max_segs, p.hkv, p.num_reqs);
  auto run = [&](auto kern, int smem) -> cudaError_t {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem + 4096 * 4);
    if (e != cudaSuccess) return e;
    if (ev_before && *ev_before) cudaEventRecord(*ev_before, s);
    // + the query fragments: 4 KB per query position
    kern<<<g1, kThreads, smem + 4096 * p.max_q_len, s>>>(maps.k, maps.v, p);
    return cudaGetLastError();
  };
  cudaError_t e;
  // the sink alone needs no change in the split kernel (it is the combine's)
  const bool feat = p.g_cache != nullptr || p.window > 0;
#define GCS_RUN3(KVF, PT, F, SQ, P1)                                                                 \
  (p.group == 8 ? run(decode_split_kernel<KVF, PT, F, 8, SQ, P1>, DecCfg<KVF, PT, F, SQ>::SMEM)       \
                : run(decode_split_kernel<KVF, PT, F, 16, SQ, P1>, DecCfg<KVF, PT, F, SQ>::SMEM))
#define GCS_RUN2(KVF, PT, F, SQ) \
  (p.log2_block_pages == 0 ? GCS_RUN3(KVF, PT, F, SQ, true) : GCS_RUN3(KVF, PT, F, SQ, false))
#define GCS_RUN(KVF, PT, F) (p.max_q_len > 2 ? GCS_RUN2(KVF, PT, F, true) : GCS_RUN2(KVF, PT, F, false))
  if (p.kv_format == 1)
    e = feat ? GCS_RUN(1, false, true) : GCS_RUN(1, false, false);
  else if (p.scale_mode == 1)
    e = feat ? GCS_RUN(0, true, true) : GCS_RUN(0, true, false);
  else
    e = feat ? GCS_RUN(0, false, true) : GCS_RUN(0, false, false);
#undef GCS_RUN
#undef GCS_RUN2
#undef GCS_RUN3
  if (ev_after && *ev_after) cudaEventRecord(*ev_after, s);
  if (e != cudaSuccess) return e;
  return launch_decode_combine(p, s);
}

cudaError_t launch_decode_combine(const DecodeParams& p, cudaStream_t s) {
  if (p.max_segs >= 32) {
    dim3 g2(p.num_reqs * p.max_q_len, p.hkv, p.group / 2);
    decode_combine_kernel<8><<<g2, 256, 0, s>>>(p);
  } else {
    dim3 g2(p.num_reqs * p.max_q_len, p.hkv, (p.group + 3) / 4);
    decode_combine_kernel<4><<<g2, 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

// Device address of the static scratch on the current device.  The first call on a
// device looks the address up (cudaGetSymbolAddress, with that device current); later
// calls reuse it.
cudaError_t decode_noalloc_scratch(void** ptr) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxScratchDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_noalloc_mu);
  if (!g_noalloc_ptr[dev]) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess) return e;
    g_noalloc_ptr[dev] = p;
  }
  *ptr = g_noalloc_ptr[dev];
  return cudaSuccess;
}

}  // namespace gcs
