// C ABI: host-side validation, workspace carving, TMA descriptor encoding and launches.
// Nothing here allocates device memory or synchronises (except gcs_get_device_status,
// which is a synchronous query by design).
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/gcs_attn.h"
#include "kernels.h"
#include "launch.h"

namespace gcs {

__device__ int g_device_status = 0;

namespace {

constexpr int kMaxDevices = 64;
int* g_status_ptr[kMaxDevices] = {nullptr};
std::mutex g_mu;

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// gcs_set_device_checks: every call first checks its index arrays on the device
std::atomic<int> g_device_checks{0};
bool device_checks_on() { return g_device_checks.load(std::memory_order_relaxed) != 0; }

// events armed by gcs_set_kernel_events for the next call of this thread
thread_local cudaEvent_t t_ev_before = nullptr, t_ev_after = nullptr;

struct KernelTimer {
  cudaStream_t s;
  cudaEvent_t b, a;
  explicit KernelTimer(cudaStream_t st) : s(st), b(t_ev_before), a(t_ev_after) {
    t_ev_before = t_ev_after = nullptr;
  }
  void before() const {
    if (b) cudaEventRecord(b, s);
  }
  void after() const {
    if (a) cudaEventRecord(a, s);
  }
};
std::once_flag g_encode_once;

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode;
}

// Element strides (token, head) of a [tokens, heads, dim] tensor with dim contiguous.
struct Layout {
  long long ts, hs;
};

// 3-D bf16 map {dim, heads, tokens} with a 64 x 1 x box_rows box and 128-byte swizzle: one
// box is 64 columns of one head for box_rows tokens, the same shared-memory tile as a 2-D box.
bool make_map(CUtensorMap* m, const void* base, int dim, int heads, int tokens, const Layout& l, uint32_t box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)l.hs * 2, (cuuint64_t)l.ts * 2};
  cuuint32_t box[3] = {64, 1, box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D fp32 map {dim, heads, tokens} of a contiguous [tokens, heads, dim] accumulator with a
// 32 x 1 x box_rows box and the 128-byte swizzle: the target of tiled reduce-adds.
bool make_map_f32(CUtensorMap* m, void* base, int dim, int heads, int tokens, uint32_t box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)dim * 4, (cuuint64_t)dim * heads * 4};
  cuuint32_t box[3] = {32, 1, box_rows};  // 32 fp32 = one 128-byte swizzle row
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Byte strides (block, kv head, slot) of a paged cache.
struct CacheLayout {
  long long bs, hs, ss;
  bool head_inner() const { return hs < ss; }
};

// 4-D byte map of a paged fp8 cache, dims in increasing stride order: {128 B, slot, kv head,
// block}, or {128 B, kv head, slot, block} when the kv head is the inner one.  One box is one
// 16-slot page of one kv head (16 x 128 B, 128-byte swizzle), the same tile either way.
bool make_page_map_u8(CUtensorMap* m, const void* base, int num_blocks, int hkv, int block_size,
                      const CacheLayout& l) {
  auto enc = encode_fn();
  if (!enc) return false;
  const bool hi = l.head_inner();
  cuuint64_t dims[4] = {128, (cuuint64_t)(hi ? hkv : block_size), (cuuint64_t)(hi ? block_size : hkv),
                        (cuuint64_t)num_blocks};
  cuuint64_t strides[3] = {(cuuint64_t)(hi ? l.hs : l.ss), (cuuint64_t)(hi ? l.ss : l.hs), (cuuint64_t)l.bs};
  cuuint32_t box[4] = {128, hi ? 1u : 16u, hi ? 16u : 1u, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same of a bf16 cache with head dim d: one box is 64 dims of a page (16 rows of 128 bytes).
bool make_page_map_bf16(CUtensorMap* m, const void* base, int num_blocks, int hkv, int block_size, int d,
                        const CacheLayout& l) {
  auto enc = encode_fn();
  if (!enc) return false;
  const bool hi = l.head_inner();
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)(hi ? hkv : block_size), (cuuint64_t)(hi ? block_size : hkv),
                        (cuuint64_t)num_blocks};
  cuuint64_t strides[3] = {(cuuint64_t)(hi ? l.hs : l.ss), (cuuint64_t)(hi ? l.ss : l.hs), (cuuint64_t)l.bs};
  cuuint32_t box[4] = {64, hi ? 1u : 16u, hi ? 16u : 1u, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D 16-bit map {dim, heads, tokens} whose box is 64 dims of `group` heads of `box_tokens` tokens: rows in
// the order (token, head), 128-byte swizzle.
bool make_query_map(CUtensorMap* m, const void* base, bool f16, int dim, int heads, int tokens, const Layout& l,
                    int group, int box_tokens) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)l.hs * 2, (cuuint64_t)l.ts * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)box_tokens};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t round_up(size_t x) { return (x + 255) & ~size_t(255); }

// Byte range [a, b) of a caller buffer; a null pointer is an empty range.
struct Span {
  uintptr_t a, b;
};
Span span(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, p ? a + bytes : a};
}
// A strided token-major tensor: byte range plus the period (token stride in bytes) and the
// bytes one token covers; period 0 = one dense range.
struct TSpan {
  uintptr_t a, b;
  unsigned long long period, width;
};
TSpan tspan(const void* p, int tokens, int heads, int dim, const Layout& l, int elt) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (!p || tokens <= 0) return TSpan{a, a, 0, 0};
  const unsigned long long w = ((unsigned long long)(heads - 1) * l.hs + dim) * elt;
  return TSpan{a, a + (unsigned long long)(tokens - 1) * l.ts * elt + w, (unsigned long long)l.ts * elt, w};
}
TSpan tspan(const Span& s) { return TSpan{s.a, s.b, 0, 0}; }
// True when two byte sets meet.  Two tensors with the same token period whose per-token ranges
// sit side by side within every period (heads of one fused buffer) do not.
bool overlap(const TSpan& x, const TSpan& y) {
  if (!(x.a < x.b && y.a < y.b && x.a < y.b && y.a < x.b)) return false;
  if (x.period != 0 && x.period == y.period && x.width <= x.period && y.width <= y.period) {
    const unsigned long long P = x.period;
    const unsigned long long d = (unsigned long long)((y.a >= x.a ? y.a - x.a : P - (x.a - y.a) % P) % P);
    return !(d >= x.width && d + y.width <= P);
  }
  return true;
}

// True when an output range overlaps an input range or another output range (kernels read
// their inputs and write their outputs concurrently, so any overlap is a race).
template <size_t NO, size_t NI>
bool outputs_overlap(const TSpan (&outs)[NO], const TSpan (&ins)[NI]) {
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (size_t j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

// Carves consecutive 256-B aligned regions out of a workspace.
struct Carver {
  uint8_t* base;
  size_t off = 0;
  template <typename T>
  T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += round_up(count * sizeof(T));
    return p;
  }
};

// {0, 0} = contiguous; otherwise token-major without overlap, 16-byte granules.
int resolve_layout(const gcs_strides& st, int heads, int dim, Layout* out) {
  if (st.token == 0 && st.head == 0) {
    *out = Layout{(long long)heads * dim, dim};
    return GCS_OK;
  }
  if (st.token < 0 || st.head < 0) return GCS_ERR_INVALID_ARG;
  if (st.head < dim || st.token < (long long)heads * st.head) return GCS_ERR_UNSUPPORTED;
  if ((st.head % 8) != 0 || (st.token % 8) != 0) return GCS_ERR_UNSUPPORTED;
  if (st.token > (1LL << 38)) return GCS_ERR_UNSUPPORTED;  // tensor-copy strides stay below 2^40 bytes
  *out = Layout{st.token, st.head};
  return GCS_OK;
}

struct PrefillLayouts {
  Layout q, k, v, o, dout, dq, dk, dv;
};

int prefill_layouts(const gcs_prefill_args* a, PrefillLayouts* l) {
  int st;
  if ((st = resolve_layout(a->q_stride, a->hq, a->dqk, &l->q)) != GCS_OK) return st;
  if ((st = resolve_layout(a->k_stride, a->hkv, a->dqk, &l->k)) != GCS_OK) return st;
  if ((st = resolve_layout(a->v_stride, a->hkv, a->dv, &l->v)) != GCS_OK) return st;
  if ((st = resolve_layout(a->o_stride, a->hq, a->dv, &l->o)) != GCS_OK) return st;
  if ((st = resolve_layout(a->do_stride, a->hq, a->dv, &l->dout)) != GCS_OK) return st;
  if ((st = resolve_layout(a->dq_stride, a->hq, a->dqk, &l->dq)) != GCS_OK) return st;
  if ((st = resolve_layout(a->dk_stride, a->hkv, a->dqk, &l->dk)) != GCS_OK) return st;
  return resolve_layout(a->dv_stride, a->hkv, a->dv, &l->dv);
}

bool supported_dims(int dqk, int dv) {
  return (dqk == 64 && dv == 64) || (dqk == 128 && dv == 128) || (dqk == 256 && dv == 256) ||
         (dqk == 256 && dv == 512) || (dqk == 512 && dv == 512);
}

int check_prefill(const gcs_prefill_args* a) {
  if (!a) return GCS_ERR_INVALID_ARG;
  if (a->num_seqs < 1 || a->total_tokens < 1 || a->max_seqlen < 1 || a->hq < 1 || a->hkv < 1)
    return GCS_ERR_INVALID_ARG;
  if (a->hq % a->hkv != 0) return GCS_ERR_INVALID_ARG;
  if (a->window < 0) return GCS_ERR_INVALID_ARG;
  if (a->deterministic != 0 && a->deterministic != 1) return GCS_ERR_INVALID_ARG;
  if (!std::isfinite(a->scale)) return GCS_ERR_INVALID_ARG;
  if (!a->cu_seqlens || !a->q || !a->k || !a->v) return GCS_ERR_INVALID_ARG;
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v)) return GCS_ERR_INVALID_ARG;
  if ((a->log_gate && !aligned16(a->log_gate)) || (a->sink && (reinterpret_cast<uintptr_t>(a->sink) & 3u)))
    return GCS_ERR_INVALID_ARG;
  if (!supported_dims(a->dqk, a->dv)) return GCS_ERR_UNSUPPORTED;
  // 32-bit element counts of the contiguous fp32 workspaces and in-kernel indices: keep every
  // tensor below 2^31 elements
  const double big = 2147483647.0;
  if ((double)a->total_tokens * a->hq * (a->dqk > a->dv ? a->dqk : a->dv) > big) return GCS_ERR_UNSUPPORTED;
  PrefillLayouts l;
  return prefill_layouts(a, &l);
}

// Byte ranges of a prefill call's inputs: q, k, v, log_gate, sink, cu_seqlens.
struct PrefillSpans {
  TSpan q, k, v, g, s, cu;
};
PrefillSpans prefill_spans(const gcs_prefill_args* a, const PrefillLayouts& l) {
  const size_t t = (size_t)a->total_tokens;
  const int T = a->total_tokens;
  return PrefillSpans{tspan(a->q, T, a->hq, a->dqk, l.q, 2),         tspan(a->k, T, a->hkv, a->dqk, l.k, 2),
                      tspan(a->v, T, a->hkv, a->dv, l.v, 2),         tspan(span(a->log_gate, t * a->hq * 4)),
                      tspan(span(a->sink, (size_t)a->hq * 4)), tspan(span(a->cu_seqlens, ((size_t)a->num_seqs + 1) * 4))};
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? GCS_OK : GCS_ERR_CUDA; }

int* status_ptr_for_current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_status_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return nullptr;
    g_status_ptr[dev] = static_cast<int*>(p);
  }
  return g_status_ptr[dev];
}

// With device checks on, every workspace ends with the checked copy of cu_seqlens / cu_q.
size_t fwd_ws(const gcs_prefill_args* a, bool chk) {
  Carver c{nullptr};
  if (a->log_gate) c.take<float>((size_t)a->hq * a->total_tokens);
  if (chk) c.take<int32_t>((size_t)a->num_seqs + 1);
  return c.off;
}

// Head dim 128 without `deterministic` takes the single-pass backward (dQ reduce-added into an
// fp32 buffer); head dim 64, and 128 with `deterministic`, the two-pass backward (dQ pass +
// dK/dV pass, no fp32 dQ buffer); wider heads the output-column roles below.
bool fused(const gcs_prefill_args* a) { return a->dqk == 128 && a->dv == 128 && a->deterministic == 0; }
bool two_pass(const gcs_prefill_args* a) { return a->dqk <= 128 && a->dv <= 128 && !fused(a); }

// Head dims above 128 take the query-stationary dQ pass when asked for a deterministic result,
// and where it is also the faster route (Dqk = 512, where the reduce-add role's 64-row steps
// cost more than the dQ pass's recompute); otherwise the dK role reduce-adds dQ in fp32.
bool wide_two_pass(const gcs_prefill_args* a) { return a->deterministic != 0 || a->dqk == 512; }

size_t bwd_ws(const gcs_prefill_args* a, bool chk) {
  Carver c{nullptr};
  const size_t ht = (size_t)a->hq * a->total_tokens;
  if (a->log_gate) c.take<float>(ht);                         // G^T
  c.take<float>(ht);                                           // delta
  if (fused(a) || (a->dqk > 128 && !wide_two_pass(a)))
    c.take<float>((size_t)a->total_tokens * a->hq * a->dqk);  // dQ accumulator
  if (a->log_gate || a->sink) c.take<float>(ht);               // row sums of dS
  if (a->log_gate) c.take<float>(ht);                          // column sums of dS
  c.take<float>((size_t)a->hq * ((a->total_tokens + 63) / 64 + a->num_seqs) * 128);  // packed vectors
  if (chk) c.take<int32_t>((size_t)a->num_seqs + 1);
  return c.off;
}

}  // namespace

int* device_status_ptr() { return status_ptr_for_current_device(); }

}  // namespace gcs

using namespace gcs;

extern "C" {

const char* gcs_status_str(int s) {
  switch (s) {
    case GCS_OK: return "ok";
    case GCS_ERR_INVALID_ARG: return "invalid argument";
    case GCS_ERR_UNSUPPORTED: return "unsupported shape, dtype or layout";
    case GCS_ERR_WORKSPACE: return "workspace missing or too small";
    case GCS_ERR_CUDA: return "CUDA error";
    case GCS_ERR_DEVICE_TIMEOUT: return "a kernel gave up on a bounded wait";
    default: return "unknown status";
  }
}

const char* gcs_version(void) { return "gcs_attn 0.1 (sm_103a)"; }

size_t attn_fwd_workspace(const gcs_prefill_args* a) {
  return (a && check_prefill(a) == GCS_OK) ? fwd_ws(a, device_checks_on()) : 0;
}

size_t attn_bwd_workspace(const gcs_prefill_args* a) {
  return (a && check_prefill(a) == GCS_OK) ? bwd_ws(a, device_checks_on()) : 0;
}

int attn_fwd(const gcs_prefill_args* a, void* o, float* lse, void* workspace, size_t workspace_bytes,
             gcs_stream_t stream) {
  int st = check_prefill(a);
  if (st != GCS_OK) return st;
  if (!o || !lse || !aligned16(o) || !aligned16(lse)) return GCS_ERR_INVALID_ARG;
  PrefillLayouts lay;
  prefill_layouts(a, &lay);
  {
    const size_t t = (size_t)a->total_tokens;
    const PrefillSpans in = prefill_spans(a, lay);
    const TSpan outs[] = {tspan(o, a->total_tokens, a->hq, a->dv, lay.o, 2), tspan(span(lse, t * a->hq * 4))};
    const TSpan ins[] = {in.q, in.k, in.v, in.g, in.s, in.cu};
    if (outputs_overlap(outs, ins)) return GCS_ERR_INVALID_ARG;
  }
  const bool chk = device_checks_on();
  const size_t need = fwd_ws(a, chk);
  if (need > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
    return GCS_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int* status = device_status_ptr();
  if (!status) return GCS_ERR_CUDA;

  Carver c{static_cast<uint8_t*>(workspace)};
  float* gT = a->log_gate ? c.take<float>((size_t)a->hq * a->total_tokens) : nullptr;
  int32_t* cu_chk = chk ? c.take<int32_t>((size_t)a->num_seqs + 1) : nullptr;

  FwdMaps maps;
  if (!make_map(&maps.q, a->q, a->dqk, a->hq, a->total_tokens, lay.q, 128) ||
      !make_map(&maps.k, a->k, a->dqk, a->hkv, a->total_tokens, lay.k, 128) ||
      !make_map(&maps.v, a->v, a->dv, a->hkv, a->total_tokens, lay.v, 128))
    return GCS_ERR_CUDA;

  // the kernels read the checked copy of cu_seqlens when device checks are on
  const int32_t* cu = a->cu_seqlens;
  if (cu_chk) {
    st = cuda_status(launch_check_prefill(a->cu_seqlens, a->num_seqs, a->total_tokens, a->max_seqlen, cu_chk, status, s));
    if (st != GCS_OK) return st;
    cu = cu_chk;
  }
  if (gT) {
    st = cuda_status(launch_gate_cumsum(a->log_gate, cu, a->num_seqs, a->total_tokens, a->hq, gT, s));
    if (st != GCS_OK) return st;
  }
  FwdParams p;
  p.cu_seqlens = cu;
  p.num_seqs = a->num_seqs;
  p.total = a->total_tokens;
  p.hq = a->hq;
  p.hkv = a->hkv;
  p.dqk = a->dqk;
  p.dv = a->dv;
  p.dv_chunk = a->dv > 256 ? 256 : a->dv;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.window = a->window;
  p.gT = gT;
  p.sink = a->sink;
  p.o = static_cast<uint16_t*>(o);
  p.o_ts = lay.o.ts;
  p.o_hs = lay.o.hs;
  p.lse = lse;
  p.status = status;
  KernelTimer timer(s);
  timer.before();
  if (a->dqk == a->dv && a->dqk <= 128) {
    st = cuda_status(launch_prefill_fwd2(p, maps, s));
  } else {
    const int num_tiles = (a->total_tokens + 127) / 128 + a->num_seqs;
    st = cuda_status(launch_prefill_fwd(p, maps, num_tiles, s));
  }
  timer.after();
  return st;
}

int attn_bwd(const gcs_prefill_args* a, const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
             float* dlog_gate, float* dsink, void* workspace, size_t workspace_bytes, gcs_stream_t stream) {
  int st = check_prefill(a);
  if (st != GCS_OK) return st;
  if (!o || !lse || !dout || !dq || !dk || !dv) return GCS_ERR_INVALID_ARG;
  if (!aligned16(o) || !aligned16(lse) || !aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return GCS_ERR_INVALID_ARG;
  if ((dlog_gate == nullptr) != (a->log_gate == nullptr)) return GCS_ERR_INVALID_ARG;
  if ((dsink == nullptr) != (a->sink == nullptr)) return GCS_ERR_INVALID_ARG;
  PrefillLayouts lay;
  prefill_layouts(a, &lay);
  {
    const size_t t = (size_t)a->total_tokens;
    const int T = a->total_tokens;
    const PrefillSpans in = prefill_spans(a, lay);
    const TSpan outs[] = {tspan(dq, T, a->hq, a->dqk, lay.dq, 2), tspan(dk, T, a->hkv, a->dqk, lay.dk, 2),
                          tspan(dv, T, a->hkv, a->dv, lay.dv, 2), tspan(span(dlog_gate, t * a->hq * 4)),
                          tspan(span(dsink, (size_t)a->hq * 4))};
    const TSpan ins[] = {in.q, in.k, in.v, in.g, in.s, in.cu, tspan(o, T, a->hq, a->dv, lay.o, 2),
                         tspan(span(lse, t * a->hq * 4)), tspan(dout, T, a->hq, a->dv, lay.dout, 2)};
    if (outputs_overlap(outs, ins)) return GCS_ERR_INVALID_ARG;
  }
  const bool chk = device_checks_on();
  const size_t need = bwd_ws(a, chk);
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return GCS_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int* status = device_status_ptr();
  if (!status) return GCS_ERR_CUDA;

  const size_t ht = (size_t)a->hq * a->total_tokens;
  Carver c{static_cast<uint8_t*>(workspace)};
  float* gT = a->log_gate ? c.take<float>(ht) : nullptr;
  float* delta = c.take<float>(ht);
  const bool fu = fused(a);
  const bool tp = two_pass(a);
  const bool wide_det = !tp && !fu && wide_two_pass(a);
  // fp32 dQ accumulator: the single-pass route and wide heads on the reduce-add route
  float* dq_acc = (tp || wide_det) ? nullptr : c.take<float>((size_t)a->total_tokens * a->hq * a->dqk);
  float* dg_row = (a->log_gate || a->sink) ? c.take<float>(ht) : nullptr;
  float* dg_col = a->log_gate ? c.take<float>(ht) : nullptr;
  const int n_qtiles = (a->total_tokens + 63) / 64 + a->num_seqs;
  float* vecp = c.take<float>((size_t)a->hq * n_qtiles * 128);
  int32_t* cu_chk = chk ? c.take<int32_t>((size_t)a->num_seqs + 1) : nullptr;

  BwdMaps maps;
  const int T = a->total_tokens;
  if (!make_map(&maps.q, a->q, a->dqk, a->hq, T, lay.q, 64) ||
      !make_map(&maps.k, a->k, a->dqk, a->hkv, T, lay.k, 128) ||
      !make_map(&maps.v, a->v, a->dv, a->hkv, T, lay.v, 128) ||
      !make_map(&maps.dout, dout, a->dv, a->hq, T, lay.dout, 64) ||
      !make_map(&maps.q128, a->q, a->dqk, a->hq, T, lay.q, 128) ||
      !make_map(&maps.dout128, dout, a->dv, a->hq, T, lay.dout, 128))
    return GCS_ERR_CUDA;
  std::memset(&maps.dq_acc, 0, sizeof(maps.dq_acc));
  if (fu && !make_map_f32(&maps.dq_acc, dq_acc, a->dqk, a->hq, T, 128)) return GCS_ERR_CUDA;

  const int32_t* cu = a->cu_seqlens;
  if (cu_chk) {
    st = cuda_status(launch_check_prefill(a->cu_seqlens, a->num_seqs, a->total_tokens, a->max_seqlen, cu_chk, status, s));
    if (st != GCS_OK) return st;
    cu = cu_chk;
  }
  PreArgs pre{};
  pre.o = static_cast<const uint16_t*>(o);
  pre.dout = static_cast<const uint16_t*>(dout);
  pre.total = a->total_tokens;
  pre.hq = a->hq;
  pre.dv = a->dv;
  pre.dqk = a->dqk;
  pre.o_ts = lay.o.ts;
  pre.o_hs = lay.o.hs;
  pre.do_ts = lay.dout.ts;
  pre.do_hs = lay.dout.hs;
  pre.delta = delta;
  pre.dq_acc = dq_acc;
  pre.dg_row = dg_row;
  pre.dg_col = dg_col;
  pre.g = a->log_gate;
  pre.cu = cu;
  pre.num_seqs = a->num_seqs;
  pre.gT = gT;
  st = cuda_status(launch_bwd_pre(pre, s));
  if (st != GCS_OK) return st;

  st = cuda_status(launch_bwd_pack(cu, a->num_seqs, a->total_tokens, a->hq, n_qtiles, lse, gT, delta,
                                   vecp, s));
  if (st != GCS_OK) return st;

  BwdParams p;
  p.cu_seqlens = cu;
  p.num_seqs = a->num_seqs;
  p.total = a->total_tokens;
  p.hq = a->hq;
  p.hkv = a->hkv;
  p.dqk = a->dqk;
  p.dv = a->dv;
  p.scale = a->scale;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.window = a->window;
  p.gT = gT;
  p.lse = lse;
  p.delta = delta;
  p.grad_q = static_cast<uint16_t*>(dq);
  p.grad_k = static_cast<uint16_t*>(dk);
  p.grad_v = static_cast<uint16_t*>(dv);
  p.dq_ts = lay.dq.ts;
  p.dq_hs = lay.dq.hs;
  p.dk_ts = lay.dk.ts;
  p.dk_hs = lay.dk.hs;
  p.dv_ts = lay.dv.ts;
  p.dv_hs = lay.dv.hs;
  p.dq_acc = dq_acc;
  p.dg_row = dg_row;
  p.dg_col = dg_col;
  p.vecp = vecp;
  p.n_qtiles = n_qtiles;
  p.status = status;
  const int num_tiles = (a->total_tokens + 127) / 128 + a->num_seqs;
  KernelTimer timer(s);
  if (fu) {
    timer.before();
    st = cuda_status(launch_prefill_bwd_fused(p, maps, num_tiles, s));
    timer.after();
  } else if (tp) {
    // dQ pass (query tiles of 128 rows), then the dK/dV pass; the timer brackets both
    BwdMaps dqmaps = maps;
    dqmaps.q = maps.q128;
    dqmaps.dout = maps.dout128;
    timer.before();
    st = cuda_status(launch_prefill_bwd_dq(p, dqmaps, num_tiles, s));
    if (st != GCS_OK) return st;
    st = cuda_status(launch_prefill_bwd(p, maps, num_tiles, s));
    timer.after();
  } else if (wide_det) {
    // dQ pass (query tiles of 64 rows), then the dK / dV roles; the timer brackets both
    timer.before();
    st = cuda_status(launch_prefill_bwd_wide_dq(p, maps, n_qtiles, s));
    if (st != GCS_OK) return st;
    st = cuda_status(launch_prefill_bwd_wide(p, maps, num_tiles, false, s));
    timer.after();
  } else {
    timer.before();
    st = cuda_status(launch_prefill_bwd_wide(p, maps, num_tiles, true, s));
    timer.after();
  }
  if (st != GCS_OK) return st;
  PostArgs post{};
  post.dq_acc = dq_acc;
  post.dq = static_cast<uint16_t*>(dq);
  post.total = a->total_tokens;
  post.hq = a->hq;
  post.dqk = a->dqk;
  post.dq_ts = lay.dq.ts;
  post.dq_hs = lay.dq.hs;
  post.cu = cu;
  post.num_seqs = a->num_seqs;
  post.dg_row = dg_row;
  post.dg_col = dg_col;
  post.dlog_gate = dlog_gate;
  post.lse = lse;
  post.delta = delta;
  post.sink = a->sink;
  post.dsink = dsink;
  return cuda_status(launch_bwd_post(post, s));
}

// Byte strides of the paged caches; all-zero element strides = contiguous
// [num_blocks, hkv, block_size, d].
static int cache_layout(const gcs_decode_args* a, CacheLayout* l) {
  const long long elt = a->kv_format == GCS_KV_BF16 ? 2 : 1;
  const long long row = (long long)a->d * elt;
  if (a->kv_stride_block == 0 && a->kv_stride_head == 0 && a->kv_stride_slot == 0) {
    *l = CacheLayout{(long long)a->hkv * a->block_size * row, (long long)a->block_size * row, row};
    return GCS_OK;
  }
  if (a->kv_stride_block < 0 || a->kv_stride_head < 0 || a->kv_stride_slot < 0) return GCS_ERR_INVALID_ARG;
  const long long b = a->kv_stride_block * elt, h = a->kv_stride_head * elt, sl = a->kv_stride_slot * elt;
  if ((b % 16) || (h % 16) || (sl % 16) || b >= (1LL << 40)) return GCS_ERR_UNSUPPORTED;
  const bool slot_inner = sl >= row && h >= (long long)a->block_size * sl;
  const bool head_inner = h >= row && sl >= (long long)a->hkv * h;
  if (!slot_inner && !head_inner) return GCS_ERR_UNSUPPORTED;
  if (b < (long long)(a->hkv - 1) * h + (long long)(a->block_size - 1) * sl + row) return GCS_ERR_UNSUPPORTED;
  *l = CacheLayout{b, h, sl};
  return GCS_OK;
}

static int check_decode(const gcs_decode_args* a) {
  if (!a) return GCS_ERR_INVALID_ARG;
  if (a->num_reqs < 1 || a->total_q < 1 || a->max_q_len < 1 || a->max_seq_len < 1 || a->max_blocks_per_req < 1 ||
      a->num_blocks < 1 || a->hq < 1 || a->hkv < 1 || a->segment_len < 1)
    return GCS_ERR_INVALID_ARG;
  if (!a->cu_q || !a->seq_lens || !a->block_table || !a->k_cache || !a->v_cache || !a->q)
    return GCS_ERR_INVALID_ARG;
  if (!std::isfinite(a->scale)) return GCS_ERR_INVALID_ARG;
  if (a->kv_format == GCS_KV_BF16) {
    // a bf16 cache carries no scales
    if (a->k_scale || a->v_scale || a->scale_mode != GCS_SCALE_PER_TOKEN) return GCS_ERR_INVALID_ARG;
  } else if (a->kv_format == GCS_KV_FP8_E4M3) {
    if (!a->k_scale || !a->v_scale) return GCS_ERR_INVALID_ARG;
    if (a->scale_mode == GCS_SCALE_PER_TOKEN) {
      if (!aligned16(a->k_scale) || !aligned16(a->v_scale)) return GCS_ERR_INVALID_ARG;
    } else if (a->scale_mode == GCS_SCALE_PER_TENSOR) {
      if ((reinterpret_cast<uintptr_t>(a->k_scale) | reinterpret_cast<uintptr_t>(a->v_scale)) & 3u)
        return GCS_ERR_INVALID_ARG;
    } else {
      return GCS_ERR_INVALID_ARG;
    }
  } else {
    return GCS_ERR_INVALID_ARG;
  }
  // per-token scales are only read on decode / short-query shapes (a prefill shape is rejected)
  if (a->max_q_len > 4) return GCS_ERR_UNSUPPORTED;
  // head dim 128; GQA groups of 16 or 8 query heads; blocks of whole 16-token pages
  if (a->d != 128 || (a->hq != 16 * a->hkv && a->hq != 8 * a->hkv)) return GCS_ERR_UNSUPPORTED;
  // cache blocks of 16 x 2^k tokens (16, 32, 64, 128, ...)
  if (a->block_size < 16 || a->block_size > 4096 || (a->block_size & (a->block_size - 1)) != 0)
    return GCS_ERR_UNSUPPORTED;
  if (a->segment_len % 16 != 0) return GCS_ERR_UNSUPPORTED;
  if ((long long)a->max_blocks_per_req * a->block_size < a->max_seq_len) return GCS_ERR_INVALID_ARG;
  if (!aligned16(a->k_cache) || !aligned16(a->v_cache) || !aligned16(a->q)) return GCS_ERR_INVALID_ARG;
  if (a->window < 0) return GCS_ERR_INVALID_ARG;
  if (a->g_cache && !aligned16(a->g_cache)) return GCS_ERR_INVALID_ARG;
  if (a->sink && (reinterpret_cast<uintptr_t>(a->sink) & 3u)) return GCS_ERR_INVALID_ARG;
  if ((double)a->num_blocks * a->hkv * a->block_size * a->d > 9.0e15) return GCS_ERR_UNSUPPORTED;
  CacheLayout cl;
  int st = cache_layout(a, &cl);
  if (st != GCS_OK) return st;
  Layout lq, lo;
  if ((st = resolve_layout(a->q_stride, a->hq, a->d, &lq)) != GCS_OK) return st;
  return resolve_layout(a->out_stride, a->hq, a->d, &lo);
}

// True when the output of a paged call overlaps one of its inputs.
static bool paged_out_overlaps(const gcs_decode_args* a, const void* out) {
  const size_t rows = (size_t)a->num_blocks * a->hkv * a->block_size;
  const size_t elt = a->kv_format == GCS_KV_BF16 ? 2 : 1;
  const size_t sc = a->scale_mode == GCS_SCALE_PER_TENSOR ? 4 : rows * 4;
  CacheLayout cl;
  Layout lq, lo;
  cache_layout(a, &cl);
  resolve_layout(a->q_stride, a->hq, a->d, &lq);
  resolve_layout(a->out_stride, a->hq, a->d, &lo);
  const size_t cache_bytes = (size_t)(a->num_blocks - 1) * cl.bs + (size_t)(a->hkv - 1) * cl.hs +
                             (size_t)(a->block_size - 1) * cl.ss + (size_t)a->d * elt;
  const TSpan outs[] = {tspan(out, a->total_q, a->hq, a->d, lo, 2)};
  const TSpan ins[] = {tspan(a->q, a->total_q, a->hq, a->d, lq, 2),
                       tspan(span(a->k_cache, cache_bytes)),
                       tspan(span(a->v_cache, cache_bytes)),
                       tspan(span(a->k_scale, sc)),
                       tspan(span(a->v_scale, sc)),
                       tspan(span(a->block_table, (size_t)a->num_reqs * a->max_blocks_per_req * 4)),
                       tspan(span(a->seq_lens, (size_t)a->num_reqs * 4)),
                       tspan(span(a->cu_q, ((size_t)a->num_reqs + 1) * 4)),
                       tspan(span(a->g_cache, (size_t)a->num_blocks * a->hq * a->block_size * 4)),
                       tspan(span(a->sink, (size_t)a->hq * 4))};
  return outputs_overlap(outs, ins);
}

// Kernel parameters common to the paged calls (segments and partial buffers set by the caller).
static void fill_paged_params(const gcs_decode_args* a, void* out, int* status, DecodeParams& p) {
  p.cu_q = a->cu_q;
  p.seq_lens = a->seq_lens;
  p.block_table = a->block_table;
  p.max_blocks = a->max_blocks_per_req;
  p.k_cache = static_cast<const uint8_t*>(a->k_cache);
  p.v_cache = static_cast<const uint8_t*>(a->v_cache);
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.kv_format = a->kv_format;
  p.scale_mode = a->scale_mode;
  p.g_cache = a->g_cache;
  p.sink = a->sink;
  p.window = a->window;
  p.num_reqs = a->num_reqs;
  p.hq = a->hq;
  p.hkv = a->hkv;
  p.max_q_len = a->max_q_len;
  p.max_segs = 1;
  p.seg_pages = 0;
  p.scale = a->scale;
  p.q = static_cast<const uint16_t*>(a->q);
  p.out = static_cast<uint16_t*>(out);
  CacheLayout cl;
  Layout lq, lo;
  cache_layout(a, &cl);
  resolve_layout(a->q_stride, a->hq, a->d, &lq);
  resolve_layout(a->out_stride, a->hq, a->d, &lo);
  p.q_ts = lq.ts;
  p.q_hs = lq.hs;
  p.out_ts = lo.ts;
  p.out_hs = lo.hs;
  p.kv_bs = cl.bs;
  p.kv_hs = cl.hs;
  p.kv_ss = cl.ss;
  p.kv_head_inner = cl.head_inner() ? 1 : 0;
  p.block_size = a->block_size;
  p.log2_block_pages = 0;
  while ((16 << p.log2_block_pages) < a->block_size) ++p.log2_block_pages;
  p.group = a->hq / a->hkv;
  p.part_acc = nullptr;
  p.part_ml = nullptr;
  p.status = status;
}

// Bytes of the split-K partials (acc, then (m, l)) of num_reqs x max_segs x hkv units.
static size_t partials_ws(const gcs_decode_args* a, int max_segs) {
  const size_t units = (size_t)a->num_reqs * max_segs * a->hkv;
  const size_t rows = (size_t)a->max_q_len * 16;
  return round_up(units * rows * 128 * sizeof(float)) + round_up(units * rows * 2 * sizeof(float));
}

// Bytes of the checked copy of cu_q that ends the workspace when device checks are on.
static size_t cu_q_copy_ws(const gcs_decode_args* a, bool chk) {
  return chk ? round_up(((size_t)a->num_reqs + 1) * sizeof(int32_t)) : 0;
}

static size_t decode_ws(const gcs_decode_args* a, bool chk, int* max_segs_out) {
  const int max_segs = (a->max_seq_len + a->segment_len - 1) / a->segment_len;
  if (max_segs_out) *max_segs_out = max_segs;
  return partials_ws(a, max_segs) + cu_q_copy_ws(a, chk);
}

// Runs the device-content checks of a paged call when they are on: p.cu_q then points to the
// checked copy at byte offset `off` of the workspace.
static PagedOperandCheck operand_check(const gcs_decode_args* a) {
  PagedOperandCheck c{};
  if (a->kv_format != GCS_KV_FP8_E4M3) return c;  // hkv 0: nothing to check
  Layout lq;
  resolve_layout(a->q_stride, a->hq, a->d, &lq);
  c.q = static_cast<const uint16_t*>(a->q);
  c.q_ts = lq.ts;
  c.q_hs = lq.hs;
  c.hq = a->hq;
  c.d = a->d;
  c.hkv = a->hkv;
  c.v_scale = a->v_scale;
  c.per_tensor = a->scale_mode == GCS_SCALE_PER_TENSOR ? 1 : 0;
  return c;
}

static int paged_checks(const gcs_decode_args* a, void* workspace, size_t off, DecodeParams& p, cudaStream_t s,
                        const SharedPrefixes& prefix = SharedPrefixes{}) {
  int32_t* cu_chk = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + off);
  const int st = cuda_status(launch_check_paged(a->cu_q, a->seq_lens, a->block_table, a->num_reqs, a->total_q,
                                                a->max_q_len, a->max_seq_len, a->max_blocks_per_req, a->num_blocks,
                                                a->block_size, a->window, operand_check(a), prefix, cu_chk, p.status,
                                                s));
  if (st == GCS_OK) p.cu_q = cu_chk;
  return st;
}

size_t attn_decode_workspace(const gcs_decode_args* a) {
  return (a && check_decode(a) == GCS_OK) ? decode_ws(a, device_checks_on(), nullptr) : 0;
}

int attn_decode_paged(const gcs_decode_args* a, void* out, void* workspace, size_t workspace_bytes,
                      gcs_stream_t stream) {
  int st = check_decode(a);
  if (st != GCS_OK) return st;
  if (!out || !aligned16(out)) return GCS_ERR_INVALID_ARG;
  if (paged_out_overlaps(a, out)) return GCS_ERR_INVALID_ARG;
  int max_segs = 0;
  const bool chk = device_checks_on();
  const size_t need = decode_ws(a, chk, &max_segs);
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return GCS_ERR_WORKSPACE;
  int* status = device_status_ptr();
  if (!status) return GCS_ERR_CUDA;
  const size_t units = (size_t)a->num_reqs * max_segs * a->hkv;
  const size_t rows = (size_t)a->max_q_len * 16;
  DecodeParams p;
  fill_paged_params(a, out, status, p);
  p.max_segs = max_segs;
  p.seg_pages = a->segment_len / 16;
  p.part_acc = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + round_up(units * rows * 128 * sizeof(float)));
  DecodeMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (a->kv_format == GCS_KV_FP8_E4M3) {
    CacheLayout cl;
    cache_layout(a, &cl);
    if (!make_page_map_u8(&maps.k, a->k_cache, a->num_blocks, a->hkv, a->block_size, cl) ||
        !make_page_map_u8(&maps.v, a->v_cache, a->num_blocks, a->hkv, a->block_size, cl))
      return GCS_ERR_CUDA;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (chk) {
    const int st2 = paged_checks(a, workspace, partials_ws(a, max_segs), p, s);
    if (st2 != GCS_OK) return st2;
  }
  KernelTimer timer(s);
  return cuda_status(launch_decode(p, maps, s, &timer.b, &timer.a));
}

int attn_decode_paged_noalloc(const gcs_decode_args* a, void* out, gcs_stream_t stream) {
  int st = check_decode(a);
  if (st != GCS_OK) return st;
  // the split-K partials must fit the library's fixed scratch
  if (decode_ws(a, device_checks_on(), nullptr) > kNoAllocScratchBytes) return GCS_ERR_WORKSPACE;
  void* scratch = nullptr;
  if (decode_noalloc_scratch(&scratch) != cudaSuccess) return GCS_ERR_CUDA;
  return attn_decode_paged(a, out, scratch, kNoAllocScratchBytes, stream);
}

// Paged chunked prefill: the decode checks with the q_len limit lifted, fp8 only, and
// segment_len 0 (automatic) or a multiple of 128 tokens (one key tile of 8 pages).
static int check_prefill_paged(const gcs_decode_args* a) {
  if (!a) return GCS_ERR_INVALID_ARG;
  if (a->max_q_len < 1 || a->segment_len < 0) return GCS_ERR_INVALID_ARG;
  gcs_decode_args b = *a;
  b.max_q_len = a->max_q_len < 4 ? a->max_q_len : 4;
  b.segment_len = a->segment_len > 0 ? a->segment_len : 128;
  const int st = check_decode(&b);
  if (st != GCS_OK) return st;
  if (a->kv_format != GCS_KV_FP8_E4M3) return GCS_ERR_UNSUPPORTED;
  if (a->segment_len % 128 != 0) return GCS_ERR_UNSUPPORTED;
  if (a->max_q_len > a->max_seq_len) return GCS_ERR_INVALID_ARG;
  return GCS_OK;
}

struct PagedPlan {
  int seg_pages = 0, max_segs = 1;  // max_segs 1: one segment per request, the kernel writes out directly
  size_t part_ws = 0;               // split-K partials (none with one segment)
  size_t ws = 0;                    // + the checked copy of cu_q with device checks on
};

// Segments of the paged prefill: the caller's, or (segment_len 0) the fewest that give
// about two CTAs per SM with the query blocks of 16 positions x kv heads x requests.
static bool plan_prefill_paged(const gcs_decode_args* a, bool chk, PagedPlan* pl) {
  const int max_pages = (a->max_seq_len + 15) / 16;
  int sp;
  if (a->segment_len > 0) {
    sp = a->segment_len / 16;
  } else {
    int dev = 0, nsm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return false;
    const long long ctas = (long long)((a->max_q_len + 15) / 16) * a->hkv * a->num_reqs;
    long long want = (2LL * nsm + ctas - 1) / ctas;
    if (want < 1) want = 1;
    sp = (int)((max_pages + want - 1) / want);
    sp = ((sp + 7) / 8) * 8;
  }
  pl->seg_pages = sp;
  pl->max_segs = (max_pages + sp - 1) / sp;
  pl->part_ws = pl->max_segs > 1 ? partials_ws(a, pl->max_segs) : 0;
  pl->ws = pl->part_ws + cu_q_copy_ws(a, chk);
  return true;
}

size_t attn_prefill_paged_workspace(const gcs_decode_args* a) {
  PagedPlan pl;
  if (!a || check_prefill_paged(a) != GCS_OK || !plan_prefill_paged(a, device_checks_on(), &pl)) return 0;
  return pl.ws;
}

int attn_prefill_paged(const gcs_decode_args* a, void* out, void* workspace, size_t workspace_bytes,
                       gcs_stream_t stream) {
  int st = check_prefill_paged(a);
  if (st != GCS_OK) return st;
  if (!out || !aligned16(out)) return GCS_ERR_INVALID_ARG;
  if (paged_out_overlaps(a, out)) return GCS_ERR_INVALID_ARG;
  PagedPlan pl;
  const bool chk = device_checks_on();
  if (!plan_prefill_paged(a, chk, &pl)) return GCS_ERR_CUDA;
  if (pl.ws > 0 && (!workspace || workspace_bytes < pl.ws || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
    return GCS_ERR_WORKSPACE;
  int* status = device_status_ptr();
  if (!status) return GCS_ERR_CUDA;
  DecodeParams p;
  fill_paged_params(a, out, status, p);
  p.max_segs = pl.max_segs;
  p.seg_pages = pl.seg_pages;
  if (pl.max_segs > 1) {
    const size_t units = (size_t)a->num_reqs * pl.max_segs * a->hkv;
    const size_t rows = (size_t)a->max_q_len * 16;
    p.part_acc = static_cast<float*>(workspace);
    p.part_ml =
        reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + round_up(units * rows * 128 * sizeof(float)));
  }
  DecodeMaps maps;
  CacheLayout cl;
  cache_layout(a, &cl);
  if (!make_page_map_u8(&maps.k, a->k_cache, a->num_blocks, a->hkv, a->block_size, cl) ||
      !make_page_map_u8(&maps.v, a->v_cache, a->num_blocks, a->hkv, a->block_size, cl))
    return GCS_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (chk) {
    const int st2 = paged_checks(a, workspace, pl.part_ws, p, s);
    if (st2 != GCS_OK) return st2;
  }
  KernelTimer timer(s);
  return cuda_status(launch_prefill_paged(p, maps, s, &timer.b, &timer.a));
}

// ------------------------------------------------------------------ decoding behind shared prefixes

static int check_shared(const gcs_decode_args* a, const gcs_prefix_args* x) {
  if (!a || !x || a->segment_len < 0) return GCS_ERR_INVALID_ARG;
  gcs_decode_args b = *a;
  if (b.segment_len == 0) b.segment_len = 16;  // the library's choice
  const int st = check_decode(&b);
  if (st != GCS_OK) return st;
  if (x->num_groups < 1 || x->max_group_q < 1 || x->max_group_q > a->total_q || x->max_prefix_len < 0 ||
      x->max_prefix_len > a->max_seq_len || x->max_suffix_len < 0 || x->max_suffix_len > a->max_seq_len)
    return GCS_ERR_INVALID_ARG;
  if (!x->cu_groups || !x->prefix_lens || (reinterpret_cast<uintptr_t>(x->cu_groups) & 3u) ||
      (reinterpret_cast<uintptr_t>(x->prefix_lens) & 3u))
    return GCS_ERR_INVALID_ARG;
  // the launch grids, and positions with a tile ahead
  if (a->num_reqs > 65535 || x->num_groups > 65535 || a->hkv > 65535 || a->max_seq_len > 1 << 30)
    return GCS_ERR_UNSUPPORTED;
  return GCS_OK;
}

struct SharedPlan {
  int pre_segs = 0, pre_seg_keys = 128;  // of the prefixes
  int max_segs = 0, seg_pages = 0;       // of what lies behind them
  size_t acc = 0, ml = 0, part = 0;      // bytes: the prefixes' partials, the others'
  size_t ws = 0;                         // + the checked copies of cu_q and cu_groups
};
// Segments: of a prefix, enough for one CTA an SM with the groups' row tiles and kv heads; behind
// it (segment_len 0), enough for the three CTAs of an SM, of 128 to 2048 tokens.
static bool plan_shared(const gcs_decode_args* a, const gcs_prefix_args* x, bool chk, SharedPlan* pl) {
  const int sms = current_sms();
  if (!sms) return false;
  if (x->max_prefix_len > 0) {
    const int rows = 256 / (a->hq / a->hkv);
    const long long base = (long long)x->num_groups * ((x->max_group_q + rows - 1) / rows) * a->hkv;
    const long long tiles = (x->max_prefix_len + 127) / 128;
    long long want = sms / base;
    want = want < 1 ? 1 : want > tiles ? tiles : want;
    pl->pre_seg_keys = (int)((tiles + want - 1) / want) * 128;
    pl->pre_segs = (x->max_prefix_len + pl->pre_seg_keys - 1) / pl->pre_seg_keys;
  }
  if (x->max_suffix_len > 0) {
    const int pages = (x->max_suffix_len + 30) / 16;  // the first may be the prefix's last
    if (a->segment_len > 0) {
      pl->seg_pages = a->segment_len / 16;
    } else {
      const long long units = (long long)a->num_reqs * a->hkv, want = (3LL * sms + units - 1) / units;
      const long long sp = (pages + want - 1) / want;
      pl->seg_pages = (int)(sp < 8 ? 8 : sp > 128 ? 128 : sp);
    }
    pl->max_segs = (pages + pl->seg_pages - 1) / pl->seg_pages;
    pl->part = partials_ws(a, pl->max_segs);
  }
  const size_t rows = (size_t)pl->pre_segs * a->total_q * a->hq;
  pl->acc = round_up(rows * 128 * sizeof(float));
  pl->ml = round_up(rows * sizeof(float2));
  pl->ws = pl->part + pl->acc + pl->ml + cu_q_copy_ws(a, chk) +
           (chk ? round_up(((size_t)x->num_groups + 1) * sizeof(int32_t)) : 0);
  return true;
}

size_t attn_decode_paged_shared_workspace(const gcs_decode_args* a, const gcs_prefix_args* x) {
  SharedPlan pl;
  return check_shared(a, x) == GCS_OK && plan_shared(a, x, device_checks_on(), &pl) ? pl.ws : 0;
}

int attn_decode_paged_shared(const gcs_decode_args* a, const gcs_prefix_args* x, void* out, void* workspace,
                             size_t workspace_bytes, gcs_stream_t stream) {
  int st = check_shared(a, x);
  if (st != GCS_OK) return st;
  if (!out || !aligned16(out)) return GCS_ERR_INVALID_ARG;
  if (paged_out_overlaps(a, out)) return GCS_ERR_INVALID_ARG;
  CacheLayout cl;
  Layout lo;
  cache_layout(a, &cl);
  resolve_layout(a->out_stride, a->hq, a->d, &lo);
  const TSpan outs[] = {tspan(out, a->total_q, a->hq, a->d, lo, 2)};
  const TSpan ins[] = {tspan(span(x->cu_groups, ((size_t)x->num_groups + 1) * 4)),
                       tspan(span(x->prefix_lens, (size_t)x->num_groups * 4))};
  if (outputs_overlap(outs, ins)) return GCS_ERR_INVALID_ARG;
  SharedPlan pl;
  const bool chk = device_checks_on();
  if (!plan_shared(a, x, chk, &pl)) return GCS_ERR_CUDA;
  if (pl.ws > 0 && (!workspace || workspace_bytes < pl.ws || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
    return GCS_ERR_WORKSPACE;
  int* status = device_status_ptr();
  if (!status) return GCS_ERR_CUDA;
  DecodeParams p{};
  fill_paged_params(a, out, status, p);
  if (p.window >= a->max_seq_len) p.window = 0;  // sees everything; position - window stays within 32 bits
  p.max_segs = pl.max_segs;
  p.seg_pages = pl.seg_pages > 0 ? pl.seg_pages : 1;
  p.num_groups = x->num_groups;
  p.cu_groups = x->cu_groups;
  p.prefix_lens = x->prefix_lens;
  p.max_prefix = x->max_prefix_len;
  p.total_q = a->total_q;
  p.max_group_q = x->max_group_q;
  p.pre_segs = pl.pre_segs;
  p.pre_seg_keys = pl.pre_seg_keys;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t units = (size_t)a->num_reqs * pl.max_segs * a->hkv;
  p.part_acc = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + round_up(units * a->max_q_len * 16 * 128 * sizeof(float)));
  p.pre_acc = reinterpret_cast<float*>(ws + pl.part);
  p.pre_ml = reinterpret_cast<float2*>(ws + pl.part + pl.acc);
  DecodeMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  auto map = [&](CUtensorMap* m, const void* base) {
    return a->kv_format == GCS_KV_BF16 ? make_page_map_bf16(m, base, a->num_blocks, a->hkv, a->block_size, a->d, cl)
                                       : make_page_map_u8(m, base, a->num_blocks, a->hkv, a->block_size, cl);
  };
  if (!map(&maps.k, a->k_cache) || !map(&maps.v, a->v_cache)) return GCS_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (chk) {
    const size_t off = pl.part + pl.acc + pl.ml;
    const SharedPrefixes prefix{x->cu_groups, x->prefix_lens, x->num_groups};
    st = paged_checks(a, workspace, off, p, s, prefix);
    if (st != GCS_OK) return st;
    int32_t* groups = reinterpret_cast<int32_t*>(ws + off + cu_q_copy_ws(a, true));
    st = cuda_status(launch_check_groups(prefix, a->seq_lens, a->block_table, a->num_reqs, a->max_blocks_per_req,
                                         a->num_blocks, a->block_size, a->total_q, x->max_group_q, x->max_prefix_len,
                                         x->max_suffix_len, a->window, operand_check(a),
                                         const_cast<int32_t*>(p.cu_q), groups, status, s));
    if (st != GCS_OK) return st;
    p.cu_groups = groups;
  }
  return cuda_status(launch_decode_shared(p, maps, s));
}

// ------------------------------------------------------------------ norm and rotation of q and k

static bool head_dim_supported(int d) { return d == 64 || d == 128 || d == 256 || d == 512; }
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// in_cache: positions may be missing (the cached positions are used).
static int check_rope(const gcs_qk_rope_args* a, bool in_cache) {
  if (!a) return GCS_ERR_INVALID_ARG;
  if (a->total_tokens < 1 || a->hq < 1 || a->hkv < 1 || a->hq % a->hkv != 0) return GCS_ERR_INVALID_ARG;
  if ((a->interleaved != 0 && a->interleaved != 1) || (a->norm != 0 && a->norm != 1)) return GCS_ERR_INVALID_ARG;
  if (!a->q || !a->k || !aligned16(a->q) || !aligned16(a->k)) return GCS_ERR_INVALID_ARG;
  if (!aligned16(a->q_weight) || !aligned16(a->k_weight) || !aligned16(a->cos_sin) || !aligned4(a->positions))
    return GCS_ERR_INVALID_ARG;
  if (a->norm) {
    if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return GCS_ERR_INVALID_ARG;
  } else if (a->q_weight || a->k_weight) {
    return GCS_ERR_INVALID_ARG;
  }
  if ((a->rotary_dim == 0) != (a->cos_sin == nullptr) || a->rotary_dim < 0) return GCS_ERR_INVALID_ARG;
  if (a->cos_sin && (a->max_pos < 1 || (!a->positions && !in_cache))) return GCS_ERR_INVALID_ARG;
  if (!head_dim_supported(a->d)) return GCS_ERR_UNSUPPORTED;
  if (a->rotary_dim > a->d) return GCS_ERR_INVALID_ARG;
  if (a->rotary_dim % 16 != 0) return GCS_ERR_UNSUPPORTED;
  // elements of a token within 32 bits
  if ((double)a->hq * a->d > 2147483647.0) return GCS_ERR_UNSUPPORTED;
  Layout l;
  int st;
  if ((st = resolve_layout(a->q_stride, a->hq, a->d, &l)) != GCS_OK) return st;
  if ((st = resolve_layout(a->k_stride, a->hkv, a->d, &l)) != GCS_OK) return st;
  if ((st = resolve_layout(a->q_out_stride, a->hq, a->d, &l)) != GCS_OK) return st;
  if ((st = resolve_layout(a->k_out_stride, a->hkv, a->d, &l)) != GCS_OK) return st;
  if ((st = resolve_layout(a->dq_stride, a->hq, a->d, &l)) != GCS_OK) return st;
  return resolve_layout(a->dk_stride, a->hkv, a->d, &l);
}

struct RopeLayouts {
  Layout q, k, q_out, k_out, dq, dk;
};
static RopeLayouts rope_layouts(const gcs_qk_rope_args* a) {
  RopeLayouts l;
  resolve_layout(a->q_stride, a->hq, a->d, &l.q);
  resolve_layout(a->k_stride, a->hkv, a->d, &l.k);
  resolve_layout(a->q_out_stride, a->hq, a->d, &l.q_out);
  resolve_layout(a->k_out_stride, a->hkv, a->d, &l.k_out);
  resolve_layout(a->dq_stride, a->hq, a->d, &l.dq);
  resolve_layout(a->dk_stride, a->hkv, a->d, &l.dk);
  return l;
}

static RopeParams rope_params(const gcs_qk_rope_args* a, const RopeLayouts& l) {
  RopeParams p{};
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.q_ts = l.q.ts, p.q_hs = l.q.hs, p.k_ts = l.k.ts, p.k_hs = l.k.hs;
  p.qo_ts = l.q_out.ts, p.qo_hs = l.q_out.hs, p.ko_ts = l.k_out.ts, p.ko_hs = l.k_out.hs;
  p.dq_ts = l.dq.ts, p.dq_hs = l.dq.hs, p.dk_ts = l.dk.ts, p.dk_hs = l.dk.hs;
  p.total = a->total_tokens;
  p.hq = a->hq;
  p.hkv = a->hkv;
  p.d = a->d;
  p.rotary_dim = a->rotary_dim;
  p.interleaved = a->interleaved;
  p.norm = a->norm;
  p.eps = a->eps;
  p.q_weight = a->q_weight;
  p.k_weight = a->k_weight;
  p.cos_sin = a->cos_sin;
  p.max_pos = a->max_pos;
  p.positions = a->positions;
  return p;
}

// Byte ranges of a rope call's inputs: q, k, the weights, the table and the positions.
struct RopeSpans {
  TSpan q, k, qw, kw, table, pos;
};
static RopeSpans rope_spans(const gcs_qk_rope_args* a, const RopeLayouts& l) {
  const int T = a->total_tokens;
  return RopeSpans{tspan(a->q, T, a->hq, a->d, l.q, 2),
                   tspan(a->k, T, a->hkv, a->d, l.k, 2),
                   tspan(span(a->q_weight, (size_t)a->d * 4)),
                   tspan(span(a->k_weight, (size_t)a->d * 4)),
                   tspan(span(a->cos_sin, (size_t)a->max_pos * a->rotary_dim * 4)),
                   tspan(span(a->positions, (size_t)T * 4))};
}

int attn_qk_norm_rope_fwd(const gcs_qk_rope_args* a, void* q_out, void* k_out, gcs_stream_t stream) {
  const int st = check_rope(a, false);
  if (st != GCS_OK) return st;
  if (!q_out || !k_out || !aligned16(q_out) || !aligned16(k_out)) return GCS_ERR_INVALID_ARG;
  const RopeLayouts l = rope_layouts(a);
  const RopeSpans in = rope_spans(a, l);
  const TSpan outs[] = {tspan(q_out, a->total_tokens, a->hq, a->d, l.q_out, 2),
                        tspan(k_out, a->total_tokens, a->hkv, a->d, l.k_out, 2)};
  const TSpan ins[] = {in.q, in.k, in.qw, in.kw, in.table, in.pos};
  if (outputs_overlap(outs, ins)) return GCS_ERR_INVALID_ARG;
  RopeParams p = rope_params(a, l);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.status = device_status_ptr();
  if (!p.status) return GCS_ERR_CUDA;
  return cuda_status(launch_norm_rope_fwd(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t attn_qk_norm_rope_bwd_workspace(const gcs_qk_rope_args* a) {
  if (check_rope(a, false) != GCS_OK || (!a->q_weight && !a->k_weight)) return 0;
  return round_up(norm_rope_bwd_partials(rope_params(a, rope_layouts(a))) * sizeof(float));
}

int attn_qk_norm_rope_bwd(const gcs_qk_rope_args* a, const void* dq_out, const void* dk_out, void* dq, void* dk,
                          float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                          gcs_stream_t stream) {
  const int st = check_rope(a, false);
  if (st != GCS_OK) return st;
  if (!dq_out || !dk_out || !dq || !dk) return GCS_ERR_INVALID_ARG;
  if (!aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) || !aligned16(dk) || !aligned4(dq_weight) ||
      !aligned4(dk_weight))
    return GCS_ERR_INVALID_ARG;
  if ((dq_weight && !a->q_weight) || (dk_weight && !a->k_weight)) return GCS_ERR_INVALID_ARG;
  const RopeLayouts l = rope_layouts(a);
  const RopeSpans in = rope_spans(a, l);
  const int T = a->total_tokens;
  const TSpan outs[] = {tspan(dq, T, a->hq, a->d, l.dq, 2), tspan(dk, T, a->hkv, a->d, l.dk, 2),
                        tspan(span(dq_weight, (size_t)a->d * 4)), tspan(span(dk_weight, (size_t)a->d * 4))};
  const TSpan ins[] = {in.q, in.k, in.qw, in.kw, in.table, in.pos, tspan(dq_out, T, a->hq, a->d, l.q_out, 2),
                       tspan(dk_out, T, a->hkv, a->d, l.k_out, 2)};
  if (outputs_overlap(outs, ins)) return GCS_ERR_INVALID_ARG;
  RopeParams p = rope_params(a, l);
  if (dq_weight || dk_weight) {
    const size_t need = norm_rope_bwd_partials(p) * sizeof(float);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
      return GCS_ERR_WORKSPACE;
    p.partials = static_cast<float*>(workspace);
  }
  p.q_out = static_cast<uint16_t*>(const_cast<void*>(dq_out));
  p.k_out = static_cast<uint16_t*>(const_cast<void*>(dk_out));
  p.dq = static_cast<uint16_t*>(dq);
  p.dk = static_cast<uint16_t*>(dk);
  p.status = device_status_ptr();
  if (!p.status) return GCS_ERR_CUDA;
  return cuda_status(launch_norm_rope_bwd(p, dq_weight, dk_weight, reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ write and read of the paged cache

// The cache strides by the rules of the paged attention calls.
static int cache_args_layout(const gcs_cache_args* a, CacheLayout* l) {
  gcs_decode_args d{};
  d.kv_format = a->kv_format;
  d.d = a->d;
  d.hkv = a->hkv;
  d.block_size = a->block_size;
  d.kv_stride_block = a->kv_stride_block;
  d.kv_stride_head = a->kv_stride_head;
  d.kv_stride_slot = a->kv_stride_slot;
  return cache_layout(&d, l);
}

static int check_cache(const gcs_cache_args* a) {
  if (!a) return GCS_ERR_INVALID_ARG;
  if (a->num_reqs < 1 || a->total_rows < 1 || a->max_rows < 1 || a->max_blocks_per_req < 1 || a->num_blocks < 1 ||
      a->hq < 1 || a->hkv < 1 || a->hq % a->hkv != 0)
    return GCS_ERR_INVALID_ARG;
  if (!a->cu_rows || !a->seq_lens || !a->block_table || !a->k_cache || !a->v_cache) return GCS_ERR_INVALID_ARG;
  if (!aligned16(a->k_cache) || !aligned16(a->v_cache) || !aligned16(a->g_cache) || !aligned4(a->cu_rows) ||
      !aligned4(a->seq_lens) || !aligned4(a->block_table) || !aligned4(a->k_scale) || !aligned4(a->v_scale))
    return GCS_ERR_INVALID_ARG;
  if (a->kv_format == GCS_KV_BF16) {
    if (a->k_scale || a->v_scale || a->scale_mode != GCS_SCALE_PER_TOKEN) return GCS_ERR_INVALID_ARG;
  } else if (a->kv_format == GCS_KV_FP8_E4M3) {
    if (!a->k_scale || !a->v_scale) return GCS_ERR_INVALID_ARG;
    if (a->scale_mode != GCS_SCALE_PER_TOKEN && a->scale_mode != GCS_SCALE_PER_TENSOR) return GCS_ERR_INVALID_ARG;
  } else {
    return GCS_ERR_INVALID_ARG;
  }
  if (!head_dim_supported(a->d)) return GCS_ERR_UNSUPPORTED;
  if (a->block_size < 16 || a->block_size > 4096 || (a->block_size & (a->block_size - 1)) != 0)
    return GCS_ERR_UNSUPPORTED;
  // rows (with the few that a warp looks ahead), heads and the gates' grid within 32 bits
  if (a->total_rows > 1 << 30 || (double)a->hq * a->d > 2147483647.0) return GCS_ERR_UNSUPPORTED;
  if (((double)a->total_rows / 64 + 2.0 * a->num_reqs) * ((a->hq + 31) / 32) > 1073741824.0 ||
      (a->hq + 31) / 32 > 65535)
    return GCS_ERR_UNSUPPORTED;
  if ((double)a->num_blocks * a->hkv * a->block_size * a->d > 9.0e15) return GCS_ERR_UNSUPPORTED;
  CacheLayout cl;
  int st = cache_args_layout(a, &cl);
  if (st != GCS_OK) return st;
  Layout l;
  if ((st = resolve_layout(a->k_stride, a->hkv, a->d, &l)) != GCS_OK) return st;
  return resolve_layout(a->v_stride, a->hkv, a->d, &l);
}

struct CacheSpans {
  TSpan k, v, ks, vs, g, table, lens, cu;
};
static CacheSpans cache_spans(const gcs_cache_args* a, const CacheLayout& cl) {
  const size_t elt = a->kv_format == GCS_KV_BF16 ? 2 : 1;
  const size_t rows = (size_t)a->num_blocks * a->hkv * a->block_size;
  const size_t sc = a->scale_mode == GCS_SCALE_PER_TENSOR ? 4 : rows * 4;
  const size_t bytes = (size_t)(a->num_blocks - 1) * cl.bs + (size_t)(a->hkv - 1) * cl.hs +
                       (size_t)(a->block_size - 1) * cl.ss + (size_t)a->d * elt;
  return CacheSpans{tspan(span(a->k_cache, bytes)),
                    tspan(span(a->v_cache, bytes)),
                    tspan(span(a->k_scale, sc)),
                    tspan(span(a->v_scale, sc)),
                    tspan(span(a->g_cache, (size_t)a->num_blocks * a->hq * a->block_size * 4)),
                    tspan(span(a->block_table, (size_t)a->num_reqs * a->max_blocks_per_req * 4)),
                    tspan(span(a->seq_lens, (size_t)a->num_reqs * 4)),
                    tspan(span(a->cu_rows, ((size_t)a->num_reqs + 1) * 4))};
}

// True when the K and V caches (same strides) share a byte.  Apart, or side by side within every
// period of one of the strides that the wider strides are multiples of, they do not.
static bool caches_meet(const gcs_cache_args* a, const CacheLayout& l, const CacheSpans& s) {
  if (!(s.k.a < s.v.b && s.v.a < s.k.b)) return false;
  const long long row = (long long)a->d * (a->kv_format == GCS_KV_BF16 ? 2 : 1);
  const bool hi = l.head_inner();
  const long long inner = hi ? l.hs : l.ss, outer = hi ? l.ss : l.hs;
  const long long n_inner = hi ? a->hkv : a->block_size, n_outer = hi ? a->block_size : a->hkv;
  const unsigned long long off = s.k.a < s.v.a ? s.v.a - s.k.a : s.k.a - s.v.a;
  auto beside = [&](long long period, long long width) {
    const long long d = (long long)(off % (unsigned long long)period);
    return d >= width && d + width <= period;
  };
  const long long w_outer = (n_inner - 1) * inner + row;              // bytes within an outer period
  const long long w_block = (n_outer - 1) * outer + w_outer;          // and within a block
  if (beside(l.bs, w_block)) return false;
  if (l.bs % outer == 0 && beside(outer, w_outer)) return false;
  return !(l.bs % inner == 0 && outer % inner == 0 && beside(inner, row));
}

static CacheParams cache_params(const gcs_cache_args* a, const CacheLayout& cl) {
  CacheParams p{};
  p.num_reqs = a->num_reqs;
  p.total = a->total_rows;
  p.hq = a->hq;
  p.hkv = a->hkv;
  p.d = a->d;
  p.cu = a->cu_rows;
  p.seq_lens = a->seq_lens;
  p.block_table = a->block_table;
  p.max_blocks = a->max_blocks_per_req;
  p.num_blocks = a->num_blocks;
  p.block_size = a->block_size;
  while ((1 << p.log2_block) < a->block_size) ++p.log2_block;
  p.capacity = (long long)a->max_blocks_per_req * a->block_size;
  p.format = a->kv_format == GCS_KV_BF16 ? kCacheBf16
             : a->scale_mode == GCS_SCALE_PER_TENSOR ? kCachePerTensor : kCachePerToken;
  p.k_cache = static_cast<uint8_t*>(a->k_cache);
  p.v_cache = static_cast<uint8_t*>(a->v_cache);
  p.kv_bs = cl.bs, p.kv_hs = cl.hs, p.kv_ss = cl.ss;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.g_cache = a->g_cache;
  Layout lk, lv;
  resolve_layout(a->k_stride, a->hkv, a->d, &lk);
  resolve_layout(a->v_stride, a->hkv, a->d, &lv);
  p.k_ts = lk.ts, p.k_hs = lk.hs, p.v_ts = lv.ts, p.v_hs = lv.hs;
  return p;
}

// Bytes of the gates' tile sums.
static size_t append_ws(const gcs_cache_args* a) {
  if (!a->g_cache || !cache_gates_need_sums(a->max_rows)) return 0;
  return round_up((size_t)cache_gate_slots(a->total_rows, a->num_reqs) * a->hq * sizeof(float));
}

size_t attn_cache_append_workspace(const gcs_cache_args* a) { return check_cache(a) == GCS_OK ? append_ws(a) : 0; }

// Both appends: r and q_out are null without the rotation, k is null with it.
static int cache_append(const gcs_cache_args* a, const gcs_qk_rope_args* r, const void* k, const void* v,
                        const float* log_gate, void* q_out, void* workspace, size_t workspace_bytes,
                        gcs_stream_t stream) {
  int st = check_cache(a);
  if (st != GCS_OK) return st;
  if (r) {
    if ((st = check_rope(r, true)) != GCS_OK) return st;
    if (r->total_tokens != a->total_rows || r->hq != a->hq || r->hkv != a->hkv || r->d != a->d)
      return GCS_ERR_INVALID_ARG;
    if (!q_out || !aligned16(q_out)) return GCS_ERR_INVALID_ARG;
  } else if (!k || !aligned16(k)) {
    return GCS_ERR_INVALID_ARG;
  }
  if (!v || !aligned16(v) || !aligned4(log_gate)) return GCS_ERR_INVALID_ARG;
  if ((log_gate == nullptr) != (a->g_cache == nullptr)) return GCS_ERR_INVALID_ARG;
  CacheLayout cl;
  cache_args_layout(a, &cl);
  const CacheSpans cs = cache_spans(a, cl);
  if (caches_meet(a, cl, cs)) return GCS_ERR_INVALID_ARG;
  CacheParams p = cache_params(a, cl);
  RopeParams q{};
  const TSpan none = tspan(Span{0, 0});
  RopeSpans rs{none, none, none, none, none, none};
  const int T = a->total_rows;
  const Layout lk{p.k_ts, p.k_hs}, lv{p.v_ts, p.v_hs};
  TSpan qo = none;
  if (r) {
    const RopeLayouts rl = rope_layouts(r);
    q = rope_params(r, rl);
    rs = rope_spans(r, rl);
    qo = tspan(q_out, T, a->hq, a->d, rl.q_out, 2);
    q.q_out = static_cast<uint16_t*>(q_out);
    p.k = q.k, p.k_ts = q.k_ts, p.k_hs = q.k_hs;
  } else {
    rs.k = tspan(k, T, a->hkv, a->d, lk, 2);
    p.k = static_cast<const uint16_t*>(k);
  }
  p.v = static_cast<const uint16_t*>(v);
  p.log_gate = log_gate;
  const bool per_token = p.format == kCachePerToken;
  // K against V was checked above; here each against everything else
  const TSpan ins[] = {rs.q, rs.k, rs.qw, rs.kw, rs.table, rs.pos, tspan(v, T, a->hkv, a->d, lv, 2),
                       tspan(span(log_gate, (size_t)T * a->hq * 4)), cs.table, cs.lens, cs.cu,
                       per_token ? none : cs.ks, per_token ? none : cs.vs};
  const TSpan outs_k[] = {cs.k, per_token ? cs.ks : none, per_token ? cs.vs : none, cs.g, qo};
  const TSpan outs_v[] = {cs.v, per_token ? cs.ks : none, per_token ? cs.vs : none, cs.g, qo};
  if (outputs_overlap(outs_k, ins) || outputs_overlap(outs_v, ins)) return GCS_ERR_INVALID_ARG;
  const size_t need = append_ws(a);
  if (need > 0) {
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
      return GCS_ERR_WORKSPACE;
    p.tile_sums = static_cast<float*>(workspace);
  }
  p.status = q.status = device_status_ptr();
  if (!p.status) return GCS_ERR_CUDA;
  return cuda_status(launch_cache_append(p, r ? &q : nullptr, reinterpret_cast<cudaStream_t>(stream)));
}

int attn_cache_append(const gcs_cache_args* a, const void* k, const void* v, const float* log_gate, void* workspace,
                      size_t workspace_bytes, gcs_stream_t stream) {
  return cache_append(a, nullptr, k, v, log_gate, nullptr, workspace, workspace_bytes, stream);
}

int attn_cache_append_rope(const gcs_cache_args* a, const gcs_qk_rope_args* r, const void* v, const float* log_gate,
                           void* q_out, void* workspace, size_t workspace_bytes, gcs_stream_t stream) {
  if (!r) return GCS_ERR_INVALID_ARG;
  return cache_append(a, r, nullptr, v, log_gate, q_out, workspace, workspace_bytes, stream);
}

int attn_cache_gather(const gcs_cache_args* a, void* k, void* v, float* log_gate, gcs_stream_t stream) {
  const int st = check_cache(a);
  if (st != GCS_OK) return st;
  if (!k || !v || !aligned16(k) || !aligned16(v) || !aligned4(log_gate)) return GCS_ERR_INVALID_ARG;
  if ((log_gate == nullptr) != (a->g_cache == nullptr)) return GCS_ERR_INVALID_ARG;
  CacheLayout cl;
  cache_args_layout(a, &cl);
  const CacheSpans cs = cache_spans(a, cl);
  CacheParams p = cache_params(a, cl);
  const int T = a->total_rows;
  const TSpan outs[] = {tspan(k, T, a->hkv, a->d, Layout{p.k_ts, p.k_hs}, 2),
                        tspan(v, T, a->hkv, a->d, Layout{p.v_ts, p.v_hs}, 2),
                        tspan(span(log_gate, (size_t)T * a->hq * 4))};
  const TSpan ins[] = {cs.k, cs.v, cs.ks, cs.vs, cs.g, cs.table, cs.lens, cs.cu};
  if (outputs_overlap(outs, ins)) return GCS_ERR_INVALID_ARG;
  p.k_out = static_cast<uint16_t*>(k);
  p.v_out = static_cast<uint16_t*>(v);
  p.log_gate_out = log_gate;
  p.status = device_status_ptr();
  if (!p.status) return GCS_ERR_CUDA;
  return cuda_status(launch_cache_gather(p, reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ eviction from the paged cache

static int log2_of(int block_size) {
  int n = 0;
  while ((1 << n) < block_size) ++n;
  return n;
}
static bool block_size_supported(int n) { return n >= 16 && n <= 4096 && (n & (n - 1)) == 0; }

// The arguments of the weights: those of the paged attention calls, without its limits on shapes and
// without the values.
static int check_weights(const gcs_decode_args* a) {
  if (!a) return GCS_ERR_INVALID_ARG;
  if (a->num_reqs < 1 || a->total_q < 1 || a->max_q_len < 1 || a->max_seq_len < 1 || a->max_blocks_per_req < 1 ||
      a->num_blocks < 1 || a->hq < 1 || a->hkv < 1 || a->hq % a->hkv != 0 || a->window < 0)
    return GCS_ERR_INVALID_ARG;
  if (!a->cu_q || !a->seq_lens || !a->block_table || !a->k_cache || !a->q) return GCS_ERR_INVALID_ARG;
  if (!std::isfinite(a->scale) || a->max_q_len > a->max_seq_len) return GCS_ERR_INVALID_ARG;
  if (!aligned16(a->k_cache) || !aligned16(a->q) || !aligned16(a->g_cache) || !aligned4(a->k_scale) ||
      !aligned4(a->sink) || !aligned4(a->cu_q) || !aligned4(a->seq_lens) || !aligned4(a->block_table))
    return GCS_ERR_INVALID_ARG;
  if (a->kv_format == GCS_KV_BF16) {
    if (a->k_scale || a->scale_mode != GCS_SCALE_PER_TOKEN) return GCS_ERR_INVALID_ARG;
  } else if (a->kv_format == GCS_KV_FP8_E4M3) {
    if (!a->k_scale) return GCS_ERR_INVALID_ARG;
    if (a->scale_mode != GCS_SCALE_PER_TOKEN && a->scale_mode != GCS_SCALE_PER_TENSOR) return GCS_ERR_INVALID_ARG;
  } else {
    return GCS_ERR_INVALID_ARG;
  }
  if (!head_dim_supported(a->d) || !block_size_supported(a->block_size)) return GCS_ERR_UNSUPPORTED;
  if ((long long)a->max_blocks_per_req * a->block_size < a->max_seq_len) return GCS_ERR_INVALID_ARG;
  // positions with a step ahead, rows x heads of a request and the launch grids within 32 bits
  if (a->max_seq_len > 1 << 30 || a->total_q > 1 << 30 || a->num_reqs > 65535 || a->hkv > 65535 ||
      (double)a->max_q_len * (a->hq / a->hkv) > 1073741824.0 || (double)a->hq * a->d > 2147483647.0)
    return GCS_ERR_UNSUPPORTED;
  if ((double)a->num_blocks * a->hkv * a->block_size * a->d > 9.0e15) return GCS_ERR_UNSUPPORTED;
  CacheLayout cl;
  const int st = cache_layout(a, &cl);
  if (st != GCS_OK) return st;
  Layout lq;
  return resolve_layout(a->q_stride, a->hq, a->d, &lq);
}

struct WeightsPlan {
  bool wide = false;  // the long form
  int seg_len = 0, segs = 0;
  size_t part = 0, rows = 0;  // bytes of the sums' parts; long form: of the rows' constants
  bool queries = false;       // long form: fp8 (in f16) or given sums (rows without one as zeros): a copy of the queries
  size_t ws = 0;              // + that copy
};
static bool plan_weights(const gcs_decode_args* a, bool with_lse, WeightsPlan* pl) {
  const int sms = current_sms();
  if (!sms) return false;
  const int group = a->hq / a->hkv;
  const long long units = (long long)a->num_reqs * a->hkv;
  const size_t rows = (size_t)a->total_q * a->hq;
  pl->wide = cache_weights_long(a->max_q_len, group, a->g_cache != nullptr);
  pl->seg_len = pl->wide ? cache_weights_long_segment(a->max_seq_len, a->max_q_len, group, a->d, units, sms)
                         : cache_weights_segment(a->max_seq_len, units, sms);
  pl->segs = (a->max_seq_len + pl->seg_len - 1) / pl->seg_len;
  pl->part = with_lse ? 0 : round_up(pl->segs * rows * sizeof(float2));
  pl->rows = pl->wide ? round_up(rows * sizeof(float2)) : 0;
  pl->queries = pl->wide && (a->kv_format != GCS_KV_BF16 || with_lse);
  pl->ws = pl->part + pl->rows + (pl->queries ? round_up(rows * a->d * 2) : 0);
  return true;
}

size_t attn_cache_weights_workspace(const gcs_decode_args* a, int with_lse) {
  WeightsPlan pl;
  return check_weights(a) == GCS_OK && plan_weights(a, with_lse != 0, &pl) ? pl.ws : 0;
}

int attn_cache_weights(const gcs_decode_args* a, const float* lse, const int32_t* first_lens, float decay,
                       float* w_cache, void* workspace, size_t workspace_bytes, gcs_stream_t stream) {
  const int st = check_weights(a);
  if (st != GCS_OK) return st;
  if (!w_cache || !aligned16(w_cache) || !aligned4(lse) || !aligned4(first_lens) || !std::isfinite(decay))
    return GCS_ERR_INVALID_ARG;
  CacheLayout cl;
  Layout lq;
  cache_layout(a, &cl);
  resolve_layout(a->q_stride, a->hq, a->d, &lq);
  const size_t rows = (size_t)a->num_blocks * a->hkv * a->block_size;
  const size_t elt = a->kv_format == GCS_KV_BF16 ? 2 : 1;
  const size_t cache_bytes = (size_t)(a->num_blocks - 1) * cl.bs + (size_t)(a->hkv - 1) * cl.hs +
                             (size_t)(a->block_size - 1) * cl.ss + (size_t)a->d * elt;
  const TSpan outs[] = {tspan(span(w_cache, rows * 4))};
  const TSpan ins[] = {tspan(a->q, a->total_q, a->hq, a->d, lq, 2),
                       tspan(span(a->k_cache, cache_bytes)),
                       tspan(span(a->k_scale, a->scale_mode == GCS_SCALE_PER_TENSOR ? 4 : rows * 4)),
                       tspan(span(a->block_table, (size_t)a->num_reqs * a->max_blocks_per_req * 4)),
                       tspan(span(a->seq_lens, (size_t)a->num_reqs * 4)),
                       tspan(span(a->cu_q, ((size_t)a->num_reqs + 1) * 4)),
                       tspan(span(a->g_cache, (size_t)a->num_blocks * a->hq * a->block_size * 4)),
                       tspan(span(a->sink, (size_t)a->hq * 4)),
                       tspan(span(lse, (size_t)a->hq * a->total_q * 4)),
                       tspan(span(first_lens, (size_t)a->num_reqs * 4))};
  if (outputs_overlap(outs, ins)) return GCS_ERR_INVALID_ARG;
  WeightsPlan pl;
  if (!plan_weights(a, lse != nullptr, &pl)) return GCS_ERR_CUDA;
  if (pl.ws > 0 && (!workspace || workspace_bytes < pl.ws || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
    return GCS_ERR_WORKSPACE;
  WeightsParams p{};
  p.cu_q = a->cu_q;
  p.seq_lens = a->seq_lens;
  p.block_table = a->block_table;
  p.max_blocks = a->max_blocks_per_req;
  p.num_blocks = a->num_blocks;
  p.block_size = a->block_size;
  p.log2_block = log2_of(a->block_size);
  p.num_reqs = a->num_reqs;
  p.total_q = a->total_q;
  p.max_q_len = a->max_q_len;
  p.max_seq_len = a->max_seq_len;
  p.hq = a->hq;
  p.hkv = a->hkv;
  p.group = a->hq / a->hkv;
  p.d = a->d;
  p.format = a->kv_format == GCS_KV_BF16 ? kCacheBf16
             : a->scale_mode == GCS_SCALE_PER_TENSOR ? kCachePerTensor : kCachePerToken;
  p.k_cache = static_cast<const uint8_t*>(a->k_cache);
  p.kv_bs = cl.bs, p.kv_hs = cl.hs, p.kv_ss = cl.ss;
  p.k_scale = a->k_scale;
  p.g_cache = a->g_cache;
  p.sink = a->sink;
  p.window = a->window < a->max_seq_len ? a->window : 0;  // sees everything; position - window stays within 32 bits
  p.scale = a->scale;
  p.decay = decay;
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_ts = lq.ts, p.q_hs = lq.hs;
  p.lse = lse;
  p.first_lens = first_lens;
  p.w_cache = w_cache;
  p.part = static_cast<float2*>(workspace);
  p.seg_len = pl.seg_len;
  p.segs = pl.segs;
  p.kv_head_inner = cl.head_inner() ? 1 : 0;
  p.status = device_status_ptr();
  if (!p.status) return GCS_ERR_CUDA;
  if (pl.wide) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.rows = reinterpret_cast<float2*>(ws + pl.part);
    p.q16 = pl.queries ? reinterpret_cast<uint16_t*>(ws + pl.part + pl.rows) : nullptr;
    const bool bf16 = a->kv_format == GCS_KV_BF16;
    WeightsMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    const Layout packed{(long long)a->hq * a->d, a->d};
    if (bf16 && !make_page_map_bf16(&maps.k, a->k_cache, a->num_blocks, a->hkv, a->block_size, a->d, cl))
      return GCS_ERR_CUDA;
    if (!make_query_map(&maps.q, p.q16 ? p.q16 : a->q, !bf16, a->d, a->hq, a->total_q, p.q16 ? packed : lq, p.group,
                        128 / p.group))
      return GCS_ERR_CUDA;
    return cuda_status(launch_cache_weights_long(p, maps, reinterpret_cast<cudaStream_t>(stream)));
  }
  return cuda_status(launch_cache_weights(p, reinterpret_cast<cudaStream_t>(stream)));
}

int attn_cache_select(const gcs_select_args* a, int32_t* kept, int32_t* kept_lens, gcs_stream_t stream) {
  if (!a || a->num_reqs < 1 || a->hkv < 1 || a->max_seq_len < 1 || a->max_blocks_per_req < 1 || a->num_blocks < 1 ||
      a->recent < 0 || a->max_keep < 1)
    return GCS_ERR_INVALID_ARG;
  if (!a->w_cache || !a->block_table || !a->seq_lens || !a->budgets || !kept || !kept_lens) return GCS_ERR_INVALID_ARG;
  if (!aligned16(a->w_cache) || !aligned4(a->block_table) || !aligned4(a->seq_lens) || !aligned4(a->budgets) ||
      !aligned4(a->first_lens) || !aligned4(kept) || !aligned4(kept_lens))
    return GCS_ERR_INVALID_ARG;
  if (!block_size_supported(a->block_size)) return GCS_ERR_UNSUPPORTED;
  if ((long long)a->max_blocks_per_req * a->block_size < a->max_seq_len) return GCS_ERR_INVALID_ARG;
  // positions, and the grid of up to 16 blocks a (request, kv head)
  if (a->max_seq_len > 1 << 30 || a->max_keep > 1 << 30 || (double)a->num_reqs * a->hkv > 134217727.0)
    return GCS_ERR_UNSUPPORTED;
  const size_t R = (size_t)a->num_reqs;
  const TSpan outs[] = {tspan(span(kept, R * a->hkv * a->max_keep * 4)), tspan(span(kept_lens, R * 4))};
  const TSpan ins[] = {tspan(span(a->w_cache, (size_t)a->num_blocks * a->hkv * a->block_size * 4)),
                       tspan(span(a->block_table, R * a->max_blocks_per_req * 4)), tspan(span(a->seq_lens, R * 4)),
                       tspan(span(a->budgets, R * 4)), tspan(span(a->first_lens, R * 4))};
  if (outputs_overlap(outs, ins)) return GCS_ERR_INVALID_ARG;
  SelectParams p{};
  p.num_reqs = a->num_reqs;
  p.hkv = a->hkv;
  p.seq_lens = a->seq_lens;
  p.block_table = a->block_table;
  p.max_blocks = a->max_blocks_per_req;
  p.num_blocks = a->num_blocks;
  p.block_size = a->block_size;
  p.log2_block = log2_of(a->block_size);
  p.max_seq_len = a->max_seq_len;
  p.w_cache = a->w_cache;
  p.budgets = a->budgets;
  p.first_lens = a->first_lens;
  p.recent = a->recent;
  p.max_keep = a->max_keep;
  p.kept = kept;
  p.kept_lens = kept_lens;
  p.status = device_status_ptr();
  if (!p.status) return GCS_ERR_CUDA;
  return cuda_status(launch_cache_select(p, reinterpret_cast<cudaStream_t>(stream)));
}

int attn_cache_compact(const gcs_cache_args* a, const int32_t* kept, const int32_t* kept_lens, int max_keep,
                       float* w_cache, gcs_stream_t stream) {
  if (!a) return GCS_ERR_INVALID_ARG;
  gcs_cache_args b = *a;  // no packed rows here
  b.cu_rows = b.seq_lens;
  b.total_rows = b.max_rows = 1;
  b.k_stride = b.v_stride = gcs_strides{0, 0};
  const int st = check_cache(&b);
  if (st != GCS_OK) return st;
  if (!kept || !kept_lens || max_keep < 1 || !aligned4(kept) || !aligned4(kept_lens) || !aligned4(w_cache) ||
      !aligned4(a->first_lens))
    return GCS_ERR_INVALID_ARG;
  // positions, and the grid of up to 8 blocks a (request, kv head) and eight vectors
  if (max_keep > 1 << 30 || (double)a->num_reqs * a->hkv > 268435455.0 || a->hq / a->hkv > 1 << 18)
    return GCS_ERR_UNSUPPORTED;
  CacheLayout cl;
  cache_args_layout(&b, &cl);
  const CacheSpans cs = cache_spans(&b, cl);
  if (caches_meet(&b, cl, cs)) return GCS_ERR_INVALID_ARG;
  const CacheParams c = cache_params(&b, cl);
  const bool per_token = c.format == kCachePerToken;
  const TSpan none = tspan(Span{0, 0});
  const size_t R = (size_t)a->num_reqs, rows = (size_t)a->num_blocks * a->hkv * a->block_size;
  const TSpan ks = per_token ? cs.ks : none, vs = per_token ? cs.vs : none, w = tspan(span(w_cache, rows * 4));
  const TSpan ins[] = {cs.table, cs.lens, tspan(span(kept, R * a->hkv * max_keep * 4)), tspan(span(kept_lens, R * 4)),
                       tspan(span(a->first_lens, R * 4))};
  // K against V was checked above
  const TSpan outs_k[] = {cs.k, ks, vs, cs.g, w}, outs_v[] = {cs.v, ks, vs, cs.g, w};
  if (outputs_overlap(outs_k, ins) || outputs_overlap(outs_v, ins)) return GCS_ERR_INVALID_ARG;
  MoveParams p{};
  p.num_reqs = a->num_reqs;
  p.hkv = a->hkv;
  p.group = a->hq / a->hkv;
  p.seq_lens = a->seq_lens;
  p.block_table = a->block_table;
  p.kept = kept;
  p.kept_lens = kept_lens;
  p.first_lens = a->first_lens;
  p.max_blocks = c.max_blocks;
  p.num_blocks = c.num_blocks;
  p.block_size = c.block_size;
  p.log2_block = c.log2_block;
  p.max_keep = max_keep;
  p.capacity = c.capacity;
  p.k_cache = c.k_cache;
  p.v_cache = c.v_cache;
  p.kv_bs = c.kv_bs, p.kv_hs = c.kv_hs, p.kv_ss = c.kv_ss;
  p.log2_units = log2_of(a->d * (c.format == kCacheBf16 ? 2 : 1) / 16);
  p.k_scale = per_token ? c.k_scale : nullptr;
  p.v_scale = per_token ? c.v_scale : nullptr;
  p.g_cache = c.g_cache;
  p.w_cache = w_cache;
  p.last_stays = c.g_cache && device_checks_on() ? 1 : 0;
  p.status = device_status_ptr();
  if (!p.status) return GCS_ERR_CUDA;
  return cuda_status(launch_cache_move(p, reinterpret_cast<cudaStream_t>(stream)));
}

int gcs_set_device_checks(int enable) {
  if (enable != 0 && enable != 1) return GCS_ERR_INVALID_ARG;
  g_device_checks.store(enable, std::memory_order_relaxed);
  return GCS_OK;
}

int gcs_get_device_checks(void) { return device_checks_on() ? 1 : 0; }

int gcs_check_prefill_inputs(const gcs_prefill_args* a, gcs_stream_t stream) {
  const int st = check_prefill(a);
  if (st != GCS_OK) return st;
  int* status = device_status_ptr();
  if (!status) return GCS_ERR_CUDA;
  return cuda_status(launch_check_prefill(a->cu_seqlens, a->num_seqs, a->total_tokens, a->max_seqlen, nullptr, status,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

int gcs_check_paged_inputs(const gcs_decode_args* a, gcs_stream_t stream) {
  // the arguments of either paged call
  if (check_decode(a) != GCS_OK) {
    const int st = check_prefill_paged(a);
    if (st != GCS_OK) return st;
  }
  int* status = device_status_ptr();
  if (!status) return GCS_ERR_CUDA;
  return cuda_status(launch_check_paged(a->cu_q, a->seq_lens, a->block_table, a->num_reqs, a->total_q, a->max_q_len,
                                        a->max_seq_len, a->max_blocks_per_req, a->num_blocks, a->block_size,
                                        a->window, operand_check(a), SharedPrefixes{}, nullptr, status,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

int gcs_set_kernel_events(void* before, void* after) {
  t_ev_before = static_cast<cudaEvent_t>(before);
  t_ev_after = static_cast<cudaEvent_t>(after);
  return GCS_OK;
}

int gcs_selftest_bounded_wait(gcs_stream_t stream) {
  int* d = device_status_ptr();
  if (!d) return GCS_ERR_CUDA;
  return cuda_status(launch_bounded_wait_selftest(d, reinterpret_cast<cudaStream_t>(stream)));
}

int gcs_get_device_status(int* status, int clear) {
  if (!status) return GCS_ERR_INVALID_ARG;
  int* d = device_status_ptr();
  if (!d) return GCS_ERR_CUDA;
  if (cudaMemcpy(status, d, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return GCS_ERR_CUDA;
  if (clear && cudaMemset(d, 0, sizeof(int)) != cudaSuccess) return GCS_ERR_CUDA;
  return GCS_OK;
}

}  // extern "C"
