// The choice of the cached tokens that stay, and their move to the front of the pages.
//
// Choice: of request r's L cached tokens n = min(budget, L) stay, for each kv head on its own: the
// last `recent`, then the first `first`, then those of the largest weight (w_cache, paged like the
// scales); of equal weights the lowest position.  The positions come out in ascending order.
// Move: position i of (request, kv head) takes what position kept[i] holds, in place.
//
// Every index that comes from a device array is checked before it is used.
#include <algorithm>

#include <cooperative_groups.h>

#include "kernels.h"
#include "sm103_ptx.cuh"

namespace gcs {
namespace {

namespace cg = cooperative_groups;

__device__ __forceinline__ void record_bad(int* status) { atomicCAS(status, kDevOk, kDevInvalidArg); }

// ------------------------------------------------------------------------------------ choice
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;          // digits of 11, 11 and 10 bits
constexpr int kMaxSlice = 40 * 1024; // keys of a block in shared memory
constexpr int kRanked = 512;         // keys up to which each counts those above it

// Weights as integers of the same order: NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  if (f != f) return 0u;
  if (f == 0.f) return 0x80000000u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One cluster for a (request, kv head): its blocks take equal slices of the positions between the
// first and the last ones, as quads of four neighbouring positions (one vector load: a quad lies in
// one cache block).  The key of rank c from the top is found by three histograms of 11, 11 and 10 bits, each
// added up over the cluster; a last walk in the order of the positions writes those above it and as
// many equal ones as are still missing.  11 bits of a positive float are its exponent and two bits
// more, so few of a warp's keys meet in a bin, and the second histogram is of few keys.
// HELD: the slice's keys stay in shared memory; otherwise (slices past kMaxSlice) each walk reads the
// weights again.  CLUSTER: more than one block.
template <bool HELD, bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint4 keys[];
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_a[kSelWarps], warp_b[kSelWarps];
  __shared__ uint32_t tot_gt, tot_eq;
  __shared__ uint32_t digit_s, above_s;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = CLUSTER ? cluster.num_blocks() : 1, rank = CLUSTER ? cluster.block_rank() : 0;
  auto all_sync = [&]() {
    if (CLUSTER) cluster.sync();
    else __syncthreads();
  };
  auto of_rank = [&](uint32_t* x, int k) { return CLUSTER ? *cluster.map_shared_rank(x, k) : *x; };
  const int row = blockIdx.x / cs;
  const int r = row / p.hkv, h = row % p.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  int L = __ldg(p.seq_lens + r);
  if (L < 0 || L > p.max_seq_len) {  // max_seq_len is within the table (checked on the host)
    if (tid == 0) record_bad(p.status);
    L = 0;
  }
  const int n = max(0, min(min(__ldg(p.budgets + r), p.max_keep), L));
  const int last = min(n, p.recent);
  const int first = p.first_lens ? max(0, __ldg(p.first_lens + r)) : 0;
  const int lead = min(n - last, min(first, L - last));
  const int need = n - last - lead;  // by weight, from the positions [lead, end)
  const int end = L - last;
  int32_t* out = p.kept + (size_t)row * p.max_keep;
  if (rank == 0 && tid == 0 && h == 0) p.kept_lens[r] = n;
  for (int i = rank * kSelThreads + tid; i < p.max_keep; i += cs * kSelThreads) {
    if (i < lead) out[i] = i;
    else if (i >= n) out[i] = -1;
    else if (i >= n - last) out[i] = L - n + i;
  }
  // the whole cluster leaves together
  if (need == 0) return;
  if (need == end - lead) {
    for (int i = rank * kSelThreads + tid; i < need; i += cs * kSelThreads) out[lead + i] = lead + i;
    return;
  }
  const int32_t* table = p.block_table + (size_t)r * p.max_blocks;
  auto weights = [&](int pos) -> const float* {  // null: never looked at, as if nothing weighed less
    const int blk = __ldg(table + (pos >> p.log2_block));
    if (blk < 0 || blk >= p.num_blocks) {
      record_bad(p.status);
      return nullptr;
    }
    return p.w_cache + (((size_t)blk * p.hkv + h) << p.log2_block) + (pos & (p.block_size - 1));
  };

  if (end - lead <= kRanked) {
    // few keys: each counts those that go before it
    if (rank != 0) return;
    const int m = end - lead;
    uint32_t mine = 0;
    if (tid < m) {
      const float* w = weights(lead + tid);
      mine = w ? order_key(__ldg(w)) : 0u;
    }
    hist[tid] = mine;
    __syncthreads();
    int before = 0;
    for (int j = 0; j < m; ++j) {
      const uint32_t k = hist[j];
      before += k > mine || (k == mine && j < tid);
    }
    const bool stays = tid < m && before < need;
    const uint32_t votes = __ballot_sync(0xffffffffu, stays);
    if (lane == 0) warp_a[warp] = __popc(votes);
    __syncthreads();
    int at = lead + __popc(votes & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) at += warp_a[w];
    if (stays) out[at] = lead + tid;
    return;
  }

  const int q0 = lead >> 2, nq = ((end + 3) >> 2) - q0;  // quads, the first and last partly outside
  const int per = (nq + cs - 1) / cs;
  const int a = q0 + min(nq, rank * per), b = q0 + min(nq, rank * per + per);
  auto load = [&](int q) -> uint4 {
    const float* at = weights(q * 4);
    if (!at) return make_uint4(0, 0, 0, 0);
    const float4 w = __ldg(reinterpret_cast<const float4*>(at));
    return make_uint4(order_key(w.x), order_key(w.y), order_key(w.z), order_key(w.w));
  };
  auto quad = [&](int q) -> uint4 { return HELD ? keys[q - a] : load(q); };
  for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
  __syncthreads();

  uint32_t prefix = 0, left = need;  // bits found so far; how many are wanted among the keys with them
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    const uint32_t digits = round == 2 ? 1023 : 2047;
    const uint32_t mask = round == 0 ? 0u : round == 1 ? 0xffe00000u : 0xfffffc00u;
    auto count = [&](int q, const uint4& k) {
      const uint32_t e[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((e[j] & mask) == prefix && q * 4 + j >= lead && q * 4 + j < end)
          atomicAdd(&hist[(e[j] >> shift) & digits], 1u);
    };
    if (HELD && round == 0) {  // the only read of the weights
      for (int q = a + tid; q < b; q += 4 * kSelThreads) {
        uint4 k[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (q + u * kSelThreads < b) k[u] = load(q + u * kSelThreads);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (q + u * kSelThreads < b) {
            keys[q + u * kSelThreads - a] = k[u];
            count(q + u * kSelThreads, k[u]);
          }
      }
    } else {
      for (int q = a + tid; q < b; q += kSelThreads) count(q, quad(q));
    }
    all_sync();
    // thread's 4 bins from the top: 2047 - 4 tid .. 2044 - 4 tid
    uint4 c = make_uint4(0, 0, 0, 0);
    const int top = kBins / 4 - 1 - tid;
    for (int k = 0; k < cs; ++k) {
      const uint4* hk = reinterpret_cast<const uint4*>(CLUSTER ? cluster.map_shared_rank(hist, k) : hist);
      const uint4 v = hk[top];
      c.x += v.x, c.y += v.y, c.z += v.z, c.w += v.w;
    }
    const uint32_t sum = c.x + c.y + c.z + c.w;
    uint32_t before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += t;
    }
    if (lane == 31) warp_a[warp] = before;
    before -= sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += warp_a[w];
    if (before < left && before + sum >= left) {  // one thread's
      const uint32_t v[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (before < left && before + v[j] >= left) {
          digit_s = kBins - 1 - 4 * tid - j;
          above_s = before;
        }
        before += v[j];
      }
    }
    all_sync();  // the bins are read
    prefix |= digit_s << shift;
    left -= above_s;
    for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
  }

  // prefix is the key of rank `need`; `left` of those equal to it stay
  const int nql = b - a, chunk = (nql + kSelWarps - 1) / kSelWarps;
  const int wa = a + min(nql, warp * chunk), wb = a + min(nql, warp * chunk + chunk);
  uint32_t gt = 0, eq = 0;
  for (int q = wa + lane; q < wb; q += 32) {
    const uint4 k = quad(q);
    const uint32_t e[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = q * 4 + j >= lead && q * 4 + j < end;
      gt += in && e[j] > prefix;
      eq += in && e[j] == prefix;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    warp_a[warp] = gt;
    warp_b[warp] = eq;
  }
  __syncthreads();
  if (CLUSTER) {
    if (tid == 0) {
      uint32_t g = 0, e = 0;
      for (int w = 0; w < kSelWarps; ++w) {
        g += warp_a[w];
        e += warp_b[w];
      }
      tot_gt = g;
      tot_eq = e;
    }
    all_sync();
  }
  uint32_t gt0 = 0, eq0 = 0;
  for (int k = 0; k < rank; ++k) {
    gt0 += of_rank(&tot_gt, k);
    eq0 += of_rank(&tot_eq, k);
  }
  for (int w = 0; w < warp; ++w) {
    gt0 += warp_a[w];
    eq0 += warp_b[w];
  }
  for (int q = wa; q < wb; q += 32) {  // the warp's quads in order
    const bool here = q + lane < wb;
    uint4 k = make_uint4(0, 0, 0, 0);
    if (here) k = quad(q + lane);
    const uint32_t e[4] = {k.x, k.y, k.z, k.w};
    const int pos = (q + lane) * 4;
    uint32_t g = 0, t = 0;  // bits
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = here && pos + j >= lead && pos + j < end;
      g |= (in && e[j] > prefix ? 1u : 0u) << j;
      t |= (in && e[j] == prefix ? 1u : 0u) << j;
    }
    const uint32_t mine = __popc(g) | __popc(t) << 16;
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t s = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += s;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, sum, 31);
    uint32_t gb = gt0 + ((sum - mine) & 0xffffu), eb = eq0 + ((sum - mine) >> 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool is_g = g >> j & 1, is_t = t >> j & 1;
      if (is_g || (is_t && eb < left)) out[lead + gb + min(eb, left)] = pos + j;
      gb += is_g;
      eb += is_t;
    }
    gt0 += all & 0xffffu;
    eq0 += all >> 16;
  }
  if (CLUSTER) all_sync();  // no block leaves while its totals are read
}

// -------------------------------------------------------------------------------------- move
constexpr int kMoveThreads = 256;
constexpr int kPieces = 4;   // 16-byte pieces of K or V a thread moves in a chunk
constexpr int kVectors = 8;  // 4-byte vectors of a block, one element each of a thread's chunk
constexpr int kDepth = 4;    // chunks on their way
constexpr int kMoveSmem = kDepth * kMoveThreads * kPieces * 16;

// A stream is one array's part of one (request, kv head): the K rows, the V rows, or up to eight of
// the 4-byte vectors (scales, weights, gates of its query heads).  A cluster takes one stream's
// target positions in ascending order, a chunk at a time, kDepth chunks ahead into shared memory; a chunk
// is written only when every block of the cluster has read it.  In place this
// is right for any kept[i] >= i: the sources of chunk c lie at or behind its first target, so no
// earlier chunk's targets hold them, and a target that is a source of its own or an earlier
// chunk has been read before it is written.  Every thread writes what it read itself: shared memory is
// only its queue, and the barrier of chunk c + 1 is under way while chunk c is written.
struct Target {
  int to, slot;  // block (-1: nothing to move) and slot
};

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool CLUSTER>
__device__ __forceinline__ void all_arrive() {
  if (CLUSTER) cg::cluster_group::barrier_arrive();
}
template <bool CLUSTER>
__device__ __forceinline__ void all_wait() {
  if (CLUSTER) cg::cluster_group::barrier_wait();
  else __syncthreads();
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kMoveThreads, 3) cache_move_kernel(const MoveParams p, int cs) {
  extern __shared__ __align__(16) uint8_t queue[];
  const int rank = CLUSTER ? blockIdx.x % cs : 0, row = CLUSTER ? blockIdx.x / cs : blockIdx.x, kind = blockIdx.y;
  const int r = row / p.hkv, h = row % p.hkv;
  const int tid = threadIdx.x;
  const int L = __ldg(p.seq_lens + r), n = __ldg(p.kept_lens + r);
  if (L < 0 || L > p.capacity || n < 0 || n > p.max_keep || n > L) {  // the same for the whole cluster
    if (tid == 0) record_bad(p.status);
    return;
  }
  const int32_t* table = p.block_table + (size_t)r * p.max_blocks;
  const int32_t* kept = p.kept + (size_t)row * p.max_keep;
  // Source of target i (from kept, read ahead): block and slot, -1 where there is nothing to move.
  auto source = [&](int i, int src) -> Target {
    if (i >= n || src == i) return Target{-1, 0};
    if (src < i || src >= L) {
      record_bad(p.status);
      return Target{-1, 0};
    }
    const int from = __ldg(table + (src >> p.log2_block)), to = __ldg(table + (i >> p.log2_block));
    if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks) {
      record_bad(p.status);
      return Target{-1, 0};
    }
    return Target{from, src & (p.block_size - 1)};
  };
  auto index = [&](int i) { return i < n ? __ldg(kept + i) : 0; };

  if (kind < 2) {
    uint8_t* cache = (kind ? p.v_cache : p.k_cache) + (size_t)h * p.kv_hs;
    const int log2_units = p.log2_units;  // 16-byte pieces of a row: 4 .. 64
    const int rows = (kMoveThreads * kPieces) >> log2_units;  // of a block's chunk
    const int unit = (tid & ((1 << log2_units) - 1)) * 16, lane_row = tid >> log2_units;
    const int step = kMoveThreads >> log2_units, stride = cs * rows;
    uint4* q = reinterpret_cast<uint4*>(queue) + tid;
    uint32_t moves = 0;  // kPieces bits a chunk, the latest lowest
    int src[kPieces];    // kept of the chunk that is read next
    int ahead = rank * rows + lane_row;  // its first target
#pragma unroll
    for (int u = 0; u < kPieces; ++u) src[u] = index(ahead + u * step);
    int at = 0;  // its place in the queue
    auto read = [&]() {
      moves <<= kPieces;
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const Target s = source(ahead + u * step, src[u]);
        if (s.to >= 0) {
          copy16(q + (at * kPieces + u) * kMoveThreads, cache + (size_t)s.to * p.kv_bs + (size_t)s.slot * p.kv_ss + unit);
          moves |= 1u << u;
        }
        src[u] = index(ahead + stride + u * step);
      }
      copies_end();
      ahead += stride;
      at = at + 1 == kDepth ? 0 : at + 1;
    };
    for (int d = 0; d < kDepth - 1; ++d) read();
    copies_wait<kDepth - 2>();
    all_arrive<CLUSTER>();
    all_wait<CLUSTER>();  // chunk 0 is read
    int i0 = rank * rows + lane_row, out = 0;
    for (int c0 = 0; c0 < n; c0 += stride) {  // c0: the cluster's chunk
      read();
      copies_wait<kDepth - 2>();  // the next chunk is here
      all_arrive<CLUSTER>();
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        if (moves >> (kPieces * (kDepth - 1) + u) & 1) {
          const int i = i0 + u * step;
          *reinterpret_cast<uint4*>(cache + (size_t)__ldg(table + (i >> p.log2_block)) * p.kv_bs +
                                    (size_t)(i & (p.block_size - 1)) * p.kv_ss + unit) =
              q[(out * kPieces + u) * kMoveThreads];
        }
      }
      i0 += stride;
      out = out + 1 == kDepth ? 0 : out + 1;
      all_wait<CLUSTER>();
    }
    copies_wait<0>();
    return;
  }

  // vectors v0 .. v0 + 7 of this (request, kv head)
  const int v0 = (kind - 2) * kVectors;
  float* base[kVectors];
  int heads[kVectors];
#pragma unroll
  for (int v = 0; v < kVectors; ++v) {
    int i = v0 + v;
    base[v] = nullptr;
    heads[v] = p.hkv;
    if (p.k_scale) {
      if (i >= 0 && i < 2) base[v] = (i ? p.v_scale : p.k_scale) + (((size_t)h) << p.log2_block);
      i -= 2;
    }
    if (p.w_cache) {
      if (i == 0) base[v] = p.w_cache + (((size_t)h) << p.log2_block);
      --i;
    }
    if (p.g_cache && i >= 0 && i < p.group) {
      base[v] = p.g_cache + (((size_t)h * p.group + i) << p.log2_block);
      heads[v] = p.hkv * p.group;
    }
  }
  auto cell = [&](int v, int blk, int slot) { return base[v] + (((size_t)blk * heads[v]) << p.log2_block) + slot; };
  float* q = reinterpret_cast<float*>(queue) + tid;
  const int stride = cs * kMoveThreads;
  int ahead = rank * kMoveThreads + tid, at = 0, out = 0, i = ahead;
  int src = index(ahead);
  uint32_t moves = 0;
  auto read = [&]() {
    const Target s = source(ahead, src);
    src = index(ahead + stride);
    moves <<= 1;
    if (s.to >= 0) {
#pragma unroll
      for (int v = 0; v < kVectors; ++v)
        if (base[v]) copy4(q + (at * kVectors + v) * kMoveThreads, cell(v, s.to, s.slot));
      moves |= 1;
    }
    copies_end();
    ahead += stride;
    at = at + 1 == kDepth ? 0 : at + 1;
  };
  for (int d = 0; d < kDepth - 1; ++d) read();
  copies_wait<kDepth - 2>();
  all_arrive<CLUSTER>();
  all_wait<CLUSTER>();
  for (int c0 = 0; c0 < n; c0 += stride) {
    read();
    copies_wait<kDepth - 2>();
    all_arrive<CLUSTER>();
    if (moves >> (kDepth - 1) & 1) {
      const int to = __ldg(table + (i >> p.log2_block)), slot = i & (p.block_size - 1);
#pragma unroll
      for (int v = 0; v < kVectors; ++v)
        if (base[v]) *cell(v, to, slot) = q[(out * kVectors + v) * kMoveThreads];
    }
    i += stride;
    out = out + 1 == kDepth ? 0 : out + 1;
    all_wait<CLUSTER>();
  }
  copies_wait<0>();
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
}

template <typename... Args, typename... Given>
cudaError_t launch_clusters(void (*kern)(Args...), dim3 grid, int threads, int cs, size_t smem, cudaStream_t s,
                            Given... given) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, given...);
}

}  // namespace

cudaError_t launch_cache_select(const SelectParams& p, cudaStream_t s) {
  const int sms = sm_count();
  if (!sms) return cudaErrorInvalidDevice;
  // blocks: about two an SM, no fewer than 2048 keys each
  const long long rows = (long long)p.num_reqs * p.hkv;
  int cs = 1;
  while (cs < 16 && rows * cs < 2 * sms && p.max_seq_len / cs > 2048) cs *= 2;
  const long long slice = ((long long)(p.max_seq_len + 3) / 4 + cs) / cs * 4 + 8;  // keys of a block, at most
  const bool held = slice <= kMaxSlice;
  auto kern = cs == 1 ? (held ? cache_select_kernel<true, false> : cache_select_kernel<false, false>)
                      : (held ? cache_select_kernel<true, true> : cache_select_kernel<false, true>);
  const size_t smem = held ? (size_t)slice * 4 : 0;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && cs > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  if (cs == 1) {
    kern<<<(unsigned)rows, kSelThreads, smem, s>>>(p);
    return cudaGetLastError();
  }
  return launch_clusters(kern, dim3((unsigned)(rows * cs)), kSelThreads, cs, smem, s, p);
}

cudaError_t launch_cache_move(const MoveParams& p, cudaStream_t s) {
  const int sms = sm_count();
  if (!sms) return cudaErrorInvalidDevice;
  const long long rows = (long long)p.num_reqs * p.hkv;
  const int vectors = (p.k_scale ? 2 : 0) + (p.w_cache ? 1 : 0) + (p.g_cache ? p.group : 0);
  const int kinds = 2 + (vectors + kVectors - 1) / kVectors;
  // blocks: about four an SM, no more than the chunks of max_keep rows
  const int chunk = (kMoveThreads * kPieces) >> p.log2_units;
  int cs = 1;
  while (cs < 8 && rows * kinds * cs < 4 * sms && p.max_keep > cs * chunk) cs *= 2;
  const dim3 grid((unsigned)(rows * cs), kinds);
  auto kern = cs > 1 ? cache_move_kernel<true> : cache_move_kernel<false>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoveSmem);
  if (e != cudaSuccess) return e;
  if (cs > 1) return launch_clusters(kern, grid, kMoveThreads, cs, kMoveSmem, s, p, cs);
  kern<<<grid, kMoveThreads, kMoveSmem, s>>>(p, cs);
  return cudaGetLastError();
}

}  // namespace gcs
