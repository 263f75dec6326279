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
constexpr int kCopies = 8;           // of the histogram, one for every eighth lane
constexpr int kMaxSlice = 40 * 1024; // keys of a block in shared memory

// Weights as integers of the same order: NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  if (f != f) return 0u;
  if (f == 0.f) return 0x80000000u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One cluster for a (request, kv head): its blocks take equal slices of the positions between the
// first and the last ones, as quads of four neighbouring positions (one vector load: a quad lies in
// one cache block).  The key of rank c from the top is found by four histograms of 8 bits, each
// added up over the cluster; a last walk in the order of the positions writes those above it and as
// many equal ones as are still missing.  HELD: the slice's keys stay in shared memory; otherwise
// (slices past kMaxSlice) each walk reads the weights again.
template <bool HELD>
__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint4 keys[];
  __shared__ uint32_t hist[256 * kCopies];
  __shared__ uint32_t bins[256];
  __shared__ uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
  __shared__ uint32_t tot_gt, tot_eq;
  __shared__ uint32_t digit_s, above_s;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = cluster.num_blocks(), rank = cluster.block_rank();
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

  const int q0 = lead >> 2, nq = ((end + 3) >> 2) - q0;  // quads, the first and last partly outside
  const int per = (nq + cs - 1) / cs;
  const int a = q0 + min(nq, rank * per), b = q0 + min(nq, rank * per + per);
  const int32_t* table = p.block_table + (size_t)r * p.max_blocks;
  auto load = [&](int q) -> uint4 {
    const int pos = q * 4;
    const int blk = __ldg(table + (pos >> p.log2_block));
    if (blk < 0 || blk >= p.num_blocks) {  // never looked at: as if nothing weighed less
      record_bad(p.status);
      return make_uint4(0, 0, 0, 0);
    }
    const float4 w = __ldg(reinterpret_cast<const float4*>(
        p.w_cache + (((size_t)blk * p.hkv + h) << p.log2_block) + (pos & (p.block_size - 1))));
    return make_uint4(order_key(w.x), order_key(w.y), order_key(w.z), order_key(w.w));
  };
  auto quad = [&](int q) -> uint4 { return HELD ? keys[q - a] : load(q); };
  if (HELD) {
    for (int q = a + tid; q < b; q += kSelThreads) keys[q - a] = load(q);
  }

  uint32_t prefix = 0, left = need;  // bits found so far; how many are wanted among the keys with them
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256 * kCopies; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int q = a + tid; q < b; q += kSelThreads) {
      const uint4 k = quad(q);
      const uint32_t e[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((e[j] & mask) == prefix && q * 4 + j >= lead && q * 4 + j < end)
          atomicAdd(&hist[((e[j] >> shift) & 255) * kCopies + (lane & (kCopies - 1))], 1u);
    }
    __syncthreads();
    if (tid < 256) {
      uint32_t s = 0;
#pragma unroll
      for (int j = 0; j < kCopies; ++j) s += hist[tid * kCopies + ((j + tid) & (kCopies - 1))];
      bins[tid] = s;
    }
    cluster.sync();
    if (warp == 0) {
      // lane's 8 bins from the top: bins 255 - 8 lane .. 248 - 8 lane
      uint32_t c[8], s = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c[j] = 0;
        for (int k = 0; k < cs; ++k) c[j] += *cluster.map_shared_rank(&bins[255 - 8 * lane - j], k);
        s += c[j];
      }
      uint32_t before = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += t;
      }
      before -= s;  // keys above this lane's bins
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (before < left && before + c[j] >= left) {
          digit_s = 255 - 8 * lane - j;
          above_s = before;
        }
        before += c[j];
      }
    }
    __syncthreads();
    prefix |= digit_s << shift;
    left -= above_s;
    cluster.sync();  // the bins are read
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
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t g = 0, e = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      g += warp_gt[w];
      e += warp_eq[w];
    }
    tot_gt = g;
    tot_eq = e;
  }
  cluster.sync();
  uint32_t gt0 = 0, eq0 = 0;
  for (int k = 0; k < rank; ++k) {
    gt0 += *cluster.map_shared_rank(&tot_gt, k);
    eq0 += *cluster.map_shared_rank(&tot_eq, k);
  }
  for (int w = 0; w < warp; ++w) {
    gt0 += warp_gt[w];
    eq0 += warp_eq[w];
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
  cluster.sync();  // no block leaves while its totals are read
}

// -------------------------------------------------------------------------------------- move
constexpr int kMoveThreads = 256;
constexpr int kPieces = 4;   // 16-byte pieces of K or V a thread holds
constexpr int kVectors = 8;  // 4-byte vectors of a block

// A stream is one array's part of one (request, kv head): the K rows, the V rows, or up to eight of
// the 4-byte vectors (scales, weights, gates of its query heads).  A cluster takes one stream's
// target positions in ascending order, a chunk at a time; a chunk is written only when every
// block of the cluster has it in its registers, and the next one is already being read.  In place this
// is right for any kept[i] >= i: the sources of chunk c lie at or behind its first target, so no
// earlier chunk's targets hold them, and a target that is a source of its own or an earlier
// chunk has been read before it is written.
struct Places {
  int to, from;            // blocks
  int to_slot, from_slot;  // -1 in `to`: nothing to move
};
__device__ __forceinline__ Places places(const MoveParams& p, int row, int i, int n, int L, const int32_t* table) {
  Places x{-1, 0, 0, 0};
  if (i >= n) return x;
  const int src = __ldg(p.kept + (size_t)row * p.max_keep + i);
  if (src == i) return x;
  if (src < i || src >= L) {
    record_bad(p.status);
    return x;
  }
  const int from = __ldg(table + (src >> p.log2_block)), to = __ldg(table + (i >> p.log2_block));
  if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks) {
    record_bad(p.status);
    return x;
  }
  return Places{to, from, i & (p.block_size - 1), src & (p.block_size - 1)};
}

__global__ void __launch_bounds__(kMoveThreads) cache_move_kernel(const MoveParams p, int cs) {
  const int rank = blockIdx.x % cs, row = blockIdx.x / cs, kind = blockIdx.y;
  const int r = row / p.hkv, h = row % p.hkv;
  const int tid = threadIdx.x;
  int L = __ldg(p.seq_lens + r), n = __ldg(p.kept_lens + r);
  if (L < 0 || L > p.capacity || n < 0 || n > p.max_keep || n > L) {  // the same for the whole cluster
    if (tid == 0) record_bad(p.status);
    return;
  }
  const int32_t* table = p.block_table + (size_t)r * p.max_blocks;

  if (kind < 2) {
    uint8_t* cache = kind ? p.v_cache : p.k_cache;
    const int log2_units = p.log2_units;  // 16-byte pieces of a row: 4 .. 64
    const int rows = (kMoveThreads * kPieces) >> log2_units;  // of a block's chunk
    const int unit = tid & ((1 << log2_units) - 1), lane_row = tid >> log2_units;
    const int step = kMoveThreads >> log2_units;
    auto at = [&](int blk, int slot) {
      return reinterpret_cast<uint4*>(cache + (size_t)blk * p.kv_bs + (size_t)h * p.kv_hs + (size_t)slot * p.kv_ss) + unit;
    };
    uint4 x[kPieces], y[kPieces];
    uint4 *to[kPieces], *to_next[kPieces];
    auto read = [&](int i0, uint4 (&d)[kPieces], uint4* (&t)[kPieces]) {
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const Places w = places(p, row, i0 + u * step + lane_row, n, L, table);
        t[u] = nullptr;
        if (w.to >= 0) {
          t[u] = at(w.to, w.to_slot);
          d[u] = *at(w.from, w.from_slot);
        }
      }
    };
    int i0 = rank * rows;
    read(i0, x, to);
    for (int c0 = 0; c0 < n; c0 += cs * rows) {  // c0: the cluster's chunk
      cg::cluster_group::barrier_arrive();
      i0 += cs * rows;
      read(i0, y, to_next);
      cg::cluster_group::barrier_wait();
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        if (to[u]) *to[u] = x[u];
        x[u] = y[u];
        to[u] = to_next[u];
      }
    }
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
      if (i < 2) base[v] = (i ? p.v_scale : p.k_scale) + (((size_t)h) << p.log2_block);
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
  float x[kVectors], y[kVectors];
  Places w{-1, 0, 0, 0}, w_next;
  auto read = [&](int i, float (&d)[kVectors], Places& t) {
    t = places(p, row, i, n, L, table);
    if (t.to < 0) return;
#pragma unroll
    for (int v = 0; v < kVectors; ++v)
      if (base[v]) d[v] = *cell(v, t.from, t.from_slot);
  };
  int i = rank * kMoveThreads + tid;
  read(i, x, w);
  for (int c0 = 0; c0 < n; c0 += cs * kMoveThreads) {
    cg::cluster_group::barrier_arrive();
    i += cs * kMoveThreads;
    read(i, y, w_next);
    cg::cluster_group::barrier_wait();
#pragma unroll
    for (int v = 0; v < kVectors; ++v) {
      if (w.to >= 0 && base[v]) *cell(v, w.to, w.to_slot) = x[v];
      x[v] = y[v];
    }
    w = w_next;
  }
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
  auto kern = held ? cache_select_kernel<true> : cache_select_kernel<false>;
  const size_t smem = held ? (size_t)slice * 4 : 0;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
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
  return launch_clusters(cache_move_kernel, dim3((unsigned)(rows * cs), kinds), kMoveThreads, cs, 0, s, p, cs);
}

}  // namespace gcs
