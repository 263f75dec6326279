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
#include "launch.h"
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
constexpr int kFew = 128;            // the same, of what a histogram leaves

// Weights as integers of the same order: NaN below everything, -0 equal to 0.  0 is left for what is
// no key at all.
constexpr uint32_t kNanKey = 1;
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);  // -0 + 0 = 0
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return f != f ? kNanKey : k;
}

// One cluster for a (request, kv head): its blocks take equal slices of the positions between the
// first and the last ones, as quads of four neighbouring positions (one vector load: a quad lies in
// one cache block).  The key of rank c from the top is found by histograms of 11, 11 and 10 bits, each
// added up in the cluster's first block, until few keys are left to be ranked; a last walk in the order
// of the positions writes those that stay.  11 bits of a positive float are its exponent and two bits
// more, so few of a warp's keys meet in a bin, and mostly one histogram is enough.
// HELD: the slice's keys stay in shared memory; otherwise (slices past kMaxSlice) each walk reads the
// weights again.  CLUSTER: more than one block.
template <bool HELD, bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads, 3) cache_select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint4 keys[];
  __shared__ __align__(16) uint32_t hist[kBins];  // read by four
  __shared__ uint32_t warp_a[kSelWarps], warp_b[kSelWarps];
  __shared__ uint2 few[kFew];  // (key, position)
  __shared__ uint32_t few_n;
  __shared__ uint3 found;         // digit, keys above it, keys with it; then the limit and its position
  __shared__ uint32_t of_block[16];  // tokens that stay (or equal the limit) in each block of the cluster
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = CLUSTER ? cluster.num_blocks() : 1, rank = CLUSTER ? cluster.block_rank() : 0;
  auto all_sync = [&]() {
    if (CLUSTER) cluster.sync();
    else __syncthreads();
  };
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
      mine = w ? order_key(__ldg(w)) : kNanKey;
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
    const int pos = q * 4;
    const float* at = weights(pos);
    uint4 k = make_uint4(kNanKey, kNanKey, kNanKey, kNanKey);
    if (at) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(at));
      k = make_uint4(order_key(w.x), order_key(w.y), order_key(w.z), order_key(w.w));
    }
    if (pos < lead || pos + 3 >= end) {  // tokens outside are below every key
      if (pos < lead) k.x = 0;
      if (pos + 1 < lead || pos + 1 >= end) k.y = 0;
      if (pos + 2 < lead || pos + 2 >= end) k.z = 0;
      if (pos + 3 < lead || pos + 3 >= end) k.w = 0;
    }
    return k;
  };
  auto quad = [&](int q) -> uint4 { return HELD ? keys[q - a] : load(q); };
  for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
  if (tid == 0) few_n = 0;
  __syncthreads();

  // The bits of the key of rank `need` found so far, and how many are wanted among the keys with
  // them.  Once those are few, they are ranked by (key, position) one against the other; the last
  // one that stays, limit, then tells for every token by itself whether it stays.
  uint32_t prefix = 0, mask = 0, left = need, same = 0;
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    const uint32_t digits = round == 2 ? 1023 : 2047;
    auto count = [&](const uint4& k) {
      const uint32_t e[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((e[j] & mask) == prefix) atomicAdd(&hist[(e[j] >> shift) & digits], 1u);
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
            count(k[u]);
          }
      }
    } else {
      for (int q = a + tid; q < b; q += kSelThreads) count(quad(q));
    }
    if (CLUSTER) {
      cluster.sync();
      if (rank != 0) {  // the first block adds up
        uint32_t* to = cluster.map_shared_rank(hist, 0);
        for (int i = tid; i < kBins; i += kSelThreads)
          if (hist[i]) atomicAdd(to + i, hist[i]);
      }
    }
    all_sync();
    if (rank == 0) {
      // thread's 4 bins from the top: 2047 - 4 tid .. 2044 - 4 tid
      const uint4 c = reinterpret_cast<const uint4*>(hist)[kBins / 4 - 1 - tid];
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
        uint3 f = make_uint3(0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (before < left && before + v[j] >= left) f = make_uint3(kBins - 1 - 4 * tid - j, before, v[j]);
          before += v[j];
        }
        for (int k = 0; k < cs; ++k) *(CLUSTER ? cluster.map_shared_rank(&found, k) : &found) = f;
      }
    }
    all_sync();
    prefix |= found.x << shift;
    mask |= digits << shift;
    left -= found.y;
    same = found.z;
    if (same <= kFew) break;
    for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
  }

  // limit: keys above it stay, and those equal to it up to position limit_at
  uint32_t limit = prefix;
  int limit_at = 0x7fffffff;
  const bool ranked = same <= kFew;  // otherwise: the many equal to it are counted below
  if (ranked) {
    // the list is in the first block; slots from any block, in any order
    uint2* list = CLUSTER ? cluster.map_shared_rank(few, 0) : few;
    uint32_t* used = CLUSTER ? cluster.map_shared_rank(&few_n, 0) : &few_n;
    for (int q = a + tid; q < b; q += kSelThreads) {
      const uint4 k = quad(q);
      const uint32_t e[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((e[j] & mask) == prefix) list[atomicAdd(used, 1u)] = make_uint2(e[j], q * 4 + j);
    }
    all_sync();
    if (rank == 0 && tid < same) {
      const uint2 mine = few[tid];
      uint32_t before = 0;
      for (int j = 0; j < (int)same; ++j) {
        const uint2 x = few[j];
        before += x.x > mine.x || (x.x == mine.x && x.y < mine.y);
      }
      if (before == left - 1)
        for (int k = 0; k < cs; ++k)
          *(CLUSTER ? cluster.map_shared_rank(&found, k) : &found) = make_uint3(mine.x, mine.y, 0);
    }
    all_sync();
    limit = found.x;
    limit_at = found.y;
  }

  // in the order of the positions, a warp's quads at a time: how many stay, then which.  Ranked: a token
  // stays iff its key is at least the limit, past limit_at one more.
  const int nql = b - a, chunk = (nql + kSelWarps - 1) / kSelWarps;
  const int wa = a + min(nql, warp * chunk), wb = a + min(nql, warp * chunk + chunk);
  auto above = [&](int q, const uint4& k) -> uint32_t {  // bits of the quad's tokens that stay
    const int pos = q * 4;
    uint32_t m = limit + (pos > limit_at);
    uint32_t v = (k.x >= m) | (k.y >= m) << 1 | (k.z >= m) << 2 | (k.w >= m) << 3;
    if (pos <= limit_at && pos + 3 > limit_at) {  // the quad that holds it
      const uint32_t strict = (k.x > m) | (k.y > m) << 1 | (k.z > m) << 2 | (k.w > m) << 3;
      const uint32_t low = (2u << (limit_at - pos)) - 1;
      v = (v & low) | (strict & ~low);
    }
    return v;
  };
  auto equal = [&](const uint4& k) -> uint32_t {
    return (k.x == limit) | (k.y == limit) << 1 | (k.z == limit) << 2 | (k.w == limit) << 3;
  };
  if (!ranked) {
    // more tokens than were ranked have the limit itself: the first `left` of them stay, and the last of
    // those is limit_at
    uint32_t eq = 0;
    for (int q = wa + lane; q < wb; q += 32) eq += __popc(equal(quad(q)));
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) warp_b[warp] = eq;
    __syncthreads();
    uint32_t eq0 = 0;
    if (CLUSTER) {
      if (tid < 32) {
        const uint32_t e = __reduce_add_sync(0xffffffffu, tid < kSelWarps ? warp_b[tid] : 0u);
        if (tid < cs) *cluster.map_shared_rank(&of_block[rank], tid) = e;
      }
      all_sync();
      for (int k = 0; k < rank; ++k) eq0 += of_block[k];
    }
    for (int w = 0; w < warp; ++w) eq0 += warp_b[w];
    if (eq0 < left && eq0 + eq >= left) {  // one warp's
      for (int q = wa; q < wb; q += 32) {
        const uint32_t t = q + lane < wb ? equal(quad(q + lane)) : 0u;
        uint32_t before = __popc(t), sum = before;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t s = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += s;
        }
        before = eq0 + sum - before;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (t >> j & 1) {
            if (before == left - 1)
              for (int k = 0; k < cs; ++k)
                *(CLUSTER ? cluster.map_shared_rank(&found, k) : &found) = make_uint3(limit, (q + lane) * 4 + j, 0);
            ++before;
          }
        }
        eq0 += __shfl_sync(0xffffffffu, sum, 31);
      }
    }
    all_sync();
    limit_at = found.y;
    if (CLUSTER) all_sync();  // of_block is written again
  }
  uint32_t stay = 0;
  for (int q = wa + lane; q < wb; q += 32) stay += __popc(above(q, quad(q)));
  stay = __reduce_add_sync(0xffffffffu, stay);
  if (lane == 0) warp_a[warp] = stay;
  __syncthreads();
  uint32_t at = lead;
  if (CLUSTER) {
    if (tid < 32) {
      const uint32_t s = __reduce_add_sync(0xffffffffu, tid < kSelWarps ? warp_a[tid] : 0u);
      if (tid < cs) *cluster.map_shared_rank(&of_block[rank], tid) = s;
    }
    all_sync();
    for (int k = 0; k < rank; ++k) at += of_block[k];
  }
  for (int w = 0; w < warp; ++w) at += warp_a[w];
  const uint32_t lower = (1u << lane) - 1;
  for (int q = wa; q < wb; q += 32) {
    const uint32_t v = q + lane < wb ? above(q + lane, quad(q + lane)) : 0u;
    const uint32_t v0 = __ballot_sync(0xffffffffu, v & 1), v1 = __ballot_sync(0xffffffffu, v & 2);
    const uint32_t v2 = __ballot_sync(0xffffffffu, v & 4), v3 = __ballot_sync(0xffffffffu, v & 8);
    int32_t* to = out + at + __popc(v0 & lower) + __popc(v1 & lower) + __popc(v2 & lower) + __popc(v3 & lower);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v >> j & 1) *to++ = (q + lane) * 4 + j;
    at += __popc(v0) + __popc(v1) + __popc(v2) + __popc(v3);
  }
}

// -------------------------------------------------------------------------------------- move
constexpr int kMoveThreads = 512;
constexpr int kPieces = 2;   // 16-byte pieces of K or V a thread moves in a chunk
constexpr int kVectors = 8;  // 4-byte vectors of a block, one element each of a thread's chunk
constexpr int kDepth = 3;    // chunks on their way
constexpr int kMoveSmem = kDepth * kMoveThreads * kPieces * 16;
static_assert(kPieces * 16 == kVectors * 4 && kPieces * kDepth <= 32, "the queue's places and the marks of what moves");

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
  // Requests that may not move, the same for all blocks of one.  The first tokens stay where they are: a request
  // that would move others to their places moves none at all (ascending positions begin with 0, 1, .. stay - 1
  // exactly where entry stay - 1 says so).  And in checked mode with gates the last token stays, from whose
  // gates the next append runs on.  (A vote of each warp: with one of the block, which keeps the threads
  // together, the kernel spills 500 bytes: 64 requests to 4096 tokens 144 us, so 135.)
  const int first = p.first_lens ? max(0, __ldg(p.first_lens + r)) : 0, stay = min(first, n);
  if (stay > 0 || (p.last_stays && n > 0)) {
    bool bad = false;
    for (int k = tid & 31; k < p.hkv; k += 32) {
      const int32_t* at = p.kept + ((size_t)r * p.hkv + k) * p.max_keep;
      bad = bad || (stay > 0 && __ldg(at + stay - 1) != stay - 1) || (p.last_stays && __ldg(at + n - 1) != L - 1);
    }
    if (__any_sync(0xffffffffu, bad)) {
      if (tid == 0) record_bad(p.status);
      return;
    }
  }
  const int32_t* table = p.block_table + (size_t)r * p.max_blocks;
  const int32_t* kept = p.kept + (size_t)row * p.max_keep;
  // Source of target i (from kept, read ahead): block and slot, -1 where there is nothing to move.
  auto source = [&](int i, int src) -> Target {
    if (i >= n || src == i) return Target{-1, 0};
    if (src < i || src >= L || i < first) {
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

template <bool HELD, bool CLUSTER>
cudaError_t launch_select(const SelectParams& p, long long rows, int cs, long long slice, cudaStream_t s) {
  auto kern = cache_select_kernel<HELD, CLUSTER>;
  const size_t smem = HELD ? (size_t)slice * 4 : 0;
  cudaError_t e = allow_smem<cache_select_kernel<HELD, CLUSTER>>(HELD ? kMaxSlice * 4 : 0);
  if (e != cudaSuccess) return e;
  if (!CLUSTER) {
    kern<<<(unsigned)rows, kSelThreads, smem, s>>>(p);
    return cudaGetLastError();
  }
  if (cs > 8 && (e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
    return e;
  return launch_clusters(kern, dim3((unsigned)(rows * cs)), kSelThreads, cs, smem, s, p);
}

}  // namespace

cudaError_t launch_cache_select(const SelectParams& p, cudaStream_t s) {
  const int sms = current_sms();
  if (!sms) return cudaErrorInvalidDevice;
  // Blocks: up to two and a half an SM, of a thousand keys or more each; a wider cluster waits longer at each
  // of its steps than its shorter slices save (64 rows of 32K keys: 4 blocks a row 20.2 us, 8 29.0, 1 26.3;
  // 192 of 16K: 1 21.0, 2 24.2; 16 of 4K: 4 15.3, 1 21.6). Slices past about 26K keys leave an SM one block at
  // a time, past kMaxSlice they are read again at each step: from 28K on they are halved however many the rows
  // (256 rows of 32K: 2 blocks 40.0, 1 44.0; of 100K: 4 92.9, 2 129.5; of 27K, below that border, 1 43.6 and 2
  // 43.5, 512 rows 82.5 and 68.2).
  const long long rows = (long long)p.num_reqs * p.hkv;
  int cs = 1;
  while (cs < 16 &&
         ((rows * cs * 4 <= 5 * sms && p.max_seq_len / cs > 1024) || p.max_seq_len / cs > 28 * 1024))
    cs *= 2;
  const long long slice = ((long long)(p.max_seq_len + 3) / 4 + cs) / cs * 4 + 8;  // keys of a block, at most
  const bool held = slice <= kMaxSlice;
  if (cs == 1)
    return held ? launch_select<true, false>(p, rows, cs, slice, s) : launch_select<false, false>(p, rows, cs, slice, s);
  return held ? launch_select<true, true>(p, rows, cs, slice, s) : launch_select<false, true>(p, rows, cs, slice, s);
}

cudaError_t launch_cache_move(const MoveParams& p, cudaStream_t s) {
  const int sms = current_sms();
  if (!sms) return cudaErrorInvalidDevice;
  const long long rows = (long long)p.num_reqs * p.hkv;
  const int vectors = (p.k_scale ? 2 : 0) + (p.w_cache ? 1 : 0) + (p.g_cache ? p.group : 0);
  const int kinds = 2 + (vectors + kVectors - 1) / kVectors;
  // blocks: about four an SM (three run at once), no more than the chunks of max_keep rows
  const int chunk = (kMoveThreads * kPieces) >> p.log2_units;
  int cs = 1;
  while (cs < 8 && rows * kinds * cs < 4 * sms && p.max_keep > cs * chunk) cs *= 2;
  const dim3 grid((unsigned)(rows * cs), kinds);
  cudaError_t e = cs > 1 ? allow_smem<cache_move_kernel<true>>(kMoveSmem) : allow_smem<cache_move_kernel<false>>(kMoveSmem);
  if (e != cudaSuccess) return e;
  if (cs > 1) return launch_clusters(cache_move_kernel<true>, grid, kMoveThreads, cs, kMoveSmem, s, p, cs);
  cache_move_kernel<false><<<grid, kMoveThreads, kMoveSmem, s>>>(p, cs);
  return cudaGetLastError();
}

}  // namespace gcs
