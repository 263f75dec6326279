// Device-content checks of the index arrays a call reads (a library diagnostic with no
// counterpart in the pages).  The host cannot read cu_seqlens, cu_q, seq_lens or the page
// table without synchronising, so one CTA reads them on the call's stream, before the call's
// kernels, and checks the preconditions the public header states for them.
//
// The CTA also writes the array of cumulative lengths (cu_seqlens or cu_q) that the call's
// kernels then read in place of the caller's: a copy when every check holds, and all zeros
// (an empty batch) when one fails, in which case it records kDevInvalidArg in the device
// status word.  In an empty batch every prefill tile and every paged request has no rows, so
// no kernel reads through an index taken from these arrays (the kernels that sweep every
// token, such as the backward's delta, stay within total_tokens, which the host checked).
#include "kernels.h"
#include "sm103_ptx.cuh"

namespace gcs {
namespace {

constexpr int kCheckThreads = 1024;

// Combines the threads' verdicts, records a failure and writes the copy (cu_out may be null).
__device__ __forceinline__ void finish_check(bool bad_here, int* bad_s, const int32_t* cu, int n1,
                                             int32_t* cu_out, int* status) {
  if (bad_here) atomicOr(bad_s, 1);
  __syncthreads();
  const bool bad = *bad_s != 0;
  if (bad && threadIdx.x == 0) atomicCAS(status, kDevOk, kDevInvalidArg);
  if (cu_out)
    for (int i = threadIdx.x; i < n1; i += blockDim.x) cu_out[i] = bad ? 0 : __ldg(cu + i);
}

// cu_seqlens: starts at 0, ends at total, and every length lies in 0 .. max_seqlen.
__global__ void __launch_bounds__(kCheckThreads) check_prefill_kernel(const int32_t* __restrict__ cu, int num_seqs,
                                                                      int total, int max_seqlen,
                                                                      int32_t* __restrict__ cu_out, int* status) {
  __shared__ int bad_s;
  if (threadIdx.x == 0) bad_s = 0;
  __syncthreads();
  bool bad = false;
  if (threadIdx.x == 0) bad = __ldg(cu) != 0 || __ldg(cu + num_seqs) != total;
  for (int s = threadIdx.x; s < num_seqs; s += blockDim.x) {
    const long long len = (long long)__ldg(cu + s + 1) - __ldg(cu + s);
    bad = bad || len < 0 || len > max_seqlen;
  }
  finish_check(bad, &bad_s, cu, num_seqs + 1, cu_out, status);
}

// Whether one of the V scales of the slots first .. end - 1 of an fp8 cache's block is not below 255 in magnitude.
__device__ __forceinline__ bool bad_scales(const PagedOperandCheck& fp8, int blk, int block_size, int first, int end) {
  bool bad = false;
  if (fp8.hkv > 0 && !fp8.per_tensor)
    for (int h = 0; h < fp8.hkv; ++h)
      for (int sl = first; sl < end; ++sl)
        bad = bad || !(fabsf(__ldg(fp8.v_scale + ((size_t)blk * fp8.hkv + h) * block_size + sl)) < 255.f);
  return bad;
}

// cu_q starts at 0 and ends at total_q; request r has 0 <= q_len <= max_q_len query rows and
// q_len <= seq_len <= max_seq_len cached tokens; the page-table entries of the pages the
// paged calls can read for it lie in [0, num_blocks).  Those pages run from the 128-key tile
// that holds the earliest key any of its query rows sees (key 0 without a window) to the
// page of its last cached token; a request with no query rows reads none.  One warp per
// request, one lane per page.
//
// With an fp8 cache (f16 operands, fp8.hkv > 0) it also checks the operand limits: every |q| at
// most 65504 (q, strided, is read in 16-byte units) and every V scale of the slots below
// seq_len in those pages below 255 in magnitude (per tensor: the one scale).
//
// With shared prefixes (prefix.num_groups > 0) the pages are those from the block of the first token behind
// the prefix on; check_groups_kernel looks at the prefix's.  cu_groups is not checked yet, so no index is taken
// from it.
__global__ void __launch_bounds__(kCheckThreads) check_paged_kernel(
    const int32_t* __restrict__ cu_q, const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ table,
    int num_reqs, int total_q, int max_q_len, int max_seq_len, int max_blocks, int num_blocks, int block_size,
    int window, PagedOperandCheck fp8, SharedPrefixes prefix, int32_t* __restrict__ cu_out, int* status) {
  __shared__ int bad_s;
  if (threadIdx.x == 0) bad_s = 0;
  __syncthreads();
  bool bad = false;
  if (threadIdx.x == 0) bad = __ldg(cu_q) != 0 || __ldg(cu_q + num_reqs) != total_q;
  if (fp8.hkv > 0) {
    // q: total_q x hq rows of d / 8 16-byte units
    const int units = fp8.d / 8;
    const long long n = (long long)total_q * fp8.hq * units;
    for (long long i = threadIdx.x; i < n; i += blockDim.x) {
      const long long row = i / units, t = row / fp8.hq, h = row % fp8.hq;
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(fp8.q + t * fp8.q_ts + h * fp8.q_hs) + i % units);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // bf16 magnitude bits above 65504 (0x477fe0), NaN included
        bad = bad || (w[k] & 0x7fffu) > 0x477fu || (w[k] >> 16 & 0x7fffu) > 0x477fu;
      }
    }
    if (fp8.per_tensor && threadIdx.x == 0) bad = bad || !(fabsf(__ldg(fp8.v_scale)) < 255.f);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
  for (int r = warp; r < num_reqs; r += nwarps) {
    const long long ql = (long long)__ldg(cu_q + r + 1) - __ldg(cu_q + r);
    const int L = __ldg(seq_lens + r);
    if (ql < 0 || ql > max_q_len || L < ql || L > max_seq_len) {
      bad = true;
      continue;
    }
    if (ql == 0) continue;
    const int first_key = window > 0 ? max(0, L - static_cast<int>(ql) - window + 1) : 0;
    int p0 = (first_key / 128) * 128 / block_size;  // block holding the first key of that tile
    int own = 0;  // first key that is read through this table
    if (prefix.num_groups > 0) {
      int lo = 0, hi = prefix.num_groups;  // the last group that starts at or before r
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(prefix.cu_groups + mid) <= r) lo = mid;
        else hi = mid;
      }
      const int P = __ldg(prefix.prefix_lens + lo);
      if (P >= L) continue;  // nothing behind it (or a prefix that the other kernel refuses)
      own = max(0, P);
      p0 = max(p0, own / block_size);
    }
    const int np = (L + block_size - 1) / block_size;  // <= max_blocks: L <= max_seq_len
    for (int pg = p0 + lane; pg < np; pg += 32) {
      const int blk = __ldg(table + (size_t)r * max_blocks + pg);
      bad = bad || blk < 0 || blk >= num_blocks;
      if (blk >= 0 && blk < num_blocks)
        bad = bad || bad_scales(fp8, blk, block_size, max(0, own - pg * block_size),
                                min(block_size, L - pg * block_size));
    }
  }
  finish_check(bad, &bad_s, cu_q, num_reqs + 1, cu_out, status);
}

// The groups of a call with shared prefixes: cu_groups starts at 0, ends at num_reqs and is sorted;
// a group has at most max_group_q query rows and a prefix of 0 .. max_prefix tokens, whose blocks the
// table of its first request holds (with V scales below 255 from the 128-key tile on that holds the earliest
// key any of the group's rows sees); every request of it has prefix <= seq_len <= prefix + max_suffix.
// cu_q is the checked copy (ending at 0: an earlier check failed).
__global__ void __launch_bounds__(kCheckThreads) check_groups_kernel(
    SharedPrefixes groups, const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ table, int num_reqs,
    int max_blocks, int num_blocks, int block_size, int total_q, int max_group_q, int max_prefix, int max_suffix,
    int window, PagedOperandCheck fp8, int32_t* cu_q, int32_t* __restrict__ groups_out, int* status) {
  const int32_t *cu_groups = groups.cu_groups, *prefix_lens = groups.prefix_lens;
  const int num_groups = groups.num_groups;
  __shared__ int bad_s;
  if (threadIdx.x == 0) bad_s = cu_q[num_reqs] != total_q;  // already recorded
  __syncthreads();
  bool bad = false;
  if (threadIdx.x == 0) bad = __ldg(cu_groups) != 0 || __ldg(cu_groups + num_groups) != num_reqs;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
  for (int g = warp; g < num_groups; g += nwarps) {
    const int a = __ldg(cu_groups + g), b = __ldg(cu_groups + g + 1), P = __ldg(prefix_lens + g);
    if (a < 0 || b < a || b > num_reqs || P < 0 || P > max_prefix) {
      bad = true;
      continue;
    }
    if (a == b) continue;
    bad = bad || (long long)cu_q[b] - cu_q[a] > max_group_q;
    bool fits = true;
    int seen = P;  // earliest key that a row sees
    for (int r = a + lane; r < b; r += 32) {
      const int L = __ldg(seq_lens + r), ql = cu_q[r + 1] - cu_q[r];
      fits = fits && P <= L && (long long)L - P <= max_suffix;
      if (ql > 0) seen = min(seen, window > 0 ? max(0, L - ql - window + 1) : 0);
    }
    if (!__all_sync(0xffffffffu, fits)) {
      bad = true;
      continue;
    }
    const int from = __reduce_min_sync(0xffffffffu, seen) / 128 * 128 / block_size;
    for (int pg = lane; pg < (P + block_size - 1) / block_size; pg += 32) {  // P <= seq_len <= the table
      const int blk = __ldg(table + (size_t)a * max_blocks + pg);
      bad = bad || blk < 0 || blk >= num_blocks;
      if (blk >= 0 && blk < num_blocks && pg >= from)
        bad = bad || bad_scales(fp8, blk, block_size, 0, min(block_size, P - pg * block_size));
    }
  }
  if (bad) atomicOr(&bad_s, 1);
  __syncthreads();
  const bool any = bad_s != 0;
  if (any && threadIdx.x == 0) atomicCAS(status, kDevOk, kDevInvalidArg);
  for (int i = threadIdx.x; i <= num_groups; i += blockDim.x) groups_out[i] = any ? 0 : __ldg(cu_groups + i);
  if (any)
    for (int i = threadIdx.x; i <= num_reqs; i += blockDim.x) cu_q[i] = 0;
}

}  // namespace

cudaError_t launch_check_groups(const SharedPrefixes& groups, const int32_t* seq_lens, const int32_t* table,
                                int num_reqs, int max_blocks, int num_blocks, int block_size, int total_q,
                                int max_group_q, int max_prefix, int max_suffix, int window,
                                const PagedOperandCheck& fp8, int32_t* cu_q, int32_t* groups_out, int* status,
                                cudaStream_t s) {
  check_groups_kernel<<<1, kCheckThreads, 0, s>>>(groups, seq_lens, table, num_reqs, max_blocks, num_blocks, block_size,
                                                  total_q, max_group_q, max_prefix, max_suffix, window, fp8, cu_q,
                                                  groups_out, status);
  return cudaGetLastError();
}

cudaError_t launch_check_prefill(const int32_t* cu, int num_seqs, int total, int max_seqlen, int32_t* cu_out,
                                 int* status, cudaStream_t s) {
  check_prefill_kernel<<<1, kCheckThreads, 0, s>>>(cu, num_seqs, total, max_seqlen, cu_out, status);
  return cudaGetLastError();
}

cudaError_t launch_check_paged(const int32_t* cu_q, const int32_t* seq_lens, const int32_t* table, int num_reqs,
                               int total_q, int max_q_len, int max_seq_len, int max_blocks, int num_blocks,
                               int block_size, int window, const PagedOperandCheck& fp8, const SharedPrefixes& prefix,
                               int32_t* cu_out, int* status, cudaStream_t s) {
  check_paged_kernel<<<1, kCheckThreads, 0, s>>>(cu_q, seq_lens, table, num_reqs, total_q, max_q_len, max_seq_len,
                                                 max_blocks, num_blocks, block_size, window, fp8, prefix, cu_out,
                                                 status);
  return cudaGetLastError();
}

}  // namespace gcs
