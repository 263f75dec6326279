// Rows of D contiguous bf16 elements (one token, one head) as the norm, rotation and cache
// kernels hold them: 16 elements a lane in registers, so D / 16 lanes share a row and a warp
// works on 512 / D rows at a time.
//
// A lane's 16 elements are two runs of 8 (one 16-byte access each), placed so that the lanes of a
// row read and write whole contiguous stretches with either access, and so that both elements of
// every pair of the rotation sit in one lane and no value has to be exchanged:
//   halves (i with i + rot / 2)   the first rot / 16 lanes: 8 s and rot / 2 + 8 s; the others
//                                 share the elements behind rot in the same way
//   neighbours (2 i with 2 i + 1) 8 s and D / 2 + 8 s
// (Runs next to each other, 16 s and 16 s + 8, make every access touch half of each 32-byte
// sector: the forward of 16384 tokens of 36 heads of 512 took 270 us that way and took 202 so.)
#pragma once

#include <cstdint>

#include "sm103_ptx.cuh"

namespace gcs {

constexpr unsigned kFullMask = 0xffffffffu;

template <int D>
struct RowLanes {
  static constexpr int kLanes = D / 16;       // lanes of a row
  static constexpr int kRows = 32 / kLanes;   // rows of a warp
};

// Element offsets of the lane's two runs, whether they are rotated, and the table's angles of
// the first and the second four of its pairs.
struct RowRuns {
  int a, b;
  bool turn_a, turn_b;
  int angle_a, angle_b;
};

template <int D>
__device__ __forceinline__ RowRuns row_runs(int sub, int rot, bool interleaved) {
  RowRuns r;
  if (interleaved) {
    r.a = 8 * sub;
    r.b = D / 2 + 8 * sub;
    r.turn_a = r.a < rot;
    r.turn_b = r.b < rot;
    r.angle_a = r.a / 2;
    r.angle_b = r.b / 2;
  } else {
    r.turn_a = r.turn_b = 16 * sub < rot;
    const int base = r.turn_a ? 0 : rot, len = r.turn_a ? rot : D - rot;
    const int i = sub - base / 16;
    r.a = base + 8 * i;
    r.b = base + len / 2 + 8 * i;
    r.angle_a = 8 * sub;
    r.angle_b = 8 * sub + 4;
  }
  return r;
}

struct RawRow {
  uint4 a, b;
};

// The rows of a warp's steps ahead, in shared memory: ROWS rows of every lane group and the table's
// row of the step's token.  Copies go in asynchronously, one step ahead of their use (two steps
// ahead measured the same or slower), so the bytes in flight do not depend on how many registers
// the arithmetic leaves for occupancy.
constexpr int kStages = 2;
template <int D, int ROWS>
struct WarpStage {
  uint4 raw[ROWS][2][32];  // a lane's two runs of each row: read by the lane that copied them
  float angles[D];         // read by the whole warp
};

__device__ __forceinline__ void copy_async16(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Starts the copy of the lane's part of a row (zeros where not valid: nothing is read).
template <int D, int ROWS>
__device__ __forceinline__ void fetch_row(WarpStage<D, ROWS>& st, int i, const uint16_t* row, const RowRuns& r,
                                          bool valid) {
  const int lane = threadIdx.x & 31;
  copy_async16(&st.raw[i][0][lane], row + r.a, valid);
  copy_async16(&st.raw[i][1][lane], row + r.b, valid);
}
// Starts the copy of a table row, by the whole warp.
template <int D, int ROWS>
__device__ __forceinline__ void fetch_angles(WarpStage<D, ROWS>& st, const float* table, long long pos, int rot) {
  for (int i = (threadIdx.x & 31) * 4; i < rot; i += 128) copy_async16(&st.angles[i], table + pos * rot + i, true);
}
template <int D, int ROWS>
__device__ __forceinline__ RawRow fetched_row(const WarpStage<D, ROWS>& st, int i) {
  const int lane = threadIdx.x & 31;
  return RawRow{st.raw[i][0][lane], st.raw[i][1][lane]};
}

__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack_row(const RawRow& w, float* x) {
  unpack8(w.a, x);
  unpack8(w.b, x + 8);
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
// The one rounding of a row to bf16 (nearest even).
__device__ __forceinline__ void store_row(uint16_t* row, const RowRuns& r, const float* x) {
  *reinterpret_cast<uint4*>(row + r.a) = pack8(x);
  *reinterpret_cast<uint4*>(row + r.b) = pack8(x + 8);
}

// Sum over the lanes of a row.
template <int L>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = L / 2; off; off >>= 1) x += __shfl_xor_sync(kFullMask, x, off);
  return x;
}

__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 u = __ldg(reinterpret_cast<const float4*>(p)), v = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
}

// The norm's weights of the lane's elements; ones without weights.
__device__ __forceinline__ void load_weights(const float* w, const RowRuns& r, float* x) {
  if (w) {
    load8(w + r.a, x);
    load8(w + r.b, x + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 1.f;
  }
}

// Cosines and sines of the lane's 8 pairs, from a row of the table (cosines, then sines).
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void read4(const float* p, float* x) {
  const float4 u = *reinterpret_cast<const float4*>(p);
  x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
}
__device__ __forceinline__ void read_angles(const float* row, int rot, const RowRuns& r, Angles& t) {
  const float* sines = row + (rot >> 1);
  if (r.turn_a) {
    read4(row + r.angle_a, t.c);
    read4(sines + r.angle_a, t.s);
  }
  if (r.turn_b) {
    read4(row + r.angle_b, t.c + 4);
    read4(sines + r.angle_b, t.s + 4);
  }
}

// (a, b) -> (a c - b s, b c + a s) for the lane's pairs; BACK: by the opposite angle.
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float x = fmaf(a, c, -b * s), y = fmaf(b, c, a * s);
  a = x, b = y;
}
template <bool BACK>
__device__ __forceinline__ void rotate_row(float* x, const RowRuns& r, const Angles& t, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < 4 ? r.turn_a : r.turn_b) rotate_pair(x[2 * i], x[2 * i + 1], t.c[i], BACK ? -t.s[i] : t.s[i]);
  } else if (r.turn_a) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rotate_pair(x[i], x[8 + i], t.c[i], BACK ? -t.s[i] : t.s[i]);
  }
}

// (mean(x^2) + eps)^(-1/2) over the row; the sum in fp32.
template <int D>
__device__ __forceinline__ float row_rstd(const float* x, float eps) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    s0 = fmaf(x[i], x[i], s0);
    s1 = fmaf(x[i + 1], x[i + 1], s1);
  }
  return rsqrtf(fmaf(row_sum<RowLanes<D>::kLanes>(s0 + s1), 1.f / D, eps));
}

}  // namespace gcs
