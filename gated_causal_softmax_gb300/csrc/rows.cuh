// Rows of D contiguous bf16 elements (one token, one head) as the norm, rotation and cache
// kernels hold them: 16 elements a lane in registers, so D / 16 lanes share a row and a warp
// works on 512 / D rows at a time.
//
// A lane's 16 elements are two runs of 8 (one 16-byte access each).  For the rotation in
// halves, which pairs element i with i + rot / 2, the runs of the first rot / 16 lanes start at
// 8 s and rot / 2 + 8 s, so both elements of every pair sit in one lane and no value has to be
// exchanged; in all other cases the two runs are neighbours.  Either way the lane's 8 pairs
// take the table's angles 8 s .. 8 s + 7.
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

// Element offsets of the lane's two runs; `rotated`: its elements are pairs of the rotation.
struct RowRuns {
  int a, b;
  bool rotated;
};

__device__ __forceinline__ RowRuns row_runs(int sub, int rot, bool interleaved) {
  RowRuns r;
  r.rotated = sub * 16 < rot;
  const bool halves = r.rotated && !interleaved;
  r.a = halves ? 8 * sub : 16 * sub;
  r.b = halves ? (rot >> 1) + 8 * sub : 16 * sub + 8;
  return r;
}

struct RawRow {
  uint4 a, b;
};

__device__ __forceinline__ RawRow load_row(const uint16_t* row, const RowRuns& r) {
  RawRow x;
  x.a = __ldg(reinterpret_cast<const uint4*>(row + r.a));
  x.b = __ldg(reinterpret_cast<const uint4*>(row + r.b));
  return x;
}

__device__ __forceinline__ RawRow zero_row() { return RawRow{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}; }

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

// Cosines and sines of the lane's 8 pairs from one row of the table (cosines, then sines).
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(const float* table, long long pos, int rot, int sub, const RowRuns& r,
                                            Angles& t) {
  if (r.rotated) {
    const float* row = table + pos * rot + 8 * sub;
    load8(row, t.c);
    load8(row + (rot >> 1), t.s);
  }
}

// (a, b) -> (a c - b s, b c + a s) for the lane's pairs; back: by the opposite angle.
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float x = fmaf(a, c, -b * s), y = fmaf(b, c, a * s);
  a = x, b = y;
}
template <bool BACK>
__device__ __forceinline__ void rotate_row(float* x, const RowRuns& r, const Angles& t, bool interleaved) {
  if (!r.rotated) return;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rotate_pair(x[2 * i], x[2 * i + 1], t.c[i], BACK ? -t.s[i] : t.s[i]);
  } else {
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
