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

#include <cuda_runtime.h>

#include <cstdint>

#include "sm103_ptx.cuh"

namespace gcs {

// A kernel that needs what the one before it on the stream wrote, launched while that one still
// runs: it waits for its end and for its writes before it reads them (grid_wait).  Where the first
// kernel says so (grid_release, by all blocks), or when its blocks have ended, the second may start.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, dim3 block, cudaStream_t s, const Args&... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = block;
  c.stream = s;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, Params(args)...);
}

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

// The rows of a warp's next step, in shared memory: ROWS rows of every lane group and the table's row
// of the step's token (or the rows of its tokens, at most one for each lane group).  Copies go in
// asynchronously a step ahead of their use (two and three steps ahead measured the same, and slower at
// d = 512), so the bytes in flight do not depend on how many registers the arithmetic leaves for
// occupancy.
template <int D, int ROWS, int TOKENS = 1>
struct WarpStage {
  uint4 raw[ROWS][2][32];  // a lane's two runs of each row: read by the lane that copied them
  float angles[TOKENS][D]; // read by the whole warp
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
template <typename Stage>
__device__ __forceinline__ void fetch_row(Stage& st, int i, const uint16_t* row, const RowRuns& r, bool valid) {
  const int lane = threadIdx.x & 31;
  copy_async16(&st.raw[i][0][lane], row + r.a, valid);
  copy_async16(&st.raw[i][1][lane], row + r.b, valid);
}
// Starts the copy of a table row, by the whole warp.
template <int D>
__device__ __forceinline__ void fetch_angles(float (&angles)[D], const float* table, int pos, int rot) {
  const float* row = table + (long long)pos * rot;
#pragma unroll
  for (int i = 0; i < D; i += 128) {
    const int j = i + (threadIdx.x & 31) * 4;
    if (j < rot) copy_async<16>(&angles[j], row + j);
  }
}
template <typename Stage>
__device__ __forceinline__ RawRow fetched_row(const Stage& st, int i) {
  const int lane = threadIdx.x & 31;
  return RawRow{st.raw[i][0][lane], st.raw[i][1][lane]};
}

// Two fp32 operations in one instruction, each rounded as usual.
__device__ __forceinline__ float2 as_f2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ unsigned long long as_u64(const float2& a) {
  unsigned long long v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a.x), "f"(a.y));
  return v;
}
__device__ __forceinline__ float2 mul2(const float2& a, const float2& b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(d);
}
__device__ __forceinline__ float2 fma2(const float2& a, const float2& b, const float2& c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
  return as_f2(d);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 neg2(const float2& a) { return make_float2(-a.x, -a.y); }

// A lane's 16 elements in fp32: e[0..3] are run a, e[4..7] run b.
struct Row {
  float2 e[8];
};
__device__ __forceinline__ Row zero_row() {
  Row x;
#pragma unroll
  for (int i = 0; i < 8; ++i) x.e[i] = both(0.f);
  return x;
}
__device__ __forceinline__ Row unpack_row(const RawRow& w) {
  const uint32_t u[8] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
  Row x;
#pragma unroll
  for (int i = 0; i < 8; ++i) x.e[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  return x;
}
// The one rounding of a row to bf16 (nearest even).
__device__ __forceinline__ uint4 pack_run(const float2* e) {
  return make_uint4(pack_bf16x2(e[0].x, e[0].y), pack_bf16x2(e[1].x, e[1].y), pack_bf16x2(e[2].x, e[2].y),
                    pack_bf16x2(e[3].x, e[3].y));
}
__device__ __forceinline__ void store_row(uint16_t* row, const RowRuns& r, const Row& x) {
  *reinterpret_cast<uint4*>(row + r.a) = pack_run(x.e);
  *reinterpret_cast<uint4*>(row + r.b) = pack_run(x.e + 4);
}

// Sums over the lanes of a row, of N values side by side.
template <int L, int N>
__device__ __forceinline__ void row_sums(float (&x)[N]) {
#pragma unroll
  for (int off = L / 2; off; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(kFullMask, x[i], off);
}

__device__ __forceinline__ void read4(const float* p, float2* x) {
  const float4 u = *reinterpret_cast<const float4*>(p);
  x[0] = make_float2(u.x, u.y);
  x[1] = make_float2(u.z, u.w);
}

// The norm's weights of the lane's elements; ones without weights.
__device__ __forceinline__ Row load_weights(const float* w, const RowRuns& r) {
  Row x;
  if (w) {
    read4(w + r.a, x.e);
    read4(w + r.a + 4, x.e + 2);
    read4(w + r.b, x.e + 4);
    read4(w + r.b + 4, x.e + 6);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x.e[i] = both(1.f);
  }
  return x;
}

// Cosines c and sines s of the lane's 8 pairs, from a row of the table (cosines, then sines), and
// n = -s; BACK: of the opposite angle.
struct Angles {
  float2 c[4], s[4], n[4];
};
template <bool BACK>
__device__ __forceinline__ Angles read_angles(const float* row, int rot, const RowRuns& r) {
  const float* sines = row + (rot >> 1);
  Angles t;
  if (r.turn_a) {
    read4(row + r.angle_a, t.c);
    read4(sines + r.angle_a, BACK ? t.n : t.s);
  }
  if (r.turn_b) {
    read4(row + r.angle_b, t.c + 2);
    read4(sines + r.angle_b, (BACK ? t.n : t.s) + 2);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BACK)
      t.s[i] = neg2(t.n[i]);
    else
      t.n[i] = neg2(t.s[i]);
  }
  return t;
}

// Pairs (a, b) -> (a c - b s, b c + a s), of U rows side by side.
template <int U>
__device__ __forceinline__ void rotate_rows(Row (&x)[U], const RowRuns& r, const Angles& t, bool interleaved) {
  if (interleaved) {
    auto turn = [](float2& p, float c, float s, float n) {
      p = make_float2(fmaf(p.y, n, p.x * c), fmaf(p.x, s, p.y * c));
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < 2 ? r.turn_a : r.turn_b) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          turn(x[u].e[2 * i], t.c[i].x, t.s[i].x, t.n[i].x);
          turn(x[u].e[2 * i + 1], t.c[i].y, t.s[i].y, t.n[i].y);
        }
      }
    }
  } else if (r.turn_a) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float2 a = x[u].e[i], b = x[u].e[4 + i];
        x[u].e[i] = fma2(b, t.n[i], mul2(a, t.c[i]));
        x[u].e[4 + i] = fma2(a, t.s[i], mul2(b, t.c[i]));
      }
  }
}

// x = R (x w) r with r = (mean(x^2) + eps)^(-1/2) over the row, the sum in fp32; without the norm
// w = 1 and r = 1.  The products and the rotation do not wait for the sum over the lanes.
template <int D, int U>
__device__ __forceinline__ void norm_rotate_rows(Row (&x)[U], const Row& w, const RowRuns& runs, const Angles& t,
                                                 bool norm, float eps, bool interleaved) {
  float r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float2 s = mul2(x[u].e[0], x[u].e[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) s = fma2(x[u].e[i], x[u].e[i], s);
    r[u] = s.x + s.y;
  }
  row_sums<RowLanes<D>::kLanes>(r);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    r[u] = norm ? rsqrtf(fmaf(r[u], 1.f / D, eps)) : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[u].e[i] = mul2(x[u].e[i], w.e[i]);
  }
  rotate_rows(x, runs, t, interleaved);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[u].e[i] = mul2(x[u].e[i], both(r[u]));
}

}  // namespace gcs
