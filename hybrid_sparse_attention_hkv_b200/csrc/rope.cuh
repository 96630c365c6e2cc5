// Rotary positions, shared by the kernels that rotate rows: the rotary kernel itself, the
// write into quantised pages and the read back from them.
//
// A thread works on two 8-column chunks of one (row, head), `lo` and `hi`, chosen so that
// both members of each of its eight pairs are its own: thread j of a head's J = d / 16 has
//   interleaved  chunks j and j + J; pairs 4 lo .. 4 lo + 3, then 4 hi .. 4 hi + 3
//   half         while j < rot/16: chunks j and j + rot/16, pairs 8 j .. 8 j + 7;
//                above: two neighbouring chunks behind the rotated columns
// so that a row is rotated in registers, with no exchange between threads, and every
// access is a whole 16-byte (bf16, fp16), 32-byte (fp32) or 8 / 4-byte (codes) vector.
// The cos and sin of a row's pairs are computed once a CTA, into shared memory, and used
// for all of the row's heads there.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace hsa {

constexpr int kRopeNone = 0;
constexpr int kRopeInterleaved = 1;
constexpr int kRopeHalf = 2;

struct ChunkPair {
  int lo, hi;           // 8-column chunks of the head
  bool rot_lo, rot_hi;  // whether they are rotated
};

template <int J, int ROPE>
__device__ __forceinline__ ChunkPair chunk_pair(const RopeArgs& r, int j) {
  ChunkPair c;
  if constexpr (ROPE == kRopeHalf) {
    const int rh = r.pairs / 8;  // chunks in each half of the rotated columns
    const bool in = j < rh;
    c.lo = in ? j : 2 * rh + 2 * (j - rh);
    c.hi = in ? j + rh : c.lo + 1;
    c.rot_lo = c.rot_hi = in;
  } else {
    c.lo = j;
    c.hi = j + J;
    c.rot_lo = ROPE == kRopeInterleaved && c.lo * 4 < r.pairs;
    c.rot_hi = ROPE == kRopeInterleaved && c.hi * 4 < r.pairs;
  }
  return c;
}

// (mscale cos, mscale sin) of a pair at a position.  The angle in quarter turns,
// pos * inv_freq * 2 / pi, is formed and reduced to [-1/2, 1/2] in fp64 (adding 1.5 * 2^52
// rounds it to an integer, whose low bits name the quarter): its error is about 2^-52 of the
// turns made (2^-21 of a turn after 2^31 of them).  The rest, at most pi / 4, goes through the
// Taylor series of sin (to the 9th power, error below 2^-29) and cos (10th, 2^-33) in fp32:
// two roundings of the angle and those of the series leave an error below 2^-22.  sign = -1
// turns backward (the gradient).
__device__ __forceinline__ float2 rope_cos_sin(const RopeArgs& r, int pos, double quarters_per_step) {
  const double quarters = (double)pos * quarters_per_step, shifted = quarters + 6755399441055744.0;
  const int q = __double2loint(shifted);
  // (clamped: beyond 2^51 quarter turns nothing is left of the angle, and the series is not to leave its range)
  const float rest = fminf(fmaxf((float)(quarters - (shifted - 6755399441055744.0)), -0.5f), 0.5f);
  const float a = rest * 1.57079632679489662f, x = a * a;
  float s = fmaf(x, 1.f / 362880, -1.f / 5040), c = fmaf(x, -1.f / 3628800, 1.f / 40320);
  s = fmaf(x, s, 1.f / 120);
  c = fmaf(x, c, -1.f / 720);
  s = fmaf(x, s, -1.f / 6);
  c = fmaf(x, c, 1.f / 24);
  s = fmaf(a * x, s, a);
  c = fmaf(x, c, -0.5f);
  c = fmaf(x, c, 1.f);
  const float cc = q & 1 ? s : c, ss = q & 1 ? c : s;
  return make_float2((q + 1) & 2 ? -cc * r.mscale : cc * r.mscale, (q & 2 ? -ss : ss) * (r.mscale * r.sign));
}

// The cos and sin of `rows` tokens from t0 on, in the order the threads read them: for each
// row four planes, plane k holding slots 2k and 2k + 1 of each of the row's J threads, so that
// the J threads' 16-byte reads of a plane are contiguous.  Slots of chunks that are not
// rotated are left out.
template <int J, int ROPE>
__device__ __forceinline__ void rope_table(const RopeArgs& r, long long t0, int rows, float4* table, int tid,
                                           int threads) {
  // a thread keeps its slot (and so its pair) and walks over rows; threads >= 8 J
  const int rows_at_once = threads / (8 * J), slot = tid % (8 * J);
  const int plane = slot / (2 * J), j = slot % (2 * J) / 2, i = 2 * plane + (slot & 1);
  const ChunkPair c = chunk_pair<J, ROPE>(r, j);
  if (tid >= rows_at_once * 8 * J || !(i < 4 ? c.rot_lo : c.rot_hi)) return;
  const int p = ROPE == kRopeHalf ? 8 * c.lo + i : 4 * (i < 4 ? c.lo : c.hi) + (i & 3);
  const int32_t* pos = r.pos + ((p >= r.end0) + (p >= r.end1)) * r.pos_stride + t0;
  const double quarters_per_step = __ldg(r.inv_freq + p) * 0.63661977236758134308;  // 2 / pi
  for (int row = tid / (8 * J); row < rows; row += rows_at_once)
    reinterpret_cast<float2*>(table)[row * 8 * J + slot] = rope_cos_sin(r, __ldg(pos + row), quarters_per_step);
}

// Rotate a thread's two chunks in fp32; row: the table's row of its token.
template <int J, int ROPE>
__device__ __forceinline__ void rotate_chunks(const ChunkPair& c, const float4* row, int j, float* lo, float* hi) {
  if constexpr (ROPE == kRopeHalf) {
    if (c.rot_lo) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 v = row[k * J + j];
        const float a0 = lo[2 * k], b0 = hi[2 * k], a1 = lo[2 * k + 1], b1 = hi[2 * k + 1];
        lo[2 * k] = a0 * v.x - b0 * v.y;
        hi[2 * k] = b0 * v.x + a0 * v.y;
        lo[2 * k + 1] = a1 * v.z - b1 * v.w;
        hi[2 * k + 1] = b1 * v.z + a1 * v.w;
      }
    }
  } else if constexpr (ROPE == kRopeInterleaved) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float* x = half ? hi : lo;
      if (half ? c.rot_hi : c.rot_lo) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 v = row[(2 * half + k) * J + j];
          const float a0 = x[4 * k], b0 = x[4 * k + 1], a1 = x[4 * k + 2], b1 = x[4 * k + 3];
          x[4 * k] = a0 * v.x - b0 * v.y;
          x[4 * k + 1] = b0 * v.x + a0 * v.y;
          x[4 * k + 2] = a1 * v.z - b1 * v.w;
          x[4 * k + 3] = b1 * v.z + a1 * v.w;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ 8 columns of a row
template <typename T>
struct Chunk;  // raw 8 elements of type T, as loaded

template <>
struct Chunk<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p) { v = *static_cast<const uint4*>(p); }
  __device__ __forceinline__ void load_split(const void* p, int) { load(p); }
  __device__ __forceinline__ void store(void* p) const { *static_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
  }
  __device__ __forceinline__ void set(const float* f) {
    v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};

template <>
struct Chunk<__half> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p) { v = *static_cast<const uint4*>(p); }
  __device__ __forceinline__ void load_split(const void* p, int) { load(p); }
  __device__ __forceinline__ void store(void* p) const { *static_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
  __device__ __forceinline__ void set(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 x = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = static_cast<const float4*>(p)[0];
    b = static_cast<const float4*>(p)[1];
  }
  // its two 16-byte vectors `step` bytes apart
  __device__ __forceinline__ void load_split(const void* p, int step) {
    a = *static_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(static_cast<const char*>(p) + step);
  }
  __device__ __forceinline__ void store(void* p) const {
    static_cast<float4*>(p)[0] = a;
    static_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void set(const float* f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

}  // namespace hsa
