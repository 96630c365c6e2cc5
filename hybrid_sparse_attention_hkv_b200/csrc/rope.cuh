// Rotary positions, shared by the kernels that rotate rows: the rotary kernel itself, the
// write into quantised pages and the read back from them.
//
// A thread works on two 8-column chunks of one (row, head), `lo` and `hi`, chosen so that
// both members of each of its eight pairs are its own: thread j of a head's d / 16 has
//   interleaved  chunks j and j + d/16; pairs 4 lo .. 4 lo + 3, then 4 hi .. 4 hi + 3
//   half         while j < rot/16: chunks j and j + rot/16, pairs 8 j .. 8 j + 7;
//                above: two neighbouring chunks behind the rotated columns
// so that a row is rotated in registers, with no exchange between threads, and every
// access is a whole 16-byte (bf16, fp16), 32-byte (fp32) or 8 / 4-byte (codes) vector.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace hsa {

struct ChunkPair {
  int lo, hi;        // 8-column chunks of the head
  bool rot_lo, rot_hi;
};

__device__ __forceinline__ ChunkPair chunk_pair(const RopeArgs& r, int j, int J) {
  ChunkPair c;
  if (r.on && r.half_layout) {
    const int rh = r.pairs / 8;  // chunks in each half of the rotated columns
    const bool in = j < rh;
    c.lo = in ? j : 2 * rh + 2 * (j - rh);
    c.hi = in ? j + rh : c.lo + 1;
    c.rot_lo = c.rot_hi = in;
  } else {
    c.lo = j;
    c.hi = j + J;
    c.rot_lo = r.on && c.lo * 4 < r.pairs;
    c.rot_hi = r.on && c.hi * 4 < r.pairs;
  }
  return c;
}

// The pair that slot i (0..7) of a thread's two chunks belongs to (only for rotated ones).
__device__ __forceinline__ int slot_pair(const RopeArgs& r, const ChunkPair& c, int i) {
  return r.half_layout ? 8 * c.lo + i : 4 * (i < 4 ? c.lo : c.hi) + (i & 3);
}

// (mscale cos, mscale sin) of pair p at token t.  The angle in turns, pos * inv_freq / 2 pi,
// is formed and reduced to [-1/2, 1/2] in fp64: its error is about 2^-52 of the turns made
// (2^-21 of a turn after 2^31 of them), and the fp32 rounding behind the reduction costs at
// most 2^-26 of a turn.  sign = -1 turns backward (the gradient).
__device__ __forceinline__ float2 rope_cos_sin(const RopeArgs& r, long long t, int p) {
  const int axis = (p >= r.end0) + (p >= r.end1);
  const double pos = (double)r.pos[axis * r.pos_stride + t];
  double turns = pos * (r.inv_freq[p] * 0.15915494309189533577);  // 1 / (2 pi)
  turns -= rint(turns);
  float s, c;
  sincospif((float)(2.0 * turns), &s, &c);
  return make_float2(c * r.mscale, s * r.mscale * r.sign);
}

// Rotate a thread's two chunks in fp32; cs[i]: cos and sin of slot i.
__device__ __forceinline__ void rotate_chunks(const RopeArgs& r, const ChunkPair& c, const float2* cs, float* lo,
                                              float* hi) {
  if (r.half_layout) {
    if (c.rot_lo) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = lo[i], b = hi[i];
        lo[i] = a * cs[i].x - b * cs[i].y;
        hi[i] = b * cs[i].x + a * cs[i].y;
      }
    }
  } else {
    if (c.rot_lo) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = lo[2 * i], b = lo[2 * i + 1];
        lo[2 * i] = a * cs[i].x - b * cs[i].y;
        lo[2 * i + 1] = b * cs[i].x + a * cs[i].y;
      }
    }
    if (c.rot_hi) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = hi[2 * i], b = hi[2 * i + 1];
        hi[2 * i] = a * cs[4 + i].x - b * cs[4 + i].y;
        hi[2 * i + 1] = b * cs[4 + i].x + a * cs[4 + i].y;
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
