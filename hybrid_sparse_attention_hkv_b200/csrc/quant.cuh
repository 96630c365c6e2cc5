// Codes of the quantised history pages: eight columns of a row at a time.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace hsa {

constexpr float kQuantTiny = 7.888609052210118e-31f;  // 2^-100: smaller groups are stored as zeros

template <int FMT>
__device__ __forceinline__ constexpr float qmax_of() {
  return FMT == HKV_QUANT_E4M3 ? 448.f : FMT == HKV_QUANT_INT8 ? 127.f : 7.f;
}
template <int FMT>
__host__ __device__ constexpr int code_bits() {
  return FMT == HKV_QUANT_INT4 ? 4 : 8;
}
// Eight codes: two words of bytes, or one of nibbles.
template <int FMT>
struct Codes8 {
  uint32_t w[FMT == HKV_QUANT_INT4 ? 1 : 2];
};

template <int FMT>
__device__ __forceinline__ void store_codes(void* p, const Codes8<FMT>& c) {
  if constexpr (FMT == HKV_QUANT_INT4) *static_cast<uint32_t*>(p) = c.w[0];
  else *static_cast<uint2*>(p) = make_uint2(c.w[0], c.w[1]);
}

// Four e4m3 bytes as two pairs of halves (exact).
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t w, uint32_t& p0, uint32_t& p1) {
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;}"
      : "=r"(p0), "=r"(p1)
      : "r"(w));
}

// code * scale of eight columns, in fp32.  Integers come out of the mantissa of 2^23 + u
// (u the code plus 128 or 8, exact), which costs a byte permute or a mask and an add where an
// integer conversion would go through the quarter-rate pipe.
template <int FMT>
__device__ __forceinline__ void decode8(const Codes8<FMT>& c, float scale, float* f) {
  if constexpr (FMT == HKV_QUANT_E4M3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h[2];
      e4m3x4_to_half2(c.w[i], h[0], h[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
        f[4 * i + 2 * k] = x.x * scale;
        f[4 * i + 2 * k + 1] = x.y * scale;
      }
    }
  } else if constexpr (FMT == HKV_QUANT_INT8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = __byte_perm(c.w[i >> 2] ^ 0x80808080u, 0x4B000000u, 0x7540u + (i & 3));
      f[i] = (__uint_as_float(u) - 8388736.f) * scale;
    }
  } else {
    // nibble i left where it is: 2^23 + 16^i (n + 8), taken off and scaled by scale / 16^i
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = i < 5 ? 4 * i : 4 * i - 20;
      const uint32_t w = i < 5 ? c.w[0] : c.w[0] >> 20;
      const float x = __uint_as_float((w & (15u << at)) ^ (0x4B000000u | (8u << at)));
      f[i] = (x - (8388608.f + (float)(8u << at))) * (scale * (1.f / (float)(1u << at)));
    }
  }
}

// round(f * inv) of eight columns; all zero where the group is not finite.
template <int FMT>
__device__ __forceinline__ Codes8<FMT> encode8(const float* f, float inv, bool finite) {
  Codes8<FMT> c;
  if constexpr (FMT == HKV_QUANT_E4M3) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t w;
      asm("{.reg .b16 a, b;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
          "mov.b32 %0, {a, b};}"
          : "=r"(w)
          : "f"(__fmul_rn(f[4 * k], inv)), "f"(__fmul_rn(f[4 * k + 1], inv)), "f"(__fmul_rn(f[4 * k + 2], inv)),
            "f"(__fmul_rn(f[4 * k + 3], inv)));
      c.w[k] = finite ? w : 0u;
    }
  } else {
    // x * inv is at most qmax (1 + 2^-20) in magnitude, so the rounded integer is at most
    // qmax.  It is read from the mantissa of 1.5 * 2^23 + x, whose addition rounds to the
    // nearest integer, ties to even.
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(__fadd_rn(__fmul_rn(f[i], inv), 12582912.f));
    if constexpr (FMT == HKV_QUANT_INT8) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t a = __byte_perm(u[4 * k], u[4 * k + 1], 0x0040);
        const uint32_t b = __byte_perm(u[4 * k + 2], u[4 * k + 3], 0x0040);
        c.w[k] = finite ? __byte_perm(a, b, 0x5410) : 0u;
      }
    } else {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) w |= (u[i] & 15u) << (4 * i);
      c.w[0] = finite ? w : 0u;
    }
  }
  return c;
}

}  // namespace hsa
