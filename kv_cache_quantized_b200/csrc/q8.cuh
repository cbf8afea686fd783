// The 8-bit cache: one code a coordinate, one fp32 scale for each block of 16 tokens and KV head; a coordinate's
// value is code * scale.  Codes are signed integers in [-127, 127], or e4m3 floats (1 sign, 4 exponent, 3 mantissa
// bits, largest 448).
//   pools  codes [num_blocks, Hkv, bt, d] uint8, scales [num_blocks, Hkv, bt / 16] fp32
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "axr_common.cuh"

namespace axr {

constexpr int kQ8Block = 16;  // tokens that share a scale (a pool block holds a whole number of them)

// The scale that the largest magnitude of a block needs: amax / 127, or the smallest power of two that holds amax
// within 448.  A power of two costs e4m3 codes no precision, and makes a later growth of the scale exact (up to
// subnormal codes).  Blocks below 2^-100 are held as zeros, so that the reciprocal of a scale is finite.
template <bool I8>
__device__ __forceinline__ float q8_need(float amax) {
  if (!(amax >= 7.888609052210118e-31f)) return 0.f;  // 2^-100
  if constexpr (I8) return __fdiv_rn(amax, 127.f);
  const uint32_t u = __float_as_uint(amax);            // normal: amax = 1.f x 2^(e - 127)
  const int e = static_cast<int>(u >> 23);
  const int up = (u & 0x7fffffu) > 0x600000u ? 1 : 0;  // 1.f > 1.75: 448 = 1.75 x 2^8
  return __uint_as_float(static_cast<uint32_t>(e - 8 + up) << 23);
}

// 4 values (already divided by the scale) to 4 codes, least significant byte first: round to nearest even, clamped;
// NaN becomes 0.
template <bool I8>
__device__ __forceinline__ uint32_t q8_pack4(const float* y) {
  if constexpr (I8) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = max(-127, min(127, __float2int_rn(y[i])));  // the conversion maps NaN to 0 and saturates
      w |= (static_cast<uint32_t>(c) & 0xffu) << (8 * i);
    }
    return w;
  } else {
    uint16_t lo, hi;
    const float a = y[0] == y[0] ? y[0] : 0.f, b = y[1] == y[1] ? y[1] : 0.f;
    const float c = y[2] == y[2] ? y[2] : 0.f, d = y[3] == y[3] ? y[3] : 0.f;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
}

// The same for finite values within the largest code's reach (up to its rounding): no clamps, no NaN.
template <bool I8>
__device__ __forceinline__ uint32_t q8_pack4_finite(const float* y) {
  if constexpr (I8) {
    const uint32_t a = __byte_perm(__float2int_rn(y[0]), __float2int_rn(y[1]), 0x0040);
    const uint32_t b = __byte_perm(__float2int_rn(y[2]), __float2int_rn(y[3]), 0x0040);
    return __byte_perm(a, b, 0x5410);
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1]), "f"(y[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3]), "f"(y[2]));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
}

// 4 codes to 4 values in fp16 (exact: integers up to 127, or 4 significant bits within fp16's range), as two half2.
template <bool I8>
__device__ __forceinline__ void q8_halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (I8) {
    // byte + 128 in the low bits of 1024's mantissa, then minus 1152
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

template <bool I8>
__device__ __forceinline__ void q8_values4(uint32_t w, float* v) {
  uint32_t lo, hi;
  q8_halves<I8>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

}  // namespace axr
