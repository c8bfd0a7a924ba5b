// Device helpers of the FP8 page cache: E8M0 page scales and E4M3 codes.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/msa.h"
#include "msa_device.cuh"

namespace msa {

constexpr int kE8m0One = 127;  // the byte of scale 1

__device__ __forceinline__ bool e8m0_ok(int byte) { return byte >= MSA_E8M0_MIN && byte <= MSA_E8M0_MAX; }

// 2^e for -126 <= e <= 127, exact
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// E8M0 byte of the smallest 2^e >= amax / 448 (e in -40..40): with amax = m 2^x, 1 <= m < 2,
// amax <= 448 * 2^e = 1.75 * 2^(e + 8) iff e >= x - 8 (m <= 1.75) or e >= x - 7.  amax >= 0;
// zero and subnormal values give the smallest, infinity the largest byte.
__device__ __forceinline__ int e8m0_for_amax(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int x = static_cast<int>(u >> 23) - 127;
  const int e = x - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e + kE8m0One, MSA_E8M0_MIN), MSA_E8M0_MAX);
}

// Four floats as E4M3 codes, the first in the low byte (round to nearest even, saturating at
// 448, NaN stays NaN).
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n"
      " .reg .b16 lo, hi;\n"
      " cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n"
      "}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}

// Four E4M3 codes -> two f16x2 (exact): r0 holds bytes 0, 1 and r1 bytes 2, 3.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& r0, uint32_t& r1) {
  asm("{\n"
      " .reg .b16 lo, hi;\n"
      " mov.b32 {lo, hi}, %2;\n"
      " cvt.rn.f16x2.e4m3x2 %0, lo;\n"
      " cvt.rn.f16x2.e4m3x2 %1, hi;\n"
      "}"
      : "=r"(r0), "=r"(r1)
      : "r"(w));
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four E4M3 codes times f, rounded to E4M3 again.
__device__ __forceinline__ uint32_t e4m3x4_times(uint32_t w, float f) {
  uint32_t h0, h1;
  e4m3x4_to_f16x4(w, h0, h1);
  const float2 a = f16x2_to_float2(h0), b = f16x2_to_float2(h1);
  return f32x4_to_e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

}  // namespace msa
