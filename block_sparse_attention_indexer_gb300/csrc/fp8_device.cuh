// Device helpers of the FP8 page cache: E8M0 page scales and E4M3 codes.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/msa.h"
#include "fp8_kernels.h"
#include "msa_device.cuh"

namespace msa {

constexpr int kE8m0One = 127;  // the byte of scale 1

__device__ __forceinline__ bool e8m0_ok(int byte) { return byte >= MSA_E8M0_MIN && byte <= MSA_E8M0_MAX; }

// A factor of the scores that float32 does not hold as its largest value: a score of 0 stays 0.  (With any other
// score the logit itself is beyond float32, or further from all others than the softmax can tell.)
__device__ __forceinline__ float finite_factor(float f) { return f == INFINITY ? 3.402823466e38f : f; }

// The reference M of the attention kernels, in P_j = 2^(e_j - M) with e_j = z_j log2(e) + b (2^b the V scale of
// the key's page).  fp16 holds P to 11 bits from 2^-14 up and to multiples of 2^-24 below, while the sum l counts
// the unrounded P, so M is kept where P uses that range, and follows the pages' V scales down as well as up:
//   * a P that would pass 2^kFp8RefMax moves M up;
//   * the row's sum so far at this page's scale, sum e^z 2^(b - M), may not be small while the page's keys are
//     rounded: M moves down first.  With that sum at least 2^s, a P below fp16's normal range is off by at most
//     2^-25 / 2^s of the row's sum, whatever the scales of its other pages are (s: fp8_stream.cu, fp8_tile.cu).
// M is an integer: moves are exact.  With Z the largest z log2(e) so far of the row's keys in the part of it that
// has its own state, Z - 55 <= M <= Z + 34 for b in -40..40 (no P passes 2^15, and M moves to a place below the
// largest e), hence
//   |O| <= 2^22 keys * 448 * 2^(Z + 40 - M) < 2^126 and l <= 2^77 do not overflow, and
//   a state whose weight 2^(M_i - M_k) underflows beside another one has no key above 2^-37 of that one's largest.
constexpr float kFp8RefMax = 15.f;

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

// 2^x (approximate to 2 ulp; -inf gives 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The top bits of the bytes of w that are NaN codes (0x7f, 0xff; no byte's sum carries), and such bits as whole bytes.
__device__ __forceinline__ uint32_t e4m3_nans(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t whole_bytes(uint32_t m) { return m | (m - (m >> 7)); }

// One 2-D tiled tensor copy global -> shared completing on `bar`, with an L2 policy (x, the byte
// offset within a key row, is always 0 here: 16-byte aligned).
__device__ __forceinline__ void tma_page(void* dst, const void* map, int y, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
      "{%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// Byte offset of 16-byte chunk c of key row r in a page as the tensor copy lands it (128-byte
// rows, 128-byte swizzle).
__device__ __forceinline__ int page_chunk(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// Whether sequence length L is one that the call can attend with (0 is a padding row).
__device__ __forceinline__ bool length_ok(const Fp8AttnArgs& a, int L) {
  return L > 0 && L >= a.q_len && L <= static_cast<int64_t>(a.max_blocks) * kBlock;
}

// Four E4M3 codes times f, rounded to E4M3 again.
__device__ __forceinline__ uint32_t e4m3x4_times(uint32_t w, float f) {
  uint32_t h0, h1;
  e4m3x4_to_f16x4(w, h0, h1);
  const float2 a = f16x2_to_float2(h0), b = f16x2_to_float2(h1);
  return f32x4_to_e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

}  // namespace msa
