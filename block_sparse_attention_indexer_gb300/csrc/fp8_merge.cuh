// The last step of units whose pages the split gave to several teams or CTAs: each left a partial
// state (O, M, l) of every row, added here.
//
// A thread takes four dims (a chunk) of a row.  A CTA has eight rows, or with many parts per unit
// (kSplit) one that its eight warps share; eight parts' states are loaded before any is used.  Bound by latency: one
// round of loads for each eight parts of a warp.
#pragma once

#include <cuda_bf16.h>

#include "fp8_device.cuh"
#include "fp8_kernels.h"

namespace msa {

constexpr int kFp8MergeThreads = 256;

// ln(2^M l); -inf for l = 0.  The powers of two meet first: M and log2 l alone may be far larger than their sum (V scales are in M).
__device__ __forceinline__ float fp8_lse(float M, float l) {
  const int e = min(static_cast<int>(__float_as_uint(l) >> 23) - 127, 127);
  return (M + static_cast<float>(e) + log2f(l * exp2_int(-e))) * 0.6931471805599453f;
}

// Parts per unit from which a CTA's warps share a row (one sequence of 4,096 tokens, 32 parts a unit:
// 12.9 us with one warp per row, 6.2 with eight; with two or three parts the extra warps only wait).
constexpr int kFp8MergeSplitParts = 12;

struct Fp8MergeShared {
  int list[kFp8MaxCtas * 3];  // the unit's partial places in order
  int n;
  float4 o[8][32];
  float m[8], l[8];
};

// Adds the states of places sh.list[0 .. n) for the thread's chunk of row `row`, float4 number `at` of a
// state of `rows` rows (O, then M, then l of the rows); with kSplit the sum is warp 0's.
template <bool kSplit>
__device__ __forceinline__ void fp8_merge_row(const float* partial, int rows, int row, int at, Fp8MergeShared& sh,
                                              float4& o, float& M, float& l) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = sh.n, first = kSplit ? warp : 0, step = kSplit ? 8 : 1;
  M = -INFINITY;
  l = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = first; i0 < n; i0 += 8 * step) {
    float ms[8], ls[8];
    float4 os[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = i0 + i * step;
      ms[i] = -INFINITY;
      ls[i] = 0.f;
      os[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < n) {
        const float* part = partial + static_cast<int64_t>(sh.list[k]) * rows * (kDim + 2);
        ms[i] = __ldcg(part + rows * kDim + row);
        ls[i] = __ldcg(part + rows * (kDim + 1) + row);
        os[i] = __ldcg(reinterpret_cast<const float4*>(part) + at);
      }
    }
    float mb = M;
#pragma unroll
    for (int i = 0; i < 8; ++i) mb = fmaxf(mb, ms[i]);
    // (no key so far: the sums hold zeros, or NaN)
    const float f = mb == -INFINITY ? 1.f : ex2(M - mb);
    l *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = mb == -INFINITY ? 1.f : ex2(ms[i] - mb);
      l += w * ls[i];
      o.x += w * os[i].x;
      o.y += w * os[i].y;
      o.z += w * os[i].z;
      o.w += w * os[i].w;
    }
    M = mb;
  }
  if (kSplit) {
    sh.o[warp][lane] = o;
    if (lane == 0) {
      sh.m[warp] = M;
      sh.l[warp] = l;
    }
    __syncthreads();
    if (warp == 0) {
      M = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) M = fmaxf(M, sh.m[i]);
      l = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = M == -INFINITY ? 1.f : ex2(sh.m[i] - M);
        l += w * sh.l[i];
        o.x += w * sh.o[i][lane].x;
        o.y += w * sh.o[i][lane].y;
        o.z += w * sh.o[i][lane].z;
        o.w += w * sh.o[i][lane].w;
      }
    }
  }
}

// A chunk of the row's output (head row hr) and, by chunk 0, its lse and statistics (index si).
__device__ __forceinline__ void fp8_write_row(const Fp8AttnArgs& a, int64_t hr, int64_t si, int chunk, const float4& o,
                                              float M, float l) {
  const bool any = l != 0.f;  // (NaN counts as any)
  const float inv = any ? 1.f / l : 0.f;
  const __nv_bfloat162 h0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), h1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  reinterpret_cast<uint2*>(a.out + hr * kDim)[chunk] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
  if (chunk == 0) {
    if (a.lse != nullptr) a.lse[hr] = fp8_lse(M, l);
    if (a.weight_out != nullptr) a.row_stat[si] = make_float2(any ? M : 0.f, inv);
  }
}

}  // namespace msa
