// FP8 cache write: the new K and V rows of every sequence as E4M3 under one power-of-two scale
// for each (page, KV head).
//
// For a touched (page, head), e is the smallest exponent with amax <= 448 * 2^e over the new
// rows, raised to the page's own exponent when it already holds older rows; when e grows, the
// older rows' codes are multiplied by 2^(e_old - e) and rounded to E4M3 again (exact but for
// codes that become subnormal).  A power of two loses nothing in a floating format (all codes
// keep their four significant bits whatever the scale) and makes that growth exact.
//
// One CTA takes one (sequence, touched block, head, K or V): its 128 x 128 new elements are
// read once into registers (four 16-element units a thread), reduced to the maximum, encoded
// and stored as 16-byte units, so that the bytes moved are the input once and the codes once.
// Bound by memory for prompt chunks, by one round of dependent loads (length -> table ->
// scale) for decode steps: 65,520 tokens of 4 heads in float32 64 us = 5.2 TB/s, a decode step of 64
// sequences 4.3 us.  Three CTAs an SM (80 registers) keep that many tiles' loads in flight; two took 76 us.
#include <cuda_bf16.h>

#include "fp8_device.cuh"
#include "fp8_kernels.h"
#include "msa_device.cuh"

namespace msa {

constexpr int kApThreads = 256;
constexpr int kApUnits = kBlock * kDim / 16 / kApThreads;  // 16-element units per thread

template <typename X>
__device__ __forceinline__ void load_unit(const X* p, float (&v)[16]);

template <>
__device__ __forceinline__ void load_unit<float>(const float* p, float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 f = __ldcs(reinterpret_cast<const float4*>(p) + j);
    v[4 * j] = f.x;
    v[4 * j + 1] = f.y;
    v[4 * j + 2] = f.z;
    v[4 * j + 3] = f.w;
  }
}

template <>
__device__ __forceinline__ void load_unit<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p) + j);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[8 * j + 2 * i] = __uint_as_float(w[i] << 16);
      v[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// 16 values times f as E4M3 codes (round to nearest even, saturating)
__device__ __forceinline__ uint4 encode16(const float (&v)[16], float f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = f32x4_to_e4m3x4(v[4 * i] * f, v[4 * i + 1] * f, v[4 * i + 2] * f, v[4 * i + 3] * f);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename X>
__global__ void __launch_bounds__(kApThreads, 3) fp8_append_kernel(const Fp8AppendArgs a, int touched) {
  __shared__ uint32_t s_amax;
  const int tid = threadIdx.x;
  if (tid == 0) s_amax = 0u;
  grid_dependency_wait();
  grid_dependents_launch();
  // blockIdx.x = ((b * touched + i) * G + g) * 2 + (0: K, 1: V)
  uint32_t idx = blockIdx.x;
  const int kv = idx & 1;
  idx >>= 1;
  const int g = idx % a.groups;
  idx /= a.groups;
  const int i = idx % touched, b = idx / touched;
  const int L = a.seq_lens[b], T = a.q_len;
  if (L == 0) return;
  if (L < T || L > static_cast<int64_t>(a.max_blocks) * kBlock) {
    if (tid == 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
    return;
  }
  const int start = L - T, n = start / kBlock + i;
  if (n > (L - 1) / kBlock) return;
  const int page = a.block_table[static_cast<int64_t>(b) * a.max_blocks + n];
  if (page < 0 || page >= a.num_pages) {
    if (tid == 0) flag_error(a.err, MSA_DEVERR_BAD_PAGE);
    return;
  }
  const int lo = max(start - n * kBlock, 0), hi = min(L - n * kBlock, kBlock);  // the new rows
  const int64_t ph = static_cast<int64_t>(page) * a.groups + g;
  uint8_t* codes = a.data[kv] + ph * kFp8PageBytes;
  const int e_old = lo > 0 ? a.scale[kv][ph] : 0;
  if (lo > 0 && !e8m0_ok(e_old)) {
    if (tid == 0) flag_error(a.err, MSA_DEVERR_BAD_SCALE);
    return;
  }
  // token of the call at row 0 of the page (may be before the first: those rows are not read)
  const X* x = static_cast<const X*>(a.x[kv]);
  const int64_t tok0 = static_cast<int64_t>(b) * T + (static_cast<int64_t>(n) * kBlock - start);

  float v[kApUnits][16];
  float m = 0.f;
#pragma unroll
  for (int u = 0; u < kApUnits; ++u) {
    const int unit = u * kApThreads + tid, row = unit >> 3, c = unit & 7;
    if (row >= lo && row < hi) {
      load_unit(x + (tok0 + row) * a.stride[kv] + g * kDim + 16 * c, v[u]);
#pragma unroll
      for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(v[u][j]));  // (fmaxf passes NaN over)
    }
  }
  const uint32_t wm = __reduce_max_sync(0xffffffffu, __float_as_uint(m));  // non-negative floats order as integers
  __syncthreads();  // s_amax is zero
  if ((tid & 31) == 0 && wm != 0u) atomicMax(&s_amax, wm);
  __syncthreads();
  const int e = max(e8m0_for_amax(__uint_as_float(s_amax)), e_old);
  if (lo > 0 && e > e_old) {  // the older rows under the larger scale
    const float f = exp2_int(e_old - e);
    for (int unit = tid; unit < lo * 8; unit += kApThreads) {
      uint4* p = reinterpret_cast<uint4*>(codes) + unit;
      const uint4 c = *p;
      *p = make_uint4(e4m3x4_times(c.x, f), e4m3x4_times(c.y, f), e4m3x4_times(c.z, f), e4m3x4_times(c.w, f));
    }
  }
  const float f = exp2_int(kE8m0One - e);
#pragma unroll
  for (int u = 0; u < kApUnits; ++u) {
    const int unit = u * kApThreads + tid, row = unit >> 3;
    if (row >= lo && row < hi) reinterpret_cast<uint4*>(codes)[unit] = encode16(v[u], f);
  }
  if (tid == 0) a.scale[kv][ph] = static_cast<uint8_t>(e);
}

cudaError_t launch_fp8_append(const Fp8AppendArgs& a, cudaStream_t s) {
  const int touched = (a.q_len + kBlock - 2) / kBlock + 1;  // blocks that q_len rows can touch
  const int64_t ctas = static_cast<int64_t>(a.batch) * touched * a.groups * 2;  // < 2^21: batch * q_len <= 65535
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kApThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a.bf16 ? cudaLaunchKernelEx(&cfg, fp8_append_kernel<__nv_bfloat16>, a, touched)
                               : cudaLaunchKernelEx(&cfg, fp8_append_kernel<float>, a, touched);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace msa
