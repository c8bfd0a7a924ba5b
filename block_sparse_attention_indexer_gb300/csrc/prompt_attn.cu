// Causal attention of packed bf16 prompts: one warp per query row (token, head), the keys one
// after another with a running maximum and sum.  A lane holds four dims.
#include <cuda_bf16.h>

#include "fp8_device.cuh"
#include "fp8_kernels.h"
#include "msa_device.cuh"
#include "prompt.h"

namespace msa {

__device__ __forceinline__ float4 bf16x4(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}

__global__ void __launch_bounds__(256) prompt_attn_kernel(const PromptArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  bool bad = false;
  for (int b = threadIdx.x; b < a.batch; b += 256)
    bad |= a.cu_q[b] < 0 || a.cu_k[b] < 0 || a.cu_q[b + 1] < a.cu_q[b] || a.cu_k[b + 1] < a.cu_k[b] ||
           a.cu_q[b + 1] > a.q_tokens || a.cu_k[b + 1] > a.k_tokens;
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
    return;
  }
  const int lane = threadIdx.x & 31, H = a.groups * a.heads_per_group;
  const int q0 = a.cu_q[0];
  const int64_t rows = static_cast<int64_t>(a.cu_q[a.batch] - q0) * H;
  for (int64_t r = blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += static_cast<int64_t>(gridDim.x) * 8) {
    const int token = q0 + static_cast<int>(r / H), h = static_cast<int>(r % H), g = h / a.heads_per_group;
    int lo = 0, n = a.batch;  // the last sequence that starts at or before the token
    while (n > 1) {
      const int half = n / 2;
      if (a.cu_q[lo + half] <= token) {
        lo += half;
        n -= half;
      } else {
        n = half;
      }
    }
    const int Lq = a.cu_q[lo + 1] - a.cu_q[lo], Lk = a.cu_k[lo + 1] - a.cu_k[lo];
    const int seen = Lk - Lq + (token - a.cu_q[lo]) + 1;
    float4 q = bf16x4(a.q + token * a.q_stride + h * kDim + 4 * lane);
    const int64_t key0 = a.cu_k[lo];
    float M = -INFINITY, was = M, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < seen; ++j) {
      const float4 k = bf16x4(a.k + (key0 + j) * a.k_stride + g * kDim + 4 * lane);
      const float4 v = bf16x4(a.v + (key0 + j) * a.v_stride + g * kDim + 4 * lane);
      float z = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
      for (int s = 16; s; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
      z *= a.scale_log2;
      M = fmaxf(M, z);  // (a NaN is left aside here and reaches the sums)
      const float ref = M == -INFINITY ? 0.f : M, f = exp2f(was - ref), p = exp2f(z - ref);
      was = M;
      l = l * f + p;
      o = make_float4(o.x * f + p * v.x, o.y * f + p * v.y, o.z * f + p * v.z, o.w * f + p * v.w);
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int64_t row = static_cast<int64_t>(token) * H + h;
    const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv, o.y * inv), y = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(a.out + row * kDim + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    if (lane == 0 && a.lse != nullptr) a.lse[row] = (M + log2f(l)) * 0.6931471805599453f;
  }
}

cudaError_t launch_prompt_attn(const PromptArgs& a, int num_sms, cudaStream_t s) {
  return launch_dependent(prompt_attn_kernel, dim3(num_sms * 8), 256, 0, s, a);
}

}  // namespace msa
