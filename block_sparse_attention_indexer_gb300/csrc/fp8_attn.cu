// Attention over the FP8 page cache: dense causal, or over selected blocks.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "fp8_device.cuh"
#include "fp8_kernels.h"
#include "msa_device.cuh"

namespace msa {

constexpr int kHeadsMax = 8;

// One CTA per (sequence, token, group): every head of the group against the visible keys, page
// by page with a running maximum and sum.  Thread j scores key j of a page, thread d keeps
// output dim d.
__global__ void __launch_bounds__(128) fp8_attn_simple_kernel(const Fp8AttnArgs a) {
  __shared__ float s_q[kHeadsMax][kDim];
  __shared__ float s_p[kHeadsMax][kBlock];
  __shared__ float s_red[2][4][kHeadsMax];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  const int g = blockIdx.x % a.groups;
  const int bt = blockIdx.x / a.groups;
  const int T = a.q_len, b = bt / T, t = bt % T, Hg = a.heads_per_group;
  const int L = a.seq_lens[b];
  const bool ok = L > 0 && L >= T && L <= static_cast<int64_t>(a.max_blocks) * kBlock;
  if (!ok && L != 0 && tid == 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
  const int pos = L - T + t;
  for (int h = 0; h < Hg; ++h) {
    const int64_t o = static_cast<int64_t>(bt) * a.q_stride + (g * Hg + h) * kDim + tid;
    s_q[h][tid] = a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[o])
                           : f16x2_to_float2(e4m3x2_to_f16x2(static_cast<const uint8_t*>(a.q)[o])).x;
  }
  __syncthreads();
  float m[kHeadsMax], l[kHeadsMax], acc[kHeadsMax];
  for (int h = 0; h < kHeadsMax; ++h) {
    m[h] = -INFINITY;
    l[h] = acc[h] = 0.f;
  }
  const bool sparse = a.selection != nullptr;
  const int places = !ok ? 0 : sparse ? kTopK : pos / kBlock + 1;
  const int64_t unit = sparse ? static_cast<int64_t>(blockIdx.x) : static_cast<int64_t>(b) * a.groups + g;
  const int64_t unit_rows = sparse ? Hg : static_cast<int64_t>(T) * Hg;
  const int64_t row0 = sparse ? 0 : static_cast<int64_t>(t) * Hg;
  for (int i = 0; i < places; ++i) {
    const int n = sparse ? a.selection[static_cast<int64_t>(blockIdx.x) * kTopK + i] : i;
    int page = -1;
    if (n >= 0 && n <= pos / kBlock) {
      page = a.block_table[static_cast<int64_t>(b) * a.max_blocks + n];
      if (page < 0 || page >= a.num_pages) {
        if (tid == 0) flag_error(a.err, MSA_DEVERR_BAD_PAGE);
        page = -1;
      }
    }
    const int64_t ph = static_cast<int64_t>(page) * a.groups + g;
    if (page >= 0 && !(e8m0_ok(a.k_scale[ph]) && e8m0_ok(a.v_scale[ph]))) {
      if (tid == 0) flag_error(a.err, MSA_DEVERR_BAD_SCALE);
      page = -1;
    }
    float2* share = a.share + ((unit * (sparse ? kTopK : a.max_blocks) + i) * unit_rows + row0);
    if (page < 0) {
      if (a.weight_out != nullptr && tid < Hg) share[tid] = make_float2(0.f, 0.f);
      continue;
    }
    const float ks = exp2_int(a.k_scale[ph] - kE8m0One) * a.scale_log2;
    const float vs = exp2_int(a.v_scale[ph] - kE8m0One);
    const int vis = min(pos - n * kBlock + 1, kBlock);  // visible keys of the page
    float z[kHeadsMax];
    for (int h = 0; h < kHeadsMax; ++h) z[h] = 0.f;
    if (tid < vis) {
      const uint8_t* k = a.k_data + ph * kFp8PageBytes + tid * kDim;
      for (int d = 0; d < kDim; d += 4) {
        uint32_t h0, h1;
        e4m3x4_to_f16x4(*reinterpret_cast<const uint32_t*>(k + d), h0, h1);
        const float2 x = f16x2_to_float2(h0), y = f16x2_to_float2(h1);
        for (int h = 0; h < Hg; ++h)
          z[h] += s_q[h][d] * x.x + s_q[h][d + 1] * x.y + s_q[h][d + 2] * y.x + s_q[h][d + 3] * y.y;
      }
    }
    for (int h = 0; h < Hg; ++h) {
      z[h] = tid < vis ? z[h] * ks : -INFINITY;
      float w = z[h];
      for (int s = 16; s; s >>= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, s));
      if (lane == 0) s_red[0][warp][h] = w;
    }
    __syncthreads();
    for (int h = 0; h < Hg; ++h) {
      const float mp = fmaxf(fmaxf(s_red[0][0][h], s_red[0][1][h]), fmaxf(s_red[0][2][h], s_red[0][3][h]));
      const float mn = fmaxf(m[h], mp);
      const float p = exp2f(z[h] - mn);
      s_p[h][tid] = p;
      float w = p;
      for (int s = 16; s; s >>= 1) w += __shfl_xor_sync(0xffffffffu, w, s);
      if (lane == 0) s_red[1][warp][h] = w;
      const float alpha = exp2f(m[h] - mn);
      l[h] *= alpha;
      acc[h] *= alpha;
      m[h] = mn;
    }
    __syncthreads();
    for (int h = 0; h < Hg; ++h) {
      const float sum = s_red[1][0][h] + s_red[1][1][h] + s_red[1][2][h] + s_red[1][3][h];
      l[h] += sum;
      if (a.weight_out != nullptr && tid == 0) share[h] = make_float2(sum, m[h]);
    }
    const uint8_t* v = a.v_data + ph * kFp8PageBytes + tid;
    float part[kHeadsMax];
    for (int h = 0; h < kHeadsMax; ++h) part[h] = 0.f;
    for (int j = 0; j < vis; ++j) {
      const float x = f16x2_to_float2(e4m3x2_to_f16x2(v[j * kDim])).x;
      for (int h = 0; h < Hg; ++h) part[h] += s_p[h][j] * x;
    }
    for (int h = 0; h < Hg; ++h) acc[h] += vs * part[h];
    __syncthreads();
  }
  for (int h = 0; h < Hg; ++h) {
    const int64_t r = static_cast<int64_t>(bt) * a.groups * Hg + g * Hg + h;
    const bool any = m[h] != -INFINITY;
    a.out[r * kDim + tid] = __bfloat16_as_ushort(__float2bfloat16_rn(any ? acc[h] / l[h] : 0.f));
    if (tid == 0 && a.lse != nullptr) a.lse[r] = any ? (m[h] + log2f(l[h])) * 0.6931471805599453f : -INFINITY;
    if (tid == 0 && a.weight_out != nullptr)
      a.row_stat[unit * unit_rows + row0 + h] = any ? make_float2(m[h], 1.f / l[h]) : make_float2(0.f, 0.f);
  }
}

// ---------------------------------------------------------------- collected block weights
// weight_out[b][n] = decay * weight_in[b][n] + sum over rows of share * 2^(ref - M) / l.  ref - M is a
// difference of two near floats, so no logarithm of a large sum is taken and rounded on the way.

__device__ __forceinline__ float decayed(const Fp8AttnArgs& a, int64_t i) {
  return a.weight_in != nullptr ? a.weight_decay * a.weight_in[i] : 0.f;
}

// Dense: one warp per (sequence, block) for few rows, else one CTA of 256 threads; each thread
// takes every 32nd (256th) (part, row) of the groups in turn, then a tree: a fixed order.
// row_tile: the rows whose pages were computed together (a row below the block's first key has
// a share only if the tile it is in reached the block).
template <int kTeam>
__global__ void __launch_bounds__(256) fp8_weights_dense_kernel(const Fp8AttnArgs a, int parts) {
  __shared__ float s_sum[8];
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t idx = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / kTeam;
  if (idx >= static_cast<int64_t>(a.batch) * a.max_blocks) return;  // whole warps (kTeam 32) or CTAs
  const int b = static_cast<int>(idx / a.max_blocks), n = static_cast<int>(idx % a.max_blocks);
  const int tid = threadIdx.x % kTeam;
  const int L = a.seq_lens[b], T = a.q_len;
  const bool ok = L > 0 && L >= T && L <= static_cast<int64_t>(a.max_blocks) * kBlock && n <= (L - 1) / kBlock;
  float sum = 0.f;
  if (ok) {
    const int rows = T * a.heads_per_group;
    // first row that sees the block: token t with L - T + t >= 128 n
    const int r0 = max(n * kBlock - (L - T), 0) * a.heads_per_group;
    for (int g = 0; g < a.groups; ++g) {
      const int64_t unit = static_cast<int64_t>(b) * a.groups + g;
      const float2* stat = a.row_stat + unit * rows;
      for (int p = 0; p < parts; ++p) {
        const float2* share = a.share + ((unit * a.max_blocks + n) * parts + p) * rows;
        for (int r = r0 + tid; r < rows; r += kTeam) {
          const float2 s = share[r], st = stat[r];
          if (s.x != 0.f) sum += s.x * exp2f(s.y - st.x) * st.y;
        }
      }
    }
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
  if (kTeam > 32) {
    if ((tid & 31) == 0) s_sum[tid >> 5] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kTeam / 32; ++w) sum += s_sum[w % 8];
  }
  if (tid == 0) a.weight_out[idx] = decayed(a, idx) + sum;
}

// Sparse: each (row of the selection, slot) adds its share to its block as a fixed-point number
// with 40 fraction bits, so that the sum does not depend on the order (a sequence collects at
// most T * H < 2^22: it fits bit 62; bit 63 marks a NaN).
__global__ void __launch_bounds__(256) fp8_weights_scatter_kernel(const Fp8AttnArgs a, int parts) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t units = static_cast<int64_t>(a.batch) * a.q_len * a.groups;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= units * kTopK) return;
  const int64_t unit = i / kTopK;
  const int bt = static_cast<int>(unit / a.groups), b = bt / a.q_len, t = bt % a.q_len;
  const int L = a.seq_lens[b], n = a.selection[i];
  if (!(L > 0 && L >= a.q_len && L <= static_cast<int64_t>(a.max_blocks) * kBlock) || n < 0 ||
      n > (L - a.q_len + t) / kBlock)
    return;
  const int Hg = a.heads_per_group;
  float sum = 0.f;
  for (int p = 0; p < parts; ++p)
    for (int h = 0; h < Hg; ++h) {
      const float2 s = a.share[(i * parts + p) * Hg + h], st = a.row_stat[unit * Hg + h];
      if (s.x != 0.f) sum += s.x * exp2f(s.y - st.x) * st.y;
    }
  unsigned long long* m = a.mass + static_cast<int64_t>(b) * a.max_blocks + n;
  if (sum != sum)
    atomicOr(m, 1ull << 63);
  else if (sum > 0.f)
    atomicAdd(m, static_cast<unsigned long long>(static_cast<double>(sum) * 1099511627776.0 + 0.5));
}

__global__ void __launch_bounds__(256) fp8_weights_sparse_kernel(const Fp8AttnArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.batch) * a.max_blocks) return;
  const unsigned long long m = a.mass[i];
  const float sum = (m >> 63) ? NAN : static_cast<float>(static_cast<double>(m) * (1.0 / 1099511627776.0));
  a.weight_out[i] = decayed(a, i) + sum;
}

// ---------------------------------------------------------------- tensor maps and dispatch

cudaError_t fp8_page_maps(const Fp8AttnArgs& a, Fp8Maps* maps) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  // row coordinates are signed 32-bit: the host has checked num_pages * G <= 2^24
  const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(a.num_pages) * a.groups * kBlock};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, kBlock};
  const cuuint32_t estr[2] = {1, 1};
  for (int i = 0; i < 2; ++i) {
    const CUresult r = encode(i ? &maps->v : &maps->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                              const_cast<uint8_t*>(i ? a.v_data : a.k_data), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

size_t fp8_attn_partial_bytes(int64_t rows) {
  (void)rows;
  return fp8_stream_partial_bytes();
}

cudaError_t launch_fp8_attn(const Fp8AttnArgs& a, int num_sms, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const int64_t blocks = static_cast<int64_t>(a.batch) * a.max_blocks;
  const bool sparse = a.selection != nullptr, weights = a.weight_out != nullptr;
  const int64_t units = static_cast<int64_t>(a.batch) * a.q_len * a.groups;
  const bool stream = sparse || a.q_len * a.heads_per_group <= kFp8StreamRows;
  const int parts = stream ? kFp8StreamParts : 1;
  if (sparse && weights && (e = cudaMemsetAsync(a.mass, 0, blocks * sizeof(*a.mass), s)) != cudaSuccess) return e;
  e = stream ? launch_fp8_stream(a, num_sms, s)
             : launch_dependent(fp8_attn_simple_kernel, dim3(static_cast<unsigned>(units)), 128, 0, s, a);
  if (e != cudaSuccess || !weights) return e;
  if (sparse) {
    e = launch_dependent(fp8_weights_scatter_kernel, dim3(static_cast<unsigned>((units * kTopK + 255) / 256)), 256, 0, s,
                         a, parts);
    if (e != cudaSuccess) return e;
    return launch_dependent(fp8_weights_sparse_kernel, dim3(static_cast<unsigned>((blocks + 255) / 256)), 256, 0, s, a);
  }
  const int64_t each = static_cast<int64_t>(a.groups) * parts * a.q_len * a.heads_per_group;
  return each <= 2048 ? launch_dependent(fp8_weights_dense_kernel<32>, dim3(static_cast<unsigned>((blocks + 7) / 8)), 256, 0,
                                         s, a, parts)
                      : launch_dependent(fp8_weights_dense_kernel<256>, dim3(static_cast<unsigned>(blocks)), 256, 0, s, a,
                                         parts);
}

}  // namespace msa
