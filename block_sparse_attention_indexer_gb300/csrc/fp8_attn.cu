// msa_fp8_attn's dispatch, the tensor maps of its pages and the kernels that turn the blocks'
// shares into collected weights.  The attention itself: fp8_stream.cu (few query rows, or a
// selection) and fp8_tile.cu (more).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "fp8_device.cuh"
#include "fp8_kernels.h"
#include "msa_device.cuh"

namespace msa {

// ---------------------------------------------------------------- collected block weights
// weight_out[b][n] = decay * weight_in[b][n] + sum over rows of share * 2^(ref - M) / l.  ref - M is a
// difference of two near floats, so no logarithm of a large sum is taken and rounded on the way.

__device__ __forceinline__ float decayed(const Fp8AttnArgs& a, int64_t i) {
  return a.weight_in != nullptr ? a.weight_decay * a.weight_in[i] : 0.f;
}

// A row whose sum is NaN collects NaN in every block with a key that it sees, also where the share is 0, but not in a page
// that was skipped.  Whether a 0 is such a share, and whether block n's page of KV head g is one:
__device__ __forceinline__ bool zero_of_nan(float2 s, float2 st) { return s.x == 0.f && st.y != st.y; }
__device__ __noinline__ bool page_counts(const Fp8AttnArgs& a, int b, int n, int g) {
  const int page = a.block_table[static_cast<int64_t>(b) * a.max_blocks + n];
  if (page < 0 || page >= a.num_pages) return false;
  const int64_t ph = static_cast<int64_t>(page) * a.groups + g;
  return e8m0_ok(a.k_scale[ph]) && e8m0_ok(a.v_scale[ph]);
}

// Dense: one warp per (sequence, block) for few shares, else one CTA of 256 threads; each thread
// takes every 32nd (256th) of the block's shares (group, part, row), then a tree: a fixed order.
// Rows before the block's first key have no share there.
template <int kTeam>
__global__ void __launch_bounds__(256) fp8_weights_dense_kernel(const __grid_constant__ Fp8AttnArgs a, int parts) {
  __shared__ float s_sum[8];
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t idx = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / kTeam;
  if (idx >= static_cast<int64_t>(a.batch) * a.max_blocks) return;  // whole warps (kTeam 32) or CTAs
  const int b = static_cast<int>(idx / a.max_blocks), n = static_cast<int>(idx % a.max_blocks);
  const int tid = threadIdx.x % kTeam;
  const int L = a.seq_lens[b], T = a.q_len;
  const bool ok = length_ok(a, L) && n <= (L - 1) / kBlock;
  float sum = 0.f;
  if (ok) {
    const int rows = T * a.heads_per_group;
    // first row that sees the block: token t with L - T + t >= 128 n
    const int r0 = max(n * kBlock - (L - T), 0) * a.heads_per_group, seen = rows - r0;
    const int all = a.groups * parts * seen;
    unsigned nan = 0u;  // bit g: a zero of a NaN row in KV head g (at most 8)
#pragma unroll 4
    for (int i = tid; i < all; i += kTeam) {
      const int gp = i / seen, r = r0 + i - gp * seen, g = gp / parts, p = gp - g * parts;
      const int64_t unit = static_cast<int64_t>(b) * a.groups + g;
      const float2 s = a.share[((unit * a.max_blocks + n) * parts + p) * rows + r], st = a.row_stat[unit * rows + r];
      sum += s.x != 0.f ? s.x * exp2f(s.y - st.x) * st.y : 0.f;
      nan |= static_cast<unsigned>(zero_of_nan(s, st)) << g;
    }
    for (; nan != 0u; nan &= nan - 1u)
      if (page_counts(a, b, n, __ffs(nan) - 1)) sum = NAN;
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
  if (kTeam > 32) {
    if ((tid & 31) == 0) s_sum[tid >> 5] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += s_sum[w];
  }
  if (tid == 0) a.weight_out[idx] = decayed(a, idx) + sum;
}

// Sparse: each entry (row of the selection, slot) adds its share to its block as a fixed-point number
// with 40 fraction bits, so that the sum does not depend on the order (a sequence collects at
// most T * H < 2^22: it fits bit 62; bit 63 marks a NaN).  Eight lanes take an entry, a head each.
constexpr float kMassOne = 1099511627776.f;  // 2^40

// The block that entry i = (b, t, g, slot) adds to (-1: none), and in its first lane what it adds.  `nan` is set where
// the lane's head has a zero of a NaN row (page_counts has then the last word).
__device__ __forceinline__ int entry_share(const Fp8AttnArgs& a, int64_t i, bool in, float& sum, bool& nan) {
  const int h = threadIdx.x & 7, Hg = a.heads_per_group;
  int n = -1;
  sum = 0.f;
  if (in) {
    const int64_t unit = i / kTopK;
    const int bt = static_cast<int>(unit / a.groups), b = bt / a.q_len, L = a.seq_lens[b];
    n = a.selection[i];
    if (!length_ok(a, L) || n > (L - a.q_len + bt - b * a.q_len) / kBlock) n = -1;
    if (n >= 0 && h < Hg) {
      const float2 st = a.row_stat[unit * Hg + h];
      float2 s[kFp8StreamParts];
#pragma unroll
      for (int p = 0; p < kFp8StreamParts; ++p) s[p] = a.share[(i * kFp8StreamParts + p) * Hg + h];
#pragma unroll
      for (int p = 0; p < kFp8StreamParts; ++p) sum += s[p].x != 0.f ? s[p].x * exp2f(s[p].y - st.x) * st.y : 0.f;
#pragma unroll
      for (int p = 0; p < kFp8StreamParts; ++p) nan |= zero_of_nan(s[p], st);
    }
  }
#pragma unroll
  for (int s = 4; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
  return h == 0 ? n : -1;
}
// Whether entry i, which has block n, is in this thread's head a zero of a NaN row that counts as NaN.
__device__ __noinline__ bool nan_entry(const Fp8AttnArgs& a, int64_t i, int n) {
  const int h = threadIdx.x & 7, Hg = a.heads_per_group;
  const int64_t unit = i / kTopK;
  const int bt = static_cast<int>(unit / a.groups), b = bt / a.q_len, L = a.seq_lens[b];
  if (h >= Hg || n < 0 || !length_ok(a, L) || n > (L - a.q_len + bt - b * a.q_len) / kBlock) return false;
  bool nan = false;
  for (int p = 0; p < kFp8StreamParts; ++p)
    nan |= zero_of_nan(a.share[(i * kFp8StreamParts + p) * Hg + h], a.row_stat[unit * Hg + h]);
  return nan && page_counts(a, b, n, static_cast<int>(unit % a.groups));
}
__device__ __forceinline__ void add_mass(unsigned long long* m, float sum) {
  if (sum != sum)
    atomicOr(m, 1ull << 63);
  else if (sum > 0.f)
    atomicAdd(m, static_cast<unsigned long long>(static_cast<double>(sum) * static_cast<double>(kMassOne) + 0.5));
}
__device__ __forceinline__ float mass_value(unsigned long long m) {
  return (m >> 63) ? NAN : static_cast<float>(static_cast<double>(m) * (1.0 / static_cast<double>(kMassOne)));
}

// Few entries per sequence: a CTA per (sequence, 2,048 blocks) goes through all of them and keeps its
// blocks' sums in shared memory.
constexpr int kMassBlocks = 2048, kMassEntries = 2048, kMassThreads = 512;
__global__ void __launch_bounds__(kMassThreads) fp8_weights_sequence_kernel(const __grid_constant__ Fp8AttnArgs a) {
  __shared__ unsigned long long s_mass[kMassBlocks];
  grid_dependency_wait();
  grid_dependents_launch();
  const int b = blockIdx.y, n0 = blockIdx.x * kMassBlocks, n1 = min(n0 + kMassBlocks, a.max_blocks);
  for (int n = threadIdx.x; n < kMassBlocks; n += kMassThreads) s_mass[n] = 0ull;
  __syncthreads();
  const int entries = a.q_len * a.groups * kTopK;
  bool nan = false;
  for (int e0 = 0; e0 < entries; e0 += kMassThreads / 8) {
    const int e = e0 + threadIdx.x / 8;
    float sum;
    const int n = entry_share(a, static_cast<int64_t>(b) * entries + e, e < entries, sum, nan);
    if (n >= n0 && n < n1) add_mass(&s_mass[n - n0], sum);
  }
  if (nan)  // this thread's head of its entries, the zeros of NaN rows among them
    for (int e = threadIdx.x / 8; e < entries; e += kMassThreads / 8) {
      const int64_t i = static_cast<int64_t>(b) * entries + e;
      const int n = a.selection[i];
      if (n >= n0 && n < n1 && nan_entry(a, i, n)) add_mass(&s_mass[n - n0], NAN);
    }
  __syncthreads();
  for (int n = n0 + threadIdx.x; n < n1; n += kMassThreads) {
    const int64_t i = static_cast<int64_t>(b) * a.max_blocks + n;
    a.weight_out[i] = decayed(a, i) + mass_value(s_mass[n - n0]);
  }
}

// Many: the entries of all sequences over the grid, into sums in the workspace that a second kernel reads.
__global__ void __launch_bounds__(256) fp8_weights_scatter_kernel(const __grid_constant__ Fp8AttnArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t all = static_cast<int64_t>(a.batch) * a.q_len * a.groups * kTopK;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / 8;
  float sum;
  bool nan = false;
  const int n = entry_share(a, i, i < all, sum, nan);
  if (nan && nan_entry(a, i, a.selection[i]))
    add_mass(a.mass + i / (static_cast<int64_t>(a.q_len) * a.groups * kTopK) * a.max_blocks + a.selection[i], NAN);
  if (n >= 0) add_mass(a.mass + i / (static_cast<int64_t>(a.q_len) * a.groups * kTopK) * a.max_blocks + n, sum);
}
__global__ void __launch_bounds__(256) fp8_weights_sparse_kernel(const Fp8AttnArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < static_cast<int64_t>(a.batch) * a.max_blocks) a.weight_out[i] = decayed(a, i) + mass_value(a.mass[i]);
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
  const size_t stream = fp8_stream_partial_bytes();  // a selection takes that form whatever the rows
  if (rows <= kFp8StreamRows) return stream;
  const size_t tile = fp8_tile_partial_bytes();
  return tile > stream ? tile : stream;
}

cudaError_t launch_fp8_attn(const Fp8AttnArgs& a, int num_sms, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const int64_t blocks = static_cast<int64_t>(a.batch) * a.max_blocks;
  const bool sparse = a.selection != nullptr, weights = a.weight_out != nullptr;
  const int64_t units = static_cast<int64_t>(a.batch) * a.q_len * a.groups;
  const bool stream = sparse || a.q_len * a.heads_per_group <= kFp8StreamRows;
  const int parts = stream ? kFp8StreamParts : 1;
  // one launch while a sequence's entries are few (64 sequences of 64 entries over 1,024 blocks: 35.1 us with
  // the attention, against 36.8 with the three of many; a CTA's 512 threads take 2,048 entries in 32 rounds,
  // where many CTAs would share them)
  const bool few = a.q_len * a.groups * kTopK <= kMassEntries;
  if (sparse && weights && !few && (e = cudaMemsetAsync(a.mass, 0, blocks * sizeof(*a.mass), s)) != cudaSuccess) return e;
  e = stream ? launch_fp8_stream(a, num_sms, s) : launch_fp8_tile(a, num_sms, s);
  if (e != cudaSuccess || !weights) return e;
  if (sparse && few)
    return launch_dependent(fp8_weights_sequence_kernel,
                            dim3(static_cast<unsigned>((a.max_blocks + kMassBlocks - 1) / kMassBlocks),
                                 static_cast<unsigned>(a.batch)), kMassThreads, 0, s, a);
  if (sparse) {
    e = launch_dependent(fp8_weights_scatter_kernel, dim3(static_cast<unsigned>((units * kTopK + 31) / 32)), 256, 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_dependent(fp8_weights_sparse_kernel, dim3(static_cast<unsigned>((blocks + 255) / 256)), 256, 0, s, a);
  }
  // a warp a block up to 128 entries (64 sequences of 4K, one token: 43.6 us with the attention, 44.5 with a
  // CTA a block; 8 of 32K: 39.6 and 40.1), a CTA from there (256 entries, 16 sequences of 16K: 61.4 us, 65.5 with
  // a warp; 1,152 entries, 46 sequences of 6 blocks: 95 and 112)
  const int64_t each = static_cast<int64_t>(a.groups) * parts * a.q_len * a.heads_per_group;
  return each <= 128 ? launch_dependent(fp8_weights_dense_kernel<32>, dim3(static_cast<unsigned>((blocks + 7) / 8)), 256, 0,
                                         s, a, parts)
                      : launch_dependent(fp8_weights_dense_kernel<256>, dim3(static_cast<unsigned>(blocks)), 256, 0, s, a,
                                         parts);
}

}  // namespace msa
