// Eviction by accumulated attention weight: each sequence's block table cut to its budget.
//
// One CTA per sequence.  Of the blocks between the forced ones (the first keep_first, the last
// keep_last) the k best by (weight descending, block ascending) stay.  The weight of the k-th
// best is found digit by digit (11 + 11 + 10 bits of the weights' order-preserving integers,
// largest first): a histogram of the digit in shared memory over the blocks that agree with
// the digits found so far, then a scan from the top.  Blocks above that weight stay, of those
// equal to it the lowest ones.  One pass then moves the blocks that stay and those that go to
// their places (prefix counts by ballot), 8192 blocks at a time: every block is read before
// anything is written at or above its place, so the outputs may be the inputs.
// Bound by latency (about ten CTA barriers and two rounds of loads); the table and the weights
// are read three to four times, from L2 after the first.
#include "fp8_kernels.h"
#include "msa_device.cuh"

namespace msa {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvItems = 8;                        // blocks per thread and step of the moving pass
constexpr int kEvBins = 2048;

struct EvShared {
  int bins[kEvBins];
  int warp_sum[2][kEvWarps];
  int digit, rest;
};

// Exclusive prefix of v over the CTA's threads (in thread order) and the total.
__device__ __forceinline__ int cta_prefix(int v, int* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int w = warp_sum[lane];  // kEvWarps == 32
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, s);
    if (lane >= s) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return x - v + (warp > 0 ? before : 0);
}

__global__ void __launch_bounds__(kEvThreads) evict_kernel(const EvictArgs a) {
  __shared__ EvShared sh;
  static_assert(kEvWarps == 32, "cta_prefix scans 32 warp sums in one warp");
  grid_dependency_wait();
  grid_dependents_launch();
  const int tid = threadIdx.x, b = blockIdx.x;
  const int64_t at = static_cast<int64_t>(b) * a.max_blocks;
  const float* weight = a.weight + at;
  const int32_t* table = a.block_table + at;
  const int MB = a.max_blocks;
  const int L = a.seq_lens[b];
  const bool ok = L >= 0 && L <= static_cast<int64_t>(MB) * kBlock;
  if (!ok && tid == 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
  const int nb = ok ? (L + kBlock - 1) / kBlock : MB;  // a bad row moves as it is
  const bool cut = ok && nb > a.budget;
  const int c0 = a.keep_first, c1 = nb - a.keep_last;  // the candidates, if cut
  const int k = a.budget - a.keep_first - a.keep_last; // places for them

  // the k-th largest order value among the candidates (k = 0: above all of them)
  uint32_t kth = 0xffffffffu;
  int equal = 0;  // how many of the candidates equal to it stay
  if (cut && k > 0) {
    uint32_t found = 0, mask = 0;
    int need = k;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      for (int i = tid; i < kEvBins; i += kEvThreads) sh.bins[i] = 0;
      __syncthreads();
      for (int i = c0 + tid; i < c1; i += kEvThreads) {
        const uint32_t o = score_order(weight[i]);
        if ((o & mask) == found) atomicAdd(&sh.bins[(o >> shift) & ((1u << bits) - 1u)], 1);
      }
      __syncthreads();
      // thread i holds the two bins 2 (1023 - i) + 1, 2 (1023 - i): counts from the top
      const int top = 2 * (kEvThreads - 1 - tid) + 1;
      const int n1 = sh.bins[top], n0 = sh.bins[top - 1];
      int total;
      const int above = cta_prefix(n1 + n0, sh.warp_sum[pass & 1], total);
      if (above < need && need <= above + n1) {
        sh.digit = top;
        sh.rest = need - above;
      } else if (above + n1 < need && need <= above + n1 + n0) {
        sh.digit = top - 1;
        sh.rest = need - above - n1;
      }
      __syncthreads();
      found |= static_cast<uint32_t>(sh.digit) << shift;
      mask |= ((1u << bits) - 1u) << shift;
      need = sh.rest;
      __syncthreads();
    }
    kth = found;
    equal = need;
  }

  int stayed = 0, gone = 0, ties = 0;
  for (int base = 0; base < nb; base += kEvThreads * kEvItems) {
    float w[kEvItems];
    int32_t page[kEvItems];
    uint32_t above = 0, tie = 0, in = 0;
    const int i0 = base + tid * kEvItems;
#pragma unroll
    for (int j = 0; j < kEvItems; ++j) {
      const int i = i0 + j;
      w[j] = 0.f;
      page[j] = -1;
      if (i < nb) {
        w[j] = weight[i];
        page[j] = table[i];
        in |= 1u << j;
        if (!cut || i < c0 || i >= c1) {
          above |= 1u << j;
        } else if (k > 0) {
          const uint32_t o = score_order(w[j]);
          if (o > kth) above |= 1u << j;
          if (o == kth) tie |= 1u << j;
        }
      }
    }
    int total;
    int rank = ties + cta_prefix(__popc(tie), sh.warp_sum[0], total);  // also: every read is done
    ties += total;
    uint32_t stay = above;
#pragma unroll
    for (int j = 0; j < kEvItems; ++j)
      if (tie >> j & 1u) {
        if (rank < equal) stay |= 1u << j;
        ++rank;
      }
    int p = stayed + cta_prefix(__popc(stay), sh.warp_sum[1], total);
    stayed += total;
    int f = gone + (i0 - base) - (p - (stayed - total));  // blocks before this thread's that go
    gone += min(nb - base, kEvThreads * kEvItems) - total;
#pragma unroll
    for (int j = 0; j < kEvItems; ++j) {
      if (!(in >> j & 1u)) continue;
      if (stay >> j & 1u) {
        a.table_out[at + p] = page[j];
        a.weight_out[at + p] = w[j];
        ++p;
      } else {
        a.freed[at + f] = page[j];
        ++f;
      }
    }
    __syncthreads();  // the warp sums are read before the next step writes them
  }
  for (int i = stayed + tid; i < MB; i += kEvThreads) {
    a.table_out[at + i] = -1;
    a.weight_out[at + i] = 0.f;
  }
  for (int i = gone + tid; i < MB; i += kEvThreads) a.freed[at + i] = -1;
  if (tid == 0) {
    a.seq_lens_out[b] = ok ? L - kBlock * gone : L;
    a.freed_count[b] = gone;
  }
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch));
  cfg.blockDim = dim3(kEvThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace msa
