// Eviction by accumulated attention weight: each sequence's block table cut to its budget.
//
// One CTA per sequence.  Of the blocks between the forced ones (the first keep_first, the last
// keep_last) the k best by (weight descending, block ascending) stay.  With the weights mapped to
// integers in their order, the k-th largest is found two bits at a time from the top, by counting the
// blocks at or above the three next candidates in registers and over the CTA; the search ends where
// exactly k blocks reach a candidate.  Long rows first find the top 12 bits by a histogram in shared
// memory (zero weights, blocks that nothing attended to, are counted by ballots: they would all meet
// in one counter), and one warp searches the bin's few blocks; where the bin holds many (equal
// weights), the CTA goes on as above from there.  Blocks above the weight
// found stay, of those equal to it the lowest ones.  One pass then moves what stays and what goes to
// its place, by ballots and prefix sums over the warps.  Every block is read before anything is
// written at or above its place, so the outputs may be the inputs.
//
// Bound by latency: the loads, then 1 to 16 counts of one barrier each, then two barriers a step to place
// the blocks.  512 rows of up to 4,096 blocks: 18.6 us, 0.9 TB/s of the bytes it cannot do without.
#include "fp8_kernels.h"
#include "msa_device.cuh"

namespace msa {

constexpr int kEvItems = 8;  // blocks per thread and step: a warp takes 256 consecutive blocks

constexpr int kEvBins = 4096;
constexpr int kEvListed = 256;  // keys of a bin that one warp takes

template <int kThreads>
using EvCounts = int[2][3][kThreads / 32];

template <int kThreads, bool kBins>
struct EvShared {
  EvCounts<kThreads> count;
};
template <int kThreads>
struct EvShared<kThreads, true> {
  EvCounts<kThreads> count;
  alignas(16) int bins[kEvBins];
  uint32_t list[kEvListed];
  int bin, rest, listed;
  uint32_t kth;
  int equal;
};

// v[0..2] summed over the CTA, in every thread.  One barrier a call: the buffers alternate.
template <int kThreads>
__device__ __forceinline__ void cta_sum3(int (&v)[3], EvCounts<kThreads>& count, int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int s = __reduce_add_sync(0xffffffffu, v[i]);
    if (lane == 0) count[turn][i][warp] = s;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) v[i] = __reduce_add_sync(0xffffffffu, lane < kThreads / 32 ? count[turn][i][lane] : 0);
  turn ^= 1;
}

// Sum of v over the warps before this one, and over all (v is warp-uniform); one barrier.
template <int kThreads>
__device__ __forceinline__ int cta_before(int v, EvCounts<kThreads>& count, int& turn, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) count[turn][0][warp] = v;
  __syncthreads();
  const int c = lane < kThreads / 32 ? count[turn][0][lane] : 0;
  total = __reduce_add_sync(0xffffffffu, c);
  turn ^= 1;
  return __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
}

template <int kThreads, bool kBins>
__global__ void __launch_bounds__(kThreads, kBins ? 2048 / kThreads : 4) evict_kernel(const EvictArgs a) {
  __shared__ EvShared<kThreads, kBins> sh;
  grid_dependency_wait();
  grid_dependents_launch();
  const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.x;
  const int64_t at = static_cast<int64_t>(b) * a.max_blocks;
  const float* weight = a.weight + at;
  const int32_t* table = a.block_table + at;
  const int MB = a.max_blocks, L = a.seq_lens[b];
  const bool ok = L >= 0 && L <= static_cast<int64_t>(MB) * kBlock;
  if (!ok && tid == 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
  const int nb = ok ? (L + kBlock - 1) / kBlock : MB;   // a bad row moves as it is
  const bool cut = ok && nb > a.budget;
  const int c0 = a.keep_first, c1 = nb - a.keep_last;   // the candidates, if cut
  const int k = a.budget - a.keep_first - a.keep_last;  // places for them
  constexpr int kStep = kThreads * kEvItems;
  const int mine = (tid >> 5) * 32 * kEvItems + lane;   // this thread's first block of a step
  int turn = 0;

  // A row of at most kStep blocks stays in registers for the search: its order values, 0 for blocks that
  // are no candidates (and for NaN, the lowest), and where the row is short also its weights and pages
  // (otherwise these are read again to be moved, so that four CTAs of 512 threads fit an SM).
  const bool once = nb <= kStep;
  const bool held = !kBins && once;
  float w[kEvItems];
  int32_t page[kEvItems];
  uint32_t order[kEvItems];
  auto fetch = [&](int base) {
#pragma unroll
    for (int j = 0; j < kEvItems; ++j) {
      const int i = base + mine + 32 * j;
      w[j] = i < nb ? weight[i] : 0.f;
      page[j] = i < nb ? table[i] : -1;
    }
  };
  // whether this warp has blocks of a step (ragged batches leave many warps none)
  auto busy = [&](int base) { return base + mine - lane < nb; };
  auto load = [&](int base) {
#pragma unroll
    for (int j = 0; j < kEvItems; ++j) order[j] = 0u;
    if (!busy(base)) return;
    float x[kEvItems];
#pragma unroll
    for (int j = 0; j < kEvItems; ++j) {
      const int i = base + mine + 32 * j;
      x[j] = i < c0 || i >= c1 ? NAN : held ? w[j] : weight[i];
    }
#pragma unroll
    for (int j = 0; j < kEvItems; ++j) order[j] = score_order(x[j]);
  };
  if (held) fetch(0);
  // Candidates with an order value above kth stay, and the lowest `equal` of those with kth itself.
  uint32_t kth = 0u;
  int equal = 0;
  // kth's bits below `shift` + 2, two at a time by counting over the CTA; then `equal`
  auto search = [&](int shift) {
    bool exact = false;
#pragma unroll 1
    for (; shift >= 0 && !exact; shift -= 2) {
      int n[3] = {0, 0, 0};
      for (int base = 0; base < nb; base += kStep) {
        if (!once) load(base);
        if (!busy(base)) continue;
#pragma unroll
        for (int j = 0; j < kEvItems; ++j)
#pragma unroll
          for (int d = 0; d < 3; ++d) n[d] += order[j] >= (kth | (static_cast<uint32_t>(d + 1) << shift)) ? 1 : 0;
      }
      cta_sum3<kThreads>(n, sh.count, turn);
      const int d = n[2] >= k ? 3 : n[1] >= k ? 2 : n[0] >= k ? 1 : 0;
      kth |= static_cast<uint32_t>(d) << shift;
      exact = d > 0 && n[d - 1] == k;  // exactly the k best are at or above it
    }
    if (exact) {
      kth -= 1;  // (above it: the same)
    } else {
      int n[3] = {0, 0, 0};  // candidates above the k-th weight (no order value is 2^32 - 1)
      for (int base = 0; base < nb; base += kStep) {
        if (!once) load(base);
#pragma unroll
        for (int j = 0; j < kEvItems; ++j) n[0] += order[j] > kth ? 1 : 0;
      }
      cta_sum3<kThreads>(n, sh.count, turn);
      equal = k - n[0];
    }
  };
  if (cut && k > 0) {
    if (!held)
      for (int i = tid * 32; i < nb; i += kThreads * 32)  // the table on its way to L2 meanwhile
        asm volatile("prefetch.global.L2 [%0];" ::"l"(table + i));
    if constexpr (!kBins) {
      if (once) load(0);
      search(30);
    } else {
      for (int i = tid; i < kEvBins / 4; i += kThreads) reinterpret_cast<int4*>(sh.bins)[i] = make_int4(0, 0, 0, 0);
      if (tid == 0) sh.listed = 0;
      __syncthreads();
      for (int base = 0; base < nb; base += kStep) {
        if (!once || base == 0) load(base);
        if (!busy(base)) continue;
#pragma unroll
        for (int j = 0; j < kEvItems; ++j) {
          const uint32_t o = order[j];
          const unsigned zeros = __ballot_sync(0xffffffffu, o == 0x80000000u);
          if (zeros != 0u && lane == 0) atomicAdd(&sh.bins[0x80000000u >> 20], __popc(zeros));
          if (o != 0u && o != 0x80000000u) atomicAdd(&sh.bins[o >> 20], 1);
        }
      }
      // NaN counts as order 0 and is in no bin: fewer than k blocks then reach a bin, and the last, 0,
      // takes the rest
      __syncthreads();
      // thread i holds the bins below kEvBins - i * kOwn: blocks from the top
      constexpr int kOwn = kEvBins / kThreads;
      int own[kOwn], sum = 0;
#pragma unroll
      for (int i = 0; i < kOwn; i += 4) {
        const int4 v = *reinterpret_cast<const int4*>(&sh.bins[kEvBins - 4 - tid * kOwn - i]);
        own[i] = v.w;
        own[i + 1] = v.z;
        own[i + 2] = v.y;
        own[i + 3] = v.x;
        sum += v.x + v.y + v.z + v.w;
      }
      int above = sum;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, above, s);
        if (lane >= s) above += y;
      }
      int total;
      const int warp_sum = __shfl_sync(0xffffffffu, above, 31);
      above += cta_before<kThreads>(warp_sum, sh.count, turn, total) - sum;
      if (above < k && above + sum >= k) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          if (above < k && above + own[i] >= k) {
            sh.bin = kEvBins - 1 - tid * kOwn - i;
            sh.rest = k - above;  // of its blocks stay
          }
          above += own[i];
        }
      }
      if (tid == 0 && total < k) {  // NaN blocks are among the k: all others stay
        sh.bin = -1;
        sh.rest = k - total;
      }
      __syncthreads();
      const int bin = sh.bin, rest = sh.rest;
      if (bin < 0) {
        equal = rest;  // kth is 0
      } else if (sh.bins[bin] == rest) {
        kth = (static_cast<uint32_t>(bin) << 20) - 1u;  // all of the bin (bin 0 holds no order value: no wrap)
      } else if (sh.bins[bin] <= kEvListed) {
        for (int base = 0; base < nb; base += kStep) {
          if (!once) load(base);
          if (!busy(base)) continue;
#pragma unroll
          for (int j = 0; j < kEvItems; ++j)
            if (order[j] >> 20 == static_cast<uint32_t>(bin) && order[j] != 0u) sh.list[atomicAdd(&sh.listed, 1)] = order[j];
        }
        __syncthreads();
        if (tid < 32) {
          constexpr int kEach = kEvListed / 32;
          uint32_t key[kEach];
#pragma unroll
          for (int j = 0; j < kEach; ++j) key[j] = lane + 32 * j < sh.listed ? sh.list[lane + 32 * j] : 0u;
          uint32_t found = static_cast<uint32_t>(bin) << 20;
          for (int shift = 18; shift >= 0; shift -= 2) {
            int n[3] = {0, 0, 0};
#pragma unroll
            for (int d = 0; d < 3; ++d) {
#pragma unroll
              for (int j = 0; j < kEach; ++j) n[d] += key[j] >= (found | (static_cast<uint32_t>(d + 1) << shift)) ? 1 : 0;
            }
#pragma unroll
            for (int d = 0; d < 3; ++d) n[d] = __reduce_add_sync(0xffffffffu, n[d]);
            found |= static_cast<uint32_t>(n[2] >= rest ? 3 : n[1] >= rest ? 2 : n[0] >= rest ? 1 : 0) << shift;
          }
          int n = 0;
#pragma unroll
          for (int j = 0; j < kEach; ++j) n += key[j] > found ? 1 : 0;
          n = __reduce_add_sync(0xffffffffu, n);
          if (lane == 0) {
            sh.kth = found;
            sh.equal = rest - n;
          }
        }
        __syncthreads();
        kth = sh.kth;
        equal = sh.equal;
      } else {
        kth = static_cast<uint32_t>(bin) << 20;
        search(18);
      }
    }
  }

  int stayed = 0, gone = 0, ties = 0;
  for (int base = 0; base < nb; base += kStep) {
    const bool some = busy(base);
    uint32_t stay = 0, tie = 0;  // bit j: block j of this thread
    int tie_here = 0;            // of the warp
    if (some) {
      if (!held) fetch(base);
#pragma unroll
      for (int j = 0; j < kEvItems; ++j) {
        const int i = base + mine + 32 * j;
        const bool in = i < nb, forced = !cut || i < c0 || i >= c1;
        const uint32_t o = score_order(w[j]);
        if (in && (forced || (k > 0 && o > kth))) stay |= 1u << j;
        if (in && !forced && k > 0 && o == kth) tie |= 1u << j;
      }
      tie_here = __reduce_add_sync(0xffffffffu, __popc(tie));
    }
    int total;
    int before = ties + cta_before<kThreads>(tie_here, sh.count, turn, total);  // (and: every block of the step is read)
    ties += total;
    int stay_here = 0;
    if (some) {
      if (tie_here > 0 && before < equal) {
#pragma unroll
        for (int j = 0; j < kEvItems; ++j) {
          const bool t = tie >> j & 1u;
          const unsigned m = __ballot_sync(0xffffffffu, t);
          if (t && before + __popc(m & ((1u << lane) - 1u)) < equal) stay |= 1u << j;
          before += __popc(m);
        }
      }
      stay_here = __reduce_add_sync(0xffffffffu, __popc(stay));
    }
    int place = stayed + cta_before<kThreads>(stay_here, sh.count, turn, total);
    int left = gone + (mine - lane) - (place - stayed);  // blocks of the step before this warp that go
    stayed += total;
    gone += min(nb - base, kStep) - total;
    if (some) {
      const unsigned below = (1u << lane) - 1u;
      int32_t* table_out = a.table_out + at;
      float* weight_out = a.weight_out + at;
      int32_t* freed = a.freed + at;
#pragma unroll
      for (int j = 0; j < kEvItems; ++j) {
        const bool in = base + mine + 32 * j < nb, s = stay >> j & 1u;
        const unsigned ms = __ballot_sync(0xffffffffu, s), mi = __ballot_sync(0xffffffffu, in);
        if (s) {
          table_out[place + __popc(ms & below)] = page[j];
          weight_out[place + __popc(ms & below)] = w[j];
        } else if (in) {
          freed[left + __popc(mi & ~ms & below)] = page[j];
        }
        place += __popc(ms);
        left += __popc(mi & ~ms);
      }
    }
  }
  for (int i = stayed + tid; i < MB; i += kThreads) {
    a.table_out[at + i] = -1;
    a.weight_out[at + i] = 0.f;
  }
  for (int i = gone + tid; i < MB; i += kThreads) a.freed[at + i] = -1;
  if (tid == 0) {
    a.seq_lens_out[b] = ok ? L - kBlock * gone : L;
    a.freed_count[b] = gone;
  }
}

// The fewest threads that hold a row in registers, up to 1024 (8,192 blocks); longer rows are
// loaded again for each count.  Rows of up to 2,048 blocks are searched by counting alone, longer ones
// begin with the histogram: 64 rows of 1,024 blocks take 7.8 us against 8.5, 512 rows of up to 4,096
// 28.0 us against 18.4.
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.batch));
  if (a.max_blocks <= 256 * kEvItems) return launch_dependent(evict_kernel<256, false>, grid, 256, 0, s, a);
  if (a.max_blocks <= 512 * kEvItems) return launch_dependent(evict_kernel<512, true>, grid, 512, 0, s, a);
  return launch_dependent(evict_kernel<1024, true>, grid, 1024, 0, s, a);
}

}  // namespace msa
