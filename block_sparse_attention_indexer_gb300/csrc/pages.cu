// The page pool: pages handed out, shared, given back and moved together.
//
// What is free is known from the reference counts alone, and pages are handed out from the lowest free number up, so
// a call needs the ranks of the free pages: a prefix sum over the counts.  page_count_kernel counts the free pages of
// each chunk of 2,048 (and copies what the call leaves in other arrays, and sums what the rows of the call need, in one more
// CTA); page_assign_kernel, a CTA for each chunk again, adds up the chunks before its own and gives every free page
// its rank and what follows from that.  A pool of one chunk is one launch.  Copies of pages (fork, compact) are a launch of
// their own, whose size the ranks decide.
// The ranks are bound by latency, a few rounds of loads and barriers: 4.2 us in a graph for 38,000 pages of which 64
// sequences take a few, 11.5 us for 890,000 of which 512 sequences take 70,000 (table and counts copied as well).  Measured
// for these: one cluster of eight CTAs that meets in distributed shared memory 7.3 and 43 us; chunks of 8,192
// pages 5.7 and 18 us.  Copies are bound by memory: a compaction that moves 500 pages in 8 buffers of 64 KB a page (and 8 of
// four bytes) 88 us, 5.9 TB/s.  Every CTA of page_assign_kernel adds up the counts of all chunks: work that grows with the square of the
// pool, nothing for a million pages (435 chunks), 17 GB read out of L2 for the 2^27 that a pool may have.
#include "fp8_kernels.h"
#include "msa_device.cuh"
#include "pages.h"

namespace msa {

constexpr int kPcThreads = 512, kPcWarps = kPcThreads / 32;
constexpr int kPcLoads = 1;                                  // int4 loads of a lane, four counts each
static_assert(kPageChunkPages == kPcThreads * kPcLoads * 4, "a chunk is what a CTA loads at once");

enum PageOp { kExtend, kFork, kCompact };

// ---------------------------------------------------------------- counts, and what the rows need

// Exclusive prefix sums of v over the CTA's threads, and their total (every thread).
__device__ __forceinline__ int cta_prefix(int v, int* warp_sum, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x = v;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  __syncthreads();  // (the last call's sums have been read)
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  const int w = lane < kPcWarps ? warp_sum[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, w);
  return x - v + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
}
__device__ __forceinline__ int cta_sum(int v, int* warp_sum) {
  const int s = __reduce_add_sync(0xffffffffu, v), lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) warp_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < kPcWarps ? warp_sum[lane] : 0);
}

// First of a lane's pages in a chunk; load i has the four pages 128 i on.
__device__ __forceinline__ int first_page(int chunk) {
  return chunk * kPageChunkPages + (threadIdx.x >> 5) * (kPageChunkPages / kPcWarps) + 4 * (threadIdx.x & 31);
}

// A lane's counts: bit 4 i + j is page at + 128 i + j, set where it is free.  `copy`, if not null, gets the counts.
__device__ __forceinline__ unsigned free_bits(const int32_t* refs, int pages, int at, int32_t* copy) {
  int4 r[kPcLoads];
#pragma unroll
  for (int i = 0; i < kPcLoads; ++i) {
    const int p = at + 128 * i;
    r[i] = make_int4(1, 1, 1, 1);
    if (p + 3 < pages) {
      r[i] = *reinterpret_cast<const int4*>(refs + p);
    } else if (p < pages) {
      r[i].x = refs[p];
      if (p + 1 < pages) r[i].y = refs[p + 1];
      if (p + 2 < pages) r[i].z = refs[p + 2];
    }
  }
  unsigned bits = 0u;
#pragma unroll
  for (int i = 0; i < kPcLoads; ++i) {
    const int p = at + 128 * i;
    bits |= ((r[i].x == 0 ? 1u : 0u) | (r[i].y == 0 ? 2u : 0u) | (r[i].z == 0 ? 4u : 0u) | (r[i].w == 0 ? 8u : 0u)) << (4 * i);
    if (copy == nullptr) continue;
    if (p + 3 < pages) {
      *reinterpret_cast<int4*>(copy + p) = r[i];
    } else if (p < pages) {
      copy[p] = r[i].x;
      if (p + 1 < pages) copy[p + 1] = r[i].y;
      if (p + 2 < pages) copy[p + 2] = r[i].z;
    }
  }
  return bits;
}

// need[r]: pages that the rows before r of an extension or a fork need; first[r]: extend, the row's first new block (-1: it
// stays as it is); fork, the parent's full blocks.
template <PageOp kOp>
__device__ __forceinline__ void row_needs(const PageArgs& a, int* warp_sum) {
  const int rows = kOp == kFork ? a.children : a.batch;
  const int64_t room = static_cast<int64_t>(a.max_blocks) * kBlock;
  int base = 0;
  for (int r0 = 0; r0 < rows; r0 += kPcThreads) {
    const int r = r0 + threadIdx.x;
    int need = 0, first = 0;
    if (r < rows && kOp == kExtend) {
      const int L = a.seq_lens[r], n = a.new_tokens != nullptr ? a.new_tokens[r] : L > 0 ? a.q_len : 0;
      const int64_t end = static_cast<int64_t>(L) + n;
      if (L < 0 || n < 0 || end > room) {
        flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
        first = -1;
      } else {
        first = (L + kBlock - 1) / kBlock;
        need = static_cast<int>((end + kBlock - 1) / kBlock) - first;
      }
    } else if (r < rows) {
      const int p = a.parents[r];
      if (p >= 0 && p < a.batch) {
        const int L = a.seq_lens[p];
        if (L < 0 || L > room) {
          flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
        } else {
          first = L / kBlock;
          if (L % kBlock != 0) {
            const int page = a.block_table[static_cast<int64_t>(p) * a.max_blocks + first];
            need = page >= 0 && page < a.num_pages;
            if (need == 0) flag_error(a.err, MSA_DEVERR_BAD_PAGE);
          }
        }
      } else if (p != -1) {
        flag_error(a.err, MSA_DEVERR_BAD_PARENT);
      }
    }
    int total;
    const int at = base + cta_prefix(need, warp_sum, total);
    if (r < rows) {
      a.need[r] = at;
      a.first[r] = first;
    }
    base += total;
  }
  if (threadIdx.x == 0) a.need[rows] = base;
}

// dst[i] = src[i], words i0, i0 + step, ...
__device__ __forceinline__ void copy_words(const int32_t* src, int32_t* dst, int64_t words, int64_t i0, int64_t step) {
  const bool wide = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
  const int64_t quads = wide ? words / 4 : 0;
  const int4* from = reinterpret_cast<const int4*>(src);
  int4* to = reinterpret_cast<int4*>(dst);
  int64_t i = i0;
  for (; i + 3 * step < quads; i += 4 * step) {
    int4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = from[i + j * step];
#pragma unroll
    for (int j = 0; j < 4; ++j) to[i + j * step] = x[j];
  }
  for (; i < quads; i += step) to[i] = from[i];
  for (i = 4 * quads + i0; i < words; i += step) dst[i] = src[i];
}

// CTA 0 sums the rows' needs, the next `chunks` count (and copy the counts), the others copy an extension's table.
template <PageOp kOp>
__global__ void __launch_bounds__(kPcThreads) page_count_kernel(const PageArgs a, int chunks) {
  __shared__ int warp_sum[kPcWarps];
  grid_dependency_wait();
  grid_dependents_launch();
  const int c = static_cast<int>(blockIdx.x) - 1;
  if (c < 0) {
    if (kOp != kCompact) row_needs<kOp>(a, warp_sum);
  } else if (c < chunks) {
    const unsigned bits = free_bits(a.refs, a.num_pages, first_page(c), a.refs != a.refs_out ? a.refs_out : nullptr);
    const int n = cta_sum(__popc(bits), warp_sum);
    if (threadIdx.x == 0) a.counts_free[c] = n;
  } else {
    copy_words(a.block_table, a.table_out, static_cast<int64_t>(a.batch) * a.max_blocks,
               static_cast<int64_t>(c - chunks) * kPcThreads + threadIdx.x,
               static_cast<int64_t>(gridDim.x - 1 - chunks) * kPcThreads);
  }
}

// ---------------------------------------------------------------- ranks

// The row that gets the new page of rank r: need[row] <= r < need[row + 1].
__device__ __forceinline__ int row_of(const int* need, int rows, int r) {
  int lo = 0, n = rows;
  while (n > 1) {
    const int h = n / 2;
    if (need[lo + h] <= r) {
      lo += h;
      n -= h;
    } else {
      n = h;
    }
  }
  return lo;
}

// Extend and fork hand out the first pages, compact lists the free pages below the number of pages in use and the pages
// in use from there on, and numbers them (page_map -2 - i: the i-th that moves).  A pool of one chunk is
// counted here as well, with all that page_count_kernel does (kOne).
template <PageOp kOp, bool kOne>
__global__ void __launch_bounds__(kPcThreads) page_assign_kernel(const PageArgs a, int chunks) {
  __shared__ int warp_sum[kPcWarps], need[kPageRows + 1], first_block[kPageRows];
  grid_dependency_wait();
  grid_dependents_launch();
  const int P = a.num_pages, rows = kOp == kFork ? a.children : a.batch, tid = threadIdx.x, lane = tid & 31;
  const int at = first_page(blockIdx.x);
  const unsigned bits = kOne ? free_bits(a.refs, P, at, a.refs != a.refs_out ? a.refs_out : nullptr)
                             : free_bits(a.refs_out, P, at, nullptr);
  if (kOne) {
    if (kOp != kCompact) row_needs<kOp>(a, warp_sum);
    if (kOp == kExtend && a.block_table != a.table_out)
      copy_words(a.block_table, a.table_out, static_cast<int64_t>(a.batch) * a.max_blocks, tid, kPcThreads);
    const int n = cta_sum(__popc(bits), warp_sum);
    if (tid == 0) a.counts_free[0] = n;
    __syncthreads();
  }
  int before = 0, all = 0;
  for (int c = tid; c < chunks; c += kPcThreads) {
    const int n = a.counts_free[c];
    all += n;
    before += c < static_cast<int>(blockIdx.x) ? n : 0;
  }
  if (kOp != kCompact)
    for (int r = tid; r <= rows; r += kPcThreads) {
      need[r] = a.need[r];
      if (r < rows) first_block[r] = a.first[r];
    }
  before = cta_sum(before, warp_sum);
  const int free_pages = cta_sum(all, warp_sum);  // (its barriers come after need[] as well)

  int given = 0;  // extend, fork: pages handed out, those of the rows whose running need fits
  const int live = P - free_pages;
  int holes = 0;  // compact: free pages below `live`, as many as pages in use from there on
  if (kOp == kCompact) {
    const int c1 = live / kPageChunkPages;  // the chunk with the border in it
    int n = 0;
    for (int c = tid; c < chunks && c < c1; c += kPcThreads) n += a.counts_free[c];
    if (c1 < chunks) {
      const int p0 = first_page(c1);
      const unsigned b1 = free_bits(a.refs_out, P, p0, nullptr);
#pragma unroll
      for (int i = 0; i < 4 * kPcLoads; ++i) n += (b1 >> i & 1u) && p0 + 128 * (i >> 2) + (i & 3) < live;
    }
    holes = cta_sum(n, warp_sum);
    if (blockIdx.x == 0 && tid == 0) {
      *a.live_count = live;
      *a.pairs = holes;
    }
  } else {
    int lo = 0, n = rows + 1;  // the last place with need[place] <= free_pages
    while (n > 1) {
      const int h = n / 2;
      if (need[lo + h] <= free_pages) {
        lo += h;
        n -= h;
      } else {
        n = h;
      }
    }
    given = need[lo];
    if (blockIdx.x == 0) {
      for (int r = tid; r < rows; r += kPcThreads) {
        const int want = need[r + 1] - need[r], first = first_block[r];
        const bool ok = want == 0 || need[r + 1] <= free_pages;
        if (!ok) flag_error(a.err, MSA_DEVERR_NO_PAGE);
        if (kOp == kExtend) {
          const int L = a.seq_lens[r], more = a.new_tokens != nullptr ? a.new_tokens[r] : L > 0 ? a.q_len : 0;
          a.seq_lens_out[r] = ok && first >= 0 ? L + more : L;
        } else {
          const int p = a.parents[r];
          const int L = p >= 0 && p < a.batch ? a.seq_lens[p] : 0;
          const bool good = L >= 0 && L <= static_cast<int64_t>(a.max_blocks) * kBlock;
          a.seq_lens_out[r] = !good ? 0 : ok ? L : first * kBlock;
          const int place = want != 0 && ok ? need[r] : -1;
          a.place[r] = place;
          if (place >= 0) {
            a.src[place] = a.block_table[static_cast<int64_t>(p) * a.max_blocks + first];
            a.tokens[place] = L % kBlock;
          }
        }
      }
      if (kOp == kFork && tid == 0) *a.pairs = given;
    }
    if (before >= given) return;  // (the whole CTA)
  }

  // every page's rank among the free ones
  int total;
  const int own = __reduce_add_sync(0xffffffffu, __popc(bits));
  const int in_cta = cta_prefix(lane == 0 ? own : 0, warp_sum, total);
  int rank = before + __shfl_sync(0xffffffffu, in_cta, 0);
  const unsigned below = (1u << lane) - 1u;
  int row = -1;  // of the lane's last page
#pragma unroll
  for (int i = 0; i < kPcLoads; ++i) {
    const unsigned b = bits >> (4 * i) & 15u;
    int r = rank;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned m = __ballot_sync(0xffffffffu, b >> j & 1u);
      r += __popc(m & below);
      rank += __popc(m);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int page = at + 128 * i + j;
      const bool is_free = b >> j & 1u;
      if (kOp == kCompact) {
        if (page < P) {
          if (is_free) {
            a.page_map[page] = -1;
            if (page < live) a.dst[r] = page;
          } else if (page < live) {
            a.page_map[page] = page;
          } else {  // pages in use and below: page - r, of them below `live`: live - holes
            const int n = page - r - (live - holes);
            a.src[n] = page;
            a.page_map[page] = -2 - n;
          }
        }
      } else if (is_free && r < given) {
        a.refs_out[page] = 1;
        if (kOp == kExtend) {
          if (row < 0) row = row_of(need, rows, r);
          while (need[row + 1] <= r) ++row;
          a.table_out[static_cast<int64_t>(row) * a.max_blocks + first_block[row] + (r - need[row])] = page;
        } else {
          a.dst[r] = page;
        }
      }
      r += is_free;
    }
  }
}

// ---------------------------------------------------------------- rows of tables, pages

// Buffers of one launch, cut into runs (of which a fork copies the first tokens) and these into chunks.
constexpr int kPageBuffers = 64, kPageChunk = 16384;
struct PageBuffers {
  struct {
    char* data;
    int64_t page_bytes;
    int32_t run_bytes, token_bytes;  // token_bytes 0: whole runs
    int32_t runs, chunks;            // of a page, of a run
  } buf[kPageBuffers];
  int32_t count;
};

// n bytes, 16 at a time where both addresses are multiples of 16, otherwise one at a time.
__device__ __forceinline__ void copy_bytes(char* dst, const char* src, int n) {
  const int tid = threadIdx.x;
  const uintptr_t d = reinterpret_cast<uintptr_t>(dst), s = reinterpret_cast<uintptr_t>(src);
  int done = 0;
  if (((d | s) & 15) == 0) {
    const int quads = n / 16;
    const uint4* from = reinterpret_cast<const uint4*>(src);
    uint4* to = reinterpret_cast<uint4*>(dst);
    for (int i0 = 0; i0 < quads; i0 += 1024) {  // a thread's four loads, then its stores
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + 256 * j + tid;
        if (i < quads) v[j] = __ldcs(from + i);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + 256 * j + tid;
        if (i < quads) __stcs(to + i, v[j]);
      }
    }
    done = quads * 16;
  }
  for (int i = done + tid; i < n; i += 256) dst[i] = src[i];
}

// Rows: fork, table_out and the references of the full blocks; compact, the renamed table, the final map and the counts of
// what moves (a page that moves is found in the map as its number among them or, already, as its new one).  Then the pages.
template <PageOp kOp>
__global__ void __launch_bounds__(256) page_move_kernel(const PageArgs a, const __grid_constant__ PageBuffers bufs, int rows_too) {
  grid_dependency_wait();
  grid_dependents_launch();
  if (rows_too) {
    const int rows = kOp == kFork ? a.children : a.batch;
    const int64_t all = static_cast<int64_t>(rows) * a.max_blocks, room = static_cast<int64_t>(a.max_blocks) * kBlock;
    const int64_t cta = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x, ctas = static_cast<int64_t>(gridDim.x) * gridDim.y;
    for (int64_t i = cta * 256 + threadIdx.x; i < all; i += ctas * 256) {
      const int r = static_cast<int>(i / a.max_blocks), n = static_cast<int>(i - static_cast<int64_t>(r) * a.max_blocks);
      int out = -1;
      if (kOp == kFork) {
        const int p = a.parents[r];
        const int L = p >= 0 && p < a.batch ? a.seq_lens[p] : 0;
        if (L > 0 && L <= room && n == L / kBlock && a.place[r] >= 0) {
          out = a.dst[a.place[r]];
        } else if (L > 0 && L <= room && n < L / kBlock) {
          const int page = a.block_table[static_cast<int64_t>(p) * a.max_blocks + n];
          if (page >= 0 && page < a.num_pages) {
            out = page;
            atomicAdd(a.refs_out + page, 1);
          } else {
            flag_error(a.err, MSA_DEVERR_BAD_PAGE);
          }
        }
      } else {
        const int L = a.seq_lens[r];
        const bool good = L >= 0 && L <= room;
        if (!good && n == 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
        if (!good || n < (L + kBlock - 1) / kBlock) {
          const int page = a.block_table[i];
          if (page >= 0 && page < a.num_pages) {
            out = __ldcg(a.page_map + page);
            if (out < -1) out = a.dst[-2 - out];
          }
          if (out < 0 && page != -1) flag_error(a.err, MSA_DEVERR_BAD_PAGE);
        }
      }
      a.table_out[i] = out;
    }
    if (kOp == kCompact) {
      const int moved = *a.pairs;
      for (int64_t i = cta * 256 + threadIdx.x; i < moved; i += ctas * 256) {
        const int from = a.src[i], to = a.dst[i];
        a.page_map[from] = to;
        a.refs_out[to] = a.refs_out[from];
        a.refs_out[from] = 0;
      }
    }
  }
  if (bufs.count == 0) return;
  const auto& b = bufs.buf[blockIdx.y];
  const int per_page = b.runs * b.chunks;
  const int64_t items = static_cast<int64_t>(*a.pairs) * per_page;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int pair = static_cast<int>(it / per_page), at = static_cast<int>(it - static_cast<int64_t>(pair) * per_page);
    const int run = at / b.chunks, lo = (at - run * b.chunks) * kPageChunk;
    int bytes = b.run_bytes;
    if (kOp == kFork && b.token_bytes > 0) bytes = a.tokens[pair] * b.token_bytes;
    const int n = min(bytes - lo, kPageChunk);
    if (n <= 0) continue;
    const int64_t off = static_cast<int64_t>(run) * b.run_bytes + lo;
    copy_bytes(b.data + a.dst[pair] * b.page_bytes + off, b.data + a.src[pair] * b.page_bytes + off, n);
  }
}

// ---------------------------------------------------------------- references given back

// A count is taken down by one and put back where it was 0 already.  Once one reference too many
// has been seen the true ones are all gone, so the final counts do not depend on the order.
__global__ void __launch_bounds__(256) page_free_kernel(const PageArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  for (int r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const int c = a.counts != nullptr ? a.counts[r] : a.width;
    if (c < 0 || c > a.width) {
      if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
      continue;
    }
    const int32_t* row = a.pages + static_cast<int64_t>(r) * a.width;
    // (64 bits: the row's end and a step of the grid together may pass 2^31)
    for (int64_t n0 = static_cast<int64_t>(blockIdx.x) * 1024 + threadIdx.x; n0 < c; n0 += static_cast<int64_t>(gridDim.x) * 1024) {
      int page[4], was[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) page[j] = n0 + 256 * j < c ? row[n0 + 256 * j] : -1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = page[j] >= 0 && page[j] < a.num_pages;
        was[j] = in ? atomicSub(a.refs_out + page[j], 1) : page[j] == -1 ? 1 : 0;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (was[j] <= 0) {
          if (page[j] >= 0 && page[j] < a.num_pages) atomicAdd(a.refs_out + page[j], 1);
          flag_error(a.err, MSA_DEVERR_BAD_PAGE);
        }
    }
  }
}

// ---------------------------------------------------------------- launches

// The counts and ranks of an operation.
template <PageOp kOp>
static cudaError_t launch_ranks(const PageArgs& a, int num_sms, cudaStream_t s) {
  const int chunks = (a.num_pages + kPageChunkPages - 1) / kPageChunkPages;
  const int64_t table = kOp == kExtend && a.block_table != a.table_out ? static_cast<int64_t>(a.batch) * a.max_blocks : 0;
  if (chunks == 1 && table <= 16 * kPcThreads)
    return launch_dependent(page_assign_kernel<kOp, true>, dim3(1), kPcThreads, 0, s, a, chunks);
  int64_t copies = (table + 4 * kPcThreads - 1) / (4 * kPcThreads);  // CTAs that copy the table, 4 words a thread (16: 13.2 us)
  if (copies > 8 * num_sms) copies = 8 * num_sms;
  const cudaError_t e = launch_dependent(page_count_kernel<kOp>, dim3(static_cast<unsigned>(1 + chunks + copies)), kPcThreads, 0, s,
                                         a, chunks);
  if (e != cudaSuccess) return e;
  return launch_dependent(page_assign_kernel<kOp, false>, dim3(static_cast<unsigned>(chunks)), kPcThreads, 0, s, a, chunks);
}

// refs into refs_out, where nothing else does it (free)
__global__ void __launch_bounds__(256) page_refs_kernel(const PageArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  copy_words(a.refs, a.refs_out, a.num_pages, static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x,
             static_cast<int64_t>(gridDim.x) * 256);
}

// Rows of a table (or list) by blockIdx.y, 1,024 entries of one by blockIdx.x.
static dim3 row_grid(int rows, int width, int num_sms) {
  const int x = width > 0 ? (width - 1) / 1024 + 1 : 1, most = num_sms * 8 / x + 1;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(rows < 1 ? 1 : rows < most ? rows : most));
}

template <PageOp kOp>
static cudaError_t launch_move(const PageArgs& a, int64_t most_pairs, int num_sms, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(kOp == kFork ? a.children : a.batch) * a.max_blocks;
  int k = 0;
  do {
    PageBuffers b;
    b.count = 0;
    int64_t most = 1;  // items of a buffer
    const bool first = k == 0;
    for (; k < a.num_buffers && b.count < kPageBuffers; ++k) {
      auto& x = b.buf[b.count++];
      x.data = static_cast<char*>(a.buffers[k].data);
      x.page_bytes = a.buffers[k].page_bytes;
      x.token_bytes = a.buffers[k].token_bytes;
      const bool runs = kOp == kFork && x.token_bytes > 0;
      x.run_bytes = runs ? x.token_bytes * kBlock : static_cast<int32_t>(x.page_bytes);
      x.runs = static_cast<int32_t>(x.page_bytes / x.run_bytes);
      x.chunks = (x.run_bytes - 1) / kPageChunk + 1;  // (run_bytes may be 2^31 - 1)
      const int64_t items = most_pairs * x.runs * x.chunks;
      most = items > most ? items : most;
    }
    const int y = b.count > 0 ? b.count : 1;
    int64_t x = first ? (rows + 256 * y - 1) / (256 * y) : 1;
    x = most > x ? most : x;
    const int64_t cap = (static_cast<int64_t>(num_sms) * 8 + y - 1) / y;
    const cudaError_t e = launch_dependent(page_move_kernel<kOp>, dim3(static_cast<unsigned>(x < cap ? x : cap), y), 256, 0, s, a,
                                           b, first ? 1 : 0);
    if (e != cudaSuccess) return e;
  } while (k < a.num_buffers);
  return cudaSuccess;
}

cudaError_t launch_extend_pages(const PageArgs& a, int num_sms, cudaStream_t s) { return launch_ranks<kExtend>(a, num_sms, s); }

cudaError_t launch_fork_pages(const PageArgs& a, int num_sms, cudaStream_t s) {
  const cudaError_t e = launch_ranks<kFork>(a, num_sms, s);
  return e != cudaSuccess ? e : launch_move<kFork>(a, a.children, num_sms, s);
}

cudaError_t launch_free_pages(const PageArgs& a, int num_sms, cudaStream_t s) {
  if (a.refs != a.refs_out) {
    const int ctas = (a.num_pages + 4095) / 4096, most = num_sms * 8;
    const cudaError_t e = launch_dependent(page_refs_kernel, dim3(static_cast<unsigned>(ctas < most ? ctas : most)), 256, 0, s, a);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(page_free_kernel, row_grid(a.rows, a.width, num_sms), 256, 0, s, a);
}

cudaError_t launch_compact_pages(const PageArgs& a, int num_sms, cudaStream_t s) {
  const cudaError_t e = launch_ranks<kCompact>(a, num_sms, s);
  return e != cudaSuccess ? e : launch_move<kCompact>(a, a.num_pages / 2, num_sms, s);
}

}  // namespace msa
