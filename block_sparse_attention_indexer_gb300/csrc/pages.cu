// The page pool: pages handed out, shared, given back and moved together.
//
// What is free is known from the reference counts alone: pages are handed out from the lowest
// free number up, so a call needs the ranks of the free pages, a prefix sum over the counts.
// page_scan_kernel makes it with one cluster of eight CTAs (a pool of 500,000 pages is then 64
// counts a thread, kept as one bit each): the CTAs' sums meet in distributed shared memory, so
// that there is one launch and no partial sum in global memory.  What follows (rows of tables,
// copies of pages) is a second launch over the whole GPU, whose size the first one decides.
#include <cooperative_groups.h>

#include "fp8_kernels.h"
#include "msa_device.cuh"
#include "pages.h"

namespace msa {

namespace cg = cooperative_groups;

constexpr int kPcCtas = 8, kPcThreads = 1024, kPcWarps = kPcThreads / 32;
constexpr int kPcIters = 16;                                   // int4 loads of a lane in a round: 64 counts, a bit each
constexpr int kPcRound = kPcCtas * kPcWarps * kPcIters * 128;  // pages of a round: 524,288

enum PageOp { kExtend, kFork, kCompact };

// ---------------------------------------------------------------- inputs whose outputs lie elsewhere

// dst[i] = src[i] for up to three arrays of 32-bit words, before the operation changes them in place.
struct PageCopies {
  const int32_t* src[3];
  int32_t* dst[3];
  int64_t words[3];
};
__global__ void __launch_bounds__(256) page_words_kernel(const PageCopies c) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<int64_t>(gridDim.x) * 256;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (c.words[k] == 0) continue;
    const bool wide = ((reinterpret_cast<uintptr_t>(c.src[k]) | reinterpret_cast<uintptr_t>(c.dst[k])) & 15) == 0;
    const int64_t quads = wide ? c.words[k] / 4 : 0;
    const int4* src = reinterpret_cast<const int4*>(c.src[k]);
    int4* dst = reinterpret_cast<int4*>(c.dst[k]);
#pragma unroll 4
    for (int64_t i = t0; i < quads; i += step) dst[i] = src[i];
    for (int64_t i = 4 * quads + t0; i < c.words[k]; i += step) c.dst[k][i] = c.src[k][i];
  }
}

// ---------------------------------------------------------------- ranks of the free pages

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
  const int w = warp_sum[lane];
  total = __reduce_add_sync(0xffffffffu, w);
  return x - v + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
}

struct PageScan {
  int warp_sum[kPcWarps];
  int cta_sum[2];              // of this CTA, read by the others: by turns, so that one barrier a sum is enough
  int need[kPageRows + 1];     // prefix sums of what the rows need
  int first[kPageRows];        // extend: a row's first new block; fork: the parent's full blocks
};

// Sum of v over the cluster (in each CTA the same on all threads), and of the CTAs before this one.
__device__ __forceinline__ int cluster_sum(cg::cluster_group& cl, PageScan& sh, int turn, int v, int& before) {
  if (threadIdx.x == 0) sh.cta_sum[turn & 1] = v;
  cl.sync();
  const int rank = static_cast<int>(cl.block_rank()), lane = threadIdx.x & 31;
  const int x = lane < kPcCtas ? *cl.map_shared_rank(&sh.cta_sum[turn & 1], lane) : 0;
  before = __reduce_add_sync(0xffffffffu, lane < rank ? x : 0);
  return __reduce_add_sync(0xffffffffu, x);
}

// What the rows of an extension or a fork need.  Every CTA sums for itself; rank 0 flags.
template <PageOp kOp>
__device__ __forceinline__ void row_needs(const PageArgs& a, PageScan& sh, bool flag) {
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
        if (flag) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
        first = -1;  // stays as it is
      } else {
        first = (L + kBlock - 1) / kBlock;
        need = static_cast<int>((end + kBlock - 1) / kBlock) - first;
      }
    } else if (r < rows) {
      const int p = a.parents[r];
      if (p >= 0 && p < a.batch) {
        const int L = a.seq_lens[p];
        if (L < 0 || L > room) {
          if (flag) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
        } else {
          first = L / kBlock;
          if (L % kBlock != 0) {
            const int page = a.block_table[static_cast<int64_t>(p) * a.max_blocks + first];
            need = page >= 0 && page < a.num_pages;
            if (flag && need == 0) flag_error(a.err, MSA_DEVERR_BAD_PAGE);
          }
        }
      } else if (p != -1 && flag) {
        flag_error(a.err, MSA_DEVERR_BAD_PARENT);
      }
    }
    int total;
    const int at = base + cta_prefix(need, sh.warp_sum, total);
    if (r < rows) {
      sh.need[r] = at;
      sh.first[r] = first;
    }
    base += total;
  }
  if (threadIdx.x == 0) sh.need[rows] = base;
  __syncthreads();
}

// One round's counts of this lane: bit 4 i + j is page at + 128 i + j, set where it is free.
__device__ __forceinline__ unsigned long long free_bits(const int32_t* refs, int pages, int at, int iters) {
  unsigned long long bits = 0ull;
#pragma unroll 4
  for (int i = 0; i < iters; ++i) {
    const int p = at + 128 * i;
    int4 r = make_int4(1, 1, 1, 1);
    if (p + 3 < pages) {
      r = __ldcg(reinterpret_cast<const int4*>(refs + p));
    } else if (p < pages) {
      r.x = refs[p];
      if (p + 1 < pages) r.y = refs[p + 1];
      if (p + 2 < pages) r.z = refs[p + 2];
    }
    const unsigned b = (r.x == 0 ? 1u : 0u) | (r.y == 0 ? 2u : 0u) | (r.z == 0 ? 4u : 0u) | (r.w == 0 ? 8u : 0u);
    bits |= static_cast<unsigned long long>(b) << (4 * i);
  }
  return bits;
}

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

// Works in place: refs_out, table_out (extend) and seq_lens_out (extend) hold the inputs.
template <PageOp kOp>
__global__ void __cluster_dims__(kPcCtas, 1, 1) __launch_bounds__(kPcThreads) page_scan_kernel(const PageArgs a) {
  __shared__ PageScan sh;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = static_cast<int>(cl.block_rank()), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  const int P = a.num_pages, rounds = (P + kPcRound - 1) / kPcRound;
  const int rows = kOp == kFork ? a.children : a.batch;
  // the warps of the cluster have equal runs of pages, one after another
  auto iters_of = [&](int round) {
    const int left = min(P - round * kPcRound, kPcRound);
    return (left + kPcCtas * kPcWarps * 128 - 1) / (kPcCtas * kPcWarps * 128);
  };
  auto first_of = [&](int round, int iters) {
    return round * kPcRound + (rank * kPcWarps + warp) * iters * 128 + 4 * lane;
  };
  if (kOp != kCompact) row_needs<kOp>(a, sh, rank == 0);

  // the free pages of the pool
  int turn = 0, before, total, mine = 0;
  unsigned long long bits = 0ull;  // of the last round: kept where there is only one
  for (int round = 0; round < rounds; ++round) {
    const int iters = iters_of(round);
    bits = free_bits(a.refs_out, P, first_of(round, iters), iters);
    mine += __popcll(bits);
  }
  cta_prefix(mine, sh.warp_sum, total);
  const int free_pages = cluster_sum(cl, sh, turn++, total, before);

  int given = 0;               // extend, fork: pages handed out
  const int live = P - free_pages;
  int holes = 0;               // compact: free pages below `live`, as many as pages in use from there on
  if (kOp == kCompact) {
    mine = 0;
    for (int round = 0; round < rounds; ++round) {
      const int iters = iters_of(round), at = first_of(round, iters);
      if (rounds > 1) bits = free_bits(a.refs_out, P, at, iters);
      for (unsigned long long b = bits; b != 0ull; b &= b - 1ull) {
        const int i = __ffsll(static_cast<long long>(b)) - 1;
        mine += at + 128 * (i >> 2) + (i & 3) < live;
      }
    }
    cta_prefix(mine, sh.warp_sum, total);
    holes = cluster_sum(cl, sh, turn++, total, before);
    if (rank == 0 && tid == 0) {
      *a.live_count = live;
      *a.pairs = holes;
    }
  } else {
    // the rows whose running need fits get theirs
    int lo = 0, n = rows + 1;  // the last place with need[place] <= free_pages
    while (n > 1) {
      const int h = n / 2;
      if (sh.need[lo + h] <= free_pages) {
        lo += h;
        n -= h;
      } else {
        n = h;
      }
    }
    given = sh.need[lo];
    if (rank == 0) {
      for (int r = tid; r < rows; r += kPcThreads) {
        const int need = sh.need[r + 1] - sh.need[r], first = sh.first[r];
        const bool ok = need == 0 || sh.need[r + 1] <= free_pages;
        if (!ok) flag_error(a.err, MSA_DEVERR_NO_PAGE);
        if (kOp == kExtend) {
          // (every CTA of the cluster has read the lengths: it met this one in cluster_sum)
          if (ok && first >= 0) {
            const int L = a.seq_lens_out[r];
            a.seq_lens_out[r] = L + (a.new_tokens != nullptr ? a.new_tokens[r] : L > 0 ? a.q_len : 0);
          }
        } else {
          const int p = a.parents[r];
          const int L = p >= 0 && p < a.batch ? a.seq_lens[p] : 0;
          const bool good = L >= 0 && L <= static_cast<int64_t>(a.max_blocks) * kBlock;
          a.seq_lens_out[r] = !good ? 0 : ok ? L : first * kBlock;
          const int place = need != 0 && ok ? sh.need[r] : -1;
          a.place[r] = place;
          if (place >= 0) {
            a.src[place] = a.block_table[static_cast<int64_t>(p) * a.max_blocks + first];
            a.tokens[place] = L % kBlock;
          }
        }
      }
      if (kOp == kFork && tid == 0) *a.pairs = given;
    }
  }

  // every page's rank among the free ones
  int base = 0;
  for (int round = 0; round < rounds; ++round) {
    const int iters = iters_of(round), at = first_of(round, iters);
    if (rounds > 1) bits = free_bits(a.refs_out, P, at, iters);
    const int own = __reduce_add_sync(0xffffffffu, __popcll(bits));
    int cta_before;
    const int in_cta = cta_prefix(lane == 0 ? own : 0, sh.warp_sum, total);
    const int all = cluster_sum(cl, sh, turn++, total, cta_before);
    int rank0 = base + cta_before + __shfl_sync(0xffffffffu, in_cta, 0);
    base += all;
    if (kOp != kCompact && rank0 >= given) continue;
    for (int i = 0; i < iters; ++i) {
      const unsigned b = static_cast<unsigned>(bits >> (4 * i)) & 15u;
      const unsigned below = (1u << lane) - 1u;
      int r = rank0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned m = __ballot_sync(0xffffffffu, b >> j & 1u);
        r += __popc(m & below);
        rank0 += __popc(m);
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
            } else {
              a.src[page - r - (live - holes)] = page;  // in use and below: page - r, of them below `live`: live - holes
            }
          }
        } else if (is_free && r < given) {
          const int row = row_of(sh.need, rows, r), first = sh.first[row];
          a.refs_out[page] = 1;
          if (kOp == kExtend)
            a.table_out[static_cast<int64_t>(row) * a.max_blocks + first + (r - sh.need[row])] = page;
          else
            a.dst[r] = page;
        }
        r += is_free;
      }
    }
  }
  if (kOp == kCompact) {
    cl.sync();  // the lists are whole
    for (int i = rank * kPcThreads + tid; i < holes; i += kPcCtas * kPcThreads) {
      const int from = __ldcg(a.src + i), to = __ldcg(a.dst + i);
      a.page_map[from] = to;
      a.refs_out[to] = a.refs_out[from];
      a.refs_out[from] = 0;
    }
  }
  cl.sync();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------- rows of tables, pages

// Buffers of one launch, cut into runs (of which a fork copies the first tokens) and these into chunks.
constexpr int kPageBuffers = 64, kPageChunk = 16384;
struct PageBuffers {
  struct {
    char* data;
    int64_t page_bytes;
    int32_t run_bytes, token_bytes;  // token_bytes 0: whole runs
    int32_t chunks;                  // of a run
    int32_t end;                     // chunks of a page in this buffer and those before it
  } buf[kPageBuffers];
  int32_t count;
};

// n bytes; both addresses have the same place within 16 bytes, or are copied byte by byte.
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

// Rows: fork, table_out and the references of the full blocks; compact, the renamed table.  Then the pages.
template <PageOp kOp>
__global__ void __launch_bounds__(256) page_move_kernel(const PageArgs a, const __grid_constant__ PageBuffers bufs, int rows_too) {
  grid_dependency_wait();
  grid_dependents_launch();
  if (rows_too) {
    const int rows = kOp == kFork ? a.children : a.batch;
    const int64_t all = static_cast<int64_t>(rows) * a.max_blocks, room = static_cast<int64_t>(a.max_blocks) * kBlock;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all; i += static_cast<int64_t>(gridDim.x) * 256) {
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
          if (page >= 0 && page < a.num_pages) out = a.page_map[page];
          if (out < 0 && page != -1) flag_error(a.err, MSA_DEVERR_BAD_PAGE);
        }
      }
      a.table_out[i] = out;
    }
  }
  if (bufs.count == 0) return;
  const int per_page = bufs.buf[bufs.count - 1].end;
  const int64_t items = static_cast<int64_t>(*a.pairs) * per_page;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int pair = static_cast<int>(it / per_page), c = static_cast<int>(it - static_cast<int64_t>(pair) * per_page);
    int k = 0;
    while (c >= bufs.buf[k].end) ++k;
    const auto& b = bufs.buf[k];
    const int at = c - (k > 0 ? bufs.buf[k - 1].end : 0), run = at / b.chunks, lo = (at - run * b.chunks) * kPageChunk;
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
  const int64_t all = static_cast<int64_t>(a.rows) * a.width;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int r = static_cast<int>(i / a.width), n = static_cast<int>(i - static_cast<int64_t>(r) * a.width);
    if (a.counts != nullptr) {
      const int c = a.counts[r];
      if (c < 0 || c > a.width) {
        if (n == 0) flag_error(a.err, MSA_DEVERR_BAD_SEQLEN);
        continue;
      }
      if (n >= c) continue;
    }
    const int page = a.pages[i];
    if (page == -1) continue;
    if (page < 0 || page >= a.num_pages) {
      flag_error(a.err, MSA_DEVERR_BAD_PAGE);
    } else if (atomicSub(a.refs_out + page, 1) <= 0) {
      atomicAdd(a.refs_out + page, 1);
      flag_error(a.err, MSA_DEVERR_BAD_PAGE);
    }
  }
}

// ---------------------------------------------------------------- launches

static unsigned grid_of(int64_t threads, int num_sms) {
  const int64_t ctas = (threads + 255) / 256, most = static_cast<int64_t>(num_sms) * 8;
  return static_cast<unsigned>(ctas < 1 ? 1 : ctas < most ? ctas : most);
}

static cudaError_t copy_words(const PageCopies& c, int num_sms, cudaStream_t s) {
  const int64_t all = c.words[0] + c.words[1] + c.words[2];
  return all == 0 ? cudaSuccess : launch_dependent(page_words_kernel, dim3(grid_of(all / 4 + 1, num_sms)), 256, 0, s, c);
}

static cudaError_t copy_refs(const PageArgs& a, int num_sms, cudaStream_t s) {
  PageCopies c{};
  if (a.refs != a.refs_out) c = PageCopies{{a.refs}, {a.refs_out}, {a.num_pages}};
  return copy_words(c, num_sms, s);
}

template <PageOp kOp>
static cudaError_t launch_move(const PageArgs& a, int64_t most_pairs, int num_sms, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(kOp == kFork ? a.children : a.batch) * a.max_blocks;
  int k = 0;
  do {
    PageBuffers b;
    b.count = 0;
    for (; k < a.num_buffers && b.count < kPageBuffers; ++k) {
      auto& x = b.buf[b.count];
      x.data = static_cast<char*>(a.buffers[k].data);
      x.page_bytes = a.buffers[k].page_bytes;
      x.token_bytes = a.buffers[k].token_bytes;
      const bool runs = kOp == kFork && x.token_bytes > 0;
      x.run_bytes = runs ? x.token_bytes * kBlock : static_cast<int32_t>(x.page_bytes);
      x.chunks = (x.run_bytes + kPageChunk - 1) / kPageChunk;
      x.end = (b.count > 0 ? b.buf[b.count - 1].end : 0) + static_cast<int32_t>(x.page_bytes / x.run_bytes) * x.chunks;
      ++b.count;
    }
    const bool first = k <= kPageBuffers;
    const int64_t items = b.count > 0 ? most_pairs * b.buf[b.count - 1].end : 0;
    const int64_t work = items * 256 > (first ? rows : 0) ? items * 256 : rows;
    const cudaError_t e = launch_dependent(page_move_kernel<kOp>, dim3(grid_of(work, num_sms)), 256, 0, s, a, b, first ? 1 : 0);
    if (e != cudaSuccess) return e;
  } while (k < a.num_buffers);
  return cudaSuccess;
}

cudaError_t launch_extend_pages(const PageArgs& a, int num_sms, cudaStream_t s) {
  PageCopies c{};
  if (a.refs != a.refs_out) {
    c.src[0] = a.refs, c.dst[0] = a.refs_out, c.words[0] = a.num_pages;
  }
  if (a.block_table != a.table_out) {
    c.src[1] = a.block_table, c.dst[1] = a.table_out, c.words[1] = static_cast<int64_t>(a.batch) * a.max_blocks;
  }
  if (a.seq_lens != a.seq_lens_out) {
    c.src[2] = a.seq_lens, c.dst[2] = a.seq_lens_out, c.words[2] = a.batch;
  }
  cudaError_t e = copy_words(c, num_sms, s);
  if (e != cudaSuccess) return e;
  PageArgs x = a;
  x.seq_lens = a.seq_lens_out;
  return launch_dependent(page_scan_kernel<kExtend>, dim3(kPcCtas), kPcThreads, 0, s, x);
}

cudaError_t launch_fork_pages(const PageArgs& a, int num_sms, cudaStream_t s) {
  cudaError_t e = copy_refs(a, num_sms, s);
  if (e != cudaSuccess) return e;
  if ((e = launch_dependent(page_scan_kernel<kFork>, dim3(kPcCtas), kPcThreads, 0, s, a)) != cudaSuccess) return e;
  return launch_move<kFork>(a, a.children, num_sms, s);
}

cudaError_t launch_free_pages(const PageArgs& a, int num_sms, cudaStream_t s) {
  const cudaError_t e = copy_refs(a, num_sms, s);
  if (e != cudaSuccess) return e;
  return launch_dependent(page_free_kernel, dim3(grid_of(static_cast<int64_t>(a.rows) * a.width, num_sms)), 256, 0, s, a);
}

cudaError_t launch_compact_pages(const PageArgs& a, int num_sms, cudaStream_t s) {
  cudaError_t e = copy_refs(a, num_sms, s);
  if (e != cudaSuccess) return e;
  if ((e = launch_dependent(page_scan_kernel<kCompact>, dim3(kPcCtas), kPcThreads, 0, s, a)) != cudaSuccess) return e;
  return launch_move<kCompact>(a, a.num_pages / 2, num_sms, s);
}

}  // namespace msa
