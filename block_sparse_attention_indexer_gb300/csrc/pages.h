// Kernel argument blocks and launchers of the page pool (extend, fork, free, compact), shared
// between the C-ABI layer (api_pages.cu) and pages.cu.  Every pointer is device memory unless
// it says otherwise.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/msa.h"

namespace msa {

// Rows whose needs a CTA sums: sequences of a call, children of a fork.
constexpr int kPageRows = 2048;
// Pages whose counts a CTA takes.
constexpr int kPageChunkPages = 2048;

struct PageArgs {
  const int32_t* refs;      // [num_pages] (or refs_out itself)
  int32_t* refs_out;
  int32_t num_pages;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int32_t batch, max_blocks, q_len;
  const int32_t* new_tokens;  // extend: [batch] or null
  const int32_t* parents;     // fork: [children]
  int32_t children;
  int32_t* table_out;
  int32_t* seq_lens_out;
  const int32_t* pages;       // free: [rows][width]
  const int32_t* counts;      // free: [rows] or null
  int32_t rows, width;
  int32_t* page_map;          // compact
  int32_t* live_count;
  // scratch.  Free pages of each chunk; extend, fork: pages that the rows before each need, and first blocks; fork,
  // compact: pages to copy, from, to, and how many tokens of each (fork); their number; fork: the child's place
  // among them, or -1
  int32_t* counts_free;
  int32_t* need;
  int32_t* first;
  int32_t* src;
  int32_t* dst;
  int32_t* tokens;
  int32_t* pairs;
  int32_t* place;
  uint32_t* err;
  const msa_page_buffer_t* buffers;  // host
  int32_t num_buffers;
};

cudaError_t launch_extend_pages(const PageArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_fork_pages(const PageArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_free_pages(const PageArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_compact_pages(const PageArgs& a, int num_sms, cudaStream_t s);

}  // namespace msa
