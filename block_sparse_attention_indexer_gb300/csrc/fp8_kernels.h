// Kernel argument blocks and launchers of the FP8 page cache (append, attention, eviction),
// shared between the C-ABI layer (api_fp8.cu) and the kernel translation units.  Every
// pointer is device memory.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/msa.h"

namespace msa {

constexpr int kFp8PageBytes = 128 * 128;  // K or V codes of one page and KV head

struct Fp8AppendArgs {
  uint8_t* data[2];      // K, V pools [P][G][128][128]
  uint8_t* scale[2];     // [P][G]
  const void* x[2];      // K, V rows
  int64_t stride[2];     // elements between tokens
  int64_t num_pages;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int32_t batch, max_blocks, q_len, groups;
  int32_t bf16;          // element type of x: 1 bfloat16, 0 float32
  uint32_t* err;
};
cudaError_t launch_fp8_append(const Fp8AppendArgs& a, cudaStream_t s);

struct Fp8AttnArgs {
  const uint8_t* k_data;       // [P][G][128][128] E4M3
  const uint8_t* k_scale;      // [P][G] E8M0
  const uint8_t* v_data;
  const uint8_t* v_scale;
  int64_t num_pages;
  const int32_t* block_table;  // [B][max_blocks]
  const int32_t* seq_lens;     // [B]
  int32_t batch, max_blocks, q_len, groups, heads_per_group;
  const void* q;               // [B][T][H][128] E4M3 or bf16, tokens q_stride elements apart
  int64_t q_stride;
  int32_t q_bf16;
  const int32_t* selection;    // [B][T][G][16], or null: dense causal
  uint16_t* out;               // [B][T][H][128] bf16
  float* lse;                  // [B][T][H] or null
  float scale_log2;            // softmax_scale * log2(e)
  uint32_t* err;
  // collected block weights (weight_out null: none wanted)
  const float* weight_in;      // [B][max_blocks] or null
  float weight_decay;
  float* weight_out;
  // Scratch.  A unit is the query rows that share a list of pages: dense, the T * Hg rows
  // (t, h) of (sequence, group); sparse, the Hg heads of (sequence, token, group).
  float* partial;              // partial softmax states of units cut by the split of the work
  float2* share;               // [unit][page place][part][row]: (sum of 2^(z - ref), ref) over the
                               // keys of a part of the page; places: block (dense) or slot (sparse)
  float2* row_stat;            // [unit][row]: (M, 1 / sum of 2^(z - M)); 0 weight for empty rows
  unsigned long long* mass;    // [B][max_blocks] fixed point (sparse)
};
// Bytes of `partial`, whatever the batch.
size_t fp8_attn_partial_bytes();
cudaError_t launch_fp8_attn(const Fp8AttnArgs& a, int num_sms, cudaStream_t s);

struct EvictArgs {
  const int32_t* block_table;
  const int32_t* seq_lens;
  const float* weight;
  int32_t batch, max_blocks, budget, keep_first, keep_last;
  int32_t* table_out;
  int32_t* seq_lens_out;
  float* weight_out;
  int32_t* freed;
  int32_t* freed_count;
  uint32_t* err;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s);

}  // namespace msa
