// Kernel argument blocks and launchers of the FP8 page cache (append, attention, eviction),
// shared between the C-ABI layer (api_fp8.cu) and the kernel translation units.  Every
// pointer is device memory.
#pragma once

#include <cuda.h>
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
  int32_t* block_prefix;       // dense, prefix sums of the work: [B + 1] blocks of the sequences before each
                               // (streaming form), [B * tile units + 1] steps of the units before each (tile form)
  float* partial;              // partial softmax states of units cut by the split of the work
  float2* share;               // [unit][page place][part][row]: (sum of 2^(z - ref), ref) over the
                               // keys of a part of the page; places: block (dense) or slot (sparse)
  float2* row_stat;            // [unit][row]: (M, 1 / sum of 2^(z - M)); 0 weight for empty rows
  unsigned long long* mass;    // [B][max_blocks] fixed point (sparse)
};
// Query rows of a unit up to which the streaming (mma.sync) form takes it; sparse units
// (at most 8 rows) always fit.
constexpr int kFp8StreamRows = 16;
// Parts of a page whose shares are kept apart.
constexpr int kFp8StreamParts = 4;
// Upper bound of the persistent grids (one CTA per SM); `partial` is sized for it.
constexpr int kFp8MaxCtas = 160;
// Bytes of `partial` for a batch with `rows` = q_len * heads_per_group rows per dense unit.
size_t fp8_attn_partial_bytes(int64_t rows);
cudaError_t launch_fp8_attn(const Fp8AttnArgs& a, int num_sms, cudaStream_t s);
// The streaming form: dense units of at most kFp8StreamRows rows, or a selection.
cudaError_t launch_fp8_stream(const Fp8AttnArgs& a, int num_sms, cudaStream_t s);
size_t fp8_stream_partial_bytes();
// The tile form: dense units of any number of rows.
cudaError_t launch_fp8_tile(const Fp8AttnArgs& a, int num_sms, cudaStream_t s);
size_t fp8_tile_partial_bytes();
int fp8_tile_units_per_seq(int64_t rows);

// Tensor maps of the K and V code pools as rows of 128 bytes ([pages * G * 128][128]), one page
// head (128 rows) per box, 128-byte swizzle.
struct Fp8Maps {
  CUtensorMap k, v;
};
cudaError_t fp8_page_maps(const Fp8AttnArgs& a, Fp8Maps* maps);

// Launch with programmatic stream serialization (every kernel here waits for the one before it).
template <typename... Par, typename... Arg>
cudaError_t launch_dependent(void (*kernel)(Par...), dim3 grid, int block, size_t smem, cudaStream_t s,
                             const Arg&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

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
