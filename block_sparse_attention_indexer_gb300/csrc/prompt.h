// Kernel arguments and launcher of the packed prompt attention, shared between the C-ABI layer
// (api_prompt.cu) and prompt_attn.cu.  Every pointer is device memory.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace msa {

struct PtCut;

struct PromptArgs {
  const int32_t* cu_q;  // [batch + 1]
  const int32_t* cu_k;
  int32_t batch, q_tokens, k_tokens, groups, heads_per_group;
  const uint16_t* q;    // bf16 [q_tokens][G * Hg][128], tokens q_stride elements apart
  const uint16_t* k;    // bf16 [k_tokens][G][128]
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;
  uint16_t* out;        // bf16 [q_tokens][G * Hg][128]
  float* lse;           // [q_tokens][G * Hg] or null
  float scale_log2;     // softmax_scale * log2(e)
  uint32_t* err;
  // scratch
  int32_t* plan;        // [0]: units and how they are spread (where a launch of its own makes the plan)
  int32_t* base;        // [batch + 1]: units of the sequences before each
  int32_t* prefix;      // [units + 1]: cost (per KV head) of the units before each
  int32_t* order;       // [kPromptSpreadUnits]: the units by falling cost
  int2* dealt;          // [CTAs][...]: each CTA's units, where they stay whole
  PtCut* cuts;   // [CTAs]: the unit inside which each CTA's range starts
  float* row_max;       // [CTAs][2][two tiles]: M of the rows of each CTA's last two units
  float* partial;       // partial softmax states of units cut by the split of the work
};

// What the start of a unit counts in the split of the work, in (tile, 128 keys) steps.
constexpr int kPromptUnitCost = 4;
// Units (of a KV head) up to which the plan puts them in order of cost.
constexpr int kPromptSpreadUnits = 2048;
// Query tokens of a tile of 128 rows (token, head), and of a unit of two tiles.
inline int prompt_tile_tokens(int heads_per_group) { return 128 / heads_per_group; }
// At least as many units as the packed sequences have.
inline int64_t prompt_max_units(int64_t q_tokens, int batch, int heads_per_group) {
  return q_tokens / (2 * prompt_tile_tokens(heads_per_group)) + batch;
}
size_t prompt_dealt_bytes();
size_t prompt_cut_bytes();
size_t prompt_row_max_bytes();
size_t prompt_partial_bytes();
cudaError_t launch_prompt_attn(const PromptArgs& a, int num_sms, cudaStream_t s);

}  // namespace msa
