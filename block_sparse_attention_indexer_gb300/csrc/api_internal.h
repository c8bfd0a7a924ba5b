// Host functions shared between the C-ABI translation units (api.cu, api_fp8.cu, noalloc.cu);
// not exported.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/msa.h"

namespace msa {

constexpr size_t kWsAlign = 256;
constexpr size_t kErrBytes = 256;  // error word + padding
inline size_t align_up(size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

msa_status_t check_config(const msa_config_t* c);
msa_status_t check_batch(const msa_batch_t* b);
int num_sms_of_current_device();           // <= 0: the query failed
float scale_log2(const msa_config_t* c);   // softmax_scale (or its default) * log2(e)

// Bytes of msa_fp8_attn's workspace, with or without the collected block weights.
size_t fp8_attn_workspace_bytes(const msa_config_t* cfg, const msa_batch_t* batch, bool weights);

// Bytes the query-major team attention needs (error word + its partial-state slots): the
// scratch of the no-allocation entry point, whatever the batch.
size_t team_attn_workspace_bytes();

// msa_sparse_attn_decode, with the block-major form of long query chunks allowed or not (the
// no-allocation entry point's fixed scratch holds only the team kernel's states).  With
// clear_error, the device error word is zeroed on the stream once every argument has passed
// validation, right before the launch (a rejected call touches nothing).
msa_status_t sparse_attn_entry(const msa_config_t* cfg, const msa_cache_t* cache, const msa_batch_t* batch,
                               const uint8_t* q, const int32_t* selection, uint16_t* out, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream, bool block_major_ok,
                               bool clear_error);

}  // namespace msa
