// C ABI of the FP8 page cache: host-side validation, workspace layout and dispatch of
// msa_fp8_append, msa_fp8_attn and msa_evict_blocks (documented in include/msa.h).
#include <cmath>
#include <cstdint>

#include "../../include/msa.h"
#include "api_internal.h"
#include "fp8_kernels.h"
#include "msa_kernels.h"

using namespace msa;

namespace {

msa_status_t check_fp8_cache(const msa_fp8_cache_t* c) {
  if (c == nullptr || c->num_pages < 1 || c->num_pages > INT32_MAX) return MSA_ERR_INVALID_ARG;
  if (c->k_data == nullptr || c->k_scale == nullptr || c->v_data == nullptr || c->v_scale == nullptr ||
      !aligned16(c->k_data) || !aligned16(c->v_data))
    return MSA_ERR_INVALID_ARG;
  return MSA_OK;
}

// token-strided rows: pointer and stride on 16-byte boundaries, tokens not overlapping
bool rows_ok(const void* p, int64_t stride, int64_t width, int elem) {
  return p != nullptr && aligned16(p) && stride >= width && stride <= (int64_t{1} << 40) && stride * elem % 16 == 0;
}

bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}

msa_status_t status_of(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

struct AttnLayout {
  size_t prefix, partial, share, stat, mass, total;
};

AttnLayout attn_layout(const msa_config_t* c, const msa_batch_t* b, bool weights) {
  AttnLayout w{};
  const int64_t rows = static_cast<int64_t>(b->q_len) * c->heads_per_group;  // per (sequence, group)
  w.prefix = kErrBytes;
  w.partial = w.prefix + align_up((static_cast<size_t>(b->batch) * fp8_tile_units_per_seq(rows) + 1) * sizeof(int32_t));
  w.total = w.partial + align_up(fp8_attn_partial_bytes(rows));
  if (!weights) return w;
  const size_t all = static_cast<size_t>(b->batch) * c->num_kv_groups * rows;
  // shares of a row: the streaming form keeps the parts of a page apart (dense, or of the 16 selected ones), the
  // tile form does not
  const size_t dense = static_cast<size_t>(b->max_blocks) * (rows <= kFp8StreamRows ? kFp8StreamParts : 1);
  const size_t sparse = static_cast<size_t>(kSelTopK) * kFp8StreamParts;
  w.share = w.total;
  w.stat = w.share + align_up(all * (dense > sparse ? dense : sparse) * sizeof(float2));
  w.mass = w.stat + align_up(all * sizeof(float2));
  w.total = w.mass + align_up(static_cast<size_t>(b->batch) * b->max_blocks * sizeof(unsigned long long));
  return w;
}

}  // namespace

size_t msa::fp8_attn_workspace_bytes(const msa_config_t* cfg, const msa_batch_t* batch, bool weights) {
  return attn_layout(cfg, batch, weights).total;
}

extern "C" {

msa_status_t msa_fp8_append(const msa_config_t* cfg, const msa_fp8_cache_t* cache, const msa_batch_t* batch,
                            const void* k, const void* v, int32_t x_type, int64_t k_stride, int64_t v_stride,
                            void* workspace, size_t workspace_bytes, void* stream) {
  msa_status_t st;
  if ((st = check_config(cfg)) != MSA_OK || (st = check_batch(batch)) != MSA_OK ||
      (st = check_fp8_cache(cache)) != MSA_OK)
    return st;
  if (x_type != MSA_TYPE_F32 && x_type != MSA_TYPE_BF16) return MSA_ERR_UNSUPPORTED;
  if (batch->batch == 0) return MSA_OK;
  const int elem = x_type == MSA_TYPE_BF16 ? 2 : 4;
  const int64_t width = static_cast<int64_t>(cfg->num_kv_groups) * cfg->head_dim;
  if (!rows_ok(k, k_stride, width, elem) || !rows_ok(v, v_stride, width, elem)) return MSA_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < kErrBytes || !aligned16(workspace)) return MSA_ERR_WORKSPACE;
  Fp8AppendArgs a{};
  a.data[0] = cache->k_data;
  a.data[1] = cache->v_data;
  a.scale[0] = cache->k_scale;
  a.scale[1] = cache->v_scale;
  a.x[0] = k;
  a.x[1] = v;
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.num_pages = cache->num_pages;
  a.block_table = batch->block_table;
  a.seq_lens = batch->seq_lens;
  a.batch = batch->batch;
  a.max_blocks = batch->max_blocks;
  a.q_len = batch->q_len;
  a.groups = cfg->num_kv_groups;
  a.bf16 = x_type == MSA_TYPE_BF16;
  a.err = static_cast<uint32_t*>(workspace);
  return status_of(launch_fp8_append(a, static_cast<cudaStream_t>(stream)));
}

msa_status_t msa_fp8_attn(const msa_config_t* cfg, const msa_fp8_cache_t* cache, const msa_batch_t* batch,
                          const void* q, int32_t q_type, int64_t q_stride, const int32_t* selection, uint16_t* out,
                          float* lse, const float* weight_in, float weight_decay, float* weight_out, void* workspace,
                          size_t workspace_bytes, void* stream) {
  msa_status_t st;
  if ((st = check_config(cfg)) != MSA_OK || (st = check_batch(batch)) != MSA_OK ||
      (st = check_fp8_cache(cache)) != MSA_OK)
    return st;
  if (q_type != MSA_TYPE_E4M3 && q_type != MSA_TYPE_BF16) return MSA_ERR_UNSUPPORTED;
  if (cache->num_pages * cfg->num_kv_groups > (1 << 24)) return MSA_ERR_UNSUPPORTED;
  // the flat list of (unit, page) steps is counted in 32 bits
  const int64_t tiles = 2 * static_cast<int64_t>(fp8_tile_units_per_seq(static_cast<int64_t>(batch->q_len) * cfg->heads_per_group));
  if (batch->batch * tiles > INT32_MAX / (static_cast<int64_t>(batch->max_blocks) * cfg->num_kv_groups))
    return MSA_ERR_UNSUPPORTED;
  if (!(weight_decay >= 0.0f && weight_decay <= 1.0f) || (weight_in != nullptr && weight_out == nullptr))
    return MSA_ERR_INVALID_ARG;
  if (batch->batch == 0) return MSA_OK;
  const int64_t width = static_cast<int64_t>(cfg->num_kv_groups) * cfg->heads_per_group * cfg->head_dim;
  if (!rows_ok(q, q_stride, width, q_type == MSA_TYPE_BF16 ? 2 : 1) || out == nullptr || !aligned16(out))
    return MSA_ERR_INVALID_ARG;
  const size_t table = static_cast<size_t>(batch->batch) * batch->max_blocks * sizeof(float);
  if (weight_in != nullptr && weight_in != weight_out && overlap(weight_in, table, weight_out, table))
    return MSA_ERR_INVALID_ARG;
  const AttnLayout w = attn_layout(cfg, batch, weight_out != nullptr);
  if (workspace == nullptr || workspace_bytes < w.total || !aligned16(workspace)) return MSA_ERR_WORKSPACE;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return MSA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Fp8AttnArgs a{};
  a.k_data = cache->k_data;
  a.k_scale = cache->k_scale;
  a.v_data = cache->v_data;
  a.v_scale = cache->v_scale;
  a.num_pages = cache->num_pages;
  a.block_table = batch->block_table;
  a.seq_lens = batch->seq_lens;
  a.batch = batch->batch;
  a.max_blocks = batch->max_blocks;
  a.q_len = batch->q_len;
  a.groups = cfg->num_kv_groups;
  a.heads_per_group = cfg->heads_per_group;
  a.q = q;
  a.q_stride = q_stride;
  a.q_bf16 = q_type == MSA_TYPE_BF16;
  a.selection = selection;
  a.out = out;
  a.lse = lse;
  a.scale_log2 = scale_log2(cfg);
  a.err = reinterpret_cast<uint32_t*>(ws);
  a.weight_in = weight_in;
  a.weight_decay = weight_decay;
  a.weight_out = weight_out;
  a.block_prefix = reinterpret_cast<int32_t*>(ws + w.prefix);
  a.partial = reinterpret_cast<float*>(ws + w.partial);
  if (weight_out != nullptr) {
    a.share = reinterpret_cast<float2*>(ws + w.share);
    a.row_stat = reinterpret_cast<float2*>(ws + w.stat);
    a.mass = reinterpret_cast<unsigned long long*>(ws + w.mass);
  }
  try {  // (the launch's bookkeeping allocates host memory: nothing may leave a C entry)
    return status_of(launch_fp8_attn(a, sms, static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return MSA_ERR_CUDA;
  }
}

msa_status_t msa_evict_blocks(const msa_batch_t* batch, const float* weight, int32_t budget, int32_t keep_first,
                              int32_t keep_last, int32_t* table_out, int32_t* seq_lens_out, float* weight_out,
                              int32_t* freed, int32_t* freed_count, void* workspace, size_t workspace_bytes,
                              void* stream) {
  msa_status_t st;
  if ((st = check_batch(batch)) != MSA_OK) return st;
  if (keep_first < 0 || keep_last < 1 || static_cast<int64_t>(keep_first) + keep_last > budget)
    return MSA_ERR_INVALID_ARG;
  if (batch->batch == 0) return MSA_OK;
  if (weight == nullptr || table_out == nullptr || seq_lens_out == nullptr || weight_out == nullptr ||
      freed == nullptr || freed_count == nullptr)
    return MSA_ERR_INVALID_ARG;
  // each output may be its own input, and nothing else may overlap
  const size_t row = static_cast<size_t>(batch->batch) * 4, table = row * batch->max_blocks;
  const struct { const void* p; size_t n; } x[8] = {
      {batch->block_table, table}, {batch->seq_lens, row}, {weight, table},        {table_out, table},
      {seq_lens_out, row},         {weight_out, table},    {freed, table},         {freed_count, row}};
  for (int i = 0; i < 8; ++i)
    for (int j = i + 1; j < 8; ++j) {
      const bool own = i < 3 && j == i + 3 && x[i].p == x[j].p;
      if ((i >= 3 || j >= 3) && !own && overlap(x[i].p, x[i].n, x[j].p, x[j].n)) return MSA_ERR_INVALID_ARG;
    }
  if (workspace == nullptr || workspace_bytes < kErrBytes || !aligned16(workspace)) return MSA_ERR_WORKSPACE;
  const EvictArgs a{batch->block_table, batch->seq_lens, weight,     batch->batch, batch->max_blocks, budget,
                    keep_first,         keep_last,       table_out,  seq_lens_out, weight_out,        freed,
                    freed_count,        static_cast<uint32_t*>(workspace)};
  return status_of(launch_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
