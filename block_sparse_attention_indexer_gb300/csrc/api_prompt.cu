// C ABI of the packed prompt attention: host-side validation, workspace layout and dispatch of
// msa_prompt_attn (documented in include/msa.h).
#include <cstdint>

#include "../../include/msa.h"
#include "api_internal.h"
#include "msa_kernels.h"
#include "prompt.h"

using namespace msa;

namespace {

constexpr int64_t kMaxTokens = int64_t{1} << 28;

msa_status_t check_packed(const msa_config_t* c, const msa_packed_t* p) {
  if (p == nullptr || p->batch < 0 || p->q_tokens < 0 || p->k_tokens < 0) return MSA_ERR_INVALID_ARG;
  if (p->batch > 0 && (p->cu_q == nullptr || p->cu_k == nullptr)) return MSA_ERR_INVALID_ARG;
  if (p->batch > kMaxBatchSmem || p->q_tokens > kMaxTokens || p->k_tokens > kMaxTokens) return MSA_ERR_UNSUPPORTED;
  // the units' cost is counted in 32 bits
  const int64_t blocks = (p->k_tokens + 127) / 128;
  if (prompt_max_units(p->q_tokens, p->batch, c->heads_per_group) * (2 * (blocks > 1 ? blocks : 1) + kPromptUnitCost) >
      INT32_MAX / c->num_kv_groups)
    return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

struct PromptLayout {
  size_t plan, base, order, dealt, prefix, cuts, row_max, partial, total;
};
PromptLayout prompt_layout(const msa_config_t* c, const msa_packed_t* p) {
  PromptLayout w;
  w.plan = kErrBytes;
  w.base = w.plan + kWsAlign;
  w.order = w.base + align_up((static_cast<size_t>(p->batch) + 1) * sizeof(int32_t));
  w.dealt = w.order + align_up(kPromptSpreadUnits * sizeof(int32_t));
  w.prefix = w.dealt + align_up(prompt_dealt_bytes());
  w.cuts = w.prefix + align_up((prompt_max_units(p->q_tokens, p->batch, c->heads_per_group) + 1) * sizeof(int32_t));
  w.row_max = w.cuts + align_up(prompt_cut_bytes());
  w.partial = w.row_max + align_up(prompt_row_max_bytes());
  w.total = w.partial + align_up(prompt_partial_bytes());
  return w;
}

// token-strided bf16 rows: pointer and stride on 16-byte boundaries, tokens not overlapping
bool rows_ok(const void* p, int64_t tokens, int64_t stride, int64_t width) {
  return (p != nullptr || tokens == 0) && aligned16(p) && stride >= width && stride <= (int64_t{1} << 37) && stride % 8 == 0;
}

bool overlap(const void* p, int64_t np, const void* q, int64_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return np > 0 && nq > 0 && a < b + static_cast<uintptr_t>(nq) && b < a + static_cast<uintptr_t>(np);
}

}  // namespace

extern "C" {

size_t msa_prompt_workspace_bytes(const msa_config_t* cfg, const msa_packed_t* packed) {
  if (check_config(cfg) != MSA_OK || check_packed(cfg, packed) != MSA_OK) return 0;
  return prompt_layout(cfg, packed).total;
}

msa_status_t msa_prompt_attn(const msa_config_t* cfg, const msa_packed_t* packed, const void* q, int64_t q_stride,
                             const void* k, int64_t k_stride, const void* v, int64_t v_stride, uint16_t* out,
                             float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  msa_status_t st;
  if ((st = check_config(cfg)) != MSA_OK || (st = check_packed(cfg, packed)) != MSA_OK) return st;
  const int64_t Nq = packed->q_tokens, Nk = packed->k_tokens;
  if (packed->batch == 0 || Nq == 0) return MSA_OK;
  const int64_t H = static_cast<int64_t>(cfg->num_kv_groups) * cfg->heads_per_group, D = cfg->head_dim;
  const int64_t qw = H * D, kw = cfg->num_kv_groups * D;
  if (!rows_ok(q, Nq, q_stride, qw) || !rows_ok(k, Nk, k_stride, kw) || !rows_ok(v, Nk, v_stride, kw) || out == nullptr ||
      !aligned16(out))
    return MSA_ERR_INVALID_ARG;
  const int64_t size = Nq * qw * 2, stats = lse != nullptr ? Nq * H * 4 : 0;
  const struct { const void* p; int64_t n; } in[3] = {{q, ((Nq - 1) * q_stride + qw) * 2},
                                                       {k, Nk > 0 ? ((Nk - 1) * k_stride + kw) * 2 : 0},
                                                       {v, Nk > 0 ? ((Nk - 1) * v_stride + kw) * 2 : 0}};
  for (const auto& x : in)
    if (overlap(out, size, x.p, x.n) || overlap(lse, stats, x.p, x.n)) return MSA_ERR_INVALID_ARG;
  if (overlap(out, size, lse, stats)) return MSA_ERR_INVALID_ARG;
  const PromptLayout w = prompt_layout(cfg, packed);
  if (workspace == nullptr || workspace_bytes < w.total || !aligned16(workspace)) return MSA_ERR_WORKSPACE;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return MSA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PromptArgs a{};
  a.cu_q = packed->cu_q;
  a.cu_k = packed->cu_k;
  a.batch = packed->batch;
  a.q_tokens = static_cast<int32_t>(Nq);
  a.k_tokens = static_cast<int32_t>(Nk);
  a.groups = cfg->num_kv_groups;
  a.heads_per_group = cfg->heads_per_group;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.out = out;
  a.lse = lse;
  a.scale_log2 = scale_log2(cfg);
  a.err = reinterpret_cast<uint32_t*>(ws);
  a.plan = reinterpret_cast<int32_t*>(ws + w.plan);
  a.base = reinterpret_cast<int32_t*>(ws + w.base);
  a.prefix = reinterpret_cast<int32_t*>(ws + w.prefix);
  a.order = reinterpret_cast<int32_t*>(ws + w.order);
  a.dealt = reinterpret_cast<int2*>(ws + w.dealt);
  a.cuts = reinterpret_cast<PtCut*>(ws + w.cuts);
  a.row_max = reinterpret_cast<float*>(ws + w.row_max);
  a.partial = reinterpret_cast<float*>(ws + w.partial);
  try {  // (the launch's bookkeeping allocates host memory: nothing may leave a C entry)
    return launch_prompt_attn(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
  } catch (...) {
    return MSA_ERR_CUDA;
  }
}

}  // extern "C"
