// C ABI of the page pool: host-side validation, workspace layout and dispatch of
// msa_extend_pages, msa_fork_pages, msa_free_pages and msa_compact_pages (documented in include/msa.h).
#include <cstdint>

#include "../../include/msa.h"
#include "api_internal.h"
#include "pages.h"

using namespace msa;

namespace {

constexpr int64_t kMaxPages = int64_t{1} << 27;
constexpr int kMaxBuffers = 4096;

msa_status_t check_pool(const msa_page_pool_t* p) {
  if (p == nullptr || p->num_pages < 1 || p->num_pages > kMaxPages || p->num_buffers < 0) return MSA_ERR_INVALID_ARG;
  if (p->num_buffers > kMaxBuffers) return MSA_ERR_UNSUPPORTED;
  if (p->refs == nullptr || p->refs_out == nullptr || !aligned16(p->refs) || !aligned16(p->refs_out))
    return MSA_ERR_INVALID_ARG;
  if (p->num_buffers > 0 && p->buffers == nullptr) return MSA_ERR_INVALID_ARG;
  for (int i = 0; i < p->num_buffers; ++i) {
    const msa_page_buffer_t& b = p->buffers[i];
    if (b.data == nullptr || b.page_bytes < 1 || b.page_bytes > INT32_MAX || b.token_bytes < 0) return MSA_ERR_INVALID_ARG;
    if (b.token_bytes > 0 && b.page_bytes % (int64_t{128} * b.token_bytes) != 0) return MSA_ERR_INVALID_ARG;
  }
  return MSA_OK;
}

struct Range {
  const void* p;
  size_t n;
};
// Whether two ranges overlap, an array on itself left aside.
bool clash(const Range& x, const Range& y, bool own) {
  if (x.p == nullptr || y.p == nullptr || x.n == 0 || y.n == 0 || (own && x.p == y.p)) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return a < b + y.n && b < a + x.n;
}
// in[i] may be out[i] where `own`; an output may overlap nothing else.
template <int kIn, int kOut>
bool arrays_ok(const Range (&in)[kIn], const Range (&out)[kOut], const bool (&own)[kOut]) {
  for (int i = 0; i < kOut; ++i) {
    for (int j = 0; j < kIn; ++j)
      if (clash(out[i], in[j], own[i] && i == j)) return false;
    for (int j = i + 1; j < kOut; ++j)
      if (clash(out[i], out[j], false)) return false;
  }
  return true;
}

struct PageLayout {
  size_t pairs, counts, need, first, src, dst, tokens, place, total;
};
PageLayout page_layout(int64_t pages, int64_t rows) {
  PageLayout w;
  const size_t pairs = align_up(static_cast<size_t>(pages / 2 > rows ? pages / 2 : rows) * sizeof(int32_t));
  const size_t row = align_up(static_cast<size_t>(rows + 1) * sizeof(int32_t));
  w.pairs = kErrBytes;
  w.counts = w.pairs + kWsAlign;
  w.need = w.counts + align_up(static_cast<size_t>(pages / kPageChunkPages + 1) * sizeof(int32_t));
  w.first = w.need + row;
  w.src = w.first + row;
  w.dst = w.src + pairs;
  w.tokens = w.dst + pairs;
  w.place = w.tokens + row;
  w.total = w.place + row;
  return w;
}

msa_status_t status_of(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

// The workspace and the pool's part of the arguments.
msa_status_t page_args(const msa_page_pool_t* pool, int64_t rows, void* workspace, size_t workspace_bytes, PageArgs* a) {
  const PageLayout w = page_layout(pool->num_pages, rows);
  if (workspace == nullptr || workspace_bytes < w.total || !aligned16(workspace)) return MSA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a->refs = pool->refs;
  a->refs_out = pool->refs_out;
  a->num_pages = static_cast<int32_t>(pool->num_pages);
  a->buffers = pool->buffers;
  a->num_buffers = pool->num_buffers;
  a->err = reinterpret_cast<uint32_t*>(ws);
  a->pairs = reinterpret_cast<int32_t*>(ws + w.pairs);
  a->counts_free = reinterpret_cast<int32_t*>(ws + w.counts);
  a->need = reinterpret_cast<int32_t*>(ws + w.need);
  a->first = reinterpret_cast<int32_t*>(ws + w.first);
  a->src = reinterpret_cast<int32_t*>(ws + w.src);
  a->dst = reinterpret_cast<int32_t*>(ws + w.dst);
  a->tokens = reinterpret_cast<int32_t*>(ws + w.tokens);
  a->place = reinterpret_cast<int32_t*>(ws + w.place);
  return MSA_OK;
}

void batch_args(const msa_batch_t* b, PageArgs* a) {
  a->block_table = b->block_table;
  a->seq_lens = b->seq_lens;
  a->batch = b->batch;
  a->max_blocks = b->max_blocks;
  a->q_len = b->q_len;
}

// Entries of a table: counted in 32 bits.
bool many(int64_t rows, int64_t width) { return rows * width > INT32_MAX; }

template <typename Launch>
msa_status_t launch(Launch f, const PageArgs& a, void* stream) {
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return MSA_ERR_CUDA;
  return status_of(f(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t msa_page_workspace_bytes(const msa_page_pool_t* pool, int32_t rows) {
  if (check_pool(pool) != MSA_OK || rows < 0) return 0;
  return page_layout(pool->num_pages, rows).total;
}

msa_status_t msa_extend_pages(const msa_page_pool_t* pool, const msa_batch_t* batch, const int32_t* new_tokens,
                              int32_t* table_out, int32_t* seq_lens_out, void* workspace, size_t workspace_bytes,
                              void* stream) {
  msa_status_t st;
  if ((st = check_pool(pool)) != MSA_OK || (st = check_batch(batch)) != MSA_OK) return st;
  if (many(batch->batch, batch->max_blocks)) return MSA_ERR_UNSUPPORTED;
  if (batch->batch > 0 && (table_out == nullptr || seq_lens_out == nullptr)) return MSA_ERR_INVALID_ARG;
  const size_t row = static_cast<size_t>(batch->batch) * 4, table = row * batch->max_blocks;
  const size_t refs = static_cast<size_t>(pool->num_pages) * 4;
  const Range in[4] = {{pool->refs, refs}, {batch->block_table, table}, {batch->seq_lens, row}, {new_tokens, row}};
  const Range out[3] = {{pool->refs_out, refs}, {table_out, table}, {seq_lens_out, row}};
  if (!arrays_ok(in, out, {true, true, true})) return MSA_ERR_INVALID_ARG;
  PageArgs a{};
  if ((st = page_args(pool, batch->batch, workspace, workspace_bytes, &a)) != MSA_OK) return st;
  batch_args(batch, &a);
  a.new_tokens = new_tokens;
  a.table_out = table_out;
  a.seq_lens_out = seq_lens_out;
  return launch(launch_extend_pages, a, stream);
}

msa_status_t msa_fork_pages(const msa_page_pool_t* pool, const msa_batch_t* batch, const int32_t* parents,
                            int32_t children, int32_t* table_out, int32_t* seq_lens_out, void* workspace,
                            size_t workspace_bytes, void* stream) {
  msa_status_t st;
  if ((st = check_pool(pool)) != MSA_OK || (st = check_batch(batch)) != MSA_OK) return st;
  if (children < 0) return MSA_ERR_INVALID_ARG;
  if (children > kPageRows || many(children, batch->max_blocks) || many(batch->batch, batch->max_blocks))
    return MSA_ERR_UNSUPPORTED;
  if (children > 0 && (parents == nullptr || table_out == nullptr || seq_lens_out == nullptr)) return MSA_ERR_INVALID_ARG;
  const size_t row = static_cast<size_t>(batch->batch) * 4, table = row * batch->max_blocks;
  const size_t kids = static_cast<size_t>(children) * 4, refs = static_cast<size_t>(pool->num_pages) * 4;
  const Range in[4] = {{pool->refs, refs}, {batch->block_table, table}, {batch->seq_lens, row}, {parents, kids}};
  const Range out[3] = {{pool->refs_out, refs}, {table_out, kids * batch->max_blocks}, {seq_lens_out, kids}};
  if (!arrays_ok(in, out, {true, false, false})) return MSA_ERR_INVALID_ARG;
  PageArgs a{};
  if ((st = page_args(pool, children, workspace, workspace_bytes, &a)) != MSA_OK) return st;
  batch_args(batch, &a);
  a.parents = parents;
  a.children = children;
  a.table_out = table_out;
  a.seq_lens_out = seq_lens_out;
  return launch(launch_fork_pages, a, stream);
}

msa_status_t msa_free_pages(const msa_page_pool_t* pool, const int32_t* pages, const int32_t* counts, int32_t rows,
                            int32_t width, void* workspace, size_t workspace_bytes, void* stream) {
  msa_status_t st;
  if ((st = check_pool(pool)) != MSA_OK) return st;
  if (rows < 0 || width < 0) return MSA_ERR_INVALID_ARG;
  if (many(rows, width)) return MSA_ERR_UNSUPPORTED;
  const size_t list = static_cast<size_t>(rows) * width * 4, refs = static_cast<size_t>(pool->num_pages) * 4;
  if (list > 0 && pages == nullptr) return MSA_ERR_INVALID_ARG;
  const Range in[3] = {{pool->refs, refs}, {pages, list}, {counts, static_cast<size_t>(rows) * 4}};
  const Range out[1] = {{pool->refs_out, refs}};
  if (!arrays_ok(in, out, {true})) return MSA_ERR_INVALID_ARG;
  PageArgs a{};
  if ((st = page_args(pool, 0, workspace, workspace_bytes, &a)) != MSA_OK) return st;
  a.pages = pages;
  a.counts = counts;
  a.rows = rows;
  a.width = width;
  return launch(launch_free_pages, a, stream);
}

msa_status_t msa_compact_pages(const msa_page_pool_t* pool, const msa_batch_t* batch, int32_t* table_out,
                               int32_t* page_map, int32_t* live_count, void* workspace, size_t workspace_bytes,
                               void* stream) {
  msa_status_t st;
  if ((st = check_pool(pool)) != MSA_OK || (st = check_batch(batch)) != MSA_OK) return st;
  if (many(batch->batch, batch->max_blocks)) return MSA_ERR_UNSUPPORTED;
  if (page_map == nullptr || live_count == nullptr || (batch->batch > 0 && table_out == nullptr)) return MSA_ERR_INVALID_ARG;
  const size_t row = static_cast<size_t>(batch->batch) * 4, table = row * batch->max_blocks;
  const size_t refs = static_cast<size_t>(pool->num_pages) * 4;
  const Range in[3] = {{pool->refs, refs}, {batch->block_table, table}, {batch->seq_lens, row}};
  const Range out[4] = {{pool->refs_out, refs}, {table_out, table}, {page_map, refs}, {live_count, 4}};
  if (!arrays_ok(in, out, {true, true, false, false})) return MSA_ERR_INVALID_ARG;
  PageArgs a{};
  if ((st = page_args(pool, 0, workspace, workspace_bytes, &a)) != MSA_OK) return st;
  batch_args(batch, &a);
  a.table_out = table_out;
  a.page_map = page_map;
  a.live_count = live_count;
  return launch(launch_compact_pages, a, stream);
}

}  // extern "C"
