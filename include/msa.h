/*
 * msa.h -- C ABI of the GB300 (sm_103a) MiniMax Sparse Attention decode library (libmsa.so).
 *
 * MSA replaces full attention with block-sparse attention.  The KV cache is split into
 * 128-token blocks; a lightweight indexer scores every key in the context with one index
 * query per GQA group against a single shared index-key head, max-pools the scores to
 * one score per block, and the main attention then runs exactly, but only over the
 * top-16 blocks, the most recent block always kept, so every query sees at most 2,048
 * keys ("vLLM liefert Day-0-Unterstützung für MiniMax-M3.1-Flash", §MSA-Grundlagen).
 * Both the main K/V cache and the index-key cache are NVFP4 (E2M1 values, one E4M3
 * scale per 16 elements); queries are FP8 E4M3 (same page, §Was ist neu in der
 * MiniMax-M3.1-Architektur and §NVIDIA-Blackwell-optimierte MSA-Kernel).
 *
 * Conventions shared by every entry point:
 *   - Every tensor pointer is DEVICE memory owned by the caller; the library allocates
 *     and frees nothing and never synchronises the device (msa_read_device_error is the
 *     one documented exception).
 *   - Work is enqueued on `stream` (a cudaStream_t passed as void*; NULL = legacy
 *     default stream) and returns immediately.
 *   - Arguments are validated on the host before anything is launched; a violation
 *     returns MSA_ERR_INVALID_ARG / MSA_ERR_UNSUPPORTED / MSA_ERR_WORKSPACE and
 *     launches nothing.  A failed launch returns MSA_ERR_CUDA.  Output contents are
 *     unspecified after a non-OK status.
 *   - Data that only the device can check (block-table entries, sequence lengths) is
 *     checked in the kernels: a bad entry sets a bit in the workspace error word, the
 *     offending page or sequence is skipped, and nothing traps.
 *   - Query position: token t (0 <= t < q_len) of sequence b sits at position
 *     pos = seq_lens[b] - q_len + t (the q_len new tokens are already in the cache);
 *     key j is visible to it iff j <= pos.  Speculative draft tokens are the q_len
 *     tokens of one request, flattened request-major ("MiniMax M3 x vLLM：百万 token 多模态
 *     推理的 Day-0 部署", §Decode Kernel 中的投机解码).
 *   - seq_lens[b] == 0 marks a padding row: its outputs are defined (scores -inf,
 *     selection -1, output 0, lse -inf) and no error is raised.
 *
 * Layouts (row-major; every pointer 16-byte aligned):
 *   index-key cache  idx_data  uint8 [num_pages][128][Di/2]   idx_scale uint8 [num_pages][128][Di/16]
 *   K (and V) cache  k_data    uint8 [num_pages][G][128][D/2] k_scale   uint8 [num_pages][G][128][D/16]
 *     byte i of a row holds element 2i in its low nibble and element 2i+1 in its high nibble;
 *     scale byte s of a row is the E4M3 scale of elements 16s..16s+15.
 *   block_table      int32 [batch][max_blocks]  logical block n of sequence b -> page
 *   seq_lens         int32 [batch]
 *   queries q        uint8 E4M3 [batch][q_len][G*Hg][D]   (head h belongs to group h / Hg)
 *   index queries    uint8 E4M3 [batch][q_len][G][Di]
 *   block_scores     float [batch][q_len][G][max_blocks]
 *   selection        int32 [batch][q_len][G][16]  ascending logical block ids, -1 padded (rows
 *                    are 16 wide, the largest top_k; entries past min(top_k, r + 1) are -1)
 *   out              bfloat16 bits (uint16) [batch][q_len][G*Hg][D]
 *   lse              float [batch][q_len][G*Hg]  natural log of the softmax denominator
 */
#ifndef MSA_H_
#define MSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MSA_ABI_VERSION 2

typedef enum {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misaligned pointer */
  MSA_ERR_UNSUPPORTED = 2,  /* a configuration the library does not implement */
  MSA_ERR_WORKSPACE = 3,    /* workspace missing or smaller than msa_workspace_bytes() */
  MSA_ERR_CUDA = 4          /* a CUDA launch or query failed */
} msa_status_t;

/* Bits of the device error word (first 4 bytes of the workspace). */
#define MSA_DEVERR_BAD_PAGE 0x1u    /* a block-table entry outside [0, num_pages) */
#define MSA_DEVERR_BAD_SEQLEN 0x2u  /* seq_len < q_len (but > 0), or > max_blocks*128 */
#define MSA_DEVERR_TIMEOUT 0x4u     /* a bounded wait inside a kernel gave up */
#define MSA_DEVERR_BAD_SCALE 0x8u   /* an FP8 page scale outside MSA_E8M0_MIN..MSA_E8M0_MAX */
#define MSA_DEVERR_NO_PAGE 0x10u    /* the page pool has fewer free pages than a call needs */
#define MSA_DEVERR_BAD_PARENT 0x20u /* msa_fork_pages: a parent outside [-1, batch) */

/* Block-score reduction over the visible keys of a block ("MiniMax M3 x vLLM：百万 token
 * 多模态推理的 Day-0 部署", §Prefill 执行 step 2: a block-level rule such as max or
 * log-sum-exp, by model configuration). */
#define MSA_SCORE_MAX 0  /* max_j s_j (the recipe) */
#define MSA_SCORE_LSE 1  /* ln sum_j e^{s_j} (natural log) */

/* Sparse configuration.  The pages' M3 recipe: block 128, top-16, init_blocks = 0,
 * local_blocks = 1, max pooling ("MiniMax M3 x vLLM：百万 token 多模态推理的 Day-0 部署",
 * §MSA 机制细节, which names init_blocks / local_blocks as configuration).
 * The library implements: num_kv_groups in 1..8, heads_per_group in 1..8,
 * head_dim = index_dim = block_size = 128, 1 <= top_k <= 16, init_blocks >= 0,
 * local_blocks >= 0 with init_blocks + local_blocks <= top_k, score_type MSA_SCORE_MAX or
 * MSA_SCORE_LSE; anything else returns MSA_ERR_UNSUPPORTED.
 * Selection of a row whose recent block is r = pos / 128: min(top_k, r + 1) blocks -- the
 * first init_blocks blocks and the last local_blocks blocks up to r (each once), and the
 * best of the other blocks up to r for the remaining places. */
typedef struct {
  int32_t num_kv_groups;    /* G */
  int32_t heads_per_group;  /* Hg */
  int32_t head_dim;         /* D */
  int32_t index_dim;        /* Di */
  int32_t block_size;       /* tokens per block and per cache page */
  int32_t top_k;            /* blocks kept per (query token, KV group), recent block included */
  int32_t init_blocks;      /* leading blocks always kept */
  int32_t local_blocks;     /* trailing (recent) blocks always kept */
  float softmax_scale;      /* logits = (q . k) * softmax_scale; 0 means 1/sqrt(head_dim) */
  int32_t score_type;       /* MSA_SCORE_MAX or MSA_SCORE_LSE */
} msa_config_t;

/* The paged NVFP4 caches (device, caller-owned, read-only for decode). */
typedef struct {
  const uint8_t* k_data;
  const uint8_t* k_scale;
  const uint8_t* v_data;
  const uint8_t* v_scale;
  const uint8_t* idx_data;
  const uint8_t* idx_scale;
  int64_t num_pages;
} msa_cache_t;

/* One decode batch (device pointers; sizes on the host). */
typedef struct {
  const int32_t* block_table;  /* [batch][max_blocks] */
  const int32_t* seq_lens;     /* [batch] */
  int32_t batch;               /* 0..2048; batch * q_len <= 65535 */
  int32_t max_blocks;          /* >= 1 */
  int32_t q_len;               /* query tokens per sequence, >= 1 */
} msa_batch_t;

typedef enum {
  MSA_OP_INDEXER_SCORES = 0,
  MSA_OP_SELECT_BLOCKS = 1,
  MSA_OP_SPARSE_ATTN = 2,
  MSA_OP_DECODE = 3,
  MSA_OP_FP8_APPEND = 4,
  MSA_OP_FP8_ATTN = 5,          /* msa_fp8_attn without weight_out */
  MSA_OP_FP8_ATTN_WEIGHTS = 6,  /* msa_fp8_attn with weight_out (or without) */
  MSA_OP_EVICT = 7,
  MSA_OP_PROMPT_ATTN = 8        /* sized by msa_prompt_workspace_bytes, not by msa_workspace_bytes */
} msa_op_t;

/* Element types of the arguments that come in more than one. */
#define MSA_TYPE_F32 0
#define MSA_TYPE_BF16 1
#define MSA_TYPE_E4M3 2

/* The paged FP8 K/V cache (device, caller-owned): E4M3 codes with one power-of-two scale for
 * each page (block of 128 tokens) and KV head, stored as an E8M0 byte; the value of a code is
 * code * 2^(scale - 127).  It shares block tables and page numbers with the NVFP4 pools
 * ("vLLM liefert Day-0-Unterstützung für MiniMax-M3.1-Flash", §Was ist neu in der
 * MiniMax-M3.1-Architektur, sizes the FP8 K/V cache it compares with at 61,440 B/token).
 *   k_data, v_data    uint8 E4M3 [num_pages][G][128][128]
 *   k_scale, v_scale  uint8 E8M0 [num_pages][G], MSA_E8M0_MIN..MSA_E8M0_MAX (2^-40 .. 2^40:
 *                     any K scale times any logit, and any V scale over any other, stays
 *                     inside float32's range)
 * The data pointers are 16-byte aligned; the scale pointers may have any alignment. */
#define MSA_E8M0_MIN 87
#define MSA_E8M0_MAX 167
typedef struct {
  uint8_t* k_data;
  uint8_t* k_scale;
  uint8_t* v_data;
  uint8_t* v_scale;
  int64_t num_pages;
} msa_fp8_cache_t;

/* Packed prompts: the query tokens of all sequences in one list and their keys in another
 * (device pointers; sizes on the host).  Sequence b has the query tokens cu_q[b] ..
 * cu_q[b + 1] - 1 and the keys cu_k[b] .. cu_k[b + 1] - 1. */
typedef struct {
  const int32_t* cu_q; /* [batch + 1] */
  const int32_t* cu_k; /* [batch + 1] */
  int32_t batch;       /* 0..2048 */
  int64_t q_tokens;    /* tokens of the query list (those behind the last sequence belong to none) */
  int64_t k_tokens;    /* tokens of the key list */
} msa_packed_t;

/* One buffer of a page pool (device): page p's bytes start at data + p * page_bytes.  With
 * token_bytes > 0 a page is page_bytes / (128 * token_bytes) runs of 128 tokens of token_bytes
 * each (a run is a KV head); with token_bytes = 0 nothing in it belongs to single tokens. */
typedef struct {
  void* data;
  int64_t page_bytes;
  int32_t token_bytes;
} msa_page_buffer_t;

/* A pool of pages that block tables share: how many references each page has (0: free), and
 * the buffers that hold the pages, of as many caches (layers, K and V, codes and scales) as go
 * by the same page numbers.  An operation reads refs and leaves the new counts in refs_out,
 * which may be refs. */
typedef struct {
  const int32_t* refs;             /* device int32 [num_pages], 16-byte aligned */
  int32_t* refs_out;               /* device int32 [num_pages], 16-byte aligned */
  int64_t num_pages;               /* 1 .. 2^27 */
  const msa_page_buffer_t* buffers; /* HOST array, read during the call */
  int32_t num_buffers;             /* 0 .. 4096 */
} msa_page_pool_t;

/* ABI version of the loaded library (MSA_ABI_VERSION). */
int32_t msa_abi_version(void);

/* Human-readable name of a status code (static string). */
const char* msa_status_string(msa_status_t status);

/* Bytes of device workspace `op` needs for this configuration and batch (host-only
 * arithmetic, no device access).  The workspace must be zero-filled once when it is
 * allocated (its first 4 bytes are the device error word); after that it may be reused
 * by every call with the same or smaller sizes.  Returns 0 for invalid arguments. */
size_t msa_workspace_bytes(msa_op_t op, const msa_config_t* cfg, const msa_batch_t* batch);

/* NVFP4 quantise-and-insert of new cache rows (the cache-write step in front of decode;
 * the pages fuse it into the QKV GEMM epilogue: "vLLM liefert Day-0-Unterstützung für
 * MiniMax-M3.1-Flash", §QKV GEMM + Norm + RoPE + KV-Insert-Fusion).
 *   x        float [n_tokens][rows_per_token][dim]   (K or V: rows = G; index keys: rows = 1)
 *   slots    int64 [n_tokens]  slot = page * block_size + offset of each token
 *   data     uint8 [num_pages][rows_per_token][block_size][dim/2]   (written)
 *   scale    uint8 [num_pages][rows_per_token][block_size][dim/16]  (written)
 * For every 16 consecutive elements: scale code = E4M3(amax/6), amax/6 in float32 rounded
 * to nearest even and saturated at 448; element code = E2M1(x/scale), x/scale in float32,
 * rounded to nearest even, saturated at +-6, sign kept; a zero scale gives zero codes.
 * Slots outside [0, num_pages*block_size) set nothing and are skipped. */
msa_status_t msa_nvfp4_insert(const float* x, int64_t n_tokens, int32_t rows_per_token, int32_t dim,
                              const int64_t* slots, uint8_t* data, uint8_t* scale, int64_t num_pages,
                              int32_t block_size, void* stream);

/* FP8 E4M3 encoding of float32 values (round to nearest even, saturating at +-448, sign kept). */
msa_status_t msa_fp8_quantize(const float* x, int64_t n, uint8_t* out, void* stream);

/* Stage 1 -- indexer score + block pooling.
 * block_scores[b][t][g][n] = max (MSA_SCORE_MAX) or log-sum-exp (MSA_SCORE_LSE) over the
 * visible keys j of block n of (qi[b][t][g] . key_j), exact products (E2M1 x E4M3 x E4M3)
 * accumulated in float32 (the log-sum-exp with expf / logf); -inf where block n has no
 * visible key (n beyond the query's own block or past the sequence end).  Entries
 * n >= ceil(seq_len/128) are written -inf too.  Any q_len works: with R = q_len x groups
 * query rows per sequence, R <= 8 (decode) takes a streaming kernel, 8 < R < 64
 * (speculative decode) a tcgen05 kernel with the keys as M, R >= 64 (chunked prefill) a
 * tcgen05 GEMM with the query rows as M; all three give the same exact products and float32
 * accumulation.  Errors: MSA_ERR_CUDA also when the driver's tensor-map encoder is not
 * available (8 < R < 64) or num_pages * 128 exceeds 2^31 rows there.
 * workspace: msa_workspace_bytes(MSA_OP_INDEXER_SCORES, ...). */
msa_status_t msa_indexer_scores(const msa_config_t* cfg, const msa_cache_t* cache, const msa_batch_t* batch,
                                const uint8_t* index_q, float* block_scores, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Stage 2 -- top-k block selection with forced blocks.
 * For each (b, t, g) with recent block r = pos / 128: the first init_blocks and the last
 * local_blocks blocks up to r are always selected (the recipe: r alone); the other places,
 * up to min(top_k, r + 1) in all, go to the blocks between them ranked by (score
 * descending, index ascending; NaN below -inf); the result is sorted ascending, -1 padded
 * to 16.  Bit-exact for given scores.  No workspace. */
msa_status_t msa_select_blocks(const msa_config_t* cfg, const msa_batch_t* batch, const float* block_scores,
                               int32_t* selection, void* stream);

/* Decode context parallelism, shard side ("vLLM liefert Day-0-Unterstützung für
 * MiniMax-M3.1-Flash", §NVFP4-Indexer-DCP: each GPU scores every index-query head over its
 * slice of the context, keeps a local top-16 per head and sends it to the head's owner, who
 * merges exactly).  On one GPU a shard is a range of logical blocks of every sequence.
 * Scores logical blocks [block_lo, block_hi) exactly as msa_indexer_scores does into
 * block_scores (same layout; -inf for blocks outside the range or past the sequence end),
 * then writes for every (b, t, g) row the shard's best top_k - 1 blocks among
 * [block_lo, min(block_hi, r)) -- r the row's recent block, which the owner adds -- ranked
 * as msa_select_blocks ranks (score descending, then index ascending; NaN below -inf), best
 * first, with their scores:
 *   cand_scores  float [batch][q_len][G][15]   cand_blocks  int32 [batch][q_len][G][15]
 *   (-inf / -1 past the end of a shorter list).
 * Supported: q_len x num_kv_groups <= 8 (decode) and the recipe's init_blocks == 0,
 * local_blocks == 1, else MSA_ERR_UNSUPPORTED; 0 <= block_lo < block_hi, else
 * MSA_ERR_INVALID_ARG.  workspace: msa_workspace_bytes(MSA_OP_INDEXER_SCORES, ...). */
msa_status_t msa_dcp_local_candidates(const msa_config_t* cfg, const msa_cache_t* cache, const msa_batch_t* batch,
                                      const uint8_t* index_q, int32_t block_lo, int32_t block_hi, float* block_scores,
                                      float* cand_scores, int32_t* cand_blocks, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* Decode context parallelism, owner side: merges the candidate lists of num_shards shards
 * (1..8; disjoint block ranges that together cover every block of every sequence) into the
 * selection: the best top_k - 1 of all candidates plus each row's recent block, ascending, -1
 * padded to 16 (every block 0 .. r when r + 1 <= top_k).
 *   cand_scores  float [num_shards][batch][q_len][G][15], cand_blocks int32 alike (the
 *   shards' outputs, concatenated in any shard order).
 * The merge is exact: top_k - 1 of the union of each shard's top_k - 1 is the global top_k - 1
 * under one strict order, so the selection is bit-identical to msa_select_blocks on the
 * unsharded scores.  Same support rules as the shard side; no workspace. */
msa_status_t msa_dcp_merge(const msa_config_t* cfg, const msa_batch_t* batch, int32_t num_shards,
                           const float* cand_scores, const int32_t* cand_blocks, int32_t* selection, void* stream);

/* Stage 3 -- exact sparse GQA attention over the selected blocks.  Every head h of group g
 * attends, with logits (q . k) * softmax_scale, to the visible keys of selection[b][t][g][:];
 * K/V are dequantised exactly from NVFP4 in the kernel.  out is rounded to bfloat16;
 * lse may be NULL.  workspace: msa_workspace_bytes(MSA_OP_SPARSE_ATTN, ...).
 * Below 64 query tokens per sequence the selected pages of all rows are split evenly across
 * the GPU (online softmax, split rows' partial states merged).  From 64 tokens on (chunked
 * prefill) the attention is KV-block-major ("MiniMax M3 x vLLM：百万 token 多模态推理的 Day-0
 * 部署", the query-major versus KV-block-major scheduling of the sparse GQA step): the
 * selections are inverted into a per-block list of (token, slot) entries, each selected
 * block is loaded once for all the tokens that chose it, and every (token, head) merges its
 * per-block partial states by log-sum-exp; its workspace then holds B*T*H*16 partial states
 * of 264 bytes (o / l in fp16, m and l in fp32) and the queries in fp16.  Both forms give
 * the same attention within the stated tolerances, and each is bit-reproducible. */
msa_status_t msa_sparse_attn_decode(const msa_config_t* cfg, const msa_cache_t* cache, const msa_batch_t* batch,
                                    const uint8_t* q, const int32_t* selection, uint16_t* out, float* lse,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* Fused decode step = stage 1 + stage 2 + stage 3 on one stream, intermediate scores and
 * selections kept in the workspace.  selection_out (may be NULL) receives the selection.
 * workspace: msa_workspace_bytes(MSA_OP_DECODE, ...): the error word, the block scores, the
 * selection, the page of every selected entry (looked up by the selection kernel for the
 * team attention kernel) and the stage-3 scratch (the stage-3 form follows the same 64-token
 * rule as msa_sparse_attn_decode).  seq_lens and block_table are read from the selection
 * kernel's start, before the indexer has finished: like q and index_q, they must be written
 * before the call's first kernel runs (any earlier stream-ordered write is).  For a small
 * batch of short rows (at most 128 (token, group) rows of at most 256 blocks, below 64 query
 * tokens) there is no selection kernel: the attention kernel's producers select their rows
 * from the block scores themselves, with the same order (the selection, written to
 * selection_out or the workspace, is the one msa_select_blocks makes). */
msa_status_t msa_decode(const msa_config_t* cfg, const msa_cache_t* cache, const msa_batch_t* batch,
                        const uint8_t* q, const uint8_t* index_q, uint16_t* out, float* lse,
                        int32_t* selection_out, void* workspace, size_t workspace_bytes, void* stream);

/* FP8 cache write: the q_len newest K and V rows of every sequence (positions
 * seq_lens[b] - q_len .. seq_lens[b] - 1) into their pages, as E4M3 with the scale of their
 * (page, KV head).
 *   k, v      float32 or bfloat16 (x_type MSA_TYPE_F32 / MSA_TYPE_BF16)
 *             [batch][q_len][G][head_dim]; the heads of a token are contiguous, token i (=
 *             b * q_len + t) starts k_stride (v_stride) elements after token i - 1, so that
 *             slices of one fused projection's rows need no copy.  Both pointers and both
 *             strides in bytes are multiples of 16; strides >= G * head_dim.
 *   cache     written: the pages holding those positions
 * For each touched (page, KV head), e is the smallest exponent in -40..40 with amax of the
 * new rows <= 448 * 2^e (NaN elements do not count; -40 for all zeros).  A page that already
 * holds older tokens of the sequence (positions before seq_lens[b] - q_len) keeps its scale
 * when that is larger than 2^e; otherwise its older rows are re-encoded under 2^e, each code
 * times 2^(e_old - e) rounded to E4M3 once more.  Codes: x * 2^-e rounded to nearest even, saturating at
 * +-448 (infinities too), the sign of zero kept, NaN as a NaN code.  Rows of the page at
 * seq_lens[b] and beyond are left as they are, and so is every other page.
 * A page is written once per call: tables that give one page to two written blocks, of one
 * sequence or of two, leave its contents unspecified.  Sequences of length 0 write nothing; an old scale
 * outside MSA_E8M0_MIN..MAX sets MSA_DEVERR_BAD_SCALE and leaves the page head alone.
 * workspace: msa_workspace_bytes(MSA_OP_FP8_APPEND, ...) (the error word). */
msa_status_t msa_fp8_append(const msa_config_t* cfg, const msa_fp8_cache_t* cache, const msa_batch_t* batch,
                            const void* k, const void* v, int32_t x_type, int64_t k_stride, int64_t v_stride,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Attention over the FP8 cache, dense or sparse: the layers that keep full attention next to
 * the MSA layers, MSA layers over an 8-bit cache, and what eviction needs to know.
 * Query row (b, t, h), position pos = seq_lens[b] - q_len + t, attends with logits
 * z_j = (q . k_j) * softmax_scale to the keys j <= pos (selection NULL: dense causal), or to
 * those of them in the blocks selection[b][t][h / Hg][:] (the layout of msa_select_blocks, -1
 * for an empty place, in any order; a block listed twice counts twice):
 *   out  = sum_j e^{z_j - lse} v_j   bfloat16 [batch][q_len][G*Hg][D]
 *   lse  = ln sum_j e^{z_j}          float [batch][q_len][G*Hg], may be NULL
 * A row with no key (padding, an empty selection, only bad pages) gives out 0 and lse -inf.
 *   q       E4M3 or bfloat16 (q_type MSA_TYPE_E4M3 / MSA_TYPE_BF16) [batch][q_len][G*Hg][D];
 *           the heads of a token are contiguous, tokens are q_stride elements apart; pointer
 *           and stride in bytes multiples of 16, q_stride >= G * Hg * D.  bfloat16 values more
 *           than 2^13 below the largest of their row may be rounded, by at most 2^-21 of that
 *           largest value (or by 2^-143, if that is more).
 *   weight_out  float [batch][max_blocks] or NULL: how much attention each block collected,
 *           weight_out[b][n] = weight_decay * weight_in[b][n]
 *                              + sum over t, h and the keys j of block n of e^{z_j - lse}
 *           for every n in 0 .. max_blocks - 1 (a missing weight_in counts as 0).  weight_in may be
 *           weight_out, but not overlap it otherwise.  weight_decay in 0..1.
 * A NaN code in K or V makes the results of the rows that see its key NaN (of V: in its dim),
 * and of no other row; codes past seq_lens[b] may be anything.  A query row with a NaN or an
 * infinity gives NaN.  A page whose table entry or scale is bad is skipped
 * (MSA_DEVERR_BAD_PAGE, MSA_DEVERR_BAD_SCALE), a sequence whose length is bad gives empty rows
 * (MSA_DEVERR_BAD_SEQLEN).
 * Results do not depend on how the work is split beyond rounding, and are the same bits in
 * every call with the same arguments on one GPU.
 * Rounding: logits, sums and lse are float32 (a logit is to stay inside its range).  A probability
 * meets its V row in fp16: it is rounded by 2^-11 of itself or, where it is small, by at most 2^-29
 * of its row's sum, whatever the page scales: before its rounding to bfloat16 out[d] is off by at most
 *   (2^-11 + twice the largest error of a logit) * sum_j p_j |v_jd| + keys * 2^-29 * max_j |v_jd|.
 * With a selection the collected weights of a sequence are summed in units of 2^-40.
 * workspace: msa_workspace_bytes(MSA_OP_FP8_ATTN_WEIGHTS, ...) with weight_out, else
 * MSA_OP_FP8_ATTN; calls that can overlap need a workspace each.  The first holds 8 bytes for every
 * query row (token, head) and place: max_blocks places (the table's width, not the lengths) for
 * dense rows, four times as many up to 16 rows of a group, or 64 for a selection, whichever is
 * more, as the operation's size does not say which it is: 0.6 GB for 4,096 tokens of 32 heads on
 * 544 blocks, 8.6 GB for 16,384 tokens of 64 heads on 1,024.  A long prompt collects its weights in
 * calls of some thousand tokens each, weight_in = weight_out and weight_decay 1.
 * Errors: MSA_ERR_UNSUPPORTED for num_pages * G > 2^24 (a tensor map's row coordinate) or
 * 2 * batch * ceil(q_len * Hg / 256) * max_blocks * G > 2^31 - 1 (the pages to visit);
 * MSA_ERR_CUDA also when the driver's tensor-map encoder is not available. */
msa_status_t msa_fp8_attn(const msa_config_t* cfg, const msa_fp8_cache_t* cache, const msa_batch_t* batch,
                          const void* q, int32_t q_type, int64_t q_stride, const int32_t* selection, uint16_t* out,
                          float* lse, const float* weight_in, float weight_decay, float* weight_out, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Eviction by accumulated attention weight: cuts every sequence to at most `budget` blocks by
 * dropping the blocks of least weight from its block table.
 * Of the ceil(seq_lens[b] / 128) blocks of a sequence with more than `budget`, the first
 * keep_first and the last keep_last stay, and the best of the others by (weight descending,
 * block ascending; NaN below -inf) up to `budget` in all; shorter sequences stay whole.
 *   weight         float [batch][max_blocks]  (msa_fp8_attn's weight_out, or any other score)
 *   table_out      int32 [batch][max_blocks]  pages of the blocks that stay, in order; -1 behind
 *   seq_lens_out   int32 [batch]              seq_lens[b] - 128 * (blocks dropped)
 *   weight_out     float [batch][max_blocks]  their weights; 0 behind
 *   freed          int32 [batch][max_blocks]  table entries of the dropped blocks, in order; -1 behind
 *   freed_count    int32 [batch]
 * table_out, seq_lens_out and weight_out may be the inputs themselves; any other overlap of
 * two arrays is MSA_ERR_INVALID_ARG.  1 <= keep_last, 0 <= keep_first, keep_first + keep_last
 * <= budget.  Keys keep the rotary position they were written with; causal order among what
 * stays is unchanged, so every entry point runs on the shorter table (the index keys of the
 * dropped pages go with them).  Table entries are moved, never followed.  A length below 0 or above
 * max_blocks * 128 sets MSA_DEVERR_BAD_SEQLEN and the row is copied as it is, nothing freed.
 * workspace: msa_workspace_bytes(MSA_OP_EVICT, ...) (the error word; cfg is only checked). */
msa_status_t msa_evict_blocks(const msa_batch_t* batch, const float* weight, int32_t budget, int32_t keep_first,
                              int32_t keep_last, int32_t* table_out, int32_t* seq_lens_out, float* weight_out,
                              int32_t* freed, int32_t* freed_count, void* workspace, size_t workspace_bytes,
                              void* stream);

/* Causal attention of packed prompts over their own bfloat16 keys and values, before (or
 * without) their way into pages: whole prompts, chunks of them behind keys that are still at
 * hand (cu_k longer than cu_q), single new tokens.
 * Query token t of sequence b, of Lq = cu_q[b+1] - cu_q[b], sits at position Lk - Lq + t of its
 * Lk = cu_k[b+1] - cu_k[b] keys, and head h attends to the keys j <= that position of KV head
 * h / Hg with logits z_j = (q . k_j) * softmax_scale:
 *   out  = sum_j e^{z_j - lse} v_j   bfloat16 [q_tokens][G*Hg][D]
 *   lse  = ln sum_j e^{z_j}          float [q_tokens][G*Hg], may be NULL
 * A row with no key (Lk < Lq: the first Lq - Lk tokens), or whose logits are all -inf and what it sees of v
 * finite, gives out 0 and lse -inf.  Rows of tokens that belong to no sequence are left as they are.
 *   q        bfloat16 [q_tokens][G*Hg][D], k, v bfloat16 [k_tokens][G][D]: the heads of a token are
 *            contiguous, tokens are q_stride (k_stride, v_stride) elements apart, so that slices of
 *            one fused projection's rows need no copy.  Pointers and strides in bytes are multiples
 *            of 16, strides at least a token's elements.  out may not overlap an input.
 * Keys that a row does not see (later ones, other sequences') do not touch it, whatever they
 * hold.  Other NaN and infinities in q or k make the rows whose logits they reach what float
 * arithmetic makes of them.  One in v makes the results of the rows that see it, in its dim, what adding its product with
 * the probability makes of them: NaN for a NaN, and for an infinity itself, or NaN where the probability is 0 (a logit
 * of -inf, alone or beside others, or one further below the row's largest than float32's exponents go; close to that either).
 * cu_q and cu_k must not decrease, start below 0 or end past q_tokens and k_tokens: otherwise
 * MSA_DEVERR_BAD_SEQLEN is set and nothing is written.
 * Rounding: logits, sums and lse are float32 (a logit that float32 does not hold, or not times log2(e), counts as infinite).
 * A probability meets its V row as bfloat16, and out is divided
 * by the sum of the rounded ones (lse has the sum before the rounding), so that before its own rounding
 * out[d] is off by at most (2^-7 + 2^-14 + twice the largest error of a logit) * sum_j p_j |v_jd|, by nothing for a
 * row of one key.  The same arguments give the same bits in every call on one GPU.
 * workspace: msa_prompt_workspace_bytes(...); calls that can overlap need one each.
 * Errors: MSA_ERR_UNSUPPORTED for q_tokens or k_tokens above 2^28, or where the call's pairs of
 * 128 query rows and 128 keys cannot be counted in 31 bits: G * (floor(q_tokens / (2 * floor(128 / Hg))) + batch) *
 * (2 * max(1, ceil(k_tokens / 128)) + 4) > 2^31 - 1 (about 1,048,000 tokens of 32 heads).  MSA_ERR_CUDA also when the
 * driver's tensor-map encoder is not available. */
size_t msa_prompt_workspace_bytes(const msa_config_t* cfg, const msa_packed_t* packed);
msa_status_t msa_prompt_attn(const msa_config_t* cfg, const msa_packed_t* packed, const void* q, int64_t q_stride,
                             const void* k, int64_t k_stride, const void* v, int64_t v_stride, uint16_t* out,
                             float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* The life of a pool's pages, on the device and without a look at them by the host: sequences
 * take pages for new tokens, go on from one another, give pages back, and the pages in use move
 * together.  Whoever holds a page of a block table holds a reference to it; a page is free when
 * its count is 0.  Pages are handed out from the lowest free number up, so that every result
 * is determined by the arguments.  A last block that is not full belongs to one sequence.
 * Overlapping arrays are MSA_ERR_INVALID_ARG, except an output that is its own input; the
 * buffers of a pool may not overlap.  A pool's calls change it one after another: on one
 * stream, or ordered by events.
 * workspace: msa_page_workspace_bytes(pool, rows), rows being the batch of the call (the
 * children of a fork); calls that can overlap need one each. */
size_t msa_page_workspace_bytes(const msa_page_pool_t* pool, int32_t rows);

/* Pages for new tokens.  Sequence b grows from L = seq_lens[b] by n = new_tokens[b] tokens
 * (new_tokens NULL: by batch->q_len, sequences of length 0 by none):
 *   seq_lens_out[b]  L + n
 *   table_out[b]     the row of block_table; blocks ceil(L/128) .. ceil((L+n)/128) - 1 get free pages,
 *                    which then have one reference
 * The i-th new block of the call, by sequence and then by block, gets the i-th free page.  When
 * the blocks that the sequences 0 .. b need are more than the free pages there are, a sequence b that needs
 * any stays as it was (MSA_DEVERR_NO_PAGE), and so does one with n < 0, L < 0 or L + n > max_blocks * 128
 * (MSA_DEVERR_BAD_SEQLEN).  table_out and seq_lens_out may be the inputs. */
msa_status_t msa_extend_pages(const msa_page_pool_t* pool, const msa_batch_t* batch, const int32_t* new_tokens,
                              int32_t* table_out, int32_t* seq_lens_out, void* workspace, size_t workspace_bytes,
                              void* stream);

/* Sequences that go on from others (samples of one prompt, beams).  Child i gets the length
 * of sequence parents[i] (int32 [children], 0..2048 of them; -1: an empty child, length 0), and
 *   table_out     int32 [children][max_blocks]: the parent's full blocks, whose pages have one reference
 *                 more per child, then, if the parent's last block is not full, a free page with one
 *                 reference and a copy of that block's tokens in every buffer of the pool (of a buffer
 *                 without tokens the whole page); -1 behind
 *   seq_lens_out  int32 [children]
 * The i-th child that needs a page gets the i-th free one; one that finds none is cut to its
 * full blocks (MSA_DEVERR_NO_PAGE).  Rows of the new pages behind the parent's tokens are left as they are.
 * A parent out of range (MSA_DEVERR_BAD_PARENT) or with a length below 0 or above max_blocks * 128
 * (MSA_DEVERR_BAD_SEQLEN) gives an empty child; a table entry outside the pool (MSA_DEVERR_BAD_PAGE)
 * becomes -1.  table_out and seq_lens_out may not overlap the inputs. */
msa_status_t msa_fork_pages(const msa_page_pool_t* pool, const msa_batch_t* batch, const int32_t* parents,
                            int32_t children, int32_t* table_out, int32_t* seq_lens_out, void* workspace,
                            size_t workspace_bytes, void* stream);

/* References given back: one for every entry of pages (int32 [rows][width]; the first counts[r]
 * entries of row r, all with counts NULL), msa_evict_blocks' freed and freed_count for example, or the
 * blocks of finished sequences.  Entries of -1 are passed over.  An entry outside the pool, or
 * one reference more than a page has (its count stays 0), sets MSA_DEVERR_BAD_PAGE; a count
 * below 0 or above width sets MSA_DEVERR_BAD_SEQLEN and its row is passed over. */
msa_status_t msa_free_pages(const msa_page_pool_t* pool, const int32_t* pages, const int32_t* counts, int32_t rows,
                            int32_t width, void* workspace, size_t workspace_bytes, void* stream);

/* Pages in use moved to the lowest numbers.  With n pages in use (count not 0), the i-th of them
 * that is numbered n or higher moves, in every buffer, to the i-th free number below n:
 *   refs_out    counts under the new numbers; 0 from n on
 *   page_map    int32 [num_pages]: the new number of every page, -1 for a free one
 *   live_count  int32 [1]: n
 *   table_out   int32 [batch][max_blocks] (may be the block table): the ceil(seq_lens[b] / 128) entries of
 *               every row under their new numbers, -1 behind; an entry of a free page or outside
 *               the pool becomes -1 (MSA_DEVERR_BAD_PAGE), unless it is -1 already.  A length
 *               below 0 or above max_blocks * 128 sets MSA_DEVERR_BAD_SEQLEN: all of the row counts.
 * Other holders of page numbers take theirs through page_map. */
msa_status_t msa_compact_pages(const msa_page_pool_t* pool, const msa_batch_t* batch, int32_t* table_out,
                               int32_t* page_map, int32_t* live_count, void* workspace, size_t workspace_bytes,
                               void* stream);

/* The stage-3 sparse attention of msa_sparse_attn_decode for callers that cannot allocate
 * device memory, or cannot hand the library a workspace: for example a plugin inside a host
 * application whose device memory all belongs to that application's own pool, or code that
 * must not allocate between decode steps.  The source pages have no counterpart; this is a
 * deployment convenience.
 * Same arguments and results as msa_sparse_attn_decode, minus the workspace: the scratch
 * (partial softmax states of rows shared by two CTAs, and the device error word) lives in
 * one library-owned device array of 8 MiB, which every GPU that loads the library holds
 * until the process exits.  Nothing is allocated or freed.
 *   - It always runs the query-major form (whatever the number of query tokens), whose
 *     scratch is 4.0 MB whatever the batch, so every valid call fits; a call whose scratch
 *     would exceed 8 MiB would be rejected with MSA_ERR_WORKSPACE before any launch.
 *   - The first call on a device looks up the array's device address (cudaGetSymbolAddress,
 *     with that device current); make that first call before any stream capture.
 *   - All calls share the one array and it keeps the last call's contents: calls that can
 *     overlap on the GPU (different streams, or different host threads, on one device) race
 *     and must be serialised by the caller.
 *   - The array's device error word (bad block-table entries, bad lengths, a wait that gave
 *     up) is zeroed on `stream` by every call that passes validation, right before its
 *     launch (a rejected call leaves it alone), and read back with
 *     msa_noalloc_read_device_error. */
msa_status_t msa_sparse_attn_decode_noalloc(const msa_config_t* cfg, const msa_cache_t* cache,
                                            const msa_batch_t* batch, const uint8_t* q, const int32_t* selection,
                                            uint16_t* out, float* lse, void* stream);

/* The device error word of the no-allocation entry point's array, as the last call on this
 * device left it (MSA_DEVERR_* bits), copied into *flags; synchronises `stream`.  Like that
 * entry point it needs no workspace, and it shares its race: a call still running on
 * another stream may change the word.  The pages have no counterpart to it either. */
msa_status_t msa_noalloc_read_device_error(uint32_t* flags, void* stream);

/* Test hook for the failure path of the bounded waits; not part of the decode path.
 * Launches the streaming indexer of msa_indexer_scores (q_len x num_kv_groups <= 8; else
 * MSA_ERR_UNSUPPORTED) with its page copies withheld and every wait capped at spin_limit
 * polls (1 .. 2^22; msa_indexer_scores uses 2^22).  Nothing then arrives on the page ring,
 * so each warp with pages to score gives up its first wait, sets MSA_DEVERR_TIMEOUT in the
 * workspace error word and returns, with no copy in flight; block_scores are unspecified
 * afterwards.  The context stays usable: the next regular call computes normally.  Same
 * arguments and workspace as msa_indexer_scores, plus spin_limit. */
msa_status_t msa_test_indexer_stall(const msa_config_t* cfg, const msa_cache_t* cache, const msa_batch_t* batch,
                                    const uint8_t* index_q, float* block_scores, void* workspace,
                                    size_t workspace_bytes, uint32_t spin_limit, void* stream);

/* Test hook for the failure path of the team attention kernel's bounded waits; not part of
 * the decode path.  Runs the query-major team attention of msa_sparse_attn_decode (whatever
 * q_len; workspace of team size: msa_workspace_bytes(MSA_OP_SPARSE_ATTN, ...) for a batch below
 * 64 query tokens) with every wait capped at spin_limit polls (1 .. 2^22) and the page copies
 * withheld: each page slot is armed for its bytes but never filled, so the consumers' first
 * waits run out, then the producers' waits for free slots.  Every wait ends, no copy is in
 * flight when a wait gives up, MSA_DEVERR_TIMEOUT is set in the workspace error word and the
 * launch returns; outputs are unspecified.  The context stays usable. */
msa_status_t msa_test_attention_stall(const msa_config_t* cfg, const msa_cache_t* cache, const msa_batch_t* batch,
                                      const uint8_t* q, const int32_t* selection, uint16_t* out, float* lse,
                                      void* workspace, size_t workspace_bytes, uint32_t spin_limit, void* stream);

/* Debug helper: copies the device error word out of `workspace` into *flags (this call
 * synchronises `stream`). */
msa_status_t msa_read_device_error(const void* workspace, uint32_t* flags, void* stream);

/* Clears the device error word (asynchronous). */
msa_status_t msa_clear_device_error(void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H_ */
