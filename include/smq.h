/*
 * smq.h: C ABI of the GB300 candidate-block sparse MQA-logits top-k indexer.
 *
 * DeepSeek-V4.1 two-level selection works like this. A candidate-source
 * indexer publishes, for every query row, its top candidate blocks. Each
 * later consumer indexer then scores only the key positions inside those
 * blocks and keeps its top-k token ids, so its work is O(candidate blocks)
 * rather than O(context). Source: the "vllm.model_executor.layers.
 * sparse_mqa_indexer" API docs, module docstring and SparseMQAIndexer.
 *
 * For a row with FP8 query q[h][d] (H heads, D = 128), per-row scale s,
 * bf16 head weights w[h] and key k[d], the score of a position is
 *     logit = sum_h w[h] * ReLU(s * q[h] . k).
 * This is the DeepSeek indexer score that the pages' MQA-logits kernels
 * compute. The pages name it but do not print it.
 *
 * Positions outside the row's key range [ks, ke), and positions in no
 * valid candidate block, are masked. The top-k token ids per row are
 * written relative to ks, padded with -1.
 *
 * Conventions of every entry point
 *  - Every pointer named "device" is CUDA device memory owned by the caller.
 *    The library allocates nothing in any call. Only smq_plan_create and
 *    smq_plan_destroy allocate or free host memory for the plan itself.
 *    (Source: "vllm/v1/attention/backends/mla/sparse_indexer.py", module
 *    docstring: the layer op allocates nothing per step.)
 *  - Every call is asynchronous on the caller's stream (a cudaStream_t
 *    passed as void*; NULL is the legacy default stream). Exceptions:
 *    smq_plan_create, smq_plan_destroy and smq_get_status.
 *  - Every call returns an smq_status code. A non-zero return means nothing
 *    was enqueued.
 *  - Errors the GPU detects are OR-ed into a status word at the start of
 *    the workspace: an out-of-range page, block-table row or block id
 *    (SMQ_ERR_BOUNDS), a pipeline wait that gave up (SMQ_ERR_TIMEOUT), or too
 *    few free pages (SMQ_ERR_NO_PAGES).
 *    The outputs of a call that raised one are unspecified.
 *    smq_get_status reads the word and clears it.
 *  - The arguments are checked once, at plan creation ("engine start").
 *    Calls only re-check pointers, alignment and sizes. (Source:
 *    sparse_indexer.py, DeepseekV41SparseIndexerMetadataBuilder: every
 *    requirement of the sparse kernels is checked at engine start rather
 *    than by falling back per step.)
 *  - Argument structs begin with struct_size. Set it to sizeof(the struct)
 *    so that later versions can append fields.
 *
 * Formats (the pages fix the element formats; the byte layout is this
 * library's)
 *  - Q: [rows][H][D] bytes, OCP FP8 E4M3 ("fn"). q_scale: [rows] float,
 *    positive and finite.
 *  - weights: [rows][H] bfloat16 (as uint16 bits).
 *  - Paged MXFP4 K cache: pages of page_size tokens. page_bytes =
 *    page_size * (D/2 + D/32), and the cache base must be 16-byte aligned.
 *    A page is
 *      values [page_size][D/2]: OCP MX FP4 E2M1, element 2i in the low
 *        nibble of byte i and element 2i+1 in the high nibble;
 *      scales [page_size][D/32]: OCP MX E8M0 exponents, byte g scaling
 *        elements [32g, 32g+32). 0xFF (NaN) must not occur.
 *    (Source: sparse_indexer.py, builder __init__: the MXFP4 indexer cache
 *    with UE8M0-packed granularity-32 scales.)
 *  - Contiguous K workspace (prefill): values [total_len][D/2] and scales
 *    [total_len][D/32] with the same encodings. This is the layout the
 *    gather writes. (Source: sparse_mqa_indexer docs,
 *    _prefill_k_workspaces.)
 *  - Candidate blocks: [rows][candidate_topk_blocks] int32 block ids, in
 *    units of candidate_block_size tokens, relative to the row's ks.
 *    Negative ids name no block. Blocks at or past the row's end are
 *    masked.
 */
#ifndef SMQ_H
#define SMQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SMQ_API __attribute__((visibility("default")))

typedef enum smq_status {
  SMQ_OK = 0,
  SMQ_ERR_INVALID_ARG = 1,         /* null or misaligned pointer, bad size */
  SMQ_ERR_UNSUPPORTED = 2,         /* shape or device this library cannot run */
  SMQ_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes < smq_workspace_size() */
  SMQ_ERR_CUDA = 4,                /* a CUDA runtime or driver call failed */
  SMQ_ERR_BOUNDS = 8,              /* device: page / row / block id out of range */
  SMQ_ERR_TIMEOUT = 16,            /* device: a pipeline wait gave up */
  SMQ_ERR_NO_PAGES = 32            /* device: a page was wanted and none was free */
} smq_status;

typedef struct smq_plan smq_plan;

/* Geometry fixed at engine start. (Source: sparse_indexer.py, builder
 * __init__: the hf config's candidate_block_size, candidate_topk_blocks and
 * index_topk; the page size of the indexer cache spec; and
 * pick_sparse_block_kv / check_deep_select_layout.) */
typedef struct smq_plan_desc {
  uint32_t struct_size;
  int32_t num_heads;             /* H: a multiple of 8 in [8, 128] */
  int32_t head_dim;              /* D: must be 128 */
  int32_t page_size;             /* tokens per cache page: a multiple of sparse_block_kv */
  int32_t candidate_block_size;  /* cbs > 0 */
  int32_t candidate_topk_blocks; /* ncb > 0 candidate blocks per row */
  int32_t topk;                  /* k: 1 <= k <= num_sparse_cols, k <= 16384 */
  int32_t sparse_block_kv;       /* sub-block size in tokens: 16, 32, 64 or 128 (else
                                    SMQ_ERR_UNSUPPORTED); 0 picks the largest of
                                    128/64/32/16 dividing both page_size and cbs */
  int32_t max_rows;              /* upper bound on rows per call (workspace sizing), <= 8192 */
  int32_t device;                /* CUDA device ordinal the plan runs on */
} smq_plan_desc;

/* Values derived at plan creation. */
typedef struct smq_plan_info {
  uint32_t struct_size;
  int32_t sparse_block_kv;   /* tokens per sparse sub-block */
  int32_t num_sparse_blocks; /* per row: ncb * (cbs / sparse_block_kv) */
  int32_t num_sparse_cols;   /* S = num_sparse_blocks * sparse_block_kv */
  int32_t page_bytes;        /* bytes per K-cache page */
  int32_t num_sms;           /* SM count of the plan's device */
} smq_plan_info;

/* Validate the descriptor and create a plan. It reads the device's SM
 * count and does no GPU work. The plan is host memory owned by the caller
 * until smq_plan_destroy. Returns SMQ_ERR_INVALID_ARG or
 * SMQ_ERR_UNSUPPORTED for a geometry this library does not run. */
SMQ_API int smq_plan_create(const smq_plan_desc *desc, smq_plan **plan);
SMQ_API int smq_plan_destroy(smq_plan *plan);
SMQ_API int smq_plan_get_info(const smq_plan *plan, smq_plan_info *info);

/* Failure-path controls of later calls with this plan (host side; not
 * thread-safe with calls in flight on other threads).
 *  - smq_plan_set_wait_limit: every pipeline wait gives up after ns
 *    nanoseconds (default 2e9) and raises SMQ_ERR_TIMEOUT; the kernel then
 *    winds down: it waits, bounded, for its own copies in flight, drains its
 *    MMAs and frees its TMEM.
 *  - smq_plan_inject_stall: for tests of that path. The loaders of the first
 *    CTA of the score kernel withhold the hand-off of its tile `tile` to the
 *    MMA, so that the MMA's wait runs out. -1 (the default) withholds
 *    nothing. The outputs of a stalled call are unspecified; zero the
 *    workspace (smq_workspace_init) before the next call. */
SMQ_API int smq_plan_set_wait_limit(smq_plan *plan, int64_t ns);
SMQ_API int smq_plan_inject_stall(smq_plan *plan, int32_t tile);

/* Device workspace bytes for calls of up to `rows` rows (<= max_rows).
 * It holds the status word, one tile counter per plan row (decode calls that
 * expand their rows in the score kernel also select their top-k there; the
 * counters find the CTA that finishes a row) and the fp32 logits scratch
 * [rows][S]. Allocate it once, then zero it with smq_workspace_init. A call
 * leaves the counters at zero; after a call whose status reports an error,
 * zero the workspace again before the next call. */
SMQ_API int smq_workspace_size(const smq_plan *plan, int32_t rows, size_t *bytes);

/* Device workspace bytes for prefill chunks of up to `rows` rows and
 * `total_len` workspace rows. It adds to smq_workspace_size(plan, rows) the
 * scratch of the window-major prefill path: per workspace position a window
 * count and a cursor (int32 each), per row a record count and its 64 head
 * weights and q_scale as float, per (row, window) pair a record (8 bytes) and
 * a group slot (32 bytes per two records). The path applies to 64-head plans
 * and total_len <= 2^20; otherwise the size equals smq_workspace_size.
 * A prefill call whose workspace is smaller than this (but at least
 * smq_workspace_size) runs the row-major path instead; both give the same
 * logits, bit for bit, and the same top-k. Errors: SMQ_ERR_INVALID_ARG for a
 * null plan or bytes, rows < 0 or > max_rows, total_len < 0. */
SMQ_API int smq_prefill_workspace_size(const smq_plan *plan, int32_t rows, int64_t total_len, size_t *bytes);

/* Zero the workspace status word and tile counters (async on stream). */
SMQ_API int smq_workspace_init(const smq_plan *plan, void *workspace, size_t workspace_bytes,
                               void *stream);

/* Synchronise `stream`, read the workspace status word into *code (a
 * bitwise OR of SMQ_ERR_BOUNDS / SMQ_ERR_TIMEOUT / SMQ_ERR_NO_PAGES, or 0),
 * then clear it. */
SMQ_API int smq_get_status(const void *workspace, void *stream, int32_t *code);

SMQ_API const char *smq_error_string(int code);

/* Shared per-step candidate expansion. (Source: sparse_indexer.py,
 * SparseMQARowsMetadata and the module docstring: the first consumer layer
 * of a step fills sparse_indices / end, and later consumer layers reuse
 * them.)
 * For each row, with L = row_ke - row_ks:
 *  - drop negative blocks and blocks starting at or past L;
 *  - sort the rest ascending without repeats;
 *  - split each into cbs/sbkv sub-blocks, dropping sub-blocks that start at
 *    or past L.
 * Outputs (device memory):
 *  - sparse_indices [rows][num_sparse_blocks] int32: sub-block ids in units
 *    of sbkv tokens, relative to row_ks, then -1 padding.
 *  - end [rows] int32: the number of valid sparse columns. Every sparse
 *    column c < end is a key position, and only the last kept sub-block
 *    can be partial.
 * Inputs (device memory):
 *  - candidate_blocks [rows][ncb] int32;
 *  - row_ks [rows] int32, or NULL for all zeros (paged decode);
 *  - row_ke [rows] int32.
 * rows may be 0, which enqueues nothing. */
SMQ_API int sparse_mqa_candidate_expand(const smq_plan *plan, const int32_t *candidate_blocks,
                                        const int32_t *row_ks, const int32_t *row_ke,
                                        int32_t rows, int32_t *sparse_indices, int32_t *end,
                                        void *workspace, size_t workspace_bytes, void *stream);

/* Paged decode: one query row per decode token. (Source: sparse_mqa_indexer
 * docs, SparseMQAIndexer.forward, the sparse_mqa_logits_paged_decode call;
 * sparse_indexer.py, SparseMQARowsMetadata and build(): row_ks is zero for
 * paged decode, row_ke is the compressed context length, block_table is
 * [rows, pages], and row_indices maps row -> request.) */
typedef struct smq_decode_args {
  uint32_t struct_size;
  int32_t rows;                   /* R >= 0 */
  const uint8_t *q;               /* device [R][H][D] E4M3 */
  const float *q_scale;           /* device [R] */
  const uint16_t *weights;        /* device [R][H] bf16 */
  const uint8_t *k_cache;         /* device [num_pages][page_bytes], 16-byte aligned (32-byte
                                    aligned lets rows that share pages use tensor copies) */
  int64_t num_pages;
  const int32_t *block_table;     /* device [bt_rows][bt_stride] page ids */
  int32_t bt_rows;
  int32_t bt_stride;              /* columns of block_table */
  const int32_t *row_indices;     /* device [R] row -> block-table row, or NULL = identity */
  const int32_t *row_ke;          /* device [R] context length of the row */
  const int32_t *candidate_blocks;/* device [R][ncb] */
  int32_t *topk_out;              /* device [R][topk_ld]; columns [0, topk) are written */
  int32_t topk_ld;                /* >= topk */
  int32_t *sparse_indices;        /* device [R][num_sparse_blocks]: written if !expansion_ready */
  int32_t *end;                   /* device [R]: written if !expansion_ready */
  int32_t expansion_ready;        /* 1: sparse_indices / end already hold this step's expansion */
  int32_t *col_indices;           /* device [R][topk] selected sparse columns, or NULL */
  float *logits_out;              /* device [R][S] fp32 logits by sparse column (columns >= end
                                     are -inf), or NULL */
  void *workspace;                /* device, >= smq_workspace_size(plan, R) bytes */
  size_t workspace_bytes;
  void *profile_events[4];        /* optional cudaEvent_t, recorded on the stream before the
                                     expansion, before the gather+score kernel, before the top-k
                                     and after it; NULL entries are skipped */
  uint16_t *logits_out_bf16;      /* device [R][S] bf16 logits by sparse column, each the fp32
                                     logit rounded to the nearest-even bf16 (columns >= end are
                                     -inf), or NULL. The top-k still selects on the fp32 logits.
                                     Read only when struct_size covers it. (Source:
                                     sparse_indexer.py, builder __init__: DeepSelect takes bf16
                                     logits.) */
} smq_decode_args;

SMQ_API int sparse_mqa_logits_topk_decode(const smq_plan *plan, const smq_decode_args *args,
                                          void *stream);

/* Paged decode for callers that cannot allocate device memory, for
 * example code running where cudaMalloc is forbidden or where memory is
 * owned by another allocator (a graph-replay engine or a runtime that hands
 * out only its own tensors). The pages have no counterpart to this call.
 *
 * It does what sparse_mqa_logits_topk_decode does, with the same arguments,
 * except that args->workspace must be NULL and args->workspace_bytes 0. The
 * library uses its own scratch instead: a static device array of 256 bytes
 * plus 8 MiB (SMQ_NOALLOC_SCRATCH_BYTES) for the tile counters and the fp32
 * logits, held on every GPU that loads the library until the process exits.
 *  - The counters (4 bytes per plan row, rounded up to 256) plus
 *    rows * num_sparse_cols * 4 must not exceed 8 MiB, for example 200 rows
 *    of 8192 columns. A larger call returns SMQ_ERR_WORKSPACE_TOO_SMALL and
 *    enqueues nothing. The limit holds whether or not logits_out is given.
 *  - The first call on a device looks up the scratch's device address
 *    (cudaGetSymbolAddress) with that device current. Make that first call
 *    before any stream capture.
 *  - Every call shares the one scratch: calls that overlap on the GPU (on
 *    different streams without ordering) race. Each call zeroes the scratch
 *    status word and counters first.
 *  - Device-detected errors (bad page or row ids, timeouts) are recorded in
 *    the scratch and not returned. Callers who need them use
 *    sparse_mqa_logits_topk_decode with a workspace.
 * It calls no cudaMalloc, cudaFree or allocating routine. */
#define SMQ_NOALLOC_SCRATCH_BYTES (8u << 20)
SMQ_API int sparse_mqa_logits_topk_decode_noalloc(const smq_plan *plan, const smq_decode_args *args,
                                                  void *stream);

/* One prefill chunk on a contiguous K workspace. (Source: sparse_mqa_indexer
 * docs, SparseMQAIndexer.forward, the sparse_mqa_logits_prefill_chunk call
 * with cu_seqlen_ks / cu_seqlen_ke.) Row r's keys are workspace rows
 * [cu_seqlen_ks[r], cu_seqlen_ke[r]). Its candidate blocks and output ids
 * are relative to cu_seqlen_ks[r].
 * With a workspace of smq_prefill_workspace_size(plan, R, total_len) bytes
 * (64-head plans) the chunk runs window-major: the rows are indexed by the
 * 128-key windows [ks + 128 u, ks + 128 u + 128) their sparse sub-blocks fall
 * in, and each window's keys stay in shared memory while the query tiles of
 * the rows that selected it stream past. Four kernels then run before the
 * top-k: record, plan and fill of the index, and the score (plus one memset
 * of the window counts); profile_events[1] is recorded after the index. */
typedef struct smq_prefill_args {
  uint32_t struct_size;
  int32_t rows;
  const uint8_t *q;               /* device [R][H][D] E4M3 */
  const float *q_scale;           /* device [R] */
  const uint16_t *weights;        /* device [R][H] bf16 */
  const uint8_t *k_values;        /* device [total_len][D/2], 32-byte aligned */
  const uint8_t *k_scales;        /* device [total_len][D/32], 4-byte aligned */
  int64_t total_len;
  const int32_t *cu_seqlen_ks;    /* device [R] */
  const int32_t *cu_seqlen_ke;    /* device [R] */
  const int32_t *candidate_blocks;/* device [R][ncb] */
  int32_t *topk_out;
  int32_t topk_ld;
  int32_t *sparse_indices;
  int32_t *end;
  int32_t expansion_ready;
  int32_t *col_indices;
  float *logits_out;
  void *workspace;
  size_t workspace_bytes;
  void *profile_events[4];        /* as in smq_decode_args */
  uint16_t *logits_out_bf16;      /* as in smq_decode_args */
} smq_prefill_args;

SMQ_API int sparse_mqa_logits_topk_prefill_chunk(const smq_plan *plan, const smq_prefill_args *args,
                                                 void *stream);

/* Paged -> contiguous K gather for a prefill chunk. (Source:
 * sparse_mqa_indexer docs, _gather_prefill_chunk_k:
 * cp_gather_indexer_k_quant_cache with the chunk's block_table and
 * local_cu_seq_lens.) Sequence s occupies workspace rows
 * [cu_seq_lens[s], cu_seq_lens[s+1]). Its position p comes from page
 * block_table[s][p / page_size].
 *  - block_table: device [num_seqs][bt_stride].
 *  - cu_seq_lens: device [num_seqs + 1], non-decreasing, with
 *    cu_seq_lens[num_seqs] == total_len.
 *  - k_values: device [total_len][D/2]. k_scales: device [total_len][D/32].
 * An out-of-range page raises SMQ_ERR_BOUNDS in the workspace status word,
 * and that position is left unwritten. */
SMQ_API int sparse_mqa_gather_k(const smq_plan *plan, const uint8_t *k_cache, int64_t num_pages,
                                const int32_t *block_table, int32_t bt_stride,
                                const int32_t *cu_seq_lens, int32_t num_seqs, int64_t total_len,
                                uint8_t *k_values, uint8_t *k_scales, void *workspace,
                                size_t workspace_bytes, void *stream);

/* The candidate source of two-level selection, on paged decode rows: a
 * dense indexer over each row's whole context [0, row_ke) that publishes the
 * row's best candidate blocks for the consumer calls above. (Source:
 * sparse_mqa_indexer docs, module docstring: the candidate-source indexer
 * publishes the top candidate blocks and later indexers pick their top-k
 * inside them; rocm_paged_mxfp4_indexer docs, RocmSparseAttnIndexer: the
 * source layer publishes its candidate pool, candidate_write.) The pages do
 * not define a block's score. This library's: block b (positions
 * [b * cbs, (b + 1) * cbs) below row_ke) scores its largest logit, the
 * logit being the one the consumer calls compute. Each row publishes its
 * candidate_topk_blocks best blocks, best first, ties to the lower block id,
 * then -1 when the context has fewer blocks. */
typedef struct smq_source_args {
  uint32_t struct_size;
  int32_t rows;                   /* R >= 0 */
  const uint8_t *q;               /* device [R][H][D] E4M3 */
  const float *q_scale;           /* device [R] */
  const uint16_t *weights;        /* device [R][H] bf16 */
  const uint8_t *k_cache;         /* device [num_pages][page_bytes], 16-byte aligned */
  int64_t num_pages;
  const int32_t *block_table;     /* device [bt_rows][bt_stride] */
  int32_t bt_rows;
  int32_t bt_stride;
  const int32_t *row_indices;     /* device [R] row -> block-table row, or NULL = identity */
  const int32_t *row_ke;          /* device [R] context length; a longer context than max_context
                                     raises SMQ_ERR_BOUNDS and is cut there */
  int32_t max_context;            /* the longest context of the call, 1 .. 1048576 */
  int32_t *candidate_blocks;      /* device [R][candidate_topk_blocks] out */
  float *block_scores;            /* device [R][ceil(max_context / cbs)] out (-inf past a row's
                                     blocks), or NULL */
  void *workspace;                /* device, >= smq_source_workspace_size(plan, R, max_context) */
  size_t workspace_bytes;
} smq_source_args;

/* Workspace bytes of a candidate-source call: the status word, the dense
 * layout of the rows and their fp32 logits [rows][max_context rounded up
 * to whole blocks]. Zero it with smq_workspace_init before the first call.
 * ceil(max_context / cbs) may not exceed 8192. */
SMQ_API int smq_source_workspace_size(const smq_plan *plan, int32_t rows, int32_t max_context, size_t *bytes);

SMQ_API int sparse_mqa_candidate_source_decode(const smq_plan *plan, const smq_source_args *args,
                                               void *stream);

/* Producers of the indexer's inputs. (Source: sparse_mqa_indexer docs,
 * SparseMQAIndexer and weights_dtype: the model writes the MXFP4 indexer K
 * cache, and a fused query kernel writes the FP8 query, its scale and the
 * bf16 weights; sparse_indexer.py, builder __init__: MXFP4 with UE8M0-packed
 * granularity-32 scales.) The pages fix the formats but not the rounding.
 * This library's rounding:
 *  - K, per group of 32 elements: the scale exponent e is the smallest
 *    integer with amax <= 6 * 2^e, stored as the UE8M0 code e + 127 clamped
 *    to [1, 254] (a group of zeros: 127). Each element x * 2^-e rounds to the
 *    nearest E2M1 value, ties to even, saturating at 6.
 *  - Q, per row: scale = amax / 448 (1 for a row of zeros). Each element
 *    x / scale (float division) rounds to the nearest E4M3 value, ties to
 *    even, saturating at 448.
 *  - weights: float to the nearest-even bfloat16.
 * The sign of an element that rounds to zero is kept. Inputs must be finite.
 * RoPE, which the pages' fused query kernel also applies, is not defined on
 * the pages and is not part of this call. */

/* Write ntok keys into the paged K cache (layout at the top of this file).
 *  - k: device [ntok][D] bfloat16 bits, 16-byte aligned.
 *  - slot_mapping: device [ntok] int64. Token t goes to page
 *    slot_mapping[t] / page_size, row slot_mapping[t] % page_size; a negative
 *    slot skips the token.
 *  - k_cache: device [num_pages][page_bytes], 16-byte aligned.
 * A slot past the cache raises SMQ_ERR_BOUNDS in the workspace status word
 * (at least smq_workspace_size(plan, 0) bytes), and that token is skipped.
 * Tokens that share a slot race. ntok may be 0. */
SMQ_API int sparse_mqa_write_k_cache(const smq_plan *plan, const uint16_t *k, const int64_t *slot_mapping,
                                     int64_t ntok, uint8_t *k_cache, int64_t num_pages, void *workspace,
                                     size_t workspace_bytes, void *stream);

/* Quantise `rows` query rows and their head weights.
 *  - q: device [rows][H][D] bfloat16 bits, 16-byte aligned.
 *  - weights: device [rows][H] float.
 *  - q_fp8: device [rows][H][D] E4M3 out, 16-byte aligned. q_scale: device
 *    [rows] float out. weights_bf16: device [rows][H] bfloat16 bits out.
 * These are the q, q_scale and weights of the decode and prefill calls.
 * rows may be 0. */
SMQ_API int sparse_mqa_quantize_q(const smq_plan *plan, const uint16_t *q, const float *weights, int32_t rows,
                                  uint8_t *q_fp8, float *q_scale, uint16_t *weights_bf16, void *stream);

/* ---------------------------------------------------------------------------
 * The attention that consumes the indexer's token ids, over its own paged
 * key-value cache: three operators that share one plan and one cache.
 *   sparse_mqa_append_kv          rotate a step's queries and keys by their
 *                                 positions; write keys and values into the cache
 *   sparse_mqa_attention_decode   one query row over its cached range [ks, ke)
 *   sparse_mqa_attention_selected one query row over selected token ids
 * (Source: sparse_mqa_indexer docs, SparseMQAIndexer: the layer returns the
 * top-k token ids to the attention layer, which reads them. The pages do not
 * show that layer; the formulas are the textbook ones.)
 *
 * With H query heads on KVH key-value heads, query head h reads key-value
 * head h / (H / KVH). For a row with queries q[h] and a set of tokens T,
 *     s[h][t] = softmax_scale * q[h] . k[t]
 *     out[h]  = sum_t exp(s[h][t] - lse[h]) v[t],  lse[h] = log sum_t exp(s[h][t]).
 * A row without tokens, or a head without a score above -infinity, gets
 * out = 0 and lse = -infinity. Products are of the
 * bfloat16 queries and the cache's elements as they are; sums, maxima and
 * scores are fp32; a weight (times its token's value scale) enters the sum of
 * the values with 16 bits, whatever the other tokens' scales are. Keys and
 * values of tokens outside T are never used, whatever they hold. An infinite
 * value makes its element of out infinite, or NaN where its token's weight is
 * too small for fp32; a score of +infinity or NaN makes out[h] and lse[h] NaN.
 * Finite values stay below 2^100, so that unnormalised sums are finite.
 *
 * The cache: keys and values are two arrays of pages [KVH][page_size][D],
 * page p at base + p * page_stride elements, so that both may be views of one
 * allocation. Elements are bfloat16, or E4M3 codes with one positive float
 * scale per token, kv head and side: [KVH][page_size] floats, page p at
 * scales + p * scale_page_stride.
 * --------------------------------------------------------------------------- */
typedef struct smq_attn_plan smq_attn_plan;

enum { SMQ_CACHE_BF16 = 0, SMQ_CACHE_E4M3 = 1 };

typedef struct smq_attn_plan_desc {
  uint32_t struct_size;
  int32_t num_heads;     /* H: a multiple of num_kv_heads, <= 1024, H / KVH <= 128 */
  int32_t num_kv_heads;  /* KVH: 1 .. 128 */
  int32_t head_dim;      /* D: 64 or 128 */
  int32_t page_size;     /* tokens per page, 1 .. 65536 */
  int32_t cache_type;    /* SMQ_CACHE_BF16 or SMQ_CACHE_E4M3 */
  int32_t max_rows;      /* upper bound on rows per call, <= 8192 */
  int32_t device;        /* CUDA device ordinal the plan runs on */
  float softmax_scale;   /* finite; 0 picks 1 / sqrt(D) */
  int32_t max_sequence_rows; /* upper bound on rows and sequences of a window or tree call below, <= 1048576; an append
                                takes as many rows as the larger bound. 0, or a struct_size that ends before it: max_rows */
} smq_attn_plan_desc;

/* As smq_plan_create / destroy / set_wait_limit / inject_stall: host memory
 * only, geometry checked once. inject_stall withholds the hand-off of the
 * first CTA's tile `tile` (a tile is 128 tokens). */
SMQ_API int smq_attn_plan_create(const smq_attn_plan_desc *desc, smq_attn_plan **plan);
SMQ_API int smq_attn_plan_destroy(smq_attn_plan *plan);
SMQ_API int smq_attn_plan_set_wait_limit(smq_attn_plan *plan, int64_t ns);
SMQ_API int smq_attn_plan_inject_stall(smq_attn_plan *plan, int32_t tile);

/* Device workspace bytes of every call with this plan: the status word and
 * the partial results of rows whose tokens several CTAs share. It does not
 * depend on rows or lengths. Zero the status word with
 * smq_attn_workspace_init; smq_get_status reads it. Calls that overlap on the
 * GPU need workspaces of their own. */
SMQ_API int smq_attn_workspace_size(const smq_attn_plan *plan, size_t *bytes);
SMQ_API int smq_attn_workspace_init(const smq_attn_plan *plan, void *workspace, size_t workspace_bytes,
                                    void *stream);

/* Rotate and append. Token t's query and key elements in the first rot_dim
 * places of a head turn by the angles of row positions[t] of cos_sin: pair i
 * (i < rot_dim / 2) is (i, i + rot_dim / 2), or (2 i, 2 i + 1) with
 * interleaved, and becomes (a c - b s, b c + a s) with c = cos_sin[i] and
 * s = cos_sin[rot_dim / 2 + i]. The other elements and the values pass
 * unchanged. Each product and sum rounds to fp32, then once to the nearest-even
 * bfloat16 for queries and a bfloat16 cache. An E4M3 cache takes, per token,
 * kv head and side, scale = amax / 448 (1 for zeros; both in float) and
 * x / scale to the nearest E4M3 value, ties to even: the rounding of
 * sparse_mqa_quantize_q. Inputs to an E4M3 cache must be finite. */
typedef struct smq_append_args {
  uint32_t struct_size;
  int32_t rows;               /* tokens, 0 .. the larger of the plan's max_rows and max_sequence_rows */
  const uint16_t *q;          /* device bf16, row t at q + t * q_stride: [H][D], 16-byte aligned; or NULL */
  const uint16_t *k;          /* device bf16, row t at k + t * k_stride: [KVH][D], 16-byte aligned */
  const uint16_t *v;          /* device bf16, row t at v + t * v_stride: [KVH][D], 16-byte aligned */
  int64_t q_stride;           /* elements, multiples of 8, at least a row's */
  int64_t k_stride;
  int64_t v_stride;
  const int64_t *positions;   /* device [rows]; one outside the table raises SMQ_ERR_BOUNDS and skips
                                 the token's query, key and value */
  const float *cos_sin;       /* device [num_positions][rot_dim]: cosines, then sines; 16-byte aligned */
  int64_t num_positions;
  int32_t rot_dim;            /* a multiple of 16, 0 .. D (0: no rotation, positions and cos_sin unread) */
  int32_t interleaved;
  const int64_t *slot_mapping;/* device [rows]: page slot / page_size, place slot % page_size. A negative
                                 slot skips the key and value; one past the cache also raises
                                 SMQ_ERR_BOUNDS. Tokens that share a slot race. */
  uint16_t *q_out;            /* device [rows][H][D] bf16, 16-byte aligned; NULL exactly when q is. It may
                                 not overlap q. */
  void *k_cache;              /* device pages, 16-byte aligned */
  void *v_cache;
  float *k_scales;            /* device scales of an E4M3 cache, else NULL */
  float *v_scales;
  int64_t num_pages;
  int64_t page_stride;        /* elements, >= KVH * page_size * D, a multiple of 16 */
  int64_t scale_page_stride;  /* floats, >= KVH * page_size (E4M3) */
  void *workspace;            /* device, the status word: at least 256 bytes */
  size_t workspace_bytes;
} smq_append_args;

SMQ_API int sparse_mqa_append_kv(const smq_attn_plan *plan, const smq_append_args *args, void *stream);

/* Attention rows. sparse_mqa_attention_decode takes T = the positions
 * [row_ks, row_ke) of the row's sequence (row_ks NULL or negative: zero; a
 * window of a sliding layer otherwise). sparse_mqa_attention_selected takes T = the
 * non-negative entries of token_ids[row][0 .. num_ids), positions in the row's
 * sequence such as topk_out of the indexer calls; -1 entries may stand
 * anywhere and an id listed twice counts twice. A position's page is
 * block_table[row_indices[row]][position / page_size]. A position past the
 * block table, or a page or table row out of range, raises SMQ_ERR_BOUNDS and
 * is left out. */
typedef struct smq_attention_args {
  uint32_t struct_size;
  int32_t rows;               /* R >= 0 */
  const uint16_t *q;          /* device bf16, row r at q + r * q_stride: [H][D], 16-byte aligned */
  int64_t q_stride;           /* elements, a multiple of 8, >= H * D */
  const void *k_cache;        /* device pages, 16-byte aligned */
  const void *v_cache;
  const float *k_scales;      /* device scales of an E4M3 cache, else NULL */
  const float *v_scales;
  int64_t num_pages;
  int64_t page_stride;        /* elements, >= KVH * page_size * D, a multiple of 16 */
  int64_t scale_page_stride;  /* floats, >= KVH * page_size (E4M3) */
  const int32_t *block_table; /* device [bt_rows][bt_stride] page ids */
  int32_t bt_rows;
  int32_t bt_stride;
  const int32_t *row_indices; /* device [R] row -> block-table row, or NULL = identity */
  const int32_t *row_ks;      /* decode: device [R] first position, or NULL; selected: NULL */
  const int32_t *row_ke;      /* decode: device [R] end position; selected: NULL */
  const int32_t *token_ids;   /* selected: device [R][ids_ld]; decode: NULL */
  int32_t num_ids;            /* selected: 1 .. 1048576 */
  int32_t ids_ld;             /* selected: >= num_ids */
  uint16_t *out;              /* device [R][H][D] bf16, 16-byte aligned */
  float *lse;                 /* device [R][H] natural log-sum-exp, or NULL */
  void *workspace;            /* device, >= smq_attn_workspace_size(plan), 16-byte aligned */
  size_t workspace_bytes;
} smq_attention_args;

SMQ_API int sparse_mqa_attention_decode(const smq_attn_plan *plan, const smq_attention_args *args, void *stream);
SMQ_API int sparse_mqa_attention_selected(const smq_attn_plan *plan, const smq_attention_args *args, void *stream);

/* ---------------------------------------------------------------------------
 * Attention of whole sequences' query rows over the same cache: several rows
 * of a sequence share its keys and values.
 *   sparse_mqa_attention_window  causal, with a sliding window and a few first
 *                                tokens that stay visible (sinks): prefill
 *                                chunks and decode steps of a sliding layer
 *   sparse_mqa_attention_tree    a tree of drafted tokens: each row sees the
 *                                context and its own ancestors
 * Formulas, heads, cache and the treatment of infinities and NaN are those of
 * sparse_mqa_attention_decode above; only the sets T differ. A weight enters
 * the sum of the values with the 8 bits of a bfloat16. Keys and values of
 * tokens that a row does not see are never used for it, whatever they hold,
 * also where another row of the same sequence sees them.
 *
 * Sequence b has the query rows cu_rows[b] .. cu_rows[b + 1] - 1, in order, and
 * seq_len[b] tokens in the cache, the tokens of those rows included: row i of n
 * is the token at position seq_len[b] - n + i. Its pages are those of table row
 * seq_indices[b] (b where NULL).
 *   window: T = { t <= position : t < sinks or t > position - window }.
 *   tree:   T = { t < seq_len - n } and { seq_len - n + j : bit j of the row's
 *           mask }: bit j % 32 of word j / 32. A row sees its own token only if
 *           its own bit says so; bits past n are not read.
 * Tokens before position 0 do not exist; a row at a negative position of a
 * window sees nothing. Rows at or past cu_rows[num_seqs] belong to no sequence
 * and their out and lse are left as they were, as are those of a sequence that
 * is refused: a sequence whose rows decrease, pass `rows` or are more than
 * max_seq_rows raises SMQ_ERR_BOUNDS. A position past the block table, or a
 * page or table row out of range (such as -1 for a page that was given back),
 * where a row would see it, raises SMQ_ERR_BOUNDS and is left out.
 * --------------------------------------------------------------------------- */
typedef struct smq_seq_attention_args {
  uint32_t struct_size;
  int32_t rows;               /* rows of q, out and lse, 0 .. the plan's max_sequence_rows */
  const uint16_t *q;          /* device bf16, row r at q + r * q_stride: [H][D], 16-byte aligned */
  int64_t q_stride;           /* elements, a multiple of 8, >= H * D */
  const void *k_cache;        /* device pages, 16-byte aligned */
  const void *v_cache;
  const float *k_scales;      /* device scales of an E4M3 cache, else NULL */
  const float *v_scales;
  int64_t num_pages;
  int64_t page_stride;        /* elements, >= KVH * page_size * D, a multiple of 16 */
  int64_t scale_page_stride;  /* floats, >= KVH * page_size (E4M3) */
  const int32_t *block_table; /* device [bt_rows][bt_stride] page ids */
  int32_t bt_rows;
  int32_t bt_stride;
  int32_t num_seqs;           /* sequences, 0 .. the plan's max_sequence_rows */
  int32_t max_seq_rows;       /* no sequence has more rows: 1 .. the plan's max_sequence_rows */
  const int32_t *seq_indices; /* device [num_seqs] sequence -> block-table row, or NULL = identity */
  const int32_t *cu_rows;     /* device [num_seqs + 1] */
  const int32_t *seq_len;     /* device [num_seqs] */
  int32_t window;             /* window call: tokens that a row sees, its own included, >= 1; tree: 0 */
  int32_t sinks;              /* window call: first tokens that stay visible, >= 0; tree: 0 */
  const int32_t *tree_mask;   /* tree call: device [rows][mask_words]; window: NULL */
  int32_t mask_words;         /* tree call: 1 .. 32, max_seq_rows <= 32 * mask_words; window: 0 */
  uint16_t *out;              /* device [rows][H][D] bf16, 16-byte aligned */
  float *lse;                 /* device [rows][H] natural log-sum-exp, or NULL */
  void *workspace;            /* device, >= smq_seq_attention_workspace_size(plan), 16-byte aligned */
  size_t workspace_bytes;
} smq_seq_attention_args;

/* Device workspace bytes of the two calls: the status word and partial results.
 * It does not depend on rows or lengths. smq_attn_workspace_init zeroes its
 * status word. Calls that overlap on the GPU need workspaces of their own. */
SMQ_API int smq_seq_attention_workspace_size(const smq_attn_plan *plan, size_t *bytes);

SMQ_API int sparse_mqa_attention_window(const smq_attn_plan *plan, const smq_seq_attention_args *args, void *stream);
SMQ_API int sparse_mqa_attention_tree(const smq_attn_plan *plan, const smq_seq_attention_args *args, void *stream);

/* ---------------------------------------------------------------------------
 * The pages of the paged caches: who holds them, and what moves between them.
 *   sparse_mqa_pages_resize   take and give back pages, so that rows of the
 *                             block table cover the tokens they are to hold
 *   sparse_mqa_pages_fork     rows that share another row's pages
 *   sparse_mqa_cache_compact  move the kept tokens of rows together
 *
 * The state is the caller's, on the device: a block table [table_rows]
 * [table_columns] of page ids, -1 where a row has no page, and a count of
 * holders for each page, page_refs [num_pages]. A page is free where its count
 * is zero; a new state is a table of -1 and counts of 0. Column c of a row
 * holds the row's positions [c * page_size, (c + 1) * page_size). The attention
 * calls, the indexer's calls and the append read the same table.
 *
 * Results do not depend on timing: new pages are the lowest-numbered ones whose
 * count was zero before the call, given out in the order in which rows are
 * listed, then columns. A page that a call gives back is free for later calls,
 * not for the same one. Where too few pages are free, SMQ_ERR_NO_PAGES is
 * raised and the entries past the last page stay -1.
 *
 * Rows are listed: distinct rows of the table. One out of range, or listed
 * again, raises SMQ_ERR_BOUNDS and is skipped. Any negative entry is no page. An
 * entry past the pool, and a count that would pass below zero, raise
 * SMQ_ERR_BOUNDS and change no count; a call's additions come before its
 * subtractions, and a page whose count was zero before it cannot be given back.
 * --------------------------------------------------------------------------- */
typedef struct smq_page_plan smq_page_plan;

typedef struct smq_page_plan_desc {
  uint32_t struct_size;
  int32_t page_size;      /* tokens per page, 1 .. 65536 */
  int64_t num_pages;      /* pages of the pool, 1 .. 2^31 - 1 */
  int32_t table_rows;     /* rows of the block table, 1 .. 8192 */
  int32_t table_columns;  /* columns of the block table, 1 .. 1048576 */
  int32_t device;         /* CUDA device ordinal the plan runs on */
} smq_page_plan_desc;

SMQ_API int smq_page_plan_create(const smq_page_plan_desc *desc, smq_page_plan **plan);
SMQ_API int smq_page_plan_destroy(smq_page_plan *plan);

/* Device workspace bytes of every call with this plan. smq_page_workspace_init
 * zeroes the status word, smq_get_status reads it. Calls that overlap on the
 * GPU need workspaces of their own (and may not share a state). */
SMQ_API int smq_page_workspace_size(const smq_page_plan *plan, size_t *bytes);
SMQ_API int smq_page_workspace_init(const smq_page_plan *plan, void *workspace, size_t workspace_bytes, void *stream);

/* Row rows[i] (i where NULL) is to cover the positions [begin, end): begin =
 * row_begin[i] (0 where NULL), end = row_end[i], both as many as the table's
 * row holds at most (more raises SMQ_ERR_BOUNDS), negative as 0. Its columns are
 * those from begin / page_size up to the one that end ends in, so that an empty
 * range that begins inside a page, as of a window that has left all tokens
 * behind, holds that page, the next token's: begin >= end in the same page. The first
 * keep_first positions stay too, as far as they are below end: the sinks of a
 * sliding layer. Wanted columns without a page take one; the others give
 * theirs back and become -1. row_end = 0 frees a row. */
typedef struct smq_pages_resize_args {
  uint32_t struct_size;
  int32_t num_rows;           /* 0 .. table_rows */
  int32_t *block_table;       /* device [table_rows][table_columns], in and out */
  int32_t *page_refs;         /* device [num_pages], in and out */
  const int32_t *rows;        /* device [num_rows], or NULL */
  const int32_t *row_begin;   /* device [num_rows], or NULL */
  const int32_t *row_end;     /* device [num_rows] */
  int32_t keep_first;         /* >= 0 */
  void *workspace;            /* device, 16-byte aligned */
  size_t workspace_bytes;
} smq_pages_resize_args;

SMQ_API int sparse_mqa_pages_resize(const smq_page_plan *plan, const smq_pages_resize_args *args, void *stream);

/* One thing that a page holds: page p at base + p * page_stride bytes, as
 * `vectors` runs (kv heads) of page_size tokens of token_bytes bytes. Keys,
 * values and scales of an attention cache are planes with KVH vectors; the
 * indexer's MXFP4 pages are two planes of one vector each: values of 64 bytes a
 * token at offset 0 and scales of 4 bytes a token at offset 64 * page_size. */
typedef struct smq_page_plane {
  void *base;             /* device, 4-byte aligned */
  int64_t page_stride;    /* bytes, a multiple of 4, >= vectors * page_size * token_bytes */
  int32_t vectors;        /* 1 .. 1024 */
  int32_t token_bytes;    /* a multiple of 4, at most 2048 */
} smq_page_plane;

enum { SMQ_MAX_PLANES = 8 };

/* Fork i makes row dst_rows[i] one that shares the first row_len[i] tokens of
 * row src_rows[i], as the rows were before the call: it holds the source's
 * whole pages too, and a new page with a copy of the tokens of the page that
 * row_len[i] ends inside, in every plane. Its other entries become -1, and what
 * it held before is given back. Columns without a page at the source (given
 * back by a window) have none in the fork. Destinations are the listed rows;
 * sources may repeat, and may be destinations themselves, so beams can change
 * places. A row forked onto itself stays as it is. A row_len past the table's
 * row raises SMQ_ERR_BOUNDS and is cut there; a negative one is 0. */
typedef struct smq_pages_fork_args {
  uint32_t struct_size;
  int32_t num_rows;           /* 0 .. table_rows */
  int32_t *block_table;       /* device [table_rows][table_columns], in and out */
  int32_t *page_refs;         /* device [num_pages], in and out */
  const int32_t *src_rows;    /* device [num_rows] */
  const int32_t *dst_rows;    /* device [num_rows] */
  const int32_t *row_len;     /* device [num_rows] tokens */
  const smq_page_plane *planes; /* host [num_planes], read during the call */
  int32_t num_planes;         /* 0 .. SMQ_MAX_PLANES */
  void *workspace;            /* device, 16-byte aligned */
  size_t workspace_bytes;
} smq_pages_fork_args;

SMQ_API int sparse_mqa_pages_fork(const smq_page_plan *plan, const smq_pages_fork_args *args, void *stream);

/* In row rows[i] (i where NULL), token keep_ids[i][j] moves to position
 * row_start[i] + j, in every plane: the accepted path of a tree, the tokens
 * that an eviction keeps. keep_ids[i] ascends strictly, has its first entry at
 * or past row_start[i] >= 0, and ends at its first negative entry. Tokens that
 * move may come from places that others move to. The table does not change;
 * sparse_mqa_pages_resize gives back what is behind. A row is moved whole or
 * not at all: a list that does not ascend, a position past the table, a page out
 * of range or a destination page with more than one holder raises SMQ_ERR_BOUNDS,
 * and the row stays as it is. A page that two listed rows hold is only read. */
typedef struct smq_cache_compact_args {
  uint32_t struct_size;
  int32_t num_rows;           /* 0 .. table_rows */
  const int32_t *block_table; /* device [table_rows][table_columns] */
  const int32_t *page_refs;   /* device [num_pages] */
  const int32_t *rows;        /* device [num_rows], or NULL */
  const int32_t *row_start;   /* device [num_rows] */
  const int32_t *keep_ids;    /* device [num_rows][keep_ld] */
  int32_t num_keep;           /* 1 .. 1048576 */
  int32_t keep_ld;            /* >= num_keep */
  const smq_page_plane *planes; /* host [num_planes], read during the call; no two share bytes */
  int32_t num_planes;         /* 1 .. SMQ_MAX_PLANES */
  void *workspace;            /* device, 16-byte aligned */
  size_t workspace_bytes;
} smq_cache_compact_args;

SMQ_API int sparse_mqa_cache_compact(const smq_page_plan *plan, const smq_cache_compact_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SMQ_H */
