/*
 * idx.h - C ABI of the GB300 sparse-attention indexer decode library (libidx.so).
 *
 * One hot path: FP8 (E4M3) index queries are scored against a paged NVFP4
 * index-K cache, and an exact top-16 of pages is selected per (query slot,
 * index head).  Sources, by page and section:
 *
 *   [GATHER]  "vllm.models.minimax_m3.nvidia.ops.gather_nvfp4_index_k",
 *             module docstring and minimax_m3_gather_nvfp4_index_k_fp8.
 *   [CP]      "vllm.models.minimax_m3.nvidia.indexer_nvfp4_decode_cp",
 *             module docstring, _local_topk_push_kernel, _merge_kernel,
 *             _page_keys, _compact_block_table_kernel.
 *   [PUBLISH] "wolfcomos/MSA PR #1", sections Summary, Changes, Behaviour
 *             changes.
 *   [MTP]     "Mojo module sparse_index_fp8_sm100", module text.
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The
 *     library never allocates, frees or synchronises; it only enqueues
 *     kernels on `stream` (a cudaStream_t; NULL = the legacy default stream),
 *     so idx_dequant_nvfp4_pages, idx_score_pages, idx_topk16_select,
 *     idx_decode_step, idx_mtp_score_fp8, idx_prefill_index_step,
 *     idx_mxfp8_quantize, idx_build_slots, idx_rope_append,
 *     idx_tree_attention, idx_verify_drafts, idx_norm_rope_append,
 *     idx_index_append, idx_logit_probs, idx_settle_drafts, idx_fork_pages
 *     and idx_release_pages can sit inside CUDA-graph capture.
 *   - Return value: IDX_OK (0) when the work was enqueued (or there was
 *     nothing to do), else a negative IDX_E_* code; on an error nothing is
 *     launched.  Argument checks are on the host and never touch the GPU.
 *   - Empty work (zero requests, rows or pages) returns IDX_OK and launches
 *     nothing.
 *   - `status` (may be NULL) is a caller-zeroed int32 in device memory; the
 *     kernels OR IDX_ST_* bits into it for problems only the device can see
 *     (for example a block id out of range).  The affected page is skipped;
 *     no kernel traps.  Read it after the stream completes.
 *   - Fixed shapes: pages of 128 tokens, index head depth 128, 8 query slots
 *     and 4 index heads per request for the decode calls.
 */
#ifndef IDX_H
#define IDX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- return codes ---- */
#define IDX_OK 0
#define IDX_E_NULL_PTR (-1)        /* a required pointer is NULL */
#define IDX_E_BAD_SHAPE (-2)       /* a size or stride is negative or inconsistent */
#define IDX_E_MISALIGNED (-3)      /* a pointer lacks the alignment stated below */
#define IDX_E_WIDTH_TOO_SMALL (-4) /* score buffer narrower than the call needs */
#define IDX_E_TOO_LARGE (-5)       /* a size beyond the supported maximum */
#define IDX_E_CUDA (-6)            /* a CUDA runtime call or launch failed */
#define IDX_E_WORKSPACE (-7)       /* workspace missing or smaller than idx_workspace_bytes() */
#define IDX_E_DEVICE (-8)          /* the current device is not an sm_103 GPU */

/* ---- device status bits (OR-ed into *status) ---- */
#define IDX_ST_BLOCK_OOR 1   /* a block-table entry outside [0, num_blocks): page skipped */
#define IDX_ST_LEN_CLAMPED 2 /* a request held more pages than the table or buffer: clamped */
#define IDX_ST_BAD_OUTPUT 4  /* an output page index outside the output buffer: skipped */
#define IDX_ST_TIMEOUT 8     /* an internal pipeline wait gave up; that CTA's outputs are incomplete */
#define IDX_ST_NO_BLOCKS 16  /* the free list ran out: block ids and slots of -1 */
#define IDX_ST_BAD_TREE 32   /* a parent outside [-1, own index), or a drafted token past 64 in a tree */
#define IDX_ST_BAD_FORK 64   /* a fork whose child is a parent or another fork's child, or out of range: not made */

/* Fixed geometry. */
#define IDX_PAGE_TOKENS 128
#define IDX_HEAD_DIM 128
#define IDX_PAGE_BYTES 9216 /* 128 tokens x (64 code bytes + 8 scale bytes) */
#define IDX_SLOTS 8
#define IDX_INDEX_HEADS 4
#define IDX_TOPK 16

/* Text for a return code. */
const char* idx_strerror(int code);

/* 1 when the library was built with the QMUL4 dequant instruction
 * (mul.rn.satfinite.e4m3x4.e2m1x4.e4m3x4), 0 when it uses the exact
 * fp32-then-round-once path.  Both give identical bytes ([GATHER]). */
int idx_have_qmul4(void);

/*
 * Wait budget of the kernels that copy ahead of their work (the decode
 * scorer, the multi-token scorer, the tree attention and idx_logit_probs, which
 * waits for its rows).  The tensor-core kernels' warp roles hand pages to one another through
 * shared-memory barriers; every such wait gives up after `polls` suspended
 * polls of at most ~20 us each (spinning roles: polls * 1024 spins), records
 * IDX_ST_TIMEOUT in the status word, and the CTA winds down: it stops taking
 * pages, waits for its own copies and MMAs to land (those waits keep the
 * default budget) and frees its tensor memory, so the stream and the context
 * stay usable.  polls == 0 makes every pipeline wait a single test, so a
 * launch times out as soon as one stage is not ready at once; that is for
 * testing the timeout path.  The default is 100,000 (about 2 s).  The value
 * is process-wide, read when a kernel is launched (a graph keeps the value
 * it was captured with).  Returns the previous value.
 */
uint32_t idx_set_wait_limit(uint32_t polls);

/*
 * Bytes of scratch workspace idx_topk16_select needs for
 * `rows` rows of `width` columns (0 when rows fit one CTA each: up to 8,192
 * columns, 4,096 when there are few rows).  Longer rows are split across
 * CTAs whose local top-16s are merged exactly through this workspace ([CP]
 * module docstring: the global top 16 lies in the union of the partial top
 * 16s).
 */
size_t idx_workspace_bytes(int32_t rows, int32_t width);

/*
 * Gather + dequantise NVFP4 index-K pages into contiguous E4M3 pages [GATHER].
 *
 *   kv            [num_blocks, 128, 72] uint8, contiguous, 16-byte aligned.
 *                 Per page: 8,192 code bytes (token t's 64 bytes at t*64,
 *                 element d in byte t*64 + d/2, low nibble for even d), then
 *                 1,024 E4M3 scale bytes, scale (t, g) at 8192 + t*8 + g,
 *                 g = d/16.  No global scale.
 *   block_table   [num_reqs, bt_stride] int32; entries [0, max_blocks) used.
 *   num_pages     [num_reqs] int32: request r gathers its first
 *                 min(num_pages[r], max_num_pages, max_blocks) logical pages.
 *   page_offsets  [num_reqs] int32: first output page of request r.
 *   out           [out_pages, 128, 128] E4M3 bytes, contiguous, 16-byte aligned.
 *                 out[page_offsets[r] + p][t][d] =
 *                   e4m3_rn_satfinite(e2m1(code) * e4m3(scale)),
 *                 a NaN scale gives 0x7F.  Pages not gathered are untouched.
 * Device checks: block id out of range -> IDX_ST_BLOCK_OOR, output page out
 * of [0, out_pages) -> IDX_ST_BAD_OUTPUT; the page is skipped.
 */
int idx_dequant_nvfp4_pages(const uint8_t* kv, int64_t num_blocks, const int32_t* block_table,
                            int64_t bt_stride, int32_t max_blocks, const int32_t* num_pages,
                            const int32_t* page_offsets, int32_t num_reqs, int32_t max_num_pages,
                            uint8_t* out, int64_t out_pages, int32_t* status, void* stream);

/*
 * Decode page scores ([CP] module docstring: the Q8KV4 decode scorer's
 * contract; the page reduction is the max over the page's keys).
 *
 *   q             [num_reqs, 8, 4, 128] E4M3 bytes, contiguous, 16-byte aligned;
 *                 slot s of request b holds query i = s - (8 - query_len).
 *   q_scale       [num_reqs, 8, 4] float32.
 *   kv, num_blocks, block_table, bt_stride, max_blocks: as above.
 *   seq_lens      [num_reqs] int32 tokens per request (the own page included).
 *   query_len     1..8: the trailing query_len slots are live.
 *   width         columns of the score buffer.
 *   scores        [num_reqs, 32, width] float32, row = slot*4 + head.
 * For request b, pages j < n_b = clamp((seq_len-1)/128, 0, min(max_blocks,
 * width)) are scored (IDX_ST_LEN_CLAMPED when the clamp bit).  For slot s
 * (query i) with own page own = floor((seq_len - query_len + i) / 128),
 *     scores[b][s*4+h][j] = max_t fp32(q_scale[b][s][h] * (q[b][s][h] . K_j[t]))
 * is stored for j < own only; every other column is left untouched.  K_j is
 * page bt[b][j] dequantised exactly as in idx_dequant_nvfp4_pages.  A page
 * with a block id out of range stores NaN (ranked as -inf) and sets
 * IDX_ST_BLOCK_OOR.  The dot product is accumulated in fp32 on the tensor
 * cores; the result is within 1e-3 * max_t sum_d |q_scale q_d k_td| of the
 * exact value.
 */
int idx_score_pages(const uint8_t* q, const float* q_scale, const uint8_t* kv, int64_t num_blocks,
                    const int32_t* block_table, int64_t bt_stride, int32_t max_blocks,
                    const int32_t* seq_lens, int32_t num_reqs, int32_t query_len, int32_t width,
                    float* scores, int32_t* status, void* stream);

/*
 * Exact top-16 per row ([PUBLISH] Changes; [CP] _page_keys).
 *
 *   scores        [rows, row_stride] float32, 4-byte aligned; columns [0, width);
 *                 row_stride >= width (else IDX_E_BAD_SHAPE, whatever the row count).
 *   valid_n       [rows] int32 or NULL: row r ranks columns [0, min(valid_n[r], width));
 *                 NULL ranks all `width` columns.  Negative counts rank nothing.
 *   force_begin/end  columns in [force_begin, force_end) rank as +inf (empty if end <= begin).
 *   out_idx       [rows, 16] int32: columns by key descending, -1 padding.
 *   out_keys      [rows, 16] uint64 or NULL: the keys, 0 padding.  Key =
 *                 ordered(score) << 32 | (0xFFFFFFFF - column) with
 *                 ordered(x) = bits(x) ^ (sign ? 0xFFFFFFFF : 0x80000000),
 *                 after NaN -> -inf, -0 -> +0, forced -> +inf.  So rows sort by
 *                 score descending, ties to the lower column.
 *   workspace     device scratch of workspace_bytes >= idx_workspace_bytes(rows, width)
 *                 (may be NULL when that is 0).  Its contents need no initialisation.
 */
int idx_topk16_select(const float* scores, int64_t row_stride, int32_t rows, int32_t width,
                      const int32_t* valid_n, int32_t force_begin, int32_t force_end, int32_t* out_idx,
                      uint64_t* out_keys, void* workspace, size_t workspace_bytes, void* stream);

/*
 * idx_topk16_select without a caller workspace, for callers that cannot
 * allocate device memory (a plugin inside a framework that owns every
 * device allocation, a serving loop that allows no allocation after
 * start-up, a captured graph replayed without a memory pool).  The pages
 * have no counterpart to this entry point; it is a packaging of the
 * selector above.
 *
 * Same arguments and results as idx_topk16_select.  Rows that need more
 * split-row scratch than IDX_NOALLOC_SCRATCH_BYTES (4 MiB; see
 * idx_workspace_bytes) are rejected with IDX_E_TOO_LARGE.  The scratch is
 * a __device__ array inside the library: every GPU that loads the library
 * holds it until exit, every call shares it (it keeps the last call's
 * contents; nothing needs clearing), and calls that overlap on the GPU race
 * on it, so serialise them.  The first call in each CUDA context (for the
 * runtime, each device's primary context) looks up the array's address
 * (cudaGetSymbolAddress, with that device current) and caches it under the
 * context's unique id; a new context -- after cudaDeviceReset, or a context
 * the caller made current with the driver API -- is looked up afresh.  Make
 * the first call in a context before any stream capture.  No allocation
 * happens in any call.
 */
#define IDX_NOALLOC_SCRATCH_BYTES (4u << 20)
int idx_topk16_select_noalloc(const float* scores, int64_t row_stride, int32_t rows, int32_t width,
                              const int32_t* valid_n, int32_t force_begin, int32_t force_end, int32_t* out_idx,
                              uint64_t* out_keys, void* stream);

/*
 * One indexer decode step: idx_score_pages, then per (request, query, head)
 * the output row ([CP] _merge_kernel):
 *   own + 1 <= 16 : pages 0..own, then -1;
 *   otherwise     : the 15 best pages below own among those scored, by
 *                   (score desc, page asc), then own.
 * The rows are ranked by the top-16 selector over the score buffer (rows
 * longer than 4,096 columns split across CTAs and merged exactly).
 *   scores_ws     [num_reqs, 32, width] float32 scratch the step scores into
 *                 (left holding the scores afterwards).
 *   out           [num_reqs, query_len, 4, 16] int32.
 *   workspace     >= idx_decode_workspace_bytes(num_reqs, query_len, width)
 *                 bytes, 8-byte aligned; its contents need no initialisation
 *                 (NULL when that is 0).
 *   flags         IDX_RANK_16BIT: rank the scores rounded to IEEE
 *                 binary16 (round to nearest even, overflow to infinity),
 *                 as the stock decode ranks 16-bit quantized scores ([CP]
 *                 module docstring); scores equal in 16 bits then rank by
 *                 page (lower first).  The score buffer keeps the fp32
 *                 scores.
 *                 IDX_PAGE_256: P256 pages ([PUBLISH] Performance: P128
 *                 and P256 pages, 672 columns at 168K tokens).  kv is
 *                 [num_blocks, 256, 72]: 18,432 bytes a page, token t's 64
 *                 code bytes at t*64, then its 8 scale bytes at
 *                 16,384 + t*8; block ids, max_blocks and width count
 *                 256-token pages; a query's own page is
 *                 floor((seq_len - query_len + i) / 256) and pages below
 *                 (seq_len-1)/256 are scored; a page's score is the max over
 *                 its 256 keys.  scores_ws is then [num_reqs, 32, 2*width],
 *                 8-byte aligned: column 2j+h holds the max over keys
 *                 [128h, 128h+128) of page j (stored where page j is, i.e.
 *                 below the own page), and the page's score is the larger
 *                 of the pair.
 *                 IDX_FUSED_SELECT: the selection runs in the scorer's own
 *                 CTAs, with no second launch ([CP] module docstring: a
 *                 local top 16 per page range, merged exactly over the
 *                 union).  Each CTA ranks the pages of its slice per
 *                 (request, row) from its own score stores, and the CTA
 *                 that finishes a request last merges the local top-16s
 *                 into the rows.  The rows are identical to the two-launch
 *                 step's.  workspace is then >=
 *                 idx_decode_fused_workspace_bytes(num_reqs) bytes, 8-byte
 *                 aligned, and ZERO-FILLED before its first use: it holds
 *                 per-request counters that every complete call leaves at
 *                 zero again (zero it again after a call whose status
 *                 reports IDX_ST_TIMEOUT, or before reusing it for another
 *                 purpose).  Not with IDX_PAGE_256 (IDX_E_BAD_SHAPE).
 *                 Other bits: IDX_E_BAD_SHAPE.
 * Other arguments as in idx_score_pages.
 *
 * idx_decode_workspace_bytes: the selector's workspace for the step's
 * num_reqs * query_len * 4 rows of `width` columns, i.e.
 * idx_workspace_bytes(num_reqs * query_len * 4, width); 0 for a bad shape.
 *
 * idx_decode_fused_workspace_bytes: the workspace of a step with
 * IDX_FUSED_SELECT: 4 bytes of counter per request (rounded up to 256
 * bytes), then (num_reqs + 512) * 32 * 16 candidate keys of 8 bytes (the
 * fused scorer runs at most 512 CTAs); 0 when num_reqs is outside
 * [1, 65535].
 */
size_t idx_decode_workspace_bytes(int32_t num_reqs, int32_t query_len, int32_t width);
size_t idx_decode_fused_workspace_bytes(int32_t num_reqs);
#define IDX_RANK_16BIT 1
#define IDX_PAGE_256 2
#define IDX_FUSED_SELECT 4
int idx_decode_step(const uint8_t* q, const float* q_scale, const uint8_t* kv, int64_t num_blocks,
                    const int32_t* block_table, int64_t bt_stride, int32_t max_blocks,
                    const int32_t* seq_lens, int32_t num_reqs, int32_t query_len, int32_t width,
                    float* scores_ws, int32_t* out, void* workspace, size_t workspace_bytes,
                    int32_t flags, int32_t* status, void* stream);

/*
 * Multi-token FP8 indexer scores [MTP]:
 *     out[t][key] = k_scale[key] * sum_h relu(q[t][h] . k[key]) * q_scale[t][h]
 *
 *   q             [num_tokens, heads, 128] E4M3 bytes, contiguous, 16-byte aligned;
 *                 heads = 64.
 *   q_scale       [num_tokens, heads] float32.
 *   k             [num_blocks, 128, 128] E4M3 bytes (128 keys per block), 16-byte aligned.
 *   k_scale       [num_blocks, 128] float32.
 *   block_table   [num_reqs, bt_stride] int32, entries [0, max_blocks) used.
 *   num_keys      [num_reqs] int32 keys of request r (clamped to max_keys and
 *                 max_blocks*128).
 *   cu_tokens     [num_reqs + 1] int32 token offsets; tokens of request r are
 *                 [cu_tokens[r], cu_tokens[r+1]).  No causal mask.
 *   out           [num_tokens, max_keys] float32; keys >= num_keys[r] untouched.
 * Accumulation in fp32 on the tensor cores; within 1e-3 * k_scale *
 * sum_h |q_scale_h| sum_d |q_hd k_d| of the exact value.
 */
int idx_mtp_score_fp8(const uint8_t* q, const float* q_scale, int32_t num_tokens, int32_t heads,
                      const uint8_t* k, const float* k_scale, int64_t num_blocks, const int32_t* block_table,
                      int64_t bt_stride, int32_t max_blocks, const int32_t* num_keys, const int32_t* cu_tokens,
                      int32_t num_reqs, int32_t max_keys, float* out, int32_t* status, void* stream);

/*
 * Q8KV8 prefill indexer chain over NVFP4 index-K pages ([GATHER] module
 * docstring: the gathered, dequantised pages feed the Q8KV8 prefill indexer;
 * [MTP] prefill / causal masking and the -inf tail-fill fusion; [PUBLISH]
 * the prefill top-k).  With nk_r = clamp(num_keys[r], 0, min(max_keys,
 * max_blocks * 128)) and token t the i-th of request r's n_r tokens, at
 * position pos_t = num_keys[r] - n_r + i:
 *     scores[t][key] = sum_h relu(q[t][h] . K_r[key]) * q_scale[t][h]
 *                                             for key <= pos_t, key < nk_r,
 *                    = -inf                   for pos_t < key < nk_r and for
 *                                             nk_r <= key < max_keys,
 *                    = NaN                    for a key of a page whose block
 *                                             id is outside [0, num_blocks)
 *                                             (IDX_ST_BLOCK_OOR; -inf where
 *                                             masked),
 * K_r[key] being key % 128 of page block_table[r][key / 128] dequantised
 * exactly as in idx_dequant_nvfp4_pages; and
 *     out[t] = the 16 best keys of [0, visible_t), visible_t = clamp(pos_t + 1,
 *              0, nk_r), in idx_topk16_select's order (score descending, NaN
 *              ranked as -inf, equal scores by lower key), padded with -1.
 *
 *   kv, num_blocks, block_table, bt_stride, max_blocks
 *                 as in idx_dequant_nvfp4_pages; row r's first
 *                 ceil(nk_r / 128) entries are read.
 *   num_keys      [num_reqs] int32 keys of request r, its new tokens included.
 *   cu_tokens     [num_reqs + 1] int32, non-decreasing, cu_tokens[0] = 0 and
 *                 cu_tokens[num_reqs] = num_tokens; tokens outside every
 *                 request get a row of -inf and no keys.
 *   q             [num_tokens, heads, 128] E4M3 bytes, 16-byte aligned;
 *                 heads in [1, 128] (64 runs on the tensor cores).
 *   q_scale       [num_tokens, heads] float32 (16-byte aligned for the
 *                 tensor-core scorer).
 *   scores        [num_tokens, max_keys] float32, every element written.
 *   out           [num_tokens, 16] int32.
 *   workspace     idx_prefill_workspace_bytes(...) bytes, 256-byte aligned,
 *                 no initialisation needed: the dequantised pages
 *                 (num_reqs * min(max_blocks, ceil(max_keys / 128)) pages of
 *                 16,384 bytes), their block table, per-token visible counts
 *                 and the selector's workspace.
 * Accumulation in fp32; a score is within 1e-3 * sum_h |q_scale_h| sum_d
 * |q_hd k_d| of the exact value.  IDX_E_WORKSPACE when workspace_bytes is
 * short; IDX_E_TOO_LARGE when the pages would pass 2^31 keys.
 *
 * idx_prefill_workspace_bytes: the workspace size for these sizes (0 for a
 * negative size).
 */
size_t idx_prefill_workspace_bytes(int32_t num_reqs, int32_t max_blocks, int32_t num_tokens, int32_t max_keys);
int idx_prefill_index_step(const uint8_t* kv, int64_t num_blocks, const int32_t* block_table, int64_t bt_stride,
                           int32_t max_blocks, const int32_t* num_keys, const int32_t* cu_tokens, int32_t num_reqs,
                           const uint8_t* q, const float* q_scale, int32_t num_tokens, int32_t heads,
                           int32_t max_keys, float* scores, int32_t* out, void* workspace, size_t workspace_bytes,
                           int32_t* status, void* stream);

/*
 * MXFP8 quantisation of bf16 rows ("vLLM PR #65508", the description of the
 * epilogue that quantises the sparse-decode attention output for o_proj):
 * per block of 32 consecutive elements of a row, with amax the largest
 * magnitude (compared on the bf16 bit patterns, sign cleared),
 *     scale = clamp(exponent_field(amax) - 8 + (mantissa(amax) > 0.75), 0, 254)
 * (an E8M0 byte; = ceil(log2(amax / 448)) + 127), and every element becomes
 *     e4m3_rn_satfinite(x * 2^(127 - scale)).
 *
 *   x_bf16        [rows, x_stride] bf16 bit patterns, 16-byte aligned,
 *                 x_stride a multiple of 8; columns [0, cols) are read.
 *   cols          a multiple of 32.
 *   out_e4m3      [rows, out_stride] E4M3 bytes, 8-byte aligned, out_stride
 *                 a multiple of 8.
 *   scales_e8m0   [rows, scale_stride] bytes, row-major: scale of block k of
 *                 row r at r * scale_stride + k.
 * Finite inputs never saturate (the scaled block's largest magnitude is at
 * most 448); an infinity becomes +-448, a NaN 0x7F.
 */
int idx_mxfp8_quantize(const uint16_t* x_bf16, int64_t rows, int64_t cols, int64_t x_stride, uint8_t* out_e4m3,
                       int64_t out_stride, uint8_t* scales_e8m0, int64_t scale_stride, void* stream);

/*
 * Dense FP8 tensor-core throughput probe.  Not a step of the indexer: the
 * pages state no tensor-core rate, and this call measures the one the
 * multi-token and prefill scorers (tcgen05.mma kind::f8f6f4) are compared
 * against.  One CTA per SM issues `iters` rounds of four M=128 x N=256 x K=32
 * E4M3 MMAs (fp32 accumulation in tensor memory) back to back; time the
 * launch with events on `stream`.
 *
 *   iters    1 .. 100,000 (IDX_E_BAD_SHAPE otherwise).
 *   check    optional (may be NULL) float in device memory, 4-byte aligned:
 *            receives accumulator element (0, 0) of the first CTA, which is
 *            32 * iters exactly (every operand element is 0.5).
 *   flops    optional host pointer: receives the launch's floating-point
 *            operations, 2 * 128 * 256 * 32 * 4 * iters * SMs.
 *   status   optional; IDX_ST_TIMEOUT if the final wait gave up.
 */
int idx_fp8_mma_probe(int32_t iters, float* check, double* flops, int32_t* status, void* stream);

/* ======================================================================
 * One step of decoding with drafted tokens, around the indexer:
 *   idx_build_slots     where the step's tokens go: block tables, slots,
 *                       positions and tree masks from the requests' lengths;
 *   idx_rope_append     rotary positions of q and k; k and v into the cache
 *                       (idx_norm_rope_append: after a norm of each head);
 *   idx_index_append    the indexer's queries, and its keys into the pages;
 *   (idx_decode_step    the pages that each drafted token looks at;)
 *   idx_tree_attention  attention of the drafted tokens over the cache;
 *   idx_logit_probs     the probabilities of the tokens after them;
 *   idx_verify_drafts   which drafted tokens stand, and the token after them;
 *   idx_settle_drafts   the rows of those that stand moved together.
 * Between steps, idx_fork_pages and idx_release_pages share a request's pages
 * with new requests and give pages back.
 *
 * Tokens of all requests are packed: request r's are cu_tokens[r] ..
 * cu_tokens[r+1]-1.  Token i of a request is stored at place seq_len - n + i
 * of the request, n being its number of tokens of this step; its place is
 * cache slot block_table[r][place / page_tokens] * page_tokens + place %
 * page_tokens.  With a tree of drafts, node 0 is the last certain token and
 * every node's parent has a lower index.  The pages of the indexer's sources
 * end where these calls begin; their formulas stand here.
 * ====================================================================== */

/* Element types of q, k, v and the attention cache. */
#define IDX_BF16 0
#define IDX_F16 1
#define IDX_F32 2

/*
 * Block tables, slot maps, positions and tree masks from request lengths.
 * With ctx, new >= 0 (negative: 0), P = page_tokens and all sums in 64 bits:
 *     need_r  = min(ceil((ctx_r + new_r) / P), max_blocks)
 *     take_r  = max(0, need_r - owned_r)
 *     first_r = *free_cursor + sum_{s < r} take_s
 *     block_table[r][owned_r + i] = free_blocks[first_r + i], i < take_r,
 *                                   or -1 from num_free on (IDX_ST_NO_BLOCKS)
 *     cu_tokens[r] = min(sum_{s < r} new_s, num_tokens)   (IDX_ST_LEN_CLAMPED:
 *                    seq_lens then count tokens that got no slot, so the step
 *                    is to be made again with room for all its tokens)
 *     seq_lens[r]  = ctx_r + new_r
 *     pages_out[r] = max(owned_r, need_r), less the blocks that were missing
 *     *cursor_out  = min(*free_cursor + sum take, num_free)
 * and for token t, the i-th of request r, at place ctx_r + i:
 *     slots[t]     = block * P + place % P, block = block_table[r][place / P];
 *                    -1 where the place has no page (IDX_ST_LEN_CLAMPED past
 *                    max_blocks) or the block is outside [0, num_blocks)
 *                    (IDX_ST_BLOCK_OOR unless it is -1)
 *     positions[t] = ctx_r + i, or with parents ctx_r + the node's depth
 *     tree_mask[t] = with parents: bit j set for j = i and each ancestor j of
 *                    i; tokens from 64 on get mask 0 and position ctx_r + i
 *                    (IDX_ST_BAD_TREE)
 * Tokens from the last request's end to num_tokens (a padded batch) get slot
 * -1, position 0 and mask 0.
 *
 *   ctx_lens, new_lens, owned_pages, seq_lens, pages_out   [num_reqs] int32
 *   block_table   [num_reqs, bt_stride] int32, in and out: entries below
 *                 owned_r are read, those taken are written
 *   free_blocks   [num_free] int32: free block ids, taken in request order
 *   free_cursor, cursor_out   int32 in device memory; different addresses (a
 *                 program swaps the two, and owned_pages and pages_out,
 *                 after the step)
 *   parents       [num_tokens] int32 or NULL: index within the request of
 *                 each token's parent, -1 for a root; one outside [-1, i)
 *                 counts as -1 (IDX_ST_BAD_TREE)
 *   cu_tokens     [num_reqs + 1] int32;  positions [num_tokens] int32
 *   slots         [num_tokens] int64;  tree_mask [num_tokens] uint64 (with
 *                 parents, else NULL)
 */
int idx_build_slots(const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* owned_pages, int32_t num_reqs,
                    int32_t* block_table, int64_t bt_stride, int32_t max_blocks, const int32_t* free_blocks,
                    int32_t num_free, const int32_t* free_cursor, int64_t num_blocks, int32_t page_tokens,
                    const int32_t* parents, int32_t num_tokens, int32_t* cu_tokens, int32_t* seq_lens,
                    int32_t* pages_out, int32_t* cursor_out, int32_t* positions, int64_t* slots,
                    uint64_t* tree_mask, int32_t* status, void* stream);

/*
 * Rotary frequencies, on the host (needs no GPU): inv_freq[i] for i in
 * [0, rotary_dim / 2) and the magnitude to pass as mscale.
 *     f_i = base^(-2i / rotary_dim)
 *   IDX_ROPE_PLAIN   inv_freq = f_i, mscale 1
 *   IDX_ROPE_LINEAR  inv_freq = f_i / factor, mscale 1 (positions interpolated)
 *   IDX_ROPE_RAMP    frequencies turning more than beta_fast times within
 *                    orig_len positions are kept, those turning less than
 *                    beta_slow times are divided by factor, a linear ramp over
 *                    the index between:  e(b) = rotary_dim ln(orig_len / (2 pi
 *                    b)) / (2 ln base), lo = max(0, floor e(beta_fast)), hi =
 *                    min(rotary_dim - 1, ceil e(beta_slow)), w_i = clamp((i -
 *                    lo) / max(hi - lo, 1e-3), 0, 1), inv_freq = f_i (1 - w_i)
 *                    + w_i f_i / factor; mscale 0.1 ln(factor) + 1 for factor
 *                    > 1, else 1
 */
#define IDX_ROPE_PLAIN 0
#define IDX_ROPE_LINEAR 1
#define IDX_ROPE_RAMP 2
int idx_rope_frequencies(int32_t rotary_dim, double base, int32_t kind, double factor, double orig_len,
                         double beta_fast, double beta_slow, double* inv_freq, double* mscale);

/*
 * Rotary positions, and the paged cache's append.  For each token t, head,
 * and pair i < rotary_dim / 2, with a = positions[t] * inv_freq[i]:
 *     y1 = mscale (x1 cos a - x2 sin a),  y2 = mscale (x2 cos a + x1 sin a)
 * computed in 32 bits and rounded once; (x1, x2) are elements i and i +
 * rotary_dim / 2 of the head, or 2i and 2i + 1 with IDX_ROPE_INTERLEAVED.
 * Elements from rotary_dim on pass unchanged.  The angle is reduced as a
 * 64-bit fraction of a turn: at positions up to 2^31 - 1 it is off by at most
 * 2^-33 turns (and fp32's rounding of the fraction).  Rotated queries go to
 * q_out; rotated keys and unchanged values go to cache slot slots[t] (NULL:
 * slot t); a negative slot is skipped, one past the cache is skipped with
 * IDX_ST_BLOCK_OOR.  Two tokens of one call must not share a slot.
 *
 *   q, q_out      [num_tokens, q_heads, head_dim] with the given strides in
 *                 elements; the head's elements contiguous; q_out may be q
 *                 (with its strides).
 *                 NULL (both) with q_heads 0.
 *   k, v          [num_tokens, kv_heads, head_dim], NULL (both, and the
 *                 caches) with kv_heads 0; v and v_cache alone may be NULL.
 *   k_cache, v_cache   [num_blocks, page_tokens, kv_heads, head_dim] with the
 *                 given strides in elements, the same for both
 *   head_dim      1..512;  rotary_dim  even, 0..head_dim
 *   inv_freq      [rotary_dim / 2] float64 in device memory, radians a
 *                 position
 *   dtype         IDX_BF16, IDX_F16 or IDX_F32, of all tensors
 *   flags         0 or IDX_ROPE_INTERLEAVED
 */
#define IDX_ROPE_INTERLEAVED 1
int idx_rope_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                    int64_t qo_token_stride, int64_t qo_head_stride, int32_t q_heads, const void* k,
                    int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                    int64_t v_head_stride, int32_t kv_heads, int32_t num_tokens, int32_t head_dim, int32_t rotary_dim,
                    const int32_t* positions, const double* inv_freq, float mscale, const int64_t* slots,
                    void* k_cache, void* v_cache, int64_t num_blocks, int32_t page_tokens, int64_t c_block_stride,
                    int64_t c_token_stride, int64_t c_head_stride, int32_t dtype, int32_t flags, int32_t* status,
                    void* stream);

/*
 * Attention of a step's tokens over the paged cache.  Token t, the i-th of
 * request r's n, sees the places p < ctx = seq_len - n, and of the places ctx
 * + j those of the drafted tokens j in its mask (bit j of tree_mask[t], j <
 * min(n, 64); with tree_mask NULL a chain: j <= i).  With pages, places
 * outside the token's listed pages are not seen.  For query head h and KV
 * head h / (q_heads / kv_heads), over the places seen,
 *     s_p = scale (q . k_p),  out = sum_p e^(s_p - L) v_p,  L = ln sum_p e^s_p
 * (scale finite; negative and zero ones too).
 * A token that sees nothing gets out 0 and L -inf (as does one whose scores
 * are all -inf).  A row with a score of NaN is NaN.  Scores, maxima, sums and
 * outputs are held in fp32; e^(s_p - M), M a maximum of the scores met so far
 * or up to 8 powers of two (fp16: 4) below it, is rounded to the cache's type
 * for the product with v; in fp16 in steps of no less than 2^-31.  Scores are
 * meant to stay below 2^24.  What is stored at places that no token sees
 * (unwritten slots of the last page, NaN and infinities among them) has no
 * effect, and what a drafted token has stored reaches only the tokens that see
 * it.
 *
 *   q, out        [num_tokens, q_heads, head_dim] with the given strides in
 *                 elements (multiples of 8), 16-byte aligned
 *   k_cache, v_cache   [num_blocks, page_tokens, kv_heads, head_dim] with the
 *                 given strides in elements (multiples of 8, the same for
 *                 both), 16-byte aligned; num_blocks >= 1
 *   page_tokens   16, 32, 64, or a multiple of 128
 *   head_dim      64 or 128;  q_heads a multiple of kv_heads, at most 128
 *                 query heads a KV head
 *   dtype         IDX_BF16 or IDX_F16 (q, caches, out)
 *   block_table   [num_reqs, bt_stride] int32, entries [0, max_blocks) used;
 *                 places past max_blocks pages are not seen
 *                 (IDX_ST_LEN_CLAMPED), nor those of a block id outside
 *                 [0, num_blocks) (IDX_ST_BLOCK_OOR)
 *   seq_lens      [num_reqs] int32 tokens per request, this step's included
 *   cu_tokens     [num_reqs + 1] int32, non-decreasing, from 0 to at most
 *                 num_tokens; rows past the last request's (a padded batch)
 *                 get out 0 and L -inf
 *   tree_mask     [num_tokens] uint64 or NULL
 *   pages         [num_tokens, page_lists, pages_per_list] int32 or NULL: the
 *                 logical pages of each token and list, as idx_decode_step
 *                 gives them ([num_reqs, query_len, 4, 16]); KV head h uses
 *                 list h / (kv_heads / page_lists); entries that are negative
 *                 or past the request's pages are skipped; an entry's
 *                 repetition within a list changes nothing.  kv_heads a
 *                 multiple of page_lists, pages_per_list 1..64, and no more
 *                 than 2^31 - 1 entries in all.
 *   lse           [num_tokens, q_heads] float32 or NULL: L
 *                 (out and lse must not overlap the inputs)
 *   workspace     >= idx_tree_attention_workspace_bytes(...) bytes, 256-byte
 *                 aligned, no initialisation needed
 */
size_t idx_tree_attention_workspace_bytes(int32_t num_reqs, int32_t num_tokens, int32_t q_heads, int32_t kv_heads,
                                          int32_t head_dim, int32_t page_lists, int32_t pages_per_list);
int idx_tree_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_cache,
                       const void* v_cache, int64_t num_blocks, int32_t page_tokens, int64_t c_block_stride,
                       int64_t c_token_stride, int64_t c_head_stride, const int32_t* block_table, int64_t bt_stride,
                       int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_tokens, int32_t num_reqs,
                       int32_t num_tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                       const uint64_t* tree_mask, const int32_t* pages, int32_t page_lists, int32_t pages_per_list,
                       float scale, int32_t dtype, void* out, int64_t o_token_stride, int64_t o_head_stride,
                       float* lse, void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/*
 * Verification of drafted tokens.  Row p = target[t] is the target's
 * distribution of the token after node t, row q = draft[t] the one from which
 * the children of node t were drawn.  From node 0 (the last certain token),
 * with c = 0 and W = 1, the children x_1, x_2, ... of the node (those whose
 * parent it is, by index) are tried in turn:
 *     child x with random number u = accept_u[x's node] stands when
 *         u W q(x) < max(p(x) - c q(x), 0);
 *     the walk then goes on at that child with c = 0, W = 1;
 *     otherwise  c <- c + W,  W <- sum_v max(p(v) - c q(v), 0).
 * Where no child stands, the next token is drawn from the residual: the
 * lowest v with  sum_{v' <= v} max(p(v') - c q(v'), 0) > sample_u[r] * W.
 * (The residual after k refused children, normalised after each, is max(p -
 * c_k q, 0) / W_k: normalising only moves c.)  With draft NULL the drafts
 * are not random: child x stands when u W < p(x), p(x) taken as 0 if a
 * refused sibling was the same token; otherwise W <- W - p(x), and the
 * residual is p without the refused tokens.  A residual without mass falls
 * back to p; p without mass gives token vocab - 1.
 * Tests of children are made in 64-bit floating point; masses and cumulative
 * sums are off by at most about 2^-45 of the sum of the row p and 2^-60 for
 * each entry and refused child (2^-42 in all for 200,000 entries and one), and
 * do not depend on anything but the inputs and the sizes of the call.  Entries
 * are probabilities: a negative or NaN entry counts as 0, and a row's sum must
 * stay below 8.
 *
 *   target, draft [num_tokens, vocab] float32, row strides in elements;
 *                 draft may be NULL
 *   tokens        [num_tokens] int32 drafted tokens (node 0's entry is not
 *                 read); one outside [0, vocab) is not tried
 *   parents       [num_tokens] int32 index within the request, or NULL for a
 *                 chain; a node whose parent is outside [0, own index) is
 *                 not tried
 *   cu_tokens     [num_reqs + 1] int32, from 0 to num_tokens; at most
 *                 IDX_VERIFY_MAX_NODES tokens a request (IDX_ST_BAD_TREE: the
 *                 rest are not tried)
 *   accept_u      [num_tokens] float32;  sample_u [num_reqs] float32, in [0, 1)
 *   out_tokens    [num_reqs, max_out] int32: the tokens that stand, the drawn
 *                 one, then -1
 *   out_nodes     [num_reqs, max_out] int32: indices of the drafted tokens
 *                 that stand, then -1
 *   num_accepted  [num_reqs] int32: how many stand, at most max_out - 1 (a
 *                 walk that got there draws from p)
 * A request without tokens gets num_accepted 0 and rows of -1.
 */
#define IDX_VERIFY_MAX_NODES 1024
int idx_verify_drafts(const float* target, int64_t target_stride, const float* draft, int64_t draft_stride,
                      int32_t vocab, const int32_t* tokens, const int32_t* parents, const int32_t* cu_tokens,
                      int32_t num_reqs, int32_t num_tokens, const float* accept_u, const float* sample_u,
                      int32_t* out_tokens, int32_t* out_nodes, int32_t max_out, int32_t* num_accepted,
                      int32_t* status, void* stream);

/*
 * idx_rope_append after a norm of each head.  With weights w, for each row x of
 * a head:
 *     n = (offset + w) x / sqrt(mean x^2 + eps)
 * and n's pairs turn as in idx_rope_append; elements from rotary_dim on are
 * those of n.  Values are not normed.  Computed in 32 bits, rounded once: a row
 * whose squares' sum passes 3e38 becomes 0, one with an infinity or NaN is not
 * finite, nor is one whose mean of squares and eps add up to 0.  Squares below
 * 2^-126 have fewer bits there, or none: rows of elements below 2^-60 need an eps
 * that covers them.  With no weights at all the values are idx_rope_append's,
 * which is the faster call.
 *
 *   q_weight, k_weight   [head_dim] of the type of all tensors, or NULL: that
 *                 side is turned only
 *   eps           >= 0;  offset  added to the weights (0, or 1 where weights
 *                 are stored less 1)
 * Other arguments as in idx_rope_append (q_out may be q, with its strides).
 */
int idx_norm_rope_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                         int64_t qo_token_stride, int64_t qo_head_stride, int32_t q_heads, const void* k,
                         int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                         int64_t v_head_stride, int32_t kv_heads, int32_t num_tokens, int32_t head_dim,
                         int32_t rotary_dim, const void* q_weight, const void* k_weight, float eps, float offset,
                         const int32_t* positions, const double* inv_freq, float mscale, const int64_t* slots,
                         void* k_cache, void* v_cache, int64_t num_blocks, int32_t page_tokens, int64_t c_block_stride,
                         int64_t c_token_stride, int64_t c_head_stride, int32_t dtype, int32_t flags, int32_t* status,
                         void* stream);

/*
 * The indexer's inputs: queries and keys of 128 elements normed and turned as
 * in idx_norm_rope_append (y), then quantised.  For a query's row, with a =
 * max |y|,
 *     q_out = e4m3_rn(448 y / a),  q_scale = scale * a / 448 * head_weights
 * and for a key's row, over each 16 consecutive elements, with a = max |y|,
 *     s = e4m3_rn_satfinite(a / 6),  code = e2m1_rn_satfinite(y / s)
 * (codes 0 where s is 0), written to the NVFP4 page of its slot.  Codes and key
 * scales are those of 64-bit arithmetic (rounded to nearest, halves to even;
 * angles as in idx_rope_append); q_scale is fp32.  A query's row that holds an
 * infinity or NaN (or whose squares' sum passes 3e38) gets codes 0x7F and a NaN
 * scale, a key's gets NaN scales and codes 0, so its scores are NaN and rank
 * last; so does a row of zeros with weights and eps 0 (a query's codes are 0).  A
 * query's row whose largest magnitude (turned, with the weights, before the norm)
 * is below 2^-100 or above 2^126 gets codes 0.  With an eps below 2^-96 queries
 * take a second launch, for rows whose squares fp32 does not hold.
 *
 *   q             [num_tokens, heads, 128], the head's elements contiguous, or
 *                 NULL with heads 0 (up to 128)
 *   k             [num_tokens, 128], or NULL (with index_k)
 *   q_weight, k_weight   [128] of the type of q and k, or NULL: no norm there
 *   rotary_dim    0..128, a multiple of 16 (of 8 with IDX_ROPE_INTERLEAVED)
 *   head_weights  [num_tokens, heads] float32 contiguous, or NULL: 1
 *   cu_tokens     [num_reqs + 1] int32, or NULL: q_out is [num_tokens, heads,
 *                 128] and q_scale [num_tokens, heads], as
 *                 idx_prefill_index_step and idx_mtp_score_fp8 take them.
 *                 With it, q_out is [num_reqs, req_slots, heads, 128] and
 *                 q_scale [num_reqs, req_slots, heads], as idx_decode_step
 *                 takes them: a request's n tokens go to its last n slots, the
 *                 others stay as they are; of more than req_slots tokens only
 *                 the last have a slot (IDX_ST_BAD_OUTPUT).  Tokens outside
 *                 every request have none.
 *   slots         [num_tokens] int64 cache slot of each key, or NULL: slot t;
 *                 a negative one is skipped, one past the pages is skipped
 *                 with IDX_ST_BLOCK_OOR; two tokens must not share one
 *   index_k       [num_blocks, page_tokens, 72] uint8 pages, page_tokens 128
 *                 (as in idx_dequant_nvfp4_pages) or 256 (IDX_PAGE_256)
 *   dtype         of q, k and the weights;  flags  0 or IDX_ROPE_INTERLEAVED
 * q_out and index_k 16-byte aligned.
 */
int idx_index_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, int32_t heads, const void* k,
                     int64_t k_token_stride, int32_t num_tokens, int32_t rotary_dim, const void* q_weight,
                     const void* k_weight, float eps, float offset, const int32_t* positions, const double* inv_freq,
                     float mscale, const float* head_weights, float scale, const int32_t* cu_tokens, int32_t num_reqs,
                     int32_t req_slots, uint8_t* q_out, float* q_scale, const int64_t* slots, uint8_t* index_k,
                     int64_t num_blocks, int32_t page_tokens, int32_t dtype, int32_t flags, int32_t* status,
                     void* stream);

/*
 * Probabilities from logits.  Row t is that of node i = t - cu_tokens[r] of
 * request r; for entry v, with c the times that the request has token v
 * already and each step rounded to fp32 in this order,
 *     x = logit
 *     seen (c > 0, or v in the prompt):  x <- x / repetition where x > 0, else
 *                                        x * repetition
 *     c > 0:  x <- x - (frequency * c + presence)
 *     x <- x + bias, for each of the request's biases of v in their order
 *     x <- -inf where the mask has no bit (whatever the logit is)
 *     p = e^(x / T - L),  L = ln sum e^(x / T)
 * With T = 0 (or below 2^-60, or NaN) p is 1 at the lowest v of the largest x
 * and 0 elsewhere, and L is that x.  With T infinite all entries above -inf get
 * the same p.  A row with nothing left gets p 0 and L -inf; one with a NaN or
 * +inf that is not masked is NaN.  x, x less the largest x, sums and p are fp32.
 * c is the count in `counts` plus, with tokens, that of v among the drafted
 * tokens of the row's path: nodes j >= 1 of tree_mask[t] (tree_mask NULL: 1 <=
 * j <= i).  Node 0's token is taken to be counted already, as idx_settle_drafts
 * does it.
 *
 *   logits        [num_tokens, vocab] of dtype, row stride in elements
 *   vocab         up to IDX_PROBS_MAX_VOCAB
 *   temperature, repetition, presence, frequency   [num_reqs] float32, each
 *                 may be NULL: 1, 1, 0, 0 (with no penalty at all counts and
 *                 tokens are not read)
 *   counts        [num_reqs, vocab] int32, row stride in elements, or NULL: the
 *                 count in the low 31 bits, the highest bit set for a token of
 *                 the prompt
 *   tokens        [num_tokens] int32 or NULL;  tree_mask [num_tokens] uint64 or
 *                 NULL (with tokens); a chain counts up to IDX_VERIFY_MAX_NODES
 *                 tokens (IDX_ST_BAD_TREE), those outside [0, vocab) not
 *   bias_cu       [num_reqs + 1] int32 or NULL: request r's biases are
 *                 bias_tokens and bias_values (int32, float32, num_bias in
 *                 all) bias_cu[r] .. bias_cu[r+1]-1
 *   allowed       [num_tokens, ceil(vocab / 32)] int32, row stride in elements,
 *                 or NULL: bit v % 32 of word v / 32
 *   probs         [num_tokens, vocab] float32; may be logits (in fp32, with its
 *                 stride).  Rows outside every request (a padded batch) get 0
 *   lse           [num_tokens] float32 or NULL: L
 */
#define IDX_PROBS_MAX_VOCAB 262144
int idx_logit_probs(const void* logits, int64_t logits_stride, int32_t dtype, int32_t vocab, int32_t num_tokens,
                    const int32_t* cu_tokens, int32_t num_reqs, const float* temperature, const float* repetition,
                    const float* presence, const float* frequency, const int32_t* counts, int64_t counts_stride,
                    const int32_t* tokens, const uint64_t* tree_mask, const int32_t* bias_cu,
                    const int32_t* bias_tokens, const float* bias_values, int32_t num_bias, const int32_t* allowed,
                    int64_t allowed_stride, float* probs, int64_t probs_stride, float* lse, int32_t* status,
                    void* stream);

/*
 * A cache whose rows the calls below move: `planes` (layers, keys and values)
 * of the same blocks, a token's row in a plane `row_bytes` contiguous bytes.
 * Strides are in bytes.  The codes and the scales of NVFP4 index-K pages are
 * two caches: 64 bytes a token from the page's begin on, and 8 from byte 64 *
 * page_tokens on.  Host memory, read during the call.
 */
#define IDX_MAX_CACHES 8
typedef struct {
  void* base;
  int64_t plane_stride, block_stride, token_stride;
  int32_t planes, row_bytes;
} idx_cache;

/*
 * After idx_verify_drafts: the rows of the nodes that stand move together in
 * every cache, from slots[cu_tokens[r] + out_nodes[r][i]] to
 * slots[cu_tokens[r] + 1 + i] for i < num_accepted[r], so that the next step's
 * context has no gaps, and
 *     ctx_out[r] = ctx_lens[r] + 1 + num_accepted[r]   (a request without
 *                  tokens in this step: ctx_lens[r])
 *     counts[r][x] += 1 for the tokens x that stand and the one drawn after
 *                  them (out_tokens[r][0 .. num_accepted[r]]), with counts
 * num_accepted is taken as at most the request's tokens, or max_out, less one.
 * A node outside [i + 1, tokens of the request) is not moved
 * (IDX_ST_BAD_TREE), nor a row whose place has no slot, or one past the caches
 * (IDX_ST_BLOCK_OOR).  Rows of other places stay as they are.
 *
 *   caches        num_caches of num_blocks blocks of page_tokens tokens
 *   slots, cu_tokens, num_tokens   as idx_build_slots gives them; without caches
 *                 nothing moves, slots are not read and may be NULL
 *   out_tokens, out_nodes [num_reqs, max_out], num_accepted   as
 *                 idx_verify_drafts gives them (out_tokens: with counts)
 *   ctx_lens, ctx_out   [num_reqs] int32; ctx_out may be ctx_lens
 *   counts        [num_reqs, vocab] int32, row stride in elements, or NULL
 */
int idx_settle_drafts(const idx_cache* caches, int32_t num_caches, int64_t num_blocks, int32_t page_tokens,
                      const int64_t* slots, const int32_t* cu_tokens, int32_t num_reqs, int32_t num_tokens,
                      const int32_t* out_tokens, const int32_t* out_nodes, int32_t max_out,
                      const int32_t* num_accepted, const int32_t* ctx_lens, int32_t* ctx_out, int32_t* counts,
                      int64_t counts_stride, int32_t vocab, int32_t* status, void* stream);

/*
 * Requests forked: child c = children[f] gets the context of p = parents[f].
 * With len = min(ctx_lens[p], owned_pages[p] * page_tokens)
 * (IDX_ST_LEN_CLAMPED), full = floor(len / page_tokens), rest = len %
 * page_tokens:
 *     block_table[c][i] = block_table[p][i], refs[that block] += 1, i < full
 *     rest > 0:  block_table[c][full] = the next free block, the first rest
 *                tokens of the parent's page `full` copied to it in every cache
 *     ctx_lens[c] = len,  owned_pages[c] = full + (rest > 0)
 *     *cursor_out = min(*free_cursor + forks with rest > 0, num_free)
 * Free blocks are taken in the forks' order; a fork for which there is none is
 * not made (IDX_ST_NO_BLOCKS): its child gets length and pages 0.  A fork whose
 * child is a parent in the same call, or the child of another fork, or that has
 * a request outside [0, num_reqs), is not made and changes nothing
 * (IDX_ST_BAD_FORK); one with child -1 is none, whatever its parent (a captured
 * call's empty places).  What a child owned before is not released.  Table
 * entries outside [0, num_blocks) are passed on, not counted, and not copied
 * from (IDX_ST_BLOCK_OOR).
 *
 *   parents, children   [num_forks] int32, up to IDX_MAX_FORKS
 *   ctx_lens, owned_pages   [num_reqs] int32, in and out
 *   block_table   [num_reqs, bt_stride] int32, in and out
 *   refs          [num_blocks] int32, in and out: holders of each block beyond
 *                 the first, >= 0 (0 for blocks fresh from the free list)
 *   free_blocks, free_cursor, cursor_out   as in idx_build_slots
 */
#define IDX_MAX_FORKS 4096
int idx_fork_pages(const idx_cache* caches, int32_t num_caches, int64_t num_blocks, int32_t page_tokens,
                   const int32_t* parents, const int32_t* children, int32_t num_forks, int32_t* ctx_lens,
                   int32_t* owned_pages, int32_t num_reqs, int32_t* block_table, int64_t bt_stride, int32_t max_blocks,
                   int32_t* refs, const int32_t* free_blocks, int32_t num_free, const int32_t* free_cursor,
                   int32_t* cursor_out, int32_t* status, void* stream);

/*
 * Pages given back: request r keeps pages_out[r] = min(owned_pages[r],
 * ceil(keep_lens[r] / page_tokens)) pages (negative lengths count as 0); of
 * each page after those one holder is taken off.  A block whose last holder
 * went (once, whatever the number of releases) goes back to the free list, its
 * refs 0: with m such blocks,
 *     *cursor_out = *free_cursor - m
 *     free_blocks[*cursor_out + i] = the i-th lowest of their ids
 * (the list's entries before the cursor are those taken from it; with more
 * blocks than entries the lowest are dropped: IDX_ST_BAD_OUTPUT).  Table
 * entries from pages_out[r] on mean nothing afterwards.  Entries of -1 are
 * skipped, others outside [0, num_blocks) too (IDX_ST_BLOCK_OOR).
 * A request that is cut back goes on in its last page, behind keep_lens[r].
 * Where that length ends inside a page with refs above 0 afterwards (a full page
 * of a fork or its parent), the request must not be given slots there: rows
 * written to them would replace tokens of the other holders.  Such a request is
 * forked at its kept length (idx_fork_pages copies the page's first tokens to a
 * block of its own) and given up for its child.
 *
 *   keep_lens, owned_pages, pages_out   [num_reqs] int32 (a finished request
 *                 keeps 0); pages_out is an array of its own
 *   block_table   [num_reqs, bt_stride] int32;  refs [num_blocks] int32, in and
 *                 out, as in idx_fork_pages
 *   free_blocks   [num_free] int32, in and out; free_cursor and cursor_out at
 *                 different addresses
 */
int idx_release_pages(const int32_t* keep_lens, const int32_t* owned_pages, int32_t num_reqs,
                      const int32_t* block_table, int64_t bt_stride, int32_t max_blocks, int32_t* refs,
                      int64_t num_blocks, int32_t* free_blocks, int32_t num_free, const int32_t* free_cursor,
                      int32_t* cursor_out, int32_t* pages_out, int32_t page_tokens, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* IDX_H */
