/*
 * idx.h -- C ABI of libidx, the GB300 (sm_103a) MXFP4 lightning-indexer path.
 *
 * The operations are those of the DSA lightning indexer with an MXFP4 K-cache as
 * described by:
 *   - vLLM PR #48558 "[Kernel] MXFP4 indexer cache for GLM-5.2 / DSA" (sections
 *     "What", "Changes", "Benefit", "Notes", and the "Live validation" comment);
 *   - Whamp/vllm PR #14 "Enable SM86 MXFP4 sparse-indexer cache" (sections
 *     "Summary", "Validation");
 *   - vLLM API docs "vllm.models.glm5next.nvidia.sparse_indexer",
 *     class SparseAttnIndexerKpool (mqa_logits, paged_mqa_logits,
 *     top_k_per_row, forward_cuda).
 *
 * Formats (fixed by this library; the pages give the sizes, not the rounding):
 *   - An indexer key or query head is 128 values.  MXFP4 stores it as 64 bytes
 *     of E2M1 codes (element 2i in the low nibble of byte i, element 2i+1 in the
 *     high nibble) and 4 UE8M0 scale bytes, one per block of 32 elements, in
 *     block order: 68 bytes instead of FP8's 132 (PR #48558, "Benefit").
 *   - Scale of a block: byte e+127 for the smallest integer e with
 *     max|x| <= 6 * 2^e, clamped to [0, 254]; an all-zero block gets byte 0.
 *   - Code of x: x / 2^e rounded to the nearest of {0,0.5,1,1.5,2,3,4,6}, ties to
 *     the even code, magnitudes above 6 saturate to 6; bit 3 is the sign of x
 *     (also when the magnitude rounds to 0).  Inf/NaN inputs are outside the
 *     contract.
 *   - Paged cache: pages of page_size = 64 tokens, 4352 bytes each: the 64x64
 *     value bytes of the page's tokens (token-major), then their 64x4 scale
 *     bytes ("block-split" layout, PR #48558 "Live validation").  Token slot
 *     s = page * 64 + offset.
 *   - logit[r, s] = sum_h w[r, h] * max(0, sum_d q^[r, h, d] * k^[s, d]) on
 *     dequantised operands, fp32 accumulation.
 *
 * Conventions for every entry point:
 *   - All data pointers are DEVICE pointers owned by the caller.  The library
 *     allocates no device memory and never synchronises; work is enqueued on
 *     `stream` (NULL = the legacy default stream) and the call returns at once.
 *     So every call other than idx_paged_logits_topk_noalloc can be captured
 *     in a CUDA graph; a replay reads its buffers afresh (the fused call's
 *     work-item counter starts over on every replay).
 *   - Argument and device errors are returned synchronously, before anything is
 *     enqueued.  IDX_ERR_CUDA reports a launch failure (the CUDA error string
 *     is available from idx_last_error_detail()).
 *   - Contract violations that only the device can see (a slot or block id out
 *     of range, a context longer than the block table or the logits row) are
 *     skipped by the kernels and counted in the optional `errors` struct.  The
 *     kernels never trap.  A pipeline wait that exceeds its limit (a library
 *     bug, not an input error) sets a bit in errors->timeouts and the kernel
 *     returns early.
 *   - Supported shapes: head_dim 128, page_size 64, H in {32, 64},
 *     next_n in {1, 2}, 1 <= k <= 2048.  Others give IDX_ERR_INVALID_ARG.
 *   - Only sm_103 devices are accepted (IDX_ERR_UNSUPPORTED_DEVICE otherwise).
 */
#ifndef IDX_H_
#define IDX_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define IDX_API __attribute__((visibility("default")))
#else
#define IDX_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t. */
typedef struct CUstream_st* idx_stream_t;

typedef enum {
  IDX_OK = 0,
  IDX_ERR_INVALID_ARG = 1,
  IDX_ERR_UNSUPPORTED_DEVICE = 2,
  IDX_ERR_WORKSPACE_TOO_SMALL = 3,
  IDX_ERR_CUDA = 4
} idx_status;

/* Device-side error counters (device memory, zeroed by the caller). */
typedef struct {
  int32_t bad_inputs; /* skipped slots / block ids / over-long contexts */
  int32_t timeouts;   /* bit mask of pipeline waits that gave up */
} idx_device_errors;

/* Library version, major * 10000 + minor * 100 + patch. */
IDX_API int idx_version(void);

/* Static description of a status code. */
IDX_API const char* idx_status_string(idx_status status);

/* Detail of the last failing call on this host thread ("" if none). */
IDX_API const char* idx_last_error_detail(void);

/* Fail-closed architecture gate (Whamp/vllm PR #14, "Summary": fail-closed
 * capability gates).  Pure host logic: IDX_OK only for compute capability
 * 10.3 (sm_103, GB300). */
IDX_API idx_status idx_arch_supported(int major, int minor);

/* Applies idx_arch_supported to `device`.  IDX_ERR_CUDA if the device cannot be
 * queried. */
IDX_API idx_status idx_check_device(int device);

/* ---------------------------------------------------------------------------
 * idx_quant_insert -- quantise indexer keys to MXFP4 and scatter them into the
 * paged cache (PR #48558, "Changes": indexer_k_quant_and_cache with scale_fmt
 * "mxfp4"; "Live validation": block-split value/scale layout).
 *   k_bf16        [n_tokens, k_row_stride] bf16; the first 128 values of each row
 *                 are the key.  Base 16-byte aligned, k_row_stride a multiple of 8.
 *   slot_mapping  [n_tokens] int64 slots; -1 = padding, skipped; any other value
 *                 outside [0, num_blocks*page_size) is skipped and counted.
 *   kcache        [num_blocks, page_size*68] bytes, 16-byte aligned.  Only the 68
 *                 bytes of each inserted token are written.
 * n_tokens == 0 is a no-op.  Slots must be distinct (duplicates race).
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_quant_insert(const void* k_bf16, int64_t n_tokens, int64_t k_row_stride,
                            const int64_t* slot_mapping, uint8_t* kcache, int64_t num_blocks,
                            int32_t page_size, idx_device_errors* errors, idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_quant_q -- quantise query heads with the same rule (PR #48558, "Notes":
 * MXFP4 q-quant; sparse_indexer forward_cuda: FP4 q is a (values, scales) pair).
 *   q_bf16    [rows, 128] bf16, contiguous, 16-byte aligned (rows = T * H).
 *   q_vals    [rows, 64] bytes out;  q_scales [rows, 4] bytes out.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_quant_q(const void* q_bf16, int64_t rows, uint8_t* q_vals, uint8_t* q_scales,
                       idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_rope_quant_q -- rotary position embedding of the query heads fused with
 * their MXFP4 quantisation (PR #48558, "Notes": a fused q-rope + MXFP4 q-quant
 * kernel could follow the PyTorch q-quant).  The pages give no rotary
 * parameters; the caller passes the table.
 *   q_bf16     [T, H, 128] bf16, contiguous, 16-byte aligned.
 *   positions  [T] int32: the table row of token t.  When rot_dim > 0, a token
 *              whose position is outside [0, num_pos) is skipped (its rows are
 *              not written) and counted in errors->bad_inputs; with rot_dim = 0
 *              positions are not read (may be any pointer, even NULL).
 *   cos_table, sin_table [num_pos, rot_dim / 2] fp32: cosine and sine of the
 *              angle of pair i at each position (may be NULL when rot_dim = 0).
 *   rot_dim    even, 0..128: dimensions [0, rot_dim) turn in pairs (2i, 2i+1):
 *              x' = x cos - y sin, y' = x sin + y cos, in fp32 with the products
 *              y sin and y cos rounded first and one fused multiply-add each;
 *              the other dimensions pass through.
 *   q_vals / q_scales [T*H, 64] / [T*H, 4] out, as idx_quant_q (row t*H + h).
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_rope_quant_q(const void* q_bf16, int64_t T, int32_t H,
                            const int32_t* positions, const float* cos_table,
                            const float* sin_table, int32_t num_pos, int32_t rot_dim,
                            uint8_t* q_vals, uint8_t* q_scales, idx_device_errors* errors,
                            idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_kpool_insert -- K-pool compressed insert (sparse_indexer docs,
 * _kpool_compress_insert): pools of kpool consecutive keys become one MXFP4
 * key, written at pool-granular slots, masked in the kernel (no compaction,
 * no synchronisation).
 *   k_bf16        [n, 128] bf16 keys of the batch in token order, contiguous.
 *   gate          [n, 128] fp32 gate scores; ape [kpool, 128] fp32 position terms.
 *   slot_mapping  [n] int64, pool-granular: row p completes a pool, and is
 *                 written, iff slot[p] >= 0 and p >= kpool - 1 (a valid slot
 *                 earlier belongs to a pool that began before the batch); a
 *                 batch with n < kpool writes nothing.  Slots past the cache are
 *                 skipped and counted.  Pool chunks start pool-aligned.
 *   Written row p: kc[d] = sum_j softmax_j(gate[p-kpool+1+j, d] + ape[j, d])
 *                 * k[p-kpool+1+j, d] over j < kpool (fp32; the pages fix the
 *                 masking, this library reads the pooling as a softmax of gate
 *                 plus position term), quantised as a key and stored at slot[p].
 *   kcache        paged cache as for idx_quant_insert.
 *   pooled        [n, 128] fp32 out, optional (NULL): kc of the written rows;
 *                 other rows are not touched.
 *   1 <= kpool <= 128.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_kpool_insert(const void* k_bf16, const float* gate, const float* ape,
                            const int64_t* slot_mapping, int64_t n, int32_t kpool,
                            uint8_t* kcache, int64_t num_blocks, int32_t page_size,
                            float* pooled, idx_device_errors* errors, idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_paged_mqa_logits -- decode logits through block tables (sparse_indexer
 * docs: paged_mqa_logits; PR #48558 "Notes": the paged MQA-logits reader).
 *   q_vals/q_scales  [B*next_n*H, 64] / [B*next_n*H, 4]: query row r = b*next_n + j,
 *                    head h at row r*H + h.
 *   kcache           paged cache as for idx_quant_insert, num_blocks pages.
 *   block_table      [B, max_blocks] int32 page ids.
 *   context_lens     [B] int32: L_b, tokens of sequence b including its next_n
 *                    new ones.  Row (b, j) sees positions [0, L_b - next_n + j].
 *   weights          [B*next_n, H] fp32.
 *   logits           [B*next_n, ld] fp32 out.  Column s < window length gets the
 *                    logit.  With clean != 0 every other column in [0, ld) gets
 *                    -inf; with clean == 0 those columns are not written.
 * A context longer than min(max_blocks*page_size, ld) is clamped and counted.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_paged_mqa_logits(const uint8_t* q_vals, const uint8_t* q_scales, int32_t B,
                                int32_t next_n, int32_t H, const uint8_t* kcache,
                                int64_t num_blocks, int32_t page_size,
                                const int32_t* block_table, int32_t max_blocks,
                                const int32_t* context_lens, const float* weights,
                                float* logits, int64_t ld, int clean,
                                idx_device_errors* errors, idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_mqa_logits -- prefill logits over contiguous keys (sparse_indexer docs:
 * mqa_logits).
 *   q_vals/q_scales  [T*H, 64] / [T*H, 4]: query t, head h at row t*H + h.
 *   k_vals/k_scales  [S, 64] / [S, 4] (e.g. from idx_gather_k), 16-byte aligned.
 *   weights          [T, H] fp32.
 *   row_start/row_end [T] int32: query t sees keys [row_start[t], row_end[t]),
 *                    0 <= start <= end <= S (windows outside are clamped and
 *                    counted in errors->bad_inputs).
 *   logits           [T, ld] fp32 out, ld >= S.  Columns in the window get the
 *                    logit; with clean != 0 the other columns of [0, S) get
 *                    -inf, otherwise they are not written.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_mqa_logits(const uint8_t* q_vals, const uint8_t* q_scales, int64_t T, int32_t H,
                          const uint8_t* k_vals, const uint8_t* k_scales, int64_t S,
                          const float* weights, const int32_t* row_start,
                          const int32_t* row_end, float* logits, int64_t ld, int clean,
                          idx_device_errors* errors, idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_mqa_logits_topk -- idx_mqa_logits followed by top-k of every row
 * (sparse_indexer docs: mqa_logits then top_k_per_row) without a logits
 * tensor: the scoring kernel keeps, per row, a threshold that only grows (the
 * k-th largest of the logits admitted so far, to within a histogram bin) and
 * appends only the logits that reach it, with their positions, to the row's
 * candidate list; a second kernel selects the k largest of each list.
 *   Arguments as for idx_mqa_logits (without logits/ld/clean) and
 *   idx_topk_rows: out_idx [T, k] int32 holds positions relative to
 *   row_start[t], in no particular order, -1 after the last valid one.
 *   workspace  at least idx_mqa_logits_topk_workspace_bytes(T, S, k) bytes,
 *              256-byte aligned, no initialisation: per row a list of up to S
 *              candidates (8 bytes each: every position of a row whose logits
 *              rise with the position is a candidate), of which typically a
 *              small part is written.  Calls that share it must not overlap.
 * ------------------------------------------------------------------------ */
IDX_API size_t idx_mqa_logits_topk_workspace_bytes(int64_t T, int64_t S, int32_t k);

IDX_API idx_status idx_mqa_logits_topk(const uint8_t* q_vals, const uint8_t* q_scales, int64_t T,
                               int32_t H, const uint8_t* k_vals, const uint8_t* k_scales,
                               int64_t S, const float* weights, const int32_t* row_start,
                               const int32_t* row_end, int32_t k, int32_t* out_idx,
                               void* workspace, size_t workspace_bytes,
                               idx_device_errors* errors, idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_topk_rows -- top-k per logits row (sparse_indexer docs: top_k_per_row
 * into topk_indices_buffer).
 *   logits           [rows, ld] fp32; only columns [row_start[r], row_end[r]) are
 *                    read (NULL row_start means 0 for every row).
 *   out_idx          [rows, k] int32 out: the columns of the k largest values,
 *                    each minus row_start[r], in no particular order.  A row
 *                    with fewer than k columns lists all of them, then -1.
 *                    Equal values may be taken in any order.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_topk_rows(const float* logits, int64_t rows, int64_t ld,
                         const int32_t* row_start, const int32_t* row_end, int32_t k,
                         int32_t* out_idx, idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_paged_logits_topk -- idx_paged_mqa_logits followed by top-k of every row,
 * without writing the logits to memory.  Arguments as for those two entries;
 * out_idx [B*next_n, k] int32 holds positions in the sequence (-1 padded).
 *   workspace        device scratch of at least
 *                    idx_paged_logits_topk_workspace_bytes(...) bytes, 256-byte
 *                    aligned; its contents need no initialisation and are
 *                    meaningless after the call.  Calls that share a workspace
 *                    must not overlap on the GPU.
 *   A batch of more than about 16 million work items (B times the items per
 *   sequence, up to 16 pages each) is rejected with IDX_ERR_INVALID_ARG.
 * ------------------------------------------------------------------------ */
IDX_API size_t idx_paged_logits_topk_workspace_bytes(int32_t B, int32_t next_n, int32_t max_blocks,
                                             int32_t page_size, int32_t k);

IDX_API idx_status idx_paged_logits_topk(const uint8_t* q_vals, const uint8_t* q_scales, int32_t B,
                                 int32_t next_n, int32_t H, const uint8_t* kcache,
                                 int64_t num_blocks, int32_t page_size,
                                 const int32_t* block_table, int32_t max_blocks,
                                 const int32_t* context_lens, const float* weights, int32_t k,
                                 int32_t* out_idx, void* workspace, size_t workspace_bytes,
                                 idx_device_errors* errors, idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_paged_logits_topk_noalloc -- idx_paged_logits_topk for callers that
 * cannot allocate device memory: an engine whose allocator is frozen after
 * start-up, a plugin host that passes raw buffers but offers no allocator, or a
 * latency-critical step that must not pay for cudaMalloc (it can block on the
 * device).  The pages have no counterpart for this entry; it only changes where
 * the scratch comes from.
 *   Arguments as for idx_paged_logits_topk, without workspace/workspace_bytes.
 *   The scratch is a 32 MiB array inside the library: every GPU that loads the
 *   library reserves it until the process exits.  Its device address is looked
 *   up on the first call in each CUDA context (the calling thread's current
 *   one) and kept for later calls in that context; a device reset ends the
 *   context, and the next call looks the address up again.
 *   A batch whose idx_paged_logits_topk_workspace_bytes exceeds 32 MiB is
 *   rejected with IDX_ERR_INVALID_ARG (the reason is in
 *   idx_last_error_detail()); use idx_paged_logits_topk with a caller
 *   workspace for it.
 *   All calls share the one scratch array: calls that overlap on the GPU race.
 *   Nothing in the scratch needs clearing between calls: the work-item counter
 *   at its start carries each call's generation and is reset by the call's
 *   select pass; the logits rows behind it are rewritten before being read.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_paged_logits_topk_noalloc(
    const uint8_t* q_vals, const uint8_t* q_scales, int32_t B, int32_t next_n, int32_t H,
    const uint8_t* kcache, int64_t num_blocks, int32_t page_size, const int32_t* block_table,
    int32_t max_blocks, const int32_t* context_lens, const float* weights, int32_t k,
    int32_t* out_idx, idx_device_errors* errors, idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_paged_decode_step -- one decode step of the indexer in two launches:
 * the step's insert (PR #48558, "Changes": indexer_k_quant_and_cache ahead of
 * the paged reader) and query quantisation ("Notes") done by the scoring
 * launch of idx_paged_logits_topk, before it scores, then its select.
 *   k_new_bf16   [B*next_n, 128] bf16, contiguous, 16-byte aligned: the step's
 *                new keys; row b*next_n + j is position L_b - next_n + j of
 *                sequence b and is written to that position's page (through
 *                the block table) and offset, as idx_quant_insert would.  A
 *                position outside the block table, or a page id outside the
 *                cache, is skipped and counted.
 *   q_bf16       [B*next_n, H, 128] bf16, contiguous, 16-byte aligned: the
 *                step's query heads, quantised as idx_quant_q would (into the
 *                workspace; nothing else of the caller's is written).
 *   The other arguments are those of idx_paged_logits_topk; context_lens
 *   count the new tokens.  out_idx [B*next_n, k] as there.
 *   workspace    at least idx_paged_decode_step_workspace_bytes(...) bytes,
 *                256-byte aligned, no initialisation, not shared by calls that
 *                overlap on the GPU.  Besides the fused call's contents it
 *                holds the quantised query heads, a chunk counter and one
 *                count per sequence (generation-tagged; the select resets
 *                them to the call's generation with no claims).
 *   The scoring launch does the step's quantisation and insert first, in
 *   small chunks that its CTAs claim from a counter in the workspace; a CTA
 *   waits for a sequence's chunks to be done before it reads any of the
 *   sequence's keys (a bounded wait; a wait that gives up sets the timeout
 *   bit).  The launch needs no co-residency of its CTAs.
 * ------------------------------------------------------------------------ */
IDX_API size_t idx_paged_decode_step_workspace_bytes(int32_t B, int32_t next_n, int32_t H,
                                             int32_t max_blocks, int32_t page_size, int32_t k);

IDX_API idx_status idx_paged_decode_step(const void* k_new_bf16, const void* q_bf16, int32_t B,
                                 int32_t next_n, int32_t H, uint8_t* kcache, int64_t num_blocks,
                                 int32_t page_size, const int32_t* block_table,
                                 int32_t max_blocks, const int32_t* context_lens,
                                 const float* weights, int32_t k, int32_t* out_idx,
                                 void* workspace, size_t workspace_bytes,
                                 idx_device_errors* errors, idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_gather_k -- copy sequences' cached tokens into contiguous value/scale
 * arrays (PR #48558 "Live validation": the shared cp_gather reader).
 *   seq_lens     [B] int32 tokens to copy per sequence (<= max_blocks*page_size).
 *   out_offsets  [B] int64 first output row of each sequence.
 *   k_vals/k_scales [out_rows, 64] / [out_rows, 4] out; rows beyond out_rows are
 *                skipped and counted.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_gather_k(const uint8_t* kcache, int64_t num_blocks, int32_t page_size,
                        const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                        const int64_t* out_offsets, int32_t B, uint8_t* k_vals,
                        uint8_t* k_scales, int64_t out_rows, idx_device_errors* errors,
                        idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_copy_async -- copy `bytes` bytes from src to dst with the GPU's SMs, for
 * the small host<->device transfers of a decode step (its inputs in, its top-k
 * indices out).  The pages have no counterpart for this entry.  On GB300 the
 * SMs reach page-locked host memory over NVLink-C2C, so for a few hundred KB
 * this costs about a kernel launch and one memory round trip, less than a
 * copy-engine transfer.
 *   dst, src   each either device memory of the current device, managed
 *              memory, or page-locked host memory mapped into the device's
 *              address space (as pinned allocations are under unified
 *              addressing), each covering `bytes` bytes of one allocation;
 *              the two ranges must not overlap.  Owned by the caller.
 *   Enqueued on `stream` in stream order (the copy reads src after the
 *   stream's previous work and later work sees dst); bytes == 0 does nothing.
 *   A pointer whose first or last byte the device cannot reach is refused
 *   with IDX_ERR_INVALID_ARG before anything is enqueued.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_copy_async(void* dst, const void* src, size_t bytes, idx_stream_t stream);

/* ===========================================================================
 * Serving operators around the indexer: the step's page bookkeeping, the
 * rotary tables, the insert into the attention's own key-value cache, and the
 * attention that reads it.  The pages have no counterpart for these entries;
 * they take and give the arrays the indexer's entries use (block tables, slot
 * maps, positions, context lengths, the selected positions).
 *
 * Value types of queries, keys and values: bf16, fp16, and for the cache also
 * FP8 E4M3 (a value is its code times the fp32 scale of its kv head) and MXFP4
 * (E2M1 codes, one UE8M0 scale byte per 32 dimensions, by the rule above).
 * ======================================================================== */
typedef enum {
  IDX_BF16 = 0,
  IDX_FP16 = 1,
  IDX_E4M3 = 2,
  IDX_MXFP4 = 3
} idx_dtype;

/* A paged key-value cache of one attention layer (a host struct, read during
 * the call).  Element (page p, kv head h, token o of the page, dimension d) of
 * the keys is k[p*k_block_stride + h*k_head_stride + o*k_token_stride + d], so
 * that a page may hold its heads one after the other or its tokens one after
 * the other; likewise v.  Strides are in elements, nonnegative, and multiples
 * of 16 bytes; k and v are 16-byte aligned.  Token slot s = page*page_size + o.
 *   page_size 16, 32, 64 or 128; head_dim 64, 128 or 256;
 *   1 <= heads <= 1024; num_blocks * page_size < 2^31.
 *   k_scale, v_scale  [heads] fp32 on the device, for IDX_E4M3 (NULL: all 1);
 *                     NULL for the other types.
 * IDX_MXFP4: a page of a head is page_size * (head_dim/2 + head_dim/32) bytes in one
 * piece, its tokens' codes (head_dim/2 bytes each, element 2i in the low nibble of byte
 * i), then its tokens' scale bytes (head_dim/32 each, 0..254); k + p*k_block_stride +
 * h*k_head_stride is where it starts; block and head strides are in bytes, token strides
 * are 0. */
typedef struct {
  void* k;
  void* v;
  const float* k_scale;
  const float* v_scale;
  int64_t num_blocks;
  int64_t k_block_stride, k_head_stride, k_token_stride;
  int64_t v_block_stride, v_head_stride, v_token_stride;
  int32_t page_size;
  int32_t heads;
  int32_t head_dim;
  int32_t dtype; /* idx_dtype */
} idx_kv_cache;

/* ---------------------------------------------------------------------------
 * idx_plan_step -- block tables, slot maps and positions of a step, built on
 * the GPU from request lengths.
 *   cached_lens  [B] int32: tokens of request b already in the cache.
 *   new_lens     [B] int32: tokens the step adds to it (0: it sits the step out).
 *   block_table  [B, max_blocks] int32, read and written: entries
 *                [0, ceil(cached/page_size)) are the request's pages; the
 *                entries of the pages the step opens are written, no others.
 *   free_pages   [num_free] int32: page ids, taken from the front in the order
 *                of the requests and, within one, of its pages, starting at
 *                entry pool_head[0].
 *   pool_head    [1] int32: entries of free_pages taken so far;
 *   pool_head_out [1] int32 out: the same after this step (another word than
 *                pool_head, which other blocks of the launch may still read).
 *   context_lens [B] int32 out: cached + new; may be cached_lens itself, whose
 *                lengths then advance in place, and one block makes the whole
 *                plan (64K tokens take 195 us, apart 4.7).
 *   query_start  [B+1] int32 out: exclusive sums of new_lens.
 *   slot_mapping [num_tokens] int64, positions [num_tokens] int32, token_seq
 *                [num_tokens] int32 out: for the step's tokens, request by
 *                request, the cache slot, the position in the request, and the
 *                request.  Entries past the step's tokens get -1, 0 and -1.
 * Skipped and counted in errors->bad_inputs: a negative length (the request
 * then counts as empty), a context past INT32_MAX (it then adds nothing), a
 * context past max_blocks pages (tokens there get slot -1), a page missing
 * from the list or outside [0, num_blocks) (block table entry -1, its tokens
 * slot -1), a token whose existing page id is outside the cache (slot -1), and
 * every token past num_tokens (not written).
 * Refused: an array that is written and overlaps another one, context_lens =
 * cached_lens apart.
 *   page_size 16, 32, 64 or 128; num_free may be 0.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_plan_step(const int32_t* cached_lens, const int32_t* new_lens, int32_t B,
                         int32_t* block_table, int32_t max_blocks, const int32_t* free_pages,
                         int32_t num_free, const int32_t* pool_head, int32_t* pool_head_out,
                         int64_t num_blocks, int32_t page_size, int32_t* context_lens,
                         int32_t* query_start, int64_t* slot_mapping, int32_t* positions,
                         int32_t* token_seq, int64_t num_tokens, idx_device_errors* errors,
                         idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_rope_table -- rotary tables, as idx_rope_quant_q and
 * idx_qk_norm_rope_insert take them.
 *   cos_out, sin_out [num_pos, rot_dim/2] fp32 out: row r, column i hold
 *              mscale * cos / sin of (pos0 + r) * w_i.
 *   w_i        base^(-2i/rot_dim), i < rot_dim/2, scaled for long contexts by
 *     IDX_ROPE_NONE    not at all;
 *     IDX_ROPE_LINEAR  w_i / factor (positions interpolated);
 *     IDX_ROPE_NTK     base * factor^(rot_dim/(rot_dim-2)) in place of base;
 *     IDX_ROPE_YARN    w_i for the columns that make at least beta_fast turns
 *                      over orig_len positions, w_i / factor for those that
 *                      make at most beta_slow, a linear blend over the column
 *                      index between (Peng et al., "YaRN", section 3.2).
 *   mscale     factor of every entry (1, or YaRN's attention factor).
 *   rot_dim    even, 2..256 (IDX_ROPE_NTK: 4..256); 0 <= pos0,
 *              pos0 + num_pos <= 2^31.
 * Angles are formed in 64-bit fixed point: beside the frequencies' own fp64
 * rounding they are off by at most 2^-32 of a turn at any position.  Entries are
 * then within 1.5 * 2^-24 where mscale is 1, else within 3.5 * 2^-24 * |mscale|.
 * ------------------------------------------------------------------------ */
typedef enum {
  IDX_ROPE_NONE = 0,
  IDX_ROPE_LINEAR = 1,
  IDX_ROPE_NTK = 2,
  IDX_ROPE_YARN = 3
} idx_rope_scaling;

IDX_API idx_status idx_rope_table(int64_t pos0, int64_t num_pos, int32_t rot_dim, double base,
                          int32_t scaling, double factor, double orig_len, double beta_fast,
                          double beta_slow, double mscale, float* cos_out, float* sin_out,
                          idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_qk_norm_rope_insert -- an attention layer's new queries, keys and values
 * made ready in one pass: RMS norm of every query and key head
 * (x * rsqrt(mean(x^2) + eps) * weight), rotary turn of their first rot_dim
 * dimensions, keys and values stored into the paged cache.
 *   q [N, Hq, D], k and v [N, Hkv, D] of type `dtype` (IDX_BF16 or IDX_FP16),
 *              D = kv->head_dim, Hkv = kv->heads; token and head strides in
 *              elements (multiples of 8), 16-byte aligned: e.g. slices of one
 *              projection's output.
 *   q_weight, k_weight [D] fp32, each may be NULL: that operand is not normed.
 *   positions  [N] int32 rows of cos_table/sin_table [num_pos, rot_dim/2] fp32.
 *   rot_dim    0..D, even; interleaved != 0 turns pairs (2i, 2i+1), else
 *              (i, i + rot_dim/2), then rot_dim is a multiple of 16.
 *              With rot_dim = 0 positions and tables are not read.
 *   slot_mapping [N] int64; -1 = no key and value to store (q is still written).
 *              The others must be distinct: of two tokens of one slot parts of
 *              both may stay (codes and scale bytes of a 4-bit block, too).
 *   q_out      [N, Hq, D], contiguous, of q's type; may be q itself where q is
 *              contiguous.
 * Arithmetic in fp32, rounded once into q_out or the cache; E4M3 codes hold
 * x / scale, rounded to nearest even, magnitudes past 448 saturate; MXFP4 codes follow
 * the rule above, by x as 64 bits give it (infinities, NaN and x past fp32's range are
 * outside the contract there, and so are values past 2^54 for the attention, which takes
 * a key's block with scale byte 0, of values below 2^-124, for zeros).
 * A token whose position is outside the table is skipped whole, one whose slot
 * is outside [0, num_blocks*page_size) stores nothing; both are counted.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_qk_norm_rope_insert(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
    int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
    int64_t v_head_stride, int64_t N, int32_t Hq, int32_t dtype, const float* q_weight,
    const float* k_weight, float eps, const int32_t* positions, const float* cos_table,
    const float* sin_table, int64_t num_pos, int32_t rot_dim, int32_t interleaved,
    const int64_t* slot_mapping, void* q_out, const idx_kv_cache* kv, idx_device_errors* errors,
    idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_paged_attention -- attention of a few new tokens per request over the
 * paged key-value cache, split over the cache's length and joined.
 *   q          [B*next_n, Hq, D] of type `dtype`; row b*next_n + j is token j
 *              of request b; token and head strides in elements (multiples of
 *              8), 16-byte aligned.  Hq is a multiple of kv->heads; query head
 *              h reads kv head h / (Hq / kv->heads).
 *   kv         the cache: of q's type, IDX_E4M3 or IDX_MXFP4.
 *   block_table [B, max_blocks], context_lens [B] int32 as for
 *              idx_paged_mqa_logits: L_b counts the new tokens, row (b, j) sees
 *              positions [0, L_b - next_n + j], with window > 0 only the last
 *              `window` of them.
 *   topk_idx   NULL, or [B*next_n, topk] int32: row r attends to exactly the
 *              positions listed (as idx_paged_logits_topk leaves them; a
 *              negative entry is none; a position listed twice counts twice).
 *              A listed position past the row's sight is skipped and counted.
 *              Needs window = 0.
 *   score      s = scale * q.k, with softcap > 0: softcap * tanh(s / softcap).
 *   out        [B*next_n, Hq, D], contiguous, of q's type: softmax(s) v.
 *   lse        [B*next_n, Hq] fp32 or NULL: ln sum exp(s).
 *              A row that sees nothing gets zeros and -inf.
 *   workspace  at least idx_paged_attention_workspace_bytes(...) bytes, 256-byte
 *              aligned, no initialisation; calls that share it must not overlap.
 * Scores, softmax statistics and sums are fp32 (scores must stay below 2^24, where an
 * fp32 rounding is a factor in the weight; a cap of any size adds at most 2^-20 of the
 * capped score); the weights enter the second
 * product as two 16-bit terms (bf16 over a bf16 or MXFP4 cache; over an fp16 or E4M3 one
 * weights below 2^-32 of a row's highest count as zero; an infinite value in a row's sight gives NaN, one
 * out of it does not reach the row).  Results do not depend on the order in which
 * blocks run.  Over-long contexts (clamped), negative ones (0) and page ids
 * outside the cache (their tokens are not seen) are counted in
 * errors->bad_inputs.
 *   1 <= next_n <= 16; 1 <= topk <= 2^20.
 * ------------------------------------------------------------------------ */
IDX_API size_t idx_paged_attention_workspace_bytes(int32_t B, int32_t next_n, int32_t Hq, int32_t Hkv,
                                           int32_t head_dim);

/* How a call of these sizes shares its work out on a device of `sms` SMs (host
 * only; topk = 0: whole contexts).  An item is a kv head of a request (with a
 * selection, of a query row) with up to `rows` of its query rows. */
typedef struct {
  int32_t split;     /* 1: items cut along their keys over all CTAs and joined */
  int32_t warps;     /* warps that share an item */
  int32_t rows;      /* query rows of an item */
  int32_t row_tiles; /* items a kv head's query rows make */
  int32_t unit;      /* keys by which a split item is cut */
  int32_t places;    /* items (split: CTAs) that run at once */
} idx_attention_form;
IDX_API idx_status idx_paged_attention_form(int32_t B, int32_t next_n, int32_t Hq, int32_t Hkv,
                               int32_t head_dim, int32_t cache_dtype, int32_t page_size,
                               int32_t max_blocks, int32_t topk, int32_t window, int32_t sms,
                               idx_attention_form* form);

IDX_API idx_status idx_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                               int32_t dtype, int32_t B, int32_t next_n, int32_t Hq,
                               const idx_kv_cache* kv, const int32_t* block_table,
                               int32_t max_blocks, const int32_t* context_lens,
                               const int32_t* topk_idx, int32_t topk, float scale, float softcap,
                               int32_t window, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, idx_device_errors* errors,
                               idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_gather_kv -- requests' cached tokens read back into contiguous keys and
 * values, as idx_prompt_attention takes them behind a cached part (idx_gather_k is
 * the same for the indexer's cache).
 *   kv          the cache: of type `dtype`, IDX_E4M3 or IDX_MXFP4.
 *   block_table [B, max_blocks] int32.
 *   key_start   [B+1] int32: request b's positions [0, key_start[b+1] - key_start[b])
 *               go to rows key_start[b] on.
 *   k_out, v_out [out_rows, heads, head_dim] of type `dtype` (IDX_BF16 or IDX_FP16),
 *               contiguous, 16-byte aligned.  Rows of no request are left as they were.
 * 16-bit values are copied; codes times their scale are rounded once (4-bit ones are exact
 * in bf16).  Starts that decrease or lie outside [0, out_rows] are taken into the range,
 * positions past max_blocks pages and those of pages outside the cache are not
 * written; all are counted in errors->bad_inputs, for keys and for values.
 *   out_rows <= 2^30, B <= 65535.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_gather_kv(const idx_kv_cache* kv, const int32_t* block_table, int32_t max_blocks,
                         const int32_t* key_start, int32_t B, int32_t dtype, void* k_out, void* v_out,
                         int64_t out_rows, idx_device_errors* errors, idx_stream_t stream);

/* ---------------------------------------------------------------------------
 * idx_prompt_attention -- attention of whole prompts, or of chunks of them behind
 * a cached part, over contiguous keys and values, sequences packed one behind
 * the other.
 *   q          [T, Hq, D], k and v [S, Hkv, D] of type `dtype` (IDX_BF16 or
 *              IDX_FP16), D = 64, 128 or 256; token and head strides in elements
 *              (positive multiples of 8), 16-byte aligned: e.g. slices of one
 *              projection's output, or what idx_gather_kv leaves.  Hq is a
 *              multiple of Hkv; query head h reads kv head h / (Hq / Hkv).
 *   query_start, key_start [B+1] int32: sequence b's new tokens are rows
 *              [query_start[b], query_start[b+1]) of q, its positions rows
 *              [key_start[b], key_start[b+1]) of k and v.  Of n new tokens and L
 *              positions, token i is position L - n + i; with causal it sees
 *              positions [0, L - n + i], with window > 0 only the last `window` of
 *              them; without causal all L (window is then 0).
 *   score      s = scale * q.k, with softcap > 0: softcap * tanh(s / softcap).
 *   out        [T, Hq, D], contiguous, of q's type: softmax(s) v; lse [T, Hq] fp32
 *              or NULL: ln sum exp(s).  A row that sees nothing gets zeros and
 *              -inf.  Rows outside all sequences are left as they were.  out may not
 *              overlap k, v or (but for q itself, where q is contiguous) q.
 * Scores, softmax statistics and sums are fp32 (scores must stay below 2^24, where an
 * fp32 rounding is a factor in the weight; a cap adds at most 2^-20 of the capped
 * score); each weight is rounded to q's type before it meets its value (by up to 2^-8
 * of itself in bf16, 2^-11 in fp16, small ones there by 2^-28 of the row's highest).
 * Outputs of finite values (bf16: up to 2^127, fp16: 2^15) are finite at any length;
 * bf16 ones are off by up to 2^-137 for every position seen besides.  An infinite or
 * NaN value in a row's sight makes that output infinite or NaN; one out of it does not
 * reach the row.  Results do not depend on the order in which blocks run.  Starts that
 * decrease or lie outside [0, T] or [0, S] are taken into the range and counted in
 * errors->bad_inputs (the rows of their sequences are unspecified).
 * How rows and keys are shared out follows T, S, B and the heads, not the starts (which
 * are on the device): few rows over many keys have their keys shared out where T and B
 * are small and S / B is long.  A call whose T or B leaves room (a captured graph's), or
 * one long sequence among many short ones, may take several times as long.
 *   T <= 2^26, S <= 2^30, B <= 65535, Hq <= 4096.
 * ------------------------------------------------------------------------ */
IDX_API idx_status idx_prompt_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                const void* k, int64_t k_token_stride, int64_t k_head_stride,
                                const void* v, int64_t v_token_stride, int64_t v_head_stride,
                                int32_t dtype, int64_t T, int64_t S, int32_t B, int32_t Hq,
                                int32_t Hkv, int32_t head_dim, const int32_t* query_start,
                                const int32_t* key_start, float scale, float softcap,
                                int32_t window, int32_t causal, void* out, float* lse,
                                idx_device_errors* errors, idx_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* IDX_H_ */
