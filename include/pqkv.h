/*
 * pqkv.h -- C-ABI of libpqkv: quantize-and-append into a paged KV cache and
 * paged decode / speculative-verify attention over it, on one GB300 (sm_103a).
 *
 * The operations follow the KV design on the ReVolta README (pages
 * "ReVolta" README and "v0.1.3" release note):
 *   - "Weight and KV formats": the KV cache is stored compressed as FP8 E4M3
 *     (calibrated per-layer K and V scales, "E4M3 KV"), INT8 ("INT8 KV") or
 *     FP16, and widened to FP16 for the arithmetic;
 *   - "Quick start", launch: MTP verify with 4 speculative tokens, i.e. one
 *     committed and four draft query positions per sequence, causally masked
 *     among themselves; GQA through the model's query / KV head counts;
 *   - "Hardware" and "Quick start": decode context parallelism splits a
 *     sequence's keys across GPUs and combines the partial results; here the
 *     split is across thread blocks of one GPU and the partials are merged by
 *     log-sum-exp;
 *   - release note "Known issues": 16-token kernel pages.
 *
 * Pool layout (this library's choice):
 *   pages[num_pages][num_kv_heads][2][page_size][head_dim]
 * where index 0 of the third axis is K and 1 is V; elements are 1-byte codes
 * (E4M3, INT8) or fp16.  Slot s of the pool is token s % page_size of page
 * s / page_size.  For one (page, kv-head) the K tile and the V tile are
 * contiguous (4 KB for 8-bit codes), which is what the attention kernel
 * streams.
 * PQKV_KV_INT8_ROW pools carry a scale area right after the codes, in the same
 * allocation (num_pages*num_kv_heads*4096 bytes from the start of `pages`):
 *   fp16 row_scale[num_pages][num_kv_heads][8][4]
 * (IEEE binary16), where [p][h][i] holds the scales of K row i, K row i+8,
 * V row i and V row i+8 of page p, kv-head h -- the order in which the
 * attention kernel's matrix fragments consume them.  That is 64 bytes per
 * (page, kv-head); the allocation is num_pages*num_kv_heads*4160 bytes.
 * PQKV_KV_INT4_GROUP pools hold 4-bit codes with an fp16 scale per group of 32
 * consecutive values of a row:
 *   pages[num_pages][num_kv_heads][2][1152 bytes]
 * (0.5625 of an 8-bit pool).  Of the 1152 bytes of a K or V tile the first 1024
 * are codes, 64 bytes a row: row r's group c is the 16-byte chunk
 * (4 (r % 2) + c) ^ (0, 5, 2, 7)[i % 4] of the 128-byte line i = r / 2.  Value
 * 8 w + 2 f + e of the group is in 32-bit word w of the chunk, half e, field f:
 * the bits of code + 8 at 6-9, 2-5, 10-13, and (lowest first) 14, 15, 0, 1 of the half
 * for f = 0 .. 3.  Behind them: fp16 scale[4 groups][16 rows].  A page is
 * contiguous with its scales, so pages may be copied as they are; tokens are
 * taken out again by pqkv_kv_read.
 *
 * Conventions for every entry point:
 *   - All tensor arguments are DEVICE pointers owned by the caller.  Nothing
 *     is allocated, freed or retained.  Between calls the library keeps only
 *     a per-device cache of device properties, and -- the one exception --
 *     the scratch area of pqkv_paged_attention_noalloc (a file-scope device
 *     array present on every GPU that loads the library, its per-device
 *     address cache and the last call's contents; see that entry point).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream), in stream order.  Most kernels are launched with
 *     programmatic dependent launch allowed: their blocks may become resident
 *     while the previous kernel on the stream finishes, but they wait for it
 *     to complete (and its writes to be visible) before touching memory, so
 *     the ordering is that of a plain launch.  The return value reports
 *     argument validation and launch errors only.
 *   - Errors that only the device can see are OR-ed as PQKV_DEV_* bits into
 *     `*status` (a device int32, may be NULL).  The offending work is skipped;
 *     no kernel traps, asserts or waits without a bound.
 */
#ifndef PQKV_H
#define PQKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* KV element formats. */
typedef enum {
  PQKV_KV_FP16 = 0,     /* fp16 values, scales ignored                          */
  PQKV_KV_FP8_E4M3 = 1, /* OCP E4M3 ("FN": max 448, no Inf), value = dec(c)*scale */
  PQKV_KV_INT8 = 2,     /* symmetric int8 in [-127, 127], value = c*scale         */
  PQKV_KV_INT8_ROW = 3, /* int8 with its own scale per (token, kv-head) row of K
                           and of V, computed when the row is written (ReVolta
                           README, "Weight and KV formats", "INT8 KV": scales
                           derived from the data at run time, no calibration);
                           value = c * row_scale.  Scale area: see the layout. */
  PQKV_KV_INT4_GROUP = 5 /* 4-bit codes in [-7, 7] with an fp16 scale per group of 32
                           consecutive values of a (token, kv-head) row, computed
                           when the row is written; value = c * scale.  (No counterpart
                           on the ReVolta pages.  4 is not a format.) */
} pqkv_kv_dtype;

/* Host-side return codes. */
enum {
  PQKV_OK = 0,
  PQKV_EINVAL = -1,       /* null pointer, bad size, misaligned pointer         */
  PQKV_EUNSUPPORTED = -2, /* valid but not implemented (head_dim != 128, ...)   */
  PQKV_ERANGE = -3,       /* a size is outside the supported range              */
  PQKV_EWORKSPACE = -4,   /* workspace missing or smaller than required         */
  PQKV_ECUDA = -5         /* a CUDA runtime call or a launch failed             */
};

/* Device-side status bits (OR-ed into *status). */
enum {
  PQKV_DEV_SLOT_RANGE = 1,    /* append: slot >= num_pages*page_size; token skipped.
                                 block tables: the free-page stack ran out or over      */
  PQKV_DEV_SEQ_RANGE = 2,     /* attention: seq_len < q_len or beyond its block-table row;
                                 shared prefix, block tables: see there                 */
  PQKV_DEV_BAD_SCALE = 4,     /* a scale is not finite and > 0; work skipped        */
  PQKV_DEV_TIMEOUT = 8,       /* a pipeline wait ran out (about 1 s); outputs invalid */
  PQKV_DEV_PAGE_RANGE = 16    /* attention: block-table entry outside [0, num_pages); read as
                                 zeros.  extend: a token's page, which gets no slot.  truncate:
                                 an entry below 0, pushed all the same                     */
};

/* Largest supported sizes. */
#define PQKV_HEAD_DIM 128
#define PQKV_PAGE_SIZE 16
#define PQKV_MAX_Q_LEN 8
#define PQKV_MAX_ROWS 32          /* (num_q_heads / num_kv_heads) * q_len        */
#define PQKV_MAX_SEQS 2048
#define PQKV_MAX_SPLITS 128
#define PQKV_MAX_SEQ_LEN 524288   /* ReVolta README, "Performance": 512K boundary */

/*
 * pqkv_kv_append_quant -- quantize new K and V tokens and write them into
 * their pool slots.  (ReVolta README, "Weight and KV formats": KV is stored
 * compressed; E4M3 uses calibrated per-layer scales, INT8 a scale per head.)
 *
 * For every token t with slot_mapping[t] >= 0, kv-head h and dim d:
 *     pages[slot/ps][h][0][slot%ps][d] = Q(fp32(k[t,h,d]) / fp32(k_scale[h']))
 *     pages[slot/ps][h][1][slot%ps][d] = Q(fp32(v[t,h,d]) / fp32(v_scale[h']))
 * where the quotient is the correctly rounded IEEE binary32 division, h' = h
 * if scale_per_head else 0, and Q is
 *     E4M3: round to nearest, ties to even, saturate to +-448 (Inf -> +-448,
 *           NaN -> 0x7F), zero keeps its sign;
 *     INT8: round half to even, clamp to [-127, 127] (NaN -> 0);
 *     FP16: the fp16 bits unchanged (scales ignored, may be NULL).
 * INT8_ROW: for each written (token, kv-head) row x of K (and of V) the row's
 * scale r = fp16(amax / 127), the binary16 value nearest the exact quotient
 * (ties to even), amax = the largest |x_d| of the row (NaNs ignored; 0 for a
 * row of zeros), is stored in the scale area at the row's slot and the codes
 * are the INT8 codes of fp32(x_d) / fp32(r).  A zero r (amax <= 127 * 2^-25)
 * gives 0/0 = NaN -> code 0 and +-x/0 -> +-127, all worth 0.  k_scale /
 * v_scale are ignored (may be NULL).  V rows with amax above 32512 exceed what the attention kernel's
 * fp16 products hold (probability <= 256 times the row scale).
 * INT4_GROUP: for each group of 32 values the scale s = min(fp16(bf16(amax/7)), 2720),
 * amax the largest |x| of the group (NaNs ignored, at most 65504) and bf16 and fp16
 * the roundings to nearest even, is stored in its tile; the codes are
 * fp32(x)/s rounded half to even and clamped to [-7, 7] (NaN -> 0; all 0 for s = 0).
 * A scale has 8 significant bits, so every value code * s is an fp16 value.
 * Values beyond +-19040 saturate.  k_scale / v_scale are ignored (may be NULL).
 * How exact: rows of N(0, 1) values are off by 9.7 % (rms, of their rms), where
 * E4M3 under one scale is off by 2.6 %, INT8 1.1 % and INT8_ROW 0.7 %; with 1 %
 * of the values twenty times as large 15.7 % (E4M3 2.6, INT8 8.0, INT8_ROW 2.1).
 *
 *   k, v            fp16 [num_tokens][num_kv_heads][head_dim]; heads and dims
 *                   contiguous, tokens `k_token_stride` / `v_token_stride`
 *                   ELEMENTS apart (>= num_kv_heads*head_dim), so K and V may
 *                   be column slices of a fused QKV buffer.
 *   slot_mapping    int64 [num_tokens]; negative = skip the token (padding).
 *                   Two tokens with the same slot: the result is unspecified.
 *   k_scale/v_scale fp32 [1] or [num_kv_heads] (device).
 *   pages           the pool (layout above); num_pages pages.
 * Requires head_dim == 128, page_size == 16, all pointers 16-byte aligned and
 * token strides multiples of 8 elements.  num_tokens == 0 is a no-op.
 */
int pqkv_kv_append_quant(const void* k, int64_t k_token_stride, const void* v,
                         int64_t v_token_stride, const int64_t* slot_mapping,
                         int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                         int32_t kv_dtype, const float* k_scale, const float* v_scale,
                         int32_t scale_per_head, void* pages, int64_t num_pages,
                         int32_t page_size, int32_t* status, void* stream);

/*
 * pqkv_kv_read -- the tokens of requests out of the pool, as contiguous fp16
 * rows: a request's cached context for a dense attention over it (the chunk of a
 * prompt that follows), or on its way to another pool, format or machine.  (The
 * ReVolta pages describe no such kernel.)
 *
 * For request s and token_offsets[s] <= t < token_offsets[s+1], with
 * pos = first_pos[s] + t - token_offsets[s], row t of k and of v receives the
 * values of the request's token pos, kv-heads and dims in order:
 *   FP16        the bits;
 *   E4M3, INT8  fp16(fp32(dec(code) * scale));
 *   INT8_ROW    fp16(code * row scale), rounded once;
 *   INT4_GROUP  code * group scale, exact.
 * Rows behind token_offsets[num_seqs] are left as they are.  So are rows whose
 * pos lies outside the request's block-table row (PQKV_DEV_SEQ_RANGE) or whose
 * scale is not finite and > 0 (PQKV_DEV_BAD_SCALE).  A block-table entry outside
 * [0, num_pages) reads as zeros (PQKV_DEV_PAGE_RANGE).  token_offsets that do
 * not start at 0, fall, or end beyond num_tokens are reported
 * (PQKV_DEV_SEQ_RANGE); then which rows are written is unspecified, but no
 * others than the num_tokens rows of k and v.
 *
 *   block_table    int32 [num_seqs][max_pages_per_seq].
 *   first_pos      int32 [num_seqs] or NULL (all 0): the first position read.
 *   token_offsets  int32 [num_seqs+1] (as pqkv_extend_block_tables writes them).
 *   k, v           fp16 [num_tokens][num_kv_heads][head_dim]; tokens
 *                  `k_token_stride` / `v_token_stride` ELEMENTS apart
 *                  (>= num_kv_heads*head_dim, multiples of 16), so they may be
 *                  column slices of a wider buffer.  32-byte aligned.
 *   k_scale, v_scale, scale_per_head  as in pqkv_kv_append_quant.
 * num_seqs <= 2048, head_dim == 128, page_size == 16, pages 16-byte aligned.
 * num_seqs == 0 or num_tokens == 0 is a no-op.  Stateless: no workspace.
 */
int pqkv_kv_read(const void* pages, int64_t num_pages, const int32_t* block_table,
                 int32_t max_pages_per_seq, const int32_t* first_pos, const int32_t* token_offsets,
                 int32_t num_seqs, int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                 int32_t page_size, int32_t kv_dtype, const float* k_scale, const float* v_scale,
                 int32_t scale_per_head, void* k, int64_t k_token_stride, void* v,
                 int64_t v_token_stride, int32_t* status, void* stream);

/*
 * pqkv_paged_attention_workspace_size -- bytes of device workspace that
 * pqkv_paged_attention needs for these sizes and split mode (0 if none).
 * num_splits as in pqkv_paged_attention.  Pure host function; for balanced
 * calls the size is that of the largest grid on any device.  The first PQKV_COUNTER_BYTES(num_seqs,
 * num_kv_heads) bytes of the workspace are merge counters: they must be zero
 * before the first call, and every call that returns with *status clean
 * leaves them zero again.  Zero the whole workspace once after allocating it
 * (and again after a call that reported PQKV_DEV_TIMEOUT).  Behind them lie
 * partial results, so calls with more counters than an earlier one need a
 * workspace of their own, or one that starts so much earlier that all calls'
 * counters end at the same byte.
 */
size_t pqkv_paged_attention_workspace_size(int32_t num_seqs, int32_t q_len,
                                           int32_t num_q_heads, int32_t num_kv_heads,
                                           int32_t head_dim, int32_t num_splits);

/*
 * pqkv_paged_attention -- decode (q_len == 1) or verify (q_len > 1)
 * attention of each sequence's new query positions over its paged,
 * quantized K/V, with GQA and split-KV partitions merged by log-sum-exp.
 * (ReVolta README, "Quick start": MTP4 verify and the FLASH_ATTN_V100
 * backend; "Weight and KV formats": K/V dequantized for compute; "Hardware":
 * decode context parallel split of the keys.)
 *
 * For sequence s with L = seq_lens[s] cached tokens (its q_len new tokens
 * already appended), query i < q_len sits at position p = L - q_len + i and
 * attends to tokens j <= p.  Query head hq reads kv-head
 * hq / (num_q_heads / num_kv_heads).  With K_j = dec(kcode_j) * k_scale and
 * V_j = dec(vcode_j) * v_scale:
 *     out[s*q_len + i][hq][:] = sum_j softmax_j(q . K_j / sqrt(head_dim)) V_j
 * computed in fp32 with fp16 tensor-core products (probabilities rounded to fp16, each
 * off by at most 2^-11 of it or 2^-25 of the row's largest; INT8_ROW: their products
 * with V's row scales), and rounded to fp16.  A V that is not finite in one of the
 * q_len new tokens also reaches the rows of the queries before it, as 0 times it.
 * A NaN among the scores of the keys that a row sees (from a NaN or an infinity in its
 * query, or in a K) makes the row NaN, however the keys are split; a row whose scores are
 * all -inf gets 0.
 * Scores may be up to 2^26 in size: from 2^28 on an fp32 step of a score is a factor that
 * fp16 probabilities do not hold.
 *
 *   q, out            fp16 [num_seqs*q_len][num_q_heads][head_dim], contiguous.
 *   pages             the pool (layout above), num_pages pages, 16-byte aligned.
 *   block_table       int32 [num_seqs][max_pages_per_seq]: the pool page of
 *                     each logical 16-token page of the sequence.
 *   seq_lens          int32 [num_seqs] (device), q_len <= L <= max_pages_per_seq*16.
 *   k_scale, v_scale  fp32 [1] or [num_kv_heads] (device); ignored for FP16,
 *                     INT8_ROW and INT4_GROUP (the last two use the scales stored
 *                     at token j's slot).
 *   num_splits        0: balanced split -- the key pages of all sequences and
 *                     kv-heads are cut into one equal contiguous share per
 *                     resident thread block, and a sequence's shares are
 *                     merged by log-sum-exp;  k >= 1: every (sequence, kv-head)
 *                     is cut into k near-equal partitions (k == 1: no merge).
 *   max_seq_len       an upper bound of seq_lens used to size the balanced
 *                     grid (0: max_pages_per_seq*16).
 *   workspace         device scratch of pqkv_paged_attention_workspace_size()
 *                     bytes (may be NULL when that size is 0), 256-byte
 *                     aligned; see the counter rule above.  Calls that share a
 *                     workspace must not overlap on the device.
 * Requires head_dim == 128, page_size == 16, 1 <= q_len <= 8,
 * (num_q_heads/num_kv_heads)*q_len <= 32, num_seqs <= 2048.
 * The result does not depend on the order of pages in the pool; for a fixed
 * split mode and device it is bitwise reproducible run to run.
 */
int pqkv_paged_attention(const void* q, void* out, const void* pages, int64_t num_pages,
                         const int32_t* block_table, int32_t max_pages_per_seq,
                         const int32_t* seq_lens, int32_t num_seqs, int32_t q_len,
                         int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                         int32_t page_size, int32_t kv_dtype, const float* k_scale,
                         const float* v_scale, int32_t scale_per_head, int32_t num_splits,
                         int32_t max_seq_len, void* workspace, size_t workspace_bytes,
                         int32_t* status, void* stream);

/*
 * pqkv_paged_attention_window -- pqkv_paged_attention with a sliding window:
 * query position p attends to the `window` most recent keys, itself included,
 * i.e. keys j with p - window < j <= p.  (ReVolta README, "DFlash2
 * speculative decoding": the drafter's sliding-window layers use a 2048-token
 * window.)  Pages that lie wholly before every query's window are not read, so
 * the cost follows the window, not the cache length.
 *
 * Same arguments as pqkv_paged_attention, plus:
 *   window   >= 1: the window in tokens; 0: no window (exactly
 *            pqkv_paged_attention); negative: PQKV_EINVAL.
 * The workspace rules are those of pqkv_paged_attention (its size query
 * covers this call).
 */
int pqkv_paged_attention_window(const void* q, void* out, const void* pages, int64_t num_pages,
                                const int32_t* block_table, int32_t max_pages_per_seq,
                                const int32_t* seq_lens, int32_t num_seqs, int32_t q_len,
                                int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                int32_t page_size, int32_t kv_dtype, const float* k_scale,
                                const float* v_scale, int32_t scale_per_head, int32_t num_splits,
                                int32_t max_seq_len, int32_t window, void* workspace,
                                size_t workspace_bytes, int32_t* status, void* stream);

/*
 * pqkv_paged_attention_partial -- one rank's part of a decode context
 * parallel split (ReVolta README, "Hardware": TP4 + DCP2; "Quick start",
 * launch: --decode-context-parallel-size 2): each rank holds a contiguous,
 * page-aligned share of every sequence's keys, attends over it, and the ranks'
 * results are combined by pqkv_lse_merge (after an all-gather across ranks).
 *
 * Same arguments as pqkv_paged_attention, except:
 *   seq_lens   int32 [num_seqs]: keys of each sequence held here (0 allowed);
 *   q_pos      int32 [num_seqs] (device): local index of query 0's position,
 *              i.e. its global position minus the global index of this
 *              share's first key; query i sees local keys j <= q_pos + i,
 *              j < seq_lens[s] (any value: a negative position sees none);
 *   out_o      fp32 [num_seqs*q_len][num_q_heads][head_dim]: O / l of the
 *              share (0 for a row that sees no key);
 *   out_lse    fp32 [num_seqs*q_len][num_q_heads]: m + ln(l), the natural-log
 *              log-sum-exp of the row's scores over the share (-inf when the
 *              row sees no key; NaN with a NaN among the scores).
 * Scores are q . K_j / sqrt(head_dim) as in pqkv_paged_attention.  out_o must
 * be 16-byte aligned.
 */
int pqkv_paged_attention_partial(const void* q, const void* pages, int64_t num_pages,
                                 const int32_t* block_table, int32_t max_pages_per_seq,
                                 const int32_t* seq_lens, const int32_t* q_pos, int32_t num_seqs,
                                 int32_t q_len, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim, int32_t page_size, int32_t kv_dtype,
                                 const float* k_scale, const float* v_scale,
                                 int32_t scale_per_head, int32_t num_splits, int32_t max_seq_len,
                                 float* out_o, float* out_lse, void* workspace,
                                 size_t workspace_bytes, int32_t* status, void* stream);

/*
 * pqkv_lse_merge -- combine partial results of the same rows (the merge step
 * of the split above): with parts p = 0 .. num_parts-1,
 *     LSE = ln sum_p e^{lse_p},   out = sum_p e^{lse_p - LSE} o_p   (fp16)
 * Parts with lse_p = -inf contribute nothing; a row whose lse_p are all -inf
 * gets out = 0 and LSE = -inf.  A NaN lse_p makes its row NaN.
 *   part_o    fp32 [num_parts][num_rows][head_dim], 16-byte aligned;
 *   part_lse  fp32 [num_parts][num_rows];
 *   out       fp16 [num_rows][head_dim], 16-byte aligned;
 *   out_lse   fp32 [num_rows] or NULL (for a further merge level).
 * num_rows = num_seqs*q_len*num_q_heads for pqkv_paged_attention_partial's
 * outputs.  Requires head_dim == 128.
 */
int pqkv_lse_merge(const float* part_o, const float* part_lse, int32_t num_parts,
                   int64_t num_rows, int32_t head_dim, void* out, float* out_lse, void* stream);

/* Size of the library-owned scratch area used by pqkv_paged_attention_noalloc
 * (16 MiB, held on every GPU that loads the library until the process exits). */
#define PQKV_NOALLOC_SCRATCH_BYTES (16u << 20)

/*
 * pqkv_paged_attention_noalloc -- pqkv_paged_attention for callers that cannot
 * allocate device memory.  (No counterpart on the ReVolta pages: an addition of
 * this library for callers such as runtimes that budget all device memory up
 * front and forbid cudaMalloc at call time, hooks running inside another
 * framework's step that must not bypass its allocator, or C callers with no
 * allocator at all.)
 *
 * Same arguments and result as pqkv_paged_attention without the workspace:
 * the library uses its own fixed scratch area of PQKV_NOALLOC_SCRATCH_BYTES, a
 * file-scope device array.  Nothing is allocated or freed, by the library or by
 * any routine it calls.
 *   - Returns PQKV_ERANGE when the workspace of the launch this call makes
 *     exceeds PQKV_NOALLOC_SCRATCH_BYTES.  That is the grid the call actually
 *     uses, not the largest one pqkv_paged_attention_workspace_size() assumes:
 *     with RP = (num_q_heads/num_kv_heads)*q_len rounded up to a multiple of
 *     8, it needs PQKV_COUNTER_BYTES(num_seqs, num_kv_heads) plus about
 *     n*RP*520 bytes, where n = num_seqs*num_kv_heads*num_splits for
 *     num_splits >= 2, and n = num_seqs*num_kv_heads + G for num_splits == 0,
 *     G the balanced grid (at most the blocks resident on the device at once:
 *     one per SM in this build); num_splits == 1 needs none.
 *   - All arguments are checked before anything is queued: a rejected call
 *     leaves the scratch area untouched.
 *   - The first call on a device that needs scratch looks up the array's
 *     device address (cudaGetSymbolAddress) with that device current; make
 *     that first call before any stream capture begins.
 *   - Every call on a device shares the one scratch area and it keeps the last
 *     call's contents; each call clears the part that must start at zero
 *     (cudaMemsetAsync on `stream`, queued just before the kernel).  Calls that
 *     overlap on the GPU (different streams, or concurrent host threads) race
 *     on it and must be serialised by the caller.
 */
int pqkv_paged_attention_noalloc(const void* q, void* out, const void* pages, int64_t num_pages,
                                 const int32_t* block_table, int32_t max_pages_per_seq,
                                 const int32_t* seq_lens, int32_t num_seqs, int32_t q_len,
                                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t page_size, int32_t kv_dtype, const float* k_scale,
                                 const float* v_scale, int32_t scale_per_head, int32_t num_splits,
                                 int32_t max_seq_len, int32_t* status, void* stream);

/*
 * pqkv_paged_attention_shared_prefix -- pqkv_paged_attention for a batch whose
 * sequences share prefixes (a system prompt, a long document): the keys of a
 * shared prefix are read once per 256 query rows of a kv-head of the sequences that
 * share it, instead of once per sequence.  (ReVolta README, "Quick start": 8 concurrent requests
 * with prefix caching; the pages describe no kernel for it.)
 *
 * The sequences come in groups of neighbours: group g holds sequences
 * group_offsets[g] .. group_offsets[g+1]-1, whose first prefix_lens[g] tokens
 * are the same tokens IN THE SAME POOL PAGES, so their block-table rows agree
 * over the first floor(prefix_lens[g]/16) entries; the entries of the group's
 * first row are the ones read.  The result is that of pqkv_paged_attention on
 * the same arguments (up to the order of the sums).  Shared are the whole pages
 * of min(prefix_lens[g], min over the group of seq_lens[s] - q_len): a prefix
 * that ends inside a page, and the q_len new tokens, stay private.
 * prefix_lens[g] < 16 shares nothing; groups may be empty.  One sequence shorter than
 * the prefix (the padding of a batch, say) cuts what its whole group shares: it belongs
 * in a group of its own, without a prefix.
 * When it pays (one GB300, 32 query heads on 8, one group): a call has four launches,
 * 24 to 30 us at least, and private keys run at about a quarter of the memory's rate.
 * Against pqkv_paged_attention on the same tables, decode gains from about 64K tokens
 * saved on (sequences times prefix; 32K for FP16 pools), verification of 5 positions
 * from the smallest batches on; below, or with private parts longer than the prefix, a
 * decode call takes up to 20 us more, and a batch that shares nothing is better off
 * with pqkv_paged_attention.
 *
 *   q, out, pages, block_table, seq_lens, k_scale, v_scale, status and the
 *   size arguments as in pqkv_paged_attention.
 *   group_offsets   int32 [num_groups+1] (device), from 0 to num_seqs, not
 *                   falling; otherwise PQKV_DEV_SEQ_RANGE, and nothing is shared
 *                   (the result is still right).
 *   prefix_lens     int32 [num_groups] (device); negative, or longer than a
 *                   sequence of the group: PQKV_DEV_SEQ_RANGE, and clamped.
 *   max_seq_len, max_prefix_len  upper bounds of seq_lens and prefix_lens
 *                   (0: unknown).  They size the grids, and no more than
 *                   max_prefix_len tokens of a prefix are shared (under 16:
 *                   none, and nothing is launched for them); the result is
 *                   right whatever they are.
 *   workspace       device scratch of at least
 *                   pqkv_paged_attention_shared_prefix_workspace_size() bytes,
 *                   256-byte aligned.  It needs no initial value and keeps
 *                   nothing between calls.  Calls that share a workspace must
 *                   not overlap on the device.
 * 1 <= num_groups <= 2048.  Bitwise reproducible run to run on one device.
 */
int pqkv_paged_attention_shared_prefix(
    const void* q, void* out, const void* pages, int64_t num_pages, const int32_t* block_table,
    int32_t max_pages_per_seq, const int32_t* seq_lens, int32_t num_seqs,
    const int32_t* group_offsets, const int32_t* prefix_lens, int32_t num_groups, int32_t q_len,
    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
    int32_t kv_dtype, const float* k_scale, const float* v_scale, int32_t scale_per_head,
    int32_t max_seq_len, int32_t max_prefix_len, void* workspace, size_t workspace_bytes,
    int32_t* status, void* stream);

/* Bytes of workspace of pqkv_paged_attention_shared_prefix for these sizes (0
 * for sizes it refuses).  Pure host function. */
size_t pqkv_paged_attention_shared_prefix_workspace_size(int32_t num_seqs, int32_t num_groups,
                                                         int32_t q_len, int32_t num_q_heads,
                                                         int32_t num_kv_heads, int32_t head_dim);

/*
 * pqkv_extend_block_tables -- grow every request by its new tokens: take the
 * pages it needs from a stack of free pages, write them into its block-table
 * row, and give every token its pool slot and its position, all on the device.
 * (ReVolta v0.1.3 release note, "Known issues": 16-token kernel pages.  The
 * pages leave the allocation to their serving engine; the stack is this
 * library's choice.)
 *
 * With L = seq_lens[s], n = new_tokens[s], have = ceil(L/16),
 * need = ceil((L+n)/16) - have, and upto the sum of need over requests 0..s:
 *   - the request is SERVED when need == 0 or upto <= free_count; its j-th new
 *     page is free_pages[free_count - 1 - (upto - need + j)] (the stack's top
 *     first), written to block_table[s][have + j];
 *   - its tokens follow those of the requests before it in slot_mapping:
 *     token i sits at position pos = L + i in slot
 *     block_table[s][pos/16]*16 + pos%16;
 *   - seq_lens_out[s] = L + n.
 * A request that is not served keeps its length, takes no page, and its n
 * tokens get slot -1 (which pqkv_kv_append_quant skips) and position -1.  It
 * is not served
 *   - when the stack runs out (PQKV_DEV_SLOT_RANGE); no later request gets
 *     pages then, while requests that need none are still served;
 *   - when L or n is negative, L + n exceeds max_pages_per_seq*16, or its
 *     tokens end beyond num_tokens (PQKV_DEV_SEQ_RANGE).
 * A token whose page id is outside [0, num_pages) gets slot and position -1
 * (PQKV_DEV_PAGE_RANGE).
 *
 *   seq_lens, new_tokens  int32 [num_seqs].
 *   block_table    int32 [num_seqs][max_pages_per_seq]; only new entries are written.
 *   free_pages     int32 [max_free_pages], the stack; entries 0..free_count-1
 *                  are free pages.  Not written.
 *   free_count     int32 [1]; outside [0, max_free_pages] it is clamped
 *                  (PQKV_DEV_SLOT_RANGE).
 *   seq_lens_out   int32 [num_seqs], free_count_out int32 [1]: the state after
 *                  the call; either may be the input itself (in place).
 *   slot_mapping   int64 [num_tokens]: one entry per token of the step's batch;
 *                  entries behind the last request's tokens become -1.
 *   positions      int32 [num_tokens] or NULL, -1 where the slot is.
 *   token_offsets  int32 [num_seqs+1] or NULL: each request's first token (and
 *                  the end), at most num_tokens.
 * The other outputs must not overlap the inputs.  num_seqs <= 2048,
 * page_size == 16.  Stateless: no workspace.
 */
int pqkv_extend_block_tables(const int32_t* seq_lens, const int32_t* new_tokens, int32_t num_seqs,
                             int32_t* block_table, int32_t max_pages_per_seq,
                             const int32_t* free_pages, const int32_t* free_count,
                             int32_t max_free_pages, int64_t num_pages, int32_t page_size,
                             int32_t* seq_lens_out, int32_t* free_count_out, int64_t* slot_mapping,
                             int32_t* positions, int32_t num_tokens, int32_t* token_offsets,
                             int32_t* status, void* stream);

/*
 * pqkv_truncate_block_tables -- shorten requests and push their pages back on
 * the stack: draft tokens that a verify step rejected, or whole requests that
 * have ended.  (ReVolta README, "Quick start": MTP verify of 4 draft tokens,
 * of which any number may be rejected.)
 *
 * Request s keeps its first keep_lens[s] tokens.  The pages with index in
 * [max(ceil(keep/16), owned_pages[s]), ceil(seq_lens[s]/16)) of its row are
 * pushed, requests in order, pages in order, from free_pages[free_count] on.
 * The row itself is left as it is.
 * A request with keep < 0, keep > seq_lens[s], or seq_lens[s] beyond its row
 * is left as it is (PQKV_DEV_SEQ_RANGE).  Pages that find no room on the stack
 * (free_count would exceed max_free_pages) are dropped (PQKV_DEV_SLOT_RANGE).
 * Page ids are pushed as the row has them; one below 0, which no pool has, is
 * reported (PQKV_DEV_PAGE_RANGE).  The pool's size is not known here: an id
 * beyond it is reported by the extend that hands it out.
 *
 *   owned_pages  int32 [num_seqs] or NULL (all 0): the row's first page that
 *                belongs to this request; the pages before it are another's
 *                (a shared prefix) and are never pushed.
 *   seq_lens_out, free_count_out  as in pqkv_extend_block_tables.
 */
int pqkv_truncate_block_tables(const int32_t* seq_lens, const int32_t* keep_lens,
                               const int32_t* owned_pages, int32_t num_seqs,
                               const int32_t* block_table, int32_t max_pages_per_seq,
                               int32_t* free_pages, const int32_t* free_count,
                               int32_t max_free_pages, int32_t page_size, int32_t* seq_lens_out,
                               int32_t* free_count_out, int32_t* status, void* stream);

/* Bytes at the start of the workspace that hold merge counters. */
#define PQKV_COUNTER_BYTES(num_seqs, num_kv_heads) \
  ((((size_t)(num_seqs) * (size_t)(num_kv_heads) * 4u) + 255u) & ~(size_t)255u)

/* Static description of a return code, or of a device status word holding any
 * combination of OR-ed PQKV_DEV_* bits ("device: a; b"); "unknown status" for
 * anything else.  The returned string lives until the process exits. */
const char* pqkv_status_string(int code);

/* Library version as "major.minor.patch". */
const char* pqkv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PQKV_H */
