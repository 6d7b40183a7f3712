/*
 * mxfp4.h - C ABI of the MXFP4 operators (MI355X, gfx950), in the same library as nvfp4.h.
 *
 * MXFP4 keeps 32 consecutive elements of a row under one power-of-two scale, where NVFP4
 * keeps 16 under an E4M3 scale and a whole tensor under an FP32 one. gfx950's scaled matrix
 * instructions multiply it as it is stored, at four times the fp16 rate, and nothing
 * outside a block is needed to quantize it, so a tensor can be quantized as it is written:
 * a projection's activations in one pass, and a key/value cache token by token.
 *
 * Conventions are those of nvfp4.h: device pointers on the current HIP device owned by the
 * caller, `stream` a hipStream_t as void*, asynchronous calls that allocate nothing, all
 * arguments validated before anything is enqueued, an nvfp4_status returned and
 * nvfp4_last_error() describing a failure. Contents of device memory are not validated on
 * the host; where a kernel takes an index from there, what happens with one out of range is
 * said below, and no access leaves the buffers described.
 *
 * Format:
 *  - Block: 32 consecutive elements of a row, A = their largest magnitude.
 *    Scale byte S = max(floor(log2 A) - 2 + 127, 0) (E8M0, value 2^(S-127); 0 for A = 0),
 *    at most 252 for finite elements. A block with an infinity or a NaN has S = 255 and
 *    codes 0 and reads back as NaN throughout. Bytes 253 and 254 are never written; the
 *    operators that read a cache expect it as the library wrote it.
 *  - Codes: E2M1 as in nvfp4.h, the magnitude nearest to |x| / 2^(S-127), ties to the even
 *    code, above 6 to 6, with the sign of x (also on zero); two per byte, the first element
 *    in the low nibble.
 *  - Value: e2m1(code) * 2^(S-127), exact in bf16 for every byte that is written.
 *  - Matrices: codes row-major [rows, k/2], not padded. Scales in the 512-byte tiles of
 *    nvfp4.h (128 rows x 4 scale columns) with C = mxfp4_scale_cols(k) columns of 32
 *    elements: byte (r, c) at
 *      ((r >> 7) * (C / 4) + (c >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (c & 3)
 *    Bytes outside real rows and columns are zero.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- sizes (pure functions; no device access) ------------------------------------- */

/* Code bytes: rows * k / 2. Returns -1 if rows < 0 or k < 0. */
int64_t mxfp4_qdata_bytes(int64_t rows, int64_t k);

/* Scale columns: roundup(k / 32, 4). Returns -1 if k < 0. */
int64_t mxfp4_scale_cols(int64_t k);

/* Scale bytes: roundup(rows, 128) * mxfp4_scale_cols(k). Returns -1 if rows < 0 or k < 0. */
int64_t mxfp4_scale_bytes(int64_t rows, int64_t k);

/* ---- quantization -------------------------------------------------------------------- */

/*
 * MXFP4 of a bf16 matrix, in one launch that reads it once.
 *
 * x_dev      : bf16 [rows, k] row-major, row stride ld_x (elements, a multiple of 8, >= k);
 *              16-byte aligned. Read only.
 * rows, k    : rows >= 0 (0: nothing is written, the pointers may be NULL), k > 0,
 *              k % 32 == 0, k and ld_x at most 2^23; ceil(rows / 128) * ceil(k / 512) < 2^21
 *              (the limits of every [rows, k] below).
 * qdata_dev  : out, mxfp4_qdata_bytes(rows, k) bytes, 16-byte aligned.
 * scales_dev : out, mxfp4_scale_bytes(rows, k) bytes, 16-byte aligned; every byte is
 *              written, padding included.
 */
int mxfp4_quantize(const void* x_dev, int64_t ld_x, int64_t rows, int64_t k, void* qdata_dev, void* scales_dev,
                   void* stream);

/* MXFP4 of y = RN_bf16(silu_bf16(gate) * up), the y of nvfp4_quantize_swiglu bit for bit
 * (silu correctly rounded to bf16), in one launch. gate and up as x in mxfp4_quantize. */
int mxfp4_quantize_swiglu(const void* gate_dev, int64_t ld_gate, const void* up_dev, int64_t ld_up, int64_t m,
                          int64_t k, void* qdata_dev, void* scales_dev, void* stream);

/* The reverse: y[r, c] = the value of element (r, c), bf16 [rows, k] with row stride ld_y
 * (a multiple of 8, >= k), 16-byte aligned. Elements of rows past k are left as they were. */
int mxfp4_dequantize(const void* qdata_dev, const void* scales_dev, int64_t rows, int64_t k, void* y_dev, int64_t ld_y,
                     void* stream);

/* ---- product -------------------------------------------------------------------------- */

/*
 * D[m, n] = RN_bf16(sum_k A[m, k] * W[n, k]), products exact, FP32 accumulation.
 *
 * a_*, w_* : matrices [m, k] and [n, k] as mxfp4_quantize writes them.
 * d_dev    : out, bf16 [m, n], row stride ld_d >= n (elements), 2-byte aligned. Rows take
 *            wide stores where d_dev is 16-byte aligned and n and ld_d are multiples of 8.
 * m >= 0 (0: nothing is done), n > 0, k > 0, k % 32 == 0, both matrices within the limits of
 * mxfp4_quantize; ceil(m / 64) * ceil(n / 64) < 2^24, ld_d at most 2^40.
 * Every element of D is summed in an order that the sizes alone decide: no atomics, no
 * workspace, no state between calls.
 */
int mxfp4_gemm_bf16out(const void* a_qdata_dev, const void* a_scales_dev, const void* w_qdata_dev,
                       const void* w_scales_dev, void* d_dev, int64_t ld_d, int64_t m, int64_t n, int64_t k,
                       void* stream);

/* ---- paged key/value cache ------------------------------------------------------------- */

/* Keys and values of many sequences in pages of page_size tokens, all in device memory:
 * codes [num_pages, kv_heads, page_size, head_dim / 2] and scales [num_pages, kv_heads,
 * page_size, head_dim / 32], contiguous, 16-byte aligned. head_dim 64, 128 or 256 (blocks
 * run along it); page_size a power of two, 16 to 32768; kv_heads at most 1024, num_pages
 * below 2^31. */
typedef struct {
  void* k_codes_dev;
  void* k_scales_dev;
  void* v_codes_dev;
  void* v_scales_dev;
  int64_t num_pages, page_size, kv_heads, head_dim;
} mxfp4_cache;

/* Rows of a packed batch. Sequence b has rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of the
 * packed tensors (tokens rows in all, batch + 1 ascending entries from 0); its cache holds
 * seq_lens[b] tokens, of which its rows are the last: row i of n has position
 * seq_lens[b] - n + i. Position p lies in page block_table[b, p / page_size]
 * (int32 [batch, max_pages], row stride table_stride >= max_pages). batch < 2^24, tokens < 2^31,
 * max_pages < 2^27, max_pages * page_size < 2^30.
 *
 * seq_lens is clamped to [0, max_pages * page_size] and cu_seqlens to [0, tokens]; a page
 * number outside [0, num_pages) is a page that is not there. Rows past the last sequence
 * belong to none. */
typedef struct {
  const int32_t* block_table_dev;
  const int32_t* seq_lens_dev;
  const int32_t* cu_seqlens_dev;
  int64_t batch, max_pages, table_stride, tokens;
} mxfp4_batch;

/*
 * Quantizes new keys and values into the cache at their rows' positions.
 *
 * k_dev, v_dev : bf16 [tokens, kv_heads, head_dim] with strides (elements, multiples of 8,
 *                at most 2^31) between tokens and between heads; 16-byte aligned. Read only.
 * tokens       : at most (2^24 - 1) * 2048 / head_dim, here and in mxfp4_cache_read.
 * Rows without a position (negative, or on a page that is not there) and rows of no
 * sequence are skipped. Nothing else of the cache is touched. Two rows at one place (a page
 * written by two sequences of the batch) leave its contents undefined.
 */
int mxfp4_cache_append(const mxfp4_cache* cache, const mxfp4_batch* batch, const void* k_dev, int64_t k_token_stride,
                       int64_t k_head_stride, const void* v_dev, int64_t v_token_stride, int64_t v_head_stride,
                       void* stream);

/* Reads the rows' keys and values back as bf16 (strides as in mxfp4_cache_append). Rows
 * without a position read as zeros; rows of no sequence are left as they were. */
int mxfp4_cache_read(const mxfp4_cache* cache, const mxfp4_batch* batch, void* k_dev, int64_t k_token_stride,
                     int64_t k_head_stride, void* v_dev, int64_t v_token_stride, int64_t v_head_stride, void* stream);

/* ---- attention over the cache ----------------------------------------------------------- */

/* Bytes of mxfp4_attention's workspace for a call of these sizes (0: none needed), with the
 * same cache, batch, heads, max_kv, window and sinks; -1 for arguments that the call itself
 * refuses. */
int64_t mxfp4_attention_workspace_bytes(const mxfp4_cache* cache, const mxfp4_batch* batch, int64_t heads,
                                        int64_t max_kv, int64_t window, int64_t sinks);

/*
 * out[i, h] = sum_t softmax_t(scale * q[i, h] . k[t, h / g]) v[t, h / g], g = heads / kv_heads,
 * over the cached tokens t of row i's sequence that it sees: t < seq_len and t <= p (with
 * causal != 0), p the row's position; with window > 0 also t > p - window or t < sinks (a
 * sliding window of `window` tokens, the row's own among them, and the first `sinks` tokens,
 * which stay visible). Tokens on a page that is not there are not seen. A row that sees
 * nothing gives zeros. A NaN in the cache reaches the rows that see it and no others.
 *
 * q_dev, out_dev : bf16 [tokens, heads, head_dim] with token and head strides (elements,
 *                  multiples of 8, at most 2^31); 16-byte aligned. out_dev may be q_dev with
 *                  the same strides. Rows of no sequence are left as they were. The rows'
 *                  own keys and values are in the cache already (mxfp4_cache_append with the
 *                  same batch, before).
 * heads          : a multiple of kv_heads, at most 65536; tokens * heads / kv_heads < 2^31 and
 *                  (tokens * heads / kv_heads / 16 + batch) * kv_heads < 2^24.
 * scale          : > 0, at most 2^127. Scores q . k are fp32 sums and have to lie in its range;
 *                  scale times them need not.
 * window, sinks  : >= 0; a window needs causal, sinks need a window.
 * max_kv         : the longest cache of the batch as far as the caller knows (> 0). It only
 *                  decides how the work is split, not the result's meaning.
 * workspace_dev  : at least mxfp4_attention_workspace_bytes(...) bytes, 16-byte aligned; may
 *                  be NULL if that is 0. Its contents before and after mean nothing. Calls
 *                  that may overlap in time need distinct workspaces.
 * Scores, the softmax and its sums are fp32; weights are rounded to bf16 for their product
 * with the values, and so for their sum: against exact weights that moves an element by at most
 * 2^-8 (sum_t w_t |v_t| + |out|). Sums of weights and values are taken before the division, of
 * weights up to 2^12: values up to 2^80 in magnitude cannot overflow them. The order of every sum
 * depends on the arguments and lengths alone.
 */
int mxfp4_attention(const mxfp4_cache* cache, const mxfp4_batch* batch, const void* q_dev, int64_t q_token_stride,
                    int64_t q_head_stride, int64_t heads, float scale, int causal, int64_t window, int64_t sinks,
                    int64_t max_kv, void* out_dev, int64_t out_token_stride, int64_t out_head_stride,
                    void* workspace_dev, int64_t workspace_bytes, void* stream);

/* ---- attention behind shared prefixes ---------------------------------------------------- */

/* Groups of consecutive sequences that begin with the same tokens (answers to one prompt,
 * questions behind one set of instructions). Group g has the sequences group_starts[g] ..
 * group_starts[g + 1] - 1 of the batch (groups + 1 ascending entries; sequences before the first
 * and from the last on are in no group); its prefix is the lens[g] tokens in the pages of row g
 * of its block table (int32 [groups, max_pages], row stride table_stride >= max_pages), of which the first
 * lens[g] / 64 * 64 are shared. groups < 2^24, max_pages < 2^27, max_pages * page_size < 2^30.
 * lens is clamped to [0, max_pages * page_size] and group_starts to [0, batch]. */
typedef struct {
  const int32_t* block_table_dev;
  const int32_t* lens_dev;
  const int32_t* group_starts_dev;
  int64_t groups, max_pages, table_stride;
} mxfp4_prefix;

/* Bytes of mxfp4_attention_prefix's workspace for a call of these sizes; -1 for arguments that
 * the call itself refuses. */
int64_t mxfp4_attention_prefix_workspace_bytes(const mxfp4_cache* cache, const mxfp4_batch* batch,
                                               const mxfp4_prefix* prefix, int64_t heads, int64_t max_prefix,
                                               int64_t max_own);

/*
 * mxfp4_attention without a window, where a sequence's shared tokens are read through its
 * group's block table and only the others through its own row of the batch's: the cached prefix is
 * read once for all rows of a group. Of a sequence whose first row does not see all of the shared
 * tokens (with causal: its position + 1 is smaller than their number; without: its length is), and of
 * one in no group, all tokens are read through its own row.
 *
 * A sequence's own row is not read below the shared tokens; above them a page that holds the first of its
 * own tokens is its own.
 * max_prefix, max_own : the longest prefix, and the most tokens of a sequence behind its own, as
 *                       far as the caller knows (> 0). They only decide how the work is split; one that is far too
 *                       large costs time (24 sequences of 4 rows, 500 tokens of their own behind 8,000: 35 us, with 8,500 49).
 * The rest as in mxfp4_attention; tokens * heads at most 2^26 - 4 and (tokens * heads / kv_heads / 16 * 2 +
 * batch + groups) * kv_heads < 2^24.
 */
int mxfp4_attention_prefix(const mxfp4_cache* cache, const mxfp4_batch* batch, const mxfp4_prefix* prefix,
                           const void* q_dev, int64_t q_token_stride, int64_t q_head_stride, int64_t heads, float scale,
                           int causal, int64_t max_prefix, int64_t max_own, void* out_dev, int64_t out_token_stride,
                           int64_t out_head_stride, void* workspace_dev, int64_t workspace_bytes, void* stream);

/* ---- norms and rotation of heads --------------------------------------------------------- */

/* n = x w / sqrt(mean(x^2) + eps) over the head_dim elements of a head. weight_dev: bf16
 * [head_dim], 16-byte aligned, or NULL for ones; eps > 0 and finite. */
typedef struct {
  const void* weight_dev;
  double eps;
} mxfp4_norm;

/* Rotation of the first rotary_dim elements of a head by pairs: (a, b) becomes
 * (a cos t - b sin t, b cos t + a sin t), t = position * freqs[j]. Pair j is (j, j + rotary_dim / 2),
 * with interleaved != 0 (2 j, 2 j + 1).
 *
 * rotary_dim    : a multiple of 16, 16 to head_dim.
 * freqs_dev     : fp32 [rotary_dim / 2], finite, 4-byte aligned.
 * axes_dev      : int32 [rotary_dim / 2], which of a row's positions turns the pair (of
 *                 time, height and width, say), clamped to [0, axes); NULL: axis 0.
 * positions_dev : int32, that of row i on axis x at [i * token_stride + x * axis_stride] (elements,
 *                 0 to 2^31); NULL in a call with a cache: the row's position in its sequence, on every axis.
 * axes          : 1 to 64.
 * Angles are taken in fp64 for every position, whatever its size, and are those of the exact product to 2^-44 of a
 * turn for frequencies up to 2^32. */
typedef struct {
  const float* freqs_dev;
  const int32_t* axes_dev;
  const int32_t* positions_dev;
  int64_t rotary_dim, axes, token_stride, axis_stride;
  int interleaved;
} mxfp4_rotation;

/*
 * out[i, h] = RN_bf16(rotation(norm(x[i, h]))), in one launch that reads x once.
 *
 * x_dev, out_dev : bf16 [tokens, heads, head_dim] with token and head strides (elements,
 *                  multiples of 8, at most 2^31); 16-byte aligned. out_dev may be x_dev with the
 *                  same strides. head_dim 64, 128 or 256; heads 1 to 65536; tokens at most 2^26 - 4.
 * norm, rotation : each may be NULL (left out).
 * Sums and products are fp32 (fp64 for heads whose squares leave its range, and with an eps above 2^100).
 * A head with an infinity or a NaN comes out as the formulas have it.
 */
int mxfp4_norm_rope(const void* x_dev, int64_t x_token_stride, int64_t x_head_stride, int64_t tokens, int64_t heads,
                    int64_t head_dim, const mxfp4_norm* norm, const mxfp4_rotation* rotation, void* out_dev,
                    int64_t out_token_stride, int64_t out_head_stride, void* stream);

/*
 * What stands between a QKV projection and mxfp4_attention, in one launch: q as mxfp4_norm_rope
 * writes it (q_norm); k likewise (k_norm), its bf16 values then quantized into the cache; v
 * quantized into the cache as it is. Places are those of mxfp4_cache_append, whose rules for
 * rows hold: rows of no sequence are left out (and their q as it was), a row without a place
 * leaves the cache as it is, and its q is written.
 *
 * q_dev, q_out_dev : bf16 [tokens, heads, head_dim]; with heads == 0 none (NULL); at most 65536. The row's
 *                    head_dim and kv_heads are the cache's; tokens at most 2^26 - 4.
 * k_dev, v_dev     : bf16 [tokens, kv_heads, head_dim].
 * Norm and rotation of k are fp64 throughout: a last bit decides the way to 4 bits.
 */
int mxfp4_norm_rope_append(const mxfp4_cache* cache, const mxfp4_batch* batch, const void* q_dev, int64_t q_token_stride,
                           int64_t q_head_stride, int64_t heads, const mxfp4_norm* q_norm, const void* k_dev,
                           int64_t k_token_stride, int64_t k_head_stride, const mxfp4_norm* k_norm, const void* v_dev,
                           int64_t v_token_stride, int64_t v_head_stride, const mxfp4_rotation* rotation,
                           void* q_out_dev, int64_t out_token_stride, int64_t out_head_stride, void* stream);

/* ---- pages --------------------------------------------------------------------------------- */

/* Which pages the sequences of a cache hold, all in device memory. A sequence is a slot: row
 * s of the block table (int32 [slots, max_pages], row stride table_stride >= max_pages) and its length
 * seq_lens[s], which is clamped to [0, max_pages * page_size]. It holds the first
 * ceil(length / page_size) entries. refs[p] (int32 [num_pages]) is how many entries
 * hold page p; a page whose count is below 1 is free. slots < 2^24, num_pages < 2^31, the rest as in
 * mxfp4_batch. Page numbers outside [0, num_pages) count as no page. Several caches (the
 * layers of a model) can go by one such record.
 *
 * Lists of slots are int32 in device memory, n < 65536 entries; entries outside [0, slots) are passed
 * over. Results do not depend on timing. done_dev says for each entry whether it was
 * carried out (1) or left everything as it was (0). */
typedef struct {
  int32_t* block_table_dev;
  int32_t* seq_lens_dev;
  int32_t* refs_dev;
  int64_t slots, max_pages, table_stride, num_pages, page_size;
} mxfp4_pages;

/* Cuts each listed sequence back to keep_dev[i] tokens (NULL: none) if it is longer; pages
 * behind them are given back, their entries become -1. A slot that is listed twice keeps the
 * smaller number. */
int mxfp4_pages_free(const mxfp4_pages* pages, const int32_t* slots_dev, const int32_t* keep_dev, int64_t n,
                     void* stream);

/* Makes slot children_dev[i] a copy of the sequence in parents_dev[i], which then share their
 * pages, a last one that is not full among them. Not done where the child's length is not 0,
 * where an earlier entry has the same child, and where the parent is itself a child in the list. */
int mxfp4_pages_fork(const mxfp4_pages* pages, const int32_t* parents_dev, const int32_t* children_dev, int64_t n,
                     int32_t* done_dev, void* stream);

/* Bytes of mxfp4_pages_reserve's workspace; -1 for arguments that the call itself refuses. */
int64_t mxfp4_pages_reserve_workspace_bytes(const mxfp4_pages* pages, int64_t n);

/*
 * Lengthens sequence slots_dev[i] to lens_dev[i] tokens, with new pages for them. A last page that is
 * not full and that other entries hold too is replaced: src_dev[i] is the page, dst_dev[i] the
 * new one, into which mxfp4_cache_copy has to copy it in every cache before its next token is written and before
 * pages are given out again; both are -1 where there is none.
 *
 * Pages are given out lowest first, in the list's order. Not done where the length is below the
 * present one or beyond max_pages * page_size, where an earlier entry has the same slot, and where it needs
 * pages and the need of the entries up to it (served or not) is more than the pages that were free.
 * workspace_dev: 16-byte aligned, mxfp4_pages_reserve_workspace_bytes bytes.
 */
int mxfp4_pages_reserve(const mxfp4_pages* pages, const int32_t* slots_dev, const int32_t* lens_dev, int64_t n,
                        int32_t* done_dev, int32_t* src_dev, int32_t* dst_dev, void* workspace_dev,
                        int64_t workspace_bytes, void* stream);

/* Bytes of mxfp4_pages_compact's workspace; -1 for arguments that the call itself refuses. */
int64_t mxfp4_pages_compact_workspace_bytes(const mxfp4_pages* pages);

/*
 * Numbers the used pages so that they are the first ones: with u in use, those at u and above move, in order, into
 * the free ones below u. Page src_dev[k] becomes dst_dev[k] (int32 [num_pages / 2] each,
 * ascending, -1 behind the last), used_dev[0] = u. The new block table and counts go to table_out_dev
 * (row stride table_out_stride >= max_pages) and refs_out_dev, which may be those of `pages`: with buffers
 * of their own the old ones stay in use until mxfp4_cache_copy has moved the pages, which
 * it does not disturb. workspace_dev: 16-byte aligned.
 * ceil(num_pages / 256) + slots * ceil(max_pages / 256) < 2^24.
 */
int mxfp4_pages_compact(const mxfp4_pages* pages, int32_t* table_out_dev, int64_t table_out_stride, int32_t* refs_out_dev,
                        int32_t* src_dev, int32_t* dst_dev, int32_t* used_dev, void* workspace_dev,
                        int64_t workspace_bytes, void* stream);

/*
 * Copies whole pages of keys and values, src_dev[i] of `from` to dst_dev[i] of `to` (int32 [n], n < 2^31),
 * which may be one cache and differ in num_pages at most. A pair with a page out of range moves
 * nothing. A page that is written by two pairs, or read by one and written by another,
 * leaves what is written undefined.
 */
int mxfp4_cache_copy(const mxfp4_cache* from, const mxfp4_cache* to, const int32_t* src_dev, const int32_t* dst_dev,
                     int64_t n, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
