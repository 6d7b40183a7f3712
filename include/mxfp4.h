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

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
