// mx_api.hip - the C ABI of the MXFP4 operators (declared in include/mxfp4.h): argument
// validation and launches. Every entry point validates all arguments before it enqueues
// anything; on an error it returns a status, enqueues nothing and writes nothing.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "api.hpp"
#include "mx_attn.hpp"
#include "mxfp4.h"

namespace nvfp4 {
int64_t mx_quant_units(int64_t m, int64_t k);
hipError_t launch_mx_quantize(const uint16_t* x, int64_t ldx, const uint16_t* up, int64_t ldu, int64_t m, int64_t k,
                              uint8_t* qdata, uint8_t* scales, const uint16_t* silu_table, hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t* qdata, const uint8_t* scales, uint16_t* y, int64_t ldy, int64_t m,
                                int64_t k, hipStream_t stream);
int64_t mx_cache_groups(int64_t tokens, int64_t head_dim);
hipError_t launch_mx_cache_append(const MxBatch& b, const MxCache& c, const uint16_t* k, int64_t k_token,
                                  int64_t k_head, const uint16_t* v, int64_t v_token, int64_t v_head,
                                  hipStream_t stream);
hipError_t launch_mx_cache_read(const MxBatch& b, const MxCache& c, uint16_t* k, int64_t k_token, int64_t k_head,
                                uint16_t* v, int64_t v_token, int64_t v_head, hipStream_t stream);
hipError_t launch_mx_gemm(const uint8_t* aq, const uint8_t* as, const uint8_t* wq, const uint8_t* ws, uint16_t* d,
                          int64_t ldd, int64_t m, int64_t n, int64_t k, hipStream_t stream);
hipError_t launch_mx_attention(const MxAttnArgs& a, const MxAttnPlan& plan, hipStream_t stream);
}  // namespace nvfp4

using nvfp4::api_device;
using nvfp4::api_fail;
using nvfp4::api_ok;

namespace {

constexpr int64_t kMostK = (int64_t)1 << 23;       // row bytes and scale columns far inside 32 bits
constexpr int64_t kMostRows = (int64_t)1 << 40;    // products of sizes stay far inside 64 bits
constexpr int64_t kMostGroups = (1 << 24) - 1;     // workgroups of 256 threads in a launch

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int check_shape(int64_t rows, int64_t k) {
  if (rows < 0 || k <= 0) return api_fail(NVFP4_ERR_INVALID_ARG, "bad shape rows=%lld k=%lld", (long long)rows, (long long)k);
  if (k % nvfp4::kMxBlock != 0) return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "k=%lld is not a multiple of 32", (long long)k);
  if (k > kMostK || rows > kMostRows || nvfp4::mx_quant_units(rows, k) > kMostGroups)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "tensor too large (rows=%lld k=%lld)", (long long)rows, (long long)k);
  return NVFP4_OK;
}

// a bf16 matrix [rows, k] with row stride ld
int check_matrix(const void* x, int64_t ld, int64_t k, const char* name) {
  if (!x) return api_fail(NVFP4_ERR_INVALID_ARG, "null %s pointer", name);
  if (ld < k) return api_fail(NVFP4_ERR_INVALID_ARG, "%s row stride %lld below k", name, (long long)ld);
  if (ld > kMostK) return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s row stride above 2^23", name);
  if (ld % 8 != 0 || !aligned16(x))
    return api_fail(NVFP4_ERR_MISALIGNED, "%s must be 16-byte aligned, its row stride a multiple of 8", name);
  return NVFP4_OK;
}

int check_packed(const void* qdata, const void* scales) {
  if (!qdata || !scales) return api_fail(NVFP4_ERR_INVALID_ARG, "null codes or scales pointer");
  if (!aligned16(qdata) || !aligned16(scales))
    return api_fail(NVFP4_ERR_MISALIGNED, "codes and scales must be 16-byte aligned");
  return NVFP4_OK;
}

int launched(hipError_t e, const char* what) {
  return e == hipSuccess ? api_ok() : api_fail(NVFP4_ERR_LAUNCH, "%s launch: %s", what, hipGetErrorString(e));
}

int quantize(const void* x, int64_t ldx, const void* up, int64_t ldu, bool swiglu, int64_t rows, int64_t k, void* qdata,
             void* scales, void* stream) {
  int rc = check_shape(rows, k);
  if (rc == NVFP4_OK && rows > 0) rc = check_matrix(x, ldx, k, swiglu ? "gate" : "x");
  if (rc == NVFP4_OK && rows > 0 && swiglu) rc = check_matrix(up, ldu, k, "up");
  if (rc == NVFP4_OK && rows > 0) rc = check_packed(qdata, scales);
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (rows == 0) return api_ok();
  return launched(nvfp4::launch_mx_quantize((const uint16_t*)x, ldx, (const uint16_t*)up, ldu, rows, k, (uint8_t*)qdata,
                                            (uint8_t*)scales, table, (hipStream_t)stream),
                  "quantize");
}

// The cache and the batch of a call; the kernels' forms of both.
int check_cache(const mxfp4_cache* c, const mxfp4_batch* b, nvfp4::MxCache* cache, nvfp4::MxBatch* batch) {
  if (!c || !b) return api_fail(NVFP4_ERR_INVALID_ARG, "null cache or batch");
  if (c->num_pages <= 0 || c->page_size <= 0 || c->kv_heads <= 0 || c->head_dim <= 0)
    return api_fail(NVFP4_ERR_INVALID_ARG, "bad cache: %lld pages of %lld tokens, %lld heads of %lld",
                    (long long)c->num_pages, (long long)c->page_size, (long long)c->kv_heads, (long long)c->head_dim);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "head_dim=%lld is not 64, 128 or 256", (long long)c->head_dim);
  if (c->page_size < 16 || c->page_size > 32768 || (c->page_size & (c->page_size - 1)) != 0)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "page_size=%lld is not a power of two from 16 to 32768",
                    (long long)c->page_size);
  if (c->kv_heads > 1024 || c->num_pages >= (int64_t)1 << 31)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "more than 1024 kv heads or 2^31 - 1 pages");
  if (!c->k_codes_dev || !c->k_scales_dev || !c->v_codes_dev || !c->v_scales_dev)
    return api_fail(NVFP4_ERR_INVALID_ARG, "null cache pointer");
  if (!aligned16(c->k_codes_dev) || !aligned16(c->k_scales_dev) || !aligned16(c->v_codes_dev) ||
      !aligned16(c->v_scales_dev))
    return api_fail(NVFP4_ERR_MISALIGNED, "cache pointers must be 16-byte aligned");
  if (b->batch < 0 || b->tokens < 0 || b->max_pages < 0 || b->table_stride < b->max_pages)
    return api_fail(NVFP4_ERR_INVALID_ARG, "bad batch: %lld sequences, %lld rows, %lld pages (stride %lld)",
                    (long long)b->batch, (long long)b->tokens, (long long)b->max_pages, (long long)b->table_stride);
  if (b->batch >= 1 << 24 || b->tokens >= (int64_t)1 << 31 || b->max_pages * c->page_size >= (int64_t)1 << 30 ||
      b->max_pages >= (int64_t)1 << 27)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "batch beyond 2^24 sequences, 2^31 rows or 2^30 tokens a sequence");
  if (b->batch > 0 && b->tokens > 0) {
    if (!b->seq_lens_dev || !b->cu_seqlens_dev || (b->max_pages > 0 && !b->block_table_dev))
      return api_fail(NVFP4_ERR_INVALID_ARG, "null batch pointer");
    if (((uintptr_t)b->seq_lens_dev & 3u) || ((uintptr_t)b->cu_seqlens_dev & 3u) || ((uintptr_t)b->block_table_dev & 3u))
      return api_fail(NVFP4_ERR_MISALIGNED, "batch pointers must be 4-byte aligned");
  }
  int shift = 0;
  while (((int64_t)1 << shift) < c->page_size) ++shift;
  *cache = nvfp4::MxCache{(uint8_t*)c->k_codes_dev, (uint8_t*)c->k_scales_dev, (uint8_t*)c->v_codes_dev,
                          (uint8_t*)c->v_scales_dev, (int)c->kv_heads, (int)c->head_dim};
  *batch = nvfp4::MxBatch{b->block_table_dev, b->seq_lens_dev, b->cu_seqlens_dev, b->table_stride, c->num_pages,
                          (int)b->batch, (int)b->max_pages, shift, b->tokens};
  return NVFP4_OK;
}

// a packed bf16 tensor [tokens, heads, head_dim]; strides between its rows
int check_packed_rows(const void* x, int64_t token, int64_t head, const char* name) {
  if (!x) return api_fail(NVFP4_ERR_INVALID_ARG, "null %s pointer", name);
  if (token < 0 || head < 0) return api_fail(NVFP4_ERR_INVALID_ARG, "negative %s stride", name);
  if (token > (int64_t)1 << 31 || head > (int64_t)1 << 31)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s stride above 2^31", name);
  if (!aligned16(x) || token % 8 != 0 || head % 8 != 0)
    return api_fail(NVFP4_ERR_MISALIGNED, "%s must be 16-byte aligned, its strides multiples of 8", name);
  return NVFP4_OK;
}

// rows written by a call must not lie in one another
int check_written_rows(int64_t token, int64_t head, int64_t heads, int64_t tokens, int64_t dim, const char* name) {
  const bool by_token = head >= dim && token >= head * (heads - 1) + dim;
  const bool by_head = token >= dim && head >= token * (tokens - 1) + dim;
  if (by_token || by_head || (heads == 1 && token >= dim) || (tokens <= 1 && head >= dim) || (heads == 1 && tokens <= 1))
    return NVFP4_OK;
  return api_fail(NVFP4_ERR_INVALID_ARG, "%s rows overlap (strides %lld, %lld)", name, (long long)token, (long long)head);
}

int move_cache(bool append, const mxfp4_cache* cache, const mxfp4_batch* batch, const void* k, int64_t kt, int64_t kh,
               const void* v, int64_t vt, int64_t vh, void* stream) {
  nvfp4::MxCache c;
  nvfp4::MxBatch b;
  int rc = check_cache(cache, batch, &c, &b);
  const bool any = rc == NVFP4_OK && b.tokens > 0 && b.batch > 0;
  if (any && nvfp4::mx_cache_groups(b.tokens, c.head_dim) > kMostGroups)
    rc = api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "too many rows for one call (%lld)", (long long)b.tokens);
  if (any && rc == NVFP4_OK) rc = check_packed_rows(k, kt, kh, "k");
  if (any && rc == NVFP4_OK) rc = check_packed_rows(v, vt, vh, "v");
  if (any && rc == NVFP4_OK && !append) rc = check_written_rows(kt, kh, c.kv_heads, b.tokens, c.head_dim, "k");
  if (any && rc == NVFP4_OK && !append) rc = check_written_rows(vt, vh, c.kv_heads, b.tokens, c.head_dim, "v");
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (!any) return api_ok();
  if (append)
    return launched(nvfp4::launch_mx_cache_append(b, c, (const uint16_t*)k, kt, kh, (const uint16_t*)v, vt, vh,
                                                  (hipStream_t)stream),
                    "cache append");
  return launched(nvfp4::launch_mx_cache_read(b, c, (uint16_t*)k, kt, kh, (uint16_t*)v, vt, vh, (hipStream_t)stream),
                  "cache read");
}

// What an attention call and its workspace query share.
int check_attention(const mxfp4_cache* cache, const mxfp4_batch* batch, int64_t heads, int64_t max_kv, int64_t window,
                    int64_t sinks, nvfp4::MxCache* c, nvfp4::MxBatch* b, nvfp4::MxAttnPlan* plan) {
  const int rc = check_cache(cache, batch, c, b);
  if (rc != NVFP4_OK) return rc;
  if (heads <= 0 || heads % c->kv_heads != 0)
    return api_fail(NVFP4_ERR_INVALID_ARG, "%lld heads are not a multiple of %d kv heads", (long long)heads, c->kv_heads);
  if (max_kv <= 0) return api_fail(NVFP4_ERR_INVALID_ARG, "max_kv=%lld", (long long)max_kv);
  if (window < 0 || sinks < 0 || (sinks > 0 && window == 0))
    return api_fail(NVFP4_ERR_INVALID_ARG, "window=%lld sinks=%lld (sinks need a window)", (long long)window,
                    (long long)sinks);
  // The workgroups of a launch: 16 packed rows each at least. (Joins have fewer: pieces are made
  // only where there are no 2048 workgroups of up to 32 rows, or 768 of 128.)
  const int64_t packed = heads > 65536 ? -1 : b->tokens * (heads / c->kv_heads);
  if (packed < 0 || packed >= (int64_t)1 << 31 || (packed / 16 + b->batch) * c->kv_heads > kMostGroups)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "too many rows and heads for one call");
  *plan = nvfp4::mx_attention_plan(b->tokens, b->batch, heads, c->kv_heads, c->head_dim, max_kv, window, sinks);
  return NVFP4_OK;
}

int64_t workspace_bytes(const nvfp4::MxBatch& b, const nvfp4::MxCache& c, int64_t heads, const nvfp4::MxAttnPlan& plan) {
  return nvfp4::mx_part_bytes(plan, b.tokens, b.batch, heads, c.kv_heads, c.head_dim);
}

}  // namespace

extern "C" {

int64_t mxfp4_qdata_bytes(int64_t rows, int64_t k) { return (rows < 0 || k < 0) ? -1 : rows * (k / 2); }
int64_t mxfp4_scale_cols(int64_t k) { return k < 0 ? -1 : (k / 32 + 3) / 4 * 4; }
int64_t mxfp4_scale_bytes(int64_t rows, int64_t k) {
  return (rows < 0 || k < 0) ? -1 : (rows + 127) / 128 * 128 * mxfp4_scale_cols(k);
}

int mxfp4_quantize(const void* x_dev, int64_t ld_x, int64_t rows, int64_t k, void* qdata_dev, void* scales_dev,
                   void* stream) {
  return quantize(x_dev, ld_x, nullptr, 0, false, rows, k, qdata_dev, scales_dev, stream);
}

int mxfp4_quantize_swiglu(const void* gate_dev, int64_t ld_gate, const void* up_dev, int64_t ld_up, int64_t m,
                          int64_t k, void* qdata_dev, void* scales_dev, void* stream) {
  return quantize(gate_dev, ld_gate, up_dev, ld_up, true, m, k, qdata_dev, scales_dev, stream);
}

int mxfp4_dequantize(const void* qdata_dev, const void* scales_dev, int64_t rows, int64_t k, void* y_dev, int64_t ld_y,
                     void* stream) {
  int rc = check_shape(rows, k);
  if (rc == NVFP4_OK && rows > 0) rc = check_packed(qdata_dev, scales_dev);
  if (rc == NVFP4_OK && rows > 0) rc = check_matrix(y_dev, ld_y, k, "y");
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (rows == 0) return api_ok();
  return launched(nvfp4::launch_mx_dequantize((const uint8_t*)qdata_dev, (const uint8_t*)scales_dev, (uint16_t*)y_dev,
                                              ld_y, rows, k, (hipStream_t)stream),
                  "dequantize");
}

int mxfp4_gemm_bf16out(const void* a_qdata_dev, const void* a_scales_dev, const void* w_qdata_dev,
                       const void* w_scales_dev, void* d_dev, int64_t ld_d, int64_t m, int64_t n, int64_t k,
                       void* stream) {
  if (n <= 0) return api_fail(NVFP4_ERR_INVALID_ARG, "bad shape n=%lld", (long long)n);
  int rc = check_shape(m, k);
  if (rc == NVFP4_OK) rc = check_shape(n, k);
  if (rc == NVFP4_OK && m > 0) rc = check_packed(a_qdata_dev, a_scales_dev);
  if (rc == NVFP4_OK && m > 0) rc = check_packed(w_qdata_dev, w_scales_dev);
  if (rc == NVFP4_OK && m > 0) {
    if (!d_dev || ld_d < n) rc = api_fail(NVFP4_ERR_INVALID_ARG, "null output, or row stride %lld below n", (long long)ld_d);
    else if ((uintptr_t)d_dev & 1u) rc = api_fail(NVFP4_ERR_MISALIGNED, "output must be 2-byte aligned");
    else if ((m + 63) / 64 * ((n + 63) / 64) > kMostGroups || ld_d > (int64_t)1 << 40)
      rc = api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "output too large (m=%lld n=%lld)", (long long)m, (long long)n);
  }
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (m == 0) return api_ok();
  return launched(nvfp4::launch_mx_gemm((const uint8_t*)a_qdata_dev, (const uint8_t*)a_scales_dev,
                                        (const uint8_t*)w_qdata_dev, (const uint8_t*)w_scales_dev, (uint16_t*)d_dev,
                                        ld_d, m, n, k, (hipStream_t)stream),
                  "gemm");
}

int mxfp4_cache_append(const mxfp4_cache* cache, const mxfp4_batch* batch, const void* k_dev, int64_t k_token_stride,
                       int64_t k_head_stride, const void* v_dev, int64_t v_token_stride, int64_t v_head_stride,
                       void* stream) {
  return move_cache(true, cache, batch, k_dev, k_token_stride, k_head_stride, v_dev, v_token_stride, v_head_stride, stream);
}

int mxfp4_cache_read(const mxfp4_cache* cache, const mxfp4_batch* batch, void* k_dev, int64_t k_token_stride,
                     int64_t k_head_stride, void* v_dev, int64_t v_token_stride, int64_t v_head_stride, void* stream) {
  return move_cache(false, cache, batch, k_dev, k_token_stride, k_head_stride, v_dev, v_token_stride, v_head_stride, stream);
}

int64_t mxfp4_attention_workspace_bytes(const mxfp4_cache* cache, const mxfp4_batch* batch, int64_t heads,
                                        int64_t max_kv, int64_t window, int64_t sinks) {
  nvfp4::MxCache c;
  nvfp4::MxBatch b;
  nvfp4::MxAttnPlan plan;
  if (check_attention(cache, batch, heads, max_kv, window, sinks, &c, &b, &plan) != NVFP4_OK) return -1;
  return workspace_bytes(b, c, heads, plan);
}

int mxfp4_attention(const mxfp4_cache* cache, const mxfp4_batch* batch, const void* q_dev, int64_t q_token_stride,
                    int64_t q_head_stride, int64_t heads, float scale, int causal, int64_t window, int64_t sinks,
                    int64_t max_kv, void* out_dev, int64_t out_token_stride, int64_t out_head_stride,
                    void* workspace_dev, int64_t workspace_size, void* stream) {
  nvfp4::MxCache c;
  nvfp4::MxBatch b;
  nvfp4::MxAttnPlan plan;
  int rc = check_attention(cache, batch, heads, max_kv, window, sinks, &c, &b, &plan);
  if (rc != NVFP4_OK) return rc;
  if (!(scale > 0.0f && scale <= 0x1p127f)) return api_fail(NVFP4_ERR_INVALID_ARG, "scale must be positive, at most 2^127");
  if (window > 0 && !causal) return api_fail(NVFP4_ERR_INVALID_ARG, "a window needs causal attention");
  const bool any = b.tokens > 0 && b.batch > 0;
  if (any) {
    rc = check_packed_rows(q_dev, q_token_stride, q_head_stride, "q");
    if (rc == NVFP4_OK) rc = check_packed_rows(out_dev, out_token_stride, out_head_stride, "out");
    if (rc == NVFP4_OK) rc = check_written_rows(out_token_stride, out_head_stride, heads, b.tokens, c.head_dim, "out");
    if (rc != NVFP4_OK) return rc;
    const int64_t need = workspace_bytes(b, c, heads, plan);
    if (need > 0 && !workspace_dev) return api_fail(NVFP4_ERR_WORKSPACE, "null workspace; %lld bytes needed", (long long)need);
    if (workspace_size < need)
      return api_fail(NVFP4_ERR_WORKSPACE, "workspace of %lld bytes; %lld needed", (long long)workspace_size, (long long)need);
    if (need > 0 && !aligned16(workspace_dev)) return api_fail(NVFP4_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  }
  const uint16_t* table = nullptr;
  rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (!any) return api_ok();
  nvfp4::MxAttnArgs a{};
  a.b = b;
  a.c = c;
  a.q = (const uint16_t*)q_dev;
  a.out = (uint16_t*)out_dev;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.out_token = out_token_stride;
  a.out_head = out_head_stride;
  a.heads = (int)heads;
  a.group = (int)(heads / c.kv_heads);
  a.scale_log2 = scale * 1.44269504f;
  a.raise = fminf(nvfp4::kMxRaise / a.scale_log2, FLT_MAX);
  // lengths stay below 2^30: a window or first tokens beyond that hide nothing more
  a.causal = causal != 0;
  a.window = (int)(window < (1 << 30) ? window : 1 << 30);
  a.sinks = (int)(sinks < (1 << 30) ? sinks : 1 << 30);
  a.splits = plan.splits;
  a.part_o = (float*)workspace_dev;
  a.part_ml = (float2*)((float*)workspace_dev + plan.splits * b.tokens * heads * c.head_dim);
  return launched(nvfp4::launch_mx_attention(a, plan, (hipStream_t)stream), "attention");
}

}  // extern "C"
