// mx_api.hip - the C ABI of the MXFP4 operators (declared in include/mxfp4.h): argument
// validation and launches. Every entry point validates all arguments before it enqueues
// anything; on an error it returns a status, enqueues nothing and writes nothing.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "api.hpp"
#include "mx_attn.hpp"
#include "mx_pages.hpp"
#include "mx_rope.hpp"
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
hipError_t launch_mx_attention_prefix(const MxAttnArgs& a, const MxPrefixPlan& plan, hipStream_t stream);
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

int check_page_size(int64_t size) {
  if (size < 16 || size > 32768 || (size & (size - 1)) != 0)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "page_size=%lld is not a power of two from 16 to 32768", (long long)size);
  return NVFP4_OK;
}

int page_shift_of(int64_t size) {
  int shift = 0;
  while (((int64_t)1 << shift) < size) ++shift;
  return shift;
}

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

int check_pages_of_cache(const mxfp4_cache* c, nvfp4::MxCache* cache) {
  if (c->num_pages <= 0 || c->page_size <= 0 || c->kv_heads <= 0 || c->head_dim <= 0)
    return api_fail(NVFP4_ERR_INVALID_ARG, "bad cache: %lld pages of %lld tokens, %lld heads of %lld",
                    (long long)c->num_pages, (long long)c->page_size, (long long)c->kv_heads, (long long)c->head_dim);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "head_dim=%lld is not 64, 128 or 256", (long long)c->head_dim);
  const int rc = check_page_size(c->page_size);
  if (rc != NVFP4_OK) return rc;
  if (c->kv_heads > 1024 || c->num_pages >= (int64_t)1 << 31)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "more than 1024 kv heads or 2^31 - 1 pages");
  if (!c->k_codes_dev || !c->k_scales_dev || !c->v_codes_dev || !c->v_scales_dev)
    return api_fail(NVFP4_ERR_INVALID_ARG, "null cache pointer");
  if (!aligned16(c->k_codes_dev) || !aligned16(c->k_scales_dev) || !aligned16(c->v_codes_dev) ||
      !aligned16(c->v_scales_dev))
    return api_fail(NVFP4_ERR_MISALIGNED, "cache pointers must be 16-byte aligned");
  *cache = nvfp4::MxCache{(uint8_t*)c->k_codes_dev, (uint8_t*)c->k_scales_dev, (uint8_t*)c->v_codes_dev,
                          (uint8_t*)c->v_scales_dev, (int)c->kv_heads, (int)c->head_dim};
  return NVFP4_OK;
}

// The cache and the batch of a call; the kernels' forms of both.
int check_cache(const mxfp4_cache* c, const mxfp4_batch* b, nvfp4::MxCache* cache, nvfp4::MxBatch* batch) {
  if (!c || !b) return api_fail(NVFP4_ERR_INVALID_ARG, "null cache or batch");
  const int rc = check_pages_of_cache(c, cache);
  if (rc != NVFP4_OK) return rc;
  if (b->batch < 0 || b->tokens < 0 || b->max_pages < 0 || b->table_stride < b->max_pages)
    return api_fail(NVFP4_ERR_INVALID_ARG, "bad batch: %lld sequences, %lld rows, %lld pages (stride %lld)",
                    (long long)b->batch, (long long)b->tokens, (long long)b->max_pages, (long long)b->table_stride);
  if (b->batch >= 1 << 24 || b->tokens >= (int64_t)1 << 31 || b->max_pages * c->page_size >= (int64_t)1 << 30 ||
      b->max_pages >= (int64_t)1 << 27)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "batch beyond 2^24 sequences, 2^31 rows or 2^30 tokens a sequence");
  if (b->batch > 0 && b->tokens > 0) {
    if (!b->seq_lens_dev || !b->cu_seqlens_dev || (b->max_pages > 0 && !b->block_table_dev))
      return api_fail(NVFP4_ERR_INVALID_ARG, "null batch pointer");
    if (!aligned4(b->seq_lens_dev) || !aligned4(b->cu_seqlens_dev) || !aligned4(b->block_table_dev))
      return api_fail(NVFP4_ERR_MISALIGNED, "batch pointers must be 4-byte aligned");
  }
  *batch = nvfp4::MxBatch{b->block_table_dev, b->seq_lens_dev, b->cu_seqlens_dev, b->table_stride, c->num_pages,
                          (int)b->batch, (int)b->max_pages, page_shift_of(c->page_size), b->tokens};
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

int check_workspace(const void* workspace, int64_t size, int64_t need) {
  if (need > 0 && !workspace) return api_fail(NVFP4_ERR_WORKSPACE, "null workspace; %lld bytes needed", (long long)need);
  if (size < need) return api_fail(NVFP4_ERR_WORKSPACE, "workspace of %lld bytes; %lld needed", (long long)size, (long long)need);
  if (need > 0 && !aligned16(workspace)) return api_fail(NVFP4_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  return NVFP4_OK;
}

int check_scale(float scale) {
  return scale > 0.0f && scale <= 0x1p127f ? NVFP4_OK : api_fail(NVFP4_ERR_INVALID_ARG, "scale must be positive, at most 2^127");
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

// the rows and scale of an attention call, and its workspace of `need` bytes
int check_attention_rows(const nvfp4::MxBatch& b, const nvfp4::MxCache& c, const void* q, int64_t qt, int64_t qh, int64_t heads,
                         const void* out, int64_t ot, int64_t oh, const void* workspace, int64_t size, int64_t need) {
  int rc = check_packed_rows(q, qt, qh, "q");
  if (rc == NVFP4_OK) rc = check_packed_rows(out, ot, oh, "out");
  if (rc == NVFP4_OK) rc = check_written_rows(ot, oh, heads, b.tokens, c.head_dim, "out");
  if (rc != NVFP4_OK) return rc;
  return check_workspace(workspace, size, need);
}

nvfp4::MxAttnArgs attention_args(const nvfp4::MxBatch& b, const nvfp4::MxCache& c, const void* q, int64_t qt, int64_t qh,
                                 int64_t heads, float scale, int causal, void* out, int64_t ot, int64_t oh, void* workspace) {
  nvfp4::MxAttnArgs a{};
  a.b = b;
  a.c = c;
  a.q = (const uint16_t*)q;
  a.out = (uint16_t*)out;
  a.q_token = qt;
  a.q_head = qh;
  a.out_token = ot;
  a.out_head = oh;
  a.heads = (int)heads;
  a.group = (int)(heads / c.kv_heads);
  a.scale_log2 = scale * 1.44269504f;
  a.raise = fminf(nvfp4::kMxRaise / a.scale_log2, FLT_MAX);
  a.causal = causal != 0;
  a.part_o = (float*)workspace;
  return a;
}

// What a call with shared prefixes and its workspace query share. Without groups it is mxfp4_attention.
int check_prefix(const mxfp4_cache* cache, const mxfp4_batch* batch, const mxfp4_prefix* prefix, int64_t heads,
                 int64_t max_prefix, int64_t max_own, nvfp4::MxCache* c, nvfp4::MxBatch* b, nvfp4::MxPrefix* x,
                 nvfp4::MxPrefixPlan* plan) {
  if (!prefix) return api_fail(NVFP4_ERR_INVALID_ARG, "null prefix");
  if (max_prefix <= 0 || max_own <= 0)
    return api_fail(NVFP4_ERR_INVALID_ARG, "max_prefix=%lld max_own=%lld", (long long)max_prefix, (long long)max_own);
  nvfp4::MxAttnPlan whole;
  const int rc = check_attention(cache, batch, heads, max_own, 0, 0, c, b, &whole);
  if (rc != NVFP4_OK) return rc;
  if (prefix->groups < 0 || prefix->max_pages < 0 || prefix->table_stride < prefix->max_pages)
    return api_fail(NVFP4_ERR_INVALID_ARG, "bad prefix: %lld groups, %lld pages (stride %lld)", (long long)prefix->groups,
                    (long long)prefix->max_pages, (long long)prefix->table_stride);
  if (prefix->groups >= 1 << 24 || prefix->max_pages >= (int64_t)1 << 27 ||
      prefix->max_pages << b->page_shift >= (int64_t)1 << 30)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "prefixes beyond 2^24 groups or 2^30 tokens");
  // of the join, four rows x heads a workgroup, and of the parts, 16 packed rows each at least
  if ((b->tokens * heads + 3) / 4 > kMostGroups ||
      (b->tokens * (heads / c->kv_heads) / 16 * 2 + b->batch + prefix->groups) * c->kv_heads > kMostGroups)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "too many rows and heads for one call");
  if (prefix->groups > 0 && b->batch > 0 && b->tokens > 0) {
    if (!prefix->lens_dev || !prefix->group_starts_dev || (prefix->max_pages > 0 && !prefix->block_table_dev))
      return api_fail(NVFP4_ERR_INVALID_ARG, "null prefix pointer");
    if (!aligned4(prefix->lens_dev) || !aligned4(prefix->group_starts_dev) || !aligned4(prefix->block_table_dev))
      return api_fail(NVFP4_ERR_MISALIGNED, "prefix pointers must be 4-byte aligned");
  }
  *x = nvfp4::MxPrefix{prefix->block_table_dev, prefix->lens_dev, prefix->group_starts_dev, prefix->table_stride,
                       (int)prefix->groups, (int)prefix->max_pages};
  constexpr int64_t most = 1 << 30;  // no sequence is longer
  if (prefix->groups > 0 && b->batch > 0 && b->tokens > 0)
    *plan = nvfp4::mx_prefix_plan(b->tokens, b->batch, prefix->groups, heads, c->kv_heads, c->head_dim,
                                  nvfp4::mx_least(max_prefix, most), nvfp4::mx_least(max_own, most));
  else
    *plan = nvfp4::MxPrefixPlan{whole, whole, false};
  return NVFP4_OK;
}

int64_t prefix_bytes(const nvfp4::MxBatch& b, const nvfp4::MxCache& c, const nvfp4::MxPrefix& x, int64_t heads,
                     const nvfp4::MxPrefixPlan& plan) {
  if (b.tokens == 0 || b.batch == 0) return 0;
  return x.groups > 0 ? nvfp4::mx_prefix_bytes(plan, b.tokens, heads, c.head_dim) : workspace_bytes(b, c, heads, plan.own);
}

int check_norm(const mxfp4_norm* n, const char* name, nvfp4::MxNorm* out) {
  *out = nvfp4::MxNorm{nullptr, 0.0, false};
  if (!n) return NVFP4_OK;
  if (!(n->eps > 0.0 && n->eps <= DBL_MAX)) return api_fail(NVFP4_ERR_INVALID_ARG, "%s eps must be positive and finite", name);
  if (!aligned16(n->weight_dev)) return api_fail(NVFP4_ERR_MISALIGNED, "%s weight must be 16-byte aligned", name);
  *out = nvfp4::MxNorm{(const uint16_t*)n->weight_dev, n->eps, true};
  return NVFP4_OK;
}

int check_rotation(const mxfp4_rotation* r, int64_t head_dim, bool cached, nvfp4::MxRopeArgs* a) {
  a->rotary = 0;
  a->axis_count = 1;
  if (!r) return NVFP4_OK;
  if (r->rotary_dim <= 0 || r->rotary_dim > head_dim || r->axes <= 0 || r->token_stride < 0 || r->axis_stride < 0)
    return api_fail(NVFP4_ERR_INVALID_ARG, "bad rotation: %lld of %lld elements, %lld axes", (long long)r->rotary_dim,
                    (long long)head_dim, (long long)r->axes);
  if (r->rotary_dim % 16 != 0 || r->axes > 64 || r->token_stride > (int64_t)1 << 31 || r->axis_stride > (int64_t)1 << 31)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "rotary_dim=%lld is not a multiple of 16, or more than 64 axes or a stride of 2^31",
                    (long long)r->rotary_dim);
  if (!r->freqs_dev || (!cached && !r->positions_dev)) return api_fail(NVFP4_ERR_INVALID_ARG, "null frequencies or positions");
  if (!aligned4(r->freqs_dev) || !aligned4(r->axes_dev) || !aligned4(r->positions_dev))
    return api_fail(NVFP4_ERR_MISALIGNED, "frequencies, axes and positions must be 4-byte aligned");
  a->freqs = r->freqs_dev;
  a->axes = r->axes_dev;
  a->positions = r->positions_dev;
  a->pos_token = r->token_stride;
  a->pos_axis = r->axis_stride;
  a->axis_count = (int)r->axes;
  a->rotary = (int)r->rotary_dim;
  return NVFP4_OK;
}

constexpr int64_t kMostRopeTokens = ((int64_t)1 << 26) - 4;  // a wave each, four to a workgroup

int check_pages(const mxfp4_pages* p, nvfp4::MxPages* out) {
  if (!p) return api_fail(NVFP4_ERR_INVALID_ARG, "null pages");
  if (p->slots <= 0 || p->max_pages <= 0 || p->num_pages <= 0 || p->table_stride < p->max_pages)
    return api_fail(NVFP4_ERR_INVALID_ARG, "bad pages: %lld slots of %lld (stride %lld), %lld in all", (long long)p->slots,
                    (long long)p->max_pages, (long long)p->table_stride, (long long)p->num_pages);
  const int rc = check_page_size(p->page_size);
  if (rc != NVFP4_OK) return rc;
  if (p->slots >= 1 << 24 || p->num_pages >= (int64_t)1 << 31 || p->max_pages >= (int64_t)1 << 27 ||
      p->max_pages * p->page_size >= (int64_t)1 << 30 || p->table_stride > (int64_t)1 << 40)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "beyond 2^24 slots, 2^31 pages or 2^30 tokens a sequence");
  if (!p->block_table_dev || !p->seq_lens_dev || !p->refs_dev) return api_fail(NVFP4_ERR_INVALID_ARG, "null pages pointer");
  if (!aligned4(p->block_table_dev) || !aligned4(p->seq_lens_dev) || !aligned4(p->refs_dev))
    return api_fail(NVFP4_ERR_MISALIGNED, "pages pointers must be 4-byte aligned");
  *out = nvfp4::MxPages{p->block_table_dev, p->seq_lens_dev, p->refs_dev, p->table_stride, p->num_pages, (int)p->slots,
                        (int)p->max_pages, page_shift_of(p->page_size)};
  return NVFP4_OK;
}

int check_list_size(int64_t n) {
  if (n < 0) return api_fail(NVFP4_ERR_INVALID_ARG, "list of %lld entries", (long long)n);
  if (n >= nvfp4::kMxMostListed) return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "list of %lld entries (65535 at most)", (long long)n);
  return NVFP4_OK;
}

int check_list(const void* list, const char* name) {
  if (!list) return api_fail(NVFP4_ERR_INVALID_ARG, "null %s pointer", name);
  if (!aligned4(list)) return api_fail(NVFP4_ERR_MISALIGNED, "%s must be 4-byte aligned", name);
  return NVFP4_OK;
}

int check_compact(const mxfp4_pages* pages, nvfp4::MxPages* p) {
  const int rc = check_pages(pages, p);
  if (rc != NVFP4_OK) return rc;
  if ((p->num_pages + 255) / 256 + p->slots * ((p->max_pages + 255) / 256) > kMostGroups)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "block table too large for one call");
  return NVFP4_OK;
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
  rc = check_scale(scale);
  if (rc != NVFP4_OK) return rc;
  if (window > 0 && !causal) return api_fail(NVFP4_ERR_INVALID_ARG, "a window needs causal attention");
  const bool any = b.tokens > 0 && b.batch > 0;
  if (any)
    rc = check_attention_rows(b, c, q_dev, q_token_stride, q_head_stride, heads, out_dev, out_token_stride, out_head_stride,
                              workspace_dev, workspace_size, workspace_bytes(b, c, heads, plan));
  if (rc != NVFP4_OK) return rc;
  const uint16_t* table = nullptr;
  rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (!any) return api_ok();
  nvfp4::MxAttnArgs a = attention_args(b, c, q_dev, q_token_stride, q_head_stride, heads, scale, causal, out_dev,
                                       out_token_stride, out_head_stride, workspace_dev);
  // lengths stay below 2^30: a window or first tokens beyond that hide nothing more
  a.window = (int)(window < (1 << 30) ? window : 1 << 30);
  a.sinks = (int)(sinks < (1 << 30) ? sinks : 1 << 30);
  a.splits = plan.splits;
  a.part_ml = (float2*)((float*)workspace_dev + plan.splits * b.tokens * heads * c.head_dim);
  return launched(nvfp4::launch_mx_attention(a, plan, (hipStream_t)stream), "attention");
}

int64_t mxfp4_attention_prefix_workspace_bytes(const mxfp4_cache* cache, const mxfp4_batch* batch,
                                               const mxfp4_prefix* prefix, int64_t heads, int64_t max_prefix,
                                               int64_t max_own) {
  nvfp4::MxCache c;
  nvfp4::MxBatch b;
  nvfp4::MxPrefix x;
  nvfp4::MxPrefixPlan plan;
  if (check_prefix(cache, batch, prefix, heads, max_prefix, max_own, &c, &b, &x, &plan) != NVFP4_OK) return -1;
  return prefix_bytes(b, c, x, heads, plan);
}

int mxfp4_attention_prefix(const mxfp4_cache* cache, const mxfp4_batch* batch, const mxfp4_prefix* prefix,
                           const void* q_dev, int64_t q_token_stride, int64_t q_head_stride, int64_t heads, float scale,
                           int causal, int64_t max_prefix, int64_t max_own, void* out_dev, int64_t out_token_stride,
                           int64_t out_head_stride, void* workspace_dev, int64_t workspace_size, void* stream) {
  nvfp4::MxCache c;
  nvfp4::MxBatch b;
  nvfp4::MxPrefix x;
  nvfp4::MxPrefixPlan plan;
  int rc = check_prefix(cache, batch, prefix, heads, max_prefix, max_own, &c, &b, &x, &plan);
  if (rc == NVFP4_OK) rc = check_scale(scale);
  const bool any = rc == NVFP4_OK && b.tokens > 0 && b.batch > 0;
  if (any)
    rc = check_attention_rows(b, c, q_dev, q_token_stride, q_head_stride, heads, out_dev, out_token_stride, out_head_stride,
                              workspace_dev, workspace_size, prefix_bytes(b, c, x, heads, plan));
  if (any && x.groups == 0 && rc == NVFP4_OK)
    return mxfp4_attention(cache, batch, q_dev, q_token_stride, q_head_stride, heads, scale, causal, 0, 0, max_own, out_dev,
                           out_token_stride, out_head_stride, workspace_dev, workspace_size, stream);
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (!any) return api_ok();
  nvfp4::MxAttnArgs a = attention_args(b, c, q_dev, q_token_stride, q_head_stride, heads, scale, causal, out_dev,
                                       out_token_stride, out_head_stride, workspace_dev);
  a.prefix = x;
  return launched(nvfp4::launch_mx_attention_prefix(a, plan, (hipStream_t)stream), "attention behind prefixes");
}

int mxfp4_norm_rope(const void* x_dev, int64_t x_token_stride, int64_t x_head_stride, int64_t tokens, int64_t heads,
                    int64_t head_dim, const mxfp4_norm* norm, const mxfp4_rotation* rotation, void* out_dev,
                    int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  if (tokens < 0 || heads <= 0 || head_dim <= 0)
    return api_fail(NVFP4_ERR_INVALID_ARG, "bad shape: %lld tokens, %lld heads of %lld", (long long)tokens, (long long)heads,
                    (long long)head_dim);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "head_dim=%lld is not 64, 128 or 256", (long long)head_dim);
  if (heads > 65536 || tokens > kMostRopeTokens)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "too many rows or heads for one call (%lld, %lld)", (long long)tokens,
                    (long long)heads);
  nvfp4::MxRopeArgs a{};
  int rc = check_norm(norm, "norm", &a.q_norm);
  if (rc == NVFP4_OK) rc = check_rotation(rotation, head_dim, tokens == 0, &a);
  if (rc == NVFP4_OK && tokens > 0) rc = check_packed_rows(x_dev, x_token_stride, x_head_stride, "x");
  if (rc == NVFP4_OK && tokens > 0) rc = check_packed_rows(out_dev, out_token_stride, out_head_stride, "out");
  if (rc == NVFP4_OK && tokens > 0)
    rc = check_written_rows(out_token_stride, out_head_stride, heads, tokens, head_dim, "out");
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (tokens == 0) return api_ok();
  a.q = (const uint16_t*)x_dev;
  a.out = (uint16_t*)out_dev;
  a.q_token = x_token_stride;
  a.q_head = x_head_stride;
  a.out_token = out_token_stride;
  a.out_head = out_head_stride;
  a.tokens = tokens;
  a.heads = (int)heads;
  a.parts = (int)nvfp4::mx_rope_parts(tokens, heads, 0, head_dim);
  return launched(nvfp4::launch_mx_rope(a, (int)head_dim, false, rotation && rotation->interleaved, (hipStream_t)stream),
                  "norm and rotation");
}

int mxfp4_norm_rope_append(const mxfp4_cache* cache, const mxfp4_batch* batch, const void* q_dev, int64_t q_token_stride,
                           int64_t q_head_stride, int64_t heads, const mxfp4_norm* q_norm, const void* k_dev,
                           int64_t k_token_stride, int64_t k_head_stride, const mxfp4_norm* k_norm, const void* v_dev,
                           int64_t v_token_stride, int64_t v_head_stride, const mxfp4_rotation* rotation,
                           void* q_out_dev, int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  nvfp4::MxRopeArgs a{};
  int rc = check_cache(cache, batch, &a.c, &a.b);
  if (rc != NVFP4_OK) return rc;
  if (heads < 0) return api_fail(NVFP4_ERR_INVALID_ARG, "%lld heads", (long long)heads);
  if (heads > 65536 || a.b.tokens > kMostRopeTokens)
    return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "too many rows or heads for one call (%lld, %lld)", (long long)a.b.tokens,
                    (long long)heads);
  const bool any = a.b.tokens > 0 && a.b.batch > 0;
  rc = check_norm(q_norm, "q", &a.q_norm);
  if (rc == NVFP4_OK) rc = check_norm(k_norm, "k", &a.k_norm);
  if (rc == NVFP4_OK) rc = check_rotation(rotation, a.c.head_dim, true, &a);
  if (any && rc == NVFP4_OK) rc = check_packed_rows(k_dev, k_token_stride, k_head_stride, "k");
  if (any && rc == NVFP4_OK) rc = check_packed_rows(v_dev, v_token_stride, v_head_stride, "v");
  if (any && rc == NVFP4_OK && heads > 0) rc = check_packed_rows(q_dev, q_token_stride, q_head_stride, "q");
  if (any && rc == NVFP4_OK && heads > 0) rc = check_packed_rows(q_out_dev, out_token_stride, out_head_stride, "q_out");
  if (any && rc == NVFP4_OK && heads > 0)
    rc = check_written_rows(out_token_stride, out_head_stride, heads, a.b.tokens, a.c.head_dim, "q_out");
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (!any) return api_ok();
  a.q = (const uint16_t*)q_dev;
  a.out = (uint16_t*)q_out_dev;
  a.k = (const uint16_t*)k_dev;
  a.v = (const uint16_t*)v_dev;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.out_token = out_token_stride;
  a.out_head = out_head_stride;
  a.k_token = k_token_stride;
  a.k_head = k_head_stride;
  a.v_token = v_token_stride;
  a.v_head = v_head_stride;
  a.tokens = a.b.tokens;
  a.heads = (int)heads;
  a.kv_heads = a.c.kv_heads;
  a.parts = (int)nvfp4::mx_rope_parts(a.tokens, heads, a.kv_heads, a.c.head_dim);
  return launched(nvfp4::launch_mx_rope(a, a.c.head_dim, true, rotation && rotation->interleaved, (hipStream_t)stream),
                  "norm, rotation and append");
}

int mxfp4_pages_free(const mxfp4_pages* pages, const int32_t* slots_dev, const int32_t* keep_dev, int64_t n,
                     void* stream) {
  nvfp4::MxPages p;
  int rc = check_pages(pages, &p);
  if (rc == NVFP4_OK) rc = check_list_size(n);
  if (rc == NVFP4_OK && n > 0) rc = check_list(slots_dev, "slots");
  if (rc == NVFP4_OK && n > 0 && keep_dev) rc = check_list(keep_dev, "keep");
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (n == 0) return api_ok();
  return launched(nvfp4::launch_mx_pages_free(p, slots_dev, keep_dev, (int)n, (hipStream_t)stream), "free");
}

int mxfp4_pages_fork(const mxfp4_pages* pages, const int32_t* parents_dev, const int32_t* children_dev, int64_t n,
                     int32_t* done_dev, void* stream) {
  nvfp4::MxPages p;
  int rc = check_pages(pages, &p);
  if (rc == NVFP4_OK) rc = check_list_size(n);
  if (rc == NVFP4_OK && n > 0) rc = check_list(parents_dev, "parents");
  if (rc == NVFP4_OK && n > 0) rc = check_list(children_dev, "children");
  if (rc == NVFP4_OK && n > 0) rc = check_list(done_dev, "done");
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (n == 0) return api_ok();
  return launched(nvfp4::launch_mx_pages_fork(p, parents_dev, children_dev, (int)n, done_dev, (hipStream_t)stream), "fork");
}

int64_t mxfp4_pages_reserve_workspace_bytes(const mxfp4_pages* pages, int64_t n) {
  nvfp4::MxPages p;
  if (check_pages(pages, &p) != NVFP4_OK || check_list_size(n) != NVFP4_OK) return -1;
  return n == 0 ? 0 : nvfp4::mx_reserve_bytes(n, p.slots, p.max_pages, p.num_pages);
}

int mxfp4_pages_reserve(const mxfp4_pages* pages, const int32_t* slots_dev, const int32_t* lens_dev, int64_t n,
                        int32_t* done_dev, int32_t* src_dev, int32_t* dst_dev, void* workspace_dev,
                        int64_t workspace_size, void* stream) {
  nvfp4::MxPages p;
  int rc = check_pages(pages, &p);
  if (rc == NVFP4_OK) rc = check_list_size(n);
  if (rc == NVFP4_OK && n > 0) rc = check_list(slots_dev, "slots");
  if (rc == NVFP4_OK && n > 0) rc = check_list(lens_dev, "lens");
  if (rc == NVFP4_OK && n > 0) rc = check_list(done_dev, "done");
  if (rc == NVFP4_OK && n > 0) rc = check_list(src_dev, "src");
  if (rc == NVFP4_OK && n > 0) rc = check_list(dst_dev, "dst");
  if (rc == NVFP4_OK && n > 0)
    rc = check_workspace(workspace_dev, workspace_size, nvfp4::mx_reserve_bytes(n, p.slots, p.max_pages, p.num_pages));
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (n == 0) return api_ok();
  return launched(nvfp4::launch_mx_pages_reserve(p, slots_dev, lens_dev, (int)n, done_dev, src_dev, dst_dev, workspace_dev,
                                                 (hipStream_t)stream),
                  "reserve");
}

int64_t mxfp4_pages_compact_workspace_bytes(const mxfp4_pages* pages) {
  nvfp4::MxPages p;
  return check_compact(pages, &p) == NVFP4_OK ? nvfp4::mx_compact_bytes(p.num_pages) : -1;
}

int mxfp4_pages_compact(const mxfp4_pages* pages, int32_t* table_out_dev, int64_t table_out_stride, int32_t* refs_out_dev,
                        int32_t* src_dev, int32_t* dst_dev, int32_t* used_dev, void* workspace_dev,
                        int64_t workspace_size, void* stream) {
  nvfp4::MxPages p;
  int rc = check_compact(pages, &p);
  if (rc == NVFP4_OK) rc = check_list(table_out_dev, "new block table");
  if (rc == NVFP4_OK && (table_out_stride < p.max_pages || table_out_stride > (int64_t)1 << 40 ||
                         (table_out_dev == p.table && table_out_stride != p.stride)))
    rc = api_fail(NVFP4_ERR_INVALID_ARG, "new block table's row stride %lld", (long long)table_out_stride);
  if (rc == NVFP4_OK) rc = check_list(refs_out_dev, "new counts");
  if (rc == NVFP4_OK && p.num_pages > 1) rc = check_list(src_dev, "src");
  if (rc == NVFP4_OK && p.num_pages > 1) rc = check_list(dst_dev, "dst");
  if (rc == NVFP4_OK) rc = check_list(used_dev, "used");
  if (rc == NVFP4_OK) rc = check_workspace(workspace_dev, workspace_size, nvfp4::mx_compact_bytes(p.num_pages));
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  return launched(nvfp4::launch_mx_pages_compact(p, table_out_dev, table_out_stride, refs_out_dev, src_dev, dst_dev, used_dev,
                                                 workspace_dev, (hipStream_t)stream),
                  "compact");
}

int mxfp4_cache_copy(const mxfp4_cache* from, const mxfp4_cache* to, const int32_t* src_dev, const int32_t* dst_dev,
                     int64_t n, void* stream) {
  nvfp4::MxCache f, t;
  if (!from || !to) return api_fail(NVFP4_ERR_INVALID_ARG, "null cache");
  int rc = check_pages_of_cache(from, &f);
  if (rc == NVFP4_OK) rc = check_pages_of_cache(to, &t);
  if (rc != NVFP4_OK) return rc;
  if (from->page_size != to->page_size || from->kv_heads != to->kv_heads || from->head_dim != to->head_dim)
    return api_fail(NVFP4_ERR_INVALID_ARG, "the caches' pages differ");
  if (n < 0) return api_fail(NVFP4_ERR_INVALID_ARG, "list of %lld entries", (long long)n);
  if (n >= (int64_t)1 << 31) return api_fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "list of %lld entries", (long long)n);
  if (n > 0) rc = check_list(src_dev, "src");
  if (n > 0 && rc == NVFP4_OK) rc = check_list(dst_dev, "dst");
  const uint16_t* table = nullptr;
  if (rc == NVFP4_OK) rc = api_device(&table);
  if (rc != NVFP4_OK) return rc;
  if (n == 0) return api_ok();
  return launched(nvfp4::launch_mx_cache_copy(f, from->num_pages, t, to->num_pages, (int)from->page_size, src_dev, dst_dev, n,
                                              (hipStream_t)stream),
                  "cache copy");
}

}  // extern "C"
