// mx_attn.hpp - arguments of the MXFP4 attention kernels and the plan of a call.
#pragma once

#include "mx.hpp"

namespace nvfp4 {

struct MxAttnArgs {
  MxBatch b;
  MxCache c;
  const uint16_t* q;
  uint16_t* out;
  int64_t q_token, q_head, out_token, out_head;  // element strides
  int heads, group;                              // group = heads / kv_heads
  float scale_log2, raise;                       // scale * log2 e; kMxRaise / scale_log2
  int causal, window, sinks;                     // window 0: none
  int splits;
  float* part_o;    // [splits, tokens, heads, head_dim]; by_seq: [splits, batch, kv_heads, 16, head_dim]
  float2* part_ml;  // [splits, tokens, heads] reference score and sum; by_seq likewise
  int skip;         // prompt form: sequences of up to so many packed rows are not its own
  bool by_seq;      // few-rows form: a workgroup a sequence and kv head, of up to 16 packed rows
};

constexpr int kMxMostSplits = 256;

// How a call is cut, from its sizes alone.
struct MxAttnPlan {
  bool few;       // the form for few rows
  int row_tiles;  // its 16-row tiles of a workgroup
  int splits;     // pieces of the token axis, joined by a second launch
  int mixed;      // prompt form: its sequences of up to 16 packed rows go to the few-rows form in
                  // so many pieces; 0: they do not
};

// Rows: the packed rows (rows x heads of a group) of an average sequence. Up to 16 of them
// (32 at head_dim 64) are one workgroup's of the few-rows form, whose four waves split the
// tokens; beyond that the prompt form gives every wave 32 rows of its own. Measured, 64
// sequences of 2048, 8 kv heads, few-rows form and prompt form: 16 rows of 128 65 and 96 us,
// 32 rows 118 and 94; of 64, 32 rows 80 and 97, 48 rows 110 and 97; of 256, 16 rows 127 and
// 233, 32 rows 251 and 225.
//
// Splits: where the rows alone do not give enough workgroups, pieces of the token axis do.
// Few rows: 8 workgroups for each of the 256 CUs (ragged lengths then even out over two
// rounds of them: 48 tokens over up to 8200 take 80 us with 5 splits, 94 with 2, 86 with 10),
// but at least two 32-token tiles a wave, so that a split is more than its own start.
// Prompts: as many as are resident at once, by registers 3, 2 or 1 a CU. But a split writes
// and reads every row once more in fp32, about head_dim tokens heads splits * 1.3 ps, which it
// has to save of the head_dim / 6 ns that a workgroup takes for a token: the sum is least at
// sqrt(128 seen / (tokens heads)) splits, and below three of them not splitting is as good.
// Measured, 32 heads of 128 over 8: 256 rows over 8192 take 180 us whole, 62 with 6 splits, 57
// with 8, 66 with 12; over 1024: 31 whole, 24 with 3; 1024 rows over 1024: 33 whole, 45 with
// 2. 28 heads over 4, 904 rows over up to 3656: 122 whole, 84 with 3, 82 with 4.
//
// Mixed: a prompt among single tokens makes the average one of prompts, whose form walks a
// single token's cache with one wave a kv head. Where caches are long a second launch takes
// the sequences of up to 16 packed rows: 2048 rows over 2048 and 31 single tokens over 8192,
// 32 heads of 128 over 8, 293 -> 133 us, over 32768 1054 -> 297. Batches without such sequences
// pay about 8 us for its launches, and over 2048 it saves nothing. A group of more than 16 heads
// has no such sequence.
inline MxAttnPlan mx_attention_plan(int64_t tokens, int64_t batch, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                    int64_t max_kv, int64_t window, int64_t sinks) {
  MxAttnPlan p{true, 1, 1, 0};
  if (tokens <= 0 || batch <= 0) return p;
  const int64_t group = heads / kv_heads;
  const int64_t rows = (tokens + batch - 1) / batch * group;
  p.row_tiles = rows <= 16 ? 1 : 2;
  p.few = p.row_tiles == 1 || (head_dim == 64 && rows <= 32);
  const int64_t per_group = p.few ? 16 * p.row_tiles : 128;
  int64_t tiles = (tokens * group + per_group - 1) / per_group;
  if (tiles < batch) tiles = batch;
  const int64_t groups = tiles * kv_heads;
  int64_t seen = max_kv < (1 << 30) ? max_kv : 1 << 30;  // no sequence is longer
  if (window > 0 && window < seen && sinks < seen) {     // a row tile's span: the window, its rows, the first tokens
    const int64_t w = window + per_group / group + sinks;
    if (w < seen) seen = w;
  }
  int64_t s, most_splits;
  if (p.few) {
    s = 2048 / groups;
    most_splits = seen / (2 * 32 * 4);
  } else {
    s = (head_dim == 64 ? 768 : head_dim == 128 ? 512 : 256) / groups;
    most_splits = 2;
    while ((most_splits + 1) * (most_splits + 1) * tokens * heads <= 128 * seen && most_splits < kMxMostSplits) ++most_splits;
    if (most_splits < 3) most_splits = 1;
  }
  if (s > most_splits) s = most_splits;
  if (s > kMxMostSplits) s = kMxMostSplits;
  p.splits = s < 1 ? 1 : (int)s;
  if (!p.few && batch > 1 && group <= 16 && seen >= 8192) {
    s = 2048 / (batch * kv_heads);
    if (s > seen / (2 * 32 * 4)) s = seen / (2 * 32 * 4);
    if (s > kMxMostSplits) s = kMxMostSplits;
    p.mixed = s < 1 ? 1 : (int)s;  // more than 1 wherever p.splits is: batch * kv_heads is below 768 / 2 there
  }
  return p;
}

// workspace of the rows' pieces, and of those of the few-rows form's sequences behind it
inline int64_t mx_prompt_part_bytes(const MxAttnPlan& p, int64_t tokens, int64_t heads, int64_t head_dim) {
  return p.splits == 1 ? 0 : (p.splits * tokens * heads * (head_dim + 2) * 4 + 15) / 16 * 16;
}

inline int64_t mx_part_bytes(const MxAttnPlan& p, int64_t tokens, int64_t batch, int64_t heads, int64_t kv_heads,
                             int64_t head_dim) {
  return mx_prompt_part_bytes(p, tokens, heads, head_dim) +
         (p.mixed > 1 ? p.mixed * batch * kv_heads * 16 * (head_dim + 2) * 4 : 0);
}

hipError_t mx_attention_prompt_setup();
hipError_t launch_mx_attention_prompt(const MxAttnArgs& a, hipStream_t stream);

// ---- device side ----

constexpr float kMxRaise = 8.0f;  // log2 of how far weights may exceed 1 before the maximum is raised

// Weights are powers of two under a reference score t, the largest of the row so far. While
// |scale_log2 t| is below 2^20 their unit is that of fl(scale_log2 t): one fma gives a weight's
// exponent with one rounding, and the reference's own, 2^-5 at most, only puts the largest
// weight that far from 1. Beyond, it would put it anywhere (2^+-128 at 2^31), or scale_log2 t be
// infinite: there the unit is that of t itself, and t is taken off first, which is exact for
// scores that count. A reference of -inf has seen nothing.
constexpr float kMxNear = 0x1p20f;

struct MxUnit {
  float base, neg;  // a weight's exponent: scale_log2 (x - base) + neg
  bool far;
};

__device__ __forceinline__ MxUnit mx_unit(const MxAttnArgs& a, float t) {
  const float e = t * a.scale_log2;
  const bool none = t == -INFINITY, far = !none && !(fabsf(e) < kMxNear);
  return MxUnit{far ? t : 0.0f, far || none ? 0.0f : -e, far};
}

// of the weight of score x
__device__ __forceinline__ float mx_exponent(const MxAttnArgs& a, float x, float base, float neg) {
  return __builtin_fmaf(x - base, a.scale_log2, neg);
}

// What weights and their sums under reference t are multiplied with to be under reference u >= t
// (anything if there are none): t's own weight is 2^off, and becomes that under u's unit. (The
// early way out matters: without it the prompt form of 64 spills, 99 us for 91.)
__device__ __forceinline__ float mx_rebase(const MxAttnArgs& a, float t, float u) {
  const MxUnit from = mx_unit(a, t);
  const float off = mx_exponent(a, t, from.base, from.neg);
  if (t == u || t == -INFINITY) return 1.0f;
  const MxUnit to = mx_unit(a, u);
  return __builtin_amdgcn_exp2f(mx_exponent(a, t, to.base, to.neg) - off);
}

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;

__device__ __forceinline__ bf16x8_t as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const u32x4_t w = {a, b, c, d};
  bf16x8_t r;
  __builtin_memcpy(&r, &w, 16);
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  bf16x2_t c;
  c[0] = (__bf16)lo;
  c[1] = (__bf16)hi;
  return as_u32(c);
}

// codes 2 sel, 2 sel + 1 of q as packed bf16
__device__ __forceinline__ uint32_t decode2(uint32_t q, float s, int sel) {
  switch (sel) {
    case 0: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
    case 1: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
    case 2: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
    default: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
  }
}

// bits -> eight bf16 that are 1 where the bit is set
__device__ __forceinline__ bf16x8_t mx_ones(uint32_t bits) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (bits >> (2 * i) & 1 ? 0x3F80u : 0u) | (bits >> (2 * i + 1) & 1 ? 0x3F800000u : 0u);
  return as_bf16x8(w[0], w[1], w[2], w[3]);
}

template <int N>
struct Words {
  uint32_t w[N];
};

template <int N>
__device__ __forceinline__ Words<N> load_words(const uint8_t* p) {
  Words<N> r;
  if constexpr (N == 1) {
    r.w[0] = *(const uint32_t*)p;
  } else if constexpr (N == 2) {
    const u32x2_t v = *(const u32x2_t*)p;
    r.w[0] = v[0];
    r.w[1] = v[1];
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4_t v = *(const u32x4_t*)(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[4 * i + j] = v[j];
    }
  }
  return r;
}

// The packed rows of a workgroup: per sequence the (row, head of the group) pairs, group
// fastest, in tiles of kRows. Sequence i's tiles are numbered from floor(start_i group /
// kRows) + i: that leaves each at least as many numbers as it has tiles, without a scan of
// the lengths; numbers without a tile have first >= count.
struct MxRows {
  int seq;
  int64_t r0;     // the sequence's first row in the packed tensors
  int count;      // packed rows of the sequence
  int first;      // the tile's first packed row
  int kv_len;
  int back;       // position of the sequence's first row
};

__device__ __forceinline__ MxRows mx_rows(const MxAttnArgs& a, int64_t tile, int rows) {
  int lo = 0, hi = a.b.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (mx_row_start(a.b, mid) * a.group / rows + mid <= tile) lo = mid;
    else hi = mid;
  }
  MxRows r;
  const int64_t r1 = mx_row_start(a.b, lo + 1);
  r.seq = lo;
  r.r0 = mx_row_start(a.b, lo);
  r.count = r1 > r.r0 ? (int)((r1 - r.r0) * a.group) : 0;
  const int64_t first = (tile - (r.r0 * a.group / rows + lo)) * rows;
  r.first = first < 0 || first > r.count ? r.count : (int)first;
  r.kv_len = mx_seq_len(a.b, lo);
  r.back = r.kv_len - (int)(r1 - r.r0);
  return r;
}

// all packed rows of a sequence
__device__ __forceinline__ MxRows mx_rows_of(const MxAttnArgs& a, int seq) {
  MxRows r;
  const int64_t r1 = mx_row_start(a.b, seq + 1);
  r.seq = seq;
  r.r0 = mx_row_start(a.b, seq);
  r.count = r1 > r.r0 ? (int)((r1 - r.r0) * a.group) : 0;
  r.first = 0;
  r.kv_len = mx_seq_len(a.b, seq);
  r.back = r.kv_len - (int)(r1 - r.r0);
  return r;
}

// What packed rows [p0, p1) of a sequence see: row at position p the tokens [low, high) and
// those below sinks, with these bounds over the rows.
struct MxSight {
  int high_min, high_max, low_min, low_max, sinks;
};

__device__ __forceinline__ int mx_high(const MxAttnArgs& a, int kv_len, int pos) {
  const int h = a.causal && pos + 1 < kv_len ? pos + 1 : kv_len;
  return h > 0 ? h : 0;
}

__device__ __forceinline__ int mx_low(const MxAttnArgs& a, int pos) {
  return a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
}

__device__ __forceinline__ MxSight mx_sight(const MxAttnArgs& a, const MxRows& r, int p0, int p1) {
  const int pos_a = r.back + p0 / a.group, pos_b = r.back + (p1 - 1) / a.group;
  return MxSight{mx_high(a, r.kv_len, pos_a), mx_high(a, r.kv_len, pos_b), mx_low(a, pos_a), mx_low(a, pos_b),
                 a.window > 0 ? a.sinks : 0};
}

// The tiles of `size` tokens that those rows see: the ones that hold first tokens, then
// from the window's start (or 0) to the last visible token.
struct MxSpan {
  int first, begin, count;  // tiles [0, first), then [begin, ...); count in all
  __device__ __forceinline__ int at(int i) const { return i < first ? i : begin + (i - first); }
};

__device__ __forceinline__ MxSpan mx_span(const MxSight& s, int size) {
  MxSpan t;
  t.first = ((s.sinks < s.high_max ? s.sinks : s.high_max) + size - 1) / size;
  t.begin = s.low_min / size > t.first ? s.low_min / size : t.first;
  const int end = (s.high_max + size - 1) / size;
  t.count = t.first + (end > t.begin ? end - t.begin : 0);
  return t;
}

// where share i of n shares of a count begins, the first ones larger by one if need be
// (count * i / n needs a 64-bit division, 200 instructions before the first load)
__device__ __forceinline__ int mx_share(int count, int i, int n) {
  const int each = (int)((unsigned)count / (unsigned)n), over = count - each * n;
  return each * i + (i < over ? i : over);
}

// first of the cache's rows for 16 tokens from t (a multiple of 16) on that page; a page
// that is not there is read as page 0, and what is read must not be used
__device__ __forceinline__ int64_t mx_cache_row(const MxAttnArgs& a, int64_t page, int head, int t) {
  return (((page < 0 ? 0 : page) * a.c.kv_heads + head) << a.b.page_shift) + (t & ((1 << a.b.page_shift) - 1));
}

}  // namespace nvfp4
