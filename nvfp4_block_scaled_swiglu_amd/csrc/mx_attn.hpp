// mx_attn.hpp - arguments of the MXFP4 attention kernels and the plan of a call.
#pragma once

#include "mx.hpp"

namespace nvfp4 {

// Groups of consecutive sequences whose first tokens are read through one block table: the
// whole kMxShared of them that every row of a sequence sees.
struct MxPrefix {
  const int32_t* block_table;  // [groups, max_pages]
  const int32_t* lens;         // [groups]
  const int32_t* starts;       // [groups + 1] first sequence of each group
  int64_t table_stride;
  int groups, max_pages;
};

constexpr int kMxShared = 64;  // tokens: whole tiles of either form

// Which tokens a launch is for: all that its rows see, a group's prefix for the rows of all of
// its sequences, what is left of each sequence, or all again, the prefix by its group's table.
enum MxPart { kMxWhole, kMxPrefix, kMxOwn, kMxThrough };

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
  int tiles;        // all but kMxWhole: row tiles of the part
  MxPrefix prefix;  // likewise (kMxPrefix and kMxOwn leave pieces always, kMxThrough where there are splits)
  int prefix_splits;        // joins: the first pieces are a prefix's, 0: none
  uint32_t* shared;         // [tokens] whether they hold for the row, written by kMxOwn for the join
};

constexpr int kMxMostSplits = 256;  // that a join takes

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

// A call with shared prefixes: what the groups' rows see of them, and the rest of the sequences.
struct MxPrefixPlan {
  MxAttnPlan prefix, own;
  bool through;  // no parts: each sequence's rows over all of their tokens, by own (prompt form); else own is few
};

// Through: rows that fill the prompt form's tiles of 128 sequence by sequence save little by filling
// them group by group, and pieces cost their way to memory and back, about what a tile takes
// for 800 tokens. 8 sequences of 288 to 512 rows x 7 heads behind 6,144 tokens: 651 us, in parts 664.
//
// Pieces, of the prefix: in the prompt form a workgroup of 128 takes 1.3 us for a tile of 64 tokens alone on its CU,
// 1.6 beside one of the rest, 2.1 beside another of the prefix, and 6 to begin and end; the rest needs 10 us
// in what is free, and after the prefix where nothing is. So one a CU up to 19 tiles each, then two: 3,072 tiles in
// 240 workgroups 28 us, 336 30, 456 33; 7,504 in 256 68 with the join, 512 57. Of 64 a CU has three, and 9 tiles
// each are best up to two: 4,512 in 240 48 us, 480 36; 3,500 in 384 29, 512 32. In the few-rows form up to 1,024 workgroups of 512
// tokens at least: 64 packed rows of 12 groups over 8,200 tokens 31 us, in 2,048 workgroups 39. Of the rest: 1,024 tokens at
// least, as its workgroups run beside the prefix's: 16 sequences over 6,000 of their own 44 us, 256 tokens
// 57, 4,096 68. (Between 12 and 29 tiles, between two and three workgroups of 64, and for heads of 256 nothing was measured.)
//
// The rest is always the few-rows form's, which has no tiles of 128 to fill. 32 heads of 128 over 8, us with the rest in
// it, in the prompt form, and of mxfp4_attention, behind 8,000 shared tokens:
//   packed rows   sequences   own tokens
//    36            8            4,000        51   60   78
//    36           64            8,000       349  567  624
//   112            8              500        58   70  102
//   112           24            4,000       211  185  251
//   112           64            8,000       783  650 1102
//   800            8            8,000       641  562  630
//   800           24              500       759  710  824
//   800           24            8,000      1852 1461 1537
//   800           64            8,000      5022 3705 3931
// So it gains up to two fifths with some 36 rows, and loses up to a third with 112 and more over long tokens of their
// own, where the call can then take longer than mxfp4_attention, which shares nothing.
constexpr int kMxJoinTokens = 800;

inline int64_t mx_least(int64_t a, int64_t b) { return a < b ? a : b; }

// row tiles of a launch, by their numbering (mx_rows)
inline int64_t mx_part_tiles(int64_t packed, int64_t sequences, int rows) {
  return (packed + rows - 1) / rows + sequences - 1;
}

inline MxPrefixPlan mx_prefix_plan(int64_t tokens, int64_t batch, int64_t groups, int64_t heads, int64_t kv_heads,
                                   int64_t head_dim, int64_t max_prefix, int64_t max_own) {
  MxPrefixPlan p;
  const int64_t listed = groups;
  groups = mx_least(groups, tokens);
  p.prefix = mx_attention_plan(tokens, groups, heads, kv_heads, head_dim, max_prefix, 0, 0);
  const int64_t rows = tokens * (heads / kv_heads);
  auto tiles = [&](int64_t sequences, int of) { return ((rows + sequences - 1) / sequences + of - 1) / of * sequences; };
  const int64_t own_tiles = tiles(batch, 128), prefix_tiles = tiles(groups, p.prefix.few ? 16 * p.prefix.row_tiles : 128);
  p.own = mx_attention_plan(tokens, batch, heads, kv_heads, head_dim, max_prefix + max_own, 0, 0);
  p.through = !p.own.few && (own_tiles - prefix_tiles) * max_prefix <= kMxJoinTokens * own_tiles;
  if (!p.through) {
    p.own.few = true;
    p.own.row_tiles = head_dim == 64 && rows > 16 * batch ? 2 : 1;
    const int64_t s = 2048 / (tiles(batch, 16 * p.own.row_tiles) * kv_heads);
    p.own.splits = (int)mx_least(s < 1 ? 1 : s, max_own < 2048 ? 1 : mx_least(max_own / 1024, kMxMostSplits / 2));
  }
  const int64_t units = prefix_tiles * kv_heads;
  int64_t s;
  if (p.prefix.few) {
    s = mx_least(1024 / units, max_prefix / 512);
  } else {
    const int64_t steps = units * (max_prefix / 64);
    int64_t most = 256;  // workgroups
    if (head_dim == 64 && steps > 9 * 256) most = mx_least(steps / 9, 512);
    if (head_dim == 128 && steps > 19 * 256) most = 512;
    s = mx_least(most / units, max_prefix / 128);
  }
  p.prefix.splits = (int)mx_least(s < 1 ? 1 : s, kMxMostSplits / 2);
  p.prefix.mixed = p.own.mixed = 0;
  // Groups and sequences without rows have tile numbers too. Many of them (10,000 groups of which one has rows) times the
  // pieces would be a launch of workgroups that only end, or none at all beyond 2^24.
  const int64_t numbers = mx_part_tiles(rows, listed, p.prefix.few ? 16 : 128) * p.prefix.splits +
                          mx_part_tiles(rows, batch, 16) * p.own.splits;
  if (!p.through && numbers * kv_heads > 1 << 15) p.prefix.splits = p.own.splits = 1;
  return p;
}

inline int64_t mx_prefix_bytes(const MxPrefixPlan& p, int64_t tokens, int64_t heads, int64_t head_dim) {
  if (p.through) return mx_prompt_part_bytes(p.own, tokens, heads, head_dim);
  return ((p.prefix.splits + p.own.splits) * tokens * heads * (head_dim + 2) * 4 + tokens * 4 + 15) / 16 * 16;
}

hipError_t mx_attention_prompt_setup();
hipError_t launch_mx_attention_prompt(const MxAttnArgs& a, hipStream_t stream);
hipError_t mx_attention_prefix_setup();
hipError_t launch_mx_attention_join_parts(const MxAttnArgs& a, hipStream_t stream);

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
// the lengths; numbers without a tile have first >= count. For a prefix a group of sequences
// takes the place of a sequence, with the rows of all of them.
struct MxRows {
  int seq;
  int64_t r0;     // the sequence's first row in the packed tensors
  int count;      // packed rows of the sequence
  int first;      // the tile's first packed row
  int kv_len;
  int back;       // position of the sequence's first row
  int from;       // kMxOwn, kMxThrough: the first token that is not its group's, a multiple of kMxShared
  bool shared;    // kMxOwn: the prefix's pieces hold for it
  int prefix;     // kMxThrough: its group
};

template <MxPart PART>
__device__ __forceinline__ int64_t mx_part_start(const MxAttnArgs& a, int i) {
  if constexpr (PART == kMxPrefix) {
    const int s = a.prefix.starts[i];
    return mx_row_start(a.b, s < 0 ? 0 : (s < a.b.batch ? s : a.b.batch));
  }
  return mx_row_start(a.b, i);
}

__device__ __forceinline__ int mx_prefix_len(const MxAttnArgs& a, int group) {
  const int64_t v = a.prefix.lens[group], most = (int64_t)a.prefix.max_pages << a.b.page_shift;
  return (int)(v < 0 ? 0 : (v > most ? most : v)) & -kMxShared;
}

// what the rows of sequence (or group) i see, and of a sequence what its group has seen for it
template <MxPart PART>
__device__ __forceinline__ void mx_rows_see(const MxAttnArgs& a, int i, int64_t r1, MxRows& r) {
  r.from = r.prefix = 0;
  r.shared = false;
  if constexpr (PART == kMxPrefix) {
    r.kv_len = mx_prefix_len(a, i);
    r.back = 0;
    return;
  }
  r.kv_len = mx_seq_len(a.b, i);
  r.back = r.kv_len - (int)(r1 - r.r0);
  if constexpr (PART == kMxOwn || PART == kMxThrough) {
    const int lo = mx_last(a.prefix.groups, [&](int g) { return a.prefix.starts[g] <= i; });
    if (a.prefix.starts[lo] <= i && i < a.prefix.starts[lo + 1]) {
      const int len = mx_prefix_len(a, lo);
      r.shared = len <= (a.causal ? r.back + 1 : r.kv_len);  // its first row sees all of it
      r.from = r.shared ? len : 0;
      r.prefix = lo;
    }
  }
}

// mx_rows of a part where there are up to 63 groups (and sequences): what the search and its answer need is in the
// lanes after one load (of starts of groups two), instead of four that wait for one another. (prefix of 6,000 behind
// 4 sequences of 5 rows each, 6 groups, heads of 64 29.8 -> 29.0 us, of 128 59.2 -> 57.8)
template <MxPart PART>
__device__ __forceinline__ MxRows mx_rows_near(const MxAttnArgs& a, int64_t tile, int rows) {
  const int lane = __lane_id(), groups = a.prefix.groups, n = PART == kMxPrefix ? groups : a.b.batch;
  const int group = a.prefix.starts[lane < groups ? lane : groups];
  const int shared = mx_prefix_len(a, lane < groups ? lane : groups - 1);
  const int len = PART == kMxPrefix ? shared : mx_seq_len(a.b, lane < n ? lane : n - 1);
  const int64_t start = mx_part_start<PART>(a, lane < n ? lane : n);
  const int below = __popcll(__ballot(lane < n && start * a.group / rows + lane <= tile));
  MxRows r;
  r.seq = below > 0 ? below - 1 : 0;
  r.r0 = __builtin_amdgcn_readlane((int)start, r.seq);
  const int r1 = __builtin_amdgcn_readlane((int)start, r.seq + 1);
  r.count = r1 > r.r0 ? (int)((r1 - r.r0) * a.group) : 0;
  const int64_t first = (tile - (r.r0 * a.group / rows + r.seq)) * rows;
  r.first = first < 0 || first > r.count ? r.count : (int)first;
  r.kv_len = __builtin_amdgcn_readlane(len, r.seq);
  r.back = r.from = r.prefix = 0;
  r.shared = false;
  if constexpr (PART == kMxPrefix) return r;
  r.back = r.kv_len - (int)(r1 - r.r0);
  const int g = __popcll(__ballot(lane < groups && group <= r.seq)) - 1;
  if (g >= 0 && r.seq < __builtin_amdgcn_readlane(group, g + 1)) {
    const int s = __builtin_amdgcn_readlane(shared, g);
    r.shared = s <= (a.causal ? r.back + 1 : r.kv_len);
    r.from = r.shared ? s : 0;
    r.prefix = g;
  }
  return r;
}

template <MxPart PART = kMxWhole>
__device__ __forceinline__ MxRows mx_rows(const MxAttnArgs& a, int64_t tile, int rows) {
  if constexpr (PART != kMxWhole)
    if (a.prefix.groups < 64 && (PART == kMxPrefix || a.b.batch < 64)) return mx_rows_near<PART>(a, tile, rows);
  int lo = 0;
  if constexpr (PART == kMxWhole) {  // (mx_last here: the prompt form of 64 spills 12 registers for 9, 95 us for 91)
    int hi = a.b.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (mx_row_start(a.b, mid) * a.group / rows + mid <= tile) lo = mid;
      else hi = mid;
    }
  } else {
    lo = mx_last(PART == kMxPrefix ? a.prefix.groups : a.b.batch,
                 [&](int i) { return mx_part_start<PART>(a, i) * a.group / rows + i <= tile; });
  }
  MxRows r;
  const int64_t r1 = mx_part_start<PART>(a, lo + 1);
  r.seq = lo;
  r.r0 = mx_part_start<PART>(a, lo);
  r.count = r1 > r.r0 ? (int)((r1 - r.r0) * a.group) : 0;
  const int64_t first = (tile - (r.r0 * a.group / rows + lo)) * rows;
  r.first = first < 0 || first > r.count ? r.count : (int)first;
  mx_rows_see<PART>(a, lo, r1, r);
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
  mx_rows_see<kMxWhole>(a, seq, r1, r);
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

// (Rows that see a group's prefix see all of it; of what is left, masks by the last token only.)
template <MxPart PART = kMxWhole>
__device__ __forceinline__ MxSight mx_sight(const MxAttnArgs& a, const MxRows& r, int p0, int p1) {
  if constexpr (PART == kMxPrefix) return MxSight{r.kv_len, r.kv_len, 0, 0, 0};
  const int pos_a = r.back + p0 / a.group, pos_b = r.back + (p1 - 1) / a.group;
  if constexpr (PART == kMxOwn) return MxSight{mx_high(a, r.kv_len, pos_a), mx_high(a, r.kv_len, pos_b), r.from, r.from, 0};
  if constexpr (PART == kMxThrough) return MxSight{mx_high(a, r.kv_len, pos_a), mx_high(a, r.kv_len, pos_b), 0, 0, 0};
  return MxSight{mx_high(a, r.kv_len, pos_a), mx_high(a, r.kv_len, pos_b), mx_low(a, pos_a), mx_low(a, pos_b),
                 a.window > 0 ? a.sinks : 0};
}

// Which piece, kv head and row tile a workgroup of a part has. Row tiles of a group read the
// same tokens, so where pieces and kv heads divide over the 8 XCDs (workgroup i is on XCD i % 8)
// those of one piece and kv head follow one another on one XCD, whose L2 then has them.
struct MxPlace {
  int split, kvh, tile;
};

__device__ __forceinline__ MxPlace mx_place(const MxAttnArgs& a, int id) {
  const int kv = a.c.kv_heads, units = a.splits * kv;
  int unit, tile;
  if (units % 8 == 0) {
    const int i = id >> 3;
    tile = i % a.tiles;
    unit = i / a.tiles * 8 + (id & 7);
  } else {
    unit = id % units;
    tile = id / units;
  }
  return MxPlace{unit / kv, unit % kv, tile};
}

__device__ __forceinline__ MxPlace mx_place_whole(const MxAttnArgs& a) {
  return MxPlace{(int)blockIdx.y, (int)blockIdx.x % a.c.kv_heads, (int)(gridDim.x - 1 - blockIdx.x) / a.c.kv_heads};
}

// the tokens [low, high) that packed row p sees (but for first tokens below sinks)
template <MxPart PART>
__device__ __forceinline__ int mx_row_high(const MxAttnArgs& a, const MxRows& r, int i) {
  return PART == kMxPrefix ? r.kv_len : mx_high(a, r.kv_len, r.back + i);
}

template <MxPart PART>
__device__ __forceinline__ int mx_row_low(const MxAttnArgs& a, const MxRows& r, int i) {
  return PART == kMxWhole ? mx_low(a, r.back + i) : PART == kMxThrough ? 0 : r.from;
}

// the block table's row of the sequence or group
template <MxPart PART>
__device__ __forceinline__ const int32_t* mx_table(const MxAttnArgs& a, const MxRows& r) {
  return PART == kMxPrefix ? a.prefix.block_table + (int64_t)r.seq * a.prefix.table_stride
                           : a.b.block_table + (int64_t)r.seq * a.b.table_stride;
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
