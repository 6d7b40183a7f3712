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
  float scale_log2;                              // scale * log2 e
  int causal, window, sinks;                     // window 0: none
  int splits;
  float* part_o;    // [splits, tokens, heads, head_dim]
  float2* part_ml;  // [splits, tokens, heads] maximum (log2) and sum
};

// How a call is cut, from its sizes alone.
struct MxAttnPlan {
  bool coop;      // a workgroup's four waves share its rows and split the tokens
  int row_tiles;  // 16-row tiles of a wave
  int splits;     // pieces of the token axis, joined by a second launch
};

// Rows: the packed rows (rows x heads of a group) of an average sequence. Up to 64 of them
// fit one wave, and the four waves of a workgroup split the tokens; beyond that every wave
// takes rows of its own.
// Splits: enough workgroups to fill 256 CUs four times where the rows alone do not, but
// at least kMinTiles 32-token tiles a wave, so that a split is more than its own start
// and its share of the join.
inline MxAttnPlan mx_attention_plan(int64_t tokens, int64_t batch, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                    int64_t max_kv, int64_t window, int64_t sinks) {
  constexpr int64_t kWanted = 1024, kMinTiles = 2, kMostSplits = 256;
  MxAttnPlan p{true, 1, 1};
  if (tokens <= 0 || batch <= 0) return p;
  const int64_t group = heads / kv_heads;
  const int64_t rows = (tokens + batch - 1) / batch * group;
  const int most = head_dim == 256 ? 2 : 4;
  p.coop = rows <= 16 * most;
  p.row_tiles = p.coop ? (rows <= 16 ? 1 : rows <= 32 ? 2 : most) : most;
  const int64_t per_group = 16 * p.row_tiles * (p.coop ? 1 : 4);
  int64_t tiles = (tokens * group + per_group - 1) / per_group;
  if (tiles < batch) tiles = batch;
  const int64_t groups = tiles * kv_heads;
  int64_t seen = max_kv;
  if (window > 0) {  // a row tile's span: the window, its rows, the first tokens
    const int64_t w = window + per_group / group + sinks;
    if (w < seen) seen = w;
  }
  const int64_t most_splits = seen / (32 * kMinTiles * (p.coop ? 4 : 1));
  int64_t s = groups >= kWanted ? 1 : kWanted / groups;
  if (s > most_splits) s = most_splits;
  if (s > kMostSplits) s = kMostSplits;
  p.splits = s < 1 ? 1 : (int)s;
  return p;
}

}  // namespace nvfp4
