// mx_rope.hpp - arguments of the head norm and rotation kernels.
#pragma once

#include "mx.hpp"

namespace nvfp4 {

struct MxNorm {
  const uint16_t* weight;  // bf16 [head_dim], or null: ones
  double eps;
  bool on;
};

struct MxRopeArgs {
  MxBatch b;  // append only, as the cache
  MxCache c;
  // rotation
  const float* freqs;        // [rotary / 2]
  const int32_t* axes;       // [rotary / 2], or null: axis 0
  const int32_t* positions;  // or null: the row's position in its sequence
  int64_t pos_token, pos_axis;
  int axis_count, rotary;    // rotary 0: none
  MxNorm q_norm, k_norm;
  const uint16_t* q;
  uint16_t* out;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_token, q_head, out_token, out_head, k_token, k_head, v_token, v_head;  // element strides
  int64_t tokens;
  int heads, kv_heads;       // kv_heads 0: no cache
  int parts;                 // waves of a token
};

// Waves of a token: one, which finds the angles once for all heads, where the tokens alone are two
// waves for every SIMD; otherwise up to one for each step of the token's work (1024 / head_dim
// heads of q, k or v), which wait side by side. 32,765 tokens of 32 and 8 heads of 128: 163 us with one, 185 with two,
// 246 with six. Of fewer tokens, into the cache, with one, two, four and all waves:
//   256 tokens   32 and 8 heads of 128  9.1   7.2   6.4   5.5    56 and 8  12.1   8.2   6.6   6.6 (here 6.0)
//   512                                 9.9   7.8   7.3   7.3              12.3   8.7   7.5   9.0
//   1,024                              10.3   8.8   8.6  10.4              12.8  10.1   9.2  12.7
//   2,048                              12.2  11.4  13.4  15.2              21.4  16.8  18.4  21.5
//   4,096                              22.6  22.7  26.0  28.0              32.1  30.6  32.0  38.5
// Heads of 64 and 256 go as 32 of 128 do; alone, without a cache, likewise.
inline int64_t mx_rope_parts(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim) {
  const int64_t per = 1024 / head_dim;
  const int64_t steps = (heads + per - 1) / per + 2 * ((kv_heads + per - 1) / per);
  int64_t parts = tokens > 0 ? (2048 + tokens - 1) / tokens : 1;
  if (parts > steps) parts = steps;
  return parts < 1 ? 1 : parts;
}

hipError_t launch_mx_rope(const MxRopeArgs& a, int head_dim, bool append, bool interleaved, hipStream_t stream);

}  // namespace nvfp4
