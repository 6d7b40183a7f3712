// mx.hpp - device helpers and host-side argument structs of the MXFP4 operators (gfx950).
//
// MXFP4: 32 consecutive elements of a row share one E8M0 scale byte S (value 2^(S-127),
// 255 is NaN); each element is an E2M1 code. For a block whose largest magnitude is A,
// S = max(floor(log2 A) - 2 + 127, 0), so the scaled block lies in [0, 8) and magnitudes
// above 6 saturate. A block that holds an infinity or a NaN gets S = 255 and codes 0, and
// reads back as NaN throughout.
//
// gfx950 converts between bf16 and E2M1 under such a scale in one instruction for two
// elements (v_cvt_scalef32_pk_fp4_bf16 and v_cvt_scalef32_pk_bf16_fp4): the scale operand
// is the float whose exponent field is S. Checked against the definition over every byte
// S and every bf16 input: nearest, ties to the even code, saturating at 6, subnormals kept,
// S = 0 meaning 2^-127 and S = 255 decoding to NaN.
#pragma once

#include "common.hpp"

namespace nvfp4 {

constexpr int kMxBlock = 32;

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;

// |x| of two packed bf16 as unsigned 16-bit patterns: order of patterns is order of values
typedef __attribute__((ext_vector_type(2))) uint16_t u16x2_t;

__device__ __forceinline__ u16x2_t mx_abs2(uint32_t w) {
  const uint32_t a = w & 0x7FFF7FFFu;
  u16x2_t r;
  __builtin_memcpy(&r, &a, 4);
  return r;
}

__device__ __forceinline__ u16x2_t mx_max2(u16x2_t a, u16x2_t b) { return __builtin_elementwise_max(a, b); }

// the largest |x| pattern of a block held by four adjacent lanes, 8 elements each
__device__ __forceinline__ uint32_t mx_quad_amax(const u32x4_t& w) {
  const u16x2_t m = mx_max2(mx_max2(mx_abs2(w[0]), mx_abs2(w[1])), mx_max2(mx_abs2(w[2]), mx_abs2(w[3])));
  uint32_t a = m[0] > m[1] ? m[0] : m[1];
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, false);  // lane ^ 1
  a = a > o ? a : o;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, false);  // lane ^ 2
  return a > o ? a : o;
}

// E8M0 byte of a block from the bf16 pattern of its largest magnitude: the exponent field
// E is floor(log2 A) + 127 for normal A; subnormal A (E = 0) clamps to byte 0 like every
// A below 2^-124; E = 255 is an infinity or a NaN
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const uint32_t E = amax >> 7;
  return E == 255u ? 255u : (E > 2u ? E - 2u : 0u);
}

__device__ __forceinline__ bf16x2_t as_bf16x2(uint32_t w) {
  bf16x2_t r;
  __builtin_memcpy(&r, &w, 4);
  return r;
}

__device__ __forceinline__ uint32_t as_u32(bf16x2_t v) {
  uint32_t r;
  __builtin_memcpy(&r, &v, 4);
  return r;
}

// 8 bf16 -> 8 E2M1 codes (element i in bits 4i .. 4i + 3)
__device__ __forceinline__ uint32_t mx_encode8(const u32x4_t& w, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, as_bf16x2(w[0]), s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, as_bf16x2(w[1]), s, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, as_bf16x2(w[2]), s, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, as_bf16x2(w[3]), s, 3);
  return byte == 255u ? 0u : q;
}

// 8 E2M1 codes -> 8 bf16 (exact for every byte that quantization writes)
__device__ __forceinline__ u32x4_t mx_decode8(uint32_t q, float s) {
  u32x4_t w;
  w[0] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
  w[1] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
  w[2] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
  w[3] = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
  return w;
}

// Sequences of a packed batch and the pages of their caches, as the callers give them.
// Device contents are not trusted: lengths are clamped to what the buffers hold, and a
// page number outside [0, num_pages) is a page that is not there.
struct MxBatch {
  const int32_t* block_table;  // [batch, max_pages]
  const int32_t* seq_lens;     // [batch] cached tokens, the call's new ones included
  const int32_t* cu_seqlens;   // [batch + 1] first row of each sequence
  int64_t table_stride;        // elements between rows of block_table
  int64_t num_pages;
  int batch;
  int max_pages;
  int page_shift;              // page_size = 1 << page_shift
  int64_t tokens;              // rows of the packed tensors
};

struct MxCache {
  uint8_t* k_codes;   // [num_pages, kv_heads, page_size, head_dim / 2]
  uint8_t* k_scales;  // [num_pages, kv_heads, page_size, head_dim / 32]
  uint8_t* v_codes;
  uint8_t* v_scales;
  int kv_heads;
  int head_dim;
};

__device__ __forceinline__ int64_t mx_row_start(const MxBatch& b, int i) {
  const int64_t v = b.cu_seqlens[i];
  return v < 0 ? 0 : (v > b.tokens ? b.tokens : v);
}

__device__ __forceinline__ int mx_seq_len(const MxBatch& b, int i) {
  const int64_t v = b.seq_lens[i], most = (int64_t)b.max_pages << b.page_shift;
  return (int)(v < 0 ? 0 : (v > most ? most : v));
}

// The last i of [0, n) for which at(i), which holds up to some i and not beyond (0 if nowhere): 64
// candidates at a time, one a lane, because every step waits for a load. All lanes take part.
template <typename F>
__device__ __forceinline__ int mx_last(int n, F at) {
  const int lane = __lane_id();
  int lo = 0;
  while (n > 1) {
    const int step = (n + 63) >> 6, i = lane * step;
    const bool yes = i < n && at(lo + i);
    const int below = __popcll(__ballot(yes));
    const int skip = below > 0 ? (below - 1) * step : 0;
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// The sequence of a packed row, found by a whole wave: the row is one of its own if it lies in [r0, r1).
// Up to 63 sequences cost one load's latency, their starts and lengths in the lanes.
struct MxSequence {
  int64_t r0, r1;
  int seq, len;
};

__device__ __forceinline__ MxSequence mx_sequence(const MxBatch& b, int64_t row) {
  if (b.batch >= 64) {
    const int i = mx_last(b.batch, [&](int k) { return b.cu_seqlens[k] <= row; });
    return MxSequence{mx_row_start(b, i), mx_row_start(b, i + 1), i, mx_seq_len(b, i)};
  }
  const int lane = __lane_id(), last = b.batch - 1;
  const int64_t start = mx_row_start(b, lane < b.batch ? lane : b.batch);
  const int len = mx_seq_len(b, lane < last ? lane : last);
  const int below = __popcll(__ballot(lane < b.batch && start <= row));
  const int i = below > 0 ? below - 1 : 0;
  return MxSequence{__builtin_amdgcn_readlane((int)start, i), __builtin_amdgcn_readlane((int)start, i + 1), i,
                    __builtin_amdgcn_readlane(len, i)};
}

// Where packed row `row` lives in the cache: its sequence is the last one that starts at
// or before it. False for a row of no sequence; otherwise pos is its position (negative
// if the sequence is shorter than its rows) and page its page, or -1 if that is not there.
__device__ __forceinline__ bool mx_locate(const MxBatch& b, int64_t row, int& pos, int64_t& page) {
  int lo = 0, hi = b.batch;  // cu_seqlens[lo] <= row, by search
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.cu_seqlens[mid] <= row) lo = mid;
    else hi = mid;
  }
  const int64_t r0 = mx_row_start(b, lo), r1 = mx_row_start(b, lo + 1);
  if (row < r0 || row >= r1) return false;
  pos = mx_seq_len(b, lo) - (int)(r1 - row);
  page = -1;
  if (pos >= 0) {
    const int64_t p = b.block_table[(int64_t)lo * b.table_stride + (pos >> b.page_shift)];
    if (p >= 0 && p < b.num_pages) page = p;
  }
  return true;
}

}  // namespace nvfp4
