// mx_quant.hip - MXFP4 quantization (plain and SwiGLU), its reverse, and the paged
// cache's append and read (gfx950). The format and the conversions are in mx.hpp.
//
// All of these move bytes: a block needs nothing from outside its 32 elements, so one
// launch reads every input once and writes every output once. Work is cut so that a wave
// always moves whole row pieces: a lane takes 8 elements (16 bytes of bf16, 4 bytes of
// codes) and four adjacent lanes share a block, whose maximum they form with two
// cross-lane moves.
#include "mx.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kUnitCols = 512;  // columns of a unit: 64 lanes of 8 elements

// The rows of a unit. The scale layout keeps rows r, r + 32, r + 64, r + 96 of a 128-row
// tile next to each other, so a unit takes 4 consecutive r and all four groups: its 16
// rows' scales are 64 consecutive bytes of each of its four 512-byte scale tiles. Wave g
// of the workgroup has the rows of group g.
__device__ __forceinline__ int64_t unit_row(int64_t tile, int sub, int g, int j) {
  return tile * 128 + g * 32 + sub * 4 + j;
}

struct QuantArgs {
  const uint16_t* x;   // the input, or the gate
  const uint16_t* up;
  int64_t ldx, ldu, m, k;
  uint8_t* qdata;
  uint8_t* scales;
  const uint16_t* silu_table;
  int col_units;       // ceil(k / kUnitCols)
  int scale_groups;    // scale columns / 4
};

// silu_bf16 of 8 packed bf16, correctly rounded: a fast fp32 evaluation, and the
// library's table where that could round the wrong way.
//   f = x * rcp(1 + exp2(t)), t = -x log2 e: each of exp2, 1 + e, rcp and the product is
//   within 1 ulp, and the rounding of t moves the result by at most |t| ulp, so f is
//   within 4 + |t| ulp; the bf16 rounding is safe if f's low 16 bits are further than
//   that from a tie. t > 120 leaves fp32's normal range on the way: also the table.
// For |x| of order 1 one element in about 5,000 takes the table; a table in LDS for all
// would cost 128 KiB of it and a persistent grid.
__device__ __forceinline__ u32x4_t silu8(const u32x4_t& gate, const uint16_t* table) {
  float f[8];
  uint32_t unsafe = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = (i & 1) ? (gate[i >> 1] & 0xFFFF0000u) : (gate[i >> 1] << 16);
    const float x = __uint_as_float(b);
    const float t = x * -1.44269504f;
    f[i] = x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
    const float d = fabsf((float)(int)(__float_as_uint(f[i]) & 0xFFFFu) - 32768.0f);
    if (!(d > 4.0f + fabsf(t)) || t > 120.0f) unsafe |= 1u << i;
  }
  u32x4_t s;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    bf16x2_t c;
    c[0] = (__bf16)f[2 * p];
    c[1] = (__bf16)f[2 * p + 1];
    s[p] = as_u32(c);
  }
  if (unsafe) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (unsafe >> i & 1) {
        const int sh = (i & 1) * 16;
        const uint32_t v = table[(gate[i >> 1] >> sh) & 0xFFFFu];
        s[i >> 1] = (s[i >> 1] & (0xFFFF0000u >> sh)) | (v << sh);
      }
    }
  }
  return s;
}

// RN_bf16(a * b) of 8 packed pairs. The fp32 product of two bf16 values is exact above
// 2^-126; below it the fp64 product is, and is rounded once.
__device__ __forceinline__ u32x4_t mul8(const u32x4_t& a, const u32x4_t& b) {
  u32x4_t y;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float a0 = __uint_as_float(a[p] << 16), a1 = __uint_as_float(a[p] & 0xFFFF0000u);
    const float b0 = __uint_as_float(b[p] << 16), b1 = __uint_as_float(b[p] & 0xFFFF0000u);
    const float p0 = a0 * b0, p1 = a1 * b1;
    bf16x2_t c;
    c[0] = (__bf16)p0;
    c[1] = (__bf16)p1;
    y[p] = as_u32(c);
    // a product that underflowed to zero keeps its sign either way
    if (fabsf(p0) < 0x1p-126f && a0 != 0.0f && b0 != 0.0f)
      y[p] = (y[p] & 0xFFFF0000u) | rn_bf16_from_double((double)a0 * (double)b0);
    if (fabsf(p1) < 0x1p-126f && a1 != 0.0f && b1 != 0.0f)
      y[p] = (y[p] & 0xFFFFu) | (rn_bf16_from_double((double)a1 * (double)b1) << 16);
  }
  return y;
}

// Quantization: one workgroup per unit of 16 rows x 512 columns, in address order. Every
// load of a unit is in flight before the first is used; there is no loop. SwiGLU of 37711 x
// 14336: 395 us, 6.2 TB/s of the 2.45 GB that it cannot do without; one row of 5376: 2.8 us.
template <bool SWIGLU>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(QuantArgs a) {
  __shared__ __align__(16) uint8_t sc[4 * 64];
  const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int64_t unit = blockIdx.x;
  const int cu = (int)(unit % a.col_units);
  const int64_t rest = unit / a.col_units, tile = rest >> 3;
  const int sub = (int)(rest & 7);
  const int64_t col = (int64_t)cu * kUnitCols + lane * 8;
  const bool col_ok = col < a.k;

  u32x4_t w[4], u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t r = unit_row(tile, sub, g, j);
    w[j] = u32x4_t{0u, 0u, 0u, 0u};
    u[j] = w[j];
    if (col_ok && r < a.m) {
      w[j] = __builtin_nontemporal_load((const u32x4_t*)(a.x + r * a.ldx + col));
      if (SWIGLU) u[j] = __builtin_nontemporal_load((const u32x4_t*)(a.up + r * a.ldu + col));
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t r = unit_row(tile, sub, g, j);
    if (SWIGLU) w[j] = mul8(silu8(w[j], a.silu_table), u[j]);
    const uint32_t byte = mx_scale_byte(mx_quad_amax(w[j]));
    const bool real = col_ok && r < a.m;
    if (real) *(uint32_t*)(a.qdata + r * (a.k >> 1) + (col >> 1)) = mx_encode8(w[j], byte);
    // bytes outside real rows and columns are zero
    if ((lane & 3) == 0) sc[(lane >> 4) * 64 + j * 16 + g * 4 + ((lane >> 2) & 3)] = real ? (uint8_t)byte : 0;
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    const int t = threadIdx.x >> 2, piece = threadIdx.x & 3;
    const int64_t group = (int64_t)cu * 4 + t;
    if (group < a.scale_groups)
      *(u32x4_t*)(a.scales + (tile * a.scale_groups + group) * 512 + sub * 64 + piece * 16) =
          *(const u32x4_t*)(sc + t * 64 + piece * 16);
  }
}

struct DequantArgs {
  const uint8_t* qdata;
  const uint8_t* scales;
  uint16_t* y;
  int64_t ldy, m, k;
  int col_units, scale_groups;
};

// The reverse, over the same units: 37711 x 14336 in 255 us, 5.4 TB/s.
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(DequantArgs a) {
  const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int64_t unit = blockIdx.x;
  const int cu = (int)(unit % a.col_units);
  const int64_t rest = unit / a.col_units, tile = rest >> 3;
  const int sub = (int)(rest & 7);
  const int64_t col = (int64_t)cu * kUnitCols + lane * 8;
  if (col >= a.k) return;
  uint32_t q[4], s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t r = unit_row(tile, sub, g, j);
    q[j] = s[j] = 0;
    if (r < a.m) {
      q[j] = *(const uint32_t*)(a.qdata + r * (a.k >> 1) + (col >> 1));
      s[j] = a.scales[(tile * a.scale_groups + (col >> 7)) * 512 + (sub * 4 + j) * 16 + g * 4 + ((lane >> 2) & 3)];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t r = unit_row(tile, sub, g, j);
    if (r < a.m)
      __builtin_nontemporal_store(mx_decode8(q[j], __uint_as_float(s[j] << 23)), (u32x4_t*)(a.y + r * a.ldy + col));
  }
}

// ---- the paged cache ----
// D / 8 lanes take a token's row of one head, 64 / (D / 8) consecutive tokens to a wave:
// their rows lie one after the other in the cache as long as they share a page, and each is
// a whole run of the packed tensor. A lane does kHeads heads of its token (one after the
// other in the packed tensor), so that the search for the token's sequence and page is done
// once for them and their loads overlap. blockIdx.y: group of heads, of K then of V.
// Five prompts, 32765 tokens in all, 8 heads of 128, K and V: appended in 42 us (170 MB, 4.0
// TB/s), read back in 29 us (5.9 TB/s); 48 single tokens 4.0 us each way, launch latency.
constexpr int kHeads = 4;

struct CacheArgs {
  MxBatch b;
  MxCache c;
  uint16_t* k;  // read by the append, written by the read
  uint16_t* v;
  int64_t k_token, k_head, v_token, v_head;  // element strides
  int head_groups;
};

template <int D, bool WRITE>
__global__ __launch_bounds__(kThreads) void mx_cache_kernel(CacheArgs a) {
  constexpr int kLanes = D / 8;  // lanes of a row
  const int sub = threadIdx.x % kLanes;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const bool is_v = (int)blockIdx.y >= a.head_groups;
  const int head0 = (is_v ? blockIdx.y - a.head_groups : blockIdx.y) * kHeads;
  const int heads = a.c.kv_heads - head0 < kHeads ? a.c.kv_heads - head0 : kHeads;
  const int64_t head_stride = is_v ? a.v_head : a.k_head;
  uint16_t* const base = (is_v ? a.v + row * a.v_token : a.k + row * a.k_token) + head0 * head_stride + sub * 8;
  const int page_size = 1 << a.b.page_shift;

  int pos = -1;
  int64_t page = -1;
  const bool known = row < a.b.tokens && mx_locate(a.b, row, pos, page);
  const bool there = known && page >= 0;
  const int64_t at = there ? (page * a.c.kv_heads + head0) * page_size + (pos & (page_size - 1)) : 0;  // head0's row
  uint8_t* const codes = (is_v ? a.c.v_codes : a.c.k_codes) + at * (D / 2) + sub * 4;
  uint8_t* const scales = (is_v ? a.c.v_scales : a.c.k_scales) + at * (D / 32);
  const int64_t code_step = (int64_t)page_size * (D / 2), scale_step = (int64_t)page_size * (D / 32);
  if (WRITE) {
    u32x4_t w[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      w[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (there && i < heads) w[i] = *(const u32x4_t*)(base + i * head_stride);
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const uint32_t byte = mx_scale_byte(mx_quad_amax(w[i]));
      const uint32_t next = __builtin_amdgcn_mov_dpp((int)byte, 0x104, 0xF, 0xF, true);  // of lane + 4, in rows of 16
      if (there && i < heads) {
        *(uint32_t*)(codes + i * code_step) = mx_encode8(w[i], byte);
        if ((sub & 7) == 0) *(uint16_t*)(scales + i * scale_step + (sub >> 2)) = (uint16_t)(byte | next << 8);
      }
    }
  } else {
    uint32_t q[kHeads], s[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      q[i] = s[i] = 0;  // a row that is not in the cache reads as zeros
      if (there && i < heads) {
        q[i] = *(const uint32_t*)(codes + i * code_step);
        s[i] = scales[i * scale_step + (sub >> 2)];
      }
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      if (known && i < heads) *(u32x4_t*)(base + i * head_stride) = mx_decode8(q[i], __uint_as_float(s[i] << 23));
  }
}

}  // namespace

// workgroups along the tokens
int64_t mx_cache_groups(int64_t tokens, int64_t head_dim) {
  const int64_t rows = kThreads / (head_dim / 8);
  return (tokens + rows - 1) / rows;
}

namespace {

template <bool WRITE>
hipError_t launch_cache(CacheArgs a, hipStream_t stream) {
  a.head_groups = (a.c.kv_heads + kHeads - 1) / kHeads;
  const dim3 grid((unsigned)mx_cache_groups(a.b.tokens, a.c.head_dim), 2 * a.head_groups);
  switch (a.c.head_dim) {
    case 64: mx_cache_kernel<64, WRITE><<<grid, kThreads, 0, stream>>>(a); break;
    case 128: mx_cache_kernel<128, WRITE><<<grid, kThreads, 0, stream>>>(a); break;
    default: mx_cache_kernel<256, WRITE><<<grid, kThreads, 0, stream>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace

int64_t mx_quant_units(int64_t m, int64_t k) { return (m + 127) / 128 * 8 * ((k + kUnitCols - 1) / kUnitCols); }

hipError_t launch_mx_quantize(const uint16_t* x, int64_t ldx, const uint16_t* up, int64_t ldu, int64_t m, int64_t k,
                              uint8_t* qdata, uint8_t* scales, const uint16_t* silu_table, hipStream_t stream) {
  QuantArgs a{x, up, ldx, ldu, m, k, qdata, scales, silu_table, (int)((k + kUnitCols - 1) / kUnitCols),
              (int)((k / kMxBlock + 3) / 4)};
  const unsigned units = (unsigned)mx_quant_units(m, k);
  if (up) mx_quantize_kernel<true><<<units, kThreads, 0, stream>>>(a);
  else mx_quantize_kernel<false><<<units, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* qdata, const uint8_t* scales, uint16_t* y, int64_t ldy, int64_t m,
                                int64_t k, hipStream_t stream) {
  DequantArgs a{qdata, scales, y, ldy, m, k, (int)((k + kUnitCols - 1) / kUnitCols), (int)((k / kMxBlock + 3) / 4)};
  mx_dequantize_kernel<<<(unsigned)mx_quant_units(m, k), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_mx_cache_append(const MxBatch& b, const MxCache& c, const uint16_t* k, int64_t k_token,
                                  int64_t k_head, const uint16_t* v, int64_t v_token, int64_t v_head,
                                  hipStream_t stream) {
  return launch_cache<true>(CacheArgs{b, c, (uint16_t*)k, (uint16_t*)v, k_token, k_head, v_token, v_head, 0}, stream);
}

hipError_t launch_mx_cache_read(const MxBatch& b, const MxCache& c, uint16_t* k, int64_t k_token, int64_t k_head,
                                uint16_t* v, int64_t v_token, int64_t v_head, hipStream_t stream) {
  return launch_cache<false>(CacheArgs{b, c, k, v, k_token, k_head, v_token, v_head, 0}, stream);
}

}  // namespace nvfp4
