// mx_rope.hip - norms of query and key heads with their rotation, in one pass, and on into
// the paged MXFP4 cache (gfx950).
//
//   n   = x w / sqrt(mean(x^2) + eps)                   of a head's D elements
//   a'  = a cos t - b sin t,  b' = b cos t + a sin t     of the pairs (a, b) of n, t = position * freq
//
// bf16 in, one rounding to bf16 out; keys and values then become MXFP4 at their place in the
// cache (mx_quant.hip does that alone).
//
// What bounds it is moving the bytes, each read and written once. A lane has 16 elements of
// one head, so D / 16 lanes share a head and a step of a wave is 1024 / D heads of a token.
// With pairs half the turned elements apart (j, j + R / 2) the 16 are the runs [8 l, + 8)
// and [R / 2 + 8 l, + 8), otherwise one run: either way both elements of 8 pairs, no
// exchange between lanes, and pair 8 l is the lane's first.
//
// A token's angles are the same for all of its heads: lane j finds cosine and sine of pair j
// once, in fp64, and the wave keeps them in LDS. Queries are then fp32 throughout; keys
// are fp64 (as fast here as unpacked fp32), because the step after their rounding to bf16 is one
// to 4 bits, where a last bit that falls the other way can move the result by half of itself.
//
// Measured: 37,810 tokens, 56 heads of 128, three axes: 220 us, 4.9 TB/s (a large copy: 5.1 to 5.2). 32,765 tokens of 32
// and 8 heads of 128 into the cache: 163 us, 4.3 TB/s; the queries alone take 107, the values' part of the cache 22 beside them
// and the keys' 36, a third of it arithmetic. One token 4.4 us, 48 tokens 4.8. One wave to a token and no more: two make
// it 185 us (the angles and the search twice), four tokens to a wave 196 (registers); loads two steps ahead change nothing.
#include <cmath>

#include "mx_rope.hpp"

namespace nvfp4 {

namespace {

constexpr int kWaves = 4;

// what one wave has in LDS
template <int D>
struct WaveLds {
  double2 turn[D > 128 ? D / 2 : 64];   // cosine, sine of each pair
  float2 turnf[D > 128 ? D / 2 : 64];
  uint16_t k[1024];      // keys on their way into blocks of 32 consecutive elements
};

// orders a wave's own LDS writes before its reads by other lanes
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// cosine and sine of position * freq. The product is exact as hi + lo (31 and 24 bits), and
// so is its first product with 1 / 2 pi as a sum; whole turns are dropped before they cost
// bits: 2^-52 of a turn at every position for frequencies up to 2^24, 2^-44 up to 2^32 (against exact rationals); from
// there on a bit is lost with each of the frequency's, as 1 / 2 pi has 107 here.
__device__ __forceinline__ double2 turn_of(int32_t position, float freq) {
  constexpr double kInv = 0.15915494309189535, kInvLo = -9.839338337591243e-18;  // 1 / 2 pi
  const double p = position, f = freq;
  const double hi = p * f, lo = fma(p, f, -hi);
  const double t = hi * kInv, e = fma(hi, kInv, -t) + fma(hi, kInvLo, lo * kInv);
  const double r = (t - rint(t)) + e;
  double s, c;
  sincospi(2.0 * r, &s, &c);
  return make_double2(c, s);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  bf16x2_t c;
  c[0] = (__bf16)lo;
  c[1] = (__bf16)hi;
  return as_u32(c);
}

// RN_bf16 of two doubles, by way of fp32. That rounding must not make or hide a tie: where it ends on one,
// the bit that it has dropped goes back in.
__device__ __forceinline__ uint32_t pack2(double lo, double hi) {
  float f[2] = {(float)lo, (float)hi};
  const double x[2] = {lo, hi};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t b = __float_as_uint(f[i]);
    if ((b & 0xFFFFu) == 0x8000u) {
      const double d = fabs(x[i]) - (double)fabsf(f[i]);
      f[i] = __uint_as_float(b + (d > 0.0 ? 1u : d < 0.0 ? -1u : 0u));
    }
  }
  return pack2(f[0], f[1]);
}

struct Sixteen {
  u32x4_t w[2];
  __device__ __forceinline__ float at(int i) const {  // bf16 element i
    const uint32_t x = w[i >> 3][(i >> 1) & 3];
    return __uint_as_float(i & 1 ? x & 0xFFFF0000u : x << 16);
  }
};

// the sum over the D / 16 lanes of a head
template <int D, typename T>
__device__ __forceinline__ T head_sum(T x) {
#pragma unroll
  for (int off = 1; off < D / 16; off <<= 1) x += __shfl_xor(x, off, 64);
  return x;
}

// 16 consecutive elements a lane into the cache
template <int D>
__device__ __forceinline__ void put(const Sixteen& x, uint8_t* codes, uint8_t* scales, int64_t row, int sub, bool there) {
  const u16x2_t m = mx_max2(mx_max2(mx_max2(mx_abs2(x.w[0][0]), mx_abs2(x.w[0][1])), mx_max2(mx_abs2(x.w[0][2]), mx_abs2(x.w[0][3]))),
                            mx_max2(mx_max2(mx_abs2(x.w[1][0]), mx_abs2(x.w[1][1])), mx_max2(mx_abs2(x.w[1][2]), mx_abs2(x.w[1][3]))));
  uint32_t top = m[0] > m[1] ? m[0] : m[1];
  const uint32_t other = (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, false);  // lane ^ 1
  top = top > other ? top : other;
  const uint32_t byte = mx_scale_byte(top);
  uint32_t all = byte << (8 * (sub >> 1 & 3));  // of the lanes of four blocks (of 64: two)
  all |= (uint32_t)__builtin_amdgcn_mov_dpp((int)all, 0x4E, 0xF, 0xF, false);  // lane ^ 2
  if (D > 64) all |= (uint32_t)__shfl_xor((int)all, 4, 64);
  if (!there) return;
  *(u32x2_t*)(codes + row * (D / 2) + sub * 8) = u32x2_t{mx_encode8(x.w[0], byte), mx_encode8(x.w[1], byte)};
  if (D == 64) {
    if (sub == 0) *(uint16_t*)(scales + row * (D / 32)) = (uint16_t)all;
  } else {
    if ((sub & 7) == 0) *(uint32_t*)(scales + row * (D / 32) + (sub >> 3) * 4) = all;
  }
}

// (Four waves a SIMD: a fifth, for which the registers of the form without a cache would do, gains nothing;
// 37,810 tokens of 56 heads, twice: 435 us with four, 440 with five.)
template <int D, bool APPEND, bool INTERLEAVED>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(4, 4))) void
mx_rope_kernel(MxRopeArgs a) {
  constexpr int L = D / 16, H = 64 / L;  // lanes of a head, heads of a step
  __shared__ __align__(16) WaveLds<D> lds[kWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  WaveLds<D>& my = lds[wave];
  const int64_t item = (int64_t)blockIdx.x * kWaves + wave;
  const int64_t token = a.parts == 1 ? item : item / a.parts;
  const int part = a.parts == 1 ? 0 : (int)(item - token * a.parts);
  if (token >= a.tokens) return;
  const int sub = lane % L, hl = lane / L;
  const bool turns = sub < a.rotary / 16;
  const int first = INTERLEAVED || !turns ? 16 * sub : 8 * sub;
  const int second = INTERLEAVED || !turns ? first + 8 : a.rotary / 2 + 8 * sub;
  const int qs = (a.heads + H - 1) / H, ks = APPEND ? (a.kv_heads + H - 1) / H : 0, steps = qs + 2 * ks;

  auto load = [&](const uint16_t* head, int at0, int at1) __attribute__((always_inline)) {
    Sixteen x;
    x.w[0] = *(const u32x4_t*)(head + at0);
    x.w[1] = *(const u32x4_t*)(head + at1);
    return x;
  };
  // what step s of the token reads; lanes without a head read the last one's
  auto fetch = [&](int s) __attribute__((always_inline)) {
    if (!APPEND || s < qs) {
      const int head = s * H + hl < a.heads ? s * H + hl : a.heads - 1;
      return load(a.q + token * a.q_token + head * a.q_head, first, second);
    }
    const bool is_v = s >= qs + ks;
    const int h = (s - (is_v ? qs + ks : qs)) * H + hl, head = h < a.kv_heads ? h : a.kv_heads - 1;
    return is_v ? load(a.v + token * a.v_token + head * a.v_head, 16 * sub, 16 * sub + 8)
                : load(a.k + token * a.k_token + head * a.k_head, first, second);
  };
  Sixteen next = fetch(part);

  // ---- what the angles need ----
  const bool angles = part < qs + ks;
  constexpr int kPairs = D > 128 ? D / 128 : 1;  // of a lane
  float freq[kPairs];
  int at[kPairs];  // position
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int j = lane + 64 * i;
    freq[i] = 0.0f;
    at[i] = 0;
    if (angles && j < a.rotary / 2) {
      freq[i] = a.freqs[j];
      if (a.positions) {
        int axis = a.axes ? a.axes[j] : 0;
        axis = axis < 0 ? 0 : axis < a.axis_count ? axis : a.axis_count - 1;
        at[i] = a.positions[token * a.pos_token + axis * a.pos_axis];
      }
    }
  }

  // ---- where the token belongs ----
  int pos = 0;
  int64_t page = -1;  // as the table has it: it is looked at when the first key is written
  if (APPEND) {
    const MxSequence q = mx_sequence(a.b, token);
    if (token < q.r0 || token >= q.r1) return;  // of no sequence
    pos = q.len - (int)(q.r1 - token);
    if (pos >= 0) page = a.b.block_table[(int64_t)q.seq * a.b.table_stride + (pos >> a.b.page_shift)];
  }

  // ---- the angles ----
  if (angles && a.rotary > 0) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const double2 t = turn_of(a.positions ? at[i] : pos, freq[i]);
      my.turn[lane + 64 * i] = t;
      my.turnf[lane + 64 * i] = make_float2((float)t.x, (float)t.y);
    }
    wave_sync();
  }

  for (int s = part; s < steps; s += a.parts) {
    const Sixteen x = next;
    if (s + a.parts < steps) next = fetch(s + a.parts);
    if (!APPEND || s < qs) {
      // ---- queries: fp32 ----
      const int head = s * H + hl;
      float y[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = x.at(i);
      if (a.q_norm.on) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum = fmaf(y[i], y[i], sum);
        sum = head_sum<D>(sum);
        Sixteen w;
        if (a.q_norm.weight) w = load(a.q_norm.weight, first, second);
        else w.w[0] = w.w[1] = u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        // Squares may have left fp32's range, or eps does (one too small for it is nothing beside such sums). A
        // head goes by its own sum, so that it comes out the same whatever stands beside it.
        const bool wide = !(sum > 0x1p-80f && sum < 0x1p100f) || a.q_norm.eps > 0x1p100;
        if (__any(wide)) {
          double d = 0.0;
#pragma unroll
          for (int i = 0; i < 16; ++i) d = fma((double)y[i], (double)y[i], d);
          const double rd = 1.0 / sqrt(head_sum<D>(d) / D + a.q_norm.eps);
          const float r = 1.0f / sqrtf(sum * (1.0f / D) + (float)a.q_norm.eps);
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = wide ? (float)((double)y[i] * rd * (double)w.at(i)) : y[i] * r * w.at(i);
        } else {
          const float r = 1.0f / sqrtf(sum * (1.0f / D) + (float)a.q_norm.eps);
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = y[i] * r * w.at(i);
        }
      }
      if (turns) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 t = my.turnf[8 * sub + j];
          float &p = y[INTERLEAVED ? 2 * j : j], &q = y[INTERLEAVED ? 2 * j + 1 : j + 8];
          const float u = p, v = q;
          p = fmaf(u, t.x, -(v * t.y));
          q = fmaf(v, t.x, u * t.y);
        }
      }
      if (head < a.heads) {
        uint16_t* dst = a.out + token * a.out_token + head * a.out_head;
        const u32x4_t lo = {pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7])};
        const u32x4_t hi = {pack2(y[8], y[9]), pack2(y[10], y[11]), pack2(y[12], y[13]), pack2(y[14], y[15])};
        // (past the caches: 32,765 tokens of 32 heads of 64 75 us, otherwise 97; such loads cost 8 %)
        __builtin_nontemporal_store(lo, (u32x4_t*)(dst + first));
        __builtin_nontemporal_store(hi, (u32x4_t*)(dst + second));
      }
      continue;
    }
    // ---- keys and values ----
    const bool is_v = s >= qs + ks;
    const int head = (s - (is_v ? qs + ks : qs)) * H + hl;
    Sixteen z = x;
    if (!is_v) {
      double y[16], r = 1.0;  // r after the rotation, which is linear
      if (a.k_norm.on) {
        Sixteen w;
        if (a.k_norm.weight) w = load(a.k_norm.weight, first, second);
        else w.w[0] = w.w[1] = u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const double u = x.at(i);
          sum = fma(u, u, sum);
          y[i] = u * (double)w.at(i);
        }
        r = rsqrt(head_sum<D>(sum) / D + a.k_norm.eps);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = x.at(i);
      }
      if (turns) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double2 t = my.turn[8 * sub + j];
          double &p = y[INTERLEAVED ? 2 * j : j], &q = y[INTERLEAVED ? 2 * j + 1 : j + 8];
          const double u = p, v = q;
          p = fma(u, t.x, -(v * t.y));
          q = fma(v, t.x, u * t.y);
        }
      }
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack2(y[2 * i] * r, y[2 * i + 1] * r);
      z.w[0] = u32x4_t{w[0], w[1], w[2], w[3]};
      z.w[1] = u32x4_t{w[4], w[5], w[6], w[7]};
      if (!INTERLEAVED && a.rotary > 0) {
        *(u32x4_t*)(my.k + hl * D + first) = z.w[0];
        *(u32x4_t*)(my.k + hl * D + second) = z.w[1];
        wave_sync();
        z = load(my.k + hl * D, 16 * sub, 16 * sub + 8);
        wave_sync();
      }
    }
    const bool there = page >= 0 && page < a.b.num_pages;
    const int64_t row = (((there ? page : 0) * a.c.kv_heads + head) << a.b.page_shift) + (pos & ((1 << a.b.page_shift) - 1));
    put<D>(z, is_v ? a.c.v_codes : a.c.k_codes, is_v ? a.c.v_scales : a.c.k_scales, row, sub,
           there && head < a.kv_heads);
  }
}

template <int D>
void launch_dim(const MxRopeArgs& a, bool append, bool interleaved, hipStream_t stream) {
  const unsigned groups = (unsigned)((a.tokens * a.parts + kWaves - 1) / kWaves);
  if (append) {
    if (interleaved) mx_rope_kernel<D, true, true><<<groups, 64 * kWaves, 0, stream>>>(a);
    else mx_rope_kernel<D, true, false><<<groups, 64 * kWaves, 0, stream>>>(a);
  } else {
    if (interleaved) mx_rope_kernel<D, false, true><<<groups, 64 * kWaves, 0, stream>>>(a);
    else mx_rope_kernel<D, false, false><<<groups, 64 * kWaves, 0, stream>>>(a);
  }
}

}  // namespace

hipError_t launch_mx_rope(const MxRopeArgs& a, int head_dim, bool append, bool interleaved, hipStream_t stream) {
  switch (head_dim) {
    case 64: launch_dim<64>(a, append, interleaved, stream); break;
    case 128: launch_dim<128>(a, append, interleaved, stream); break;
    default: launch_dim<256>(a, append, interleaved, stream); break;
  }
  return hipGetLastError();
}

}  // namespace nvfp4
