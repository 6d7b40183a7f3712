// mx_attn_prompt.hip - attention over a paged MXFP4 cache, for many rows of a sequence
// (gfx950): prompts and prompt chunks. The operator and the packing of rows and heads are
// those of mx_attn.hip.
//
// What bounds it is arithmetic: the two matrix products, and one exp2 per score beside them.
// A workgroup has 128 RB packed rows, 32 RB to a wave, and walks the tokens 64 at a time. A
// tile's codes are decoded once for the workgroup, into bf16 in LDS, and the products run on
// v_mfma_f32_32x32x16_bf16 in the transposed form, lane (n, h) = (lane & 31, lane >> 5):
//
//   S^T = K Q^T    A: token n, elements 16 s + 8 h .. + 7 of step s, a 16-byte LDS read.
//                  S^T comes out with lane (n, h) holding packed row n and, of 32 tokens,
//                  8 (i / 4) + 4 h + i % 4 in register i.
//   O^T = V^T P^T  B: P as S^T left it: registers 8 s .. 8 s + 7 are the lane's 8 of the 16
//                  tokens of step s. A: element n of a block of 32, the same 8 tokens - V is
//                  laid in LDS by element with its tokens in that order, again one read.
//
// Each wave reads the whole tile from LDS for its 32 RB rows; with 64 rows (RB = 2) that is
// half of what LDS can deliver in the time of the products. O, Q, two halves' scores and the
// weights are then about 330 registers: one wave a SIMD, so overlap comes from the
// instruction stream. A tile goes in two halves of 32 tokens; the scores of the next half
// are multiplied while this one's exponentials are taken, and the next tile is decoded
// beside the products with V:
//
//   barrier | S1 = K[t]1 Q     ||  P = exp2(S0) | O += V[t]0 P  ||  decode K[t + 1]
//   barrier | S0 = K[t + 1]0 Q ||  P = exp2(S1) | O += V[t]1 P  ||  decode V[t + 1]
//
// Masks are put into S as -inf, only in tiles that some row does not see whole. Arithmetic
// and the raising of the maximum are those of mx_attn.hip.
#include "mx_attn.hpp"

namespace nvfp4 {

namespace {

constexpr int kWaves = 4;
constexpr int kTile = 64;  // tokens per step: 16 to a wave when they are decoded

// position of 16-byte chunk c of K row t (D / 8 chunks) and of V row d (8 chunks): the 16
// rows that a read phase meets lie in different banks
template <int D>
__device__ __forceinline__ int k_chunk(int t, int c) {
  return c ^ (D == 64 ? (t >> 1) & 7 : t & 15);
}
__device__ __forceinline__ int v_chunk(int d, int c) { return c ^ (((d >> 1) ^ (d >> 3)) & 7); }

template <int D>
struct Lds {
  static constexpr int K = kTile * D * 2, V = D * kTile * 2;  // bytes of a tile
  static constexpr int Nan = D / 32 * kTile;                  // V bytes that are NaN, [block][token]
  static constexpr int VAt = 2 * K, NanAt = VAt + 2 * V, FlagAt = NanAt + 2 * Nan, Bytes = FlagAt + 2 * 4 * kWaves;
};

template <int D, int RB>
__global__ __launch_bounds__(64 * kWaves, 1) void mx_attention_prompt_kernel(MxAttnArgs a) {
  using L = Lds<D>;
  constexpr int KS = D / 16, DB = D / 32;
  constexpr int kRows = 32 * RB * kWaves;
  extern __shared__ __align__(16) uint8_t smem[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 31, h = lane >> 5;
  const int kvh = blockIdx.x % a.c.kv_heads;
  const int split = blockIdx.y;
  const int g = a.group;
  // within a causal sequence the last tiles see the most tokens: they are started first
  const MxRows rows = mx_rows(a, (gridDim.x - 1 - blockIdx.x) / a.c.kv_heads, kRows);
  if (rows.first >= rows.count) return;  // the whole workgroup
  const int wg_end = rows.first + kRows < rows.count ? rows.first + kRows : rows.count;
  const MxSight all = mx_sight(a, rows, rows.first, wg_end);
  const MxSpan span = mx_span(all, kTile);
  const int begin = (int)((int64_t)span.count * split / a.splits);
  const int end = (int)((int64_t)span.count * (split + 1) / a.splits);

  // ---- the wave's rows ----
  const int p0 = rows.first + wave * 32 * RB;
  const int p1 = p0 + 32 * RB < rows.count ? p0 + 32 * RB : rows.count;
  MxSight sight{0, 0, 0, 0, 0};  // a wave without rows sees nothing
  if (p0 < p1) sight = mx_sight(a, rows, p0, p1);
  if (p1 - p0 < 32 * RB) sight.high_min = 0;
  bf16x8_t q[RB][KS];
  int high[RB], low[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int p = p0 + r * 32 + n;
    const bool real = p < rows.count;
    const int i = p / g;
    const uint16_t* src = a.q + (rows.r0 + i) * a.q_token + (int64_t)(kvh * g + p % g) * a.q_head + 8 * h;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4_t w = {0u, 0u, 0u, 0u};
      if (real) w = *(const u32x4_t*)(src + 16 * s);
      q[r][s] = as_bf16x8(w[0], w[1], w[2], w[3]);
    }
    high[r] = real ? mx_high(a, rows.kv_len, rows.back + i) : 0;
    low[r] = mx_low(a, rows.back + i);
  }

  // ---- a tile's way into LDS: wave w brings tokens 16 w .. 16 w + 15 ----
  // K: a lane takes a quarter of a token's codes; V: D / 16 elements of four tokens
  const int kt = lane >> 2, kq = lane & 3;          // K: token of the 16, quarter
  const int vc = lane & 15, vq = lane >> 4;         // V: elements [vc D/16, + D/16), tokens 4 vq .. + 3
  const int vblk = vc * (D / 16) / 32;
  struct Raw {
    Words<D / 32> k;
    uint32_t ks[D == 256 ? 2 : 1];
    uint32_t v[4][D == 256 ? 2 : 1];
    uint32_t vs[4];
    bool there;  // V's page exists
  };
  auto load_k = [&](Raw& x, int tile) __attribute__((always_inline)) {
    const int t = tile * kTile + wave * 16;
    const int64_t row = mx_cache_row(a, mx_page(a, rows, t), kvh, t) + kt;
    x.k = load_words<D / 32>(a.c.k_codes + row * (D / 2) + kq * (D / 8));
    const uint8_t* s = a.c.k_scales + row * (D / 32) + kq * (D / 4) / 32;
#pragma unroll
    for (int b = 0; b < (D == 256 ? 2 : 1); ++b) x.ks[b] = s[b];
  };
  auto load_v = [&](Raw& x, int tile) __attribute__((always_inline)) {
    const int t = tile * kTile + wave * 16;
    const int64_t page = mx_page(a, rows, t), row = mx_cache_row(a, page, kvh, t) + 4 * vq;
    x.there = page >= 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* p = a.c.v_codes + (row + i) * (D / 2) + vc * (D / 32);
      if constexpr (D == 64) x.v[i][0] = *(const uint16_t*)p;
      else {
        const Words<D / 128> w = load_words<D / 128>(p);
#pragma unroll
        for (int j = 0; j < D / 128; ++j) x.v[i][j] = w.w[j];
      }
      x.vs[i] = a.c.v_scales[(row + i) * (D / 32) + vblk];
    }
  };
  auto store_k = [&](const Raw& x, int buf) __attribute__((always_inline)) {
    uint8_t* dst = smem + buf * L::K + (wave * 16 + kt) * (D * 2);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const u32x4_t w = mx_decode8(x.k.w[e], __uint_as_float(x.ks[D == 256 ? e >> 2 : 0] << 23));
      *(u32x4_t*)(dst + k_chunk<D>(wave * 16 + kt, kq * (D / 32) + e) * 16) = w;
    }
  };
  // V by element. The products must not meet a NaN: 0 * NaN would reach rows that do not
  // see it. NaN blocks go in as zeros (scale 0) and are marked; tokens past the last and on
  // pages that are not there may hold anything and go in under scale 0 too.
  auto store_v = [&](const Raw& x, int buf, int tile) __attribute__((always_inline)) {
    uint8_t* dst = smem + L::VAt + buf * L::V;
    const int t = tile * kTile + wave * 16 + 4 * vq;
    float s[4];
    uint32_t marks = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool nan = x.vs[i] == 255u, token = x.there && t + i < rows.kv_len;
      if (nan && token) marks |= 1u << (8 * i);
      s[i] = __uint_as_float(nan || !token ? 0u : x.vs[i] << 23);
    }
    if ((vc & (16 / DB - 1)) == 0) *(uint32_t*)(smem + L::NanAt + buf * L::Nan + vblk * kTile + wave * 16 + 4 * vq) = marks;
    const uint64_t any = __ballot(marks != 0);
    if (lane == 0) *(uint32_t*)(smem + L::FlagAt + (buf * kWaves + wave) * 4) = any != 0;
    // tokens 4 vq .. + 3 of the 16: lane half vq & 1, first or second four
    const int c = 2 * wave + (vq & 1), off = (vq >> 1) * 8;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) {  // elements 2 d, 2 d + 1 of the lane's
      uint32_t two[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) two[i] = decode2(x.v[i][D == 256 ? d >> 2 : 0], s[i], d & 3);
      const int e = vc * (D / 16) + 2 * d;
      *(u32x2_t*)(dst + e * 128 + v_chunk(e, c) * 16 + off) =
          u32x2_t{__builtin_amdgcn_perm(two[1], two[0], 0x05040100u), __builtin_amdgcn_perm(two[3], two[2], 0x05040100u)};
      *(u32x2_t*)(dst + (e + 1) * 128 + v_chunk(e + 1, c) * 16 + off) =
          u32x2_t{__builtin_amdgcn_perm(two[1], two[0], 0x07060302u), __builtin_amdgcn_perm(two[3], two[2], 0x07060302u)};
    }
  };

  // ---- state ----
  f32x16_t o[RB][DB];
  f32x16_t s0[RB], s1[RB];  // scores of a tile's halves
  float m[RB], l[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[r][d][i] = 0.0f;
  }

  auto scores = [&](f32x16_t (&x)[RB], int buf, int half) __attribute__((always_inline)) {
    const uint8_t* src = smem + buf * L::K;
    const int t = half * 32 + n;
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[r][i] = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const bf16x8_t kf = *(const bf16x8_t*)(src + t * (D * 2) + k_chunk<D>(t, 2 * k + h) * 16);
#pragma unroll
      for (int r = 0; r < RB; ++r) x[r] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, q[r][k], x[r], 0, 0, 0);
    }
  };
  // which 16-token groups of the tile have a page
  auto there_of = [&](int tile) __attribute__((always_inline)) {
    uint32_t there = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) there |= mx_page(a, rows, tile * kTile + 16 * w) >= 0 ? 1u << w : 0u;
    return there;
  };
  // (no short-circuits: selects, not branches around the accumulators)
  auto sees = [&](int r, int t, uint32_t there, int group) __attribute__((always_inline)) {
    return (t < high[r]) & ((t >= low[r]) | (t < sight.sinks)) & ((there >> group & 1u) != 0);
  };
  // register i of a half is its token 8 (i / 4) + 4 h + i % 4
  auto mask = [&](f32x16_t (&x)[RB], int tile, int half, uint32_t there) __attribute__((always_inline)) {
    const int t0 = tile * kTile + half * 32;
    if ((there >> (2 * half) & 3u) == 3u && t0 + 32 <= sight.high_min &&
        (t0 >= sight.low_max || t0 + 32 <= sight.sinks))
      return;
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        x[r][i] = sees(r, t0 + 8 * (i >> 2) + 4 * h + (i & 3), there, 2 * half + (i >> 3)) ? x[r][i] : -INFINITY;
  };
  auto raise = [&](const f32x16_t (&x)[RB]) __attribute__((always_inline)) {
    float top[RB];
    bool need = false;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      top[r] = x[r][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top[r] = fmaxf(top[r], x[r][i]);
      top[r] *= a.scale_log2;
      need |= top[r] > m[r] + kMxRaise;
    }
    if (!__any(need)) return;
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const float next = fmaxf(m[r], fmaxf(top[r], __shfl_xor(top[r], 32, 64)));
      const float f = m[r] == next ? 1.0f : __builtin_amdgcn_exp2f(m[r] - next);  // m = -inf: o and l are 0
      m[r] = next;
      l[r] *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[r][d] *= f;
    }
  };
  bf16x8_t pf[RB][2];
  auto weights = [&](const f32x16_t (&x)[RB]) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const float neg = m[r] == -INFINITY ? 0.0f : -m[r];  // nothing seen yet: every weight is exp2(-inf)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r][8 * k + i], a.scale_log2, neg));
        l[r] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        pf[r][k] = as_bf16x8(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7]));
      }
    }
  };
  auto values = [&](int buf, int half) __attribute__((always_inline)) {
    const uint8_t* src = smem + L::VAt + buf * L::V;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        const int e = d * 32 + n;
        const bf16x8_t vf = *(const bf16x8_t*)(src + e * 128 + v_chunk(e, 4 * half + 2 * k + h) * 16);
#pragma unroll
        for (int r = 0; r < RB; ++r) o[r][d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[r][k], o[r][d], 0, 0, 0);
      }
  };
  // Marked blocks: a product of "is NaN" with "is seen" tells the rows that get one, for the
  // whole block of 32 elements at once.
  auto nans = [&](int buf, int tile) __attribute__((always_inline)) {
    const u32x4_t flag = *(const u32x4_t*)(smem + L::FlagAt + buf * kWaves * 4);
    if (__builtin_amdgcn_readfirstlane(flag[0] | flag[1] | flag[2] | flag[3]) == 0) return;
    const uint32_t there = there_of(tile);
#pragma nounroll
    for (int k = 0; k < 4; ++k) {
      bf16x8_t seen[RB];
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int t = tile * kTile + 16 * k + 8 * (i >> 2) + 4 * h + (i & 3);
          bits |= sees(r, t, there, k) ? 1u << i : 0u;
        }
        seen[r] = mx_ones(bits);
      }
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          bits |= smem[L::NanAt + buf * L::Nan + d * kTile + 16 * k + 8 * (i >> 2) + 4 * h + (i & 3)] ? 1u << i : 0u;
        const bf16x8_t is_nan = mx_ones(bits);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          f32x16_t hit;
#pragma unroll
          for (int i = 0; i < 16; ++i) hit[i] = 0.0f;
          hit = __builtin_amdgcn_mfma_f32_32x32x16_bf16(is_nan, seen[r], hit, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[r][d][i] = hit[i] > 0.0f ? NAN : o[r][d][i];
        }
      }
    }
  };
  auto barrier = [&]() __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's writes are in LDS, its reads done
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // ---- the walk ----
  if (begin < end) {
    Raw x;
    auto clamp = [&](int i) __attribute__((always_inline)) { return span.at(i < end ? i : end - 1); };
    int tile = span.at(begin);
    uint32_t there = there_of(tile);
    load_k(x, tile);
    load_v(x, tile);
    store_k(x, 0);
    store_v(x, 0, tile);
    load_k(x, clamp(begin + 1));
    load_v(x, clamp(begin + 1));
    barrier();
    scores(s0, 0, 0);
    mask(s0, tile, 0, there);
    int buf = 0;
    for (int i = begin; i < end; ++i) {
      const int next = clamp(i + 1);
      // V[i] is in LDS; no wave reads K[i - 1] or V[i - 1] any more
      if (i > begin) barrier();
      nans(buf, tile);
      raise(s0);
      scores(s1, buf, 1);
      weights(s0);
      values(buf, 0);
      store_k(x, buf ^ 1);
      load_k(x, clamp(i + 2));
      mask(s1, tile, 1, there);
      barrier();  // K[i + 1] is in LDS
      raise(s1);
      there = there_of(next);
      scores(s0, buf ^ 1, 0);
      weights(s1);
      values(buf, 1);
      store_v(x, buf ^ 1, next);
      load_v(x, clamp(i + 2));
      mask(s0, next, 0, there);
      tile = next;
      buf ^= 1;
    }
  }

  // ---- the rows' results: lane (n, h) has elements 32 d + 8 k + 4 h .. + 3 of row n ----
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const float sum = l[r] + __shfl_xor(l[r], 32, 64);
    const int p = p0 + r * 32 + n;
    if (p >= rows.count) continue;
    const int64_t token = rows.r0 + p / g;
    const int head = kvh * g + p % g;
    if (a.splits > 1) {
      const int64_t at = ((int64_t)split * a.b.tokens + token) * a.heads + head;
      if (h == 0) a.part_ml[at] = make_float2(m[r], sum);
      if (sum != 0.0f) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *(f32x4_t*)(a.part_o + at * D + 32 * d + 8 * k + 4 * h) =
                f32x4_t{o[r][d][4 * k], o[r][d][4 * k + 1], o[r][d][4 * k + 2], o[r][d][4 * k + 3]};
      }
    } else {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      uint16_t* dst = a.out + token * a.out_token + (int64_t)head * a.out_head;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *(u32x2_t*)(dst + 32 * d + 8 * k + 4 * h) =
              u32x2_t{pack_bf16(o[r][d][4 * k] * inv, o[r][d][4 * k + 1] * inv),
                      pack_bf16(o[r][d][4 * k + 2] * inv, o[r][d][4 * k + 3] * inv)};
    }
  }
}

template <int D, int RB>
hipError_t launch_prompt(const MxAttnArgs& a, hipStream_t stream) {
  const int64_t tiles = a.b.tokens * a.group / (32 * RB * kWaves) + a.b.batch;
  mx_attention_prompt_kernel<D, RB>
      <<<dim3((unsigned)(tiles * a.c.kv_heads), a.splits), 64 * kWaves, Lds<D>::Bytes, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t mx_attention_setup() {
  hipError_t e = hipFuncSetAttribute((const void*)mx_attention_prompt_kernel<64, 2>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, Lds<64>::Bytes);
  if (e == hipSuccess)
    e = hipFuncSetAttribute((const void*)mx_attention_prompt_kernel<128, 2>,
                            hipFuncAttributeMaxDynamicSharedMemorySize, Lds<128>::Bytes);
  if (e == hipSuccess)
    e = hipFuncSetAttribute((const void*)mx_attention_prompt_kernel<256, 1>,
                            hipFuncAttributeMaxDynamicSharedMemorySize, Lds<256>::Bytes);
  return e;
}

hipError_t launch_mx_attention_prompt(const MxAttnArgs& a, hipStream_t stream) {
  switch (a.c.head_dim) {
    case 64: return launch_prompt<64, 2>(a, stream);
    case 128: return launch_prompt<128, 2>(a, stream);
    default: return launch_prompt<256, 1>(a, stream);
  }
}

}  // namespace nvfp4
