// mx_attn_prompt.hip - attention over a paged MXFP4 cache, for many rows of a sequence
// (gfx950): prompts and prompt chunks. The operator and the packing of rows and heads are
// those of mx_attn.hip.
//
// What bounds it is the issue of instructions: the two matrix products, one exp2 per score
// and the rounding of its result, and the reads from LDS go side by side (taking any one of
// them out gains less than a tenth). A workgroup has 128 packed rows, 32 to a wave, and walks
// the tokens 64 at a time. A tile's codes are decoded once for the workgroup, into bf16 in
// LDS, and the products run on v_mfma_f32_32x32x16_bf16 in the transposed form, lane
// (n, h) = (lane & 31, lane >> 5):
//
//   S^T = K Q^T    A: token n, elements 16 s + 8 h .. + 7 of step s, a 16-byte LDS read.
//                  S^T comes out with lane (n, h) holding packed row n and, of 32 tokens,
//                  8 (i / 4) + 4 h + i % 4 in register i.
//   O^T = V^T P^T  B: P as S^T left it: registers 8 s .. 8 s + 7 are the lane's 8 of the 16
//                  tokens of step s. A: element n of a block of 32, the same 8 tokens - V is
//                  laid in LDS by element with its tokens in that order, again one read.
//
// Each wave reads the whole tile from LDS for its 32 rows. 64 rows to a wave would halve
// that, and eight waves the decoding; but then a CU has one or two workgroups where it has
// two or three, with nothing to run beside a barrier or a workgroup's start. Measured, 56
// heads of 128 over 8, 2 ragged prompts: 787 us, eight waves 802, 64 rows 1171. 32 heads over
// 8, 1,500 tokens eight times: 213 us and eight waves 227; of 64, 139 us and 64 rows 158 (they
// gain from 4,096 tokens on only, 9 % at most).
// Waves are few all the same, so overlap comes from the instruction stream as well. A tile
// goes in two halves of 32 tokens, each in two phases of D / 16 matrix instructions beside
// what else is due:
//
//   1  S1 = K[t]1 Q       ||  P = exp2(S0)                  ||  read V[t]0
//   2  O += V[t]0 P       ||  decode V[t + 1] into LDS      ||  read K[t + 1]0   | barrier
//   3  S0 = K[t + 1]0 Q   ||  P = exp2(S1)                  ||  read V[t]1
//   4  O += V[t]1 P       ||  decode K[t + 2] into LDS      ||  read K[t + 1]1   | barrier
//
// Weights are taken under the maximum as it stands, and their sum, which is needed anyway,
// tells afterwards whether a score exceeded it by too much: then the maximum is raised and
// the half's weights are taken again. So most halves look for no maximum at all. The sum is
// of the weights as rounded for the product, two to an instruction (v_dot2_f32_bf16, fp32).
//
// Masks are put into S as -inf, only in halves that some row does not see whole. Arithmetic
// is that of mx_attn.hip.
#include <type_traits>

#include "mx_attn.hpp"

namespace nvfp4 {

namespace {

constexpr int kTile = 64;  // tokens per step
constexpr int kWaves = 4, kRows = 32 * kWaves;

// A raise is due when the weights of a lane's 16 tokens add up to more: some weight is then
// above 2^8, and none that passes is above 2^12.
constexpr float kMostSum = 4096.0f;

// K rows are padded by 16 bytes; in V rows (64 tokens, 128 bytes) the 16-byte pieces are
// permuted by element. Either way the 16 rows that a phase of a 16-byte read meets lie in
// different banks (16 in order, or the rows whose bits 2, 3 and 4 have an even sum), and of V
// so do those that 32 lanes write, 4 or 16 elements apart.
__device__ __forceinline__ int v_chunk(int e, int c) { return c ^ (((e >> 1) ^ (e >> 4) ^ (e >> 7)) & 7); }

template <int D>
struct Lds {
  static constexpr int KRow = D * 2 + 16;
  static constexpr int K = kTile * KRow, V = D * kTile * 2;   // bytes of a tile
  static constexpr int Nan = D / 32 * kTile;                  // V bytes that are NaN, [block][token]
  static constexpr int VAt = 2 * K, NanAt = VAt + 2 * V, FlagAt = NanAt + 2 * Nan;
  static constexpr int RefAt = FlagAt + 2 * 4 * kWaves, Bytes = RefAt + 64 * kWaves * 4;  // reference scores, by lane
  static_assert(Bytes <= 160 * 1024, "LDS");
};

constexpr int waves_per_simd(int d) { return d == 64 ? 3 : d == 128 ? 2 : 1; }  // by registers

template <int D>
__global__ __launch_bounds__(64 * kWaves, waves_per_simd(D)) void mx_attention_prompt_kernel(MxAttnArgs a) {
  using L = Lds<D>;
  constexpr int KS = D / 16, DB = D / 32;
  extern __shared__ __align__(16) uint8_t smem[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 31, h = lane >> 5;
  const int kvh = blockIdx.x % a.c.kv_heads;
  const int split = blockIdx.y;
  const int g = a.group;
  // within a causal sequence the last tiles see the most tokens: they are started first
  const MxRows rows = mx_rows(a, (gridDim.x - 1 - blockIdx.x) / a.c.kv_heads, kRows);
  if (rows.first >= rows.count || rows.count <= a.skip) return;  // the whole workgroup
  const int wg_end = rows.first + kRows < rows.count ? rows.first + kRows : rows.count;
  const MxSight all = mx_sight(a, rows, rows.first, wg_end);
  const MxSpan span = mx_span(all, kTile);
  const int begin = mx_share(span.count, split, a.splits), end = mx_share(span.count, split + 1, a.splits);

  // ---- the wave's rows ----
  const int p0 = rows.first + wave * 32;
  const int p1 = p0 + 32 < rows.count ? p0 + 32 : rows.count;
  MxSight sight{0, 0, 0, 0, 0};  // a wave without rows sees nothing
  if (p0 < p1) sight = mx_sight(a, rows, p0, p1);
  if (p1 - p0 < 32) sight.high_min = 0;
  const int pn = p0 + n;
  const bool real = pn < rows.count;
  bf16x8_t q[KS];
  {
    const uint16_t* src = a.q + (rows.r0 + pn / g) * a.q_token + (int64_t)(kvh * g + pn % g) * a.q_head + 8 * h;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4_t w = {0u, 0u, 0u, 0u};
      if (real) w = *(const u32x4_t*)(src + 16 * s);
      q[s] = as_bf16x8(w[0], w[1], w[2], w[3]);
    }
  }
  const int high = real ? mx_high(a, rows.kv_len, rows.back + pn / g) : 0;
  const int low = mx_low(a, rows.back + pn / g);

  // ---- a tile's way into LDS: wave w brings tokens 16 w .. + 15 ----
  // K: four lanes to a token, D / 4 elements each; V: D / 16 elements of four tokens
  constexpr int KE = D / 4, VE = D / 16;  // elements of a lane
  const int kt = lane >> 2, k0 = (lane & 3) * KE;
  const int vq = (lane >> 4 & 1) * 2 + (lane >> 5), v0 = (lane & 15) * VE;
  const int vblk = v0 / 32;
  struct Raw {
    Words<KE / 8> k;
    uint32_t ks[KE > 32 ? 2 : 1];
    uint32_t v[4][VE > 8 ? 2 : 1];
    uint32_t vs[4];
  };
  // The block table, 64 entries at a time, one a lane. Of a tile: the cache row of the wave's
  // 16 tokens (on page 0 if their page is not there) and which of the four 16-token groups
  // have a page.
  struct Pages {
    int64_t row;
    uint32_t there;
  };
  const int32_t* table = a.b.block_table + (int64_t)rows.seq * a.b.table_stride;
  const int pages = (rows.kv_len + (1 << a.b.page_shift) - 1) >> a.b.page_shift;
  int entry = 0, base = -64;
  bool holes = false;  // among the 64
  auto pages_of = [&](int tile) __attribute__((always_inline)) {
    const int t = tile * kTile, first = t >> a.b.page_shift, last = (t + 48) >> a.b.page_shift;
    if ((first < base) | (last >= base + 64)) {  // uniform
      base = first;
      entry = first + lane < pages ? table[first + lane] : 0;  // past the last page: never seen
      if (entry >= a.b.num_pages) entry = -1;
      holes = __any(entry < 0);
    }
    Pages x;
    x.there = 15u;
    if (holes) {
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (__builtin_amdgcn_readlane(entry, ((t + 16 * w) >> a.b.page_shift) - base) < 0) x.there &= ~(1u << w);
    }
    x.row = mx_cache_row(a, __builtin_amdgcn_readlane(entry, ((t + 16 * wave) >> a.b.page_shift) - base), kvh,
                         t + 16 * wave);
    return x;
  };
  auto load_k = [&](Raw& x, const Pages& pg) __attribute__((always_inline)) {
    x.k = load_words<KE / 8>(a.c.k_codes + pg.row * (D / 2) + (kt * (D / 2) + k0 / 2));
    const uint8_t* s = a.c.k_scales + pg.row * (D / 32) + (kt * (D / 32) + k0 / 32);
#pragma unroll
    for (int b = 0; b < (KE > 32 ? 2 : 1); ++b) x.ks[b] = s[b];
  };
  auto load_v = [&](Raw& x, const Pages& pg) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* p = a.c.v_codes + pg.row * (D / 2) + ((4 * vq + i) * (D / 2) + v0 / 2);
      if constexpr (VE == 4) x.v[i][0] = *(const uint16_t*)p;
      else {
        const Words<VE / 8> w = load_words<VE / 8>(p);
#pragma unroll
        for (int j = 0; j < VE / 8; ++j) x.v[i][j] = w.w[j];
      }
      x.vs[i] = (a.c.v_scales + pg.row * (D / 32))[(4 * vq + i) * (D / 32) + vblk];
    }
  };
  auto store_k = [&](const Raw& x, int buf, int e) __attribute__((always_inline)) {  // piece e of KE / 8
    uint8_t* dst = smem + buf * L::K + (wave * 16 + kt) * L::KRow + k0 * 2;
    *(u32x4_t*)(dst + e * 16) = mx_decode8(x.k.w[e], __uint_as_float(x.ks[KE > 32 ? e >> 2 : 0] << 23));
  };
  // V by element. The products must not meet a NaN: 0 * NaN would reach rows that do not
  // see it. NaN blocks go in as zeros (scale 0) and are marked; tokens past the last and on
  // pages that are not there may hold anything and go in under scale 0 too.
  auto mark_v = [&](Raw& x, int buf, int tile, const Pages& pg) __attribute__((always_inline)) {
    const int t0 = tile * kTile + wave * 16;
    if ((t0 + 16 > rows.kv_len) | ((pg.there >> wave & 1u) == 0)) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x.vs[i] = ((t0 + 4 * vq + i < rows.kv_len) & ((pg.there >> wave & 1u) != 0)) ? x.vs[i] : 0u;
    }
    const uint32_t most = max(max(x.vs[0], x.vs[1]), max(x.vs[2], x.vs[3]));
    const uint32_t any = __any(most == 255u);
    if (any) {
      uint32_t marks = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        marks |= x.vs[i] == 255u ? 1u << (8 * i) : 0u;
        x.vs[i] = x.vs[i] == 255u ? 0u : x.vs[i];
      }
      *(uint32_t*)(smem + L::NanAt + buf * L::Nan + vblk * kTile + wave * 16 + 4 * vq) = marks;  // the same from a block's lanes
    }
    *(uint32_t*)(smem + L::FlagAt + (buf * 4 + wave) * 4) = any;
  };
  auto store_v = [&](const Raw& x, int buf, int d) __attribute__((always_inline)) {  // elements 2 d, 2 d + 1 of the lane's
    // tokens 4 vq .. + 3 of the 16: lane half vq & 1, first or second four
    uint8_t* dst = smem + L::VAt + buf * L::V + (vq >> 1) * 8;
    const int c = 2 * wave + (vq & 1), e = v0 + 2 * d;
    uint32_t two[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) two[i] = decode2(x.v[i][VE > 8 ? d >> 2 : 0], __uint_as_float(x.vs[i] << 23), d & 3);
    *(u32x2_t*)(dst + e * 128 + v_chunk(e, c) * 16) =
        u32x2_t{__builtin_amdgcn_perm(two[1], two[0], 0x05040100u), __builtin_amdgcn_perm(two[3], two[2], 0x05040100u)};
    *(u32x2_t*)(dst + (e + 1) * 128 + v_chunk(e + 1, c) * 16) =
        u32x2_t{__builtin_amdgcn_perm(two[1], two[0], 0x07060302u), __builtin_amdgcn_perm(two[3], two[2], 0x07060302u)};
  };

  // ---- state ----
  f32x16_t o[DB];
  f32x16_t s0, s1;  // scores of a tile's halves
  float neg = 0.0f, l = 0.0f;  // the unit of the reference score, the sum of the lane's tokens
  // the score itself is needed when it is raised, and waits in LDS (in a register instead of neg,
  // its unit taken in every half: D = 64 spills, 100 us for 91)
  float* const ref = (float*)(smem + L::RefAt) + (wave * 64 + h * 32 + n);
  *ref = -INFINITY;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  bool wary = true;  // some row has seen nothing yet, or its reference is far

  bf16x8_t kf[KS], vf[KS];  // fragments of a half: K by step, V by (16 tokens, block)
  auto read_k = [&](int buf, int half, int k) __attribute__((always_inline)) {
    kf[k] = *(const bf16x8_t*)(smem + buf * L::K + (half * 32 + n) * L::KRow + h * 16 + k * 32);
  };
  auto read_v = [&](int buf, int half, int k) __attribute__((always_inline)) {
    const int e = k % DB * 32 + n;
    vf[k] = *(const bf16x8_t*)(smem + L::VAt + buf * L::V + e * 128 + v_chunk(e, 4 * half + 2 * (k / DB) + h) * 16);
  };
  auto zero = [&](f32x16_t& x) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.0f;
  };
  auto scores = [&](f32x16_t& x, int k) __attribute__((always_inline)) {  // step k
    x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[k], q[k], x, 0, 0, 0);
  };
  // (no short-circuits: selects, not branches around the accumulators)
  auto sees = [&](int t, uint32_t there, int group) __attribute__((always_inline)) {
    return (t < high) & ((t >= low) | (t < sight.sinks)) & ((there >> group & 1u) != 0);
  };
  // register i of a half is its token 8 (i / 4) + 4 h + i % 4
  auto mask = [&](f32x16_t& x, int tile, int half, uint32_t there) __attribute__((always_inline)) {
    const int t0 = tile * kTile + half * 32;
    if ((there >> (2 * half) & 3u) == 3u && t0 + 32 <= sight.high_min &&
        (t0 >= sight.low_max || t0 + 32 <= sight.sinks))
      return;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      x[i] = sees(t0 + 8 * (i >> 2) + 4 * h + (i & 3), there, 2 * half + (i >> 3)) ? x[i] : -INFINITY;
  };
  uint32_t pw[8];  // the weights, packed
  float sum;       // of the lane's 16
  // weights 4 j .. 4 j + 3: taken (the exponentials), then summed and packed
  auto take = [&](const f32x16_t& x, int j, float (&p)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[4 * j + i], a.scale_log2, neg));
  };
  auto add = [&](int j, const float (&p)[4]) __attribute__((always_inline)) {
    const uint32_t w0 = pack_bf16(p[0], p[1]), w1 = pack_bf16(p[2], p[3]);
    const bf16x2_t one = as_bf16x2(0x3F803F80u);
    const float t = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(w0), one, j == 0 ? 0.0f : sum, false);
    sum = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(w1), one, t, false);
    pw[2 * j] = w0;
    pw[2 * j + 1] = w1;
  };
  // after the weights of x: raises the maximum and takes them again if that is due
  bf16x8_t pf[2];
  auto settle = [&](f32x16_t& x) __attribute__((always_inline)) {
    if (__any(wary | !(sum <= kMostSum))) {
      float top = x[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
      const float m = *ref, next = fmaxf(m, fmaxf(top, __shfl_xor(top, 32, 64)));
      const float f = mx_rebase(a, m, next);  // m = -inf: o and l are 0
      *ref = next;
      const MxUnit unit = mx_unit(a, next);
      neg = unit.neg;
      wary = __any(((next == -INFINITY) & (high > 0)) | unit.far);
      x -= unit.base;  // 0 unless far, when every half comes here
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float p[4];
        take(x, j, p);
        add(j, p);
      }
    }
    l += sum;
#pragma unroll
    for (int k = 0; k < 2; ++k) pf[k] = as_bf16x8(pw[4 * k], pw[4 * k + 1], pw[4 * k + 2], pw[4 * k + 3]);
  };
  auto values = [&](int k) __attribute__((always_inline)) {  // 16 tokens k / DB, block k % DB
    o[k % DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[k], pf[k / DB], o[k % DB], 0, 0, 0);
  };
  // The phases, in steps of a matrix instruction each with its share of the rest, fenced so
  // that the order stands: left alone the instructions gather by kind, and one wave a SIMD
  // then does first the one and then the other (D = 256: 196 us for 188).
  auto fence = []() __attribute__((always_inline)) { __builtin_amdgcn_sched_barrier(0); };
  auto phase_scores = [&](f32x16_t& x, const f32x16_t& y, int vbuf, int half) __attribute__((always_inline)) {
    constexpr int G = 4;  // groups of weights, over KS steps; packed a step after they are taken
    float p[2][4];
    zero(x);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      scores(x, k);
      read_v(vbuf, half, k);
#pragma unroll
      for (int j = k * G / KS; j < (k + 1) * G / KS; ++j) {
        if (j > 0) add(j - 1, p[(j - 1) & 1]);
        take(y, j, p[j & 1]);
      }
      fence();
    }
    add(G - 1, p[(G - 1) & 1]);
  };

  // Marked blocks: a product of "is NaN" with "is seen" tells the rows that get one, for the
  // whole block of 32 elements at once.
  u32x4_t flag;  // of V[t], one word for 16 tokens
  auto read_flag = [&](int buf) __attribute__((always_inline)) {
    flag = *(const u32x4_t*)(smem + L::FlagAt + buf * 16);
  };
  auto nans = [&](int buf, int tile, uint32_t there) __attribute__((always_inline)) {
    if (__builtin_amdgcn_readfirstlane(flag[0] | flag[1] | flag[2] | flag[3]) == 0) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (__builtin_amdgcn_readfirstlane(flag[k]) == 0) continue;
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        bits |= sees(tile * kTile + 16 * k + 8 * (i >> 2) + 4 * h + (i & 3), there, k) ? 1u << i : 0u;
      const bf16x8_t seen = mx_ones(bits);
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        bits = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          bits |= smem[L::NanAt + buf * L::Nan + d * kTile + 16 * k + 8 * (i >> 2) + 4 * h + (i & 3)] ? 1u << i : 0u;
        f32x16_t hit;
#pragma unroll
        for (int i = 0; i < 16; ++i) hit[i] = 0.0f;
        hit = __builtin_amdgcn_mfma_f32_32x32x16_bf16(mx_ones(bits), seen, hit, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = hit[i] > 0.0f ? NAN : o[d][i];
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
    int tile = span.at(begin), next = clamp(begin + 1), far = clamp(begin + 2);
    Pages at = pages_of(tile), an = pages_of(next), af = pages_of(far);  // of the three tiles
    load_k(x, at);
    load_v(x, at);
#pragma unroll
    for (int d = 0; d < KE / 8; ++d) store_k(x, 0, d);
    mark_v(x, 0, tile, at);
#pragma unroll
    for (int d = 0; d < VE / 2; ++d) store_v(x, 0, d);
    load_k(x, an);
#pragma unroll
    for (int d = 0; d < KE / 8; ++d) store_k(x, 1, d);
    load_v(x, an);
    load_k(x, af);
    barrier();
    zero(s0);
#pragma unroll
    for (int k = 0; k < KS; ++k) read_k(0, 0, k);
#pragma unroll
    for (int k = 0; k < KS; ++k) scores(s0, k);
    mask(s0, tile, 0, at.there);
#pragma unroll
    for (int k = 0; k < KS; ++k) read_k(0, 1, k);
    read_flag(0);
    auto body = [&](int i, auto buffer) __attribute__((always_inline)) {
      constexpr int buf = decltype(buffer)::value;
      nans(buf, tile, at.there);
      const int beyond = clamp(i + 3);
      const Pages ab = pages_of(beyond);
      // 1
      fence();
      phase_scores(s1, s0, buf, 0);
      settle(s0);
      mask(s1, tile, 1, at.there);
      // 2
      fence();
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        values(k);
        read_k(buf ^ 1, 0, k);
        if (k == 0) mark_v(x, buf ^ 1, next, an);
        if ((k & 1) && (k >> 1) < VE / 2) store_v(x, buf ^ 1, k >> 1);
        fence();
      }
      load_v(x, af);
      barrier();
      // 3
      read_flag(buf ^ 1);
      fence();
      phase_scores(s0, s1, buf, 1);
      settle(s1);
      mask(s0, next, 0, an.there);
      // 4
      fence();
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        values(k);
        read_k(buf ^ 1, 1, k);
        if ((k & 1) && (k >> 1) < KE / 8) store_k(x, buf, k >> 1);
        fence();
      }
      load_k(x, ab);
      barrier();
      tile = next;
      next = far;
      far = beyond;
      at = an;
      an = af;
      af = ab;
    };
    for (int i = begin; i < end; i += 2) {
      body(i, std::integral_constant<int, 0>());
      if (i + 1 < end) body(i + 1, std::integral_constant<int, 1>());
    }
  }

  // ---- the rows' results: lane (n, h) has elements 32 d + 8 k + 4 h .. + 3 of row n ----
  const float all_sum = l + __shfl_xor(l, 32, 64);
  if (!real) return;
  const int64_t token = rows.r0 + pn / g;
  const int head = kvh * g + pn % g;
  if (a.splits > 1) {
    const int64_t at = ((int64_t)split * a.b.tokens + token) * a.heads + head;
    if (h == 0) a.part_ml[at] = make_float2(*ref, all_sum);
    if (all_sum != 0.0f) {
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *(f32x4_t*)(a.part_o + at * D + 32 * d + 8 * k + 4 * h) =
              f32x4_t{o[d][4 * k], o[d][4 * k + 1], o[d][4 * k + 2], o[d][4 * k + 3]};
    }
  } else {
    const float inv = all_sum == 0.0f ? 0.0f : 1.0f / all_sum;
    uint16_t* dst = a.out + token * a.out_token + (int64_t)head * a.out_head;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *(u32x2_t*)(dst + 32 * d + 8 * k + 4 * h) =
            u32x2_t{pack_bf16(o[d][4 * k] * inv, o[d][4 * k + 1] * inv),
                    pack_bf16(o[d][4 * k + 2] * inv, o[d][4 * k + 3] * inv)};
  }
}

template <int D>
hipError_t launch_prompt(const MxAttnArgs& a, hipStream_t stream) {
  const int64_t tiles = a.b.tokens * a.group / kRows + a.b.batch;
  mx_attention_prompt_kernel<D>
      <<<dim3((unsigned)(tiles * a.c.kv_heads), a.splits), 64 * kWaves, Lds<D>::Bytes, stream>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t setup_prompt() {
  return hipFuncSetAttribute((const void*)mx_attention_prompt_kernel<D>, hipFuncAttributeMaxDynamicSharedMemorySize,
                             Lds<D>::Bytes);
}

}  // namespace

hipError_t mx_attention_prompt_setup() {
  hipError_t e = setup_prompt<64>();
  if (e == hipSuccess) e = setup_prompt<128>();
  if (e == hipSuccess) e = setup_prompt<256>();
  return e;
}

hipError_t launch_mx_attention_prompt(const MxAttnArgs& a, hipStream_t stream) {
  switch (a.c.head_dim) {
    case 64: return launch_prompt<64>(a, stream);
    case 128: return launch_prompt<128>(a, stream);
    default: return launch_prompt<256>(a, stream);
  }
}

}  // namespace nvfp4
