// mx_attn.hip - attention over a paged MXFP4 cache, for few rows of a sequence (gfx950):
// single tokens of a decoding batch, a few drafted ones. Many rows: mx_attn_prompt.hip.
//
//   o[i, h] = sum_t softmax_t(scale * q[i, h] . k[t, h / g]) v[t, h / g]
//
// over the tokens t that row i of its sequence sees. The (row, head of the group) pairs of a
// sequence and kv head are packed into one axis, so a single token of a grouped model fills
// a 16-wide matrix tile. A workgroup has RT tiles of 16 packed rows; its four waves split
// the tokens and join at the end, and the token axis is split further over workgroups where
// the batch alone does not fill the device.
//
// What bounds it is reading the cache: every visible token once per kv head, 17/32 bytes an
// element. A wave moves its codes and scales to a ring of its own in LDS, 32 tokens a slot,
// with direct-to-LDS loads that need no register while they fly and no barrier (six
// instructions for 32 tokens of 128 elements, every one of whole runs): 16 waves x 2 slots
// x 4.25 KiB in flight per CU. 48 single tokens over up to 8200, 56 heads of 128 over 8: 77
// us and 5 of joining, 4.2 TB/s of the cache; the loads alone take 63, the rest alone 69.
//
// One pass with the running maximum and sum of the softmax, in the transposed form with
// v_mfma_f32_16x16x32_bf16, lane (n, u) = (lane & 15, lane >> 4):
//
//   S^T = K Q^T    A: lane (n, u) holds token n, elements [u D/4, (u + 1) D/4) - the
//                  contraction order is free, so a lane takes D/8 bytes of codes in one run
//                  under at most two scales. S^T comes out with lane (n, u) holding packed
//                  row n, tokens 4u .. 4u + 3.
//   O^T = V^T P^T  B: P as S^T left it, without a move: lane (n, u) has tokens 4u .. 4u + 3
//                  of both 16-token halves, its 8 of the 32. A: lane (c, u) takes the same
//                  8 tokens, elements [c D/16, (c + 1) D/16): whole bytes of each token's
//                  codes, decoded in pairs along the head and paired along the tokens by
//                  byte permutes.
//
// Packed row n stays in the lanes n + 16 u from the scores to the output, and lane (n, u)
// ends with elements [u D/4, (u + 1) D/4) of its row. Codes become exact bf16
// (v_cvt_scalef32_pk_bf16_fp4); scores, maxima, sums and o are fp32. P is rounded to bf16
// for the product (2^-8 of each weight at most, the size of o's own rounding); its sum is of
// the same rounded weights, so that they still add up to one.
//
// The maximum is raised only when a weight under it would exceed 2^8: until then weights up to
// 2^8 are as exact as those below 1, and most tiles skip the cross-lane maximum and the
// rescaling of O.
#include <type_traits>

#include "mx_attn.hpp"

namespace nvfp4 {

namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;  // tokens per step

typedef __attribute__((address_space(3))) void lds_ptr_t;

// A ring slot: K codes, V codes, K scales, V scales of 32 tokens, in the cache's order.
template <int D>
struct Slot {
  static constexpr int Codes = kTile * D / 2, Half = Codes / 2;   // bytes; Half: of 16 tokens
  static constexpr int Scales = kTile * D / 32, SHalf = Scales / 2;
  static constexpr int V = Codes, KS = 2 * Codes, VS = KS + Scales, Bytes = VS + Scales;
  // instructions for a run of tokens: 16 bytes a lane of codes, 4 of scales
  static constexpr int loads(int tokens) { return 2 * ((tokens * D / 2 + 1023) / 1024 + (tokens * D / 32 + 255) / 256); }
};

// Workgroups of a CU, by registers, and the ring slots of a wave that then fit. Measured on 48
// single tokens over up to 8200 of 128: four workgroups with 2 slots 85 us, three with 2 the
// same, three with 3 slots 91 - more waves hide more than more slots.
constexpr int groups_per_cu(int d, int rt) { return d == 256 ? 2 : rt == 1 ? 4 : 3; }
constexpr int ring_slots(int d) { return d == 64 ? 4 : 2; }

// LDS of a workgroup: the rings, where the waves' outputs meet afterwards, and their references,
// sums, and exponents of the references' own weights. (Dynamic: of static LDS the compiler knows
// which object a load into it writes, and waits for all loads in flight before any read of that
// object.)
template <int D, int RT>
struct FewLds {
  static constexpr int Rings = kWaves * ring_slots(D) * Slot<D>::Bytes, Red = kWaves * (D / 4) * 64 * 4;
  static constexpr int Ring = Rings > Red ? Rings : Red, Bytes = Ring + 3 * kWaves * RT * 16 * 4;
};

template <int N>
__device__ __forceinline__ void wait_loads() {  // vmcnt(N)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}

template <int D, int RT>
__global__ __launch_bounds__(64 * kWaves, groups_per_cu(D, RT)) void mx_attention_few_kernel(MxAttnArgs a) {
  using S = Slot<D>;
  constexpr int NJ = D / 16, KS = D / 32, E = D / 4, R = ring_slots(D);
  constexpr int kRows = 16 * RT;  // packed rows of the workgroup
  extern __shared__ __align__(16) uint8_t smem[];
  float* const ml = (float*)(smem + FewLds<D, RT>::Ring);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, u = lane >> 4;
  const int kvh = blockIdx.x % a.c.kv_heads;
  const int split = blockIdx.y;
  const int g = a.group;
  // the longest contexts are not known here; the last tiles come first, as in the prompt form
  const int tile = (gridDim.x - 1 - blockIdx.x) / a.c.kv_heads;
  const MxRows rows = a.by_seq ? mx_rows_of(a, tile) : mx_rows(a, tile, kRows);
  const int p0 = rows.first;
  if (p0 >= rows.count || (a.by_seq && rows.count > kRows)) return;  // the whole workgroup
  const int p1 = p0 + kRows < rows.count ? p0 + kRows : rows.count;

  // ---- the rows ----
  bf16x8_t q[RT][KS];
  int high[RT], low[RT];  // visible: [low, high) and t < sinks
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int p = p0 + r * 16 + n;
    const bool real = p < rows.count;
    const int i = p / g;
    const uint16_t* src = a.q + (rows.r0 + i) * a.q_token + (int64_t)(kvh * g + p % g) * a.q_head + u * E;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4_t w = {0u, 0u, 0u, 0u};
      if (real) w = *(const u32x4_t*)(src + 8 * s);
      q[r][s] = as_bf16x8(w[0], w[1], w[2], w[3]);
    }
    high[r] = real ? mx_high(a, rows.kv_len, rows.back + i) : 0;
    low[r] = mx_low(a, rows.back + i);
  }
  const MxSight sight = mx_sight(a, rows, p0, p1);
  const int high_min = p1 - p0 < kRows ? 0 : sight.high_min;  // rows that are not there see nothing
  const MxSpan span = mx_span(sight, kTile);
  const int from = mx_share(span.count, split, a.splits), to = mx_share(span.count, split + 1, a.splits);
  const int begin = from + (to - from) * wave / kWaves, end = from + (to - from) * (wave + 1) / kWaves;

  // ---- loads ----
  // 64 entries of the block table at a time, one a lane
  const int32_t* table = a.b.block_table + (int64_t)rows.seq * a.b.table_stride;
  const int pages = (rows.kv_len + (1 << a.b.page_shift) - 1) >> a.b.page_shift;
  int entry = -1, held = -64;
  auto page_of = [&](int t) __attribute__((always_inline)) -> int {
    const int p = t >> a.b.page_shift;
    if (p < held || p >= held + 64) {  // uniform
      held = p;
      entry = p + lane < pages ? table[p + lane] : -1;
      if (entry >= a.b.num_pages) entry = -1;
    }
    return __builtin_amdgcn_readlane(entry, p - held);
  };
  uint8_t* const ring = smem + wave * (R * S::Bytes);
  const bool halves = a.b.page_shift == 4;  // else the halves of a tile share a page
  uint32_t there_bits = 0;  // bits 2 slot, 2 slot + 1: the page of each 16-token half exists
  auto load = [&](int slot, int tile) __attribute__((always_inline)) {
    const int t0 = tile * kTile;
    int64_t row[2];
    int page = page_of(t0);  // of a token that some row sees
    uint32_t there = page >= 0 ? 3u : 0u;
    row[0] = mx_cache_row(a, page, kvh, t0);
    row[1] = row[0] + 16;
    if (halves) {
      page = t0 + 16 < rows.kv_len ? page_of(t0 + 16) : -1;
      there = (there & 1u) | (page >= 0 ? 2u : 0u);
      row[1] = mx_cache_row(a, page, kvh, t0 + 16);
    }
    there_bits = (there_bits & ~(3u << (2 * slot))) | (there << (2 * slot));
    uint8_t* dst = ring + slot * S::Bytes;
    // (buffer loads: behind global loads into LDS the compiler would wait for all of them
    // at each of the step's reads)
    auto move_all = [&](int64_t row, int token, auto tokens) __attribute__((always_inline)) {
      constexpr int kCodes = decltype(tokens)::value * D / 2, kScales = decltype(tokens)::value * D / 32;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const __amdgpu_buffer_rsrc_t from = __builtin_amdgcn_make_buffer_rsrc(
            (kv ? a.c.v_codes : a.c.k_codes) + row * (D / 2), 0, kCodes, 0x00020000);
        uint8_t* to = dst + (kv ? S::V : 0) + token * (D / 2);
#pragma unroll
        for (int at = 0; at < kCodes; at += 1024)
          if (kCodes - at >= 1024 || lane * 16 < kCodes - at)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr_t*)(to + at), 16, at + lane * 16, 0, 0, 0);
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const __amdgpu_buffer_rsrc_t from = __builtin_amdgcn_make_buffer_rsrc(
            (kv ? a.c.v_scales : a.c.k_scales) + row * (D / 32), 0, kScales, 0x00020000);
        if (lane * 4 < kScales)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr_t*)(dst + (kv ? S::VS : S::KS) + token * (D / 32)), 4,
                                                   lane * 4, 0, 0, 0);
      }
    };
    if (halves) {
      move_all(row[0], 0, std::integral_constant<int, 16>());
      move_all(row[1], 16, std::integral_constant<int, 16>());
    } else {
      move_all(row[0], 0, std::integral_constant<int, kTile>());
    }
  };

  // ---- state ----
  f32x4_t o[RT][NJ];
  float m[RT], l[RT];       // m: the reference score, agreed by the four lanes of a row; l: the lane's own tokens
  float base[RT], neg[RT];  // its unit
  float most[RT];           // the score up to which it stays
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = most[r] = -INFINITY;
    l[r] = base[r] = neg[r] = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) o[r][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const int vblk = n * (D / 16) / 32;  // the block of the lane's V elements

  auto step = [&](int slot, int tile) __attribute__((always_inline)) {
    const int t0 = tile * kTile;
    const uint8_t* x = ring + slot * S::Bytes;
    const uint32_t there = there_bits >> (2 * slot) & 3u;
    f32x4_t s[RT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const Words<D / 32> kc = load_words<D / 32>(x + h * S::Half + n * (D / 2) + u * (D / 8));
      float ks[D == 256 ? 2 : 1];
#pragma unroll
      for (int b = 0; b < (D == 256 ? 2 : 1); ++b)
        ks[b] = __uint_as_float((uint32_t)x[S::KS + h * S::SHalf + n * (D / 32) + u * (D / 4) / 32 + b] << 23);
#pragma unroll
      for (int r = 0; r < RT; ++r) s[r][h] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < KS; ++e) {
        const u32x4_t w = mx_decode8(kc.w[e], ks[D == 256 ? e >> 2 : 0]);
        const bf16x8_t kf = as_bf16x8(w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int r = 0; r < RT; ++r) s[r][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[r][e], s[r][h], 0, 0, 0);
      }
    }
    const bool full = there == 3u && t0 + kTile <= high_min && (t0 >= sight.low_max || t0 + kTile <= sight.sinks);
    auto sees = [&](int r, int j) __attribute__((always_inline)) {
      const int t = t0 + 16 * (j >> 2) + 4 * u + (j & 3);
      return (t < high[r]) & ((t >= low[r]) | (t < sight.sinks)) & ((there >> (j >> 2) & 1u) != 0);
    };
    if (!full) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          s[r][j >> 2][j & 3] = sees(r, j) ? s[r][j >> 2][j & 3] : -INFINITY;
    }
    bf16x8_t pf[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float top = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                        fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3])));
      if (__any(top > most[r])) {
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float next = fmaxf(m[r], top);
        const MxUnit unit = mx_unit(a, next);
        // mx_rebase with the units at hand, without a branch; m = -inf: o and l are 0
        const float e = mx_exponent(a, m[r], unit.base, unit.neg) - mx_exponent(a, m[r], base[r], neg[r]);
        const float f = m[r] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(e);
        m[r] = next;
        base[r] = unit.base;
        neg[r] = unit.neg;
        most[r] = next + a.raise;
        l[r] *= f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) o[r][j] *= f;
      }
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        p[j] = __builtin_amdgcn_exp2f(mx_exponent(a, s[r][j >> 2][j & 3], base[r], neg[r]));
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = pack_bf16(p[2 * j], p[2 * j + 1]);
        l[r] = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(w[j]), as_bf16x2(0x3F803F80u), l[r], false);
      }
      pf[r] = as_bf16x8(w[0], w[1], w[2], w[3]);
    }
    uint32_t vc[8][D == 256 ? 2 : 1];
    float vs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int t = 4 * u + (j & 3);
      const uint8_t* p = x + S::V + (j >> 2) * S::Half + t * (D / 2) + n * (D / 32);
      if constexpr (D == 64) vc[j][0] = *(const uint16_t*)p;
      else {
        const Words<D / 128> w = load_words<D / 128>(p);
#pragma unroll
        for (int k = 0; k < D / 128; ++k) vc[j][k] = w.w[k];
      }
      vs[j] = __uint_as_float((uint32_t)x[S::VS + (j >> 2) * S::SHalf + t * (D / 32) + vblk] << 23);
    }
    // 0 * NaN is NaN, and a row must not meet a NaN that it does not see (another row's
    // token, or what lies behind the last one): where not all rows see all, NaN blocks leave
    // the product (their scale becomes 0), and a second product of "is NaN" with "is seen"
    // tells the rows that get one. The lane's elements all lie in one block, so its answer
    // holds for all of them.
    // Tokens that no row sees may hold anything, infinite values too: their scale becomes 0.
    uint32_t nans = 0;  // bit j: the lane's block of its token j is NaN
    if (!full) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool none = (t0 + 16 * (j >> 2) + 4 * u + (j & 3) >= sight.high_max) | ((there >> (j >> 2) & 1u) == 0);
        vs[j] = none ? 0.0f : vs[j];
        nans |= __float_as_uint(vs[j]) == 255u << 23 ? 1u << j : 0u;
      }
    }
    if (!full && __any(nans != 0)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) vs[j] = (nans >> j & 1) ? 0.0f : vs[j];
      const bf16x8_t is_nan = mx_ones(nans);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        uint32_t seen = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) seen |= sees(r, j) ? 1u << j : 0u;
        const f32x4_t hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(is_nan, mx_ones(seen),
                                                                    f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j) o[r][j][i] = hit[i] > 0.0f ? NAN : o[r][j][i];
      }
    }
#pragma unroll
    for (int d = 0; d < NJ / 2; ++d) {
      uint32_t two[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) two[j] = decode2(vc[j][D == 256 ? d >> 2 : 0], vs[j], d & 3);
      uint32_t ev[4], od[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        ev[w] = __builtin_amdgcn_perm(two[2 * w + 1], two[2 * w], 0x05040100u);
        od[w] = __builtin_amdgcn_perm(two[2 * w + 1], two[2 * w], 0x07060302u);
      }
      const bf16x8_t ve = as_bf16x8(ev[0], ev[1], ev[2], ev[3]), vo = as_bf16x8(od[0], od[1], od[2], od[3]);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        o[r][2 * d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ve, pf[r], o[r][2 * d], 0, 0, 0);
        o[r][2 * d + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vo, pf[r], o[r][2 * d + 1], 0, 0, 0);
      }
    }
  };

  // ---- the walk ----
  static_assert((R - 1) * 2 * S::loads(16) <= 63, "vmcnt");
  // Slots are filled R tiles ahead; past the end the last tile is loaded again, so that the
  // count of loads in flight stays what the waits assume. A slot is refilled once its reads
  // have returned (lgkmcnt(0)).
  if (begin < end) {
    page_of(span.at(begin) * kTile);
    wait_loads<0>();  // the rows are here: no step waits for them, and with them for the ring
#pragma unroll
    for (int i = 0; i < R; ++i) load(i, span.at(begin + i < end ? begin + i : end - 1));
    int slot = 0;
    for (int i = begin; i < end; ++i) {
      if (halves) wait_loads<(R - 1) * S::loads(16) * 2>();
      else wait_loads<(R - 1) * S::loads(32)>();
      step(slot, span.at(i));
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xC07F);
      asm volatile("" ::: "memory");
      load(slot, span.at(i + R < end ? i + R : end - 1));
      slot = slot + 1 == R ? 0 : slot + 1;
    }
    wait_loads<0>();  // before the ring's memory is used again
  }

  // ---- join the waves, 16 rows at a time: wave w adds up and stores elements
  // [(4u + w) D/16, + D/16) of each row ----
  float* red = (float*)smem;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    l[r] += __shfl_xor(l[r], 16, 64);
    l[r] += __shfl_xor(l[r], 32, 64);
    if (u == 0) {
      ml[(wave * RT + r) * 16 + n] = m[r];
      ml[(kWaves * RT + wave * RT + r) * 16 + n] = l[r];
      ml[(2 * kWaves * RT + wave * RT + r) * 16 + n] =
          m[r] == -INFINITY ? 0.0f : mx_exponent(a, m[r], base[r], neg[r]);  // 0: its f is 2^-inf
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    __syncthreads();  // every wave has left its ring, or the last round's reads
    float top = -INFINITY, sum = 0.0f, f[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ml[(w * RT + r) * 16 + n]);
    const MxUnit unit = mx_unit(a, top);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float mw = ml[(w * RT + r) * 16 + n];
      f[w] = __builtin_amdgcn_exp2f(mx_exponent(a, mw, unit.base, unit.neg) - ml[(2 * kWaves * RT + w * RT + r) * 16 + n]);
      sum += f[w] * ml[(kWaves * RT + w * RT + r) * 16 + n];
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[((wave * 4 + i) * NJ + j) * 64 + lane] = o[r][j][i];
    __syncthreads();
    float y[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      y[j] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) y[j] += f[w] * red[((w * 4 + wave) * NJ + j) * 64 + lane];
    }
    const int p = p0 + r * 16 + n;
    if (p >= rows.count) continue;
    const int64_t token = rows.r0 + p / g;
    const int head = kvh * g + p % g;
    const int e0 = (4 * u + wave) * NJ;
    if (a.splits > 1) {
      const int64_t at = a.by_seq ? (((int64_t)split * a.b.batch + rows.seq) * a.c.kv_heads + kvh) * 16 + n
                                  : ((int64_t)split * a.b.tokens + token) * a.heads + head;
      if (u == 0 && wave == 0) a.part_ml[at] = make_float2(top, sum);
      if (sum != 0.0f) {
#pragma unroll
        for (int j = 0; j < NJ; j += 4)
          *(f32x4_t*)(a.part_o + at * D + e0 + j) = f32x4_t{y[j], y[j + 1], y[j + 2], y[j + 3]};
      }
    } else {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      uint16_t* dst = a.out + token * a.out_token + (int64_t)head * a.out_head + e0;
      if constexpr (NJ == 4) {
        *(u32x2_t*)dst = u32x2_t{pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
      } else {
#pragma unroll
        for (int j = 0; j < NJ; j += 8)
          *(u32x4_t*)(dst + j) = u32x4_t{pack_bf16(y[j] * inv, y[j + 1] * inv), pack_bf16(y[j + 2] * inv, y[j + 3] * inv),
                                         pack_bf16(y[j + 4] * inv, y[j + 5] * inv),
                                         pack_bf16(y[j + 6] * inv, y[j + 7] * inv)};
      }
    }
  }
}

// Which row and head the pair of a join is; false if there is none, or it is not its own.
__device__ __forceinline__ bool pair_of(const MxAttnArgs& a, int64_t pair, int64_t& token, int& head) {
  if (a.by_seq) {
    const int place = (int)(pair / 16), n = (int)(pair % 16), seq = place / a.c.kv_heads;
    const MxRows rows = mx_rows_of(a, seq);
    if (n >= rows.count || rows.count > 16) return false;  // no such row, or not of this form
    token = rows.r0 + n / a.group;
    head = (place - seq * a.c.kv_heads) * a.group + n % a.group;
    return true;
  }
  token = pair / a.heads;
  head = (int)(pair - token * a.heads);
  return token >= mx_row_start(a.b, 0) && token < mx_row_start(a.b, a.b.batch);  // of no sequence: stays as it was
}

// Joins up to kJoinWave splits of each (row, head): a wave per pair. D/4 lanes take a split's
// row, four elements each, 256 / D splits at a time. 1,800 tokens, 24 heads of 64, attention
// in 2 pieces: 54 us, with a workgroup a pair 86.
constexpr int kJoinWave = 16;

template <int D>
__global__ __launch_bounds__(256) void mx_attention_join_few_kernel(MxAttnArgs a, int64_t pairs) {
  constexpr int L = D / 4, P = 64 / L;
  const int lane = threadIdx.x & 63;
  const int64_t pair = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t token;
  int head;
  if (pair >= pairs || !pair_of(a, pair, token, head)) return;
  float2 v = make_float2(-INFINITY, 0.0f);
  if (lane < a.splits) v = a.part_ml[lane * pairs + pair];
  if (v.y == 0.0f) v.x = -INFINITY;  // saw nothing; its o was not written
  float top = v.x;
#pragma unroll
  for (int off = kJoinWave / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  top = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(top)));
  const float f = v.y == 0.0f ? 0.0f : mx_rebase(a, v.x, top);
  float sum = v.y == 0.0f ? 0.0f : f * v.y;
#pragma unroll
  for (int off = kJoinWave / 2; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
  sum = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(sum)));
  const float weight = v.y == 0.0f ? -1.0f : f;
  // what a split that saw nothing left there is read and not used
  f32x4_t y = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* src = a.part_o + pair * D + (lane % L) * 4;
  for (int s0 = lane / L; s0 < kJoinWave; s0 += 4 * P) {
    if (s0 - lane / L >= a.splits) break;  // uniform
    f32x4_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int s = s0 + q * P;
      o[q] = *(const f32x4_t*)(src + (s < a.splits ? s : 0) * pairs * D);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float w = __shfl(weight, s0 + q * P, 64);  // -1 past the last
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] += w == -1.0f ? 0.0f : w * o[q][i];
    }
  }
#pragma unroll
  for (int off = L; off < 64; off <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] += __shfl_xor(y[i], off, 64);
  if (lane >= L) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  *(u32x2_t*)(a.out + token * a.out_token + (int64_t)head * a.out_head + lane * 4) =
      u32x2_t{pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
}

// The same for more splits: a workgroup per pair, 1024 / D splits at a time.
template <int D>
__global__ __launch_bounds__(256) void mx_attention_join_kernel(MxAttnArgs a) {
  constexpr int L = D / 4, P = 256 / L;
  __shared__ float weight[kMxMostSplits];
  __shared__ float red[4];
  __shared__ f32x4_t part[256];
  const int tid = threadIdx.x;
  const int64_t pair = blockIdx.x, pairs = gridDim.x;
  int64_t token;
  int head;
  if (!pair_of(a, pair, token, head)) return;
  float2 v = make_float2(-INFINITY, 0.0f);
  if (tid < a.splits) v = a.part_ml[tid * pairs + pair];
  if (v.y == 0.0f) v.x = -INFINITY;  // saw nothing; its o was not written
  auto all = [&](float x, bool max) __attribute__((always_inline)) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const float y = __shfl_xor(x, off, 64);
      x = max ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if ((tid & 63) == 0) red[tid >> 6] = x;
    __syncthreads();
    return max ? fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])) : (red[0] + red[1]) + (red[2] + red[3]);
  };
  const float top = all(v.x, true);
  const float f = v.y == 0.0f ? 0.0f : mx_rebase(a, v.x, top);
  const float sum = all(v.y == 0.0f ? 0.0f : f * v.y, false);
  if (tid < a.splits) weight[tid] = v.y == 0.0f ? -1.0f : f;
  __syncthreads();
  // what a split that saw nothing left there is read and not used
  f32x4_t y = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* src = a.part_o + pair * D + (tid % L) * 4;
#pragma unroll 8
  for (int s = tid / L; s < a.splits; s += P) {
    const float w = weight[s];
    const f32x4_t o = *(const f32x4_t*)(src + s * pairs * D);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] += w == -1.0f ? 0.0f : w * o[i];
  }
  part[tid] = y;
  __syncthreads();
  if (tid >= L) return;
#pragma unroll
  for (int p = 1; p < P; ++p) y += part[p * L + tid];
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  *(u32x2_t*)(a.out + token * a.out_token + (int64_t)head * a.out_head + tid * 4) =
      u32x2_t{pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
}

template <int D, int RT>
hipError_t launch_few(const MxAttnArgs& a, hipStream_t stream) {
  const int64_t tiles = a.by_seq ? a.b.batch : a.b.tokens * a.group / (16 * RT) + a.b.batch;
  mx_attention_few_kernel<D, RT>
      <<<dim3((unsigned)(tiles * a.c.kv_heads), a.splits), 64 * kWaves, FewLds<D, RT>::Bytes, stream>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t join(const MxAttnArgs& a, hipStream_t stream) {
  if (a.splits == 1) return hipSuccess;
  const int64_t pairs = a.by_seq ? (int64_t)a.b.batch * a.c.kv_heads * 16 : a.b.tokens * a.heads;
  if (a.splits <= kJoinWave) mx_attention_join_few_kernel<D><<<(unsigned)((pairs + 3) / 4), 256, 0, stream>>>(a, pairs);
  else mx_attention_join_kernel<D><<<(unsigned)pairs, 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t launch_dim(MxAttnArgs a, const MxAttnPlan& plan, hipStream_t stream) {
  hipError_t e;
  if (plan.few) {
    if (plan.row_tiles == 1) e = launch_few<D, 1>(a, stream);
    else e = launch_few<D, D == 64 ? 2 : 1>(a, stream);  // two: only of 64
    return e == hipSuccess ? join<D>(a, stream) : e;
  }
  MxAttnArgs few = a;
  if (plan.mixed > 0) {
    a.skip = 16;
    few.by_seq = true;
    few.splits = plan.mixed;
    few.part_o = (float*)((uint8_t*)a.part_o + mx_prompt_part_bytes(plan, a.b.tokens, a.heads, D));
    few.part_ml = (float2*)(few.part_o + (int64_t)plan.mixed * a.b.batch * a.c.kv_heads * 16 * D);
    e = launch_few<D, 1>(few, stream);
    if (e != hipSuccess) return e;
  }
  e = launch_mx_attention_prompt(a, stream);
  // Of the few-rows form's sequences the first join writes what nobody left for it; where
  // there is one (few groups, long caches) those are in pieces too, and the second is right.
  if (e == hipSuccess) e = join<D>(a, stream);
  if (e == hipSuccess && plan.mixed > 0) e = join<D>(few, stream);
  return e;
}

template <int D, int RT>
hipError_t setup_few() {
  return hipFuncSetAttribute((const void*)mx_attention_few_kernel<D, RT>, hipFuncAttributeMaxDynamicSharedMemorySize,
                             FewLds<D, RT>::Bytes);
}

}  // namespace

hipError_t mx_attention_setup() {
  hipError_t e = setup_few<64, 1>();
  if (e == hipSuccess) e = setup_few<64, 2>();
  if (e == hipSuccess) e = setup_few<128, 1>();
  if (e == hipSuccess) e = setup_few<256, 1>();
  if (e == hipSuccess) e = mx_attention_prompt_setup();
  return e;
}

hipError_t launch_mx_attention(const MxAttnArgs& a, const MxAttnPlan& plan, hipStream_t stream) {
  switch (a.c.head_dim) {
    case 64: return launch_dim<64>(a, plan, stream);
    case 128: return launch_dim<128>(a, plan, stream);
    default: return launch_dim<256>(a, plan, stream);
  }
}

}  // namespace nvfp4
