// mx_attn.hip - attention over a paged MXFP4 cache (gfx950).
//
//   o[i, h] = sum_t softmax_t(scale * q[i, h] . k[t, h / g]) v[t, h / g]
//
// over the tokens t that row i of its sequence sees: t < kv_len, t <= p_i (causal), and
// with a window t > p_i - window or t < sinks; p_i = kv_len - rows + i. g = heads /
// kv_heads query heads share a kv head. A row that sees nothing gives zeros.
//
// One pass over the cache with the running maximum and sum of the softmax, all of it in
// registers. The (row, head of the group) pairs of a sequence and kv head are packed into
// one axis, so a single token of a grouped model fills a 16-wide matrix tile and a long
// prompt fills many. A wave owns RT tiles of 16 packed rows and walks the tokens 32 at a
// time with v_mfma_f32_16x16x32_bf16, in the transposed form:
//
//   S^T = K Q^T    A: lane (n, u) = (lane & 15, lane >> 4) holds token n, elements
//                  [u D/4, (u + 1) D/4) - the contraction order is free, so a lane takes
//                  the codes it loads (D/8 bytes) and at most two scales. S^T comes out
//                  with lane (n, u) holding packed row n, tokens 4u .. 4u + 3.
//   O^T = V^T P^T  B: P as S^T left it, without a move: lane (n, u) has tokens 4u .. 4u + 3
//                  of both 16-token halves, its 8 of the 32. A: lane (c, u) takes the same
//                  8 tokens, elements [c D/16, (c + 1) D/16): whole bytes of each token's
//                  codes, decoded in pairs along the head and paired along the tokens by
//                  byte permutes.
//
// Packed row n then stays in the lanes n + 16 u from the scores to the output, and lane
// (n, u) ends with elements [u D/4, (u + 1) D/4) of its row. Codes become exact bf16
// (v_cvt_scalef32_pk_bf16_fp4); scores, maxima, sums and o are fp32. P is rounded to bf16
// for the product (2^-9 of each weight, below the rounding of o); its sum takes the
// unrounded weights.
//
// The maximum is raised only when a score exceeds it by more than 2^8: until then weights
// up to 2^8 are as exact as those below 1, and most tiles skip the cross-lane maximum and
// the rescaling of O.
#include <type_traits>

#include "mx_attn.hpp"

namespace nvfp4 {

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;

constexpr int kWaves = 4;
constexpr float kRaise = 8.0f;  // log2 of how far weights may exceed 1
constexpr int kTile = 32;       // tokens per step

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

// codes 2 sel, 2 sel + 1 of q as packed bf16
__device__ __forceinline__ uint32_t decode2(uint32_t q, float s, int sel) {
  switch (sel) {
    case 0: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
    case 1: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
    case 2: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
    default: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
  }
}

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

// What a lane holds of 32 tokens. vs: D = 64 has two tokens' scales in a dword, D = 128
// one token's four, D = 256 the half of a token's eight that the lane's block is in.
template <int D>
struct Tile {
  Words<D / 32> k[2];
  uint32_t ks[2][D == 256 ? 2 : 1];
  uint32_t v[8][D == 256 ? 2 : 1];
  uint32_t vs[D == 64 ? 4 : 8];
  int t0;
  bool there[2];  // the page of each 16-token half exists
};

// The tile list of a wave's rows: tiles that hold the first tokens, then those from the
// window's start (or 0) to the last visible token.
struct Span {
  int first, begin, count;  // tiles [0, first), then [begin, ...); count in all
  __device__ __forceinline__ int at(int i) const { return i < first ? i : begin + (i - first); }
};

template <int D, int RT, bool COOP>
__global__ __launch_bounds__(64 * kWaves, COOP ? (RT == 4 ? 1 : 2) : 1) void mx_attention_kernel(MxAttnArgs a) {
  constexpr int NJ = D / 16, KS = D / 32, E = D / 4;
  constexpr int kRows = 16 * RT * (COOP ? 1 : kWaves);  // packed rows of the workgroup
  __shared__ float red[COOP ? kWaves * E * 64 : 1];
  __shared__ float ml[COOP ? 2 * kWaves * RT * 16 : 1];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, u = lane >> 4;
  const int kvh = blockIdx.x % a.c.kv_heads;
  const int split = blockIdx.y;
  const int g = a.group;

  // The row tile's sequence. Sequence i's tiles are numbered from floor(start_i g / kRows)
  // + i: that leaves each at least as many numbers as it has tiles, without a scan of the
  // lengths. The longest contexts (the last tiles) are started first.
  const int64_t tile = (gridDim.x - 1 - blockIdx.x) / a.c.kv_heads;
  int lo = 0, hi = a.b.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (mx_row_start(a.b, mid) * g / kRows + mid <= tile) lo = mid;
    else hi = mid;
  }
  const int64_t r0 = mx_row_start(a.b, lo), r1 = mx_row_start(a.b, lo + 1);
  const int64_t rows64 = r1 > r0 ? (r1 - r0) * g : 0;
  const int64_t p064 = (tile - (r0 * g / kRows + lo)) * kRows + (COOP ? 0 : wave * 16 * RT);
  if (p064 >= rows64 || p064 < 0) return;  // COOP: the whole workgroup; else no barrier follows
  const int rows = (int)rows64, p0 = (int)p064;
  const int kv_len = mx_seq_len(a.b, lo);
  const int back = kv_len - (int)(r1 - r0);  // position of the sequence's first row

  // ---- the rows ----
  bf16x8_t q[RT][KS];
  int high[RT], low[RT];  // visible: [low, high) and t < sinks
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int p = p0 + r * 16 + n;
    const bool real = p < rows;
    const int i = p / g;
    const uint16_t* src = a.q + (r0 + i) * a.q_token + (int64_t)(kvh * g + p % g) * a.q_head + u * E;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4_t w = {0u, 0u, 0u, 0u};
      if (real) w = *(const u32x4_t*)(src + 8 * s);
      q[r][s] = as_bf16x8(w[0], w[1], w[2], w[3]);
    }
    const int pos = back + i;
    const int h = a.causal && pos + 1 < kv_len ? pos + 1 : kv_len;
    high[r] = real && h > 0 ? h : 0;
    low[r] = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
  }
  const int last_row = (p0 + 16 * RT < rows ? p0 + 16 * RT : rows) - 1;
  const int pos_a = back + p0 / g, pos_b = back + last_row / g;
  const int high_min = p0 + 16 * RT > rows ? 0 : (a.causal && pos_a + 1 < kv_len ? pos_a + 1 : kv_len);
  int high_max = a.causal && pos_b + 1 < kv_len ? pos_b + 1 : kv_len;
  if (high_max < 0) high_max = 0;
  const int low_min = a.window > 0 && pos_a - a.window + 1 > 0 ? pos_a - a.window + 1 : 0;
  const int low_max = a.window > 0 && pos_b - a.window + 1 > 0 ? pos_b - a.window + 1 : 0;
  Span span;
  const int sinks = a.window > 0 ? a.sinks : 0;
  span.first = ((sinks < high_max ? sinks : high_max) + kTile - 1) / kTile;
  span.begin = low_min / kTile > span.first ? low_min / kTile : span.first;
  const int end_tile = (high_max + kTile - 1) / kTile;
  span.count = span.first + (end_tile > span.begin ? end_tile - span.begin : 0);
  const int begin = (int)((int64_t)span.count * split / a.splits) + (COOP ? wave : 0);
  const int end = (int)((int64_t)span.count * (split + 1) / a.splits);
  constexpr int kStep = COOP ? kWaves : 1;

  // ---- loads ----
  const int32_t* table = a.b.block_table + (int64_t)lo * a.b.table_stride;
  const int page_mask = (1 << a.b.page_shift) - 1;
  const int vblk = n * (D / 16) / 32;  // the block of the lane's V elements
  auto page_of = [&](int t) __attribute__((always_inline)) -> int64_t {
    if (t >= kv_len) return -1;
    const int64_t p = table[t >> a.b.page_shift];
    return p >= 0 && p < a.b.num_pages ? p : -1;
  };
  auto load = [&](Tile<D>& x, int tile_no, int64_t pg0, int64_t pg1) __attribute__((always_inline)) {
    x.t0 = tile_no * kTile;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t pg = h ? pg1 : pg0;
      x.there[h] = pg >= 0;
      // a page that is not there is read as page 0 and masked
      const int64_t row = ((pg < 0 ? 0 : pg) * a.c.kv_heads + kvh) * (int64_t)(page_mask + 1) +
                          ((x.t0 + 16 * h) & page_mask);
      const uint8_t* kc = a.c.k_codes + row * (D / 2);
      const uint8_t* ks = a.c.k_scales + row * (D / 32);
      const uint8_t* vc = a.c.v_codes + row * (D / 2);
      const uint8_t* vs = a.c.v_scales + row * (D / 32);
      x.k[h] = load_words<D / 32>(kc + n * (D / 2) + u * (D / 8));
      if constexpr (D == 64) x.ks[h][0] = ks[n * 2 + (u >> 1)];
      else if constexpr (D == 128) x.ks[h][0] = ks[n * 4 + u];
      else {
        const uint32_t two = *(const uint16_t*)(ks + n * 8 + u * 2);
        x.ks[h][0] = two & 0xFFu;
        x.ks[h][1] = two >> 8;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* p = vc + (4 * u + i) * (D / 2) + n * (D / 32);
        if constexpr (D == 64) x.v[4 * h + i][0] = *(const uint16_t*)p;
        else {
          const Words<D / 128> w = load_words<D / 128>(p);
#pragma unroll
          for (int j = 0; j < D / 128; ++j) x.v[4 * h + i][j] = w.w[j];
        }
      }
      if constexpr (D == 64) {
        const Words<2> w = load_words<2>(vs + 4 * u * 2);
        x.vs[2 * h] = w.w[0];
        x.vs[2 * h + 1] = w.w[1];
      } else if constexpr (D == 128) {
        const Words<4> w = load_words<4>(vs + 4 * u * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) x.vs[4 * h + i] = w.w[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x.vs[4 * h + i] = *(const uint32_t*)(vs + (4 * u + i) * 8 + (vblk >> 2) * 4);
      }
    }
  };
  auto v_byte = [&](const Tile<D>& x, int j) __attribute__((always_inline)) -> uint32_t {
    if constexpr (D == 64) return (x.vs[j >> 1] >> (16 * (j & 1) + 8 * vblk)) & 0xFFu;
    else return (x.vs[j] >> (8 * (vblk & 3))) & 0xFFu;
  };

  // ---- state ----
  f32x4_t o[RT][NJ];
  float m[RT], l[RT];  // m: agreed by the four lanes of a row; l: the lane's own tokens
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) o[r][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // One tile. FULL: every row sees every token of it.
  auto step = [&](const Tile<D>& x, auto full_tag) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(full_tag)::value;
    f32x4_t s[RT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int r = 0; r < RT; ++r) s[r][h] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < KS; ++e) {
        const u32x4_t w = mx_decode8(x.k[h].w[e], __uint_as_float(x.ks[h][D == 256 ? e >> 2 : 0] << 23));
        const bf16x8_t kf = as_bf16x8(w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int r = 0; r < RT; ++r) s[r][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[r][e], s[r][h], 0, 0, 0);
      }
    }
    bf16x8_t pf[RT];
    uint32_t seen[RT];  // bit j: the lane's row sees its token j (not kept when FULL)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      if constexpr (!FULL) {
        seen[r] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = x.t0 + 16 * (j >> 2) + 4 * u + (j & 3);
          const bool v = t < high[r] && (t >= low[r] || t < sinks) && x.there[j >> 2];
          if (v) seen[r] |= 1u << j;
          else s[r][j >> 2][j & 3] = -INFINITY;
        }
      }
      float top = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                        fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3]))) * a.scale_log2;
      if (__any(top > m[r] + kRaise)) {
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float next = fmaxf(m[r], top);
        // nothing to keep yet where m is -inf (o and l are 0)
        const float f = m[r] == next ? 1.0f : __builtin_amdgcn_exp2f(m[r] - next);
        m[r] = next;
        l[r] *= f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) o[r][j] *= f;
      }
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][j >> 2][j & 3], a.scale_log2, -m[r]));
        if constexpr (!FULL) p[j] = (seen[r] >> j & 1) ? p[j] : 0.0f;
      }
      l[r] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
      pf[r] = as_bf16x8(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7]));
    }
    float vsc[8];
    uint32_t nans = 0;  // bit j: the lane's block of its token j is NaN
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t byte = v_byte(x, j);
      if constexpr (!FULL) {
        const int t = x.t0 + 16 * (j >> 2) + 4 * u + (j & 3);
        // tokens that no row sees hold anything: scale 0 makes them finite
        if (t >= high_max || !x.there[j >> 2]) byte = 0;
        if (byte == 255u) {
          nans |= 1u << j;
          byte = 0;
        }
      }
      vsc[j] = __uint_as_float(byte << 23);
    }
    if constexpr (!FULL) {
      // 0 * NaN is NaN, and a row must not meet a NaN that it does not see: NaN blocks
      // leave the product (their codes are 0), and a second product of "is NaN" with "is
      // seen" tells the rows that get one. The lane's elements all lie in one block, so
      // its answer holds for all of them.
      if (__any(nans != 0)) {
        auto ones = [](uint32_t bits) __attribute__((always_inline)) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = (bits >> (2 * i) & 1 ? 0x3F80u : 0u) | (bits >> (2 * i + 1) & 1 ? 0x3F800000u : 0u);
          return as_bf16x8(w[0], w[1], w[2], w[3]);
        };
        const bf16x8_t is_nan = ones(nans);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const f32x4_t hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(is_nan, ones(seen[r]),
                                                                      f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) o[r][j][i] = hit[i] > 0.0f ? NAN : o[r][j][i];
        }
      }
    }
#pragma unroll
    for (int d = 0; d < NJ / 2; ++d) {
      uint32_t two[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) two[j] = decode2(x.v[j][D == 256 ? d >> 2 : 0], vsc[j], d & 3);
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
  auto run = [&](const Tile<D>& x) __attribute__((always_inline)) {
    const bool full = x.there[0] && x.there[1] && x.t0 + kTile <= high_min &&
                      (x.t0 >= low_max || x.t0 + kTile <= sinks);
    if (full) step(x, std::integral_constant<bool, true>());
    else step(x, std::integral_constant<bool, false>());
  };

  // ---- the walk: the next tile's loads are in flight while one is computed, and its
  // pages were looked up a tile earlier ----
  if (begin < end) {
    Tile<D> xa, xb;
    int t = span.at(begin);
    load(xa, t, page_of(t * kTile), page_of(t * kTile + 16));
    t = span.at(begin + kStep < end ? begin + kStep : begin);
    int64_t pg0 = page_of(t * kTile), pg1 = page_of(t * kTile + 16);
    for (int i = begin; i < end; i += 2 * kStep) {
      if (i + kStep < end) {
        load(xb, t, pg0, pg1);
        t = span.at(i + 2 * kStep < end ? i + 2 * kStep : begin);
        pg0 = page_of(t * kTile);
        pg1 = page_of(t * kTile + 16);
      }
      run(xa);
      if (i + kStep < end) {
        if (i + 2 * kStep < end) {
          load(xa, t, pg0, pg1);
          t = span.at(i + 3 * kStep < end ? i + 3 * kStep : begin);
          pg0 = page_of(t * kTile);
          pg1 = page_of(t * kTile + 16);
        }
        run(xb);
      }
    }
  }

  // ---- the rows' results ----
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    l[r] += __shfl_xor(l[r], 16, 64);
    l[r] += __shfl_xor(l[r], 32, 64);
  }
  auto row_of = [&](int r, int64_t& token, int& head) __attribute__((always_inline)) -> bool {
    const int p = p0 + r * 16 + n;
    token = r0 + p / g;
    head = kvh * g + p % g;
    return p < rows;
  };
  if constexpr (!COOP) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      int64_t token;
      int head;
      if (!row_of(r, token, head)) continue;
      if (a.splits > 1) {
        const int64_t at = ((int64_t)split * a.b.tokens + token) * a.heads + head;
        if (u == 0) a.part_ml[at] = make_float2(m[r], l[r]);
        if (l[r] != 0.0f) {
#pragma unroll
          for (int e = 0; e < E; e += 4)
            *(f32x4_t*)(a.part_o + at * D + u * E + e) =
                f32x4_t{o[r][e % NJ][e / NJ], o[r][(e + 1) % NJ][(e + 1) / NJ], o[r][(e + 2) % NJ][(e + 2) / NJ],
                        o[r][(e + 3) % NJ][(e + 3) / NJ]};
        }
      } else {
        const float inv = l[r] == 0.0f ? 0.0f : 1.0f / l[r];
        uint16_t* dst = a.out + token * a.out_token + (int64_t)head * a.out_head + u * E;
#pragma unroll
        for (int e = 0; e < E; e += 8) {
          u32x4_t w;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int e0 = e + 2 * k, e1 = e0 + 1;
            w[k] = pack_bf16(o[r][e0 % NJ][e0 / NJ] * inv, o[r][e1 % NJ][e1 / NJ] * inv);
          }
          *(u32x4_t*)(dst + e) = w;
        }
      }
    }
  } else {
    // The four waves walked different tokens of the same rows: join them, 16 rows at a
    // time. Wave w adds up and stores elements [(4u + w) D/16, + D/16) of each row.
    if (u == 0) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        ml[(wave * RT + r) * 16 + n] = m[r];
        ml[(kWaves * RT + wave * RT + r) * 16 + n] = l[r];
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float top = -INFINITY, sum = 0.0f, f[kWaves];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ml[(w * RT + r) * 16 + n]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float mw = ml[(w * RT + r) * 16 + n];
        f[w] = mw == top ? 1.0f : __builtin_amdgcn_exp2f(mw - top);
        sum += f[w] * ml[(kWaves * RT + w * RT + r) * 16 + n];
      }
      if (r > 0) __syncthreads();  // the last round's reads are done
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
      int64_t token;
      int head;
      if (!row_of(r, token, head)) continue;
      const int e0 = (4 * u + wave) * NJ;
      if (a.splits > 1) {
        const int64_t at = ((int64_t)split * a.b.tokens + token) * a.heads + head;
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
}

// Joins the splits of each (row, head): a wave per pair, D / 64 elements a lane.
template <int D>
__global__ __launch_bounds__(256) void mx_attention_join_kernel(MxAttnArgs a) {
  constexpr int W = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t pair = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), pairs = a.b.tokens * a.heads;
  if (pair >= pairs) return;
  const int64_t token = pair / a.heads;
  const int head = (int)(pair - token * a.heads);
  int pos;
  int64_t page;
  if (!mx_locate(a.b, token, pos, page)) return;  // a row of no sequence stays as it was
  float top = -INFINITY;
  for (int s = lane; s < a.splits; s += 64) top = fmaxf(top, a.part_ml[s * pairs + pair].x);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  float sum = 0.0f, y[W];
#pragma unroll
  for (int j = 0; j < W; ++j) y[j] = 0.0f;
  for (int s = 0; s < a.splits; ++s) {
    const float2 v = a.part_ml[s * pairs + pair];
    if (v.y == 0.0f) continue;  // saw nothing; its o was not written
    const float f = v.x == top ? 1.0f : __builtin_amdgcn_exp2f(v.x - top);
    sum += f * v.y;
    const float* o = a.part_o + (s * pairs + pair) * D + lane * W;
#pragma unroll
    for (int j = 0; j < W; ++j) y[j] += f * o[j];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* dst = a.out + token * a.out_token + (int64_t)head * a.out_head + lane * W;
  if constexpr (W == 1) {
    *dst = (uint16_t)pack_bf16(y[0] * inv, 0.0f);
  } else {
#pragma unroll
    for (int j = 0; j < W; j += 2) *(uint32_t*)(dst + j) = pack_bf16(y[j] * inv, y[j + 1] * inv);
  }
}

template <int D, int RT, bool COOP>
hipError_t launch_form(const MxAttnArgs& a, hipStream_t stream) {
  constexpr int kRows = 16 * RT * (COOP ? 1 : kWaves);
  const int64_t tiles = a.b.tokens * a.group / kRows + a.b.batch;
  mx_attention_kernel<D, RT, COOP><<<dim3((unsigned)(tiles * a.c.kv_heads), a.splits), 64 * kWaves, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  mx_attention_join_kernel<D><<<(unsigned)((a.b.tokens * a.heads + 3) / 4), 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t launch_dim(const MxAttnArgs& a, const MxAttnPlan& plan, hipStream_t stream) {
  if (!plan.coop) return launch_form<D, D == 256 ? 2 : 4, false>(a, stream);
  switch (plan.row_tiles) {
    case 1: return launch_form<D, 1, true>(a, stream);
    case 2: return launch_form<D, 2, true>(a, stream);
    default: return launch_form<D, D == 256 ? 2 : 4, true>(a, stream);
  }
}

}  // namespace

hipError_t launch_mx_attention(const MxAttnArgs& a, const MxAttnPlan& plan, hipStream_t stream) {
  switch (a.c.head_dim) {
    case 64: return launch_dim<64>(a, plan, stream);
    case 128: return launch_dim<128>(a, plan, stream);
    default: return launch_dim<256>(a, plan, stream);
  }
}

}  // namespace nvfp4
