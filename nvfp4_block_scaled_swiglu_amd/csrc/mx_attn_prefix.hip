// mx_attn_prefix.hip - attention over a paged MXFP4 cache where groups of sequences share their
// first tokens (gfx950).
//
// The softmax of a row falls into parts that are taken apart and joined: over tokens of part p with
// the largest score m_p, l_p = sum exp(s_t - m_p) and o_p = sum exp(s_t - m_p) v_t, and
// o = sum_p e^(m_p - m) o_p / sum_p e^(m_p - m) l_p. One part is the shared prefix: the rows of all
// sequences of a group are packed into one axis for it, as the rows and heads of one sequence are
// otherwise, so its tokens are read and decoded once for (sequences x heads of the group) rows. The other
// part is the rest of each sequence. Both are the forms of mx_attn_few.hpp and mx_attn_prompt.hpp,
// whose pieces of the token axis are such parts already.
//
// What bounds it, 48 single tokens of 56 heads of 128 over 8 behind 8,200: the prefix's workgroups take 26 us (20 of them
// 13 tiles, the rest their start and end), the sequences' own 10 us each in the CUs' other half, then 5 of joining: 35 us,
// where mxfp4_attention reads the prefix 48 times in 80. 16 tokens of 32 heads of 128 over 4 behind 131,071: 45 us of
// the prefix at 0.76 PFLOP/s, 8 of the rest behind it, 7.4 of joining 129 pieces: 56 to 62.
#include "mx_attn_few.hpp"
#include "mx_attn_prompt.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
static_assert(few::kWaves * 64 == kThreads && prompt::kWaves * 64 == kThreads, "one launch");

// Both parts in one launch: workgroups [0, first) for the prefixes, the others for what is left. (Two launches: 54 us
// for 42 in the first case above.)
// RT 0: the prompt form.
template <int D, int RT, MxPart PART>
__device__ __forceinline__ void attend(const MxAttnArgs& a, int id) {
  if constexpr (RT == 0) prompt::attend<D, PART>(a, mx_place(a, id));
  else few::attend<D, RT, PART>(a, mx_place(a, id));
}

constexpr int waves_per_simd(int d, int rt) { return rt == 0 ? prompt::waves_per_simd(d) : few::groups_per_cu(d, rt); }
constexpr int least(int a, int b) { return a < b ? a : b; }

template <int D, int RTP, int RTO>
__global__ __launch_bounds__(kThreads, least(waves_per_simd(D, RTP), waves_per_simd(D, RTO))) void
mx_attention_parts_kernel(MxAttnArgs prefix, MxAttnArgs own, int first) {
  if ((int)blockIdx.x < first) attend<D, RTP, kMxPrefix>(prefix, blockIdx.x);
  else attend<D, RTO, kMxOwn>(own, blockIdx.x - first);
}

template <int D, int RT>
constexpr int lds_bytes() {
  if constexpr (RT == 0) return prompt::Lds<D>::Bytes;
  else return few::FewLds<D, RT>::Bytes;
}

template <int D, int RTP, int RTO>
constexpr int both_lds() {
  return lds_bytes<D, RTP>() > lds_bytes<D, RTO>() ? lds_bytes<D, RTP>() : lds_bytes<D, RTO>();
}

// Rows that fill the prompt form's tiles sequence by sequence gain nothing from sharing them over
// a group: their sequences are walked through, the first tokens by the group's table, without pieces to join.
template <int D>
__global__ __launch_bounds__(kThreads, prompt::waves_per_simd(D)) void mx_attention_through_kernel(MxAttnArgs a) {
  prompt::attend<D, kMxThrough>(a, mx_place(a, blockIdx.x));
}

template <int RT>
int tiles(const MxAttnArgs& a, int64_t sequences) {
  return (int)mx_part_tiles(a.b.tokens * a.group, sequences, RT == 0 ? prompt::kRows : 16 * RT);
}

template <int D, int RTP, int RTO>
hipError_t launch_both(MxAttnArgs x, MxAttnArgs y, hipStream_t stream) {
  x.tiles = tiles<RTP>(x, x.prefix.groups);
  y.tiles = tiles<RTO>(y, y.b.batch);
  const int first = x.tiles * x.c.kv_heads * x.splits, rest = y.tiles * y.c.kv_heads * y.splits;
  mx_attention_parts_kernel<D, RTP, RTO><<<(unsigned)(first + rest), kThreads, both_lds<D, RTP, RTO>(), stream>>>(x, y, first);
  return hipGetLastError();
}

// the row tiles of a plan's form; two only of 64
int form(const MxAttnPlan& p, int d) { return !p.few ? 0 : d == 64 ? p.row_tiles : 1; }

template <int D>
hipError_t launch_through(MxAttnArgs a, const MxAttnPlan& plan, hipStream_t stream) {
  a.splits = plan.splits;
  a.part_ml = (float2*)(a.part_o + plan.splits * a.b.tokens * a.heads * D);
  a.tiles = tiles<0>(a, a.b.batch);
  mx_attention_through_kernel<D><<<(unsigned)(a.tiles * a.c.kv_heads * a.splits), kThreads, prompt::Lds<D>::Bytes, stream>>>(a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess && a.splits > 1 ? launch_mx_attention_join_parts(a, stream) : e;
}

template <int D>
hipError_t launch_dim(const MxAttnArgs& a, const MxPrefixPlan& plan, hipStream_t stream) {
  if (plan.through) return launch_through<D>(a, plan.own, stream);
  const int64_t rows = a.b.tokens * a.heads;
  const int pieces = plan.prefix.splits + plan.own.splits;
  MxAttnArgs x = a;
  x.part_ml = (float2*)(a.part_o + pieces * rows * D);
  x.splits = plan.prefix.splits;
  x.shared = (uint32_t*)(x.part_ml + pieces * rows);
  x.prefix_splits = x.splits;
  MxAttnArgs y = x;
  y.part_o += x.splits * rows * D;
  y.part_ml += x.splits * rows;
  y.splits = plan.own.splits;
  const int p = form(plan.prefix, D), o = form(plan.own, D);
  constexpr int T = D == 64 ? 2 : 1;
  hipError_t e;
  if (o == 1) e = p == 0 ? launch_both<D, 0, 1>(x, y, stream)
                         : p == 1 ? launch_both<D, 1, 1>(x, y, stream) : launch_both<D, T, 1>(x, y, stream);
  else e = p == 0 ? launch_both<D, 0, T>(x, y, stream) : launch_both<D, T, T>(x, y, stream);
  if (e != hipSuccess) return e;
  x.splits = pieces;
  return launch_mx_attention_join_parts(x, stream);
}

template <int D, int RTP, int RTO>
hipError_t setup_both() {
  return hipFuncSetAttribute((const void*)mx_attention_parts_kernel<D, RTP, RTO>, hipFuncAttributeMaxDynamicSharedMemorySize,
                             both_lds<D, RTP, RTO>());
}

template <int D>
hipError_t setup_dim() {
  constexpr int T = D == 64 ? 2 : 1;
  hipError_t e = setup_both<D, 0, 1>();
  if (e == hipSuccess) e = setup_both<D, 1, 1>();
  if (e == hipSuccess) e = setup_both<D, T, 1>();
  if (e == hipSuccess) e = setup_both<D, 0, T>();
  if (e == hipSuccess) e = setup_both<D, T, T>();
  if (e == hipSuccess)
    e = hipFuncSetAttribute((const void*)mx_attention_through_kernel<D>, hipFuncAttributeMaxDynamicSharedMemorySize,
                            prompt::Lds<D>::Bytes);
  return e;
}

}  // namespace

hipError_t mx_attention_prefix_setup() {
  hipError_t e = setup_dim<64>();
  if (e == hipSuccess) e = setup_dim<128>();
  if (e == hipSuccess) e = setup_dim<256>();
  return e;
}

hipError_t launch_mx_attention_prefix(const MxAttnArgs& a, const MxPrefixPlan& plan, hipStream_t stream) {
  switch (a.c.head_dim) {
    case 64: return launch_dim<64>(a, plan, stream);
    case 128: return launch_dim<128>(a, plan, stream);
    default: return launch_dim<256>(a, plan, stream);
  }
}

}  // namespace nvfp4
