// mx_attn.hip - launches of the attention over a paged MXFP4 cache, and the join of the pieces
// that the token axis was cut into (gfx950). The forms are in mx_attn_few.hpp (few rows of a
// sequence) and mx_attn_prompt.hpp (many).
#include "mx_attn_few.hpp"

namespace nvfp4 {

namespace {

using few::FewLds;
constexpr int kWaves = few::kWaves;

template <int D, int RT>
__global__ __launch_bounds__(64 * kWaves, few::groups_per_cu(D, RT)) void mx_attention_few_kernel(MxAttnArgs a) {
  // the longest contexts are not known here; the last tiles come first, as in the prompt form
  few::attend<D, RT, kMxWhole>(a, mx_place_whole(a));
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
  token = pair < (int64_t)1 << 32 ? (uint32_t)pair / (uint32_t)a.heads : pair / a.heads;
  head = (int)(pair - token * a.heads);
  return token >= mx_row_start(a.b, 0) && token < mx_row_start(a.b, a.b.batch);  // of no sequence: stays as it was
}

// Joins up to kJoinWave splits of each (row, head): a wave per pair. D/4 lanes take a split's
// row, four elements each, 256 / D splits at a time. 1,800 tokens, 24 heads of 64, attention
// in 2 pieces: 54 us, with a workgroup a pair 86.
constexpr int kJoinWave = 16;

template <int D, int J = kJoinWave>
__global__ __launch_bounds__(256) void mx_attention_join_few_kernel(MxAttnArgs a, int64_t pairs) {
  constexpr int L = D / 4, P = 64 / L;
  const int lane = threadIdx.x & 63;
  const int64_t pair = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (pair >= pairs) return;
  // The pieces are read before anything is known of them (otherwise after the row's sequence, the sums and the weights:
  // 2,688 pairs of 11 pieces 5.9 -> 5.4 us, with the launch before it 36.6 -> 34.8), also for pairs that turn out to be none and past the last piece, where
  // the first is read again; what a piece that saw nothing left there is not used. By sequence most pairs are none, and
  // are looked up first (32 sequences of 8 kv heads, 4 rows or none of 16 each, 8 pieces: 5.4 us, otherwise 5.8; 8 of
  // them in 32 pieces 5.2 and 6.0).
  int64_t token;
  int head;
  if (a.by_seq && !pair_of(a, pair, token, head)) return;
  float2 v = make_float2(-INFINITY, 0.0f);
  if (lane < a.splits) v = a.part_ml[lane * pairs + pair];
  constexpr int kFirst = J / P < 8 ? J / P : 8;  // splits of a lane that are read so
  f32x4_t o[kFirst];
  const float* src = a.part_o + pair * D + (lane % L) * 4;
#pragma unroll
  for (int q = 0; q < kFirst; ++q) {
    const int s = lane / L + q * P;
    o[q] = *(const f32x4_t*)(src + (s < a.splits ? s : 0) * pairs * D);
  }
  if (!a.by_seq && !pair_of(a, pair, token, head)) return;
  if (lane < a.prefix_splits && !a.shared[token]) v.y = 0.0f;
  if (v.y == 0.0f) v.x = -INFINITY;  // saw nothing; its o was not written
  float top = v.x;
#pragma unroll
  for (int off = J / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  top = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(top)));
  const float f = v.y == 0.0f ? 0.0f : mx_rebase(a, v.x, top);
  float sum = v.y == 0.0f ? 0.0f : f * v.y;
#pragma unroll
  for (int off = J / 2; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
  sum = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(sum)));
  const float weight = v.y == 0.0f ? -1.0f : f;
  f32x4_t y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < kFirst; ++q) {
    const float w = __shfl(weight, lane / L + q * P, 64);  // -1 past the last
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] += w == -1.0f ? 0.0f : w * o[q][i];
  }
  if constexpr (kFirst * P < J) {
    for (int s0 = lane / L + kFirst * P; s0 - lane / L < a.splits; s0 += 4 * P) {  // uniform
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int s = s0 + q * P;
        o[q] = *(const f32x4_t*)(src + (s < a.splits ? s : 0) * pairs * D);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float w = __shfl(weight, s0 + q * P, 64);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] += w == -1.0f ? 0.0f : w * o[q][i];
      }
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
  if (a.by_seq && !pair_of(a, pair, token, head)) return;  // (as above)
  float2 v = make_float2(-INFINITY, 0.0f);
  if (tid < a.splits) v = a.part_ml[tid * pairs + pair];
  constexpr int kFirst = 8;  // splits of a thread that are read ahead
  f32x4_t o[kFirst];
  const float* src = a.part_o + pair * D + (tid % L) * 4;
#pragma unroll
  for (int q = 0; q < kFirst; ++q) {
    const int s = tid / L + q * P;
    o[q] = *(const f32x4_t*)(src + (s < a.splits ? s : 0) * pairs * D);
  }
  if (!a.by_seq && !pair_of(a, pair, token, head)) return;
  if (tid < a.prefix_splits && !a.shared[token]) v.y = 0.0f;
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
  f32x4_t y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < kFirst; ++q) {
    const int s = tid / L + q * P;
    const float w = s < a.splits ? weight[s] : -1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] += w == -1.0f ? 0.0f : w * o[q][i];
  }
#pragma unroll 8
  for (int s = tid / L + kFirst * P; s < a.splits; s += P) {
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

// the pieces of two parts
template <int D>
hipError_t join_parts(const MxAttnArgs& a, hipStream_t stream) {
  const int64_t pairs = a.b.tokens * a.heads;
  if (a.splits <= kJoinWave || a.splits > 64) return join<D>(a, stream);
  mx_attention_join_few_kernel<D, 64><<<(unsigned)((pairs + 3) / 4), 256, 0, stream>>>(a, pairs);
  return hipGetLastError();
}

}  // namespace

hipError_t mx_attention_setup() {
  hipError_t e = setup_few<64, 1>();
  if (e == hipSuccess) e = setup_few<64, 2>();
  if (e == hipSuccess) e = setup_few<128, 1>();
  if (e == hipSuccess) e = setup_few<256, 1>();
  if (e == hipSuccess) e = mx_attention_prompt_setup();
  if (e == hipSuccess) e = mx_attention_prefix_setup();
  return e;
}

hipError_t launch_mx_attention(const MxAttnArgs& a, const MxAttnPlan& plan, hipStream_t stream) {
  switch (a.c.head_dim) {
    case 64: return launch_dim<64>(a, plan, stream);
    case 128: return launch_dim<128>(a, plan, stream);
    default: return launch_dim<256>(a, plan, stream);
  }
}

hipError_t launch_mx_attention_join_parts(const MxAttnArgs& a, hipStream_t stream) {
  switch (a.c.head_dim) {
    case 64: return join_parts<64>(a, stream);
    case 128: return join_parts<128>(a, stream);
    default: return join_parts<256>(a, stream);
  }
}

}  // namespace nvfp4
