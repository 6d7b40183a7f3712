// mx_attn_prompt.hip - launches of the attention's form for many rows (mx_attn_prompt.hpp).
#include "mx_attn_prompt.hpp"

namespace nvfp4 {

namespace {

using prompt::Lds;
using prompt::kRows;
using prompt::kWaves;

template <int D>
__global__ __launch_bounds__(64 * kWaves, prompt::waves_per_simd(D)) void mx_attention_prompt_kernel(MxAttnArgs a) {
  // within a causal sequence the last tiles see the most tokens: they are started first
  prompt::attend<D, kMxWhole>(a, mx_place_whole(a));
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
