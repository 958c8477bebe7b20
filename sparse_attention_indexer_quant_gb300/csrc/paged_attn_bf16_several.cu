// Paged attention over a cache of bf16 values, several new tokens a request.
#include "paged_attn.cuh"

namespace idx {
cudaError_t launch_attn_bf16_several(const AttnArgs& a, cudaStream_t stream) {
  return attn::launch_type<IDX_BF16, attn::kSeveralTokens>(a, stream);
}
}  // namespace idx
