// Paged attention over a cache of e4m3 values, several new tokens a request.
#include "paged_attn.cuh"

namespace idx {
cudaError_t launch_attn_e4m3_several(const AttnArgs& a, cudaStream_t stream) {
  return attn::launch_type<IDX_E4M3, attn::kSeveralTokens>(a, stream);
}
}  // namespace idx
