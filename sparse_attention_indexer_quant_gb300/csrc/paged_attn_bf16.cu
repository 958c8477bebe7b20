// Paged attention over a cache of bf16 values.
#include "paged_attn.cuh"

namespace idx {
cudaError_t launch_attn_bf16(const AttnArgs& a, cudaStream_t stream) {
  return attn::launch_type<IDX_BF16>(a, stream);
}
}  // namespace idx
