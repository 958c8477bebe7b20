// Paged attention over a cache of fp16 values.
#include "paged_attn.cuh"

namespace idx {
cudaError_t launch_attn_fp16(const AttnArgs& a, cudaStream_t stream) {
  return attn::launch_type<IDX_FP16>(a, stream);
}
}  // namespace idx
