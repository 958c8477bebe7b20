// Paged attention over a cache of bf16 values.
#include "paged_attn.cuh"

namespace idx {
cudaError_t launch_attn_bf16(const AttnArgs& a, cudaStream_t stream) {
  if (a.topk_idx) return attn::launch_type<IDX_BF16, attn::kSelection>(a, stream);
  return a.next_n > 1 ? launch_attn_bf16_several(a, stream)
                      : attn::launch_type<IDX_BF16, attn::kOneToken>(a, stream);
}
}  // namespace idx
