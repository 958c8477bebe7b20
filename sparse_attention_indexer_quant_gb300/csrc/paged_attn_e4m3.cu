// Paged attention over a cache of e4m3 values.
#include "paged_attn.cuh"

namespace idx {
cudaError_t launch_attn_e4m3(const AttnArgs& a, cudaStream_t stream) {
  if (a.topk_idx) return attn::launch_type<IDX_E4M3, attn::kSelection>(a, stream);
  return a.next_n > 1 ? launch_attn_e4m3_several(a, stream)
                      : attn::launch_type<IDX_E4M3, attn::kOneToken>(a, stream);
}
}  // namespace idx
