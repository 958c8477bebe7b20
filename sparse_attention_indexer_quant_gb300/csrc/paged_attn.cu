// Paged attention: the join of split items (the streaming kernel is in
// paged_attn.cuh).
#include "paged_attn.cuh"

namespace idx {

namespace {

constexpr int kJoinThreads = 128;

// One block per query row of one item: the parts' maxima first, then the
// parts' sums weighted by 2^(m_part - m) in part order within each of the
// block's lane groups, and the groups in order.  A split item has a handful of
// parts (up to one per CTA for a lone long request); they were written a
// moment ago and come from L2.  The segment counter is left at this call's
// generation with no claims, for a replay of the call.
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnArgs a) {
  __shared__ float s_max[kJoinThreads / 32];
  __shared__ float4 s_acc[kJoinThreads];
  __shared__ float s_l[kJoinThreads];
  const int tid = threadIdx.x, D = a.kv.head_dim;
  const int HR = a.kv.heads * a.row_tiles;
  const int item = blockIdx.x, req = item / HR, hr = item % HR;
  const int h = hr / a.row_tiles, rr = (hr % a.row_tiles) * a.part_rows + blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  if (item == 0 && blockIdx.y == 0 && tid == 0) *a.counter = a.gen << kItemBits;
  const int2 desc = a.desc[item];
  if (desc.y <= 1 || rr >= a.rows) return;
  // part i of the item: its first CTA's, then the first part of each following CTA
  auto part_row = [&](int i) -> int64_t {
    const int part = i == 0 ? desc.x : 2 * (desc.x / 2 + i);
    return (int64_t)part * a.part_rows + blockIdx.y;
  };
  float mx = -INFINITY;
  for (int i = tid; i < desc.y; i += kJoinThreads) mx = fmaxf(mx, a.part_ml[part_row(i) * 2]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
  if ((tid & 31) == 0) s_max[tid >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) mx = fmaxf(mx, s_max[w]);

  const int quads = D / 4, groups = kJoinThreads / quads;
  const int q = tid % quads, grp = tid / quads;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float lsum = 0.f;
#pragma unroll 4
  for (int i = grp; i < desc.y; i += groups) {
    const int64_t r = part_row(i);
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + r * 2);
    const float4 x = *reinterpret_cast<const float4*>(a.part_o + r * D + 4 * q);
    // a part that saw nothing of the row has weight 0 (and reference -inf)
    const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : attn::ex2(ml.x - mx);
    lsum += ml.y * f;
    acc.x += x.x * f;
    acc.y += x.y * f;
    acc.z += x.z * f;
    acc.w += x.w * f;
  }
  s_acc[tid] = acc;
  s_l[tid] = lsum;
  __syncthreads();
  if (grp != 0) return;
  for (int w = 1; w < groups; ++w) {
    const float4 x = s_acc[w * quads + q];
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
    lsum += s_l[w * quads + q];
  }
  const int tok = a.topk_idx ? req : req * a.next_n + rr / a.group;
  const int64_t orow = (int64_t)tok * a.Hq + h * a.group + rr % a.group;
  float inv = lsum == 0.f ? 0.f : 1.f / lsum;
  if (a.kv.dtype == IDX_E4M3 && a.kv.v_scale) inv *= __ldg(a.kv.v_scale + h);
  uint2 w;
  if (a.q_bf16) {
    w.x = pack2<true>(acc.x * inv, acc.y * inv);
    w.y = pack2<true>(acc.z * inv, acc.w * inv);
  } else {
    w.x = pack2<false>(acc.x * inv, acc.y * inv);
    w.y = pack2<false>(acc.z * inv, acc.w * inv);
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + 4 * q) = w;
  if (a.lse && q == 0) a.lse[orow] = lsum == 0.f ? -INFINITY : (mx + log2f(lsum)) * attn::kLn2;
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs& a, cudaStream_t stream) {
  const int items = (a.topk_idx ? a.B * a.next_n : a.B) * a.kv.heads * a.row_tiles;
  return launch_dependent(attn_join_kernel, dim3(items, a.part_rows), dim3(kJoinThreads), 0, stream,
                          a);
}

}  // namespace idx
