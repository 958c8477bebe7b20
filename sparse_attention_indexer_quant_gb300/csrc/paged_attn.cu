// Paged attention: the join of split items (the streaming kernel is in
// paged_attn.cuh).
#include "paged_attn.cuh"

namespace idx {

namespace {

// One block per query row of one item: the parts' maxima, their weights
// 2^(m_part - m), then the weighted sums, in part order within each of the
// block's lane groups, and the groups in order.  A split item has a handful of
// parts (up to a few hundred for a lone long request); they were written a
// moment ago and come from L2.  The segment counter is left at this call's
// generation with no claims, for a replay of the call.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) attn_join_kernel(const __grid_constant__ AttnArgs a) {
  __shared__ float s_max[THREADS / 32], s_l[THREADS / 32];
  __shared__ float s_f[kAttnLevels * kAttnMaxCtas];  // an item has at most one part per segment
  __shared__ float4 s_acc[THREADS];
  const int tid = threadIdx.x, D = a.kv.head_dim;
  const int HR = a.kv.heads * a.row_tiles;
  const int item = blockIdx.x, req = item / HR, hr = item % HR;
  const int h = hr / a.row_tiles, rr = (hr % a.row_tiles) * a.part_rows + blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  if (item == 0 && blockIdx.y == 0 && tid == 0) *a.counter = a.gen << kItemBits;
  const int2 desc = a.desc[item];
  if (desc.y <= 1 || rr >= a.rows) return;
  // part i of the item: its first segment's, then the first part of each following one
  auto part_row = [&](int i) -> int64_t {
    const int part = i == 0 ? desc.x : 2 * (desc.x / 2 + i);
    return (int64_t)part * a.part_rows + blockIdx.y;
  };
  float mx = -INFINITY;
  for (int i = tid; i < desc.y; i += THREADS) mx = fmaxf(mx, a.part_ml[part_row(i) * 2]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
  if ((tid & 31) == 0) s_max[tid >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) mx = fmaxf(mx, s_max[w]);
  float lsum = 0.f;
  for (int i = tid; i < desc.y; i += THREADS) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + part_row(i) * 2);
    // a part that saw nothing of the row has weight 0 (and reference -inf)
    const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : attn::ex2(ml.x - mx);
    s_f[i] = f;
    lsum += ml.y * f;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) lsum += __shfl_xor_sync(~0u, lsum, d);
  if ((tid & 31) == 0) s_l[tid >> 5] = lsum;
  __syncthreads();
  lsum = 0.f;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) lsum += s_l[w];

  const int quads = D / 4, groups = THREADS / quads;
  const int q = tid % quads, grp = tid / quads;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = grp; i < desc.y; i += groups) {
    const float4 x = *reinterpret_cast<const float4*>(a.part_o + part_row(i) * D + 4 * q);
    const float f = s_f[i];
    acc.x += x.x * f;
    acc.y += x.y * f;
    acc.z += x.z * f;
    acc.w += x.w * f;
  }
  s_acc[tid] = acc;
  __syncthreads();
  if (grp != 0) return;
  for (int w = 1; w < groups; ++w) {
    const float4 x = s_acc[w * quads + q];
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
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
  const dim3 grid(items, a.part_rows);
  // few rows have many parts each: more loads in flight per row
  if ((int64_t)items * a.part_rows <= 512)
    return launch_dependent(attn_join_kernel<512>, grid, dim3(512), 0, stream, a);
  return launch_dependent(attn_join_kernel<128>, grid, dim3(128), 0, stream, a);
}

}  // namespace idx
