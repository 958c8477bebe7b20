// Paged attention: the join of split items (the streaming kernel is in
// paged_attn.cuh).
#include "paged_attn.cuh"

namespace idx {

namespace {

struct JoinRow {
  int req, h, rr;  // request (or query row, with a selection), kv head, row of the kv head
};

__device__ __forceinline__ JoinRow join_row(const AttnArgs& a, int item, int r) {
  const int HR = a.kv.heads * a.row_tiles, req = item / HR, hr = item - req * HR;
  const int h = hr / a.row_tiles;
  return JoinRow{req, h, (hr - h * a.row_tiles) * a.part_rows + r};
}
// Row of part i of an item in the partial arrays: its first segment's, then the
// first part of each following segment.
__device__ __forceinline__ int64_t part_row(const AttnArgs& a, int2 desc, int i, int r) {
  const int part = i == 0 ? desc.x : 2 * (desc.x / 2 + i);
  return (int64_t)part * a.part_rows + r;
}
// A part's weight; one that saw nothing of the row has weight 0 (and reference -inf).
__device__ __forceinline__ float part_weight(float2 ml, float mx) {
  return ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : attn::ex2(ml.x - mx);
}
template <int N>
__device__ __forceinline__ void store_row(const AttnArgs& a, JoinRow w, int d, const float (&acc)[N],
                                          float mx, float lsum) {
  const int tok = a.topk_idx ? w.req : w.req * a.next_n + w.rr / a.group;
  const int64_t orow = (int64_t)tok * a.Hq + w.h * a.group + w.rr % a.group;
  float inv = lsum == 0.f ? 0.f : 1.f / lsum;
  // an empty row stays zero whatever the scale
  if (a.kv.dtype == IDX_E4M3 && a.kv.v_scale && lsum != 0.f) inv *= __ldg(a.kv.v_scale + w.h);
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + orow * a.kv.head_dim + d);
#pragma unroll
  for (int i = 0; i < N; i += 2)
    out[i / 2] = a.q_bf16 ? pack2<true>(acc[i] * inv, acc[i + 1] * inv)
                          : pack2<false>(acc[i] * inv, acc[i + 1] * inv);
  if (a.lse && d == 0) a.lse[orow] = lsum == 0.f ? -INFINITY : (mx + log2f(lsum)) * attn::kLn2;
}

// The join.  Parts were written a moment ago and come from L2; weights are
// 2^(m_part - m), sums run in the order of the parts.  The segment counter is
// left at this call's generation with no claims, for a replay of the call.
//
// One warp per query row of one item: most items have a handful of parts.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join_rows_kernel(
    const __grid_constant__ AttnArgs a, int n) {
  constexpr int VL = D / 32;  // values per lane
  const int w = blockIdx.x * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  if (w == 0 && lane == 0) *a.counter = a.gen << kItemBits;
  if (w >= n) return;
  const int item = w / a.part_rows, r = w - item * a.part_rows;
  const int2 desc = a.desc[item];
  const JoinRow row = join_row(a, item, r);
  if (desc.y <= 1 || row.rr >= a.rows) return;
  // the first 32 parts' statistics stay in the lanes
  float2 mine = make_float2(-INFINITY, 0.f);
  float mx = -INFINITY;
  for (int i = lane; i < desc.y; i += 32) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + part_row(a, desc, i, r) * 2);
    if (i < 32) mine = ml;
    mx = fmaxf(mx, ml.x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
  float acc[VL], lsum = 0.f;
#pragma unroll
  for (int v = 0; v < VL; ++v) acc[v] = 0.f;
  const float* base = a.part_o + lane * VL;
#pragma unroll 4
  for (int i = 0; i < desc.y; ++i) {
    const int64_t pr = part_row(a, desc, i, r);
    float2 ml = make_float2(__shfl_sync(~0u, mine.x, i & 31), __shfl_sync(~0u, mine.y, i & 31));
    if (i >= 32) ml = *reinterpret_cast<const float2*>(a.part_ml + pr * 2);
    const float f = part_weight(ml, mx);
    lsum += ml.y * f;
    const float2* x = reinterpret_cast<const float2*>(base + pr * D);
#pragma unroll
    for (int v = 0; v < VL; v += 2) {
      const float2 y = x[v / 2];
      acc[v] += y.x * f;
      acc[v + 1] += y.y * f;
    }
  }
  store_row(a, row, lane * VL, acc, mx, lsum);
}

// One block per query row, for batches of few rows: their items have up to a
// few hundred parts, whose loads the block's lane groups share.
constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) attn_join_long_kernel(
    const __grid_constant__ AttnArgs a) {
  __shared__ float s_max[kJoinThreads / 32], s_l[kJoinThreads / 32];
  __shared__ float s_f[kAttnLevels * kAttnMaxCtas];  // an item has at most one part per segment
  __shared__ float4 s_acc[kJoinThreads];
  const int tid = threadIdx.x, D = a.kv.head_dim, r = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0 && r == 0 && tid == 0) *a.counter = a.gen << kItemBits;
  const int2 desc = a.desc[blockIdx.x];
  const JoinRow row = join_row(a, blockIdx.x, r);
  if (desc.y <= 1 || row.rr >= a.rows) return;
  float mx = -INFINITY;
  for (int i = tid; i < desc.y; i += kJoinThreads)
    mx = fmaxf(mx, a.part_ml[part_row(a, desc, i, r) * 2]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
  if ((tid & 31) == 0) s_max[tid >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) mx = fmaxf(mx, s_max[w]);
  float lsum = 0.f;
  for (int i = tid; i < desc.y; i += kJoinThreads) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + part_row(a, desc, i, r) * 2);
    const float f = part_weight(ml, mx);
    s_f[i] = f;
    lsum += ml.y * f;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) lsum += __shfl_xor_sync(~0u, lsum, d);
  if ((tid & 31) == 0) s_l[tid >> 5] = lsum;
  __syncthreads();
  lsum = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) lsum += s_l[w];

  const int quads = D / 4, groups = kJoinThreads / quads;
  const int q = tid % quads, grp = tid / quads;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = grp; i < desc.y; i += groups) {
    const float4 x = *reinterpret_cast<const float4*>(a.part_o + part_row(a, desc, i, r) * D + 4 * q);
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
  const float v[4] = {acc.x, acc.y, acc.z, acc.w};
  store_row(a, row, 4 * q, v, mx, lsum);
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs& a, cudaStream_t stream) {
  const int items = (a.topk_idx ? a.B * a.next_n : a.B) * a.kv.heads * a.row_tiles;
  const int64_t n = (int64_t)items * a.part_rows;
  if (n <= 512)
    return launch_dependent(attn_join_long_kernel, dim3(items, a.part_rows), dim3(kJoinThreads), 0,
                            stream, a);
  const dim3 grid((unsigned)((n + kJoinWarps - 1) / kJoinWarps)), block(kJoinWarps * 32);
  switch (a.kv.head_dim) {
    case 64: return launch_dependent(attn_join_rows_kernel<64>, grid, block, 0, stream, a, (int)n);
    case 128: return launch_dependent(attn_join_rows_kernel<128>, grid, block, 0, stream, a, (int)n);
    default: return launch_dependent(attn_join_rows_kernel<256>, grid, block, 0, stream, a, (int)n);
  }
}

}  // namespace idx
