// Cached keys and values of requests into contiguous 16-bit rows, as prompt attention takes
// them: what a request's pages hold of positions [0, key_start[b+1] - key_start[b]) to
// rows key_start[b] on.
//
// Every 16 bytes of output are one lane's: eight values of a head, read as 16, 8 or 4
// bytes (and a 4-bit block's scale byte).  16-bit values are copied; E4M3 codes are
// multiplied by their head's scale in fp32 and rounded once; 4-bit codes times their power
// of two are exact in bf16, rounded once in fp16.
//
// Bound by HBM.  A block takes 16 tokens (one page holds them all) of all heads, keys and
// values, so that the request and the page are looked up once; the rows it writes lie
// together.  Which request rows belong to is found by searching key_start.  262144 4-bit tokens
// of 8 heads of 128 (1.35 GB) take 201 us, the measured copy rate.
#include "common.cuh"
#include "launch.h"
#include "serving.h"
#include "value_types.cuh"

namespace idx {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;

template <int D, int CT, bool BF16>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const __grid_constant__ KvGatherArgs a) {
  __shared__ int s_seq;
  pdl_launch_dependents();
  pdl_wait();  // inputs may come from the previous kernel
  // Groups of 16 tokens are numbered so that request b's start at floor(key_start[b] / 16) + b.
  const int num = blockIdx.x;
  auto start_of = [&](int b) -> int64_t {
    const int64_t x = __ldg(a.key_start + b);
    return x < 0 ? 0 : (x > a.out_rows ? a.out_rows : x);
  };
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {
    int lo = 0, hi = a.B;
    bool found = true;
    while (found) {
      const int step = (hi - lo + 31) / 32, b = lo + lane * step;
      const bool ok = b < hi && start_of(b) / kTokens + b <= num;
      const unsigned votes = __ballot_sync(~0u, ok);
      if (votes == 0) {
        found = false;
      } else {
        lo += (31 - __clz(votes)) * step;
        hi = min(hi, lo + step);
        if (step == 1) break;
      }
    }
    if (lane == 0) s_seq = found ? lo : -1;
  }
  if (blockIdx.x == gridDim.x - 1) {
    int bad = 0;
    const int64_t cap = (int64_t)a.max_blocks << a.page_shift;
    for (int b = tid; b < a.B; b += kThreads) {
      const int64_t x = __ldg(a.key_start + b), y = __ldg(a.key_start + b + 1);
      bad += x < 0 || y < x || y > a.out_rows || y - x > cap;
    }
    count_bad_input(a.errors, bad);
  }
  __syncthreads();
  const int b = s_seq;
  if (b < 0) return;
  const int64_t row0 = start_of(b), cap = (int64_t)a.max_blocks << a.page_shift;
  int64_t len = start_of(b + 1) - row0;
  if (len > cap) len = cap;
  const int64_t t0 = (num - (row0 / kTokens + b)) * kTokens;
  if (t0 >= len) return;
  const int n = (int)(len - t0 < kTokens ? len - t0 : kTokens);
  const int64_t page = __ldg(a.block_table + (int64_t)b * a.max_blocks + (t0 >> a.page_shift));
  if (page < 0 || page >= a.kv.num_blocks) {
    // counted once a page, by its first group
    if (tid == 0 && (t0 & ((1 << a.page_shift) - 1)) == 0) count_bad_input(a.errors);
    return;
  }
  const int off0 = (int)(t0 & ((1 << a.page_shift) - 1));

  constexpr int LQ = D / 8;                       // lanes per head's row
  constexpr int EB = CT == IDX_BF16 || CT == IDX_FP16 ? 2 : 1;
  const int heads = a.kv.heads, per_token = heads * LQ, all = n * per_token;
  const bool is_v = blockIdx.y != 0;
  const uint8_t* base = static_cast<const uint8_t*>(is_v ? a.kv.v : a.kv.k) +
                        page * (is_v ? a.kv.v_block_stride : a.kv.k_block_stride) * EB;
  const int64_t hs = (is_v ? a.kv.v_head_stride : a.kv.k_head_stride) * EB;
  const int64_t ts = CT == IDX_MXFP4 ? D / 2 : (is_v ? a.kv.v_token_stride : a.kv.k_token_stride) * EB;
  const float* scale = is_v ? a.kv.v_scale : a.kv.k_scale;
  uint4* out = reinterpret_cast<uint4*>(is_v ? a.v_out : a.k_out) + (row0 + t0) * per_token;
  // four rows' loads in flight a lane
  constexpr int U = 4;
#pragma unroll 1
  for (int i0 = tid; i0 < all; i0 += U * kThreads) {
    uint4 raw[U];
    uint32_t byte[U];
    float f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= all) break;
      // heads first within a token: the output's order
      const int t = i / per_token, h = i % per_token / LQ, part = i % LQ;
      const uint8_t* p = base + h * hs + (off0 + t) * ts;
      if (EB == 2) {
        raw[u] = __ldg(reinterpret_cast<const uint4*>(p) + part);
      } else if (CT == IDX_E4M3) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(p) + part);
        raw[u].x = x.x;
        raw[u].y = x.y;
        f[u] = scale ? __ldg(scale + h) : 1.f;
      } else {
        raw[u].x = __ldg(reinterpret_cast<const uint32_t*>(p) + part);
        byte[u] = __ldg(base + h * hs + ((D / 2) << a.page_shift) + (off0 + t) * (D / 32) + part / 4);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= all) break;
      if (EB == 2) {
        out[i] = raw[u];
        continue;
      }
      float x[8];
      if (CT == IDX_E4M3) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = e < 2 ? raw[u].x : raw[u].y;
          const float2 y = unpack2<false>(e4m3x2_to_f16x2((uint16_t)(e & 1 ? w >> 16 : w & 0xFFFF)));
          x[2 * e] = y.x * f[u];
          x[2 * e + 1] = y.y * f[u];
        }
      } else {
        uint32_t c[4];
        e2m1x8_to_f16x2(raw[u].x, c);
        // 2^(byte - 127); 2^-127, of the byte 0, is half of the smallest normal number
        const float two = byte[u] == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte[u] << 23);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 y = unpack2<false>(c[e]);
          x[2 * e] = y.x * two;
          x[2 * e + 1] = y.y * two;
        }
      }
      out[i] = pack8<BF16>(x);
    }
  }
}

template <int D, int CT, bool BF16>
cudaError_t launch(const KvGatherArgs& a, cudaStream_t stream) {
  const int64_t groups = a.out_rows / kTokens + a.B;
  return launch_dependent(kv_gather_kernel<D, CT, BF16>, dim3((unsigned)groups, 2), dim3(kThreads), 0, stream, a);
}
template <int CT, bool BF16>
cudaError_t launch_dim(const KvGatherArgs& a, cudaStream_t stream) {
  switch (a.kv.head_dim) {
    case 64: return launch<64, CT, BF16>(a, stream);
    case 128: return launch<128, CT, BF16>(a, stream);
    default: return launch<256, CT, BF16>(a, stream);
  }
}

}  // namespace

cudaError_t launch_kv_gather(const KvGatherArgs& a, cudaStream_t stream) {
  switch (a.kv.dtype) {
    case IDX_E4M3: return a.out_bf16 ? launch_dim<IDX_E4M3, true>(a, stream) : launch_dim<IDX_E4M3, false>(a, stream);
    case IDX_MXFP4: return a.out_bf16 ? launch_dim<IDX_MXFP4, true>(a, stream) : launch_dim<IDX_MXFP4, false>(a, stream);
    default: return launch_dim<IDX_BF16, true>(a, stream);  // 16-bit values are copied
  }
}

}  // namespace idx
