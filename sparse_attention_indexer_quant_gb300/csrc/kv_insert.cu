// Per-head RMS norm of queries and keys, rotary turn, and the insert of keys
// and values into the paged cache, in one pass over the new tokens.
//
// A head is one vector of D values on D/8 consecutive lanes, eight values
// (16 bytes) a lane.  The mean square is summed over the lanes with butterfly
// shuffles; an interleaved pair (2i, 2i+1) lies in one lane, a pair
// (i, i + rot_dim/2) in two lanes rot_dim/16 apart, which exchange their
// values; values pass through fp32 and are rounded once, into q_out or the
// cache (a page's row, by the token's slot).
//
// Bound by HBM: each value is read once and written once (the tables' rows
// are shared by a token's heads and come from L1/L2).  A group of lanes takes
// VPT heads of one token, so that it reads the position, the slot and the
// table row once and keeps VPT 16-byte loads per lane in flight.
#include "common.cuh"
#include "launch.h"
#include "serving.h"
#include "value_types.cuh"

namespace idx {
namespace {

constexpr int kThreads = 256;

template <int D, bool BF16, bool CACHE8, int VPT>
__global__ void __launch_bounds__(kThreads) kv_insert_kernel(const __grid_constant__ KvInsertArgs a,
                                                             int groups_per_token) {
  constexpr int kLanes = D / 8;
  const int part = threadIdx.x % kLanes;
  const int64_t group = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int64_t t = group / groups_per_token;
  const int h0 = (int)(group - t * groups_per_token) * VPT;
  const int Hkv = a.kv.heads, Hqk = a.Hq + Hkv, Hall = Hqk + Hkv;
  const bool live = t < a.N;
  pdl_launch_dependents();
  pdl_wait();  // inputs may come from the previous kernel

  uint4 raw[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int h = h0 + u;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (live && h < Hall) {
      const uint16_t* src =
          h < a.Hq ? static_cast<const uint16_t*>(a.q) + t * a.q_ts + h * a.q_hs
          : h < Hqk ? static_cast<const uint16_t*>(a.k) + t * a.k_ts + (h - a.Hq) * a.k_hs
                    : static_cast<const uint16_t*>(a.v) + t * a.v_ts + (h - Hqk) * a.v_hs;
      raw[u] = reinterpret_cast<const uint4*>(src)[part];
    }
  }
  int64_t slot = -1;
  int32_t pos = 0;
  if (live) {
    slot = __ldg(a.slots + t);
    if (a.rot_dim > 0) pos = __ldg(a.positions + t);
  }
  const bool pos_ok = a.rot_dim == 0 || (pos >= 0 && pos < a.num_pos);
  const bool slot_ok = slot >= 0 && slot < (a.kv.num_blocks << a.page_shift);
  if (live && h0 == 0 && part == 0 && (!pos_ok || (slot != -1 && !slot_ok)))
    count_bad_input(a.errors);

  // the token's angles for this lane's eight dimensions; dimensions past
  // rot_dim are not multiplied at all (an infinity there stays one)
  const int half = a.rot_dim >> 1;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  int partner = 0;  // lanes to the other half of a pair
  if (live && pos_ok && 8 * part < a.rot_dim) {
    const int64_t row = (int64_t)pos * half;
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * part + i < half) {
          c[2 * i] = c[2 * i + 1] = __ldg(a.cs + row + 4 * part + i);
          s[2 * i] = s[2 * i + 1] = __ldg(a.sn + row + 4 * part + i);
        }
    } else {
      // rot_dim is a multiple of 16, so a lane is wholly in one half
      const bool second = 8 * part >= half;
      const int col = 8 * part - (second ? half : 0);
      partner = second ? -(half / 8) : half / 8;
      // rows of the table start on 32 bytes (half is a multiple of 8) when the table does
      if (((reinterpret_cast<uintptr_t>(a.cs) | reinterpret_cast<uintptr_t>(a.sn)) & 15) == 0) {
        const float4* cp = reinterpret_cast<const float4*>(a.cs + row + col);
        const float4* sp = reinterpret_cast<const float4*>(a.sn + row + col);
        const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
        c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
        c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
        s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
        s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = __ldg(a.cs + row + col + i);
          s[i] = __ldg(a.sn + row + col + i);
        }
      }
    }
  }

#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int h = h0 + u;
    const bool is_q = h < a.Hq, is_k = !is_q && h < Hqk;
    float x[8];
    unpack8<BF16>(raw[u], x);
    // every lane of the warp takes part in the shuffles, whatever its head
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) ss += __shfl_xor_sync(~0u, ss, d);
    const float* weight = is_q ? a.q_weight : (is_k ? a.k_weight : nullptr);
    if (weight != nullptr) {
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * r * __ldg(weight + 8 * part + i);
    }
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float e = x[i], o = x[i + 1];
        if ((is_q || is_k) && 4 * part + i / 2 < half) {
          x[i] = e * c[i] - o * s[i];
          x[i + 1] = e * s[i] + o * c[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(~0u, x[i], part + partner, kLanes);
        if ((is_q || is_k) && partner != 0)
          x[i] = partner > 0 ? x[i] * c[i] - y * s[i] : x[i] * c[i] + y * s[i];
      }
    }
    if (!live || h >= Hall || !pos_ok) continue;
    if (is_q) {
      uint16_t* dst = static_cast<uint16_t*>(a.q_out) + (t * a.Hq + h) * D;
      reinterpret_cast<uint4*>(dst)[part] = pack8<BF16>(x);
    } else if (slot_ok) {
      const int kvh = is_k ? h - a.Hq : h - Hqk;
      const int64_t page = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
      const int64_t at = is_k ? page * a.kv.k_block_stride + kvh * a.kv.k_head_stride + off * a.kv.k_token_stride
                              : page * a.kv.v_block_stride + kvh * a.kv.v_head_stride + off * a.kv.v_token_stride;
      void* base = is_k ? a.kv.k : a.kv.v;
      if (CACHE8) {
        const float* scale = is_k ? a.kv.k_scale : a.kv.v_scale;
        const float sc = scale ? __ldg(scale + kvh) : 1.f;
        // a true division, as the definition says: a product with 1/scale can
        // fall on the other side of a code's border
        uint2 w;
        w.x = pack_e4m3x2(__fdiv_rn(x[0], sc), __fdiv_rn(x[1], sc)) |
              pack_e4m3x2(__fdiv_rn(x[2], sc), __fdiv_rn(x[3], sc)) << 16;
        w.y = pack_e4m3x2(__fdiv_rn(x[4], sc), __fdiv_rn(x[5], sc)) |
              pack_e4m3x2(__fdiv_rn(x[6], sc), __fdiv_rn(x[7], sc)) << 16;
        reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at)[part] = w;
      } else {
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at)[part] = pack8<BF16>(x);
      }
    }
  }
}

template <int D, bool BF16, bool CACHE8>
cudaError_t launch_d(const KvInsertArgs& a, int sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);  // per block
  const int heads = a.Hq + 2 * a.kv.heads;
  // four heads a group once that still gives every SM its eight blocks
  const int64_t g4 = (heads + 3) / 4;
  if (a.N * g4 >= (int64_t)sms * 8 * kGroups) {
    const int64_t grid = (a.N * g4 + kGroups - 1) / kGroups;
    return launch_dependent(kv_insert_kernel<D, BF16, CACHE8, 4>, dim3((unsigned)grid),
                            dim3(kThreads), 0, stream, a, (int)g4);
  }
  const int64_t grid = (a.N * heads + kGroups - 1) / kGroups;
  return launch_dependent(kv_insert_kernel<D, BF16, CACHE8, 1>, dim3((unsigned)grid),
                          dim3(kThreads), 0, stream, a, heads);
}

template <bool BF16, bool CACHE8>
cudaError_t launch_t(const KvInsertArgs& a, int sms, cudaStream_t stream) {
  switch (a.kv.head_dim) {
    case 64: return launch_d<64, BF16, CACHE8>(a, sms, stream);
    case 128: return launch_d<128, BF16, CACHE8>(a, sms, stream);
    default: return launch_d<256, BF16, CACHE8>(a, sms, stream);
  }
}

}  // namespace

cudaError_t launch_kv_insert(int dtype, const KvInsertArgs& a, int sms, cudaStream_t stream) {
  const bool c8 = a.kv.dtype == IDX_E4M3;
  if (dtype == IDX_BF16)
    return c8 ? launch_t<true, true>(a, sms, stream) : launch_t<true, false>(a, sms, stream);
  return c8 ? launch_t<false, true>(a, sms, stream) : launch_t<false, false>(a, sms, stream);
}

}  // namespace idx
