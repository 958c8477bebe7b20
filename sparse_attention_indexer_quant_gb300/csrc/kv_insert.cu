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
// VPT heads of one kind (query, key or value) of one token, so that it reads
// the position, the slot, the table row and the weights once and keeps VPT
// 16-byte loads per lane in flight; value heads are copied as they are.
// 32768 tokens of 32 + 2 x 8 heads of 128 (bf16, 816 MB) take 134 us, 0.89 of
// the copy rate; in blocks of 256 threads 149 us, of 512 158, of 32 200 (the
// rate at which blocks start), as resident blocks that load the next group
// ahead 161 - 255; by twos instead of fours 201.
#include "common.cuh"
#include "launch.h"
#include "serving.h"
#include "value_types.cuh"

namespace idx {
namespace {

constexpr int kThreads = 128;

enum : int { kQuery = 0, kKey = 1, kValue = 2 };

// Eight consecutive floats; 16-byte loads where the base allows them (the
// offset is a multiple of four floats).
__device__ __forceinline__ void load8(const float* p, bool vec, float (&x)[8]) {
  if (vec) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __ldg(p + i);
  }
}
__device__ __forceinline__ bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int D, bool BF16, bool CACHE8, bool PAIRS, int VPT>
__global__ void __launch_bounds__(kThreads, CACHE8 ? 9 : 8) kv_insert_kernel(
    const __grid_constant__ KvInsertArgs a, int q_groups, int k_groups) {
  constexpr int kLanes = D / 8;
  const unsigned part = threadIdx.x % kLanes;
  const unsigned per_token = q_groups + 2 * k_groups;
  const unsigned group = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const unsigned tok = group / per_token;
  int gi = (int)(group - tok * per_token);
  const int64_t t = tok;
  const bool live = t < a.N;
  int kind = kQuery, heads = a.Hq;
  if (gi >= q_groups) {
    gi -= q_groups;
    kind = kKey;
    heads = a.kv.heads;
    if (gi >= k_groups) {
      gi -= k_groups;
      kind = kValue;
    }
  }
  const int h0 = gi * VPT;
  const int n = live ? min(VPT, heads - h0) : 0;  // heads of this group
  pdl_launch_dependents();
  pdl_wait();  // inputs may come from the previous kernel

  int64_t slot = -1;
  int32_t pos = 0;
  auto load_place = [&]() {
    if (live) {
      slot = __ldg(a.slots + t);
      if (a.rot_dim > 0) pos = __ldg(a.positions + t);
    }
  };
  // the table's row waits for the position: where it is long (16 values a lane)
  // the position goes first (147 us, after the heads 153), where short it does
  // not pay (136 and 134)
  if (!PAIRS) load_place();
  const int64_t hs = kind == kQuery ? a.q_hs : (kind == kKey ? a.k_hs : a.v_hs);
  const uint16_t* src = kind == kQuery ? static_cast<const uint16_t*>(a.q) + t * a.q_ts
                        : kind == kKey ? static_cast<const uint16_t*>(a.k) + t * a.k_ts
                                       : static_cast<const uint16_t*>(a.v) + t * a.v_ts;
  src += h0 * hs + part * 8;
  uint4 raw[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u)
    raw[u] = u < n ? *reinterpret_cast<const uint4*>(src + u * hs) : make_uint4(0, 0, 0, 0);
  if (PAIRS) load_place();
  const bool pos_ok = a.rot_dim == 0 || (pos >= 0 && pos < a.num_pos);
  const bool slot_ok = slot >= 0 && slot < (a.kv.num_blocks << a.page_shift);
  if (live && kind == kQuery && h0 == 0 && part == 0 && (!pos_ok || (slot != -1 && !slot_ok)))
    count_bad_input(a.errors);

  // where the group's first head goes
  uint8_t* dst;
  int64_t dst_hs;  // bytes between heads
  if (kind == kQuery) {
    dst = static_cast<uint8_t*>(a.q_out) + ((t * a.Hq + h0) * D + part * 8) * 2;
    dst_hs = D * 2;
  } else {
    constexpr int EB = CACHE8 ? 1 : 2;
    const int64_t page = slot_ok ? slot >> a.page_shift : 0, off = slot & ((1 << a.page_shift) - 1);
    if (kind == kKey) {
      dst = static_cast<uint8_t*>(a.kv.k) + (page * a.kv.k_block_stride + off * a.kv.k_token_stride) * EB;
      dst_hs = a.kv.k_head_stride * EB;
    } else {
      dst = static_cast<uint8_t*>(a.kv.v) + (page * a.kv.v_block_stride + off * a.kv.v_token_stride) * EB;
      dst_hs = a.kv.v_head_stride * EB;
    }
    dst += h0 * dst_hs + part * 8 * EB;
  }
  const bool store = live && pos_ok && (kind == kQuery || slot_ok);

  // the lane's angles: of its four pairs, or of its eight dimensions (the sine
  // then carries the sign of the turn); dimensions past rot_dim are not
  // multiplied at all (an infinity there stays one)
  const int half = a.rot_dim >> 1;
  constexpr int NC = PAIRS ? 4 : 8;
  float c[NC], s[NC];
  const bool turns = kind != kValue && live && pos_ok && 8 * (int)part < a.rot_dim;
  unsigned other = part;  // lane with the other half of a pair
  if (turns) {
    const int64_t row = (int64_t)pos * half;
    if constexpr (PAIRS) {
      const float* cp = a.cs + row + 4 * part;
      const float* sp = a.sn + row + 4 * part;
      if (half % 4 == 0 && on16(a.cs) && on16(a.sn)) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(cp));
        const float4 sv = __ldg(reinterpret_cast<const float4*>(sp));
        c[0] = cv.x; c[1] = cv.y; c[2] = cv.z; c[3] = cv.w;
        s[0] = sv.x; s[1] = sv.y; s[2] = sv.z; s[3] = sv.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = 4 * (int)part + i < half;
          c[i] = in ? __ldg(cp + i) : 1.f;
          s[i] = in ? __ldg(sp + i) : 0.f;
        }
      }
    } else {
      // rot_dim is a multiple of 16, so a lane is wholly in one half and the
      // table's rows start on 32 bytes where the table does
      const bool second = 8 * (int)part >= half;
      const int col = 8 * part - (second ? half : 0);
      other = second ? part - half / 8 : part + half / 8;
      load8(a.cs + row + col, on16(a.cs), c);
      load8(a.sn + row + col, on16(a.sn), s);
      if (!second) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = -s[i];
      }
    }
  }
  const float* weight = kind == kQuery ? a.q_weight : (kind == kKey ? a.k_weight : nullptr);
  float w[8];
  if (weight != nullptr) load8(weight + 8 * part, on16(weight), w);

  // warps that hold value heads alone copy; in the others every lane takes
  // part in the shuffles
  const bool works = __any_sync(~0u, kind != kValue);
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    float x[8];
    if (works || CACHE8) unpack8<BF16>(raw[u], x);
    if (works) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) ss += __shfl_xor_sync(~0u, ss, d);
      if (weight != nullptr) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
      }
      if constexpr (PAIRS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = x[2 * i], o = x[2 * i + 1];
          if (turns && 4 * (int)part + i < half) {
            x[2 * i] = e * c[i] - o * s[i];
            x[2 * i + 1] = e * s[i] + o * c[i];
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = __shfl_sync(~0u, x[i], other, kLanes);
          if (turns) x[i] = x[i] * c[i] + y * s[i];
        }
      }
    }
    if (!store || u >= n) continue;
    if (CACHE8 && kind != kQuery) {
      const float* scale = kind == kKey ? a.kv.k_scale : a.kv.v_scale;
      const float sc = scale ? __ldg(scale + h0 + u) : 1.f;
      // a true division, as the definition says: a product with 1/scale can
      // fall on the other side of a code's border
      uint2 v;
      v.x = pack_e4m3x2(__fdiv_rn(x[0], sc), __fdiv_rn(x[1], sc)) |
            pack_e4m3x2(__fdiv_rn(x[2], sc), __fdiv_rn(x[3], sc)) << 16;
      v.y = pack_e4m3x2(__fdiv_rn(x[4], sc), __fdiv_rn(x[5], sc)) |
            pack_e4m3x2(__fdiv_rn(x[6], sc), __fdiv_rn(x[7], sc)) << 16;
      *reinterpret_cast<uint2*>(dst + u * dst_hs) = v;
    } else {
      *reinterpret_cast<uint4*>(dst + u * dst_hs) = kind == kValue ? raw[u] : pack8<BF16>(x);
    }
  }
}

template <int D, bool BF16, bool CACHE8, bool PAIRS>
cudaError_t launch_d(const KvInsertArgs& a, int sms, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);  // per block
  // Four heads a group once they fill every SM's eight blocks, else one.  4000
  // tokens of 32 + 2 x 8 heads of 128: 18.4 us by fours, 28.4 by ones; 1000
  // tokens 6.2 and 7.8; 200 tokens 5.7 and 5.5 (few blocks, one long chain each).
  // Where fours would be half empty, ones: 20000 tokens of 2 + 2 x 2 heads 17.5
  // us, by fours 19.4; of 5 + 2 x 2 heads 16.7 and 15.4.
  const int q4 = (a.Hq + 3) / 4, k4 = (a.kv.heads + 3) / 4;
  const int64_t n4 = a.N * (q4 + 2 * k4);
  if (n4 >= (int64_t)sms * 8 * kGroups && 2 * (q4 + 2 * k4) < a.Hq + 2 * a.kv.heads)
    return launch_dependent(kv_insert_kernel<D, BF16, CACHE8, PAIRS, 4>,
                            dim3((unsigned)((n4 + kGroups - 1) / kGroups)), dim3(kThreads), 0, stream,
                            a, q4, k4);
  const int64_t n1 = a.N * (a.Hq + 2 * a.kv.heads);
  return launch_dependent(kv_insert_kernel<D, BF16, CACHE8, PAIRS, 1>,
                          dim3((unsigned)((n1 + kGroups - 1) / kGroups)), dim3(kThreads), 0, stream, a,
                          a.Hq, a.kv.heads);
}

template <bool BF16, bool CACHE8, bool PAIRS>
cudaError_t launch_p(const KvInsertArgs& a, int sms, cudaStream_t stream) {
  switch (a.kv.head_dim) {
    case 64: return launch_d<64, BF16, CACHE8, PAIRS>(a, sms, stream);
    case 128: return launch_d<128, BF16, CACHE8, PAIRS>(a, sms, stream);
    default: return launch_d<256, BF16, CACHE8, PAIRS>(a, sms, stream);
  }
}

template <bool BF16, bool CACHE8>
cudaError_t launch_t(const KvInsertArgs& a, int sms, cudaStream_t stream) {
  return a.interleaved ? launch_p<BF16, CACHE8, true>(a, sms, stream)
                       : launch_p<BF16, CACHE8, false>(a, sms, stream);
}

}  // namespace

cudaError_t launch_kv_insert(int dtype, const KvInsertArgs& a, int sms, cudaStream_t stream) {
  const bool c8 = a.kv.dtype == IDX_E4M3;
  if (dtype == IDX_BF16)
    return c8 ? launch_t<true, true>(a, sms, stream) : launch_t<true, false>(a, sms, stream);
  return c8 ? launch_t<false, true>(a, sms, stream) : launch_t<false, false>(a, sms, stream);
}

}  // namespace idx
