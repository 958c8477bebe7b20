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
//
// A 4-bit cache takes a block of 32 values from four lanes: their largest magnitude by two
// butterfly shuffles gives the scale byte, each lane stores four bytes of codes and the first
// of the four the byte; warps of queries alone do not.  Keys are encoded twice, at both ends of
// what their fp32 roundings leave open, and again in 64 bits where the two differ, so that codes
// are those of the unrounded key (32768 tokens of 32 + 2 x 8 heads of 128, 707 MB: 168 us, 0.63 of
// the copy rate; without this 142, where some 15 codes in 17 million fall to the other side of
// their border; encoding in every warp 11 more; E4M3 143).
#include "common.cuh"
#include "launch.h"
#include "mxfp4_encode.cuh"
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

// The heads that a thread's lanes work on together: n from h0 on, of token t.
template <int D, int VPT>
struct Group {
  int64_t t;
  int kind, h0, n;
  bool live;
  __device__ __forceinline__ Group(const KvInsertArgs& a, int q_groups, int k_groups) {
    constexpr int kLanes = D / 8;
    const unsigned per_token = q_groups + 2 * k_groups;
    const unsigned group = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    const unsigned tok = group / per_token;
    int gi = (int)(group - tok * per_token), heads = a.Hq;
    t = tok;
    live = t < a.N;
    kind = kQuery;
    if (gi >= q_groups) {
      gi -= q_groups;
      kind = kKey;
      heads = a.kv.heads;
      if (gi >= k_groups) {
        gi -= k_groups;
        kind = kValue;
      }
    }
    h0 = gi * VPT;
    n = live ? min(VPT, heads - h0) : 0;
  }
};

// Where a lane's eight values of a group's first head go in a 4-bit cache, and a head's store.
struct Place4 {
  uint8_t *codes, *scale;
  int64_t hs;
  __device__ __forceinline__ Place4(const KvInsertArgs& a, bool key, int64_t slot, int h0, int part, int D) {
    const int64_t page = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
    hs = key ? a.kv.k_head_stride : a.kv.v_head_stride;
    uint8_t* p = static_cast<uint8_t*>(key ? a.kv.k : a.kv.v) +
                 page * (key ? a.kv.k_block_stride : a.kv.v_block_stride) + h0 * hs;
    codes = p + off * (D / 2) + part * 4;
    scale = p + ((D / 2) << a.page_shift) + off * (D / 32) + part / 4;  // behind the page's codes
  }
  __device__ __forceinline__ void store(int u, uint32_t c, uint32_t byte, int part) const {
    *reinterpret_cast<uint32_t*>(codes + u * hs) = c;
    if (part % 4 == 0) scale[u * hs] = (uint8_t)byte;
  }
};

// Stores the codes and scale bytes of the warp's keys in its groups' heads `which` (bits) as 64-bit
// arithmetic gives them.  A sum is cut to fp32 with its last bit set where it is not exact,
// which leaves it on its side of every border between codes.  Everything is found anew: what
// would be kept for so rare a call costs the kernel registers.
template <int D, bool BF16, bool PAIRS, int VPT>
__device__ __noinline__ void store_exactly(const KvInsertArgs& a, int q_groups, int k_groups, uint32_t which) {
  constexpr int kLanes = D / 8;
  const int part = threadIdx.x % kLanes, half = a.rot_dim >> 1;
  const Group<D, VPT> gr(a, q_groups, k_groups);
  const bool key = gr.kind == kKey && gr.live;
  const int64_t slot = key ? __ldg(a.slots + gr.t) : -1;
  const int32_t pos = key && a.rot_dim > 0 ? __ldg(a.positions + gr.t) : 0;
  const bool pos_ok = a.rot_dim == 0 || (pos >= 0 && pos < a.num_pos);
  const bool turns = key && pos_ok && 8 * part < a.rot_dim;
  const bool store = key && pos_ok && slot >= 0 && slot < (a.kv.num_blocks << a.page_shift);
  const float *cs = a.cs + (int64_t)pos * half, *sn = a.sn + (int64_t)pos * half;
#pragma unroll 1
  for (; which != 0; which &= which - 1) {
    const int u = __ffs(which) - 1;
    float f[8] = {};
    if (key && u < gr.n)
      unpack8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.k) + gr.t * a.k_ts +
                                                    (gr.h0 + u) * a.k_hs + part * 8), f);
    double x[8], ss = 0.;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = f[i];
      ss += x[i] * x[i];
    }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) ss += __shfl_xor_sync(~0u, ss, d);
    if (!__any_sync(~0u, ss != 0.)) {  // zeros, which need no arithmetic
      if (store && u < gr.n) Place4(a, true, slot, gr.h0, part, D).store(u, 0, 0, part);
      continue;
    }
    if (a.k_weight != nullptr) {
      const double r = 1. / sqrt(ss / D + (double)a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= r * (double)__ldg(a.k_weight + 8 * part + i);
    }
    if constexpr (PAIRS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double e = x[2 * i], o = x[2 * i + 1];
        if (turns && 4 * part + i < half) {
          const double c = __ldg(cs + 4 * part + i), s = __ldg(sn + 4 * part + i);
          x[2 * i] = e * c - o * s;
          x[2 * i + 1] = e * s + o * c;
        }
      }
    } else {
      const bool second = 8 * part >= half;
      const int other = !turns ? part : (second ? part - half / 8 : part + half / 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double y = __shfl_sync(~0u, x[i], other, kLanes);
        if (turns) {
          const int col = 8 * part - (second ? half : 0) + i;
          const double s = __ldg(sn + col);
          x[i] = x[i] * (double)__ldg(cs + col) + y * (second ? s : -s);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = __double2float_rz(x[i]);
      if ((double)f[i] != x[i]) f[i] = __uint_as_float(__float_as_uint(f[i]) | 1u);
    }
    uint32_t byte;
    const uint32_t codes = encode8_block(f, &byte);
    if (store && u < gr.n) Place4(a, true, slot, gr.h0, part, D).store(u, codes, byte, part);
  }
}

// BITS of a cached value
template <int D, bool BF16, int BITS, bool PAIRS, int VPT>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 9 : 8) kv_insert_kernel(
    const __grid_constant__ KvInsertArgs a, int q_groups, int k_groups) {
  constexpr int kLanes = D / 8;
  constexpr bool CACHE8 = BITS == 8, CACHE4 = BITS == 4;
  const unsigned part = threadIdx.x % kLanes;
  const Group<D, VPT> gr(a, q_groups, k_groups);
  const int64_t t = gr.t;
  const bool live = gr.live;
  const int kind = gr.kind, h0 = gr.h0, n = gr.n;
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
    constexpr int EB = BITS == 16 ? 2 : 1;  // bytes of a stride's unit
    const int64_t page = slot_ok ? slot >> a.page_shift : 0, off = slot & ((1 << a.page_shift) - 1);
    if (kind == kKey) {
      dst = static_cast<uint8_t*>(a.kv.k) + (page * a.kv.k_block_stride + off * a.kv.k_token_stride) * EB;
      dst_hs = a.kv.k_head_stride * EB;
    } else {
      dst = static_cast<uint8_t*>(a.kv.v) + (page * a.kv.v_block_stride + off * a.kv.v_token_stride) * EB;
      dst_hs = a.kv.v_head_stride * EB;
    }
    if (CACHE4) dst += off * (D / 2);
    dst += h0 * dst_hs + part * BITS;
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
  const bool encodes = CACHE4 && __any_sync(~0u, kind != kQuery);
  // Normed or turned keys are off by their fp32 roundings, in units of 2^-24: 13 by the norm's
  // factor (half of 8 products' and sums', 5 shuffled sums' and eps's 14; 4 by rsqrtf; 2
  // products), 2 by the turn, 1 by the bounds below, in all 16 of the magnitudes that enter.
  // Where a code or a scale could differ within 17, for one or two vectors in a thousand, 64-bit
  // arithmetic decides afterwards, and so it does where fp32 may be off by more: a mean square that
  // overflows or, its eps letting it, is below 2^-100 (squares lose bits), a block whose largest is
  // outside [2^-50, 2^60) and not zero (so may products lose bits, or overflow with a weight's).
  // (32768 tokens 168 us, without these three 163.)
  const bool inexact = CACHE4 && kind == kKey && (weight != nullptr || turns);
  const bool checks = CACHE4 && __any_sync(~0u, inexact);
  uint32_t unsure = 0;  // heads of the lane's group
  const uint32_t least = a.eps >= 0x1p-100f ? 0 : 0x0D800000u;  // 2^-100
  float bound = inexact ? 0x1.1p-20f : 0.f;
  if (turns) {
    float top = 1.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) top = fmaxf(top, fmaxf(fabsf(c[i]), fabsf(s[i])));
    bound *= top;
  }
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    float x[8], off[4];
    bool far = false;
    if (works || BITS < 16) unpack8<BF16>(raw[u], x);
    if (works) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) ss += __shfl_xor_sync(~0u, ss, d);
      if (weight != nullptr) {
        const float ms = ss * (1.f / D) + a.eps, r = rsqrtf(ms);
        far = __float_as_uint(ms) - least >= 0x7F800000u - least;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
      }
      if (checks) {
#pragma unroll
        for (int i = 0; i < 4; ++i) off[i] = (fabsf(x[2 * i]) + fabsf(x[2 * i + 1])) * bound;
        if (!PAIRS) {  // what may enter any of the lane's eight
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
          off[0] = (top + __shfl_sync(~0u, top, other, kLanes)) * bound;
        }
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
    uint32_t codes = 0, byte = 0;
    if (CACHE4 && encodes) {  // every lane takes part in the shuffles
      if (checks) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = copysignf(off[PAIRS ? i / 2 : 0], x[i]);
          y[i] = x[i] - d;
          x[i] += d;
        }
        uint32_t low;
        const bool same = encode8_block(y, &low) == (codes = encode8_block(x, &byte));
        bool lost = !same || low != byte || far;
        if (byte - 77u >= 110u && inexact) {
          // (x has moved away from zero: where it is zero still, nothing came near the least code)
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
          lost = lost || top != 0.f;
        }
        if (lost) unsure |= 1u << u;
      } else {
        codes = encode8_block(x, &byte);
      }
    }
    if (!store || u >= n) continue;
    if (CACHE4 && kind != kQuery) {
      *reinterpret_cast<uint32_t*>(dst + u * dst_hs) = codes;
      // the scales lie behind the page's codes
      const int64_t at = slot & ((1 << a.page_shift) - 1);
      if (part % 4 == 0)
        dst[u * dst_hs - part * 4 - at * (D / 2) + ((D / 2) << a.page_shift) + at * (D / 32) + part / 4] = (uint8_t)byte;
    } else if (CACHE8 && kind != kQuery) {
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
  if (CACHE4 && checks) {
    unsure = __reduce_or_sync(~0u, unsure);
    if (unsure != 0) store_exactly<D, BF16, PAIRS, VPT>(a, q_groups, k_groups, unsure);
  }
}

template <int D, bool BF16, int BITS, bool PAIRS>
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
    return launch_dependent(kv_insert_kernel<D, BF16, BITS, PAIRS, 4>,
                            dim3((unsigned)((n4 + kGroups - 1) / kGroups)), dim3(kThreads), 0, stream,
                            a, q4, k4);
  const int64_t n1 = a.N * (a.Hq + 2 * a.kv.heads);
  return launch_dependent(kv_insert_kernel<D, BF16, BITS, PAIRS, 1>,
                          dim3((unsigned)((n1 + kGroups - 1) / kGroups)), dim3(kThreads), 0, stream, a,
                          a.Hq, a.kv.heads);
}

template <bool BF16, int BITS, bool PAIRS>
cudaError_t launch_p(const KvInsertArgs& a, int sms, cudaStream_t stream) {
  switch (a.kv.head_dim) {
    case 64: return launch_d<64, BF16, BITS, PAIRS>(a, sms, stream);
    case 128: return launch_d<128, BF16, BITS, PAIRS>(a, sms, stream);
    default: return launch_d<256, BF16, BITS, PAIRS>(a, sms, stream);
  }
}

template <bool BF16, int BITS>
cudaError_t launch_t(const KvInsertArgs& a, int sms, cudaStream_t stream) {
  return a.interleaved ? launch_p<BF16, BITS, true>(a, sms, stream)
                       : launch_p<BF16, BITS, false>(a, sms, stream);
}

template <bool BF16>
cudaError_t launch_bits(const KvInsertArgs& a, int sms, cudaStream_t stream) {
  switch (a.kv.dtype) {
    case IDX_E4M3: return launch_t<BF16, 8>(a, sms, stream);
    case IDX_MXFP4: return launch_t<BF16, 4>(a, sms, stream);
    default: return launch_t<BF16, 16>(a, sms, stream);
  }
}

}  // namespace

cudaError_t launch_kv_insert(int dtype, const KvInsertArgs& a, int sms, cudaStream_t stream) {
  return dtype == IDX_BF16 ? launch_bits<true>(a, sms, stream) : launch_bits<false>(a, sms, stream);
}

}  // namespace idx
