// Attention of a few new tokens over a paged key-value cache.
//
// Work.  An item is one kv head of one request with its query rows (next_n
// tokens times the heads of the group; with a selection, one token's group),
// up to 16 * MT of them.  Its keys are cut into units of 8 * KS, numbered item
// by item over the whole batch, and CTA c of A takes units [c U / A, (c+1) U / A):
// every CTA streams the same number of bytes whatever the requests' lengths.
// A CTA that covers an item alone writes the result; an item that spans CTAs
// leaves one partial (running maximum, weight, weighted sum) per CTA in the
// workspace and a second, dependent launch joins them in the order of their
// keys, so the result does not depend on the order in which CTAs run.
//
// Arithmetic.  o = sum_s p_s v_s / sum_s p_s with p_s = 2^(x_s - m), one pass
// with a running reference m per row that is raised (and the sums rescaled)
// only when a score passes it by more than 2^8, which fp32 sums hold easily:
// most tiles need one vote instead of two shuffle reductions.  Scores and sums
// are fp32 accumulators of m16n8k16 products with the query rows on M.  p goes
// into the second product as two 16-bit terms, hi = round(p) and lo =
// round(p - hi): one term's rounding (2^-9 in bf16) would be as large as the
// rounding of the output itself.  8-bit codes are exact in fp16; queries are
// then brought to fp16 by a power of two per row, which loses nothing of a
// bf16 value within 2^-29 of the row's largest.
//
// Memory.  2 G flops per byte of cache (G query heads per kv head) is far
// below the tensor pipes' ridge, so the kernel is built as a stream: each of
// the CTA's eight warps owns KS keys of every unit and a private ring of
// half stages (KS keys' K or V rows, 16-byte cp.async, XOR-swizzled for
// ldmatrix); no barrier stands between warps until the item ends.  Rows that
// no query sees are zero-filled, never read, so whatever a page holds past the
// context (NaN included) cannot reach a sum.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "serving.h"
#include "value_types.cuh"

namespace idx {
namespace attn {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTab = 2048;  // page groups (or listed positions) resolved at a time
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;  // log2 of how far a score may pass the reference

template <int D, int CT>
constexpr int row_bytes() { return D * (CT == IDX_E4M3 ? 1 : 2); }
// keys per warp and unit: 4 KB half stages where rows are short
template <int D, int CT>
constexpr int tile_keys() { return row_bytes<D, CT>() >= 256 ? 16 : 32; }

template <int D, int CT, int MT>
struct Cfg {
  static constexpr bool kF8 = CT == IDX_E4M3;
  static constexpr bool kMmaBf16 = CT == IDX_BF16;
  static constexpr int kRowB = row_bytes<D, CT>();
  static constexpr int kKS = tile_keys<D, CT>();
  static constexpr int kUnit = kWarps * kKS;
  static constexpr int kRows = 16 * MT;
  static constexpr int kHalf = kRowB * kKS;  // bytes of a half stage
  // two CTAs per SM where 128 registers a thread hold the accumulators
  static constexpr int kOcc = (MT == 1 && D <= 128) ? 2 : 1;
  static constexpr int kStages = (kOcc == 2 ? 12288 : 24576) / kHalf;
  static constexpr int kRing = kStages * kHalf;
  static constexpr int kPitch = D + 8;  // floats of a row of the merge buffer
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kSmem = kWarps * kRing + kQBytes + kTab * 4;
  static_assert(kRows * kPitch * 4 <= kRing, "a warp's sums fit its ring");
  static_assert(kStages >= 3, "");
};

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(full ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory offset of 16-byte chunk c of row r: the chunk index is XORed
// with the row so that eight rows' equal chunks lie in eight bank groups
// (64-byte rows: two rows per 128 bytes).
template <int ROWB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if (ROWB >= 128) return (uint32_t)(r * ROWB + ((c ^ (r & 7)) << 4));
  return (uint32_t)(r * ROWB + ((c ^ ((r >> 1) & 3)) << 4));
}

// Sum over a warp's lanes below / over the block, for 64-bit values.
__device__ __forceinline__ long long warp_incl_sum(long long x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// A request as an item sees it.
struct Span {
  int len;    // clamped context
  int t0;     // first unit of its keys
  int units;  // units (at least one, so that an empty request's rows are written)
};

template <int D, int CT, int MT>
__global__ void __launch_bounds__(kThreads, (Cfg<D, CT, MT>::kOcc))
paged_attn_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<D, CT, MT>;
  constexpr bool F8 = C::kF8, MB = C::kMmaBf16;
  constexpr int KS = C::kKS, ROWB = C::kRowB, NS = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long s_warp[kWarps];
  __shared__ long long s_base;
  __shared__ int s_req;
  __shared__ float s_mult[C::kRows];
  __shared__ float2 s_ml[kWarps][C::kRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* ring = smem + warp * C::kRing;
  const uint32_t ring_u = smem_u32(ring);
  uint8_t* q_sm = smem + kWarps * C::kRing;
  const uint32_t q_u = smem_u32(q_sm);
  int* tab = reinterpret_cast<int*>(q_sm + C::kQBytes);

  const bool listed = a.topk_idx != nullptr;
  const int Hkv = a.kv.heads, HR = Hkv * a.row_tiles;
  const int page_mask = (1 << a.page_shift) - 1;
  const long long cap = (long long)a.max_blocks << a.page_shift;
  pdl_wait();  // inputs may come from the previous kernel; it may still read the workspace

  auto span_of = [&](int b) -> Span {
    Span s;
    const int L = __ldg(a.context_lens + b);
    s.len = L < 0 ? 0 : (L > cap ? (int)cap : L);
    const int first = a.window > 0 ? max(0, s.len - a.next_n + 1 - a.window) : 0;
    s.t0 = first / C::kUnit;
    s.units = max(1, (int)(((long long)s.len + C::kUnit - 1) / C::kUnit) - s.t0);
    return s;
  };

  // ---- this CTA's units [u0, u1), and the request the first belongs to
  const int reqs = listed ? a.B * a.next_n : a.B;
  const int list_units = (a.topk + C::kUnit - 1) / C::kUnit;
  long long u0, u1, U, A, base;  // base: first unit of request `req`
  int req;
  if (!a.split) {
    U = 0;  // one CTA per item, which knows its units below
  } else if (listed) {
    U = (long long)reqs * HR * list_units;
  } else {
    long long sum = 0;
    for (int b = tid; b < reqs; b += kThreads) sum += span_of(b).units;
    sum = warp_incl_sum(sum, lane);
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    U = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) U += s_warp[w];
    U *= HR;
  }
  A = gridDim.x;
  if (a.split) {
    // no more CTAs than units
    if (A > U) A = U;
    if ((long long)blockIdx.x >= A) {
      pdl_launch_dependents();
      return;
    }
    u0 = (long long)blockIdx.x * U / A;
    u1 = ((long long)blockIdx.x + 1) * U / A;
  } else {
    const int units = listed ? list_units : span_of(blockIdx.x / HR).units;
    u0 = (long long)(blockIdx.x % HR) * units;
    u1 = u0 + units;
  }
  if (!a.split) {
    req = blockIdx.x / HR;
    base = 0;
  } else if (listed) {
    req = (int)(u0 / ((long long)HR * list_units));
    base = (long long)req * HR * list_units;
  } else {
    long long before = 0;  // units of the requests before this round's
    for (int b0 = 0;; b0 += kThreads) {
      const int b = b0 + tid;
      const long long mine = b < reqs ? (long long)span_of(b).units * HR : 0;
      long long incl = warp_incl_sum(mine, lane);
      __syncthreads();
      if (lane == 31) s_warp[warp] = incl;
      __syncthreads();
      long long total = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) incl += s_warp[w];
        total += s_warp[w];
      }
      const long long start = before + incl - mine;
      if (mine > 0 && start <= u0 && u0 < start + mine) {
        s_req = b;
        s_base = start;
      }
      before += total;
      if (before > u0) break;
    }
    __syncthreads();
    req = s_req;
    base = s_base;
  }

  const int g = lane >> 2, c4 = lane & 3;  // fragment row and column group
  const bool use_cap = a.softcap > 0.f;

  for (long long u = u0; u < u1;) {
    // ---- the item at unit u, and the part of it that is this CTA's
    const int b = listed ? req / a.next_n : req;
    const int tok0 = listed ? req : req * a.next_n;  // query row of the item's first row
    const int n_tok = listed ? 1 : a.next_n;
    const Span sp = span_of(b);
    const int units = listed ? list_units : sp.units;
    const int hr = (int)((u - base) / units);
    const int h = hr / a.row_tiles, rt = hr % a.row_tiles;
    const int ta = (int)((u - base) - (long long)hr * units);
    const int tb = (int)min((long long)units, ta + (u1 - u));
    const int row0 = rt * C::kRows;
    const int rows = min(C::kRows, a.rows - row0);
    const uint8_t* kbase = static_cast<const uint8_t*>(a.kv.k) + h * a.kv.k_head_stride * (F8 ? 1 : 2);
    const uint8_t* vbase = static_cast<const uint8_t*>(a.kv.v) + h * a.kv.v_head_stride * (F8 ? 1 : 2);
    const int64_t k_bs = a.kv.k_block_stride * (F8 ? 1 : 2), v_bs = a.kv.v_block_stride * (F8 ? 1 : 2);
    const int64_t k_ts = a.kv.k_token_stride * (F8 ? 1 : 2), v_ts = a.kv.v_token_stride * (F8 ? 1 : 2);
    // sight of query token j: [end_j - window, end_j), end_j = end0 + j
    const int end0 = listed ? 0 : sp.len - a.next_n + 1;
    const int lo_all = a.window > 0 ? max(0, end0 - a.window) : 0;
    const int* bt = a.block_table + (int64_t)b * a.max_blocks;

    if (tid == 0 && hr == 0 && ta == 0 && (!listed || req % a.next_n == 0)) {
      const int L = __ldg(a.context_lens + b);
      if (L < 0 || L > cap) count_bad_input(a.errors);
    }

    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }

    // keys per sub-range whose page ids (or list entries) fit the table
    constexpr int kSub = kTab / C::kUnit;            // units of listed positions
    const int sub = listed ? kSub : kSub * 16;       // units of 16-key groups
    bool q_loaded = false;
    for (int sa = ta; sa < tb; sa += sub) {
      const int sb = min(tb, sa + sub);
      __syncthreads();  // the table and the query rows of the previous range are done with
      if (listed) {
        const int* list = a.topk_idx + (int64_t)req * a.topk;
        const int my_end = max(0, sp.len - a.next_n + 1 + req % a.next_n);
        for (int i = tid; i < (sb - sa) * C::kUnit; i += kThreads) {
          const int at = sa * C::kUnit + i;
          int slot = -1;
          const int p = at < a.topk ? __ldg(list + at) : -1;
          if (p >= 0) {
            bool ok = p < my_end;
            if (ok) {
              const int id = __ldg(bt + (p >> a.page_shift));
              ok = id >= 0 && id < a.kv.num_blocks;
              slot = ok ? (id << a.page_shift) + (p & page_mask) : -1;
            }
            if (!ok && hr == 0) count_bad_input(a.errors);
          }
          tab[i] = slot;
        }
      } else {
        const int g0 = (sp.t0 + sa) * (C::kUnit / 16), ng = (sb - sa) * (C::kUnit / 16);
        for (int i = tid; i < ng; i += kThreads) {
          const int key = (g0 + i) * 16;
          int id = -1;
          if (key < sp.len && key + 16 > lo_all) {
            id = __ldg(bt + (key >> a.page_shift));
            if (id < 0 || id >= a.kv.num_blocks) {
              // counted once per page, by its first group that is in sight
              if (hr == 0 && ((key & page_mask) == 0 || key <= lo_all)) count_bad_input(a.errors);
              id = -1;
            }
          }
          tab[i] = id;
        }
      }
      __syncthreads();

      // ---- the warp's stream: half stage 2 t is unit sa + t's keys, 2 t + 1 its values
      const int halves = 2 * (sb - sa);
      int put = 0, get = 0;  // ring positions
      auto issue = [&](int i) {
        if (i < halves) {
          const int t = i >> 1;
          const bool is_v = i & 1;
          const uint8_t* src0 = is_v ? vbase : kbase;
          const int64_t bs = is_v ? v_bs : k_bs, ts = is_v ? v_ts : k_ts;
          constexpr int LPR = ROWB / 16, RPI = 32 / LPR;  // lanes per row, rows per pass
          const uint32_t dst = ring_u + put * C::kHalf;
          const int rl = lane / LPR, cl = lane % LPR;
          if (listed) {
#pragma unroll
            for (int j = 0; j < KS / RPI; ++j) {
              const int r = j * RPI + rl;
              const int slot = tab[t * C::kUnit + warp * KS + r];
              const bool ok = slot >= 0;
              const uint8_t* src = src0 + (ok ? (slot >> a.page_shift) * bs + (slot & page_mask) * ts : 0);
              cp_async_16_zfill(dst + swz<ROWB>(r, cl), src + cl * 16, ok);
            }
          } else {
#pragma unroll
            for (int gr = 0; gr < KS / 16; ++gr) {
              const int grp = t * (C::kUnit / 16) + warp * (KS / 16) + gr;
              const int id = tab[grp];
              const int key = (sp.t0 + sa) * C::kUnit + grp * 16;
              const uint8_t* src =
                  src0 + (id >= 0 ? id * bs + (key & page_mask) * ts : 0) + rl * ts + cl * 16;
#pragma unroll
              for (int j = 0; j < 16 / RPI; ++j) {
                const int r = j * RPI + rl;
                const bool ok = id >= 0 && key + r < sp.len && key + r >= lo_all;
                cp_async_16_zfill(dst + swz<ROWB>(gr * 16 + r, cl), ok ? src + (int64_t)(j * RPI) * ts : src0, ok);
              }
            }
          }
        }
        cp_async_commit();
        put = put + 1 == NS ? 0 : put + 1;
      };
#pragma unroll
      for (int i = 0; i < NS; ++i) issue(i);

      if (!q_loaded) {
        q_loaded = true;
        // ---- query rows to shared memory, one warp per row at a time
        for (int r = warp; r < C::kRows; r += kWarps) {
          constexpr int VL = D / 32;  // values per lane
          float x[VL];
          uint32_t raw[(VL + 1) / 2];
          const int rr = row0 + r;
          const int j = rr / a.group, head = h * a.group + rr % a.group;
          if (r < rows) {
            const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(tok0 + j) * a.q_ts +
                                  (int64_t)head * a.q_hs + lane * VL;
            const uint32_t* s32 = reinterpret_cast<const uint32_t*>(src);
#pragma unroll
            for (int i = 0; i < VL / 2; ++i) raw[i] = s32[i];
          } else {
#pragma unroll
            for (int i = 0; i < VL / 2; ++i) raw[i] = 0;
          }
          float mult = a.scale;
          if (F8) {
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < VL / 2; ++i) {
              const float2 f = a.q_bf16 ? unpack2<true>(raw[i]) : unpack2<false>(raw[i]);
              x[2 * i] = f.x;
              x[2 * i + 1] = f.y;
              amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
            // largest magnitude to [2^14, 2^15): all products with codes stay finite
            int e = 0;
            if (a.q_bf16 && amax > 0.f && amax < INFINITY) e = 14 - ilogbf(amax);
#pragma unroll
            for (int i = 0; i < VL / 2; ++i)
              raw[i] = pack2<false>(ldexpf(x[2 * i], e), ldexpf(x[2 * i + 1], e));
            mult *= a.kv.k_scale ? __ldg(a.kv.k_scale + h) : 1.f;
            mult = ldexpf(mult, -e);
          }
          if (lane == 0) s_mult[r] = use_cap ? mult / a.softcap : mult * kLog2e;
#pragma unroll
          for (int i = 0; i < VL / 2; ++i) {
            int d = lane * VL + 2 * i;
            // 8-bit keys come from ldmatrix four codes a lane: dimension 4c+i of a
            // 16-block sits at k index 2c+i (i < 2) or 8+2c+i-2
            if (F8) d = (d & ~15) + ((d & 2) ? 8 : 0) + ((d & 15) >> 2) * 2;
            *reinterpret_cast<uint32_t*>(q_sm + swz<D * 2>(r, d >> 3) + (d & 7) * 2) = raw[i];
          }
        }
        __syncthreads();
      }
      float mult[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mult[mt][0] = s_mult[mt * 16 + g];
        mult[mt][1] = s_mult[mt * 16 + g + 8];
      }

      for (int t = 0; t < sb - sa; ++t) {
        // ---- scores of KS keys
        float s[MT][KS / 8][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < KS / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][i][e] = 0.f;
        cp_async_wait_group<NS - 1>();
        __syncwarp();
        {
          const uint32_t kt = ring_u + get * C::kHalf;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t qa[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              ldsm4(q_u + swz<D * 2>(mt * 16 + (lane & 15), 2 * ks + (lane >> 4)), qa[mt]);
            if (F8) {
              // one matrix: 8 keys x 16 codes; a lane's four codes are its k16 operand pair
#pragma unroll
              for (int kg = 0; kg < KS / 32; ++kg) {
                uint32_t kb[4];
                ldsm4(kt + swz<ROWB>(kg * 32 + lane, ks), kb);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const uint32_t b0 = e4m3x2_to_f16x2((uint16_t)(kb[i] & 0xFFFF));
                  const uint32_t b1 = e4m3x2_to_f16x2((uint16_t)(kb[i] >> 16));
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt) mma16816<MB>(s[mt][kg * 4 + i], qa[mt], b0, b1);
                }
              }
              if (KS == 16) {
                // 16 keys: two matrices of this step and two of the next would fit one
                // load; the second pair is loaded again there instead
                uint32_t kb[4];
                ldsm4(kt + swz<ROWB>(lane & 15, ks), kb);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t b0 = e4m3x2_to_f16x2((uint16_t)(kb[i] & 0xFFFF));
                  const uint32_t b1 = e4m3x2_to_f16x2((uint16_t)(kb[i] >> 16));
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt) mma16816<MB>(s[mt][i], qa[mt], b0, b1);
                }
              }
            } else {
#pragma unroll
              for (int kg = 0; kg < KS / 16; ++kg) {
                uint32_t kb[4];
                ldsm4(kt + swz<ROWB>(kg * 16 + (lane & 7) + ((lane >> 4) << 3),
                                     2 * ks + ((lane >> 3) & 1)), kb);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  mma16816<MB>(s[mt][kg * 2], qa[mt], kb[0], kb[1]);
                  mma16816<MB>(s[mt][kg * 2 + 1], qa[mt], kb[2], kb[3]);
                }
              }
            }
          }
        }
        __syncwarp();
        get = get + 1 == NS ? 0 : get + 1;
        issue(2 * t + NS);

        // ---- log2 scores, masked
        const int tile0 = t * C::kUnit + warp * KS;  // within the sub-range
        const int key0 = (sp.t0 + sa) * C::kUnit + tile0;
        bool whole;  // every key of the tile is seen by every row
        if (listed) {
          bool ok = true;
          if (lane < KS) ok = tab[tile0 + lane] >= 0;
          whole = __all_sync(~0u, ok);
        } else {
          bool ok = true;
#pragma unroll
          for (int gr = 0; gr < KS / 16; ++gr) ok = ok && tab[tile0 / 16 + gr] >= 0;
          whole = ok && key0 + KS <= end0 &&
                  (a.window == 0 || key0 >= end0 + n_tok - 1 - a.window);
        }
        bool raise = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int i = 0; i < KS / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x = s[mt][i][e] * mult[mt][e >> 1];
              if (use_cap) x = a.softcap * kLog2e * tanhf(x);
              s[mt][i][e] = x;
            }
          if (!whole) {
            int end[2], lo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int j = (row0 + mt * 16 + g + 8 * e) / a.group;
              end[e] = end0 + j;
              lo[e] = a.window > 0 ? end[e] - a.window : 0;
            }
#pragma unroll
            for (int i = 0; i < KS / 8; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int kk = i * 8 + 2 * c4 + (e & 1);
                bool seen;
                if (listed) {
                  seen = tab[tile0 + kk] >= 0;
                } else {
                  const int key = key0 + kk;
                  seen = key < end[e >> 1] && key >= lo[e >> 1] && tab[(tile0 + kk) / 16] >= 0;
                }
                if (!seen) s[mt][i][e] = -INFINITY;
              }
          }
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < KS / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[mt][i][e]);
          raise = raise || mx[0] > m[mt][0] + kSlack || mx[1] > m[mt][1] + kSlack;
        }
        if (__any_sync(~0u, raise)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = m[mt][e];
#pragma unroll
              for (int i = 0; i < KS / 8; ++i)
                mx = fmaxf(mx, fmaxf(s[mt][i][2 * e], s[mt][i][2 * e + 1]));
              mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
              mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
              const float f = m[mt][e] == -INFINITY ? 0.f : ex2(m[mt][e] - mx);
              m[mt][e] = mx;
              l[mt][e] *= f;
#pragma unroll
              for (int i = 0; i < D / 8; ++i) {
                o[mt][i][2 * e] *= f;
                o[mt][i][2 * e + 1] *= f;
              }
            }
        }
        uint32_t ph[MT][KS / 16][4], pl[MT][KS / 16][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float m0 = m[mt][0] == -INFINITY ? 0.f : m[mt][0];
          const float m1 = m[mt][1] == -INFINITY ? 0.f : m[mt][1];
#pragma unroll
          for (int i = 0; i < KS / 8; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p0 = ex2(s[mt][i][2 * e] - (e ? m1 : m0));
              const float p1 = ex2(s[mt][i][2 * e + 1] - (e ? m1 : m0));
              l[mt][e] += p0 + p1;
              const uint32_t hi = pack2<MB>(p0, p1);
              const float2 back = unpack2<MB>(hi);
              ph[mt][i / 2][(i & 1) * 2 + e] = hi;
              pl[mt][i / 2][(i & 1) * 2 + e] = pack2<MB>(p0 - back.x, p1 - back.y);
            }
          }
        }

        // ---- weighted sum of the values
        cp_async_wait_group<NS - 1>();
        __syncwarp();
        {
          const uint32_t vt = ring_u + get * C::kHalf;
#pragma unroll
          for (int kg = 0; kg < KS / 16; ++kg)
            if (F8) {
              // a matrix of 8 keys x 16 codes transposed gives a lane the codes of two
              // keys at dimensions 2n, 2n+1: even dimensions feed one product, odd the next
#pragma unroll
              for (int db = 0; db < D / 32; ++db) {
                uint32_t vb[4];
                ldsm4t(vt + swz<ROWB>(kg * 16 + (lane & 15), 2 * db + (lane >> 4)), vb);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const uint32_t w0 = __byte_perm(vb[2 * half], 0, 0x3120);
                  const uint32_t w1 = __byte_perm(vb[2 * half + 1], 0, 0x3120);
                  const uint32_t e0 = e4m3x2_to_f16x2((uint16_t)(w0 & 0xFFFF));
                  const uint32_t e1 = e4m3x2_to_f16x2((uint16_t)(w1 & 0xFFFF));
                  const uint32_t o0 = e4m3x2_to_f16x2((uint16_t)(w0 >> 16));
                  const uint32_t o1 = e4m3x2_to_f16x2((uint16_t)(w1 >> 16));
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt) {
                    const int i = (2 * db + half) * 2;
                    mma16816<MB>(o[mt][i], ph[mt][kg], e0, e1);
                    mma16816<MB>(o[mt][i + 1], ph[mt][kg], o0, o1);
                    mma16816<MB>(o[mt][i], pl[mt][kg], e0, e1);
                    mma16816<MB>(o[mt][i + 1], pl[mt][kg], o0, o1);
                  }
                }
              }
            } else {
#pragma unroll
              for (int db = 0; db < D / 16; ++db) {
                uint32_t vb[4];
                ldsm4t(vt + swz<ROWB>(kg * 16 + (lane & 15), 2 * db + (lane >> 4)), vb);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  mma16816<MB>(o[mt][2 * db], ph[mt][kg], vb[0], vb[1]);
                  mma16816<MB>(o[mt][2 * db + 1], ph[mt][kg], vb[2], vb[3]);
                  mma16816<MB>(o[mt][2 * db], pl[mt][kg], vb[0], vb[1]);
                  mma16816<MB>(o[mt][2 * db + 1], pl[mt][kg], vb[2], vb[3]);
                }
              }
            }
        }
        __syncwarp();
        get = get + 1 == NS ? 0 : get + 1;
        issue(2 * t + 1 + NS);
      }
      cp_async_wait_group<0>();
      __syncwarp();
    }

    // ---- the warps' sums become one: each leaves its own in its ring
    {
      float* buf = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float s = l[mt][e];
          s += __shfl_xor_sync(~0u, s, 1);
          s += __shfl_xor_sync(~0u, s, 2);
          if (c4 == 0) s_ml[warp][mt * 16 + g + 8 * e] = make_float2(m[mt][e], s);
          float* row = buf + (mt * 16 + g + 8 * e) * C::kPitch;
#pragma unroll
          for (int i = 0; i < D / 8; i += 2) {
            if (F8) {
              *reinterpret_cast<float4*>(row + i * 8 + 4 * c4) =
                  make_float4(o[mt][i][2 * e], o[mt][i + 1][2 * e], o[mt][i][2 * e + 1],
                              o[mt][i + 1][2 * e + 1]);
            } else {
              *reinterpret_cast<float2*>(row + i * 8 + 2 * c4) =
                  make_float2(o[mt][i][2 * e], o[mt][i][2 * e + 1]);
              *reinterpret_cast<float2*>(row + i * 8 + 8 + 2 * c4) =
                  make_float2(o[mt][i + 1][2 * e], o[mt][i + 1][2 * e + 1]);
            }
          }
        }
      }
    }
    __syncthreads();
    const bool complete = ta == 0 && tb == units;
    // partial 2c is a CTA's first part, 2c + 1 its last; an item's parts are its
    // first CTA's last (or only) part, then the following CTAs' first parts
    const int part = 2 * (int)blockIdx.x + (u == u0 ? 0 : 1);
    if (a.split && ta == 0 && tid == 0) {
      const long long last = u + units - 1;  // the item's last unit
      const int owner = (int)(((last + 1) * A - 1) / U);
      a.desc[(long long)req * HR + hr] = make_int2(part, owner - (int)blockIdx.x + 1);
    }
    constexpr int QPR = D / 4;  // float4 quads per row
    for (int i = tid; i < rows * QPR; i += kThreads) {
      const int r = i / QPR, d = (i % QPR) * 4;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_ml[w][r].x);
      float lsum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = s_ml[w][r];
        if (ml.x == -INFINITY && ml.y == 0.f) continue;  // the warp saw nothing of this row
        const float f = ml.x == -INFINITY ? 1.f : ex2(ml.x - mx);
        const float4 x = *reinterpret_cast<const float4*>(smem + w * C::kRing + (r * C::kPitch + d) * 4);
        lsum += ml.y * f;
        acc.x += x.x * f;
        acc.y += x.y * f;
        acc.z += x.z * f;
        acc.w += x.w * f;
      }
      if (complete) {
        const int rr = row0 + r;
        const int64_t orow = (int64_t)(tok0 + rr / a.group) * a.Hq + h * a.group + rr % a.group;
        float inv = lsum == 0.f ? 0.f : 1.f / lsum;
        if (F8 && a.kv.v_scale) inv *= __ldg(a.kv.v_scale + h);
        uint2 w;
        if (MB || (F8 && a.q_bf16)) {
          w.x = pack2<true>(acc.x * inv, acc.y * inv);
          w.y = pack2<true>(acc.z * inv, acc.w * inv);
        } else {
          w.x = pack2<false>(acc.x * inv, acc.y * inv);
          w.y = pack2<false>(acc.z * inv, acc.w * inv);
        }
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + d) = w;
        if (a.lse && d == 0) a.lse[orow] = lsum == 0.f ? -INFINITY : (mx + log2f(lsum)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(a.part_o + ((int64_t)part * C::kRows + r) * D + d) = acc;
        if (d == 0)
          *reinterpret_cast<float2*>(a.part_ml + ((int64_t)part * C::kRows + r) * 2) = make_float2(mx, lsum);
      }
    }
    __syncthreads();  // the rings are refilled next

    u += tb - ta;
    if (u - base >= (long long)units * HR) {
      base += (long long)units * HR;
      ++req;
    }
  }
  pdl_launch_dependents();
}

template <int D, int CT, int MT>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
  using C = Cfg<D, CT, MT>;
  static const cudaError_t attr = cudaFuncSetAttribute(
      paged_attn_kernel<D, CT, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (attr != cudaSuccess) return attr;
  return launch_dependent(paged_attn_kernel<D, CT, MT>, dim3(a.grid), dim3(kThreads), C::kSmem,
                          stream, a);
}

template <int CT>
cudaError_t launch_type(const AttnArgs& a, cudaStream_t stream) {
  const bool two = attn_rows_per_item(a.kv.head_dim, a.rows) == 32;
  switch (a.kv.head_dim) {
    case 64: return two ? launch<64, CT, 2>(a, stream) : launch<64, CT, 1>(a, stream);
    case 128: return two ? launch<128, CT, 2>(a, stream) : launch<128, CT, 1>(a, stream);
    default: return launch<256, CT, 1>(a, stream);
  }
}

}  // namespace attn
}  // namespace idx
