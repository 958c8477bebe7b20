// Attention of whole prompts over contiguous keys and values, packed sequences.
//
//   o[t, h] = sum_s p_s v[s] / sum_s p_s,  p_s = exp(scale * q[t, h].k[s]),
//   s over the positions of t's own sequence that t sees.
//
// Work.  A CTA takes 128 or 256 query rows of one kv head: rows are (token, head
// of the group) pairs, tokens outermost, so that the heads of a group share the
// keys that are loaded and a few tokens already fill a tile.  Keys and values
// stream once per CTA through a ring of tiles.  Tiles of a sequence are numbered so
// that no list of them is needed: sequence b's start at floor(query_start[b] / c) + b
// (c tokens a CTA), which leaves at least ceil(n_b / c) numbers to it; CTAs past
// its end leave at once.  Numbers are taken from the end, where causal rows are
// longest, so that short items fill the gaps at the end of the call.
//
// Arithmetic.  S = Q K^T and O += P V are tcgen05 products with fp32 accumulators in
// tensor memory; P (16-bit) takes the place of the scores it was made from.  A
// thread holds one row of S, half a tile at a time.  Weights are 2^(x - m) with a running
// reference m per row, the highest score when it was last raised.  No maximum is taken
// of later scores: their weights' sum tells whether one passes m by too much, and only
// then are they read again, m raised and O rescaled in tensor memory.
// (Comparisons run at half rate: with a maximum before the exponentials a tile's softmax
// took 1280 cycles of latency, and the tensor core waited for it.)
// P is rounded to one 16-bit term: each weight is off by at most 2^-8 (bf16) or 2^-11
// (fp16) of itself, as much as the output's own rounding and less where several keys
// share the weight; a second term would add half of the tensor work again.  Sums of
// weights are fp32 and taken before the rounding.
//
// Bound by the tensor core and the power: 16384 tokens, 32 heads on 8 of 128, causal, 1390 us one
// call after another, 1.58 PFLOP/s (0.82 of the measured burst, 0.90 of the sustained rate); 8192
// tokens 343 us, 1.60, where the tensor pipe is busy 69 % of the time, starts and ends of CTAs
// included (5 us each); head_dim 64 1.12 PFLOP/s, by the hand-overs between the roles, 1000
// cycles a step (a lane for each row tile's products, or no exponentials at all: 0.83 of the
// time at best); head_dim 256 1.54.
//
// A position that a row does not see has weight zero, but zero times an infinity is
// NaN: in tiles where some row's sight begins or ends two warps look through the
// values and set such ones to zero before the product; rows that do see
// them get them added at the end (never the fast path).
//
// Few rows over many keys would leave most SMs idle: then the CTAs of a cluster take a
// part each of the same rows' keys and join them through distributed shared memory, in the
// order of the keys (16 new tokens behind 32768: 37 us, by one CTA each 226).
//
// Roles (384 threads with two row tiles, 256 with one): warps 0-3 and 4-7 the softmax
// of row tile 0 and 1; then a warp whose elected lane issues the products, one that
// loads (TMA, 128-byte swizzle), two that look through values.  Steps n = 0, 1, ... take the
// tiles of keys in turn, for both row tiles one after the other; step n's scores lie in
// place n mod B of tensor memory, its weights over them, and once its product with the
// values is issued the scores of step n + B follow: while one row tile's softmax
// runs, the tensor core works on the other's.  With head_dim 64 there is room for three
// places and no row tile waits for its own products; with 256 the sums of one row
// tile fill half of tensor memory: one row tile, two places.
#pragma once

#include "attn_math.cuh"
#include "common.cuh"
#include "launch.h"
#include "paged_core.cuh"
#include "serving.h"
#include "tcgen05_f16.cuh"
#include "value_types.cuh"

#include <type_traits>

namespace idx {
namespace prompt {

using attn::ex2;
using attn::kCapNear;
using attn::kLn2;

// log2 of the weight that a raise gives the highest score, and of how far weights' sums
// may pass it before the next raise (which costs 2900 cycles).
// fp16: the sum of half a tile; weights must stay below 2^16, and under 2^-24 they are lost.
// bf16: the sum of all weights so far, so that it never exceeds 1/2 and sums of values up to
// 2^127 are finite at any length.  A raise leaves it 2^-15 or more, of which fp32's least step is
// half of bf16's: small values keep what bf16 holds of them.  (Keys of equal scores raise it after
// 16384 of them, then 16384 times as many.  Raises at 2^-1 over 2^-12 instead: 16384 tokens, 32/8
// heads of 128, 1440 us for 1404, head_dim 256 with window and cap 185 for 180.)
template <bool BF16>
constexpr float kLift = BF16 ? -15.f : 3.f;
template <bool BF16>
constexpr float kSlack = BF16 ? 14.f : 12.f;

// mbar_wait (common.cuh) with the limit in cycles of the SM: reading the global timer
// costs as much as a short wait, and every tile waits several times.
constexpr long long kWaitCycles = 2000000000ll;  // about a second
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (mbar_test(bar, parity)) return true;
    if ((it & 15u) == 0) {
      if (*abort) return false;
      if (clock64() - t0 > kWaitCycles) {
        *abort = 1;
        return false;
      }
    }
  }
}

// Which of four barriers' phases of the given parities are over, without waiting, as bits.
// Looked at together: one look takes some 190 cycles while the tensor core reads its operands.
__device__ __forceinline__ uint32_t passed4(const uint32_t (&bar)[4], const uint32_t (&parity)[4]) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q, s, t;\n\t.reg .b32 a, b;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %5;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%2], %6;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 s, [%3], %7;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 t, [%4], %8;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tselp.u32 a, 2, 0, q;\n\tselp.u32 b, 4, 0, s;\n\tor.b32 %0, %0, a;\n\t"
      "selp.u32 a, 8, 0, t;\n\tor.b32 %0, %0, b;\n\tor.b32 %0, %0, a;\n\t}"
      : "=&r"(r)
      : "r"(bar[0]), "r"(bar[1]), "r"(bar[2]), "r"(bar[3]), "r"(parity[0]), "r"(parity[1]), "r"(parity[2]),
        "r"(parity[3])
      : "memory");
  return r;
}

template <int D>
struct Cfg {
  static constexpr int kQ = prompt_row_tiles(D);  // row tiles of a CTA
  static constexpr int kN = kPromptTileKeys;
  static constexpr int kPlaces = D == 64 ? 3 : 2;  // of scores
  static constexpr int kParts = D == 256 ? 2 : 1;  // loads of a tile, of 64 or 128 dimensions
  static constexpr int kDims = D / kParts;
  // Pieces in which a tile's weights are handed over.  Two let the product with the values
  // start while the second is made; with three places nothing waits for it, and one piece
  // saves a barrier's cost (head_dim 64, 8192 tokens: 273 us when it was
  // taken, 286 in two).
  static constexpr int kPieces = kPlaces > 2 ? 1 : 2;
  static constexpr uint32_t kQBytes = 128 * D * 2;
  static constexpr uint32_t kStage = kN * kDims * 2;
  static constexpr int kRoom = 224 * 1024 - kQ * kQBytes;
  static constexpr int kStages = kRoom / (int)kStage < 8 ? kRoom / (int)kStage : 8;
  static constexpr int kSoftmaxWarps = 4 * kQ;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
  // 384 threads are launched with 168 registers each: 216 for a softmax thread's scores, 64
  // for the others (256 * 216 + 128 * 64 <= 384 * 168)
  static constexpr bool kSplitRegs = kQ == 2;
  // tensor memory: scores (and weights in their place), then sums
  static constexpr uint32_t kCols = 512;
  __host__ __device__ static constexpr uint32_t s_col(int place) { return (uint32_t)(place * kN); }
  __host__ __device__ static constexpr uint32_t o_col(int q) { return (uint32_t)(kPlaces * kN + q * D); }
  static_assert(kPlaces * kN + kQ * D <= 512, "");
  static_assert(kStages >= 5, "");
  // shared memory
  static constexpr size_t kKv = kQ * kQBytes;
  static constexpr size_t kBars = kKv + (size_t)kStages * kStage;
  // scores per place; weights and their products per place and half of a tile; full, empty
  // and checked per stage
  enum : int { kQFull = 0, kScores = 2, kWeights = kScores + kPlaces, kSums = kWeights + 2 * kPlaces };
  enum : int { kDrain = kSums + 2 * kPlaces, kFull = kDrain + 1, kEmpty = kFull + kStages };
  enum : int { kChecked = kEmpty + kStages, kNumBars = kChecked + kStages };
  static constexpr size_t kMisc = kBars + 8 * kNumBars;
  static constexpr size_t kSmem = kMisc + 64 + 1024;
  static_assert(kSmem <= 227 * 1024, "");
  static_assert(kQ * 128 * D * 4 <= kStages * (int)kStage, "the sums of a part fit the stages");
};

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// The order of a CTA's loads, tile by tile: as many tiles of keys ahead of the values as the
// places for scores allow, then in turn.
struct Order {
  int tiles, ahead;
  __device__ int keys(int t) const { return t + max(0, t - ahead); }
  __device__ int values(int t) const { return t + min(tiles, t + ahead + 1); }
};

// Keys a row tile sees: tiles [lo, hi); those in [w0, w1) are seen whole by every row.
struct Reach {
  int lo, hi, w0, w1;
  __device__ bool whole(int j) const { return j >= w0 && j < w1; }
};

template <int D, bool BF16, bool CAP>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PromptArgs a) {
  using C = Cfg<D>;
  constexpr int N = C::kN, NQ = C::kQ, ST = C::kStages, NP = C::kPlaces, PARTS = C::kParts;
  uint8_t* sm = aligned_smem_base();
  const uint32_t sq = smem_u32(sm), skv = sq + (uint32_t)C::kKv, bars = sq + (uint32_t)C::kBars;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  auto full_bar = [&](int s) { return bar(C::kFull + s); };
  auto empty_bar = [&](int s) { return bar(C::kEmpty + s); };
  auto checked_bar = [&](int s) { return bar(C::kChecked + s); };
  int* misc = reinterpret_cast<int*>(sm + C::kMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort = misc + 1;
  int* poisoned = misc + 2;
  int* s_seq = misc + 3;
  const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int tid = threadIdx.x;

  // ---- the CTA's sequence, tokens and head
  const int heads = a.Hkv * a.subs, split = a.split;
  const unsigned item = split > 1 ? blockIdx.x / (unsigned)split : blockIdx.x;
  const int rank = split > 1 ? (int)cluster_ctarank() : 0;
  const int hx = (int)(item % (unsigned)heads);
  const int64_t num = a.numbers - 1 - (int64_t)(item / (unsigned)heads);
  const int kvh = hx / a.subs, sub = hx % a.subs;
  const int per_cta = a.row_tiles * a.tile_tokens;
  const int rows = a.tile_tokens * a.pack;
  if (warp == C::kSoftmaxWarps) {
    tmem_alloc(smem_u32(tmem_slot), C::kCols);
    tmem_relinquish();
  } else if (warp == C::kSoftmaxWarps + 1) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  } else if (warp == C::kSoftmaxWarps + 2) {
    for (int i = lane; i < C::kNumBars; i += 32) {
      const bool p = i >= C::kWeights && i < C::kSums;
      mbar_init(bar(i), p ? 4 : (i >= C::kChecked ? 2 : (i >= C::kEmpty ? 3 : 1)));
    }
    if (lane == 0) {
      *abort = 0;
      *poisoned = 0;
    }
    fence_mbar_init();
  } else if (warp == 0) {
    // The sequence that owns this CTA's number, and its starts.  32 at a time are looked at
    // together; with up to 32 sequences that is all.
    pdl_wait();  // inputs may come from the previous kernel
    auto start_of = [&](const int32_t* s, int b, int64_t most) -> int {
      const int x = __ldg(s + b);
      return x < 0 ? 0 : (x > most ? (int)most : x);
    };
    int lo = 0, hi = a.B, at[4] = {0, 0, 0, 0};
    bool found = true;
    while (found) {
      const int step = (hi - lo + 31) / 32, b = lo + lane * step;
      if (b < hi) {
        at[0] = start_of(a.query_start, b, a.T);
        if (step == 1) {
          at[1] = start_of(a.query_start, b + 1, a.T);
          at[2] = start_of(a.key_start, b, a.S);
          at[3] = start_of(a.key_start, b + 1, a.S);
        }
      }
      const unsigned votes = __ballot_sync(~0u, b < hi && at[0] / per_cta + b <= num);
      if (votes == 0) {
        found = false;
      } else {
        const int top = 31 - __clz(votes);
        lo += top * step;
        hi = min(hi, lo + step);
        if (step == 1) {
          // the tokens of the sequence before this CTA's, and the starts
          if (lane == top) {
            const int64_t before = (num - (at[0] / per_cta + lo)) * per_cta;
            s_seq[0] = before < at[1] - at[0] ? (int)before : -1;
#pragma unroll
            for (int i = 0; i < 4; ++i) s_seq[1 + i] = at[i];
          }
          break;
        }
      }
    }
    if (!found && lane == 0) s_seq[0] = -1;
  }
  if (rows < 128) {  // rows of a short tile
    const int words = (128 - rows) * 8;  // 16 bytes each
    for (int i = tid; i < NQ * (D / 64) * words; i += C::kThreads)
      *reinterpret_cast<uint4*>(sm + (i / words) * 16384 + rows * 128 + (i % words) * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  pdl_wait();  // (no one writes before the previous kernel is done with what this one writes)
  if (blockIdx.x == gridDim.x - 1) {  // one of the lightest CTAs looks through the starts
    int bad = 0;
    for (int b = tid; b < a.B; b += C::kThreads) {
      const int q0 = __ldg(a.query_start + b), q1 = __ldg(a.query_start + b + 1);
      const int k0 = __ldg(a.key_start + b), k1 = __ldg(a.key_start + b + 1);
      bad += q0 < 0 || q1 < q0 || q1 > a.T || k0 < 0 || k1 < k0 || k1 > a.S;
    }
    count_bad_input(a.errors, bad);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();  // (the tensor memory is this CTA's before another kernel's may ask for some)
  const uint32_t tmem = __shfl_sync(~0u, *tmem_slot, 0);
  const int t0 = s_seq[0];  // the CTA's first token
  if (t0 < 0) {  // a number that no tokens need
    if (warp == C::kSoftmaxWarps) tmem_dealloc(tmem, C::kCols);
    return;
  }
  const int64_t q0 = s_seq[1], k0 = s_seq[3];
  const int n = s_seq[2] - s_seq[1], nk = max(0, s_seq[4] - s_seq[3]);
  auto load_q = [&](int q) {
    mbar_arrive_expect_tx(bar(C::kQFull + q), (uint32_t)(D / 64 * rows * 128));
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      tma_load_3d(sq + q * C::kQBytes + c * 16384, &tm_q, c * 64, kvh * a.group + sub * a.pack,
                  (int)q0 + t0 + q * a.tile_tokens, bar(C::kQFull + q));
  };
  // The first product waits for these loads: the queries are asked for before what the rows
  // see is worked out, the first keys as soon as it is.
  const bool loader = warp == C::kSoftmaxWarps + 1 && lane == 0;
  if (loader) load_q(0);

  // ---- what each row tile sees
  auto end_of = [&](int t) -> int { return a.causal ? max(0, nk - n + t + 1) : nk; };
  auto low_of = [&](int end) -> int { return a.window > 0 ? max(0, end - a.window) : 0; };
  Reach reach[NQ];
  int jl = INT32_MAX, jh = 0;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int ta = t0 + q * a.tile_tokens, tb = min(n, ta + a.tile_tokens);
    reach[q] = Reach{0, 0, 0, 0};
    if (q >= a.row_tiles || ta >= tb) continue;
    const int e0 = end_of(ta), e1 = end_of(tb - 1), l0 = low_of(e0), l1 = low_of(e1);
    if (e1 == 0) continue;
    reach[q].lo = l0 / N;
    reach[q].hi = (e1 + N - 1) / N;
    reach[q].w0 = (l1 + N - 1) / N;
    reach[q].w1 = e0 / N;
    jl = min(jl, reach[q].lo);
    jh = max(jh, reach[q].hi);
  }
  if (jl > jh) jl = jh;
  if (split > 1) {  // this CTA's part
    const int all = jh - jl;
    jh = jl + all * (rank + 1) / split;
    jl += all * rank / split;
  }
  // Tiles [u0, u1) are seen whole by every row of the CTA; in the others some row's sight
  // may begin or end.
  int u0 = 0, u1 = INT32_MAX;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
    if (reach[q].hi > reach[q].lo) {
      u0 = max(u0, reach[q].w0);
      u1 = min(u1, reach[q].w1);
    }
  auto cut = [&](int j) -> bool { return j < u0 || j >= u1; };

  const int tiles = jh - jl;
  const int two = NQ == 2 && a.row_tiles == 2 && t0 + a.tile_tokens < n;  // whether the second row tile has rows
  const Order order{tiles, (NP - 1) >> two};
  // part c of a tile of keys or values into a stage
  auto load_part = [&](const CUtensorMap* tm, int t, int c, int st) {
    mbar_arrive_expect_tx(full_bar(st), C::kStage);
#pragma unroll
    for (int d = 0; d < C::kDims; d += 64)
      tma_load_3d(skv + (uint32_t)st * C::kStage + d * N * 2, tm, c * C::kDims + d, kvh, (int)k0 + (jl + t) * N,
                  full_bar(st));
  };
  if (loader && tiles > 0) {
#pragma unroll
    for (int c = 0; c < PARTS; ++c) load_part(&tm_k, 0, c, c);
  }

  if (C::kSplitRegs && warp >= C::kSoftmaxWarps) leave_registers<64>();
  if (warp < C::kSoftmaxWarps) {
    // ---------------------------------------------------------- softmax
    if (C::kSplitRegs) take_registers<216>();
    const int q = warp / 4, r = (warp % 4) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp % 4) * 32) << 16);
    // a row's token in its tile: r / pack, exact below 128
    auto token_of = [&](int r) -> int { return r * a.pack_inv >> 16; };
    const int tok = t0 + q * a.tile_tokens + token_of(r), head = r - token_of(r) * a.pack;
    const bool live = q <= two && r < rows && tok < n;
    const int end = live ? end_of(tok) : 0, low = low_of(end);
    const Reach re = reach[q];
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    // (the lanes of a warp go on or leave together)
    auto wait = [&](int which, int count) -> bool {
      return __all_sync(~0u, wait_bar(bar(which), (uint32_t)count & 1, abort));
    };
    constexpr int W = N / C::kPieces;  // scores at a time
    auto step = [&](int i) -> int { return (i << two) + q; };  // of the row tile's i-th tile
    // products of half h of the row tile's i-th tile
    auto sums = [&](int i, int h) -> bool { return wait(C::kSums + 2 * (step(i) % NP) + h, step(i) / NP); };
    const float mult = CAP ? 1.f : a.mult, most = live ? exp2f(kLift<BF16> + kSlack<BF16>) : INFINITY;
    if (!live) m = 0.f;  // its row never asks for a raise
    bool unset = true;   // some row of the warp has no reference yet
    int i = 0;
    for (int j = jl; j < jh && ok && q <= two; ++j, ++i) {
      const int place = step(i) % NP;
      if (!wait(C::kScores + place, step(i) / NP)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool whole = re.whole(j);
      // a piece's scores of the row, in log2 units once multiplied by mult
      auto scores = [&](float(&s)[W], int h) {
#pragma unroll
        for (int c = 0; c < W; c += 32)
          tmem_ld32(lanes + C::s_col(place) + h * W + c, *reinterpret_cast<float(*)[32]>(&s[c]));
        tmem_wait_ld();
        tmem_take(s);
        if (CAP) {
          // the near form by way of the products' own units, its factors times mult:
          // s (f0 + z (f1 + z (f2 + ...))), z = (s / cap)^2.  Where some score of the warp's is past
          // half a cap (one that a row does not see, perhaps another sequence's), those below go by
          // the same operations all the same, so that no score's bits depend on its neighbours.
          float top = 0.f;
#pragma unroll
          for (int c = 0; c < W; ++c) top = fmaxf(top, fabsf(s[c]));
          const float k = a.cap_unit;
          if (__all_sync(~0u, top * k < kCapNear)) {
          const float f0 = a.mult, f1 = attn::kCapNear1 * f0, f2 = attn::kCapNear2 * f0;
          const float f3 = attn::kCapNear3 * f0, f4 = attn::kCapNear4 * f0;
#pragma unroll
            for (int c = 0; c < W; c += 2) {
              const float2 x = make_float2(s[c], s[c + 1]), y = mul2(x, make_float2(k, k)), z = mul2(y, y);
              float2 p = fma2(make_float2(f4, f4), z, make_float2(f3, f3));
              p = fma2(p, z, make_float2(f2, f2));
              p = fma2(p, z, make_float2(f1, f1));
              p = fma2(p, z, make_float2(f0, f0));
              p = mul2(p, x);
              s[c] = p.x;
              s[c + 1] = p.y;
            }
          } else {
#pragma unroll
            for (int c = 0; c < W; ++c) {
              const float f0 = a.mult, f1 = attn::kCapNear1 * f0, f2 = attn::kCapNear2 * f0;
              const float f3 = attn::kCapNear3 * f0, f4 = attn::kCapNear4 * f0;
              const float y = s[c] * k, z = y * y;
              const float near = fmaf(fmaf(fmaf(fmaf(f4, z, f3), z, f2), z, f1), z, f0) * s[c];
              const float far = fmaf(__fdividef(-2.f, 1.f + ex2(2.f * attn::kLog2e * fabsf(y))), a.cap_log2, a.cap_log2);
              s[c] = fabsf(y) < kCapNear ? near : copysignf(far, y);
            }
          }
        }
        if (!whole) {
          const int to = end - j * N - h * W, from = low - j * N - h * W;
          auto below = [](int x) -> uint32_t { return x >= 32 ? ~0u : (x <= 0 ? 0u : (1u << x) - 1); };
#pragma unroll
          for (int g = 0; g < W; g += 32) {
            const uint32_t seen = below(to - g) & ~below(from - g);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(seen >> c & 1)) s[g + c] = -INFINITY;
          }
        }
      };
      // 2^(s mult + ref), rounded, and their sum before that
      auto weights = [&](const float(&s)[W], float ref, uint32_t(&p)[W / 2]) -> float {
        float2 part[4] = {};
#pragma unroll
        for (int c = 0; c < W; c += 2) {
          const float2 t = fma2(make_float2(s[c], s[c + 1]), make_float2(mult, mult), make_float2(ref, ref));
          const float2 y = make_float2(ex2(t.x), ex2(t.y));
          part[(c / 2) & 3] = add2(part[(c / 2) & 3], y);
          p[c / 2] = pack2<BF16>(y.x, y.y);
        }
        part[0] = add2(add2(part[0], part[1]), add2(part[2], part[3]));
        return part[0].x + part[0].y;
      };
      auto store = [&](uint32_t at, const uint32_t(&p)[W / 2]) {
#pragma unroll
        for (int c = 0; c < W / 2; c += 16) tmem_st16(at + c, *reinterpret_cast<const uint32_t(*)[16]>(&p[c]));
      };
#pragma unroll
      for (int h = 0; h < C::kPieces; ++h) {
        const uint32_t at_p = lanes + C::s_col(place) + h * (W / 2);
        bool slow = false;
        if (unset) slow = unset = __any_sync(~0u, m == -INFINITY);  // a row without a reference
        if (!slow) {
          float s[W];
          scores(s, h);
          uint32_t p[W / 2];
          const float room = BF16 ? most - l : most;  // (known before the sum is)
          const float sum = weights(s, -m, p);
          slow = __any_sync(~0u, sum > room);
          if (!slow) {
            l += sum;
            store(at_p, p);
          }
        }
        if (slow) {
          // ---- the reference is raised: scores once more, for their maximum and by the new one
          float s[W];
          scores(s, h);
          float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c < W; ++c) top[c & 3] = fmaxf(top[c & 3], s[c]);
          const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * mult;
          float up = live ? fmaxf(mx - kLift<BF16>, m) : m;
          // (half a tile's new weights sum to 2^(lift + 7) at most; so may the earlier ones)
          if (BF16 && live && l > exp2f(kLift<BF16> + 7.f)) up = fmaxf(up, m + __log2f(l) - kLift<BF16>);
          const float w = m == -INFINITY ? 0.f : ex2(m - up);
          if (i + h > 0) {
            if (!(h ? sums(i, 0) : sums(i - 1, C::kPieces - 1))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tmem_ld16(lanes + C::o_col(q) + c, o);
              tmem_wait_ld();
              tmem_take(o);
              // (a row that has seen nothing yet has sums of zero)
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = m == -INFINITY ? 0.f : o[e] * w;
              tmem_st16(lanes + C::o_col(q) + c, *reinterpret_cast<const uint32_t(*)[16]>(&o[0]));
            }
          }
          m = up;
          uint32_t p[W / 2];
          l = l * w + weights(s, m == -INFINITY ? 0.f : -m, p);
          store(at_p, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kWeights + 2 * place + h));
      }
    }
    float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t head0 = (int64_t)kvh * a.group + sub * a.pack;
    if (split == 1 && live && a.lse)
      a.lse[(q0 + tok) * a.Hq + head0 + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    asm volatile("" : "+f"(inv));  // (made while the last product runs)
    // without tiles the queries were loaded all the same, to where the rows go
    if (ok) ok = i > 0 ? sums(i - 1, C::kPieces - 1) : q > 0 || wait(C::kQFull, 0);
    if (!ok && lane == 0) flag_timeout(a.errors, kTimeoutEpilogue);
    const bool fix = *reinterpret_cast<volatile int*>(poisoned) != 0;
    // infinities and NaN that were kept out of the products, dimensions c ..
    auto mend = [&](float* o, auto n, int c) {
#pragma unroll 1
      for (int j = jl; j < jh; ++j) {
        if (!cut(j)) continue;
        for (int key = max(low, j * N); key < min(end, (j + 1) * N); ++key) {
          const uint16_t* v = static_cast<const uint16_t*>(a.v) + (k0 + key) * a.v_ts + kvh * a.v_hs + c;
#pragma unroll
          for (int e = 0; e < decltype(n)::value; e += 2) {
            const float2 x = unpack2<BF16>((uint32_t)v[e] | (uint32_t)v[e + 1] << 16);
            if (!(fabsf(x.x) < INFINITY)) o[e] += x.x;
            if (!(fabsf(x.y) < INFINITY)) o[e + 1] += x.y;
          }
        }
      }
    };
    if (split > 1) {
      // ---- the parts are joined: every CTA's references and weights, its sums by the joint
      // ones in fp32, then each CTA adds up a share of the rows
      if (!ok) l = 0.f;
      uint8_t* stats = sm + q * C::kQBytes;  // (the row tile's queries are done with)
      *reinterpret_cast<float2*>(stats + r * 8) = make_float2(l == 0.f ? -INFINITY : m, l);
      cluster_sync_all();
      // the highest reference and the sum of weights of row r of tile q
      auto joint = [&](int q, int r) -> float2 {
        float top = -INFINITY, sum = 0.f;
        for (int k = 0; k < split; ++k)
          top = fmaxf(top, ld_cluster_f2(cluster_map(sq + q * C::kQBytes + r * 8, k)).x);
        for (int k = 0; k < split; ++k) {
          const float2 x = ld_cluster_f2(cluster_map(sq + q * C::kQBytes + r * 8, k));
          if (x.y != 0.f) sum += x.y * (x.x == top ? 1.f : ex2(x.x - top));
        }
        return make_float2(top, sum);
      };
      const uint32_t sums_sm = (uint32_t)C::kKv;  // 16-byte chunks of a row, XORed with it
      if (q <= two) {
        const float2 all = joint(q, r);
        const float f = l == 0.f ? 0.f : (m == all.x ? 1.f : ex2(m - all.x)) / all.y;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          if (i > 0 && ok) {
            tmem_ld32(lanes + C::o_col(q) + c, o);
            tmem_wait_ld();
            tmem_take(o);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0.f : o[e] * f;
          if (fix && live) mend(o, std::integral_constant<int, 32>(), c);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(sm + sums_sm + (q * 128 + r) * D * 4 + ((((c + e) / 4) ^ (r & 7)) << 4)) =
                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      cluster_sync_all();
      for (int y = rank * C::kSoftmaxWarps + warp; y < 128 << two; y += split * C::kSoftmaxWarps) {
        const int yq = y >> 7, yr = y & 127, tk = token_of(yr), t = t0 + yq * a.tile_tokens + tk;
        if (yr >= rows || t >= n) continue;
        const int64_t row = (q0 + t) * a.Hq + head0 + yr - tk * a.pack;
#pragma unroll
        for (int x = lane; x < D / 4; x += 32) {
          const uint32_t at = sq + sums_sm + (uint32_t)(y * D * 4 + ((x ^ (yr & 7)) << 4));
          uint4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < split) v[k] = ld_cluster_v4(cluster_map(at, k));
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < split) {
              s.x += __uint_as_float(v[k].x);
              s.y += __uint_as_float(v[k].y);
              s.z += __uint_as_float(v[k].z);
              s.w += __uint_as_float(v[k].w);
            }
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + x * 4) =
              make_uint2(pack2<BF16>(s.x, s.y), pack2<BF16>(s.z, s.w));
        }
        if (a.lse && lane == 0) {
          const float2 all = joint(yq, yr);
          a.lse[row] = all.y == 0.f ? -INFINITY : (all.x + log2f(all.y)) * kLn2;
        }
      }
      cluster_sync_all();  // no CTA leaves while others read its shared memory
    } else if (ok) {
      // ---- the row's sums leave
      tc_fence_after();
      // By way of the row tile's queries' place in shared memory (its products are done), so
      // that whole rows are stored together: a lane storing its own row took 5000 cycles.
      uint8_t* rows_sm = sm + q * C::kQBytes;
      auto place_of = [&](int r, int c) -> uint8_t* {  // 16-byte chunk c of row r
        return rows_sm + (c / 8) * 16384 + r * 128 + (((c ^ r) & 7) << 4);
      };
      constexpr int OC = 64;
      const bool none = __any_sync(~0u, l == 0.f);  // a row of the warp saw nothing
#pragma unroll 1
      for (int c = 0; c < D; c += OC) {
        float o[OC];
        if (i > 0) {
#pragma unroll
          for (int e = 0; e < OC; e += 32)
            tmem_ld32(lanes + C::o_col(q) + c + e, *reinterpret_cast<float(*)[32]>(&o[e]));
          tmem_wait_ld();
          tmem_take(o);
        }
#pragma unroll
        for (int e = 0; e < OC; ++e) o[e] *= inv;
        if (none) {
#pragma unroll
          for (int e = 0; e < OC; ++e) o[e] = l == 0.f ? 0.f : o[e];
        }
        if (fix && live) mend(o, std::integral_constant<int, OC>(), c);
#pragma unroll
        for (int e = 0; e < OC; e += 8)
          *reinterpret_cast<uint4*>(place_of(r, (c + e) / 8)) = pack8<BF16>(*reinterpret_cast<const float(*)[8]>(&o[e]));
      }
      __syncwarp();
      constexpr int LR = D / 8, RI = 32 / LR;  // lanes per row, rows at a time
      const int mine = live ? (tok - t0) * a.Hq + head : -1;  // this lane's row, counted from the CTA's first
      uint16_t* out = static_cast<uint16_t*>(a.out) + ((q0 + t0) * a.Hq + head0) * D + lane % LR * 8;
      constexpr int G = 32 / RI < 8 ? 32 / RI : 8;  // loads in flight
#pragma unroll 1
      for (int x = lane / LR; x < 32; x += G * RI) {
        uint4 v[G];
        int at[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
          at[g] = __shfl_sync(~0u, mine, x + g * RI);
          v[g] = *reinterpret_cast<const uint4*>(place_of((warp % 4) * 32 + x + g * RI, lane % LR));
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (at[g] >= 0) *reinterpret_cast<uint4*>(out + (int64_t)at[g] * D) = v[g];
      }
    }
  } else if (warp == C::kSoftmaxWarps) {
    // ---------------------------------------------------------- products
    // One lane; loads are taken in the order in which they were made.
    if (elect_one()) {
      constexpr uint32_t qk_pos = f16_idesc(N, BF16, false, false), qk_neg = f16_idesc(N, BF16, false, true);
      constexpr uint32_t pv = f16_idesc(C::kDims, BF16, true, false);
      constexpr uint32_t high = desc_high(1024, kLayoutSw128);
      const uint32_t qk = a.neg ? qk_neg : qk_pos;
      auto wait = [&](int which, uint32_t parity) -> bool { return wait_bar(bar(which), parity, abort); };
      // Places, stages and their parities are stepped, not divided out: what this lane
      // computes between two products the tensor core may have to wait for.
      struct Ring {
        int at = 0;
        uint32_t ph = 0;
        __device__ void step(int by, int size) {
          at += by;
          if (at >= size) {
            at -= size;
            ph ^= 1;
          }
        }
      };
      Ring ks, vs, sp, vp;  // stages of keys and values, places of scores and weights
      vs.step(min(tiles, order.ahead + 1) * PARTS % ST, ST);
      const uint32_t al = desc_low(sq, 16);
      int kt = 0, vt = 0;  // tiles
      // `ready`: the barriers were seen passed already
      auto scores = [&](int q, bool ready) -> bool {
#pragma unroll
        for (int c = 0; c < PARTS; ++c) {
          Ring k = ks;
          k.step(c, ST);
          if (q == 0 && !ready && !wait(C::kFull + k.at, k.ph)) return false;
          const uint32_t bl = desc_low(skv + k.at * C::kStage, 16);
#pragma unroll
          for (int e = 0; e < C::kDims / 16; ++e)
            mma_f16_ss(tmem + C::s_col(sp.at), al + q * (C::kQBytes / 16) + ((c * C::kDims / 64 + e / 4) * 16384 + (e % 4) * 32) / 16,
                       bl + ((e / 4) * N * 128 + (e % 4) * 32) / 16, high, qk, c + e > 0);
          if (q == two) mma_commit(empty_bar(k.at));
        }
        mma_commit(bar(C::kScores + sp.at));
        sp.step(1, NP);
        if (q == two) ks.step(PARTS * (++kt <= order.ahead ? 1 : 2), ST);
        return true;
      };
      // the barrier of part c of the tile's values: loaded, and checked where some row's sight is cut
      auto values_bar = [&](const Ring& v) -> int { return (cut(jl + vt) ? C::kChecked : C::kFull) + v.at; };
      auto products = [&]() -> bool {
        int left = tiles << two;  // scores to issue
        for (int i = 0; i < NP && left > 0; ++i, --left) {
          if (i <= two && !wait(C::kQFull + i, 0)) return false;
          if (!scores(i & two, false)) return false;
        }
        // row tiles take turns
        for (int n = 0; n < tiles << two; ++n) {
          const int q = n & two, next = (n + NP) & two;
          // the step's barriers: weights, values (and their second part), the next scores' keys
          // (whose second part is waited for)
          const int wb = C::kWeights + 2 * vp.at;
          Ring v1 = vs;
          v1.step(1, ST);
          const uint32_t bars4[4] = {bar(wb), C::kPieces > 1 ? bar(wb + 1) : bar(values_bar(v1)),
                                     bar(values_bar(vs)), bar(C::kFull + ks.at)};
          const uint32_t par4[4] = {vp.ph, C::kPieces > 1 ? vp.ph : v1.ph, vs.ph, ks.ph};
          const uint32_t seen = passed4(bars4, par4);
          const bool w0 = seen & 1, w1 = seen & 2, kr = PARTS == 1 && (seen & 8);
          if (q == 0) {
            if (!(seen & 4) && !wait(values_bar(vs), vs.ph)) return false;
            if (PARTS > 1 && !wait(values_bar(v1), v1.ph)) return false;
          }
#pragma unroll
          for (int h = 0; h < C::kPieces; ++h) {
            if (!(h ? w1 : w0) && !wait(C::kWeights + 2 * vp.at + h, vp.ph)) return false;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < PARTS; ++c) {
              Ring v = vs;
              v.step(c, ST);
              const uint32_t bl = desc_low(skv + v.at * C::kStage, N * 128);
#pragma unroll
              for (int k = h * (N / 16 / C::kPieces); k < (h + 1) * (N / 16 / C::kPieces); ++k)
                mma_f16_ts(tmem + C::o_col(q) + c * C::kDims, tmem + C::s_col(vp.at) + 8 * k, bl + k * 2048 / 16,
                           high, pv, vt > 0 || k > 0);
            }
            mma_commit(bar(C::kSums + 2 * vp.at + h));
          }
          vp.step(1, NP);
          if (q == two) {
#pragma unroll
            for (int c = 0; c < PARTS; ++c) {
              Ring v = vs;
              v.step(c, ST);
              mma_commit(empty_bar(v.at));
            }
            ++vt;
            vs.step(PARTS * (vt + order.ahead < tiles ? 2 : 1), ST);
          }
          if (left > 0) {
            if (!scores(next, kr)) return false;
            --left;
          }
        }
        return true;
      };
      if (!products()) flag_timeout(a.errors, kTimeoutMma);
      mma_commit(bar(C::kDrain));
      if (!mbar_wait_drain(bar(C::kDrain), 0)) flag_timeout(a.errors, kTimeoutDrain);
    }
    __syncwarp();
  } else if (warp == C::kSoftmaxWarps + 1) {
    // ---------------------------------------------------------- loads
    if (lane == 0) {
      int at = PARTS;  // (the first tile of keys is on its way)
      auto load = [&](const CUtensorMap* tm, int t) -> bool {
#pragma unroll
        for (int c = 0; c < PARTS; ++c, ++at) {
          const int st = at % ST;
          if (!wait_bar(empty_bar(st), ((uint32_t)(at / ST) & 1) ^ 1, abort)) return false;
          load_part(tm, t, c, st);
        }
        return true;
      };
      bool ok = true;
      if (two && tiles > 0) load_q(1);
      for (int t = 1; t <= order.ahead && t < tiles; ++t) ok = ok && load(&tm_k, t);
      for (int t = 0; t < tiles && ok; ++t) {
        ok = load(&tm_v, t);
        if (t + order.ahead + 1 < tiles) ok = ok && load(&tm_k, t + order.ahead + 1);
      }
      if (!ok) flag_timeout(a.errors, kTimeoutProducer);
      // nothing of the CTA's may be in flight when it leaves
      if (tiles == 0) at = 0;
      for (int q = 0; q <= (tiles > 0 ? two : 0); ++q)
        if (!mbar_wait_drain(bar(C::kQFull + q), 0)) flag_timeout(a.errors, kTimeoutDrain);
      for (int i = at > ST ? at - ST : 0; i < at; ++i)
        if (!mbar_wait_drain(full_bar(i % ST), (uint32_t)(i / ST) & 1)) flag_timeout(a.errors, kTimeoutDrain);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- values that are not finite
    // Every load passes here, so that a stage is neither refilled before these warps
    // have seen it nor taken for its next filling.
    const int half = warp - C::kSoftmaxWarps - 2;
    int t = 0;  // the next tile of values
    for (int at = 0; at < 2 * tiles * PARTS; ++at) {
      const int st = at % ST;
      if (!__all_sync(~0u, wait_bar(full_bar(st), (uint32_t)(at / ST) & 1, abort))) break;
      const bool values = at / PARTS == order.values(t);
      if (values && cut(jl + t)) {
        uint8_t* tile = sm + C::kKv + (size_t)st * C::kStage + half * (C::kStage / 2);
        // the largest magnitudes' bits tell: infinities and NaN lie above every number
        uint32_t top[2] = {0, 0};
#pragma unroll 8
        for (int i = lane; i < (int)C::kStage / 32; i += 32) {
          const uint4 x = *reinterpret_cast<const uint4*>(tile + i * 16);
          top[0] = __vmaxu2(top[0], x.x & 0x7FFF7FFFu);
          top[1] = __vmaxu2(top[1], x.y & 0x7FFF7FFFu);
          top[0] = __vmaxu2(top[0], x.z & 0x7FFF7FFFu);
          top[1] = __vmaxu2(top[1], x.w & 0x7FFF7FFFu);
        }
        if (not_finite16<BF16>(top[0]) || not_finite16<BF16>(top[1])) {
#pragma unroll 1
          for (int i = lane; i < (int)C::kStage / 32; i += 32) {
            uint16_t* p = reinterpret_cast<uint16_t*>(tile + i * 16);
#pragma unroll 1
            for (int e = 0; e < 8; ++e)
              if (not_finite16<BF16>(p[e])) p[e] = 0;
          }
          *reinterpret_cast<volatile int*>(poisoned) = 1;
          fence_proxy_async_smem();
          __threadfence_block();
        }
      }
      if (values && at % PARTS == PARTS - 1) ++t;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(checked_bar(st));
        mbar_arrive(empty_bar(st));
      }
    }
  }

  if (split > 1 && warp >= C::kSoftmaxWarps) {  // (the join's barriers)
    cluster_sync_all();
    cluster_sync_all();
    cluster_sync_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kSoftmaxWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int D, bool BF16, bool CAP>
cudaError_t launch(const CUtensorMap* tm, const PromptArgs& a, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kern = prompt_attn_kernel<D, BF16, CAP>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.numbers * a.Hkv * a.subs * a.split));
  if (a.split > 1)
    return launch_dependent_cluster(kern, grid, dim3(C::kThreads), C::kSmem, stream, (unsigned)a.split, tm[0],
                                    tm[1], tm[2], a);
  return launch_dependent(kern, grid, dim3(C::kThreads), C::kSmem, stream, tm[0], tm[1], tm[2], a);
}

template <int D, bool BF16>
cudaError_t launch_cap(const CUtensorMap* tm, const PromptArgs& a, cudaStream_t stream) {
  return a.cap_unit > 0.f ? launch<D, BF16, true>(tm, a, stream) : launch<D, BF16, false>(tm, a, stream);
}

template <bool BF16>
cudaError_t launch_type(int D, const CUtensorMap* tm, const PromptArgs& a, cudaStream_t stream) {
  switch (D) {
    case 64: return launch_cap<64, BF16>(tm, a, stream);
    case 128: return launch_cap<128, BF16>(tm, a, stream);
    default: return launch_cap<256, BF16>(tm, a, stream);
  }
}

}  // namespace prompt
}  // namespace idx
