// Attention of a few new tokens over a paged key-value cache.
//
// Work.  An item is one kv head of one request with its query rows (next_n
// tokens times the heads of the group; with a selection, one token's group),
// up to 8 * NT of them.  An item is taken whole by a team of W = 8, 4, 2 or 1
// warps, their order left to the hardware: long items by eight warps, short ones by
// few, so that some teams of an SM set items up while others stream.  Where that would leave SMs idle (few or long items; the caller
// estimates both) the items are split: their keys are cut into units of 8 * KS
// (64 KB of cache for most shapes), numbered item by item over the whole batch,
// and the units into segments (see Cut).  With R resident CTAs the first R segments take
// three quarters of the units, one segment per CTA; the rest are cut into
// levels of R segments of 1/8, 1/16, ... that the CTAs claim from a counter as
// they finish: with equal shares alone the first CTA was done after 614 us and
// the last after 817 (64 requests of 8K - 32K keys), as CTAs stream at
// different rates; 817 became 705.  Which units form a segment depends on the
// lengths alone, so results do not depend on the order in which CTAs run.  A
// segment that holds an item whole writes its result; an item that spans
// segments leaves one partial (running maximum, weight, weighted sum) per
// segment in the workspace and a second, dependent launch joins them in the
// order of their keys.
//
// Arithmetic.  o = sum_s p_s v_s / sum_s p_s with p_s = 2^(x_s - m), one pass
// with a running reference m per row that is raised (and the sums rescaled)
// only when a score passes the highest at the last raise by more than 2^8, which
// fp32 sums hold easily: most tiles need one vote instead of shuffle reductions.
// Scores and sums are fp32 accumulators of m16n8k16 products.  Up to eight rows:
// keys (then value dimensions) on M, query rows on N, so that eight rows fill a
// tile: S^T = K Q^T, then O^T = V^T P^T, P passing from one product's result layout to the
// other's operand layout by a register transpose (movmatrix).  More rows: query
// rows on M.  p goes into the second product as two 16-bit terms, hi = round(p)
// and lo = round(p - hi): one term's rounding (2^-9 in bf16) would be as large
// as the rounding of the output itself.  8-bit codes are exact in fp16; queries
// are then brought to fp16 by a power of two per row, which loses nothing of a
// bf16 value within 2^-29 of the row's largest.  4-bit codes (E2M1, one power of two 2^e
// per 32 dimensions) are exact in both types: keys in fp16, a block's part of a score
// times its key's 2^e in fp32 after the products over the block; values in bf16, the
// weights' terms times 2^e before the product (exact, bf16 having fp32's range; values from
// scale byte 0 up to 2^54 leave room for the weights').
//
// Memory.  2 G flops per byte of cache (G query heads per kv head) is far
// below the tensor pipes' ridge, so the kernel is built as a stream: each of
// the CTA's eight warps owns KS keys of every unit and a private ring of
// half stages (KS keys' K or V rows, 16-byte cp.async, XOR-swizzled for
// ldmatrix); no barrier stands between warps until the item ends.  Rows that
// no query sees are zero-filled, never read, so whatever a page holds past the
// context (NaN included) cannot reach a sum.
//
// Measured (one call, new inputs in turn): 64 requests of 8K - 32K keys, 32/8
// heads of 128, bf16, 5.2 GB: 724 us, 7.19 TB/s; 64 x 2048 selected positions
// (0.54 GB) 86 us, 6.3 TB/s, items whole by four warps each (split and joined
// 94).  Rows gathered one by one take 0.92 of the copy rate at 256 bytes, 0.95 at
// 512, 0.70 - 0.74 at 128.  The tensor pipe is 13 - 15 % busy with up to eight rows, 50 % with sixteen over an E4M3 cache; it binds
// from 32 rows over an E4M3 cache on (0.53 of the copy rate).  Over 4-bit values the
// way from codes to operands binds: 64 requests of 20480 keys 383 us, 0.55 of the copy rate, the
// issue slots 72 % and the logic pipe 59 % busy (476 instructions for 16 keys of 128 dimensions, half
// of them on that way, in chains that 16 warps an SM do not hide); selected positions by two places gathered a row, codes and scales.
#pragma once

#include <float.h>

#include "attn_math.cuh"
#include "common.cuh"
#include "launch.h"
#include "paged_core.cuh"
#include "serving.h"
#include "value_types.cuh"

namespace idx {
namespace attn {

constexpr int kWarps = 8;
constexpr int kTab = 2048;  // words of the table of resolved page groups / listed positions
constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr float kSlack = 8.f;  // log2 of how far a score may pass the highest at the last raise
// log2 of the weight that a raise gives the highest score: with fp16 operands as
// high as their range allows (2^15 after the slack), since what lies under 2^-25
// is lost: 2^-32 of the highest weight and less.  Over 4-bit values 2^32, so that the second
// term of a weight times a scale byte's 2^-127 is still a normal number, and 2^31 keys' weights of
// up to 2^40 times values of 2^54 are finite (brought back when the sums leave).
template <bool PB, bool F4 = false>
constexpr float kLift = F4 ? 32.f : (PB ? 0.f : 7.f);
constexpr float kLiftDown = 2.3283064365386963e-10f;  // 2^-32

template <int D, int CT>
constexpr int row_bytes() { return attn_row_bytes(D, CT); }  // of codes or values
// shared memory of a key's scale bytes (4-bit codes; copies are of at least 4 bytes)
template <int D, int CT>
__host__ __device__ constexpr int scale_room() { return CT != IDX_MXFP4 ? 0 : D == 64 ? 4 : D / 32; }

// W warps (a team) share an item.  A CTA is one team; where rows of at most 128
// bytes are gathered one by one and a team is less than eight warps, it is all the
// teams of an SM, of neighbouring heads, whose rows lie close together: 64 x 2048
// selected from an E4M3 cache 56 us, as CTAs of one team 66; of head_dim 64 53 and
// 63, from a 4-bit one 80 and 95 (rows of 256 bytes 87 and 86; contexts, whose lengths differ, gain by single
// teams: 128 of 100 - 250 keys 14.9, two teams a CTA 16.7).
template <int D, int CT, int NT, bool listed, int W>
struct Cfg {
  static_assert(W == kWarps || W == 4 || W == 2 || W == 1, "");
  static constexpr bool kF8 = CT == IDX_E4M3, kF4 = CT == IDX_MXFP4;
  static constexpr bool kMmaBf16 = CT == IDX_BF16;
  static constexpr int kRowB = row_bytes<D, CT>();
  // keys per warp and unit: 4 KB half stages where rows are short and the sums
  // leave room for 32 keys' scores
  static constexpr int kKS = attn_keys_per_tile(D, CT, NT, W);
  static constexpr int kUnit = W * kKS;
  static constexpr int kRows = 8 * NT;
  static constexpr int kHalf = (kRowB + scale_room<D, CT>()) * kKS;  // bytes of a half stage
  // two CTAs per SM where 128 registers a thread hold the accumulators
  static constexpr int kOcc = attn_occupancy(D, CT, NT);
  static constexpr int kPitch = W < kWarps ? D : D + 4;  // floats of a row of the merge buffer
  static constexpr int kSums = kRows * kPitch * 4;
  static constexpr int kTeams = listed && kRowB <= 128 && W < kWarps ? kOcc * kWarps / W : 1;
  static constexpr int kThreads = 32 * W * kTeams;
  static constexpr int kCtas = kOcc * kWarps / (W * kTeams);  // resident per SM
  static constexpr int kQBytes = kRows * D * 2;
  // words of a team's table; halved for four and two warps, whose stream then starts
  // after one round of loads (64 x 2048 selected from an E4M3 cache 56 us, else 61)
  static constexpr int kTabWords = (W == 2 || W == 4 ? kTab / 2 : kTab) * W / kWarps;
  // a warp's ring: 12 KB, of a small team 8 (16 rows, 64 x 2048 selected 94 us, with
  // 12 KB 104; 8 rows 87 and 89; 64 contexts of 100 - 500 15.4 and 16.1), with one CTA
  // an SM twice that, or what the query rows leave
  static constexpr int kMost = (W == kWarps ? 12288 : 8192) * (kOcc == 2 ? 1 : 2);
  static constexpr int kRoom = (222 * 1024 / kCtas / kTeams - kQBytes - kTabWords * 4) / W;
  static constexpr int kStages = (kRoom < kMost ? kRoom : kMost) / kHalf;
  static constexpr int kRing = kStages * kHalf > kSums ? kStages * kHalf : kSums;
  static constexpr int kSmem = kTeams * (W * kRing + kQBytes + kTabWords * 4);
  static_assert(kSums <= kRing, "a warp's sums fit its ring");
  static_assert(kStages >= 2 && kRing % 16 == 0, "");
  static_assert(kSmem * kCtas <= 222 * 1024, "");
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(full ? 16 : 0)
               : "memory");
}
template <int N>  // 4 or 8 bytes
__device__ __forceinline__ void cp_async_few_zfill(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(full ? N : 0)
               : "memory");
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
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
// An 8 x 8 matrix of 16-bit values held two to a lane, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
// Shared-memory offset of 16-byte chunk c of row r: the chunk index is XORed
// with the row so that eight rows' equal chunks lie in eight bank groups
// (64-byte rows: two rows per 128 bytes, 32-byte rows four).
template <int ROWB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if (ROWB >= 128) return (uint32_t)(r * ROWB + ((c ^ (r & 7)) << 4));
  if (ROWB == 32) return (uint32_t)(r * ROWB + ((c ^ ((r >> 2) & 1)) << 4));
  return (uint32_t)(r * ROWB + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ int warp_incl_sum(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// An item costs its units and about as much time again as kSetup of them: query
// rows, table, first loads, the sums of eight warps.  Cuts weigh it so, the
// setup first.
constexpr int kSetup = 3;

// The cut of U units (setups counted) into segments by R CTAs.  One level of A = min(R, U)
// equal segments, or K + 1 levels of R: 3/4 of the units, then 1/8, 1/16, ...,
// 2^-(K+1), 2^-(K+1), as far as the smallest segments keep kMinSegment units.
// Segments weigh whole 2^-(K+1) / R parts of the units, the first `rem` parts
// one unit more than the others.
//
// With one level (few units a CTA) segments are first tried along the items:
// every item in pieces of q units, at most R pieces in all, q from the equal
// share up to about a quarter more.  A piece lies in one item, so no CTA sets a
// second one up.
constexpr int kMinSegment = 5;
struct Cut {
  int R, K, U, part, rem;
  __device__ Cut(int units, int ctas) : R(ctas), K(0), U(units) {
#pragma unroll
    for (int k = 2; k < kAttnLevels; ++k)
      if (U >> (k + 1) >= kMinSegment * R) K = k;
    if (K == 0 && R > U) R = U;
    const int parts = K == 0 ? R : R << (K + 1);
    part = U / parts;
    rem = U - part * parts;
  }
  __device__ int segments() const { return R * (K + 1); }
  // parts of one segment of level l, and of all segments before level l (per CTA)
  __device__ int weight(int l) const { return l == 0 ? (K == 0 ? 1 : 3 << (K - 1)) : (l < K ? 1 << (K - 1 - l) : 1); }
  __device__ int before(int l) const { return l == 0 ? 0 : (2 << K) - (1 << (K - l)); }
  // first unit of segment s (s = segments(): U)
  __device__ int start(int s) const {
    const int l = s / R;
    if (l > K) return U;
    const int x = R * before(l) + (s - l * R) * weight(l);
    return x * part + min(x, rem);
  }
  // the segment that holds unit u
  __device__ int owner(int u) const {
    const int x = u < rem * (part + 1) ? u / (part + 1) : rem + (u - rem * (part + 1)) / part;
    int l = 0;
    while (l < K && x >= R * before(l + 1)) ++l;
    return l * R + (x - R * before(l)) / weight(l);
  }
};

// A request as an item sees it.
struct Span {
  int len;    // clamped context
  int t0;     // first unit of its keys
  int units;  // units (at least one, so that an empty request's rows are written)
};

// What a tile's masking goes by: key kk of the tile (keys key0 ..) is seen by
// row r where the table has its place and, of a whole context, where it lies in
// [end_r - window, end_r).
template <bool listed>
struct Sight {
  const uint32_t* tab;  // of the sub-range
  const int* end;       // per row of the item, in shared memory
  int tile0, key0, window;
  __device__ __forceinline__ bool there(int kk) const {
    return tab[listed ? tile0 + kk : (tile0 + kk) / 16] != kNone;
  }
  __device__ __forceinline__ bool in(int kk, int r) const {
    const int key = key0 + kk, e = end[r];
    return listed || (key < e && (window == 0 || key >= e - window));
  }
};

// Whether one of a word's packed values is infinite or NaN (E4M3: NaN).
template <int CT>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  if (CT == IDX_E4M3)  // a byte of all ones but the sign: the byte sum carries into its sign place
    return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
  return not_finite16<CT == IDX_BF16>(w);
}

// Keys that some of an item's rows see and others do not: a weight of zero times an
// infinite or NaN value would be NaN, so a tile's such values become zeros, and
// marks[row][dimension] says which sums of the rows that see them are to be NaN.
// The keys are [lo0, lo1), past the later tokens' windows, and [hi0, hi1), the later
// tokens' own: fewer than n_tok each, looked through 16 bytes a lane.  Calls of several
// tokens pay 0 - 6 % for it (64 contexts of 100 - 500 keys, 2 tokens 13.6 -> 14.2 us,
// 64 of 1000 - 8000, 4 tokens, E4M3 111 -> 113); with the NaN set in the sums
// themselves, the tile's keys taken one by one, 14.2 and 119; rows done again after a
// sum that is not finite 14.4 and 126 (registers that must then outlive the stream).
// In kernels of its own: as a branch of one kernel it cost calls of one token up to 6 %.
template <int D, int CT, int ROWS>
__device__ __forceinline__ void keep_apart(uint8_t* vt, const Sight<false>& v, int lo0, int lo1, int hi0,
                                           int hi1, uint32_t (*marks)[D / 32], int* marked, int lane) {
  constexpr int ROWB = D * (CT == IDX_E4M3 ? 1 : 2), CH = ROWB / 16;
  const int lows = max(0, lo1 - lo0), n = lows + max(0, hi1 - hi0);
  auto row_of = [&](int i) -> int { return (i < lows ? lo0 + i : hi0 + i - lows) - v.key0; };
  bool bad = false;
#pragma unroll 1
  for (int c = lane; c < n * CH; c += 32) {
    const uint4 x = *reinterpret_cast<const uint4*>(vt + swz<ROWB>(row_of(c / CH), c % CH));
    bad = bad || not_finite<CT>(x.x) || not_finite<CT>(x.y) || not_finite<CT>(x.z) || not_finite<CT>(x.w);
  }
  if (!__any_sync(~0u, bad)) return;
#pragma unroll 1
  for (int i = lane; i < n * D; i += 32) {
    const int kk = row_of(i / D), d = i % D, at = d * (CT == IDX_E4M3 ? 1 : 2);
    uint8_t* p = vt + swz<ROWB>(kk, at >> 4) + (at & 15);
    const uint32_t x = CT == IDX_E4M3 ? *p : *reinterpret_cast<uint16_t*>(p);
    if (!not_finite<CT>(x)) continue;
    if (CT == IDX_E4M3) *p = 0; else *reinterpret_cast<uint16_t*>(p) = 0;
    *marked = 1;
#pragma unroll 1
    for (int r = 0; r < ROWS; ++r)
      if (v.in(kk, r)) atomicOr(&marks[r][d / 32], 1u << (d % 32));
  }
  __syncwarp();
}

// The scale bytes of a key's blocks [4 w, 4 w + 4) (head_dim 64: both its bytes).
template <int D>
__device__ __forceinline__ uint32_t scale_word(uint32_t scales, int key, int w) {
  return D == 64 ? lds16(scales + key * 2) : lds32(scales + key * (D / 32) + 4 * w);
}
// 2^e of a word's byte b (of a byte of 0: zero, such a block of a key counts as zeros).
__device__ __forceinline__ float scale_of(uint32_t w, int b) {
  return __uint_as_float((b < 3 ? w << (23 - 8 * b) : w >> 1) & 0x7F800000u);
}
// 2^e of byte b of two keys' words, in bf16.
__device__ __forceinline__ uint32_t scales_of(uint32_t w0, uint32_t w1, int b) {
  uint32_t r;
  const uint16_t two = (uint16_t)__byte_perm(w0, w1, (uint32_t)(b | (b + 4) << 4));
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"(two));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Of a word with four codes of one key below four of another: the pairs of the same
// place, in bf16.  A code's three low bits moved to a bf16's bits 6 - 8 are 2^-126 of its
// value (the least of them a subnormal number); its sign is six places further up, so one
// multiplication by 65 moves both (products run beside the logic operations, which bind).
// A product with 2^126 gives the value itself: left to the sums, the factor would cost the small
// values their bits there (64 contexts of 20480 keys 365 us, 383 with it: those of 2^-64 came short of
// some, from 2^-87 on they were zero.  A power of two per block of dimensions that follows the
// scale bytes as the reference follows the scores: 376, and small values beside large ones still lost).
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t (&v)[4]) {
  constexpr uint32_t keep = 0x81C081C0u, up = 0x7E807E80u;  // 2^126
  const uint32_t u = w >> 8;
  v[0] = mul_bf16x2(((w & 0x000F000Fu) * (65u << 6)) & keep, up);
  v[1] = mul_bf16x2(((w & 0x00F000F0u) * (65u << 2)) & keep, up);
  v[2] = mul_bf16x2(((u & 0x000F000Fu) * (65u << 6)) & keep, up);
  v[3] = mul_bf16x2(((u & 0x00F000F0u) * (65u << 2)) & keep, up);
}
// The scale words of N keys for two blocks' worth of code chunks (c2), loaded once for
// every four blocks.
template <int D, int N, class Key>
__device__ __forceinline__ void scale_words(uint32_t (&w)[N], uint32_t scales, int c2, Key key) {
  if (c2 % 2 != 0) return;
#pragma unroll
  for (int j = 0; j < N; ++j) w[j] = scale_word<D>(scales, key(j), c2 / 2);
}
// d = a b, sums from zero.
template <bool BF16>
__device__ __forceinline__ void mma16816_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// A tile's scale bytes before they are used: those of keys that no row sees become
// zero (their codes are zero, but a page may hold any byte there, and zero times infinity
// is NaN); selected keys of head_dim 64, copied with a neighbour's, are put in place.
template <int D, bool listed>
__device__ __forceinline__ void settle_scales(uint8_t* scales, const Sight<listed>& v, int keys, int lo, int len,
                                              bool clear, int lane) {
  constexpr int SB = D / 32;
  const bool mine = lane < keys;
  bool seen = true;
  uint32_t two = 0;
  if (mine) {
    seen = v.there(lane) && (listed || (v.key0 + lane < len && v.key0 + lane >= lo));
    if (listed && D == 64)
      two = *reinterpret_cast<const uint32_t*>(scales + 4 * lane) >> (v.tab[v.tile0 + lane] & 1 ? 16 : 0);
  }
  __syncwarp();
  if (mine && D == 64) {
    if (listed) *reinterpret_cast<uint16_t*>(scales + 2 * lane) = clear && !seen ? 0 : (uint16_t)two;
    else if (clear && !seen) *reinterpret_cast<uint16_t*>(scales + 2 * lane) = 0;
  } else if (mine && clear && !seen) {
#pragma unroll
    for (int i = 0; i < SB / 4; ++i) *reinterpret_cast<uint32_t*>(scales + SB * lane + 4 * i) = 0;
  }
  __syncwarp();
}

// Two weights of one row pair or key pair, as the fp16/bf16 term and the rest.
template <bool MB>
__device__ __forceinline__ void two_terms(float p0, float p1, uint32_t* hi, uint32_t* lo) {
  *hi = pack2<MB>(p0, p1);
  const float2 back = unpack2<MB>(*hi);
  *lo = pack2<MB>(p0 - back.x, p1 - back.y);
}

// One warp's running sums over its tiles, for at most eight query rows: keys
// (then value dimensions) on M, rows on N.  A lane holds keys g, g + 8 of a
// 16-key group and rows 2 c4, 2 c4 + 1.
template <int D, int CT, int KS>
struct KeysOnM {
  static constexpr bool F8 = CT == IDX_E4M3, F4 = CT == IDX_MXFP4;
  static constexpr bool MB = CT == IDX_BF16, PB = MB || F4;  // the first and second product in bf16
  static constexpr int ROWB = row_bytes<D, CT>();
  static constexpr bool kQRegs = D <= 128;  // query operands stay in registers
  float o[D / 16][4], s[KS / 16][4], m[2], l[2];
  uint32_t qf[kQRegs ? D / 8 : 1];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }
  __device__ __forceinline__ void load_q(uint32_t q_u, int lane) {
    if (!kQRegs) return;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t r[4];
      ldsm4(q_u + swz<D * 2>(lane & 7, 4 * i + (lane >> 3)), r);
#pragma unroll
      for (int j = 0; j < 4; ++j) qf[4 * i + j] = r[j];
    }
  }
  __device__ __forceinline__ void scores(uint32_t kt, uint32_t q_u, int lane) {
#pragma unroll
    for (int kg = 0; kg < KS / 16; ++kg)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[kg][e] = 0.f;
    if constexpr (F4) {
#pragma unroll
      for (int kg = 0; kg < KS / 16; ++kg) {
        uint32_t w[2];
#pragma unroll
        for (int c2 = 0; c2 < D / 64; ++c2) {  // two blocks of 32 dimensions at a time
          // a lane's eight codes of a key are its operand values of two k16 steps
          uint32_t r[4];
          ldsm4(kt + swz<ROWB>(kg * 16 + (lane & 15), 2 * c2 + (lane >> 4)), r);
          scale_words<D>(w, kt + KS * ROWB, c2, [&](int j) { return kg * 16 + 8 * j + (lane >> 2); });
#pragma unroll
          for (int bl = 0; bl < 2; ++bl) {
            uint32_t ka[2][4], x[4], y[4];
            e2m1x8_to_f16x2(r[2 * bl], x);
            e2m1x8_to_f16x2(r[2 * bl + 1], y);
            float t[4];
            uint32_t qb[4];
            if (kQRegs) {
#pragma unroll
              for (int j = 0; j < 4; ++j) qb[j] = qf[kQRegs ? 4 * (2 * c2 + bl) + j : 0];
            } else {
              ldsm4(q_u + swz<D * 2>(lane & 7, 4 * (2 * c2 + bl) + (lane >> 3)), qb);
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              ka[ks][0] = x[2 * ks];
              ka[ks][1] = y[2 * ks];
              ka[ks][2] = x[2 * ks + 1];
              ka[ks][3] = y[2 * ks + 1];
              if (ks == 0) mma16816_new<MB>(t, ka[ks], qb[2 * ks], qb[2 * ks + 1]);
              else mma16816<MB>(t, ka[ks], qb[2 * ks], qb[2 * ks + 1]);
            }
            const int by = D == 64 ? bl : (2 * c2 + bl) % 4;
            const float f0 = scale_of(w[0], by), f1 = scale_of(w[1], by);
            s[kg][0] = fmaf(t[0], f0, s[kg][0]);
            s[kg][1] = fmaf(t[1], f0, s[kg][1]);
            s[kg][2] = fmaf(t[2], f1, s[kg][2]);
            s[kg][3] = fmaf(t[3], f1, s[kg][3]);
          }
        }
      }
    } else {
#pragma unroll
    for (int k2 = 0; k2 < D / 32; ++k2) {  // 32 dimensions at a time
      uint32_t qb[4];
      if (kQRegs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) qb[j] = qf[4 * k2 + j];
      } else {
        ldsm4(q_u + swz<D * 2>(lane & 7, 4 * k2 + (lane >> 3)), qb);
      }
#pragma unroll
      for (int kg = 0; kg < KS / 16; ++kg) {
        uint32_t ka[2][4];
        if (F8) {
          // one matrix: 8 keys x 16 codes; a lane's four codes are its operand
          // values of both halves of a k16 step
          uint32_t r[4];
          ldsm4(kt + swz<ROWB>(kg * 16 + (lane & 15), 2 * k2 + (lane >> 4)), r);
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              ka[ks][hf] = e4m3x2_to_f16x2((uint16_t)(r[2 * ks + hf] & 0xFFFF));
              ka[ks][2 + hf] = e4m3x2_to_f16x2((uint16_t)(r[2 * ks + hf] >> 16));
            }
        } else {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
            ldsm4(kt + swz<ROWB>(kg * 16 + (lane & 15), 4 * k2 + 2 * ks + (lane >> 4)), ka[ks]);
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) mma16816<MB>(s[kg], ka[ks], qb[2 * ks], qb[2 * ks + 1]);
      }
    }
    }
  }
  __device__ __forceinline__ void cap(float c, float inv, const float* mult, int lane) {
    const float2 f = *reinterpret_cast<const float2*>(mult + 2 * (lane & 3));
    float most = 0.f;
#pragma unroll
    for (int kg = 0; kg < KS / 16; ++kg)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[kg][e] *= e & 1 ? f.y : f.x;
        most = fmaxf(most, fabsf(s[kg][e]));
      }
    if (__all_sync(~0u, most * inv < kCapNear)) {
#pragma unroll
      for (int kg = 0; kg < KS / 16; ++kg)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[kg][e] = capped_near(s[kg][e], inv);
    } else {
#pragma unroll
      for (int kg = 0; kg < KS / 16; ++kg)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[kg][e] = capped(s[kg][e], c, inv);
    }
  }
  template <bool LISTED>
  __device__ __forceinline__ void mask(const Sight<LISTED>& v, int lane) {
    const int g = lane >> 2, c4 = lane & 3;
#pragma unroll
    for (int kg = 0; kg < KS / 16; ++kg)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int kk = kg * 16 + hf * 8 + g;
        const bool there = v.there(kk);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!there || !v.in(kk, 2 * c4 + e)) s[kg][2 * hf + e] = -INFINITY;
      }
  }
  // Reference raised where needed, weights, and their product with the values.
  // Log2 scores are s * mult.
  __device__ __forceinline__ void values(uint32_t vt, float2 mult, int lane) {
    const float f[2] = {mult.x, mult.y};
    float mx[2];
    bool raise = false;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = fmaxf(s[0][e], s[0][2 + e]);
#pragma unroll
      for (int kg = 1; kg < KS / 16; ++kg) x = fmaxf(x, fmaxf(s[kg][e], s[kg][2 + e]));
      mx[e] = x * f[e];
      raise = raise || mx[e] > m[e] + (kLift<PB, F4> + kSlack);
    }
    if (__any_sync(~0u, raise)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(mx[e] - kLift<PB, F4>, m[e]);
        x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
        x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
        x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
        const float w = m[e] == -INFINITY ? 0.f : ex2(m[e] - x);
        m[e] = x;
        l[e] *= w;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[i][e] *= w;
          o[i][2 + e] *= w;
        }
      }
    }
    const float r0 = m[0] == -INFINITY ? 0.f : -m[0], r1 = m[1] == -INFINITY ? 0.f : -m[1];
#pragma unroll
    for (int kg = 0; kg < KS / 16; ++kg) {
      uint32_t ph[2], pl[2];  // the weights in the second product's operand layout
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float p0 = ex2(fmaf(s[kg][2 * hf], f[0], r0));
        const float p1 = ex2(fmaf(s[kg][2 * hf + 1], f[1], r1));
        l[0] += p0;
        l[1] += p1;
        uint32_t hi, lo;
        two_terms<PB>(p0, p1, &hi, &lo);
        ph[hf] = transpose8x8(hi);
        pl[hf] = transpose8x8(lo);
      }
      if constexpr (F4) {
        // a matrix of 8 keys x 32 codes transposed gives a lane two keys' codes at
        // dimensions 4g .. 4g + 3: rows g and g + 8 of two operands
        uint32_t w[4];
#pragma unroll
        for (int c2 = 0; c2 < D / 64; ++c2) {
          uint32_t r[4];
          ldsm4t(vt + swz<ROWB>(kg * 16 + (lane & 15), 2 * c2 + (lane >> 4)), r);
          scale_words<D>(w, vt + KS * ROWB, c2,
                         [&](int j) { return kg * 16 + 2 * (lane & 3) + (j & 1) + (j & 2) * 4; });
#pragma unroll
          for (int bl = 0; bl < 2; ++bl) {
            const int by = D == 64 ? bl : (2 * c2 + bl) % 4;
            const uint32_t f0 = scales_of(w[0], w[1], by), f1 = scales_of(w[2], w[3], by);
            const uint32_t h0 = mul_bf16x2(ph[0], f0), h1 = mul_bf16x2(ph[1], f1);
            const uint32_t l0 = mul_bf16x2(pl[0], f0), l1 = mul_bf16x2(pl[1], f1);
            uint32_t x[4], y[4];
            code_pairs(r[2 * bl], x);
            code_pairs(r[2 * bl + 1], y);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t va[4] = {x[2 * hf], x[2 * hf + 1], y[2 * hf], y[2 * hf + 1]};
              const int i = 4 * c2 + 2 * bl + hf;
              mma16816<PB>(o[i], va, h0, h1);
              mma16816<PB>(o[i], va, l0, l1);
            }
          }
        }
      } else if (F8) {
        // a matrix of 8 keys x 16 codes transposed gives a lane two keys' codes at
        // dimensions 2g, 2g+1: the even one is row g of the operand, the odd g + 8
#pragma unroll
        for (int db = 0; db < D / 32; ++db) {
          uint32_t r[4];
          ldsm4t(vt + swz<ROWB>(kg * 16 + (lane & 15), 2 * db + (lane >> 4)), r);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t va[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w = __byte_perm(r[2 * hf + j], 0, 0x3120);
              va[2 * j] = e4m3x2_to_f16x2((uint16_t)(w & 0xFFFF));
              va[2 * j + 1] = e4m3x2_to_f16x2((uint16_t)(w >> 16));
            }
            mma16816<MB>(o[2 * db + hf], va, ph[0], ph[1]);
            mma16816<MB>(o[2 * db + hf], va, pl[0], pl[1]);
          }
        }
      } else {
#pragma unroll
        for (int db = 0; db < D / 16; ++db) {
          uint32_t va[4];
          ldsm4t(vt + swz<ROWB>(kg * 16 + (lane & 7) + ((lane >> 4) << 3),
                                2 * db + ((lane >> 3) & 1)), va);
          mma16816<MB>(o[db], va, ph[0], ph[1]);
          mma16816<MB>(o[db], va, pl[0], pl[1]);
        }
      }
    }
  }
  // This lane's factors of the rows it holds.
  __device__ __forceinline__ float2 factors(const float* mult, int lane) const {
    return *reinterpret_cast<const float2*>(mult + 2 * (lane & 3));
  }
  __device__ __forceinline__ void leave(float* buf, int pitch, float2* ml, int rows, int lane) {
    const int g = lane >> 2, c4 = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * c4 + e;
      float x = l[e];
      x += __shfl_xor_sync(~0u, x, 4);
      x += __shfl_xor_sync(~0u, x, 8);
      x += __shfl_xor_sync(~0u, x, 16);
      if (r < rows) {
        if (g == 0) ml[r] = F4 ? make_float2(m[e] + kLift<PB, F4>, x * kLiftDown) : make_float2(m[e], x);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          if (F4) {
            if (i % 2 == 0)
              *reinterpret_cast<float4*>(buf + r * pitch + i * 16 + 4 * g) =
                  make_float4(o[i][e] * kLiftDown, o[i][2 + e] * kLiftDown, o[(i + 1) % (D / 16)][e] * kLiftDown,
                              o[(i + 1) % (D / 16)][2 + e] * kLiftDown);
          } else if (F8) {
            *reinterpret_cast<float2*>(buf + r * pitch + i * 16 + 2 * g) = make_float2(o[i][e], o[i][2 + e]);
          } else {
            buf[r * pitch + i * 16 + g] = o[i][e];
            buf[r * pitch + i * 16 + 8 + g] = o[i][2 + e];
          }
        }
      }
    }
  }
};

// The same for 16 * MT rows, which fill M themselves: S = Q K^T, O = P V, and
// P is already in the second product's operand layout.  A lane holds rows g,
// g + 8 of a tile and keys 2 c4, 2 c4 + 1 of each group of eight.  (Keys on M
// cost these 12 % more time: a transpose for every eight weights.)
template <int D, int CT, int KS, int MT>
struct RowsOnM {
  static constexpr bool F8 = CT == IDX_E4M3, F4 = CT == IDX_MXFP4;
  static constexpr bool MB = CT == IDX_BF16, PB = MB || F4;  // the first and second product in bf16
  static constexpr int ROWB = row_bytes<D, CT>();
  float o[MT][D / 8][4], s[MT][KS / 8][4], m[MT][2], l[MT][2];

  struct Factors {
    float f[MT][2];
  };
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }
  }
  __device__ __forceinline__ void load_q(uint32_t, int) {}
  __device__ __forceinline__ void scores(uint32_t kt, uint32_t q_u, int lane) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < KS / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][i][e] = 0.f;
    if constexpr (F4) {
      uint32_t w[KS / 4];  // of keys 2 c4, 2 c4 + 1 of each group of eight
#pragma unroll
      for (int c2 = 0; c2 < D / 64; ++c2) {
        scale_words<D>(w, kt + KS * ROWB, c2, [&](int j) { return j / 2 * 8 + 2 * (lane & 3) + j % 2; });
        uint32_t r[KS / 16][4];
#pragma unroll
        for (int kg = 0; kg < KS / 16; ++kg)
          ldsm4(kt + swz<ROWB>(kg * 16 + (lane & 15), 2 * c2 + (lane >> 4)), r[kg]);
#pragma unroll
        for (int bl = 0; bl < 2; ++bl) {
          uint32_t qa[2][MT][4];
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              ldsm4(q_u + swz<D * 2>(mt * 16 + (lane & 15), 4 * (2 * c2 + bl) + 2 * ks + (lane >> 4)), qa[ks][mt]);
          const int by = D == 64 ? bl : (2 * c2 + bl) % 4;
#pragma unroll
          for (int kg = 0; kg < KS / 16; ++kg)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float f0 = scale_of(w[4 * kg + 2 * n], by), f1 = scale_of(w[4 * kg + 2 * n + 1], by);
              uint32_t x[4];
              e2m1x8_to_f16x2(r[kg][2 * bl + n], x);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                float t[4];
                mma16816_new<MB>(t, qa[0][mt], x[0], x[1]);
                mma16816<MB>(t, qa[1][mt], x[2], x[3]);
                float(&d)[4] = s[mt][2 * kg + n];
                d[0] = fmaf(t[0], f0, d[0]);
                d[1] = fmaf(t[1], f1, d[1]);
                d[2] = fmaf(t[2], f0, d[2]);
                d[3] = fmaf(t[3], f1, d[3]);
              }
            }
        }
      }
    } else {
#pragma unroll
    for (int k2 = 0; k2 < D / 32; ++k2) {
      uint32_t qa[2][MT][4];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          ldsm4(q_u + swz<D * 2>(mt * 16 + (lane & 15), 4 * k2 + 2 * ks + (lane >> 4)), qa[ks][mt]);
#pragma unroll
      for (int kg = 0; kg < KS / 16; ++kg) {
        uint32_t kb[2][4];  // per k16 step: operand pairs of two groups of eight keys
        if (F8) {
          uint32_t r[4];
          ldsm4(kt + swz<ROWB>(kg * 16 + (lane & 15), 2 * k2 + (lane >> 4)), r);
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              kb[ks][2 * n] = e4m3x2_to_f16x2((uint16_t)(r[2 * ks + n] & 0xFFFF));
              kb[ks][2 * n + 1] = e4m3x2_to_f16x2((uint16_t)(r[2 * ks + n] >> 16));
            }
        } else {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
            ldsm4(kt + swz<ROWB>(kg * 16 + (lane & 7) + ((lane >> 4) << 3),
                                 4 * k2 + 2 * ks + ((lane >> 3) & 1)), kb[ks]);
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < 2; ++n)
              mma16816<MB>(s[mt][2 * kg + n], qa[ks][mt], kb[ks][2 * n], kb[ks][2 * n + 1]);
      }
    }
    }
  }
  __device__ __forceinline__ Factors factors(const float* mult, int lane) const {
    Factors f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) f.f[mt][e] = mult[mt * 16 + (lane >> 2) + 8 * e];
    return f;
  }
  __device__ __forceinline__ void cap(float c, float inv, const float* mult, int lane) {
    const Factors f = factors(mult, lane);
    float most = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < KS / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[mt][i][e] *= f.f[mt][e >> 1];
          most = fmaxf(most, fabsf(s[mt][i][e]));
        }
    if (__all_sync(~0u, most * inv < kCapNear)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < KS / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][i][e] = capped_near(s[mt][i][e], inv);
    } else {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < KS / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][i][e] = capped(s[mt][i][e], c, inv);
    }
  }
  template <bool LISTED>
  __device__ __forceinline__ void mask(const Sight<LISTED>& v, int lane) {
    const int g = lane >> 2, c4 = lane & 3;
#pragma unroll
    for (int i = 0; i < KS / 8; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int kk = i * 8 + 2 * c4 + k;
        const bool there = v.there(kk);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!there || !v.in(kk, mt * 16 + g + 8 * e)) s[mt][i][2 * e + k] = -INFINITY;
      }
  }
  __device__ __forceinline__ void values(uint32_t vt, const Factors& f, int lane) {
    float mx[MT][2];
    bool raise = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(s[mt][0][2 * e], s[mt][0][2 * e + 1]);
#pragma unroll
        for (int i = 1; i < KS / 8; ++i) x = fmaxf(x, fmaxf(s[mt][i][2 * e], s[mt][i][2 * e + 1]));
        mx[mt][e] = x * f.f[mt][e];
        raise = raise || mx[mt][e] > m[mt][e] + (kLift<PB, F4> + kSlack);
      }
    if (__any_sync(~0u, raise)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(mx[mt][e] - kLift<PB, F4>, m[mt][e]);
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 2));
          const float w = m[mt][e] == -INFINITY ? 0.f : ex2(m[mt][e] - x);
          m[mt][e] = x;
          l[mt][e] *= w;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[mt][i][2 * e] *= w;
            o[mt][i][2 * e + 1] *= w;
          }
        }
    }
#pragma unroll
    for (int kg = 0; kg < KS / 16; ++kg) {
      uint32_t ph[MT][4], pl[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float r = m[mt][e] == -INFINITY ? 0.f : -m[mt][e];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float p0 = ex2(fmaf(s[mt][2 * kg + n][2 * e], f.f[mt][e], r));
            const float p1 = ex2(fmaf(s[mt][2 * kg + n][2 * e + 1], f.f[mt][e], r));
            l[mt][e] += p0 + p1;
            two_terms<PB>(p0, p1, &ph[mt][2 * n + e], &pl[mt][2 * n + e]);
          }
        }
      if constexpr (F4) {
        // dimensions 4n .. 4n + 3 of a 32-block feed four products
        uint32_t w[4];
#pragma unroll
        for (int c2 = 0; c2 < D / 64; ++c2) {
          uint32_t r[4];
          ldsm4t(vt + swz<ROWB>(kg * 16 + (lane & 15), 2 * c2 + (lane >> 4)), r);
          scale_words<D>(w, vt + KS * ROWB, c2,
                         [&](int j) { return kg * 16 + 2 * (lane & 3) + (j & 1) + (j & 2) * 4; });
#pragma unroll
          for (int bl = 0; bl < 2; ++bl) {
            const int by = D == 64 ? bl : (2 * c2 + bl) % 4;
            const uint32_t f[2] = {scales_of(w[0], w[1], by), scales_of(w[2], w[3], by)};
            uint32_t x[4], y[4];
            code_pairs(r[2 * bl], x);
            code_pairs(r[2 * bl + 1], y);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t ha[4], la[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                ha[j] = mul_bf16x2(ph[mt][j], f[j / 2]);
                la[j] = mul_bf16x2(pl[mt][j], f[j / 2]);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                mma16816<PB>(o[mt][4 * (2 * c2 + bl) + j], ha, x[j], y[j]);
                mma16816<PB>(o[mt][4 * (2 * c2 + bl) + j], la, x[j], y[j]);
              }
            }
          }
        }
      } else if (F8) {
        // dimensions 2n, 2n + 1 of a 16-block: even ones feed one product, odd the next
#pragma unroll
        for (int db = 0; db < D / 32; ++db) {
          uint32_t r[4];
          ldsm4t(vt + swz<ROWB>(kg * 16 + (lane & 15), 2 * db + (lane >> 4)), r);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t w0 = __byte_perm(r[2 * hf], 0, 0x3120);
            const uint32_t w1 = __byte_perm(r[2 * hf + 1], 0, 0x3120);
            const uint32_t e0 = e4m3x2_to_f16x2((uint16_t)(w0 & 0xFFFF));
            const uint32_t e1 = e4m3x2_to_f16x2((uint16_t)(w1 & 0xFFFF));
            const uint32_t o0 = e4m3x2_to_f16x2((uint16_t)(w0 >> 16));
            const uint32_t o1 = e4m3x2_to_f16x2((uint16_t)(w1 >> 16));
            const int i = (2 * db + hf) * 2;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16816<MB>(o[mt][i], ph[mt], e0, e1);
              mma16816<MB>(o[mt][i + 1], ph[mt], o0, o1);
              mma16816<MB>(o[mt][i], pl[mt], e0, e1);
              mma16816<MB>(o[mt][i + 1], pl[mt], o0, o1);
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
            mma16816<MB>(o[mt][2 * db], ph[mt], vb[0], vb[1]);
            mma16816<MB>(o[mt][2 * db + 1], ph[mt], vb[2], vb[3]);
            mma16816<MB>(o[mt][2 * db], pl[mt], vb[0], vb[1]);
            mma16816<MB>(o[mt][2 * db + 1], pl[mt], vb[2], vb[3]);
          }
        }
      }
    }
  }
  __device__ __forceinline__ void leave(float* buf, int pitch, float2* ml, int rows, int lane) {
    const int g = lane >> 2, c4 = lane & 3;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mt * 16 + g + 8 * e;
        float x = l[mt][e];
        x += __shfl_xor_sync(~0u, x, 1);
        x += __shfl_xor_sync(~0u, x, 2);
        if (r < rows) {
          if (c4 == 0)
            ml[r] = F4 ? make_float2(m[mt][e] + kLift<PB, F4>, x * kLiftDown) : make_float2(m[mt][e], x);
          float* row = buf + r * pitch;
#pragma unroll
          for (int i = 0; i < D / 8; i += 2) {
            if (F4) {
              // columns 2 c4, 2 c4 + 1 of four products: eight dimensions in turn
              const int f = i & ~3, k = (i & 2) / 2;
              *reinterpret_cast<float4*>(row + f * 8 + 8 * c4 + 4 * k) =
                  make_float4(o[mt][f][2 * e + k] * kLiftDown, o[mt][f + 1][2 * e + k] * kLiftDown,
                              o[mt][f + 2][2 * e + k] * kLiftDown, o[mt][f + 3][2 * e + k] * kLiftDown);
            } else if (F8) {
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
};

template <int D, int CT, int NT, int KS>
struct TileOf {
  using type = RowsOnM<D, CT, KS, NT / 2>;
};
template <int D, int CT, int KS>
struct TileOf<D, CT, 1, KS> {
  using type = KeysOnM<D, CT, KS>;
};

// several: more than one new token a request, whose sights differ (whole contexts)
template <int D, int CT, int NT, bool listed, int W, bool several>
__global__ void __launch_bounds__((Cfg<D, CT, NT, listed, W>::kThreads), (Cfg<D, CT, NT, listed, W>::kCtas))
paged_attn_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<D, CT, NT, listed, W>;
  constexpr bool F8 = C::kF8, F4 = C::kF4, MB = C::kMmaBf16;
  constexpr int KS = C::kKS, ROWB = C::kRowB, NS = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int s_warp[W], s_pieces[W][4], s_lasts[C::kTeams][W];
  __shared__ int s_base, s_req, s_seg;
  __shared__ uint32_t s_marks[several ? C::kRows : 1][D / 32];  // see keep_apart
  __shared__ int s_marked;
  // log2 score per product, and ones for capped scores
  __shared__ __align__(8) float s_mults[C::kTeams][C::kRows], s_one[C::kRows];
  __shared__ int s_ends[C::kTeams][C::kRows];  // first key past a row's sight
  __shared__ float2 s_mls[C::kTeams][W][C::kRows];
  constexpr int TT = 32 * W;
  // the team, and this thread's and warp's place in it
  const int team = (int)threadIdx.x / TT, tid = (int)threadIdx.x % TT, lane = tid & 31, warp = tid >> 5;
  auto sync = [&]() {
    if (W == 1) __syncwarp();
    else if (C::kTeams == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(TT) : "memory");
  };
  float* s_mult = s_mults[team];
  int* s_end = s_ends[team];
  int* s_last = s_lasts[team];
  float2(*s_ml)[C::kRows] = s_mls[team];
  uint8_t* rings = smem + team * (W * C::kRing);
  uint8_t* ring = rings + warp * C::kRing;
  const uint32_t ring_u = smem_u32(ring);
  uint8_t* q_sm = smem + C::kTeams * (W * C::kRing) + team * C::kQBytes;
  const uint32_t q_u = smem_u32(q_sm);
  uint32_t* tab = reinterpret_cast<uint32_t*>(smem + C::kTeams * (W * C::kRing + C::kQBytes)) +
                  team * C::kTabWords;
  // offsets into k and v: one table where both have the same strides
  uint32_t* vtab = a.one_table ? tab : tab + C::kTabWords / 2;
  const int tab_words = a.one_table ? C::kTabWords : C::kTabWords / 2;

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

  const int reqs = listed ? a.B * a.next_n : a.B;
  const int list_units = (a.topk + C::kUnit - 1) / C::kUnit;
  int U = 0;  // below 2^31, as the caller has checked
  const bool split = W == kWarps && a.split;
  if (split) {
    if (listed) {
      U = reqs * HR * (list_units + kSetup);
    } else {
      int sum = 0;
      for (int b = tid; b < reqs; b += TT) sum += span_of(b).units + kSetup;
      sum = warp_incl_sum(sum, lane);
      if (lane == 31) s_warp[warp] = sum;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) U += s_warp[w];
      U *= HR;
    }
  }
  const Cut cut(split ? U : (int)gridDim.x, (int)gridDim.x);
  // q > 0: units of a piece
  int q = 0, segments = W < kWarps ? reqs * HR : cut.segments();
  if (split && cut.K == 0) {
    const int real = U - reqs * HR * kSetup;
    const int q0 = (real + (int)gridDim.x - 1) / (int)gridDim.x, step = max(1, q0 / 12);
    int pieces[4] = {0, 0, 0, 0};
    if (listed) {
#pragma unroll
      for (int j = 0; j < 4; ++j) pieces[j] = reqs * ((list_units + q0 + j * step - 1) / (q0 + j * step));
    } else {
      for (int b = tid; b < reqs; b += TT) {
        const int units = span_of(b).units;
#pragma unroll
        for (int j = 0; j < 4; ++j) pieces[j] += (units + q0 + j * step - 1) / (q0 + j * step);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        pieces[j] = __reduce_add_sync(~0u, pieces[j]);
        if (lane == 0) s_pieces[warp][j] = pieces[j];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        pieces[j] = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) pieces[j] += s_pieces[w][j];
      }
    }
#pragma unroll
    for (int j = 3; j >= 0; --j)
      if (pieces[j] <= (int)gridDim.x / HR) {
        q = q0 + j * step;
        segments = pieces[j] * HR;
      }
  }
  // every CTA is running: the join may take the room of those that finish first
  pdl_launch_dependents();
  const bool use_cap = a.cap_inv > 0.f;
  auto clear_marks = [&]() {
    for (int i = tid; i < C::kRows * (D / 32); i += TT) s_marks[0][i] = 0;
    if (tid == 0) s_marked = 0;
  };
  if (several) clear_marks();

  // units of setup that count in this call's segments
  const int setup = split && q == 0 ? kSetup : 0;
  // The last thread, which has the least to do when sums are joined, fetches the
  // CTA's next segment.
  auto claim = [&]() {
    if (split && cut.K > 0 && tid == TT - 1) {
      const uint32_t t = claim_item(a.counter, a.gen, a.errors);
      s_seg = t >= (uint32_t)(cut.segments() - cut.R) ? cut.segments() : cut.R + (int)t;
    }
  };
  for (int seg = blockIdx.x * C::kTeams + team; seg < segments;) {
    // ---- the segment's units [u0, u1), and the request its first unit belongs to
    int u0, u1, base, req;  // base: first unit of request `req`
    if (!split) {  // one team per item; units are counted from its request's first
      const int units = listed ? list_units : span_of(seg / HR).units;
      req = seg / HR;
      base = 0;
      u0 = (seg % HR) * units;
      u1 = u0 + units;
    } else {
      // requests weigh their units or pieces; the one that holds unit or piece x
      const int x = q > 0 ? seg : cut.start(seg);
      auto weight = [&](int units) -> int { return (q > 0 ? (units + q - 1) / q : units + setup) * HR; };
      if (listed) {
        req = x / weight(list_units);
        base = req * weight(list_units);
      } else {
        int before = 0;  // weights of the requests before these
        if (tid == 0) s_req = -1;
        for (int b0 = 0; b0 < reqs; b0 += TT) {
          const int b = b0 + tid;
          const int mine = b < reqs ? weight(span_of(b).units) : 0;
          int incl = warp_incl_sum(mine, lane);
          __syncthreads();
          if (lane == 31) s_warp[warp] = incl;
          __syncthreads();
          int total = 0;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            if (w < warp) incl += s_warp[w];
            total += s_warp[w];
          }
          const int first = before + incl - mine;
          if (mine > 0 && first <= x && x < first + mine) {
            s_req = b;
            s_base = first;
          }
          before += total;
          if (before > x) break;
        }
        __syncthreads();
        req = s_req;
        base = s_base;
        if (req < 0) break;  // the lengths changed during the call
      }
      u0 = x;
      u1 = q > 0 ? x + 1 : cut.start(seg + 1);
      if (q > 0) {  // the piece's units, counted from its request's first
        const int units = listed ? list_units : span_of(req).units, per = (units + q - 1) / q;
        const int hr = (x - base) / per, piece = x - base - hr * per;
        base = 0;
        u0 = hr * units + piece * q;
        u1 = hr * units + min(units, (piece + 1) * q);
      }
    }

    bool claimed = false;
    for (int u = u0; u < u1;) {
      // ---- the item at unit u, and the part of it that is this segment's
      int req_next = req;
      const int b = listed ? req / a.next_n : req;
      const int tok0 = listed ? req : req * a.next_n;  // query row of the item's first row
      const int n_tok = listed ? 1 : a.next_n;
      const Span sp = span_of(b);
      const int units = listed ? list_units : sp.units;
      const int cost = setup + units, hr = (u - base) / cost;
      const int off = u - base - hr * cost, stop = min(cost, off + (u1 - u));
      const int h = hr / a.row_tiles, rt = hr % a.row_tiles;
      const int ta = max(0, off - setup), tb = max(0, stop - setup);
      const bool first_item = u == u0;
      u += stop - off;
      if (u - base >= cost * HR) {
        base += cost * HR;
        ++req_next;
      }
      if (ta == tb) {  // the segment ends in the item's setup
        req = req_next;
        continue;
      }
      const int row0 = rt * C::kRows;
      const int rows = min(C::kRows, a.rows - row0);
      constexpr int EB = F8 || F4 ? 1 : 2;  // bytes of a cached value (4-bit: strides are in bytes)
      const uint8_t* kbase = static_cast<const uint8_t*>(a.kv.k) + h * a.kv.k_head_stride * EB;
      const uint8_t* vbase = static_cast<const uint8_t*>(a.kv.v) + h * a.kv.v_head_stride * EB;
      const int64_t k_ts = a.kv.k_token_stride * EB, v_ts = a.kv.v_token_stride * EB;
      // a page's or token's place in 2^off_shift bytes
      // (4-bit: the token's slot, from which both its codes' and its scales' places follow)
      auto k_off = [&](int64_t page, int off) -> uint32_t {
        if (F4) return (uint32_t)((int)page << a.page_shift | off);
        return (uint32_t)((page * a.kv.k_block_stride * EB + off * k_ts) >> a.off_shift);
      };
      auto v_off = [&](int64_t page, int off) -> uint32_t {
        return (uint32_t)((page * a.kv.v_block_stride * EB + off * v_ts) >> a.off_shift);
      };
      // sight of query token j: [end_j - window, end_j), end_j = end0 + j
      const int end0 = listed ? 0 : sp.len - a.next_n + 1;
      const int lo_all = a.window > 0 ? max(0, end0 - a.window) : 0;
      const int* bt = a.block_table + (int64_t)b * a.max_blocks;
      if (tid == 0 && hr == 0 && ta == 0 && (!listed || req % a.next_n == 0)) {
        const int L = __ldg(a.context_lens + b);
        if (L < 0 || L > cap) count_bad_input(a.errors);
      }

      // ---- the item's query rows; a CTA's are on their way while the table is made
      constexpr int LQ = D / 8;  // lanes per row, 16 bytes each
      constexpr int QP = (C::kRows * LQ + TT - 1) / TT;
      auto q_chunk = [&](int i) -> uint4 {
        const int r = (i * TT + tid) / LQ, rr = row0 + r;
        if (r >= rows) return make_uint4(0, 0, 0, 0);
        const uint16_t* src = static_cast<const uint16_t*>(a.q) +
                              (int64_t)(tok0 + rr / a.group) * a.q_ts +
                              (int64_t)(h * a.group + rr % a.group) * a.q_hs;
        return __ldg(reinterpret_cast<const uint4*>(src) + tid % LQ);
      };
      uint4 qraw[W < kWarps ? 1 : QP];
      if (W == kWarps) {
#pragma unroll
        for (int i = 0; i < QP; ++i) qraw[W < kWarps ? 0 : i] = q_chunk(i);
      }

      typename TileOf<D, CT, NT, KS>::type tile;
      tile.clear();

      // units whose page groups of 16 keys (or listed positions) fit the table
      const int sub = tab_words / (listed ? C::kUnit : C::kUnit / 16);
      for (int sa = ta; sa < tb; sa += sub) {
        int sb = min(tb, sa + sub);
        if (sa > ta) sync();  // the previous range's table is done with
        // four entries at a time, their loads issued together (a list entry and
        // then its page id are two dependent round trips)
        constexpr int TB = 4;
        int last = -1;  // last position found in this thread's entries
        if (listed) {
          const int* list = a.topk_idx + (int64_t)req * a.topk;
          const int my_end = max(0, sp.len - a.next_n + 1 + req % a.next_n);
          const int n = (sb - sa) * C::kUnit;
          for (int i0 = tid; i0 < n; i0 += TB * TT) {
            int p[TB], id[TB];
#pragma unroll
            for (int j = 0; j < TB; ++j) {
              const int i = i0 + j * TT, at = sa * C::kUnit + i;
              p[j] = i < n && at < a.topk ? __ldg(list + at) : -1;
            }
#pragma unroll
            for (int j = 0; j < TB; ++j)
              id[j] = p[j] >= 0 && p[j] < my_end ? __ldg(bt + (p[j] >> a.page_shift)) : -1;
#pragma unroll
            for (int j = 0; j < TB; ++j) {
              const int i = i0 + j * TT;
              if (i >= n) break;
              const bool ok = id[j] >= 0 && id[j] < a.kv.num_blocks;
              if (!ok && p[j] >= 0 && hr == 0) count_bad_input(a.errors);
              if (ok) last = i;
              tab[i] = ok ? k_off(id[j], p[j] & page_mask) : kNone;
              if (!a.one_table) vtab[i] = ok ? v_off(id[j], p[j] & page_mask) : kNone;
            }
          }
        } else {
          const int g0 = (sp.t0 + sa) * (C::kUnit / 16), n = (sb - sa) * (C::kUnit / 16);
          for (int i0 = tid; i0 < n; i0 += TB * TT) {
            int id[TB];
#pragma unroll
            for (int j = 0; j < TB; ++j) {
              const int i = i0 + j * TT, key = (g0 + i) * 16;
              id[j] = i < n && key < sp.len && key + 16 > lo_all ? __ldg(bt + (key >> a.page_shift)) : -1;
            }
#pragma unroll
            for (int j = 0; j < TB; ++j) {
              const int i = i0 + j * TT, key = (g0 + i) * 16;
              if (i >= n) break;
              const bool ok = id[j] >= 0 && id[j] < a.kv.num_blocks;
              // counted once per page, by its first group that is in sight
              if (!ok && key < sp.len && key + 16 > lo_all && hr == 0 &&
                  ((key & page_mask) == 0 || key <= lo_all))
                count_bad_input(a.errors);
              tab[i] = ok ? k_off(id[j], key & page_mask) : kNone;
              if (!a.one_table) vtab[i] = ok ? v_off(id[j], key & page_mask) : kNone;
            }
          }
        }
        if (sa == ta) {
          // ---- query rows to shared memory
#pragma unroll(W < kWarps && QP > 2 ? 2 : QP)
          for (int i = 0; i < QP; ++i) {
            const int r = (i * TT + tid) / LQ, part = tid % LQ;
            float mult = a.scale;
            const uint4 raw = W < kWarps ? q_chunk(i) : qraw[W < kWarps ? 0 : i];
            uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            if (F8 || F4) {
              float x[8], amax = 0.f;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 f = a.q_bf16 ? unpack2<true>(w[j]) : unpack2<false>(w[j]);
                x[2 * j] = f.x;
                x[2 * j + 1] = f.y;
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
#pragma unroll
              for (int d = LQ / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
              // largest magnitude to [2^14, 2^15): all products with codes stay finite
              // (tiny rows: times 2^126; rows with an infinity or NaN: as they are)
              int e = 0;
              if (a.q_bf16 && amax < INFINITY) e = min(126, 141 - (int)(__float_as_uint(amax) >> 23));
              const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = pack2<false>(x[2 * j] * up, x[2 * j + 1] * up);
              mult *= (F8 && a.kv.k_scale ? __ldg(a.kv.k_scale + h) : 1.f) *
                      __uint_as_float((uint32_t)(127 - e) << 23);
            }
            if (QP * TT == C::kRows * LQ || r < C::kRows) {
              if (part == 0) {
                // a masked score (-inf) times the factor must stay one: at least FLT_MIN
                s_mult[r] = fmaxf(fabsf(mult) * kLog2e, FLT_MIN);
                s_one[r] = 1.f;  // every team's the same
                s_end[r] = end0 + (row0 + r) / a.group;
              }
              // a factor's sign is carried by the queries, and so is a NaN (of a key scale)
              const uint32_t flip = mult < 0.f ? 0x80008000u : 0u, nan = mult != mult ? 0x7FFF7FFFu : 0u;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                int d = part * 8 + 2 * j;
                // 8-bit keys come from ldmatrix four codes a lane: dimension 4c+i of a
                // 16-block sits at k index 2c+i (i < 2) or 8+2c+i-2
                if (F8) d = (d & ~15) + ((d & 2) ? 8 : 0) + ((d & 15) >> 2) * 2;
                // 4-bit ones eight a lane: dimension 8c+i of a 32-block in its half i / 4, there
                // at 2c+i%4 (i%4 < 2) or 8+2c+i%4-2
                if (F4) d = (d & ~31) + ((d & 4) ? 16 : 0) + ((d & 2) ? 8 : 0) + ((d & 31) >> 3) * 2;
                *reinterpret_cast<uint32_t*>(q_sm + swz<D * 2>(r, d >> 3) + (d & 7) * 2) = (w[j] ^ flip) | nan;
              }
            }
          }
        }
        if (listed) {
          // units past the last listed position (a short row's list ends in -1) are
          // not streamed at all
          last = __reduce_max_sync(~0u, last);
          if (lane == 0) s_last[warp] = last;
        }
        sync();
        if (listed) {
#pragma unroll
          for (int w = 0; w < W; ++w) last = max(last, s_last[w]);
          sb = min(sb, sa + last / C::kUnit + (last < 0 ? 0 : 1));
        }

        // ---- the warp's stream: half stage 2 t is unit sa + t's keys, 2 t + 1 its values
        const int halves = 2 * (sb - sa);
        int put = 0, get = 0;  // ring positions
        auto issue = [&](int i) {
          if (i < halves) {
            const int t = i >> 1;
            const bool is_v = i & 1;
            const uint8_t* src0 = is_v ? vbase : kbase;
            const uint32_t* tb_ = is_v ? vtab : tab;
            constexpr int LPR = ROWB / 16, RPI = 32 / LPR;  // lanes per row, rows per pass
            const int rl = lane / LPR, cl = lane % LPR;
            const uint32_t dst = ring_u + put * C::kHalf;
            src0 += cl * 16;
            if constexpr (F4) {
              // codes of a token at page + off * ROWB, its scales behind the page's codes
              constexpr int SB = D / 32;
              const int64_t bs = is_v ? a.kv.v_block_stride : a.kv.k_block_stride;
              const int codes = ROWB << a.page_shift;  // of a page
              const uint32_t dst_s = dst + KS * ROWB;
              auto page_of = [&](uint32_t e) -> const uint8_t* { return src0 + (int64_t)(e >> a.page_shift) * bs; };
              if (listed) {
                const uint32_t* e0 = tb_ + t * C::kUnit + warp * KS;
#pragma unroll
                for (int j = 0; j < KS / RPI; ++j) {
                  const uint32_t e = e0[j * RPI + rl];
                  const bool ok = e != kNone;
                  cp_async_16_zfill(dst + swz<ROWB>(j * RPI + rl, cl),
                                    ok ? page_of(e) + (e & page_mask) * ROWB : src0, ok);
                }
                if (lane < KS) {  // (head_dim 64: with its neighbour's)
                  const uint32_t e = e0[lane];
                  const bool ok = e != kNone;
                  constexpr int N = scale_room<D, CT>();
                  cp_async_few_zfill<N>(dst_s + lane * N,
                                        (ok ? page_of(e) + codes + ((int)(e & page_mask) * SB & ~(N - 1)) : src0) - cl * 16, ok);
                }
              } else {
                const uint32_t* e0 = tb_ + t * (C::kUnit / 16) + warp * (KS / 16);
                const int key0 = (sp.t0 + sa + t) * C::kUnit + warp * KS;
                uint32_t e[KS / 16];
                bool all = key0 >= lo_all && key0 + KS <= sp.len;  // every key is seen by some query
#pragma unroll
                for (int gr = 0; gr < KS / 16; ++gr) {
                  e[gr] = e0[gr];
                  all = all && e[gr] != kNone;
                }
                if (all) {
                  const uint32_t to = dst + swz<ROWB>(rl, cl), to_s = dst_s + lane * 16;
#pragma unroll
                  for (int gr = 0; gr < KS / 16; ++gr) {
                    const uint8_t* pg = page_of(e[gr]);
                    const int off = e[gr] & page_mask;
                    const uint8_t* src = pg + (off + rl) * ROWB;
                    // (rows 8 apart have the same swizzle; RPI = 4, 8 or 16)
#pragma unroll
                    for (int j = 0; j < 16 / RPI; ++j)
                      cp_async_16((RPI % 8 == 0 ? to + (gr * 16 + j * RPI) * ROWB : dst + swz<ROWB>(gr * 16 + j * RPI + rl, cl)),
                                  src + j * RPI * ROWB);
                    if (lane < SB)  // the group's scales, 16 bytes a lane
                      cp_async_16(to_s + gr * 16 * SB, pg + (codes + off * SB + lane * 16 - cl * 16));
                  }
                } else {
#pragma unroll 1
                  for (int gr = 0; gr < KS / 16; ++gr) {
                    const uint32_t x = e0[gr];
                    const int key = key0 + gr * 16 + rl;
                    const uint8_t* pg = x != kNone ? page_of(x) : src0;
                    const int off = x != kNone ? (int)(x & page_mask) : 0;
                    const uint8_t* src = pg + (off + rl) * ROWB;
                    // rows of the group that some query sees: [from, to)
                    const int from = x != kNone ? lo_all - key : 16, to = sp.len - key;
#pragma unroll
                    for (int j = 0; j < 16 / RPI; ++j) {
                      const bool ok = j * RPI >= from && j * RPI < to;
                      cp_async_16_zfill(dst + swz<ROWB>(gr * 16 + j * RPI + rl, cl), ok ? src + j * RPI * ROWB : src0, ok);
                    }
                    if (lane < SB)
                      cp_async_16_zfill(dst_s + gr * 16 * SB + lane * 16,
                                        x != kNone ? pg - cl * 16 + codes + off * SB + lane * 16 : src0, x != kNone);
                  }
                }
              }
            } else if (listed) {
              const uint32_t* e0 = tb_ + t * C::kUnit + warp * KS + rl;
#pragma unroll
              for (int j = 0; j < KS / RPI; ++j) {
                const uint32_t e = e0[j * RPI];
                const bool ok = e != kNone;
                cp_async_16_zfill(dst + swz<ROWB>(j * RPI + rl, cl),
                                  src0 + (ok ? (uint64_t)e * a.off_unit : 0), ok);
              }
            } else {
              const int64_t ts = is_v ? v_ts : k_ts;
#pragma unroll
              for (int gr = 0; gr < KS / 16; ++gr) {
                const int grp = t * (C::kUnit / 16) + warp * (KS / 16) + gr;
                const uint32_t e = tb_[grp];
                const int key = (sp.t0 + sa) * C::kUnit + grp * 16 + rl;
                const uint8_t* src = src0 + (e != kNone ? (uint64_t)e * a.off_unit + rl * ts : 0);
                if (e != kNone && key - rl >= lo_all && key - rl + 16 <= sp.len) {
#pragma unroll
                  for (int j = 0; j < 16 / RPI; ++j) {
                    cp_async_16(dst + swz<ROWB>(gr * 16 + j * RPI + rl, cl), src);
                    src += RPI * ts;
                  }
                } else {
                  // rows of the group that some query sees: [from, to)
                  const int from = e != kNone ? lo_all - key : 16, to = sp.len - key;
#pragma unroll
                  for (int j = 0; j < 16 / RPI; ++j) {
                    const bool ok = j * RPI >= from && j * RPI < to;
                    cp_async_16_zfill(dst + swz<ROWB>(gr * 16 + j * RPI + rl, cl), ok ? src : src0, ok);
                    src += RPI * ts;
                  }
                }
              }
            }
          }
          cp_async_commit();
          put = put + 1 == NS ? 0 : put + 1;
        };
#pragma unroll 1
        for (int i = 0; i < NS; ++i) issue(i);

        tile.load_q(q_u, lane);
        for (int t = 0; t < sb - sa; ++t) {
          cp_async_wait_group<NS - 1>();
          __syncwarp();
          const int tile0 = t * C::kUnit + warp * KS;  // within the sub-range
          const int key0 = (sp.t0 + sa) * C::kUnit + tile0;
          const Sight<listed> sight{tab, s_end, tile0, key0, a.window};
          if constexpr (F4 && listed && D == 64)
            settle_scales<D, listed>(ring + get * C::kHalf + KS * ROWB, sight, KS, lo_all, sp.len, false, lane);
          tile.scores(ring_u + get * C::kHalf, q_u, lane);
          __syncwarp();
          get = get + 1 == NS ? 0 : get + 1;
          issue(2 * t + NS);

          bool whole;  // every key of the tile is seen by every row
          if (listed) {
            bool ok = true;
            if (lane < KS) ok = tab[tile0 + lane] != kNone;
            whole = __all_sync(~0u, ok);
          } else {
            bool ok = true;
#pragma unroll
            for (int gr = 0; gr < KS / 16; ++gr) ok = ok && tab[tile0 / 16 + gr] != kNone;
            whole = ok && key0 + KS <= end0 &&
                    (a.window == 0 || key0 >= end0 + n_tok - 1 - a.window);
          }
          if (use_cap) tile.cap(a.cap_log2, a.cap_inv, s_mult, lane);
          if (!whole) tile.mask(sight, lane);

          cp_async_wait_group<NS - 1>();
          __syncwarp();
          if constexpr (F4) {
            if (!whole || (listed && D == 64))
              settle_scales<D, listed>(ring + get * C::kHalf + KS * ROWB, sight, KS, lo_all, sp.len, !whole, lane);
          }
          if constexpr (several) {
            if (!whole)
              keep_apart<D, CT, C::kRows>(ring + get * C::kHalf, sight, max(lo_all, key0),
                                          a.window > 0 ? min(end0 + min(n_tok - 1 - a.window, 0), key0 + KS) : 0,
                                          max(end0, key0), min(sp.len, key0 + KS), s_marks, &s_marked, lane);
          }
          tile.values(ring_u + get * C::kHalf, tile.factors(use_cap ? s_one : s_mult, lane), lane);
          __syncwarp();
          get = get + 1 == NS ? 0 : get + 1;
          issue(2 * t + 1 + NS);
        }
        cp_async_wait_group<0>();
        __syncwarp();
      }

      // ---- the warps' sums become one: each leaves its own in its ring
      tile.leave(reinterpret_cast<float*>(ring), C::kPitch, s_ml[warp], rows, lane);
      if (u + setup >= u1) {  // nothing more in this segment
        claimed = true;
        claim();  // while the sums are joined
      }
      sync();
      const bool complete = ta == 0 && tb == units;
      // partial 2 s is a segment's first part, 2 s + 1 its last; an item's parts are its
      // first segment's last (or only) part, then the following segments' first parts
      const int item_end = u + cost - stop;  // in the cut's units
      const int part = 2 * seg + (first_item ? 0 : 1);
      if (split && ta == 0 && tid == TT - 1)
        a.desc[req * HR + hr] =
            make_int2(part, q > 0 ? (units + q - 1) / q : cut.owner(item_end - 1) - seg + 1);
      const bool marked = several && s_marked != 0;
      constexpr int QPR = D / 4;  // float4 quads per row
      for (int i = tid; i < rows * QPR; i += TT) {
        const int r = i / QPR, d = (i % QPR) * 4;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) mx = fmaxf(mx, s_ml[w][r].x);
        float lsum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float2 ml = s_ml[w][r];
          if (ml.x == -INFINITY && ml.y == 0.f) continue;  // the warp saw nothing of this row
          const float f = ml.x == -INFINITY ? 1.f : ex2(ml.x - mx);
          const float4 x = *reinterpret_cast<const float4*>(rings + w * C::kRing + (r * C::kPitch + d) * 4);
          lsum += ml.y * f;
          acc.x += x.x * f;
          acc.y += x.y * f;
          acc.z += x.z * f;
          acc.w += x.w * f;
        }
        if (marked) {
          const uint32_t bits = s_marks[0][r * (D / 32) + d / 32] >> (d % 32);
          const float nan = __int_as_float(0x7FFFFFFF);
          if (bits & 1) acc.x = nan;
          if (bits & 2) acc.y = nan;
          if (bits & 4) acc.z = nan;
          if (bits & 8) acc.w = nan;
        }
        if (complete) {
          const int rr = row0 + r;
          const int64_t orow = (int64_t)(tok0 + rr / a.group) * a.Hq + h * a.group + rr % a.group;
          float inv = lsum == 0.f ? 0.f : 1.f / lsum;
          // an empty row stays zero whatever the scale
          if (F8 && a.kv.v_scale && lsum != 0.f) inv *= __ldg(a.kv.v_scale + h);
          uint2 w;
          if (MB || ((F8 || F4) && a.q_bf16)) {
            w.x = pack2<true>(acc.x * inv, acc.y * inv);
            w.y = pack2<true>(acc.z * inv, acc.w * inv);
          } else {
            w.x = pack2<false>(acc.x * inv, acc.y * inv);
            w.y = pack2<false>(acc.z * inv, acc.w * inv);
          }
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + d) = w;
          if (a.lse && d == 0) a.lse[orow] = lsum == 0.f ? -INFINITY : (mx + log2f(lsum)) * kLn2;
        } else {
          const int64_t prow = (int64_t)part * a.part_rows + r;
          *reinterpret_cast<float4*>(a.part_o + prow * D + d) = acc;
          if (d == 0) *reinterpret_cast<float2*>(a.part_ml + prow * 2) = make_float2(mx, lsum);
        }
      }
      sync();  // the rings, the table and the query rows are refilled next
      if (marked) clear_marks();  // the next marks come after the table's barrier

      req = req_next;
    }
    if (!split || cut.K == 0) break;
    if (!claimed) {
      claim();
      __syncthreads();
    }
    seg = s_seg;
    __syncthreads();  // read by all before the next claim
  }
}

template <int D, int CT, int NT, bool listed, int W, bool several>
cudaError_t launch_items(const AttnArgs& a, cudaStream_t stream) {
  using C = Cfg<D, CT, NT, listed, W>;
  auto kern = paged_attn_kernel<D, CT, NT, listed, W, several>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3((a.grid + C::kTeams - 1) / C::kTeams), dim3(C::kThreads), C::kSmem,
                          stream, a);
}

// A call's kernels by what its items see: one token's context each, several tokens'
// contexts, a selection.
enum Sights : int { kOneToken = 0, kSeveralTokens = 1, kSelection = 2 };

template <int D, int CT, int NT, int S>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
  constexpr bool listed = S == kSelection, several = S == kSeveralTokens;
  switch (a.warps) {
    case 1: return launch_items<D, CT, NT, listed, 1, several>(a, stream);
    case 2: return launch_items<D, CT, NT, listed, 2, several>(a, stream);
    case 4: return launch_items<D, CT, NT, listed, 4, several>(a, stream);
  }
  return launch_items<D, CT, NT, listed, kWarps, several>(a, stream);
}

template <int D, int CT, int S>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t stream) {
  switch (attn_row_tiles(D, a.rows)) {
    case 1: return launch<D, CT, 1, S>(a, stream);
    case 2: return launch<D, CT, 2, S>(a, stream);
  }
  if constexpr (D <= 128) return launch<D, CT, 4, S>(a, stream);
  return cudaErrorInvalidValue;
}

template <int CT, int S>
cudaError_t launch_type(const AttnArgs& a, cudaStream_t stream) {
  switch (a.kv.head_dim) {
    case 64: return launch_rows<64, CT, S>(a, stream);
    case 128: return launch_rows<128, CT, S>(a, stream);
    default: return launch_rows<256, CT, S>(a, stream);
  }
}

}  // namespace attn
}  // namespace idx
