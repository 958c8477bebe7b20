// C ABI of the serving operators (declared in include/idx.h): argument checks,
// workspace layout and dispatch.  Nothing here allocates device memory or
// synchronises.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "idx.h"
#include "launch.h"
#include "serving.h"

namespace {

using idx::fail;
using idx::ok;

idx_status from_cuda(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ok();
  return fail(IDX_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int page_shift_of(int32_t page_size) {
  switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
  }
  return -1;
}

struct Range {
  const void* p;
  int64_t bytes;
  const char* name;
};
bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes &&
         y < x + (uintptr_t)a.bytes;
}

bool stride_ok(int64_t stride, int elt) {
  return stride >= 0 && stride <= (int64_t)1 << 48 && (stride * elt) % 16 == 0;
}

// q_dtype: the type the cache must have unless it is E4M3.
idx_status check_kv(const idx_kv_cache* kv, int32_t q_dtype) {
  if (!kv) return fail(IDX_ERR_INVALID_ARG, "null kv");
  if (q_dtype != IDX_BF16 && q_dtype != IDX_FP16)
    return fail(IDX_ERR_INVALID_ARG, "dtype=%d (bf16 or fp16)", q_dtype);
  if (kv->dtype != q_dtype && kv->dtype != IDX_E4M3)
    return fail(IDX_ERR_INVALID_ARG, "cache dtype=%d (the queries' type or E4M3)", kv->dtype);
  if (page_shift_of(kv->page_size) < 0)
    return fail(IDX_ERR_INVALID_ARG, "page_size=%d (16, 32, 64 or 128)", kv->page_size);
  if (kv->head_dim != 64 && kv->head_dim != 128 && kv->head_dim != 256)
    return fail(IDX_ERR_INVALID_ARG, "head_dim=%d (64, 128 or 256)", kv->head_dim);
  if (kv->heads < 1 || kv->heads > 1024)
    return fail(IDX_ERR_INVALID_ARG, "kv heads=%d outside [1, 1024]", kv->heads);
  if (kv->num_blocks <= 0 || kv->num_blocks > (int64_t)INT32_MAX / kv->page_size)
    return fail(IDX_ERR_INVALID_ARG, "num_blocks=%lld", (long long)kv->num_blocks);
  const int elt = kv->dtype == IDX_E4M3 ? 1 : 2;
  const int64_t strides[6] = {kv->k_block_stride, kv->k_head_stride, kv->k_token_stride,
                              kv->v_block_stride, kv->v_head_stride, kv->v_token_stride};
  for (int64_t s : strides)
    if (!stride_ok(s, elt))
      return fail(IDX_ERR_INVALID_ARG, "cache stride %lld (nonnegative, a multiple of 16 bytes)",
                  (long long)s);
  if (kv->dtype != IDX_E4M3 && (kv->k_scale || kv->v_scale))
    return fail(IDX_ERR_INVALID_ARG, "scales belong to an E4M3 cache");
  return IDX_OK;
}

idx_status check_kv_pointers(const idx_kv_cache* kv) {
  if (!kv->k || !kv->v) return fail(IDX_ERR_INVALID_ARG, "null cache");
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16))
    return fail(IDX_ERR_INVALID_ARG, "alignment: k and v need 16 bytes");
  if (!aligned(kv->k_scale, 4) || !aligned(kv->v_scale, 4))
    return fail(IDX_ERR_INVALID_ARG, "alignment: scales need 4 bytes");
  return IDX_OK;
}

// Workspace of the attention: the segment counter, the items' descriptors, then
// the partials (rows of the larger of the two row layouts: whole groups of
// next_n tokens, or one token's group with a selection).
struct AttnWs {
  unsigned long long* counter;
  int2* desc;
  float* ml;
  float* o;
};
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
int64_t part_rows_of(int D, int64_t rows) {
  const int64_t most = 8 * idx::attn_row_tiles(D, (int)rows);
  return rows < most ? rows : most;
}
size_t attn_ws(void* base, int64_t B, int64_t next_n, int64_t Hq, int64_t Hkv, int D, AttnWs* w) {
  const int64_t group = Hq / Hkv;
  const int64_t rows = part_rows_of(D, group * next_n), one = part_rows_of(D, group);
  const int64_t dense = B * Hkv * ((group * next_n + rows - 1) / rows);
  const int64_t listed = B * next_n * Hkv * ((group + one - 1) / one);
  const size_t items = (size_t)(dense > listed ? dense : listed);
  const size_t o_desc = 256;
  const size_t o_ml = o_desc + up256(items * sizeof(int2));
  const size_t o_o = o_ml + up256(idx::kAttnMaxParts * (size_t)rows * 2 * sizeof(float));
  if (w) {
    uint8_t* p = static_cast<uint8_t*>(base);
    *w = AttnWs{reinterpret_cast<unsigned long long*>(p), reinterpret_cast<int2*>(p + o_desc),
                reinterpret_cast<float*>(p + o_ml), reinterpret_cast<float*>(p + o_o)};
  }
  return o_o + idx::kAttnMaxParts * (size_t)rows * (size_t)D * sizeof(float);
}

// The largest power of two (at least 16 bytes, at most 2^30) that divides both.
int common_shift(int64_t x, int64_t y) {
  int s = 4;
  while (s < 30 && ((x | y) >> s & 1) == 0) ++s;
  return s;
}

// Warps that share an item: 8 (a CTA), 4, 2 or 1, or 0: items split over all CTAs
// and joined.  By an estimate of the call's microseconds for `items` items of up
// to `bytes` bytes of cache: 5 to start; 2.5 to set an item up; 7.1 TB/s in all and
// what a warp's ring and products let it stream: 6.2 GB/s, 5.2 with 16 rows, 5 with
// 32; 12.4, 7.8 and 7 where one CTA an SM leaves more room; of E4M3 codes 0.7 of
// that; 15 to start, cut and join.  Selected positions are as many for every item,
// and a last wave of few items costs its whole time.  Contexts are taken to fill
// half of their room on average, and the longest, which may come last, costs 0.4 of
// its time.  Over 277 measured cases of types, head layouts and lengths this choice
// takes 1.7 % more time than the best of the five on average (26 % at most, where
// contexts fill little of their room) and 13 % less than splitting always (14 % more
// at most).
//   us (8 heads, 8 rows of 128, bf16)     split   8 warps   4     2     1
//   64 x 2048 selected                      94      88      86   100   153
//   80 x 2048 selected                     113     120     135   116   162
//   64 x 512 selected                       33      30      26    30    44
//   128 x 128 selected                      23      23      15    13    15
//   304 x 512 selected                     114     114     107   103   104
//   128 contexts of 64 - 512                38      35      31    31    38
//   128 of 128 - 1024                       57      52      53    54    68
//   64 of 256 - 2048                        54      53      52    66   109
//   256 of 2048                            307     297     299   295   310
//   8 of 8192 - 32768                      103     203     413   788  1554
int attn_warps(int64_t items, double bytes, bool listed, int ctas, int occ, int nt, bool f8) {
  const double setup = 2.5;
  const double ring = nt == 4 ? (occ == 2 ? 5.0e3 : 7.0e3)
                      : nt == 2 ? (occ == 2 ? 5.2e3 : 7.8e3) : (occ == 2 ? 6.2e3 : 12.4e3);
  const double warp_rate = f8 ? 0.7 * ring : ring;
  const double rate = fmin(7.1e6, ctas * 8 * warp_rate);
  const double all = (double)items * bytes / rate * (listed ? 1.0 : 0.5);
  double best = 15.0 + setup * (double)items / ctas + all;
  int warps = 0;
  for (int w = 8; w >= 1; w /= 2) {
    const int64_t slots = (int64_t)ctas * (8 / w);
    const double alone = bytes / (w * warp_rate);
    double t = 5.0;
    if (listed) {
      const int64_t waves = items / slots, rest = items % slots;
      t += (double)waves * (setup + fmax((double)slots * bytes / rate, alone));
      if (rest) t += setup + fmax((double)rest * bytes / rate, alone);
    } else {
      const double waves = (double)items / (double)slots;
      t += setup * (waves > 1.0 ? waves + 0.5 : 1.0) + fmax(all + 0.4 * alone, alone);
    }
    if (t < best) {
      best = t;
      warps = w;
    }
  }
  return warps;
}

// How a call shares its items out.
struct AttnForm {
  int rows, nt, part_rows, row_tiles;  // query rows of a kv head, in tiles of eight, an item's, items a head
  int window;                          // 0 where no context can pass it
  int unit, ctas;                      // keys of a CTA's unit, CTAs the device holds at once
  int64_t keys, items, units, grid;    // keys an item can have at most
  int warps;                           // that share an item
  bool split;
};
AttnForm attn_form(int64_t B, int next_n, int group, int heads, int D, int dtype, int page_size,
                   int max_blocks, int topk, int window, int sms) {
  AttnForm f;
  const int elt = dtype == IDX_E4M3 ? 1 : 2;
  f.rows = topk > 0 ? group : group * next_n;
  f.nt = idx::attn_row_tiles(D, f.rows);
  f.part_rows = (int)part_rows_of(D, f.rows);
  f.row_tiles = (f.rows + 8 * f.nt - 1) / (8 * f.nt);
  f.window = window >= max_blocks * page_size ? 0 : window;
  f.unit = idx::attn_unit_keys(D, dtype, f.nt);
  f.keys = topk > 0 ? topk : (int64_t)max_blocks * page_size;
  if (topk == 0 && f.window > 0 && f.keys > (int64_t)f.window + next_n + f.unit)
    f.keys = (int64_t)f.window + next_n + f.unit;  // sight of all rows, first unit cut
  f.units = (f.keys + f.unit - 1) / f.unit;
  f.items = (topk > 0 ? B * next_n : B) * heads * f.row_tiles;
  const int occ = idx::attn_occupancy(D, dtype, f.nt);
  f.ctas = sms * occ < idx::kAttnMaxCtas ? sms * occ : idx::kAttnMaxCtas;
  const int warps = attn_warps(f.items, (double)f.keys * D * 2 * elt, topk > 0, f.ctas, occ, f.nt,
                               dtype == IDX_E4M3);
  f.split = f.units > 2 && warps == 0;
  f.warps = warps == 0 ? 8 : warps;
  f.grid = f.split ? (f.units * f.items < f.ctas ? f.units * f.items : f.ctas) : f.items;
  return f;
}

bool attn_shape_ok(int64_t B, int64_t next_n, int64_t Hq, int64_t Hkv, int D) {
  return B >= 0 && B <= 65535 && next_n >= 1 && next_n <= 16 && Hkv >= 1 && Hkv <= 1024 &&
         Hq >= Hkv && Hq <= 4096 && Hq % Hkv == 0 && (D == 64 || D == 128 || D == 256) &&
         B * next_n * Hq <= (int64_t)1 << 24;
}

}  // namespace

extern "C" {

idx_status idx_plan_step(const int32_t* cached_lens, const int32_t* new_lens, int32_t B,
                         int32_t* block_table, int32_t max_blocks, const int32_t* free_pages,
                         int32_t num_free, const int32_t* pool_head, int32_t* pool_head_out,
                         int64_t num_blocks, int32_t page_size, int32_t* context_lens,
                         int32_t* query_start, int64_t* slot_mapping, int32_t* positions,
                         int32_t* token_seq, int64_t num_tokens, idx_device_errors* errors,
                         idx_stream_t stream) {
  if (B < 0 || B > 65535) return fail(IDX_ERR_INVALID_ARG, "B=%d outside [0, 65535]", B);
  if (max_blocks <= 0 || max_blocks > (1 << 24))
    return fail(IDX_ERR_INVALID_ARG, "max_blocks=%d", max_blocks);
  if (num_free < 0) return fail(IDX_ERR_INVALID_ARG, "num_free=%d", num_free);
  const int shift = page_shift_of(page_size);
  if (shift < 0)
    return fail(IDX_ERR_INVALID_ARG, "page_size=%d (16, 32, 64 or 128)", page_size);
  if (num_blocks <= 0 || num_blocks > (int64_t)INT32_MAX)
    return fail(IDX_ERR_INVALID_ARG, "num_blocks=%lld", (long long)num_blocks);
  if (num_tokens < 0 || num_tokens > (int64_t)INT32_MAX)
    return fail(IDX_ERR_INVALID_ARG, "num_tokens=%lld", (long long)num_tokens);
  // Every block reads all inputs while others write: an array that is written overlaps
  // no other one, but for context_lens = cached_lens (then one block does it all).
  const Range written[7] = {{context_lens, 4ll * B, "context_lens"},
                            {query_start, 4ll * B + 4, "query_start"},
                            {slot_mapping, 8 * num_tokens, "slot_mapping"},
                            {positions, 4 * num_tokens, "positions"},
                            {token_seq, 4 * num_tokens, "token_seq"},
                            {pool_head_out, 4, "pool_head_out"},
                            {block_table, 4ll * B * max_blocks, "block_table"}};
  const Range read[4] = {{cached_lens, 4ll * B, "cached_lens"},
                         {new_lens, 4ll * B, "new_lens"},
                         {free_pages, 4ll * num_free, "free_pages"},
                         {pool_head, 4, "pool_head"}};
  for (int i = 0; i < 7; ++i) {
    for (const Range& r : read)
      if (overlap(written[i], r) && !(i == 0 && &r == read && context_lens == cached_lens))
        return fail(IDX_ERR_INVALID_ARG, "%s overlaps %s", written[i].name, r.name);
    for (int j = 0; j < i; ++j)
      if (overlap(written[i], written[j]))
        return fail(IDX_ERR_INVALID_ARG, "%s overlaps %s", written[i].name, written[j].name);
  }
  int sms = 0;
  idx_status s = idx::current_device_ok(&sms);
  if (s != IDX_OK) return s;
  if (!pool_head || !pool_head_out || !query_start ||
      (B > 0 && (!cached_lens || !new_lens || !block_table || !context_lens)) ||
      (num_free > 0 && !free_pages) ||
      (num_tokens > 0 && (!slot_mapping || !positions || !token_seq)))
    return fail(IDX_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(cached_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) ||
      !aligned(free_pages, 4) || !aligned(pool_head, 4) || !aligned(pool_head_out, 4) ||
      !aligned(context_lens, 4) || !aligned(query_start, 4) || !aligned(slot_mapping, 8) ||
      !aligned(positions, 4) || !aligned(token_seq, 4))
    return fail(IDX_ERR_INVALID_ARG, "alignment: slot_mapping 8 bytes, the rest 4 bytes");
  idx::PlanArgs a{};
  a.cached = cached_lens;
  a.fresh = new_lens;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.head = pool_head;
  a.head_out = pool_head_out;
  a.context_lens = context_lens;
  a.query_start = query_start;
  a.slots = slot_mapping;
  a.positions = positions;
  a.token_seq = token_seq;
  a.num_tokens = num_tokens;
  a.num_blocks = num_blocks;
  a.B = B;
  a.max_blocks = max_blocks;
  a.num_free = num_free;
  a.page_shift = shift;
  a.errors = errors;
  return from_cuda(idx::launch_plan_step(a, sms, (cudaStream_t)stream), "plan_step launch");
}

idx_status idx_rope_table(int64_t pos0, int64_t num_pos, int32_t rot_dim, double base,
                          int32_t scaling, double factor, double orig_len, double beta_fast,
                          double beta_slow, double mscale, float* cos_out, float* sin_out,
                          idx_stream_t stream) {
  const double kPi = 3.14159265358979323846;
  if (pos0 < 0 || num_pos < 0 || pos0 > (int64_t)1 << 31 || num_pos > ((int64_t)1 << 31) - pos0)
    return fail(IDX_ERR_INVALID_ARG, "positions [%lld, +%lld) outside [0, 2^31)", (long long)pos0,
                (long long)num_pos);
  if (rot_dim < 2 || rot_dim > 2 * idx::kMaxRopeCols || rot_dim % 2 != 0)
    return fail(IDX_ERR_INVALID_ARG, "rot_dim=%d (even, 2..256)", rot_dim);
  if (!(base > 1.0) || !isfinite(base)) return fail(IDX_ERR_INVALID_ARG, "base=%g (> 1)", base);
  if (scaling < IDX_ROPE_NONE || scaling > IDX_ROPE_YARN)
    return fail(IDX_ERR_INVALID_ARG, "scaling=%d", scaling);
  if (scaling != IDX_ROPE_NONE && (!(factor > 0.0) || !isfinite(factor)))
    return fail(IDX_ERR_INVALID_ARG, "factor=%g (> 0)", factor);
  if (scaling == IDX_ROPE_NTK && rot_dim < 4)
    return fail(IDX_ERR_INVALID_ARG, "rot_dim=%d (NTK scaling needs 4)", rot_dim);
  if (scaling == IDX_ROPE_YARN &&
      (!(orig_len > 0.0) || !isfinite(orig_len) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) ||
       !isfinite(beta_fast)))
    return fail(IDX_ERR_INVALID_ARG, "orig_len=%g, beta_fast=%g, beta_slow=%g", orig_len,
                beta_fast, beta_slow);
  if (!isfinite(mscale)) return fail(IDX_ERR_INVALID_ARG, "mscale=%g", mscale);
  int sms = 0;
  idx_status s = idx::current_device_ok(&sms);
  if (s != IDX_OK) return s;
  if (num_pos == 0) return ok();
  if (!cos_out || !sin_out) return fail(IDX_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(cos_out, 4) || !aligned(sin_out, 4))
    return fail(IDX_ERR_INVALID_ARG, "alignment: outputs need 4 bytes");

  idx::RopeTableArgs a{};
  a.half = rot_dim / 2;
  double b = base, lo = 0.0, hi = 0.0;
  if (scaling == IDX_ROPE_NTK) b = base * pow(factor, (double)rot_dim / (rot_dim - 2));
  if (scaling == IDX_ROPE_YARN) {
    // column index (in dimensions) at which a frequency makes `beta` turns over orig_len
    auto dim_of = [&](double beta) {
      return rot_dim * log(orig_len / (beta * 2.0 * kPi)) / (2.0 * log(base));
    };
    lo = fmax(floor(dim_of(beta_fast)), 0.0);
    hi = fmin(ceil(dim_of(beta_slow)), (double)(rot_dim - 1));
  }
  for (int i = 0; i < a.half; ++i) {
    double w = pow(b, -2.0 * i / rot_dim);
    if (scaling == IDX_ROPE_LINEAR) w /= factor;
    if (scaling == IDX_ROPE_YARN) {
      const double ramp = fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
      w = w * (1.0 - ramp) + w / factor * ramp;
    }
    const double turns = w / (2.0 * kPi);
    // below 1, times 2^64 fits 64 bits (a double just under 1 has spare low bits)
    a.turns[i] = (unsigned long long)ldexp(turns - floor(turns), 64);
  }
  a.pos0 = pos0;
  a.num_pos = num_pos;
  a.mscale = (float)mscale;
  a.cos_out = cos_out;
  a.sin_out = sin_out;
  return from_cuda(idx::launch_rope_table(a, sms, (cudaStream_t)stream), "rope_table launch");
}

idx_status idx_qk_norm_rope_insert(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
    int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
    int64_t v_head_stride, int64_t N, int32_t Hq, int32_t dtype, const float* q_weight,
    const float* k_weight, float eps, const int32_t* positions, const float* cos_table,
    const float* sin_table, int64_t num_pos, int32_t rot_dim, int32_t interleaved,
    const int64_t* slot_mapping, void* q_out, const idx_kv_cache* kv, idx_device_errors* errors,
    idx_stream_t stream) {
  idx_status s = check_kv(kv, dtype);
  if (s != IDX_OK) return s;
  if (N < 0 || N > (int64_t)1 << 26) return fail(IDX_ERR_INVALID_ARG, "N=%lld", (long long)N);
  if (Hq < 1 || Hq > 4096) return fail(IDX_ERR_INVALID_ARG, "Hq=%d outside [1, 4096]", Hq);
  if (rot_dim < 0 || rot_dim > kv->head_dim || rot_dim % 2 != 0)
    return fail(IDX_ERR_INVALID_ARG, "rot_dim=%d (even, 0..head_dim)", rot_dim);
  if (!interleaved && rot_dim % 16 != 0)
    return fail(IDX_ERR_INVALID_ARG, "rot_dim=%d (a multiple of 16 for halves)", rot_dim);
  if (num_pos < 0 || num_pos > (int64_t)1 << 31)
    return fail(IDX_ERR_INVALID_ARG, "num_pos=%lld", (long long)num_pos);
  if (!(eps >= 0.f) || isinf(eps)) return fail(IDX_ERR_INVALID_ARG, "eps=%g", (double)eps);
  const int64_t strides[6] = {q_token_stride, q_head_stride, k_token_stride,
                              k_head_stride,  v_token_stride, v_head_stride};
  for (int64_t st : strides)
    if (!stride_ok(st, 2))
      return fail(IDX_ERR_INVALID_ARG, "stride %lld (nonnegative, a multiple of 8)", (long long)st);
  // groups of lanes per block; the grid is one block per that many heads
  if (N * (Hq + 2 * (int64_t)kv->heads) > (int64_t)INT32_MAX)
    return fail(IDX_ERR_INVALID_ARG, "N=%lld: too many heads in all", (long long)N);
  int sms = 0;
  s = idx::current_device_ok(&sms);
  if (s != IDX_OK) return s;
  if (N == 0) return ok();
  if ((s = check_kv_pointers(kv)) != IDX_OK) return s;
  if (!q || !k || !v || !slot_mapping || !q_out ||
      (rot_dim > 0 && (!positions || !cos_table || !sin_table)))
    return fail(IDX_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16))
    return fail(IDX_ERR_INVALID_ARG, "alignment: q, k, v and q_out need 16 bytes");
  if (!aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(positions, 4) ||
      !aligned(cos_table, 4) || !aligned(sin_table, 4) || !aligned(slot_mapping, 8))
    return fail(IDX_ERR_INVALID_ARG, "alignment: slot_mapping 8 bytes, the rest 4 bytes");
  idx::KvInsertArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.k_ts = k_token_stride;
  a.k_hs = k_head_stride;
  a.v_ts = v_token_stride;
  a.v_hs = v_head_stride;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.positions = positions;
  a.cs = cos_table;
  a.sn = sin_table;
  a.num_pos = num_pos;
  a.slots = slot_mapping;
  a.q_out = q_out;
  a.kv = *kv;
  a.N = N;
  a.Hq = Hq;
  a.rot_dim = rot_dim;
  a.interleaved = interleaved;
  a.page_shift = page_shift_of(kv->page_size);
  a.errors = errors;
  return from_cuda(idx::launch_kv_insert(dtype, a, sms, (cudaStream_t)stream),
                   "qk_norm_rope_insert launch");
}

size_t idx_paged_attention_workspace_bytes(int32_t B, int32_t next_n, int32_t Hq, int32_t Hkv,
                                           int32_t head_dim) {
  if (!attn_shape_ok(B, next_n, Hq, Hkv, head_dim)) return 0;
  return attn_ws(nullptr, B, next_n, Hq, Hkv, head_dim, nullptr);
}

idx_status idx_paged_attention_form(int32_t B, int32_t next_n, int32_t Hq, int32_t Hkv,
                                    int32_t head_dim, int32_t cache_dtype, int32_t page_size,
                                    int32_t max_blocks, int32_t topk, int32_t window, int32_t sms,
                                    idx_attention_form* form) {
  if (!form) return fail(IDX_ERR_INVALID_ARG, "null form");
  if (!attn_shape_ok(B, next_n, Hq, Hkv, head_dim))
    return fail(IDX_ERR_INVALID_ARG, "B=%d, next_n=%d, Hq=%d, Hkv=%d, head_dim=%d", B, next_n, Hq, Hkv, head_dim);
  if (cache_dtype < IDX_BF16 || cache_dtype > IDX_E4M3)
    return fail(IDX_ERR_INVALID_ARG, "cache dtype=%d", cache_dtype);
  if (page_shift_of(page_size) < 0)
    return fail(IDX_ERR_INVALID_ARG, "page_size=%d (16, 32, 64 or 128)", page_size);
  if (max_blocks <= 0 || max_blocks > (INT32_MAX - 4096) / page_size)
    return fail(IDX_ERR_INVALID_ARG, "max_blocks=%d", max_blocks);
  if (topk < 0 || topk > (1 << 20) || window < 0 || (topk > 0 && window > 0))
    return fail(IDX_ERR_INVALID_ARG, "topk=%d, window=%d", topk, window);
  if (sms < 1 || sms > 1024) return fail(IDX_ERR_INVALID_ARG, "sms=%d", sms);
  const AttnForm f = attn_form(B, next_n, Hq / Hkv, Hkv, head_dim, cache_dtype, page_size, max_blocks,
                               topk, window, sms);
  *form = idx_attention_form{f.split, f.warps, f.part_rows, f.row_tiles, f.unit,
                             f.split ? (int32_t)f.grid : f.ctas * 8 / f.warps};
  return ok();
}

idx_status idx_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                               int32_t dtype, int32_t B, int32_t next_n, int32_t Hq,
                               const idx_kv_cache* kv, const int32_t* block_table,
                               int32_t max_blocks, const int32_t* context_lens,
                               const int32_t* topk_idx, int32_t topk, float scale, float softcap,
                               int32_t window, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, idx_device_errors* errors,
                               idx_stream_t stream) {
  idx_status s = check_kv(kv, dtype);
  if (s != IDX_OK) return s;
  const int D = kv->head_dim;
  if (B < 0 || B > 65535) return fail(IDX_ERR_INVALID_ARG, "B=%d outside [0, 65535]", B);
  if (next_n < 1 || next_n > 16) return fail(IDX_ERR_INVALID_ARG, "next_n=%d outside [1, 16]", next_n);
  if (Hq < 1 || Hq % kv->heads != 0)
    return fail(IDX_ERR_INVALID_ARG, "Hq=%d is no multiple of the %d kv heads", Hq, kv->heads);
  if (!attn_shape_ok(B, next_n, Hq, kv->heads, D))
    return fail(IDX_ERR_INVALID_ARG, "B=%d, next_n=%d, Hq=%d: too many query rows", B, next_n, Hq);
  if (!stride_ok(q_token_stride, 2) || !stride_ok(q_head_stride, 2))
    return fail(IDX_ERR_INVALID_ARG, "q strides %lld, %lld (nonnegative, multiples of 8)",
                (long long)q_token_stride, (long long)q_head_stride);
  // positions, rounded up to whole units, stay below 2^31
  if (max_blocks <= 0 || max_blocks > (INT32_MAX - 4096) / kv->page_size)
    return fail(IDX_ERR_INVALID_ARG, "max_blocks=%d", max_blocks);
  if (!isfinite(scale)) return fail(IDX_ERR_INVALID_ARG, "scale=%g", (double)scale);
  if (!(softcap >= 0.f) || isinf(softcap))
    return fail(IDX_ERR_INVALID_ARG, "softcap=%g (>= 0)", (double)softcap);
  if (window < 0) return fail(IDX_ERR_INVALID_ARG, "window=%d", window);
  if (topk_idx) {
    if (topk < 1 || topk > (1 << 20))
      return fail(IDX_ERR_INVALID_ARG, "topk=%d outside [1, 2^20]", topk);
    if (window != 0) return fail(IDX_ERR_INVALID_ARG, "a selection takes no window");
  }
  int sms = 0;
  s = idx::current_device_ok(&sms);
  if (s != IDX_OK) return s;
  if (B == 0) return ok();
  if ((s = check_kv_pointers(kv)) != IDX_OK) return s;
  if (!q || !block_table || !context_lens || !out)
    return fail(IDX_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return fail(IDX_ERR_INVALID_ARG, "alignment: q and out need 16 bytes, workspace 256");
  if (!aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(topk_idx, 4) ||
      !aligned(lse, 4))
    return fail(IDX_ERR_INVALID_ARG, "alignment: integer arrays and lse need 4 bytes");
  // page and token offsets as 32-bit multiples of a power of two
  const int elt = kv->dtype == IDX_E4M3 ? 1 : 2;
  const bool one_table = kv->k_block_stride == kv->v_block_stride &&
                         kv->k_token_stride == kv->v_token_stride;
  const int shift_k = common_shift(kv->k_block_stride * elt, kv->k_token_stride * elt);
  const int shift_v = common_shift(kv->v_block_stride * elt, kv->v_token_stride * elt);
  const int off_shift = shift_k < shift_v ? shift_k : shift_v;
  auto span = [&](int64_t bs, int64_t ts) {
    return (double)(kv->num_blocks - 1) * (double)bs + (double)(kv->page_size - 1) * (double)ts;
  };
  const double far = fmax(span(kv->k_block_stride, kv->k_token_stride),
                          span(kv->v_block_stride, kv->v_token_stride)) * elt;
  if (far >= ldexp(4294967295.0, off_shift))
    return fail(IDX_ERR_INVALID_ARG, "the cache spans %g bytes: strides must then be multiples of more than %d bytes",
                far, 1 << off_shift);
  AttnWs w;
  const size_t need = attn_ws(workspace, B, next_n, Hq, kv->heads, D, &w);
  if (!workspace || workspace_bytes < need)
    return fail(IDX_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu",
                workspace ? workspace_bytes : (size_t)0, need);

  idx::AttnArgs a{};
  a.q = q;
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.kv = *kv;
  a.block_table = block_table;
  a.context_lens = context_lens;
  a.topk_idx = topk_idx;
  a.out = out;
  a.lse = lse;
  a.counter = w.counter;
  a.gen = idx::next_item_generation();
  a.desc = w.desc;
  a.part_ml = w.ml;
  a.part_o = w.o;
  a.scale = scale;
  if (softcap > 0.f) {
    const double cap = (double)softcap * 1.4426950408889634;
    a.cap_log2 = cap < FLT_MAX ? (float)cap : FLT_MAX;
    a.cap_inv = (float)fmin(1.0 / cap, FLT_MAX);
  }
  const AttnForm f = attn_form(B, next_n, Hq / kv->heads, kv->heads, D, kv->dtype, kv->page_size,
                               max_blocks, topk_idx ? topk : 0, window, sms);
  a.window = f.window;
  a.topk = topk_idx ? topk : 0;
  a.B = B;
  a.next_n = next_n;
  a.Hq = Hq;
  a.group = Hq / kv->heads;
  a.rows = f.rows;
  a.part_rows = f.part_rows;
  a.row_tiles = f.row_tiles;
  a.max_blocks = max_blocks;
  a.page_shift = page_shift_of(kv->page_size);
  a.off_shift = off_shift;
  a.off_unit = 1u << off_shift;
  a.one_table = one_table;
  a.q_bf16 = dtype == IDX_BF16;
  a.errors = errors;

  if ((f.units + 64) * f.items > INT32_MAX || f.items * f.part_rows > INT32_MAX)
    return fail(IDX_ERR_INVALID_ARG, "%lld query row tiles of up to %lld keys: too much for one call",
                (long long)f.items, (long long)f.keys);
  a.split = f.split;
  a.warps = f.warps;
  a.grid = (int32_t)f.grid;
  cudaError_t e = kv->dtype == IDX_BF16   ? idx::launch_attn_bf16(a, (cudaStream_t)stream)
                  : kv->dtype == IDX_FP16 ? idx::launch_attn_fp16(a, (cudaStream_t)stream)
                                          : idx::launch_attn_e4m3(a, (cudaStream_t)stream);
  if (e == cudaSuccess && a.split) e = idx::launch_attn_join(a, (cudaStream_t)stream);
  return from_cuda(e, "paged_attention launch");
}

}  // extern "C"
