// Internal launchers of the serving operators (argument checking happens in
// serving_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "idx.h"

namespace idx {

struct PlanArgs {
  const int32_t* cached;
  const int32_t* fresh;  // new tokens per request
  int32_t* block_table;
  const int32_t* free_pages;
  const int32_t* head;
  int32_t* head_out;
  int32_t* context_lens;
  int32_t* query_start;
  int64_t* slots;
  int32_t* positions;
  int32_t* token_seq;
  int64_t num_tokens;
  int64_t num_blocks;
  int32_t B;
  int32_t max_blocks;
  int32_t num_free;
  int32_t page_shift;  // log2 of the page size
  idx_device_errors* errors;
};
cudaError_t launch_plan_step(const PlanArgs& a, int sms, cudaStream_t stream);

constexpr int kMaxRopeCols = 128;
// Turns per position of every table column as 64-bit fractions: the angle at
// position p is 2 pi * (p * turns[i] mod 2^64) / 2^64.
struct RopeTableArgs {
  unsigned long long turns[kMaxRopeCols];
  int64_t pos0;
  int64_t num_pos;
  int32_t half;
  float mscale;
  float* cos_out;
  float* sin_out;
};
cudaError_t launch_rope_table(const RopeTableArgs& a, int sms, cudaStream_t stream);

struct KvInsertArgs {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;  // elements
  const float* q_weight;
  const float* k_weight;
  float eps;
  const int32_t* positions;
  const float* cs;
  const float* sn;
  int64_t num_pos;
  const int64_t* slots;
  void* q_out;
  idx_kv_cache kv;
  int64_t N;
  int32_t Hq;
  int32_t rot_dim;
  int32_t interleaved;
  int32_t page_shift;
  idx_device_errors* errors;
};
cudaError_t launch_kv_insert(int dtype, const KvInsertArgs& a, int sms, cudaStream_t stream);

// Paged attention: resident CTAs over the device, and the levels of segments
// they claim (see paged_attn.cuh), are bounded by these, so that the
// workspace's size depends on neither the device nor the lengths.
constexpr int kAttnMaxCtas = 320;
constexpr int kAttnLevels = 5;
constexpr int kAttnMaxParts = 2 * kAttnLevels * kAttnMaxCtas;
struct AttnArgs {
  const void* q;
  int64_t q_ts, q_hs;  // elements
  idx_kv_cache kv;
  const int32_t* block_table;
  const int32_t* context_lens;
  const int32_t* topk_idx;  // null: the whole context
  void* out;
  float* lse;
  float* part_o;   // [kAttnMaxParts][part_rows][D] partial sums of split items
  float* part_ml;  // [kAttnMaxParts][part_rows][2] their running maxima and weights
  int2* desc;      // [items] first partial and number of partials
  unsigned long long* counter;  // generation-tagged count of claimed segments
  unsigned long long gen;       // this call's generation
  float scale;
  float cap_log2;  // the cap in log2 units, and its reciprocal (0: no cap)
  float cap_inv;
  int32_t window;
  int32_t topk;
  int32_t B;        // requests
  int32_t next_n;
  int32_t Hq;
  int32_t group;    // query heads per kv head
  int32_t rows;     // query rows of one kv head: next_n * group, or group (top-k)
  int32_t row_tiles;
  int32_t part_rows;  // query rows of an item: at most 8 * attn_row_tiles()
  int32_t max_blocks;
  int32_t page_shift;
  int32_t off_shift;  // every page and token offset is a multiple of 2^off_shift bytes,
  uint32_t off_unit;  // off_unit, and fits 32 bits in that unit
  int32_t one_table;  // k and v have the same page and token strides
  int32_t q_bf16;     // type of q and out
  int32_t split;      // 0: items whole, no join
  int32_t warps;      // warps that share an item: 8, 4, 2 or 1 (fewer than 8 only with split = 0)
  int32_t grid;       // teams
  idx_device_errors* errors;
};
// Tiles of eight query rows an item of `rows` rows takes: 1, 2 or 4 (head_dim
// 256: 1 or 2, where four would not fit the registers).
constexpr int attn_row_tiles(int head_dim, int rows) {
  return rows <= 8 ? 1 : (rows <= 16 || head_dim > 128 ? 2 : 4);
}
// keys of a warp's tile, with `warps` warps sharing an item
constexpr int attn_keys_per_tile(int head_dim, int cache_dtype, int nt, int warps) {
  return head_dim * (cache_dtype == IDX_E4M3 ? 1 : 2) >= 256 || nt == 4 || warps < 8 ? 16 : 32;
}
// Resident CTAs per SM: two where the sums take at most 64 registers a thread
// and three half stages fit 12 KB of shared memory a warp.
constexpr int attn_occupancy(int head_dim, int cache_dtype, int nt) {
  return head_dim * nt <= 256 && 3 * head_dim * (cache_dtype == IDX_E4M3 ? 1 : 2) *
                                         attn_keys_per_tile(head_dim, cache_dtype, nt, 8) <= 12288 ? 2 : 1;
}
// keys a CTA handles at a time (the unit in which an item's length is split)
constexpr int attn_unit_keys(int head_dim, int cache_dtype, int nt) {
  return 8 * attn_keys_per_tile(head_dim, cache_dtype, nt, 8);
}
cudaError_t launch_attn_bf16(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_fp16(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_e4m3(const AttnArgs& a, cudaStream_t stream);
// whole contexts, several new tokens a request (translation units of their own)
cudaError_t launch_attn_bf16_several(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_fp16_several(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_e4m3_several(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_join(const AttnArgs& a, cudaStream_t stream);

}  // namespace idx
