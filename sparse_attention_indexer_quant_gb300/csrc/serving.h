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

// Paged attention: resident CTAs over the device are bounded by this, so that
// the workspace's size does not depend on the device.
constexpr int kAttnMaxCtas = 320;
struct AttnArgs {
  const void* q;
  int64_t q_ts, q_hs;  // elements
  idx_kv_cache kv;
  const int32_t* block_table;
  const int32_t* context_lens;
  const int32_t* topk_idx;  // null: the whole context
  void* out;
  float* lse;
  float* part_o;   // [2 * kAttnMaxCtas][rows][D] partial sums of split items
  float* part_ml;  // [2 * kAttnMaxCtas][rows][2] their running maxima and weights
  int2* desc;      // [items] first partial and number of partials
  float scale;
  float softcap;
  int32_t window;
  int32_t topk;
  int32_t B;        // requests
  int32_t next_n;
  int32_t Hq;
  int32_t group;    // query heads per kv head
  int32_t rows;     // query rows of one item's kv head: next_n * group, or group (top-k)
  int32_t row_tiles;
  int32_t max_blocks;
  int32_t page_shift;
  int32_t q_bf16;   // type of q and out
  int32_t split;    // 0: one CTA per item, no join
  int32_t grid;
  idx_device_errors* errors;
};
// keys one CTA handles at a time (the unit in which an item's length is split)
int attn_unit_keys(int head_dim, int cache_dtype);
int attn_rows_per_item(int head_dim, int rows);
int attn_ctas_per_sm(int head_dim, int rows);
cudaError_t launch_attn_bf16(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_fp16(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_e4m3(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_join(const AttnArgs& a, int rows_per_item, cudaStream_t stream);

}  // namespace idx
