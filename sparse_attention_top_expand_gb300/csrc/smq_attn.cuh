// Parameter blocks and launchers of the attention operators: the append of
// rotated keys and values (smq_append.cu) and the attention over the paged
// cache (smq_attn.cu). Shared with their host side (smq_attn_api.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace smq {

constexpr int kAttnTile = 128;  // tokens per tile

struct AppendParams {
  int32_t rows;
  int32_t heads;
  int32_t kv_heads;
  int32_t page_size;
  int32_t rot_dim;
  int32_t interleaved;
  int64_t num_positions;
  int64_t num_pages;
  int64_t page_stride;        // elements
  int64_t scale_page_stride;  // floats
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  const int64_t* positions;
  const float* cos_sin;
  const int64_t* slot_mapping;
  uint16_t* q_out;
  void* k_cache;
  void* v_cache;
  float* k_scales;
  float* v_scales;
  int32_t* status;
};

struct AttnParams {
  int32_t rows;
  int32_t kv_heads;
  int32_t group;      // query heads per kv head
  int32_t head_dim;
  int32_t page_size;
  int32_t page_shift;  // log2 of page_size, or -1
  float scale_log2;   // softmax_scale * log2(e)
  const uint16_t* q;
  int64_t q_stride;
  const void* k_cache;
  const void* v_cache;
  const float* k_scales;
  const float* v_scales;
  int64_t num_pages;
  int64_t page_stride;        // elements
  int64_t scale_page_stride;  // floats
  const int32_t* block_table;
  int32_t bt_rows;
  int32_t bt_stride;
  const int32_t* row_indices;  // may be null
  const int32_t* row_ks;       // may be null
  const int32_t* row_ke;       // null: selected
  const int32_t* token_ids;    // null: decode
  int32_t num_ids;
  int32_t ids_ld;
  uint16_t* out;
  float* lse;  // may be null
  // partial results: CTA c leaves slot 2 c for an item that an earlier CTA began and slot 2 c + 1 for
  // one that a later CTA continues; seg_info[c] = (row, kv head, CTAs that continue it, 0) of the latter
  int4* seg_info;    // [grid]
  float2* part_ml;   // [2 grid][group] running maximum (log2) and sum
  float* part_o;     // [2 grid][group][head_dim]
  int32_t* status;
  // failure path: every wait gives up after wait_ns; with stall_tile >= 0 the loaders of CTA 0
  // withhold that tile's keys (tests of the failure path only)
  int64_t wait_ns;
  int32_t stall_tile;
};

cudaError_t launch_append(const AppendParams& p, int head_dim, bool e4m3, int num_sms, cudaStream_t stream);
cudaError_t prepare_attention(int head_dim, bool e4m3, int group);  // raise the dynamic-smem limit, once per plan
cudaError_t launch_attention(const AttnParams& p, bool e4m3, int grid, cudaStream_t stream);

}  // namespace smq
