// Internal declarations of the decode-step calls (include/xfer_decode.h).
#pragma once

#include "internal.h"
#include "xfer_decode.h"

namespace xfer {

// ---- norms, rotation and the cache's rows (rope_store.hip)
struct CacheView {
  uint8_t *k, *v;
  const float *k_scale, *v_scale;
  uint64_t page_stride, token_stride, head_stride;  // bytes
  uint32_t n_pages, page_log2, kv_heads, head_dim;
};
struct RopeStoreArgs {
  CacheView cache;
  const uint16_t *q, *k, *v, *q_weight, *k_weight;
  uint64_t q_ld, k_ld, v_ld, q_out_ld;
  const float *cos_sin;
  const int32_t *positions;
  const int64_t *slots;
  uint16_t *q_out;
  uint32_t tokens, q_heads, max_pos, rot_dim;
  float eps;
};
// Workgroups of the launch (0 heads or tokens: 0).
uint64_t rope_store_workgroups(uint32_t tokens, uint32_t heads, uint32_t head_dim);
hipError_t launch_rope_store(const RopeStoreArgs &a, int kind, int style, hipStream_t stream);

// ---- attention of one new token over a paged cache (attn_paged.hip)
// How a call's work is cut up: query heads of a kv head in m_groups of 16 *
// m_tiles; workgroups of `waves`, of `heads` kv heads side by side, that share the visible tokens (of vis_max a
// row, at most) evenly; whether a (row, kv head) may fall to several of them;
// how many of these an XCD gets at a time if not; whether the cache is read past
// the caches.
struct AttnShape {
  uint32_t m_tiles, m_groups, part_heads, waves, heads, deal;
  uint64_t workgroups;
  bool joined, stream;
};
AttnShape attn_shape(uint32_t rows, uint32_t kv_heads, uint32_t group, uint32_t head_dim, int kind,
                     uint64_t vis_max, uint64_t head_stride);
uint64_t attn_workspace_bytes(const AttnShape &s, uint32_t rows, uint32_t kv_heads, uint32_t head_dim);
struct AttnArgs {
  CacheView cache;
  const uint32_t *page_table, *lens;
  uint64_t table_ld;
  uint32_t rows, max_len, window, sinks;  // window: UINT32_MAX for every token
  const uint16_t *q;
  uint64_t q_ld, out_ld;
  uint32_t q_heads, group;  // group = q_heads / kv_heads
  float scale;
  void *out;
  int out_mode;
  float *part_ml, *part_o;  // (max, sum) of each query head of each part, and its weighted sum
  void *parts;              // where each (row, kv head)'s parts are (NULL: none has two)
};
hipError_t launch_attn(const AttnArgs &a, int kind, const AttnShape &s, hipStream_t stream);

// ---- sampling (sample.hip)
// Workgroups of the widest launch for each row, and the workspace.
uint32_t sample_slices(uint32_t ncols0, uint32_t ncols1);
uint64_t sample_workspace_bytes(uint32_t rows, uint32_t ncols0, uint32_t ncols1);
struct SampleArgs {
  ArgmaxShard s[2];
  uint32_t rows;
  const xfer_sample_params *params;
  const float *u;
  xfer_sampled *out;
  void *workspace;
};
hipError_t launch_sample(const SampleArgs &a, hipStream_t stream);

}  // namespace xfer
