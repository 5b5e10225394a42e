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

}  // namespace xfer
