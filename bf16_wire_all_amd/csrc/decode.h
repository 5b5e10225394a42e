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

// ---- attention of rows with shared prefixes (attn_shared.hip)
constexpr uint32_t kMaxGroups = 4096;
constexpr uint32_t kNoGroup = 0xFFFFFFFFu;
// Tokens first .. first + n - 1 of a row's pages, seen by all query heads of
// q_rows rows from q_row on: a row's own tokens, or a group's shared ones.
struct SharedEntry {
  uint64_t unit0;  // the first of its units, over all entries
  uint32_t row, first, n, q_row, q_rows;
  uint32_t part0;  // its first (kv head, tile of heads) among all entries'
  uint32_t group;  // whose shared tokens the row also sees (kNoGroup: none)
  uint32_t reserved;
};
static_assert(sizeof(SharedEntry) % 8 == 0, "entries lie one after the other");
struct SharedParts {
  uint32_t slot, n;    // its first run's, and how many parts: one of each run,
  uint32_t wgs, lead;  // but of `wgs` workgroups after the first `lead` runs
};
struct SharedArgs {
  CacheView cache;
  const uint32_t *page_table, *lens;
  uint64_t table_ld;
  uint32_t rows, max_len;
  const uint32_t *starts, *shared;
  uint32_t groups;
  const uint16_t *q;
  uint64_t q_ld, out_ld;
  uint32_t q_heads, group;  // group = q_heads / kv_heads
  float scale;
  void *out;
  int out_mode;
  // set by the launch
  uint32_t slot_heads;  // query heads of a slot for parts of few
  uint32_t *many_places;  // workgroups of each XCD that take groups of many query heads
  uint32_t places_of_xcd, unit_cost, many_unit_cost;
  SharedEntry *entries;  // of rows, then of groups of few query heads
  SharedEntry *many;     // of groups of many (NULL: there is none)
  SharedParts *parts;
  uint32_t many_part0;
  float *part_ml, *part_o;
  uint64_t many_place0, whole0;  // the first places of groups of many, and of results that one workgroup has whole
};
bool shared_launches(uint32_t rows, uint32_t groups, uint32_t kv_heads, uint32_t group, uint32_t head_dim, int kind);
uint64_t shared_workspace_bytes(uint32_t rows, uint32_t groups, uint32_t kv_heads, uint32_t group, uint32_t head_dim,
                                int kind);
hipError_t launch_shared(const SharedArgs &a, int kind, void *workspace, hipStream_t stream);

// ---- a cache's slots as records for the wire, and back (kv_wire.hip)
struct WireArgs {
  CacheView cache;
  const int64_t *slots;
  uint8_t *records;  // written by quantize, read by restore
  uint64_t record_ld;
  uint32_t tokens;
  // set by the launch: log2 of the lanes that share a head's row, and what divides by a record's rows
  uint32_t lanes_log2, magic, magic_shift;
};
uint64_t wire_workgroups(uint32_t tokens, uint32_t kv_heads, uint32_t head_dim, int kind, int bits);
hipError_t launch_wire(const WireArgs &a, int kind, int bits, bool restore, hipStream_t stream);

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

// ---- log probabilities (logprobs.hip)
constexpr uint32_t kMaxTokens = 16, kMaxTop = 32;  // of a row
struct LogprobArgs {
  ArgmaxShard s[2];
  uint32_t rows, n_tokens, n_top;
  const float *temperature;
  const int32_t *tokens;
  xfer_token_logprob *token_out;
  xfer_top_logprob *top_out;
  float *entropy;
  // set by the launch: how rows are cut up, and the workspace of rows in several parts
  uint32_t parts, slices[2], width[2];
  void *sums;
  uint64_t *keys;
  uint32_t *ranks;
};
uint64_t logprobs_workgroups(uint32_t rows, uint32_t ncols0, uint32_t ncols1);
uint64_t logprobs_workspace_bytes(uint32_t rows, uint32_t ncols0, uint32_t ncols1, uint32_t n_tokens, uint32_t n_top);
hipError_t launch_logprobs(const LogprobArgs &a, void *workspace, hipStream_t stream);

}  // namespace xfer
