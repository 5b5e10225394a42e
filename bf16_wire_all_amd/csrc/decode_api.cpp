// Exported entry points of the decode-step calls: argument checks in the order
// the header documents, then the kernel launches.  Every check runs on the
// host before anything is enqueued.
#include <algorithm>
#include <cmath>

#include "decode.h"

namespace {

constexpr uint64_t kMaxExtent = 1ull << 47;

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

bool overlaps(uintptr_t a, uint64_t na, uintptr_t b, uint64_t nb) {
  if (na == 0 || nb == 0) return false;
  return a < b + nb && b < a + na;
}

uint32_t element_bytes(int kind) { return kind == XFER_KV_BF16 ? 2 : 1; }

// The checks that every call makes of a cache; on XFER_OK *extent holds the
// bytes from k (and from v) to the end of the last slot.
int cache_checks(const xfer_kv_cache *c, uint64_t *extent) {
  if (!c) return XFER_E_INVAL;
  if (c->kind != XFER_KV_BF16 && c->kind != XFER_KV_E4M3) return XFER_E_INVAL;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return XFER_E_INVAL;
  if (c->page_stride % 16 || c->token_stride % 16 || c->head_stride % 16) return XFER_E_INVAL;
  if (c->n_pages == 0 || c->page_tokens == 0 || c->kv_heads == 0) return XFER_E_INVAL;
  if (c->page_tokens & (c->page_tokens - 1)) return XFER_E_INVAL;
  if (c->kind == XFER_KV_BF16 && (c->k_scale || c->v_scale)) return XFER_E_INVAL;
  if ((uintptr_t)c->k_scale % 4 || (uintptr_t)c->v_scale % 4) return XFER_E_INVAL;
  if (c->reserved) return XFER_E_INVAL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return XFER_E_UNSUPPORTED;
  if (c->page_tokens > 65536) return XFER_E_UNSUPPORTED;
  uint64_t n = (uint64_t)c->head_dim * element_bytes(c->kind);
  const uint64_t step[3][2] = {{c->page_stride, c->n_pages}, {c->token_stride, c->page_tokens},
                               {c->head_stride, c->kv_heads}};
  for (const auto &s : step) {
    uint64_t reach;
    if (__builtin_mul_overflow(s[0], s[1] - 1, &reach) || reach > kMaxExtent) return XFER_E_INVAL;
    n += reach;
  }
  if (n > kMaxExtent) return XFER_E_INVAL;
  *extent = n;
  return XFER_OK;
}

// Whether every element of the cache has bytes of its own: from the smallest
// stride up, each stride must pass the extent of what lies inside it.
bool slots_disjoint(const xfer_kv_cache *c) {
  struct Step {
    uint64_t stride, count;
  } s[3] = {{c->page_stride, c->n_pages}, {c->token_stride, c->page_tokens}, {c->head_stride, c->kv_heads}};
  std::sort(s, s + 3, [](const Step &a, const Step &b) { return a.stride < b.stride; });
  uint64_t extent = (uint64_t)c->head_dim * element_bytes(c->kind);
  for (const Step &t : s) {
    if (t.count == 1) continue;
    if (t.stride < extent) return false;
    extent += t.stride * (t.count - 1);
  }
  return true;
}

// Whether an element of the values shares a byte with one of the keys, whose
// elements are disjoint among themselves: `by` bytes lie between two elements,
// and from stride `level` of s (in descending order) inwards each may still be
// moved either way.
struct Stride {
  uint64_t bytes, count;
};
bool values_touch(const Stride *s, int level, int64_t by, int64_t row) {
  if (level == 3) return by < row && -by < row;
  const int64_t step = (int64_t)s[level].bytes, most = (int64_t)s[level].count - 1;
  if (most == 0) return values_touch(s, level + 1, by, row);
  int64_t inner = row;  // bytes of what lies inside one step
  for (int i = level + 1; i < 3; ++i) inner += (int64_t)s[i].bytes * ((int64_t)s[i].count - 1);
  const int64_t near = -by / step;  // only steps about there can bring them together
  for (int64_t t = std::max(near - 1, -most); t <= std::min(near + 1, most); ++t) {
    const int64_t d = by + t * step;
    if (d < inner && -d < inner && values_touch(s, level + 1, d, row)) return true;
  }
  return false;
}
bool values_apart(const xfer_kv_cache *c) {
  Stride s[3] = {{c->page_stride, c->n_pages}, {c->token_stride, c->page_tokens}, {c->head_stride, c->kv_heads}};
  std::sort(s, s + 3, [](const Stride &a, const Stride &b) { return a.bytes > b.bytes; });
  return !values_touch(s, 0, (int64_t)((uintptr_t)c->v - (uintptr_t)c->k),
                       (int64_t)c->head_dim * element_bytes(c->kind));
}

// Rows of `len` bytes, `pitch` apart.
struct Rows {
  uintptr_t at;
  uint64_t pitch, len, n;
  uint64_t extent() const { return n ? (n - 1) * pitch + len : 0; }
};

// Whether a row of a shares a byte with a row of b.  Slices of one buffer
// (equal pitches) interleave without touching; with other pitches the whole
// extents must be apart.
bool rows_touch(const Rows &a, const Rows &b) {
  if (!a.n || !b.n || !a.len || !b.len || !overlaps(a.at, a.extent(), b.at, b.extent())) return false;
  if (a.pitch != b.pitch || a.n == 1 || b.n == 1) return true;
  const uint64_t d = b.at >= a.at ? (b.at - a.at) % a.pitch : (a.pitch - (a.at - b.at) % a.pitch) % a.pitch;
  return d < a.len || a.pitch - d < b.len;
}

// An ld (elements) of `rows` rows of `row` BF16 elements: a multiple of 8, and
// not so small that rows overlap or so large that they pass the extent limit.
bool ld_ok(uint64_t ld, uint64_t rows, uint64_t row) {
  if (ld % 8) return false;
  if (rows <= 1) return true;
  return ld >= row && ld <= kMaxExtent / 2 && (rows - 1) <= kMaxExtent / 2 / ld;
}

uint32_t log2_of(uint32_t x) { return (uint32_t)__builtin_ctz(x); }

xfer::CacheView view_of(const xfer_kv_cache *c) {
  xfer::CacheView v{};
  v.k = static_cast<uint8_t *>(c->k);
  v.v = static_cast<uint8_t *>(c->v);
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.page_stride = c->page_stride;
  v.token_stride = c->token_stride;
  v.head_stride = c->head_stride;
  v.n_pages = c->n_pages;
  v.page_log2 = log2_of(c->page_tokens);
  v.kv_heads = c->kv_heads;
  v.head_dim = c->head_dim;
  return v;
}

// The sizes of an attention call that the workspace follows from; on XFER_OK
// fills *s.
int attn_sizes(const xfer_kv_cache *c, const xfer_paged_batch *b, uint32_t q_heads, xfer::AttnShape *s) {
  if (q_heads == 0 || q_heads % c->kv_heads) return XFER_E_INVAL;
  if (b->sinks && !b->window) return XFER_E_INVAL;
  if (b->max_len == 0 || b->max_len > 0x7FFFFFFFu) return XFER_E_INVAL;
  uint64_t vis = b->max_len;
  if (b->window) vis = std::min<uint64_t>(vis, (uint64_t)b->window + b->sinks);
  *s = xfer::attn_shape(b->rows, c->kv_heads, q_heads / c->kv_heads, c->head_dim, c->kind, vis, c->head_stride);
  return XFER_OK;
}

// Whether both launches of an attention call are within a grid's limit.
bool attn_launches(const xfer::AttnShape &s, uint64_t rows, uint32_t q_heads) {
  return s.workgroups <= xfer::kMaxGridBlocks && rows * q_heads <= xfer::kMaxGridBlocks;
}

// The pointers and row distances that attention's calls share.
int attn_pointers(const xfer_kv_cache *c, const xfer_paged_batch *b, const void *q, uint64_t q_ld, const void *out,
                  uint64_t out_ld, uint64_t row) {
  const uint64_t R = b->rows, pages = ((uint64_t)b->max_len + c->page_tokens - 1) / c->page_tokens;
  if (!b->page_table || !b->lens || (uintptr_t)b->page_table % 4 || (uintptr_t)b->lens % 4) return XFER_E_INVAL;
  if (R > 1 && (b->table_ld < pages || b->table_ld > kMaxExtent / 4 || R - 1 > kMaxExtent / 4 / b->table_ld))
    return XFER_E_INVAL;
  if (!q || !out || !aligned16(q) || !aligned16(out) || !ld_ok(q_ld, R, row) || !ld_ok(out_ld, R, row))
    return XFER_E_INVAL;
  return XFER_OK;
}

// Whether the output or the workspace (w, need bytes) shares a byte with an
// input, the cache, its scales or one another.
bool attn_outputs_touch(const xfer_kv_cache *c, uint64_t extent, const Rows &o, uintptr_t w, uint64_t need,
                        const Rows *ins, int n) {
  for (int i = 0; i < n; ++i)
    if (rows_touch(o, ins[i]) || overlaps(w, need, ins[i].at, ins[i].extent())) return true;
  for (uintptr_t k : {(uintptr_t)c->k, (uintptr_t)c->v})
    if (overlaps(k, extent, o.at, o.extent()) || overlaps(k, extent, w, need)) return true;
  for (const float *scales : {c->k_scale, c->v_scale})
    if (scales && (overlaps((uintptr_t)scales, c->kv_heads * 4ull, o.at, o.extent()) ||
                   overlaps((uintptr_t)scales, c->kv_heads * 4ull, w, need)))
      return true;
  return overlaps(w, need, o.at, o.extent());
}

// The sizes of a call with shared prefixes.
int shared_sizes(const xfer_kv_cache *c, const xfer_paged_batch *b, const xfer_prefix_groups *g, uint32_t q_heads) {
  if (q_heads == 0 || q_heads % c->kv_heads || g->reserved) return XFER_E_INVAL;
  if (b->max_len == 0 || b->max_len > 0x7FFFFFFFu || (b->sinks && !b->window)) return XFER_E_INVAL;
  if (b->window || !xfer::shared_launches(b->rows, g->groups, c->kv_heads, q_heads / c->kv_heads, c->head_dim, c->kind))
    return XFER_E_UNSUPPORTED;
  return XFER_OK;
}

// The checks of two logit shards that xfer_sample_merge and xfer_logprobs_merge
// share, up to their pointers'.
int shard_checks(const xfer_shard *const (&s)[2]) {
  for (const xfer_shard *x : s)
    if (x->ncols == 0 || (uint64_t)x->col_offset + x->ncols > (1ull << 31)) return XFER_E_INVAL;
  if (s[0]->col_offset < s[1]->col_offset + (uint64_t)s[1]->ncols &&
      s[1]->col_offset < s[0]->col_offset + (uint64_t)s[0]->ncols)
    return XFER_E_INVAL;
  for (const xfer_shard *x : s)
    if (x->ncols > xfer::kArgmaxMaxShardCols) return XFER_E_UNSUPPORTED;
  return XFER_OK;
}

// Bytes of a token's record: its elements, a scale for each 32 of them, and
// zeros up to a multiple of 16.
uint64_t record_bytes(const xfer_kv_cache *c, int bits) {
  const uint64_t n = 2ull * c->kv_heads * c->head_dim;
  return (n * (uint64_t)bits / 8 + n / 32 + 15) / 16 * 16;
}

// Both directions of the wire; the records are read by one and written by the other.
int wire_call(const xfer_kv_cache *cache, const int64_t *slots, uint32_t tokens, int bits, void *records,
              uint64_t record_ld, bool restore, hipStream_t stream) {
  uint64_t extent = 0;
  const int st = cache_checks(cache, &extent);
  if (st != XFER_OK) return st;
  if (bits != XFER_WIRE_E4M3 && bits != XFER_WIRE_E2M1) return XFER_E_INVAL;
  if (restore && (!slots_disjoint(cache) || !values_apart(cache))) return XFER_E_OVERLAP;
  if (tokens == 0) return XFER_OK;
  const uint64_t need = record_bytes(cache, bits);
  if (need > 0x7FFFFFFFu ||
      xfer::wire_workgroups(tokens, cache->kv_heads, cache->head_dim, cache->kind, bits) > xfer::kMaxGridBlocks)
    return XFER_E_UNSUPPORTED;
  if (!slots || (uintptr_t)slots % 8 || !records || !aligned16(records) || record_ld % 16) return XFER_E_INVAL;
  if (tokens > 1 && (record_ld < need || record_ld > kMaxExtent || tokens - 1 > kMaxExtent / record_ld))
    return XFER_E_INVAL;
  const Rows rec{(uintptr_t)records, record_ld, need, tokens};
  const Rows others[3] = {{(uintptr_t)slots, 8, 8, tokens},
                          {(uintptr_t)cache->k_scale, 4, 4, cache->k_scale ? cache->kv_heads : 0},
                          {(uintptr_t)cache->v_scale, 4, 4, cache->v_scale ? cache->kv_heads : 0}};
  const uintptr_t caches[2] = {(uintptr_t)cache->k, (uintptr_t)cache->v};
  for (uintptr_t c : caches) {
    if (overlaps(c, extent, rec.at, rec.extent())) return XFER_E_INVAL;
    for (const Rows &o : others)
      if (restore && overlaps(c, extent, o.at, o.extent())) return XFER_E_INVAL;
  }
  for (const Rows &o : others)
    if (!restore && rows_touch(rec, Rows{o.at, 0, o.extent(), o.n ? 1u : 0u})) return XFER_E_INVAL;

  xfer::WireArgs a{};
  a.cache = view_of(cache);
  a.slots = slots;
  a.records = static_cast<uint8_t *>(records);
  a.record_ld = record_ld;
  a.tokens = tokens;
  if (xfer::launch_wire(a, cache->kind, bits, restore, stream) != hipSuccess) return XFER_E_DEVICE;
  return XFER_OK;
}

}  // namespace

extern "C" {

int xfer_qkv_rope_store(const xfer_kv_cache *cache, const xfer_qkv *in, const xfer_rope *rope, const int64_t *slots,
                        uint16_t *q_out, uint64_t q_out_ld, hipStream_t stream) {
  uint64_t extent = 0;
  const int st = cache_checks(cache, &extent);
  if (st != XFER_OK) return st;
  if (!slots_disjoint(cache) || !values_apart(cache)) return XFER_E_OVERLAP;
  if (!in || !rope || in->reserved || rope->reserved) return XFER_E_INVAL;
  if (rope->style != XFER_ROPE_HALVES && rope->style != XFER_ROPE_PAIRS) return XFER_E_INVAL;
  if (!(in->eps >= 0.0f) || !std::isfinite(in->eps)) return XFER_E_INVAL;
  if (rope->rot_dim % 8 || rope->rot_dim > cache->head_dim) return XFER_E_INVAL;
  if (in->tokens == 0) return XFER_OK;
  const uint64_t T = in->tokens, q_row = (uint64_t)in->q_heads * cache->head_dim;
  const uint64_t kv_row = (uint64_t)cache->kv_heads * cache->head_dim;
  if (rope->rot_dim && (!rope->cos_sin || !aligned16(rope->cos_sin) || !rope->positions ||
                        (uintptr_t)rope->positions % 4 || !rope->max_pos))
    return XFER_E_INVAL;
  if (!slots || (uintptr_t)slots % 8 || !in->k || !in->v || !aligned16(in->k) || !aligned16(in->v)) return XFER_E_INVAL;
  if (in->q_heads && (!in->q || !q_out || !aligned16(in->q) || !aligned16(q_out))) return XFER_E_INVAL;
  if (!aligned16(in->q_weight) || !aligned16(in->k_weight)) return XFER_E_INVAL;
  if (!ld_ok(in->k_ld, T, kv_row) || !ld_ok(in->v_ld, T, kv_row)) return XFER_E_INVAL;
  if (in->q_heads && (!ld_ok(in->q_ld, T, q_row) || !ld_ok(q_out_ld, T, q_row))) return XFER_E_INVAL;

  const uint64_t nq = in->q_heads ? T : 0;
  const Rows out{(uintptr_t)q_out, q_out_ld * 2, q_row * 2, nq};
  const Rows ins[3] = {{(uintptr_t)in->q, in->q_ld * 2, q_row * 2, nq},
                       {(uintptr_t)in->k, in->k_ld * 2, kv_row * 2, T},
                       {(uintptr_t)in->v, in->v_ld * 2, kv_row * 2, T}};
  const bool in_place = nq && q_out == in->q && (q_out_ld == in->q_ld || T == 1);
  for (int i = 0; i < 3; ++i)
    if (!(i == 0 && in_place) && rows_touch(out, ins[i])) return XFER_E_INVAL;
  const uintptr_t caches[2] = {(uintptr_t)cache->k, (uintptr_t)cache->v};
  for (uintptr_t c : caches) {
    if (overlaps(c, extent, out.at, out.extent())) return XFER_E_INVAL;
    for (const Rows &r : ins)
      if (overlaps(c, extent, r.at, r.extent())) return XFER_E_INVAL;
  }
  const uint64_t dim_bytes = cache->head_dim * 2ull, scale_bytes = cache->kv_heads * 4ull;
  const struct {
    const void *at;
    uint64_t bytes;
  } others[7] = {{slots, T * 8},
                 {rope->rot_dim ? rope->positions : nullptr, T * 4},
                 {rope->rot_dim ? rope->cos_sin : nullptr, (uint64_t)rope->max_pos * rope->rot_dim * 4},
                 {in->q_weight, dim_bytes},
                 {in->k_weight, dim_bytes},
                 {cache->k_scale, scale_bytes},
                 {cache->v_scale, scale_bytes}};
  for (const auto &o : others) {
    if (!o.at) continue;
    if (rows_touch(out, Rows{(uintptr_t)o.at, 0, o.bytes, 1})) return XFER_E_INVAL;
    for (uintptr_t c : caches)
      if (overlaps(c, extent, (uintptr_t)o.at, o.bytes)) return XFER_E_INVAL;
  }
  const uint64_t heads = (uint64_t)in->q_heads + 2ull * cache->kv_heads;
  if (heads > UINT32_MAX ||
      xfer::rope_store_workgroups(in->tokens, (uint32_t)heads, cache->head_dim) > xfer::kMaxGridBlocks)
    return XFER_E_UNSUPPORTED;

  xfer::RopeStoreArgs a{};
  a.cache = view_of(cache);
  a.q = in->q;
  a.k = in->k;
  a.v = in->v;
  a.q_weight = in->q_weight;
  a.k_weight = in->k_weight;
  a.q_ld = in->q_ld;
  a.k_ld = in->k_ld;
  a.v_ld = in->v_ld;
  a.q_out_ld = q_out_ld;
  a.cos_sin = rope->cos_sin;
  a.positions = rope->positions;
  a.slots = slots;
  a.q_out = q_out;
  a.tokens = in->tokens;
  a.q_heads = in->q_heads;
  a.max_pos = rope->max_pos;
  a.rot_dim = rope->rot_dim;
  a.eps = in->eps;
  if (xfer::launch_rope_store(a, cache->kind, rope->style, stream) != hipSuccess) return XFER_E_DEVICE;
  return XFER_OK;
}

size_t xfer_attn_workspace_bytes(const xfer_kv_cache *cache, const xfer_paged_batch *batch, uint32_t q_heads) {
  uint64_t extent = 0;
  xfer::AttnShape s{};
  if (!batch || cache_checks(cache, &extent) != XFER_OK || attn_sizes(cache, batch, q_heads, &s) != XFER_OK ||
      !attn_launches(s, batch->rows, q_heads))
    return 0;
  return (size_t)xfer::attn_workspace_bytes(s, batch->rows, cache->kv_heads, cache->head_dim);
}

int xfer_attn_paged(const xfer_kv_cache *cache, const xfer_paged_batch *batch, const uint16_t *q, uint64_t q_ld,
                    uint32_t q_heads, float scale, void *out, uint64_t out_ld, int out_mode, void *workspace,
                    size_t workspace_bytes, hipStream_t stream) {
  uint64_t extent = 0;
  int st = cache_checks(cache, &extent);
  if (st != XFER_OK) return st;
  if (!batch || (out_mode != XFER_OUT_F32 && out_mode != XFER_OUT_BF16)) return XFER_E_INVAL;
  if (!std::isfinite(scale)) return XFER_E_INVAL;
  xfer::AttnShape s{};
  if ((st = attn_sizes(cache, batch, q_heads, &s)) != XFER_OK) return st;
  if (batch->rows == 0) return XFER_OK;
  const uint64_t R = batch->rows, row = (uint64_t)q_heads * cache->head_dim;
  const uint64_t pages = ((uint64_t)batch->max_len + cache->page_tokens - 1) / cache->page_tokens;
  if ((st = attn_pointers(cache, batch, q, q_ld, out, out_ld, row)) != XFER_OK) return st;
  const uint64_t need = xfer::attn_workspace_bytes(s, batch->rows, cache->kv_heads, cache->head_dim);
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return XFER_E_INVAL;

  const uint64_t ob = out_mode == XFER_OUT_F32 ? 4 : 2;
  const Rows o{(uintptr_t)out, out_ld * ob, row * ob, R};
  const Rows ins[3] = {{(uintptr_t)q, q_ld * 2, row * 2, R},
                       {(uintptr_t)batch->page_table, batch->table_ld * 4, pages * 4, R},
                       {(uintptr_t)batch->lens, 4, 4, R}};
  if (attn_outputs_touch(cache, extent, o, (uintptr_t)workspace, need, ins, 3)) return XFER_E_INVAL;
  if (!attn_launches(s, R, q_heads)) return XFER_E_UNSUPPORTED;

  xfer::AttnArgs a{};
  a.cache = view_of(cache);
  a.page_table = batch->page_table;
  a.lens = batch->lens;
  a.table_ld = batch->table_ld;
  a.rows = batch->rows;
  a.max_len = batch->max_len;
  a.window = batch->window ? batch->window : UINT32_MAX;
  a.sinks = batch->sinks;
  a.q = q;
  a.q_ld = q_ld;
  a.out_ld = out_ld;
  a.q_heads = q_heads;
  a.group = q_heads / cache->kv_heads;
  a.scale = scale;
  a.out = out;
  a.out_mode = out_mode;
  a.part_ml = static_cast<float *>(workspace);
  if (xfer::launch_attn(a, cache->kind, s, stream) != hipSuccess) return XFER_E_DEVICE;
  return XFER_OK;
}

size_t xfer_attn_shared_workspace_bytes(const xfer_kv_cache *cache, const xfer_paged_batch *batch,
                                        const xfer_prefix_groups *groups, uint32_t q_heads) {
  uint64_t extent = 0;
  if (!batch || !groups || cache_checks(cache, &extent) != XFER_OK ||
      shared_sizes(cache, batch, groups, q_heads) != XFER_OK || batch->rows == 0)
    return 0;
  return (size_t)xfer::shared_workspace_bytes(batch->rows, groups->groups, cache->kv_heads, q_heads / cache->kv_heads,
                                              cache->head_dim, cache->kind);
}

int xfer_attn_shared(const xfer_kv_cache *cache, const xfer_paged_batch *batch, const xfer_prefix_groups *groups,
                     const uint16_t *q, uint64_t q_ld, uint32_t q_heads, float scale, void *out, uint64_t out_ld,
                     int out_mode, void *workspace, size_t workspace_bytes, hipStream_t stream) {
  uint64_t extent = 0;
  int st = cache_checks(cache, &extent);
  if (st != XFER_OK) return st;
  if (!batch || !groups || (out_mode != XFER_OUT_F32 && out_mode != XFER_OUT_BF16) || !std::isfinite(scale))
    return XFER_E_INVAL;
  if ((st = shared_sizes(cache, batch, groups, q_heads)) != XFER_OK) return st;
  if (batch->rows == 0) return XFER_OK;
  const uint64_t R = batch->rows, G = groups->groups, row = (uint64_t)q_heads * cache->head_dim;
  const uint64_t pages = ((uint64_t)batch->max_len + cache->page_tokens - 1) / cache->page_tokens;
  if ((st = attn_pointers(cache, batch, q, q_ld, out, out_ld, row)) != XFER_OK) return st;
  if (G && (!groups->starts || !groups->shared || (uintptr_t)groups->starts % 4 || (uintptr_t)groups->shared % 4))
    return XFER_E_INVAL;
  const uint64_t need = xfer::shared_workspace_bytes(batch->rows, groups->groups, cache->kv_heads,
                                                     q_heads / cache->kv_heads, cache->head_dim, cache->kind);
  if (!workspace || !aligned16(workspace) || workspace_bytes < need) return XFER_E_INVAL;
  const uint64_t ob = out_mode == XFER_OUT_F32 ? 4 : 2;
  const Rows o{(uintptr_t)out, out_ld * ob, row * ob, R};
  const Rows ins[5] = {{(uintptr_t)q, q_ld * 2, row * 2, R},
                       {(uintptr_t)batch->page_table, batch->table_ld * 4, pages * 4, R},
                       {(uintptr_t)batch->lens, 4, 4, R},
                       {(uintptr_t)groups->starts, 4, 4, G ? G + 1 : 0},
                       {(uintptr_t)groups->shared, 4, 4, G}};
  if (attn_outputs_touch(cache, extent, o, (uintptr_t)workspace, need, ins, 5)) return XFER_E_INVAL;

  xfer::SharedArgs a{};
  a.cache = view_of(cache);
  a.page_table = batch->page_table;
  a.lens = batch->lens;
  a.table_ld = batch->table_ld;
  a.rows = batch->rows;
  a.max_len = batch->max_len;
  a.starts = groups->starts;
  a.shared = groups->shared;
  a.groups = groups->groups;
  a.q = q;
  a.q_ld = q_ld;
  a.out_ld = out_ld;
  a.q_heads = q_heads;
  a.group = q_heads / cache->kv_heads;
  a.scale = scale;
  a.out = out;
  a.out_mode = out_mode;
  if (xfer::launch_shared(a, cache->kind, workspace, stream) != hipSuccess) return XFER_E_DEVICE;
  return XFER_OK;
}

size_t xfer_kv_record_bytes(const xfer_kv_cache *cache, int bits) {
  uint64_t extent = 0;
  if (cache_checks(cache, &extent) != XFER_OK || (bits != XFER_WIRE_E4M3 && bits != XFER_WIRE_E2M1)) return 0;
  const uint64_t need = record_bytes(cache, bits);
  return need > 0x7FFFFFFFu ? 0 : (size_t)need;
}

int xfer_kv_quantize(const xfer_kv_cache *cache, const int64_t *slots, uint32_t tokens, int bits, void *records,
                     uint64_t record_ld, hipStream_t stream) {
  return wire_call(cache, slots, tokens, bits, records, record_ld, false, stream);
}

int xfer_kv_restore(const void *records, uint64_t record_ld, uint32_t tokens, int bits, const xfer_kv_cache *cache,
                    const int64_t *slots, hipStream_t stream) {
  return wire_call(cache, slots, tokens, bits, const_cast<void *>(records), record_ld, true, stream);
}

size_t xfer_sample_workspace_bytes(uint32_t rows, uint32_t ncols0, uint32_t ncols1) {
  if (!ncols0 || !ncols1 || ncols0 > xfer::kArgmaxMaxShardCols || ncols1 > xfer::kArgmaxMaxShardCols) return 0;
  return (size_t)xfer::sample_workspace_bytes(rows, ncols0, ncols1);
}

int xfer_sample_merge(const xfer_shard *s0, const xfer_shard *s1, const xfer_sample_params *params, const float *u,
                      void *out, void *workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!s0 || !s1 || s0->rows != s1->rows) return XFER_E_INVAL;
  const uint64_t R = s0->rows;
  if (R == 0) return XFER_OK;
  const xfer_shard *s[2] = {s0, s1};
  const int st = shard_checks(s);
  if (st != XFER_OK) return st;
  if (R * xfer::sample_slices(s0->ncols, s1->ncols) > xfer::kMaxGridBlocks) return XFER_E_UNSUPPORTED;
  for (const xfer_shard *x : s)
    if (!x->ptr || !aligned16(x->ptr) || !ld_ok(x->ld, R, x->ncols)) return XFER_E_INVAL;
  if (!params || !aligned16(params) || !u || (uintptr_t)u % 4 || !out || !aligned16(out)) return XFER_E_INVAL;
  const uint64_t need = xfer::sample_workspace_bytes((uint32_t)R, s0->ncols, s1->ncols);
  if (!workspace || !aligned16(workspace) || workspace_bytes < need) return XFER_E_INVAL;
  const uintptr_t o = (uintptr_t)out, w = (uintptr_t)workspace;
  const uint64_t out_bytes = R * sizeof(xfer_sampled);
  const Rows ins[4] = {{(uintptr_t)s0->ptr, s0->ld * 2, (uint64_t)s0->ncols * 2, R},
                       {(uintptr_t)s1->ptr, s1->ld * 2, (uint64_t)s1->ncols * 2, R},
                       {(uintptr_t)params, sizeof(xfer_sample_params), sizeof(xfer_sample_params), R},
                       {(uintptr_t)u, 4, 4, R}};
  for (const Rows &r : ins)
    if (overlaps(o, out_bytes, r.at, r.extent()) || overlaps(w, need, r.at, r.extent())) return XFER_E_INVAL;
  if (overlaps(o, out_bytes, w, need)) return XFER_E_INVAL;

  xfer::SampleArgs a{};
  for (int i = 0; i < 2; ++i) a.s[i] = xfer::ArgmaxShard{s[i]->ptr, s[i]->ld, s[i]->ncols, s[i]->col_offset};
  a.rows = (uint32_t)R;
  a.params = params;
  a.u = u;
  a.out = static_cast<xfer_sampled *>(out);
  a.workspace = workspace;
  if (xfer::launch_sample(a, stream) != hipSuccess) return XFER_E_DEVICE;
  return XFER_OK;
}

size_t xfer_logprobs_workspace_bytes(uint32_t rows, uint32_t ncols0, uint32_t ncols1, uint32_t n_tokens,
                                     uint32_t n_top) {
  if (!rows || !ncols0 || !ncols1 || ncols0 > xfer::kArgmaxMaxShardCols || ncols1 > xfer::kArgmaxMaxShardCols ||
      n_tokens > xfer::kMaxTokens || n_top > xfer::kMaxTop ||
      xfer::logprobs_workgroups(rows, ncols0, ncols1) > xfer::kMaxGridBlocks)
    return 0;
  return (size_t)xfer::logprobs_workspace_bytes(rows, ncols0, ncols1, n_tokens, n_top);
}

int xfer_logprobs_merge(const xfer_shard *s0, const xfer_shard *s1, const float *temperature, const int32_t *tokens,
                        uint32_t n_tokens, uint32_t n_top, void *token_out, void *top_out, float *entropy,
                        void *workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!s0 || !s1 || s0->rows != s1->rows) return XFER_E_INVAL;
  const uint64_t R = s0->rows;
  if (R == 0) return XFER_OK;
  const xfer_shard *s[2] = {s0, s1};
  const int st = shard_checks(s);
  if (st != XFER_OK) return st;
  if (n_tokens > xfer::kMaxTokens || n_top > xfer::kMaxTop ||
      xfer::logprobs_workgroups((uint32_t)R, s0->ncols, s1->ncols) > xfer::kMaxGridBlocks)
    return XFER_E_UNSUPPORTED;
  for (const xfer_shard *x : s)
    if (!x->ptr || !aligned16(x->ptr) || !ld_ok(x->ld, R, x->ncols)) return XFER_E_INVAL;
  if ((uintptr_t)temperature % 4 || (uintptr_t)entropy % 4) return XFER_E_INVAL;
  if (n_tokens && (!tokens || (uintptr_t)tokens % 4 || !token_out || (uintptr_t)token_out % 8)) return XFER_E_INVAL;
  if (n_top && (!top_out || (uintptr_t)top_out % 8)) return XFER_E_INVAL;
  const uint64_t need = xfer::logprobs_workspace_bytes((uint32_t)R, s0->ncols, s1->ncols, n_tokens, n_top);
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return XFER_E_INVAL;
  struct Buffer {
    uintptr_t at;
    uint64_t bytes;
  };
  const Buffer outs[4] = {{(uintptr_t)token_out, R * n_tokens * sizeof(xfer_token_logprob)},
                          {(uintptr_t)top_out, R * n_top * sizeof(xfer_top_logprob)},
                          {(uintptr_t)entropy, entropy ? R * 4 : 0},
                          {(uintptr_t)workspace, need}};
  const Rows ins[4] = {{(uintptr_t)s0->ptr, s0->ld * 2, (uint64_t)s0->ncols * 2, R},
                       {(uintptr_t)s1->ptr, s1->ld * 2, (uint64_t)s1->ncols * 2, R},
                       {(uintptr_t)temperature, 4, 4, temperature ? R : 0},
                       {(uintptr_t)tokens, 4ull * n_tokens, 4ull * n_tokens, n_tokens ? R : 0}};
  for (int i = 0; i < 4; ++i) {
    for (const Rows &r : ins)
      if (overlaps(outs[i].at, outs[i].bytes, r.at, r.extent())) return XFER_E_INVAL;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i].at, outs[i].bytes, outs[j].at, outs[j].bytes)) return XFER_E_INVAL;
  }

  xfer::LogprobArgs a{};
  for (int i = 0; i < 2; ++i) a.s[i] = xfer::ArgmaxShard{s[i]->ptr, s[i]->ld, s[i]->ncols, s[i]->col_offset};
  a.rows = (uint32_t)R;
  a.n_tokens = n_tokens;
  a.n_top = n_top;
  a.temperature = temperature;
  a.tokens = tokens;
  a.token_out = static_cast<xfer_token_logprob *>(token_out);
  a.top_out = static_cast<xfer_top_logprob *>(top_out);
  a.entropy = entropy;
  if (xfer::launch_logprobs(a, workspace, stream) != hipSuccess) return XFER_E_DEVICE;
  return XFER_OK;
}

}  // extern "C"
