// Attention of one new token over a paged cache for rows in groups that begin
// with the same tokens: what a group shares is read once for all its rows.
//
// A softmax over a row's tokens splits into sums over any parts of them, each
// with a maximum of its own, so a row is its group's shared tokens and the
// rest of its own, and three steps make it up:
//   1. plan: one workgroup turns the groups and lengths into two lists of
//      entries, a run of tokens with the query heads that see all of it: a row's
//      own tokens with its heads, a group's shared tokens with the heads of
//      all its rows.  Rows that do not see all of the shared tokens are kept
//      out of them and read theirs alone, so no entry needs a mask;
//   2. walk: the entries' units (128 tokens of a kv head and up to 16 or 32
//      query heads) are one line that is cut into equal runs, as the attention
//      of one token cuts its rows, and with the same walk;
//   3. join: a workgroup for each (row, query head) scales the parts of the
//      shared tokens and of the row's own to the largest maximum and adds
//      them up, in a fixed order.
#include "attn_tile.h"

namespace xfer {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr uint32_t kUnit = kTile * kWaves;       // tokens of a unit
constexpr uint32_t kComputeUnits = 256;
constexpr uint32_t kXcds = 8;
constexpr int kPlanThreads = 1024;
constexpr int kParts = 3;  // BF16 numbers of a weight: exact, and no slower, since the memory bounds the walk

// Groups of more than kFewHeads query heads for a kv head go another way, kManyHeads of them and
// kManyUnit tokens at a time, and at least kManyLeast such units to a workgroup.
constexpr uint32_t kFewHeads = 32, kManyHeads = 128, kManyUnit = 64, kManyLeast = 4;

constexpr uint32_t kZeros = 16;  // bytes that stand for tokens that are not there

// ------------------------------------------------------------------- plan

// What a number of entries comes to, in the list whose workgroups take `tile`
// heads and `unit` tokens at a time: units, and tiles of heads of a kv head.
struct Extent {
  uint64_t units;
  uint32_t tiles;
};
__device__ __forceinline__ Extent operator+(const Extent &x, const Extent &y) { return {x.units + y.units, x.tiles + y.tiles}; }
__device__ __forceinline__ Extent extent_of(const SharedArgs &a, const SharedEntry &e, uint32_t tile, uint32_t unit) {
  const uint32_t tiles = (uint32_t)(((uint64_t)e.q_rows * a.group + tile - 1) / tile);
  return {(uint64_t)((e.n + unit - 1) / unit) * a.cache.kv_heads * tiles, tiles};
}

// Sums (or maxima) over the lanes up to each, by DPP moves; lanes that a move does not reach give 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ Extent dpp(const Extent &x) {
  const uint32_t lo = dpp<CTRL, ROWS>((uint32_t)x.units), hi = dpp<CTRL, ROWS>((uint32_t)(x.units >> 32));
  return {(uint64_t)hi << 32 | lo, dpp<CTRL, ROWS>(x.tiles)};
}
template <typename T, typename F>
__device__ __forceinline__ T wave_scan(T x, F &&op) {
  x = op(x, dpp<0x111, 0xF>(x));
  x = op(x, dpp<0x112, 0xF>(x));
  x = op(x, dpp<0x114, 0xF>(x));
  x = op(x, dpp<0x118, 0xF>(x));
  x = op(x, dpp<0x142, 0xA>(x));
  return op(x, dpp<0x143, 0xC>(x));
}

__global__ __launch_bounds__(kPlanThreads) void shared_plan_kernel(SharedArgs a) {
  constexpr uint32_t kPlanWaves = kPlanThreads / 64;
  __shared__ uint32_t start[kMaxGroups + 1], prefix[kMaxGroups];
  __shared__ uint32_t wave_top[kPlanWaves];
  __shared__ Extent wave_sum[3][kPlanWaves];
  const uint32_t tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  if (tid < kZeros / 4) reinterpret_cast<uint32_t *>(a.zeros)[tid] = 0;
  // This thread's starts, groups and rows.  Loads that depend on nothing first.
  const uint32_t n_starts = a.groups + 1, s_each = (n_starts + kPlanThreads - 1) / kPlanThreads;
  const uint32_t s0 = min(tid * s_each, n_starts), s1 = min(s0 + s_each, n_starts);
  const uint32_t g0 = min(s0, a.groups), g1 = min(s1, a.groups);
  const uint32_t r_each = (a.rows + kPlanThreads - 1) / kPlanThreads;
  const uint32_t r0 = min(tid * r_each, a.rows), r1 = min(r0 + r_each, a.rows);
  const uint32_t first_len = r0 < r1 ? a.lens[r0] : 0, first_shared = g0 < g1 ? a.shared[g0] : 0;
  // The groups' first rows: a start below the one before counts as that one,
  // so that no row is in two groups, whatever the caller's numbers are.
  auto given = [&](uint32_t i) { return a.groups ? min(a.starts[i], a.rows) : a.rows; };
  auto larger = [](uint32_t x, uint32_t y) { return max(x, y); };
  uint32_t top = 0;
  for (uint32_t i = s0; i < s1; ++i) start[i] = top = max(top, given(i));
  const uint32_t through = wave_scan(top, larger);
  if (lane == 63) wave_top[wave] = through;
  __syncthreads();
  uint32_t before = __shfl_up(through, 1);  // by all lanes: one that sits out gives nothing
  if (lane == 0) before = 0;
  for (uint32_t w = 0; w < wave; ++w) before = max(before, wave_top[w]);
  for (uint32_t i = s0; i < s1; ++i) start[i] = max(start[i], before);
  __syncthreads();
  for (uint32_t g = g0; g < g1; ++g) {
    const uint32_t row = start[g], n = start[g + 1] - row;
    uint32_t p = n > 1 ? min(g == g0 ? first_shared : a.shared[g], a.max_len) : 0;
    if (p) p = min(p, a.lens[row]);  // the first row's pages are read
    prefix[g] = p;
  }
  __syncthreads();
  // A group's shared tokens, if its rows' heads are in the list of many or the other.
  auto of_group = [&](uint32_t g, bool many) {
    SharedEntry e{};
    const uint32_t rows = start[g + 1] - start[g];
    if (!prefix[g] || ((uint64_t)rows * a.group > kFewHeads) != many) return e;
    e.n = prefix[g];
    e.row = e.q_row = start[g];
    e.q_rows = rows;
    return e;
  };
  auto of_row = [&](uint32_t i) {
    SharedEntry e{};
    uint32_t lo = 0, hi = n_starts;  // the first start past row i
    while (lo < hi) {
      const uint32_t mid = (lo + hi) / 2;
      if (start[mid] <= i)
        lo = mid + 1;
      else
        hi = mid;
    }
    const uint32_t len = min(i == r0 ? first_len : a.lens[i], a.max_len);
    const uint32_t p = lo > 0 && lo <= a.groups ? prefix[lo - 1] : 0;
    e.first = p <= len ? p : 0;
    e.n = len - e.first;
    e.row = e.q_row = i;
    e.q_rows = 1;
    e.group = e.first ? lo - 1 : kNoGroup;
    return e;
  };
  // Where each entry's units and parts begin: rows, groups of few heads after them, and groups of many.
  Extent mine[3] = {};
  for (uint32_t i = r0; i < r1; ++i) mine[0] = mine[0] + extent_of(a, of_row(i), a.tile, kUnit);
  for (uint32_t g = g0; g < g1; ++g) {
    mine[1] = mine[1] + extent_of(a, of_group(g, false), a.tile, kUnit);
    mine[2] = mine[2] + extent_of(a, of_group(g, true), kManyHeads, kManyUnit);
  }
  Extent at[3], all[3];
  auto add = [](const Extent &x, const Extent &y) { return x + y; };
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    at[k] = wave_scan(mine[k], add);
    if (lane == 63) wave_sum[k][wave] = at[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const Extent waves = wave_scan(lane < kPlanWaves ? wave_sum[k][lane] : Extent{}, add);  // up to each wave
    auto of_wave = [&](uint32_t w) -> Extent {
      const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)waves.units, w),
                     hi = __builtin_amdgcn_readlane((uint32_t)(waves.units >> 32), w);
      return {(uint64_t)hi << 32 | lo, (uint32_t)__builtin_amdgcn_readlane(waves.tiles, w)};
    };
    all[k] = of_wave(kPlanWaves - 1);
    const Extent before_wave = wave ? of_wave(wave - 1) : Extent{};
    at[k] = {at[k].units - mine[k].units + before_wave.units, at[k].tiles - mine[k].tiles + before_wave.tiles};
  }
  at[1] = at[1] + all[0];
  auto put = [&](SharedEntry &to, SharedEntry e, Extent &from, uint32_t part0, uint32_t tile, uint32_t unit) {
    e.unit0 = from.units;
    e.part0 = part0 + from.tiles * a.cache.kv_heads;
    to = e;
    from = from + extent_of(a, e, tile, unit);
  };
  for (uint32_t i = r0; i < r1; ++i) put(a.entries[i], of_row(i), at[0], 0, a.tile, kUnit);
  for (uint32_t g = g0; g < g1; ++g) {
    put(a.entries[a.rows + g], of_group(g, false), at[1], 0, a.tile, kUnit);
    if (a.many) put(a.many[g], of_group(g, true), at[2], a.many_part0, kManyHeads, kManyUnit);
  }
  if (tid == 0) {
    a.entries[a.rows + a.groups].unit0 = all[0].units + all[1].units;
    if (a.many) {
      a.many[a.groups].unit0 = all[2].units;
      // Both lists' workgroups are to end together, by what a unit of each costs.
      const double few = (double)(all[0].units + all[1].units) * a.unit_cost, many = (double)all[2].units * a.many_unit_cost;
      uint32_t n = few + many > 0 ? (uint32_t)(a.places_of_xcd * (many / (few + many)) + 0.5) : 0;
      if (all[2].units) n = max(n, 1u);
      if (few > 0) n = min(n, a.places_of_xcd - 1);
      *a.many_places = n;
    }
  }
}

// ------------------------------------------------------------------- walk

// What a (entry, kv head, tile of heads) that fell to several workgroups leaves:
// its first part's slot (kWhole: one workgroup did it all), and how many parts.
constexpr uint32_t kWhole = 0xFFFFFFFFu;

template <int D, int TILES>
struct WalkLds {
  static constexpr int kPad = 4;  // floats between rows of the exchange, so that 16 rows' stores fall on all banks
  float o[kWaves][16][D + kPad];
  float m[TILES][kWaves][16], l[TILES][kWaves][16];
};

// The entry that unit `from` of a list falls to; by all threads.
__device__ __forceinline__ uint32_t entry_at(const SharedEntry *entries, uint32_t n, uint64_t from) {
  __shared__ uint32_t start;
  for (uint32_t i = threadIdx.x; i < n; i += kThreads)
    if (entries[i].unit0 <= from && from < entries[i + 1].unit0) start = i;
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(start);
}

// The run of workgroup wg of n_wg.
template <int D, int KIND, int TILES>
__device__ __forceinline__ void walk(const SharedArgs &a, uint32_t wg, uint32_t n_wg, WalkLds<D, TILES> &lds) {
  using L = Layout<D, KIND>;
  using R = Residence<D, KIND, TILES>;
  constexpr int MR = TILES;
  constexpr uint32_t kHeads = 16 * TILES;
  auto &lds_o = lds.o;
  auto &lds_all_m = lds.m;
  auto &lds_all_l = lds.l;
  const uint32_t n_entries = a.rows + a.groups;
  const uint64_t all = a.entries[n_entries].unit0, per = (all + n_wg - 1) / n_wg, from = wg * per;
  if (from >= all) return;
  uint64_t left = min(per, all - from);
  uint32_t index = entry_at(a.entries, n_entries, from);
  SharedEntry e = a.entries[index];
  uint64_t at = from - e.unit0;

  const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64, n = lane % 16,
                 g = lane / 16;
  // The queries, in the lanes' order, where the exchange lies later.
  v4u *const lds_q = reinterpret_cast<v4u *>(&lds_o[0][0][0]);
  static_assert(!R::kQInLds || MR * L::kMfmaK * 64 * 16 <= (int)sizeof(lds_o), "they fit");
  bool first_segment = true;

#pragma unroll 1
  while (left) {
    const uint32_t heads = e.q_rows * a.group, m_groups = (heads + kHeads - 1) / kHeads;
    const uint32_t units = (e.n + kUnit - 1) / kUnit, inner_n = m_groups * a.cache.kv_heads;
    uint32_t inner = __builtin_amdgcn_readfirstlane((uint32_t)(at / units));
    uint32_t unit = __builtin_amdgcn_readfirstlane((uint32_t)(at % units));
#pragma unroll 1
    for (; inner < inner_n && left; ++inner, unit = 0) {
      const uint32_t take = (uint32_t)min(left, (uint64_t)(units - unit));
      const uint32_t kvh = inner / m_groups, h0 = inner % m_groups * kHeads;
      const uint32_t v0 = unit * kUnit, v1 = min((unit + take) * kUnit, e.n);
      const Visible vis{e.n, 0, e.first};
      // Q: query head h0 + 16 * r + n of the entry, the dims that this lane's K loads hold.
      v4u q[R::kQInLds ? 1 : MR][L::kMfmaK];
      auto load_q = [&](int r, int k) {
        const uint32_t h = h0 + 16 * r + n;
        const uint32_t d = KIND == XFER_KV_BF16 ? k * 32 + g * 8 : (k / 2) * 64 + g * 16 + (k % 2) * 8;
        if (h >= heads) return v4u{0, 0, 0, 0};
        return *reinterpret_cast<const v4u *>(a.q + (e.q_row + h / a.group) * a.q_ld +
                                              (uint64_t)(kvh * a.group + h % a.group) * D + d);
      };
      if constexpr (R::kQInLds) {
        for (int k = wave; k < MR * L::kMfmaK; k += kWaves) lds_q[k * 64 + lane] = load_q(k / L::kMfmaK, k % L::kMfmaK);
        __syncthreads();
      } else {
#pragma unroll
        for (int r = 0; r < MR; ++r)
#pragma unroll
          for (int k = 0; k < L::kMfmaK; ++k) q[r][k] = load_q(r, k);
      }
      float scale2 = a.scale * 1.4426950408889634f;
      if (KIND == XFER_KV_E4M3 && a.cache.k_scale) scale2 *= a.cache.k_scale[kvh];
      const uint32_t *table = a.page_table + e.row * a.table_ld;
      v4f o[MR][L::kMfmaV];
      float mx[MR], sum[MR];
      attn_walk<D, KIND, MR, kParts, kUnit, false>(a.cache, kvh, table, vis, v0 + wave * kTile, v1, scale2, n, g, lane, q,
                                                   lds_q, o, mx, sum);

      // The waves' results, joined in LDS.
      const bool whole = take == units;
      const uint32_t slot = 2 * wg + (first_segment ? 0 : 1);
      if (unit == 0 && tid == 0)
        a.parts[e.part0 + inner] = whole ? SharedParts{kWhole, 1} : SharedParts{slot, 1 + (uint32_t)((units - take + per - 1) / per)};
#pragma unroll
      for (int r = 0; r < MR; ++r) {
        sum[r] += __shfl_xor(sum[r], 16);
        sum[r] += __shfl_xor(sum[r], 32);
        if (g == 0) {
          lds_all_m[r][wave][n] = mx[r];
          lds_all_l[r][wave][n] = sum[r];
        }
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < MR; ++r) {
        auto &lds_m = lds_all_m[r];
        auto &lds_l = lds_all_l[r];
        if (r) __syncthreads();
        {
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) top = fmaxf(top, lds_m[w][n]);
          const float f = mx[r] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[r] - top);
#pragma unroll
          for (int j = 0; j < L::kMfmaV; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) lds_o[wave][n][dim_of<D, KIND>(j, 4 * g + i)] = o[r][j][i] * f;
        }
        __syncthreads();
#pragma unroll
        for (uint32_t i = tid; i < 4 * D; i += kThreads) {
          const uint32_t hq = i / (D / 4), d = i % (D / 4) * 4, h = h0 + 16 * r + hq;
          if (h >= heads) continue;
          float top = -INFINITY, total = 0;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) top = fmaxf(top, lds_m[w][hq]);
          v4f v = {0, 0, 0, 0};
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            const float mw = lds_m[w][hq];
            total += mw == -INFINITY ? lds_l[w][hq] : lds_l[w][hq] * __builtin_amdgcn_exp2f(mw - top);
            v += *reinterpret_cast<const v4f *>(&lds_o[w][hq][d]);
          }
          if constexpr (KIND == XFER_KV_BF16) {
            if (isnan(v.x + v.y + v.z + v.w)) v = with_infinities<KIND>(a.cache, kvh, table, vis, v0, v1, v, d);
          }
          // a whole one's place is its row's and head's, in the half for shared or own tokens
          const uint64_t mine = (uint64_t)(e.q_row + h / a.group) * a.q_heads + kvh * a.group + h % a.group;
          const uint64_t to = whole ? a.whole0 + (index < a.rows ? 0 : (uint64_t)a.rows * a.q_heads) + mine
                                    : (uint64_t)slot * kHeads + 16 * r + hq;
          *reinterpret_cast<v4f *>(a.part_o + to * D + d) = v;
          if (d == 0) {
            a.part_ml[2 * to] = top;
            a.part_ml[2 * to + 1] = total;
          }
        }
      }
      left -= take;
      first_segment = false;
      if (left) __syncthreads();  // LDS is written again
    }
    at = 0;
    if (left) {
      do e = a.entries[++index];
      while (e.n == 0);  // there is one with tokens as long as units are left
    }
  }
}

// --------------------------------------------------- many heads' shared tokens

// Four waves take 32 query heads each of the same tokens, 64 at a time, which go
// through LDS in BF16, a row for each token.  Scores are K Q^T (32x32x16), so a lane
// holds 16 tokens' scores of one query in each of two blocks, and in the order in
// which it holds them they are the operand of V^T P^T: a lane's eight tokens are two
// fours, and each four of a dim is what one transposing read of LDS (4 rows of 16
// columns for 16 lanes) gives.  Nothing crosses lanes but the two halves' maxima.
// BF16 rows go from memory to LDS without a register; the next tile is on its way
// while one is used.  A row's pieces of 16 bytes are placed by the token's last three
// bits, so that eight lanes side by side that read a column of pieces touch all banks.
template <int D, int KIND>
struct Many {
  static constexpr int kBytes = KIND == XFER_KV_BF16 ? 2 : 1;
  static constexpr int kEach = D / 32;                             // pieces of keys, and of values, of a thread
  static constexpr uint32_t kRowLanes = D / 8;                     // that hold a row of pieces
  static constexpr uint32_t kRows = 64 / kRowLanes;                // rows that a wave moves at once
  static constexpr int kPerSimd = D == 256 ? 1 : D == 128 ? 2 : 3;
  static constexpr uint32_t kTileBytes = kManyUnit * D * 2;        // of keys, and of values
};

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v16f mfma32(v4u a, v4u b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}
// Element `lane % 16` of the rows that the lanes of 16 point into, four lanes to a row.
__device__ __forceinline__ v2u column4(const uint8_t *p) {
  typedef __attribute__((address_space(3))) v4s *Lds;
  return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)p));
}

// The run of workgroup wg of n_wg; lds0 and lds1 are two variables, not one of two: then the compiler knows that what
// is on its way to one does not change the other.
template <int D, int KIND, int PARTS>
__device__ __forceinline__ void walk_many(const SharedArgs &a, uint32_t wg, uint32_t n_wg, uint8_t *lds0, uint8_t *lds1) {
  using M = Many<D, KIND>;
  constexpr int kDims = D / 32;   // blocks of dims
  constexpr int kSteps = D / 16;  // of a score
  __shared__ __align__(8) uint16_t lds_gone[2][kWaves];  // a bit for each token of 16 that is not there
  const uint64_t all = a.many[a.groups].unit0, share = (all + n_wg - 1) / n_wg;
  const uint64_t per = share < kManyLeast ? kManyLeast : share, from = wg * per;
  if (from >= all) return;
  uint64_t left = min(per, all - from);
  uint32_t index = entry_at(a.many, a.groups, from);
  SharedEntry e = a.many[index];
  uint64_t at = from - e.unit0;

  const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64, n = lane % 32,
                 hf = lane / 32;
  // This lane moves tokens 16 * wave + kRows * i + row of a tile, the pieces that lie at its place.
  const uint32_t row = lane / M::kRowLanes, place = lane % M::kRowLanes;
  const uint32_t slot_mask = (1u << a.cache.page_log2) - 1;
  // Where its operands lie: a step's keys at key0 ^ 32 * step, a dim block's values at value0 ^ 64 * block; other tokens' 2 D
  // bytes further on for each.
  const uint32_t key0 = n * 2 * D + (hf ^ (n & 7)) * 16;
  const uint32_t four = 4 * hf + lane % 16 / 4, column = 2 * (lane / 16 & 1) + lane % 4 / 2;
  const uint32_t value0 = four * 2 * D + (column ^ four) * 16 + lane % 2 * 8;
  bool first_segment = true;

#pragma unroll 1
  while (left) {
    const uint32_t heads = e.q_rows * a.group, tiles = (heads + kManyHeads - 1) / kManyHeads;
    const uint32_t units = (e.n + kManyUnit - 1) / kManyUnit, inner_n = tiles * a.cache.kv_heads;
    uint32_t inner = __builtin_amdgcn_readfirstlane((uint32_t)(at / units));
    uint32_t unit = __builtin_amdgcn_readfirstlane((uint32_t)(at % units));
#pragma unroll 1
    for (; inner < inner_n && left; ++inner, unit = 0) {
      const uint32_t take = (uint32_t)min(left, (uint64_t)(units - unit));
      const uint32_t kvh = inner / tiles, h = inner % tiles * kManyHeads + 32 * wave + n;  // this lane's query head
      const uint64_t head = (uint64_t)kvh * a.group + h % a.group;
      const uint32_t *table = a.page_table + e.row * a.table_ld;
      const uint8_t *kbase = a.cache.k + kvh * a.cache.head_stride, *vbase = a.cache.v + kvh * a.cache.head_stride;

      // The pages of this lane's tokens of the tile from token t on.
      struct Pages {
        uint32_t page[M::kEach];
      };
      auto look_up = [&](uint32_t t) {
        Pages p;
#pragma unroll
        for (int i = 0; i < M::kEach; ++i)
          p.page[i] = table[min(t + 16 * wave + M::kRows * i + row, e.n - 1) >> a.cache.page_log2];
        return p;
      };
      // Moves a tile to buffer b: BF16 at once, E4M3 by way of registers and put().
      uint32_t held[2][M::kEach][2];
      auto fetch = [&](uint32_t t, const Pages &p, uint8_t *lds, uint16_t *lds_gone) {
        uint32_t gone = 0;
#pragma unroll
        for (int i = 0; i < M::kEach; ++i) {
          const uint32_t local = 16 * wave + M::kRows * i + row, token = t + local;
          const bool there = token < e.n && p.page[i] < a.cache.n_pages;
          const uint64_t absent = __ballot(!there);
          if (absent) {
#pragma unroll
            for (uint32_t r = 0; r < M::kRows; ++r) gone |= (uint32_t)(absent >> (r * M::kRowLanes) & 1) << (M::kRows * i + r);
          }
          const uint64_t off = p.page[i] * a.cache.page_stride + (token & slot_mask) * a.cache.token_stride +
                               (place ^ (local & 7)) * 8 * M::kBytes;
          // one that is not there is all zeros: no weight times it is NaN
          const uint8_t *key = there ? kbase + off : a.zeros, *value = there ? vbase + off : a.zeros;
          if constexpr (KIND == XFER_KV_BF16) {
            typedef const __attribute__((address_space(1))) void *Global;
            typedef __attribute__((address_space(3))) void *Lds;
            uint8_t *to = lds + (wave * M::kEach + i) * 1024;
            __builtin_amdgcn_global_load_lds((Global)key, (Lds)to, 16, 0, 0);
            __builtin_amdgcn_global_load_lds((Global)value, (Lds)(to + M::kTileBytes), 16, 0, 0);
          } else {
            const v2u k = *reinterpret_cast<const v2u *>(key), v = *reinterpret_cast<const v2u *>(value);
            held[0][i][0] = k.x, held[0][i][1] = k.y;
            held[1][i][0] = v.x, held[1][i][1] = v.y;
          }
        }
        if (lane == 0) lds_gone[wave] = (uint16_t)gone;
      };
      auto put = [&](uint8_t *lds) {
        if constexpr (KIND == XFER_KV_E4M3) {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv)
#pragma unroll
            for (int i = 0; i < M::kEach; ++i) {
              const uint32_t w0 = held[kv][i][0], w1 = held[kv][i][1];
              *reinterpret_cast<v4u *>(lds + kv * M::kTileBytes + (wave * M::kEach + i) * 1024 + lane * 16) =
                  v4u{e4m3x2_to_bf16<false>(w0), e4m3x2_to_bf16<true>(w0), e4m3x2_to_bf16<false>(w1), e4m3x2_to_bf16<true>(w1)};
            }
        }
        // What goes to LDS on its own counts as a load, which a barrier need not wait for.
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
      };

      const uint32_t t0 = unit * kManyUnit, t1 = t0 + take * kManyUnit;
      fetch(t0, look_up(t0), lds0, lds_gone[0]);
      Pages next = look_up(t0 + kManyUnit);
      float scale2 = a.scale * 1.4426950408889634f;
      if (KIND == XFER_KV_E4M3 && a.cache.k_scale) scale2 *= a.cache.k_scale[kvh];
      // a negative scale's sign goes to the queries, so that the largest product is the largest score
      const uint32_t flip = scale2 < 0 ? 0x80008000u : 0;
      scale2 = __builtin_fabsf(scale2);
      v4u q[kSteps];
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        q[k] = v4u{0, 0, 0, 0};
        if (h < heads) q[k] = *reinterpret_cast<const v4u *>(a.q + (e.q_row + h / a.group) * a.q_ld + head * D + 16 * k + 8 * hf);
        q[k] ^= flip;
      }
      v16f o[kDims];
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[d] = v16f{};
      float mx = -INFINITY, sum = 0;
      put(lds0);
      // The tile from token t on, which is in `tile`, while the next goes to `other`.
      auto step = [&](uint32_t t, const uint8_t *tile, const uint16_t *tile_gone, uint8_t *other, uint16_t *other_gone) {
        if (t + kManyUnit < t1) {
          fetch(t + kManyUnit, next, other, other_gone);
          next = look_up(t + 2 * kManyUnit);
        }
        const uint8_t *keys = tile, *values = tile + M::kTileBytes;
        const v2u out = *reinterpret_cast<const v2u *>(tile_gone);
        // Operands are read from LDS a group of products ahead; the barriers keep the compiler from reading each where it is used.
        v16f s[2] = {v16f{}, v16f{}};
        v4u key[2][4];
        auto read_keys = [&](int g) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            key[g % 2][i] = *reinterpret_cast<const v4u *>(keys + (key0 ^ 32 * (2 * g + i / 2)) + i % 2 * 64 * D);
        };
        read_keys(0);
#pragma unroll
        for (int g = 0; g < kSteps / 2; ++g) {
          if (g + 1 < kSteps / 2) read_keys(g + 1);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i % 2] = mfma32(key[g % 2][i], q[2 * g + i / 2], s[i % 2]);
          __builtin_amdgcn_sched_barrier(0);
        }
        v4u value[2][kDims];
        auto read_values = [&](int g) {  // 16 tokens
#pragma unroll
          for (int d = 0; d < kDims; ++d) {
            const uint8_t *p = values + (value0 ^ 64 * d) + 16 * g * 2 * D;
            const v2u lo = column4(p), hi = column4(p + 8 * 2 * D);
            value[g % 2][d] = v4u{lo.x, lo.y, hi.x, hi.y};
          }
        };
        read_values(0);
        if ((out.x | out.y) != 0) {
#pragma unroll
          for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (out[blk] >> (8 * (i / 4) + 4 * hf + i % 4) & 1) s[blk][i] = -INFINITY;
        }
        // Scores above the running maximum; where one passes it by kRaise, the maximum moves and they with it.
        float base = mx == -INFINITY ? 0.0f : mx, top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[0][i] = fmaf(s[0][i], scale2, -base);
          s[1][i] = fmaf(s[1][i], scale2, -base);
          top = fmaxf(top, fmaxf(s[0][i], s[1][i]));
        }
        if (__any(top + base > mx + kRaise)) {
          top = fmaxf(top, __shfl_xor(top, 32)) + base;
          const float raised = fmaxf(mx, top);
          const float f = mx == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx - raised);
          const float by = base - (raised == -INFINITY ? 0.0f : raised);
          mx = raised;
          sum *= f;
#pragma unroll
          for (int d = 0; d < kDims; ++d) o[d] *= f;
          s[0] += by;
          s[1] += by;
        }
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          v4u w[PARTS][2];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float x0 = __builtin_amdgcn_exp2f(s[blk][2 * i]), x1 = __builtin_amdgcn_exp2f(s[blk][2 * i + 1]);
            sum += x0 + x1;
#pragma unroll
            for (int c = 0; c < PARTS; ++c) {
              const uint32_t two = bf16x2(x0, x1);
              w[c][i / 4][i % 4] = two;
              x0 -= __uint_as_float(two << 16);
              x1 -= __uint_as_float(two & 0xFFFF0000u);
            }
          }
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const int g = 2 * blk + st;
            if (g < 3) read_values(g + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < PARTS; ++c)
#pragma unroll
              for (int d = 0; d < kDims; ++d) o[d] = mfma32(value[g % 2][d], w[c][st], o[d]);
            if (g == 0) __builtin_amdgcn_sched_barrier(0);
          }
        }
        put(other);
      };
#pragma unroll 1
      for (uint32_t t = t0; t < t1; t += 2 * kManyUnit) {
        step(t, lds0, lds_gone[0], lds1, lds_gone[1]);
        if (t + kManyUnit < t1) step(t + kManyUnit, lds1, lds_gone[1], lds0, lds_gone[0]);
      }

      // This wave's results: lane n, hf holds dims 32 d + 8 (i / 4) + 4 hf + i % 4 of query n.
      const bool whole = take == units;
      const uint32_t slot = 2 * wg + (first_segment ? 0 : 1);
      if (unit == 0 && tid == 0)
        a.parts[e.part0 + inner] = whole ? SharedParts{kWhole, 1} : SharedParts{slot, 1 + (uint32_t)((units - take + per - 1) / per)};
      sum += __shfl_xor(sum, 32);
      if (h < heads) {
        const uint64_t to = whole ? a.whole0 + ((uint64_t)a.rows + e.q_row + h / a.group) * a.q_heads + head
                                  : a.many_place0 + (uint64_t)slot * kManyHeads + 32 * wave + n;
        if (hf == 0) {
          a.part_ml[2 * to] = mx;
          a.part_ml[2 * to + 1] = sum;
        }
        const Visible vis{e.n, 0, 0};
#pragma unroll
        for (int d = 0; d < kDims; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v4f x = {o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
            const uint32_t dim = 32 * d + 8 * j + 4 * hf;
            if constexpr (KIND == XFER_KV_BF16) {
              if (isnan(x.x + x.y + x.z + x.w) && !isnan(sum))
                x = with_infinities<KIND>(a.cache, kvh, table, vis, t0, min(t1, e.n), x, dim);
            }
            *reinterpret_cast<v4f *>(a.part_o + to * D + dim) = x;
          }
      }
      left -= take;
      first_segment = false;
    }
    at = 0;
    if (left) {
      do e = a.many[++index];
      while (e.n == 0);  // there is one with tokens as long as units are left
    }
  }
}

// Neighbouring runs on one XCD: its L2 then serves the tokens that the heads of an entry have in common.
template <int D, int KIND, int TILES>
__global__ __launch_bounds__(kThreads, (Residence<D, KIND, TILES>::kPerSimd)) void shared_walk_kernel(SharedArgs a) {
  __shared__ WalkLds<D, TILES> lds;
  walk<D, KIND, TILES>(a, blockIdx.x % kXcds * (gridDim.x / kXcds) + blockIdx.x / kXcds, gridDim.x, lds);
}

// Both lists at once, so that one's loads and the other's products share the compute units: of the workgroups
// that are resident, as many take the list of many heads as the plan found, spread evenly over the others.
template <int D, int KIND, int TILES, int PARTS>
__global__ __launch_bounds__(kThreads, (Many<D, KIND>::kPerSimd)) void shared_both_kernel(SharedArgs a) {
  constexpr uint32_t kTile = 2 * Many<D, KIND>::kTileBytes;
  __shared__ __align__(16) uint8_t lds0[kTile < sizeof(WalkLds<D, TILES>) ? sizeof(WalkLds<D, TILES>) : kTile];
  __shared__ __align__(16) uint8_t lds1[kTile];
  const uint32_t xcd = blockIdx.x % kXcds, place = blockIdx.x / kXcds, places = gridDim.x / kXcds;
  const uint32_t many = *a.many_places;  // of an XCD's places
  const uint32_t before = place * many / places;
  if ((place + 1) * many / places > before)
    walk_many<D, KIND, PARTS>(a, xcd * many + before, kXcds * many, lds0, lds1);
  else
    walk<D, KIND, TILES>(a, xcd * (places - many) + place - before, kXcds * (places - many),
                         *reinterpret_cast<WalkLds<D, TILES> *>(lds0));
}

// ------------------------------------------------------------------- join

// kJoinWaves (or one) for each (row, query head): its parts of the shared tokens, then of its own, each scaled to
// the largest maximum, in a fixed order.  One wave where there are many heads to join, since each has few parts then
// (6336 heads of 64: 6 us with a wave each, 18 with four); four where few heads are cut into many parts.
constexpr uint32_t kJoinHeads = 4096;  // from which on a wave takes a whole one

template <int D, int WAVES>
__global__ __launch_bounds__(kThreads) void shared_join_kernel(SharedArgs a) {
  constexpr uint32_t kLanes = D / 4, kAtOnce = 64 / kLanes;  // of a part, and parts of a wave at once
  __shared__ float lds_top[kWaves], lds_total[kWaves];
  __shared__ v4f lds_o[WAVES][kLanes];
  const uint32_t lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64) % WAVES;
  const uint32_t item = WAVES == 1 ? blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : blockIdx.x;
  if (item >= a.rows * a.q_heads) return;  // by waves that share nothing
  const uint32_t row = item / a.q_heads, head = item % a.q_heads, kvh = head / a.group, h = head % a.group;
  const SharedEntry own = a.entries[row];
  struct Source {
    uint32_t n;                 // parts
    uint64_t at0, at1, stride;  // places: part 0's; part p's at1 + p * stride
  };
  auto source = [&](const SharedEntry &e, bool prefix, uint32_t tile, uint64_t cut0) {
    Source s{};
    if (!e.n) return s;
    const uint32_t heads = e.q_rows * a.group, m_groups = (heads + tile - 1) / tile;
    const uint32_t i = (row - e.q_row) * a.group + h;
    const SharedParts p = a.parts[e.part0 + kvh * m_groups + i / tile];
    s.n = p.n;
    if (p.slot == kWhole) {
      s.at0 = a.whole0 + (prefix ? (uint64_t)a.rows * a.q_heads : 0) + (uint64_t)row * a.q_heads + head;
    } else {
      // Part p > 0 is the first thing that the workgroup p further on did.
      s.at0 = cut0 + (uint64_t)p.slot * tile + i % tile;
      s.at1 = cut0 + (uint64_t)(p.slot / 2 * 2) * tile + i % tile;
      s.stride = 2 * tile;
    }
    return s;
  };
  Source pre{};
  if (own.group != kNoGroup) {
    const SharedEntry e = a.entries[a.rows + own.group];
    pre = e.n ? source(e, true, a.tile, 0) : source(a.many[own.group], true, kManyHeads, a.many_place0);
  }
  const Source mine = source(own, false, a.tile, 0);
  const uint32_t n = pre.n + mine.n;
  auto place = [&](uint32_t p) -> uint64_t {
    const Source &s = p < pre.n ? pre : mine;
    const uint32_t k = p < pre.n ? p : p - pre.n;
    return k ? s.at1 + k * s.stride : s.at0;
  };

  // Lane l of wave w has part p0 + l * WAVES + w of every 64 * WAVES.
  float top = -INFINITY;
#pragma unroll 1
  for (uint32_t p0 = 0; p0 < n; p0 += 64 * WAVES) {
    const uint32_t p = p0 + lane * WAVES + wave;
    top = fmaxf(top, p < n ? a.part_ml[2 * place(p)] : -INFINITY);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
  if constexpr (WAVES > 1) {
    if (lane == 0) lds_top[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = fmaxf(top, lds_top[w]);
  }
  float total = 0;
  v4f r = {0, 0, 0, 0};
  const uint32_t sub = lane / kLanes, d4 = lane % kLanes;
#pragma unroll 1
  for (uint32_t p0 = 0; p0 < n; p0 += 64 * WAVES) {
    const uint32_t p = p0 + lane * WAVES + wave;
    float f = 0;
    if (p < n) {
      const uint64_t at = place(p);
      const float m = a.part_ml[2 * at], l = a.part_ml[2 * at + 1];
      f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
      total += m == -INFINITY ? l : l * f;
      if (f == 0.0f) f = __uint_as_float(1);  // a part's infinity stays one, however small its weights
    }
    const uint32_t count = wave < n - p0 ? min((n - p0 - wave + WAVES - 1) / WAVES, 64u) : 0;
#pragma unroll 4
    for (uint32_t k0 = 0; k0 < count; k0 += kAtOnce) {
      const uint32_t k = k0 + sub;
      const float fk = __shfl(f, k);
      if (k < count) r += fk * *reinterpret_cast<const v4f *>(a.part_o + place(p0 + k * WAVES + wave) * D + 4 * d4);
    }
  }
#pragma unroll
  for (uint32_t d = kLanes; d < 64; d *= 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] += __shfl_xor(r[i], d);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d);
  if constexpr (WAVES > 1) {
    if (lane == 0) lds_total[wave] = total;
    if (sub == 0) lds_o[wave][d4] = r;
    __syncthreads();
    if (wave != 0) return;
    total = lds_total[0];
    if (sub == 0) {
#pragma unroll
      for (int w = 1; w < WAVES; ++w) r += lds_o[w][d4];
    }
#pragma unroll
    for (int w = 1; w < WAVES; ++w) total += lds_total[w];
  }
  if (sub != 0) return;
  const float v_scale = a.cache.v_scale ? a.cache.v_scale[kvh] : 1.0f;
  r = total == 0.0f ? v4f{0, 0, 0, 0} : r * (v_scale / total);
  const uint64_t at = row * a.out_ld + (uint64_t)head * D + 4 * d4;
  if (a.out_mode == XFER_OUT_F32)
    *reinterpret_cast<v4f *>(static_cast<float *>(a.out) + at) = r;
  else
    *reinterpret_cast<v2u *>(static_cast<uint16_t *>(a.out) + at) = v2u{bf16x2(r.x, r.y), bf16x2(r.z, r.w)};
}

// ----------------------------------------------------------------- launches

template <int D, int KIND>
hipError_t launch_kind(const SharedArgs &a, uint32_t workgroups, uint32_t many_workgroups, hipStream_t stream) {
  const dim3 block(kThreads);
  if (!a.many)
    return a.tile == 16 ? launch(shared_walk_kernel<D, KIND, 1>, dim3(workgroups), block, 0, stream, a)
                        : launch(shared_walk_kernel<D, KIND, 2>, dim3(workgroups), block, 0, stream, a);
  const dim3 grid(many_workgroups);
  if (a.out_mode == XFER_OUT_F32)
    return a.tile == 16 ? launch(shared_both_kernel<D, KIND, 1, 3>, grid, block, 0, stream, a)
                        : launch(shared_both_kernel<D, KIND, 2, 3>, grid, block, 0, stream, a);
  return a.tile == 16 ? launch(shared_both_kernel<D, KIND, 1, 2>, grid, block, 0, stream, a)
                      : launch(shared_both_kernel<D, KIND, 2, 2>, grid, block, 0, stream, a);
}
template <int D>
hipError_t launch_dim(const SharedArgs &a, int kind, uint32_t workgroups, uint32_t many_workgroups, hipStream_t stream) {
  hipError_t e = launch(shared_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
  if (e != hipSuccess) return e;
  e = kind == XFER_KV_BF16 ? launch_kind<D, XFER_KV_BF16>(a, workgroups, many_workgroups, stream)
                           : launch_kind<D, XFER_KV_E4M3>(a, workgroups, many_workgroups, stream);
  if (e != hipSuccess) return e;
  const uint32_t items = a.rows * a.q_heads;
  if (items >= kJoinHeads)
    return launch(shared_join_kernel<D, 1>, dim3((items + kWaves - 1) / kWaves), dim3(kThreads), 0, stream, a);
  return launch(shared_join_kernel<D, kWaves>, dim3(items), dim3(kThreads), 0, stream, a);
}

struct Shape {
  uint32_t tile, workgroups, many_workgroups;
  uint64_t parts, many_part0;             // (entry, kv head, tile)s at most, and where those of many heads begin
  uint64_t places, many_place0, whole0;   // query heads of all parts, and where those of many heads and whole ones begin
};
template <int D, int KIND>
uint32_t per_simd(uint32_t tile) {
  return tile == 16 ? Residence<D, KIND, 1>::kPerSimd : Residence<D, KIND, 2>::kPerSimd;
}
template <int KIND>
uint32_t per_simd(uint32_t head_dim, uint32_t tile) {
  return head_dim == 64 ? per_simd<64, KIND>(tile) : head_dim == 128 ? per_simd<128, KIND>(tile) : per_simd<256, KIND>(tile);
}
Shape shape_of(uint32_t rows, uint32_t groups, uint32_t kv_heads, uint32_t group, uint32_t head_dim, int kind) {
  Shape s{};
  // 32 heads at a time where a row or the average group has more than 16
  s.tile = group > 16 ? 32 : 16;
  s.workgroups = kComputeUnits * (kind == XFER_KV_BF16 ? per_simd<XFER_KV_BF16>(head_dim, s.tile)
                                                       : per_simd<XFER_KV_E4M3>(head_dim, s.tile));
  const uint64_t row_tiles = (group + s.tile - 1) / s.tile;
  s.many_part0 = kv_heads * (rows * row_tiles + (uint64_t)rows * group / s.tile + groups);
  s.parts = s.many_part0;
  s.many_place0 = 2ull * s.workgroups * s.tile;
  s.whole0 = s.many_place0;
  if (groups && (uint64_t)rows * group > kFewHeads) {  // some group may be that large
    s.workgroups = s.many_workgroups = kComputeUnits * (head_dim == 256 ? 1 : head_dim == 128 ? 2 : 3);
    s.many_place0 = 2ull * s.workgroups * s.tile;
    s.whole0 = s.many_place0;
    s.parts += kv_heads * ((uint64_t)rows * group / kManyHeads + groups);
    s.whole0 += 2ull * s.many_workgroups * kManyHeads;
  }
  s.places = s.whole0 + 2ull * rows * kv_heads * group;
  return s;
}
uint64_t up16(uint64_t x) { return (x + 15) / 16 * 16; }

}  // namespace

bool shared_launches(uint32_t rows, uint32_t groups, uint32_t kv_heads, uint32_t group, uint32_t head_dim, int kind) {
  return groups <= kMaxGroups && (uint64_t)rows * kv_heads * group <= kMaxGridBlocks &&
         shape_of(rows, groups, kv_heads, group, head_dim, kind).parts <= UINT32_MAX;
}

// Layout: the entries, the parts of each (entry, kv head, tile), (max, sum) of each part, the weighted sums.
uint64_t shared_workspace_bytes(uint32_t rows, uint32_t groups, uint32_t kv_heads, uint32_t group, uint32_t head_dim,
                                int kind) {
  const Shape s = shape_of(rows, groups, kv_heads, group, head_dim, kind);
  return 2 * kZeros + up16(((uint64_t)rows + 2ull * groups + 2) * sizeof(SharedEntry)) + up16(s.parts * sizeof(SharedParts)) + up16(s.places * 8) +
         s.places * head_dim * 4;
}

hipError_t launch_shared(const SharedArgs &in, int kind, void *workspace, hipStream_t stream) {
  SharedArgs a = in;
  const Shape s = shape_of(a.rows, a.groups, a.cache.kv_heads, a.group, a.cache.head_dim, kind);
  a.tile = s.tile;
  a.whole0 = s.whole0;
  uint8_t *at = static_cast<uint8_t *>(workspace);
  a.zeros = at;
  a.many_places = reinterpret_cast<uint32_t *>(at + kZeros);
  a.places_of_xcd = s.many_workgroups / kXcds;
  a.unit_cost = kUnit * 2 * a.cache.head_dim * (kind == XFER_KV_BF16 ? 2 : 1) / 64;
  a.many_unit_cost = a.cache.head_dim * (a.out_mode == XFER_OUT_F32 ? 4 : 3) * 2;
  a.entries = reinterpret_cast<SharedEntry *>(at += 2 * kZeros);
  a.parts = reinterpret_cast<SharedParts *>(at += up16(((uint64_t)a.rows + 2ull * a.groups + 2) * sizeof(SharedEntry)));
  if (s.many_workgroups) a.many = a.entries + a.rows + a.groups + 1;
  a.many_part0 = (uint32_t)s.many_part0;
  a.many_place0 = s.many_place0;
  a.part_ml = reinterpret_cast<float *>(at += up16(s.parts * sizeof(SharedParts)));
  a.part_o = reinterpret_cast<float *>(at + up16(s.places * 8));
  if (a.cache.head_dim == 64) return launch_dim<64>(a, kind, s.workgroups, s.many_workgroups, stream);
  if (a.cache.head_dim == 128) return launch_dim<128>(a, kind, s.workgroups, s.many_workgroups, stream);
  return launch_dim<256>(a, kind, s.workgroups, s.many_workgroups, stream);
}

}  // namespace xfer
