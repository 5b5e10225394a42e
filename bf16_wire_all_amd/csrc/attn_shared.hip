// Attention of one new token over a paged cache for rows in groups that begin
// with the same tokens: what a group shares is read once for all its rows.
//
// A softmax over a row's tokens splits into sums over any parts of them, each
// with a maximum of its own, so a row is its group's shared tokens and the
// rest of its own, and three steps make it up:
//   1. plan: the groups and lengths become entries, a run of tokens with the
//      query heads that see all of it: a row's own tokens with its heads, a
//      group's shared tokens with the heads of all its rows.  Rows that do not
//      see all of the shared tokens are kept out of them and read theirs
//      alone, so no entry needs a mask.  Up to 255 rows and groups, every
//      workgroup of the walk makes the plan itself (64 answers: 41.3 us; by a
//      launch of its own 5.2 us and then 39.8); for more a workgroup of
//      shared_plan_kernel does (6.4 us for 300);
//   2. walk, two ways in one launch:
//      - entries of up to 32 query heads for a kv head (or of one row): their
//        units (32 tokens of a kv head and up to 16 or 32 query heads) are one
//        line that is cut into equal runs, one for each wave, with the walk of
//        the attention of one token; four runs of one kind are joined in LDS.  The memory bounds it, or, where runs
//        are short, its latency: 2.5 us for a unit;
//      - groups of more: units of 64 tokens and 128 query heads through LDS,
//        a run for each workgroup.  The matrix cores and the weights between
//        the products bound it.
//      The resident workgroups are shared out between the two so that both end
//      together (in one launch after the other 64 answers took 85 us, so 58);
//   3. join: one or four waves for each (row, query head) scale the parts of the
//      shared tokens and of the row's own to the largest maximum and add
//      them up, in a fixed order.
//
// 64 answers to a prompt of 8192 tokens (32 query heads on 8 of 128, 124 MB):
// 42-45 us of walk and 9.4 of join, on two sets of inputs in turn or on three;
// 24 rows over 131056 shared tokens in F32 (548 MB, 129 GFLOP with the weights in
// three parts): 164-195 + 12 us.
#include "attn_tile.h"

#include <type_traits>

namespace xfer {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr uint32_t kUnit = kTile;                // tokens of a unit
// Units of a wave's run, at least: 4 drafted positions each of 4 requests of up to 6000 tokens 23.6 us and 9.9 of join;
// 4 units 28.7 + 7.5, 8 units 39.8 + 6.5 (measured where each run left a part).
constexpr uint32_t kLeast = 2;
constexpr uint32_t kComputeUnits = 256;
constexpr uint32_t kXcds = 8;
constexpr int kPlanThreads = 1024;
// BF16 numbers of a weight in the walk of few heads: exact.  With two, 2^-17, drafted positions take 22.0 us for 23.2, and 64
// answers and 300 rows as long as now.
constexpr int kParts = 3;

// Groups of more than kFewHeads query heads for a kv head go another way, kManyHeads of them and
// kManyUnit tokens at a time (groups of 40 heads of 128: 74 us over 8 x 8000 tokens and 40 over 30000, 32 heads at a time 99
// and 59; of 64 in E4M3 45, 32 at a time 40), and at least kManyLeast such units to a workgroup (of a group that has as
// many; with 1 in 64 answers' 16 shared tokens 25 us, with 4 whatever there is 35).
constexpr uint32_t kFewHeads = 32, kManyHeads = 128, kManyUnit = 64, kManyLeast = 4;
// Scores in powers of two up to which the maximum's own rounding, 2^-18, moves no weight by more than that.  Beside larger
// ones all are rounded as it is: 64 answers 42.0 us so, 41.5 with fused products alone, which made alike scores of 2^9 weigh
// differently from tile to tile and those of 2^31 infinite.
constexpr float kRounded = 128.0f;

__device__ const v4u kZeros = {0, 0, 0, 0};  // stands for tokens that are not there

// ------------------------------------------------------------------- plan

// What a number of entries comes to, in the list whose workgroups take `tile`
// heads and `unit` tokens at a time: units, and tiles of heads of a kv head.
struct Extent {
  uint64_t units;
  uint32_t tiles;
};
__device__ __forceinline__ Extent operator+(const Extent &x, const Extent &y) { return {x.units + y.units, x.tiles + y.tiles}; }
__device__ __forceinline__ Extent extent_of(const SharedArgs &a, const SharedEntry &e, uint32_t tile, uint32_t unit) {
  const uint32_t tiles = (e.q_rows * a.group + tile - 1) >> (31 - __builtin_clz(tile));  // a power of two
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

// Query heads of a tile in the list of few: 16 at a time, or 32 where there are more, so that their tokens are read once
// (16 groups of 20 heads over 6000 tokens each 92 us, 16 at a time 128; 4 such groups of up to 6000, which leave workgroups
// without work, 24 and 22.6).
__device__ __forceinline__ uint32_t tile_of(uint32_t heads) { return heads > 16 ? 32 : 16; }

template <int THREADS>
struct PlanLds {
  static constexpr uint32_t kGroups = THREADS == kPlanThreads ? kMaxGroups : THREADS;
  uint32_t start[kGroups + 1], prefix[kGroups];
  uint32_t len[THREADS == kPlanThreads ? 1 : THREADS];  // of the rows, where each thread has one at most
  uint32_t wave_top[THREADS / 64], longest;
  Extent wave_sum[2][THREADS / 64];
};

// The lists, by all threads of a workgroup: begin(units of rows and groups of few heads, of groups of many, most tokens of
// one of those), then put(many, index, entry) by one thread for each entry.
template <int THREADS, typename Begin, typename Put>
__device__ __forceinline__ void plan(const SharedArgs &a, PlanLds<THREADS> &lds, Begin &&begin, Put &&put) {
  constexpr uint32_t kPlanWaves = THREADS / 64;
  constexpr bool kOne = THREADS != kPlanThreads;  // a thread has one row and one start at most
  auto &start = lds.start;
  auto &prefix = lds.prefix;
  const uint32_t tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  // This thread's starts, groups and entries (rows, then groups).  Loads that depend on nothing first.
  const uint32_t n_starts = a.groups + 1, s_each = kOne ? 1 : (n_starts + THREADS - 1) / THREADS;
  const uint32_t s0 = min(tid * s_each, n_starts), s1 = min(s0 + s_each, n_starts);
  const uint32_t g0 = min(s0, a.groups), g1 = min(s1, a.groups);
  const uint32_t n_entries = a.rows + a.groups, e_each = kOne ? 1 : (n_entries + THREADS - 1) / THREADS;
  const uint32_t e0 = min(tid * e_each, n_entries), e1 = min(e0 + e_each, n_entries);
  const uint32_t first_len = e0 < a.rows ? a.lens[e0] : 0, first_shared = g0 < g1 ? a.shared[g0] : 0;
  // The groups' first rows: a start below the one before counts as that one,
  // so that no row is in two groups, whatever the caller's numbers are.
  auto given = [&](uint32_t i) { return a.groups ? min(a.starts[i], a.rows) : a.rows; };
  auto larger = [](uint32_t x, uint32_t y) { return max(x, y); };
  uint32_t top = 0;
  for (uint32_t i = s0; i < s1; ++i) start[i] = top = max(top, given(i));
  if (kOne) lds.len[tid] = first_len;
  const uint32_t through = wave_scan(top, larger);
  if (lane == 63) lds.wave_top[wave] = through;
  if (tid == 0) lds.longest = 0;
  __syncthreads();
  uint32_t before = __shfl_up(through, 1);  // by all lanes: one that sits out gives nothing
  if (lane == 0) before = 0;
  for (uint32_t w = 0; w < wave; ++w) before = max(before, lds.wave_top[w]);
  for (uint32_t i = s0; i < s1; ++i) start[i] = max(start[i], before);
  __syncthreads();
  for (uint32_t g = g0; g < g1; ++g) {
    const uint32_t row = start[g], n = start[g + 1] - row;
    uint32_t p = n > 1 ? min(g == g0 ? first_shared : a.shared[g], a.max_len) : 0;
    if (p) p = min(p, kOne ? lds.len[row] : a.lens[row]);  // the first row's pages are read
    prefix[g] = p;
    if (p && n * a.group > kFewHeads) atomicMax(&lds.longest, p);
  }
  __syncthreads();
  // A group's shared tokens, if its rows' heads are in the list of many or the other.
  auto of_group = [&](uint32_t g, bool many) {
    SharedEntry e{};
    const uint32_t rows = start[g + 1] - start[g];
    if (!prefix[g] || (rows * a.group > kFewHeads) != many) return e;
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
    const uint32_t len = min(i == e0 ? first_len : a.lens[i], a.max_len);
    const uint32_t p = lo > 0 && lo <= a.groups ? prefix[lo - 1] : 0;
    e.first = p <= len ? p : 0;
    e.n = len - e.first;
    e.row = e.q_row = i;
    e.q_rows = 1;
    e.group = e.first ? lo - 1 : kNoGroup;
    return e;
  };
  auto of = [&](uint32_t i) { return i < a.rows ? of_row(i) : of_group(i - a.rows, false); };
  // Where each entry's units and parts begin, in either list.
  auto few = [&](const SharedEntry &e) { return extent_of(a, e, tile_of(e.q_rows * a.group), kUnit); };
  auto many = [&](const SharedEntry &e) { return extent_of(a, e, kManyHeads, kManyUnit); };
  const SharedEntry first = e0 < e1 ? of(e0) : SharedEntry{};
  Extent at[2] = {}, all[2] = {};
  for (uint32_t i = e0; i < e1; ++i) {
    at[0] = at[0] + few(i == e0 ? first : of(i));
    if (i >= a.rows) at[1] = at[1] + many(of_group(i - a.rows, true));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const Extent mine = at[k];
    at[k] = wave_scan(mine, [](const Extent &x, const Extent &y) { return x + y; });
    if (lane == 63) lds.wave_sum[k][wave] = at[k];
    at[k] = {at[k].units - mine.units, at[k].tiles - mine.tiles};
  }
  __syncthreads();
  const uint32_t longest = lds.longest;
#pragma unroll
  for (uint32_t w = 0; w < kPlanWaves; ++w)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (w == wave) at[k] = at[k] + all[k];
      all[k] = all[k] + lds.wave_sum[k][w];
    }
  begin(all[0].units, all[1].units, longest);
  auto place = [&](SharedEntry &e, Extent &from, uint32_t part0, const Extent &extent) {
    e.unit0 = from.units;
    e.part0 = part0 + from.tiles * a.cache.kv_heads;
    from = from + extent;
  };
  for (uint32_t i = e0; i < e1; ++i) {
    SharedEntry e = i == e0 ? first : of(i);
    place(e, at[0], 0, few(e));
    put(false, i, e);
    if (i < a.rows || !a.many) continue;
    e = of_group(i - a.rows, true);
    place(e, at[1], a.many_part0, many(e));
    put(true, i - a.rows, e);
  }
}

// Of an XCD's workgroups, those that take the list of many: both lists' are to end together, by what a unit of each costs.
__device__ __forceinline__ uint32_t many_places(const SharedArgs &a, uint64_t few_units, uint64_t many_units) {
  const float few = (float)few_units * (float)a.unit_cost, many = (float)many_units * (float)a.many_unit_cost;
  uint32_t n = few + many > 0 ? (uint32_t)((float)a.places_of_xcd * (many / (few + many)) + 0.5f) : 0;
  if (many_units) n = max(n, 1u);
  if (few_units) n = min(n, a.places_of_xcd - 1);
  return n;
}

__global__ __launch_bounds__(kPlanThreads) void shared_plan_kernel(SharedArgs a) {
  __shared__ PlanLds<kPlanThreads> lds;
  plan<kPlanThreads>(
      a, lds,
      [&](uint64_t few_units, uint64_t many_units, uint32_t longest) {
        if (threadIdx.x != 0) return;
        a.entries[a.rows + a.groups].unit0 = few_units;
        if (!a.many) return;
        a.many[a.groups].unit0 = many_units;
        a.many[a.groups].n = longest;
        *a.many_places = many_places(a, few_units, many_units);
      },
      [&](bool many, uint32_t i, const SharedEntry &e) { (many ? a.many : a.entries)[i] = e; });
}

// The list that a workgroup of the walk takes, in LDS: where each thread has one row and one start at most, every
// workgroup makes it itself, which costs no more than to read it and saves a launch; the first one also
// writes both lists for the join.
struct LocalPlan {
  SharedEntry list[kThreads + 1];
};
// choose(many_places): whether this workgroup takes the list of many.
template <typename Choose>
__device__ __forceinline__ bool plan_here(const SharedArgs &a, LocalPlan &to, PlanLds<kThreads> &lds, Choose &&choose) {
  bool takes_many = false;
  plan<kThreads>(
      a, lds,
      [&](uint64_t few_units, uint64_t many_units, uint32_t longest) {
        takes_many = choose(a.many ? many_places(a, few_units, many_units) : 0);
        if (threadIdx.x != 0) return;
        SharedEntry &end = to.list[takes_many ? a.groups : a.rows + a.groups];
        end.unit0 = takes_many ? many_units : few_units;
        end.n = longest;
      },
      [&](bool many, uint32_t i, const SharedEntry &e) {
        if (many == takes_many) to.list[i] = e;
        if (blockIdx.x == 0) (many ? a.many : a.entries)[i] = e;
      });
  __syncthreads();
  return takes_many;
}

// ------------------------------------------------------------------- walk

// What a (entry, kv head, tile of heads) that fell to several runs leaves:
// its first part's slot (kWhole: one run did it all), and how many parts.
constexpr uint32_t kWhole = 0xFFFFFFFFu;

template <int D, int KIND, int TILES, bool JOIN>
union WalkLds {
  static constexpr int kPad = 4;  // floats between rows of the exchange, so that 16 rows' stores fall on all banks
  static constexpr int kMost = TILES == 2 && Residence<D, KIND, 2>::kQInLds ? 2 : Residence<D, KIND, 1>::kQInLds ? 1 : 0;
  v4u q[kMost ? kWaves : 1][kMost ? kMost * Layout<D, KIND>::kMfmaK * 64 : 1];  // queries that registers do not hold, of each wave
  struct {
    float o[JOIN ? kWaves : 1][16][D + kPad];
    float m[kWaves][16], l[kWaves][16];
  } exchange;
};

// Query heads of a slot for what a wave has of a tile's tokens.
constexpr uint32_t slot_heads(int tiles) { return 16 * tiles; }

// An entry that is the same for all lanes.
__device__ __forceinline__ SharedEntry scalar(const SharedEntry &e) {
  static_assert(sizeof(SharedEntry) % 4 == 0, "words");
  uint32_t w[sizeof(SharedEntry) / 4];
  __builtin_memcpy(w, &e, sizeof(e));
#pragma unroll
  for (uint32_t &x : w) x = __builtin_amdgcn_readfirstlane(x);
  SharedEntry s;
  __builtin_memcpy(&s, w, sizeof(s));
  return s;
}
// The entry that unit `from` of a list falls to, by a wave: the last whose units begin there or before.
__device__ __forceinline__ uint32_t entry_at(const SharedEntry *entries, uint32_t n, uint64_t from) {
  uint32_t first = 0;
#pragma unroll 1
  for (uint32_t left = n; left > 1;) {
    const uint32_t step = (left + 63) / 64, i = threadIdx.x % 64 * step;
    const uint32_t before = (uint32_t)__popcll(__ballot(i < left && entries[first + i].unit0 <= from)) - 1;
    first += before * step;
    left = min(step, left - before * step);
  }
  return first;
}

// x / y, most often of 32 bits.
__device__ __forceinline__ uint32_t quotient(uint64_t x, uint64_t y) {
  return (x | y) >> 32 ? (uint32_t)(x / y) : (uint32_t)x / (uint32_t)y;
}

// The runs of workgroup wg of n_wg, one of each wave.  TILES: 16 query heads at a time, or (2) 32 of the entries that
// have more.  JOIN: a workgroup whose four runs are of one (entry, kv head, tile of heads) leaves one part (two answers
// to 16,000 tokens 17.2 us and 7.2 of join, otherwise 17.4 and 15.4; drafted positions 23.2 + 6.3 and 23.7 + 9.6).
template <int D, int KIND, int TILES, bool JOIN>
__device__ __forceinline__ void walk(const SharedArgs &a, const SharedEntry *entries, uint32_t wg, uint32_t n_wg,
                                     WalkLds<D, KIND, TILES, JOIN> &lds) {
  using L = Layout<D, KIND>;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, n = lane % 16, g = lane / 16;
  const uint32_t n_entries = a.rows + a.groups, n_runs = n_wg * kWaves, run = wg * kWaves + wave;
  const uint64_t all = entries[n_entries].unit0, share = (all + n_runs - 1) / n_runs;
  const uint64_t per = share < kLeast ? kLeast : share, per_wg = kWaves * per, from_wg = wg * per_wg;
  const uint64_t from = run * per;
  uint32_t index = 0;
  SharedEntry e;
  bool together = false;
  if (JOIN && from_wg + (kWaves - 1) * per < all) {
    index = entry_at(entries, n_entries, from_wg);
    e = scalar(entries[index]);
    const uint64_t at = from_wg - e.unit0, takes = min(per_wg, all - from_wg);
    const uint32_t units = (e.n + kUnit - 1) / kUnit;
    together = takes <= units && at - (uint64_t)quotient(at, units) * units + takes <= units;
  }
  if (from >= all) return;  // by no wave of those that are joined
  if (!together) {
    index = entry_at(entries, n_entries, from);
    e = scalar(entries[index]);
  }
  uint64_t at = from - e.unit0;
  uint64_t left = min(per, all - from);
  v4u *const lds_q = WalkLds<D, KIND, TILES, JOIN>::kMost ? lds.q[wave] : lds.q[0];
  bool first_segment = true;

  // What is left of an entry, MR times 16 heads at a time.
  auto entry = [&](auto tiles) {
    constexpr int MR = decltype(tiles)::value;
    using R = Residence<D, KIND, MR>;
    constexpr uint32_t kHeads = 16 * MR;
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
#pragma unroll
      for (int r = 0; r < MR; ++r) {
        const uint32_t h = h0 + 16 * r + n;
        const uint16_t *from_q = a.q + (e.q_row + h / a.group) * a.q_ld + (uint64_t)(kvh * a.group + h % a.group) * D;
#pragma unroll
        for (int k = 0; k < L::kMfmaK; ++k) {
          const uint32_t d = KIND == XFER_KV_BF16 ? k * 32 + g * 8 : (k / 2) * 64 + g * 16 + (k % 2) * 8;
          const v4u x = h < heads ? *reinterpret_cast<const v4u *>(from_q + d) : v4u{0, 0, 0, 0};
          if constexpr (R::kQInLds)
            lds_q[(r * L::kMfmaK + k) * 64 + lane] = x;  // which this lane reads again
          else
            q[r][k] = x;
        }
      }
      float scale2 = a.scale * 1.4426950408889634f;
      if (KIND == XFER_KV_E4M3 && a.cache.k_scale) scale2 *= a.cache.k_scale[kvh];
      const uint32_t *table = a.page_table + e.row * a.table_ld;
      v4f o[MR][L::kMfmaV];
      float mx[MR], sum[MR];
      attn_walk<D, KIND, MR, kParts, kUnit, false>(a.cache, kvh, table, vis, v0, v1, scale2, n, g, lane, q, lds_q, o, mx, sum);

      // made anew, or the places of all results would be ready, and held, while the tokens are walked through
      uint32_t en = n, eg = g;
      if (JOIN) asm volatile("" : "+v"(en), "+v"(eg));
      const bool whole = take == units;
      const uint32_t slot = 2 * run + (first_segment ? 0 : 1);
      if (unit == 0 && lane == 0) {
        SharedParts parts{whole ? kWhole : slot, 1 + (uint32_t)((units - take + per - 1) / per), 0};
        // The workgroups that leave one part, of those that begin here, and the runs before them; counted from this one on.
        const uint64_t begin = e.unit0 + (uint64_t)inner * units, span = begin + units - from_wg;
        const uint32_t first = begin > from_wg;
        uint32_t last = span < per_wg ? 0 : quotient(span, per_wg);
        if (begin + units == all && last * per_wg + (kWaves - 1) * per < span) ++last;
        if (JOIN && last > first) {
          parts.wgs = last - first;
          parts.lead = (wg + first) * kWaves - run;
          parts.n -= min(parts.n - parts.lead, parts.wgs * kWaves) - parts.wgs;
        }
        a.parts[e.part0 + inner] = parts;
      }
      auto put = [&](uint64_t to, uint32_t d, v4f v, float total, uint32_t t0, uint32_t t1) {
        if constexpr (KIND == XFER_KV_BF16) {
          if (isnan(v.x + v.y + v.z + v.w) && !isnan(total)) v = with_infinities<KIND>(a.cache, kvh, table, vis, t0, t1, v, d);
        }
        *reinterpret_cast<v4f *>(a.part_o + to * D + d) = v;
      };
#pragma unroll
      for (int r = 0; r < MR; ++r) {
        sum[r] += __shfl_xor(sum[r], 16);
        sum[r] += __shfl_xor(sum[r], 32);
        const uint32_t h = h0 + 16 * r + en;
        if (together) {
          auto &x = lds.exchange;
          __syncthreads();
          if (eg == 0) {
            x.m[wave][en] = mx[r];
            x.l[wave][en] = sum[r];
          }
          __syncthreads();
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) top = fmaxf(top, x.m[w][en]);
          const float f = mx[r] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[r] - top);
#pragma unroll
          for (int j = 0; j < L::kMfmaV; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) x.o[wave][en][dim_of<D, KIND>(j, 4 * eg + i)] = o[r][j][i] * f;
          __syncthreads();
#pragma unroll
          for (uint32_t i = threadIdx.x; i < 4 * D; i += kThreads) {
            const uint32_t hq = i / (D / 4), d = i % (D / 4) * 4;
            if (h0 + 16 * r + hq >= heads) continue;
            float best = -INFINITY, total = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) best = fmaxf(best, x.m[w][hq]);
            v4f v = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
              const float mw = x.m[w][hq];
              total += mw == -INFINITY ? x.l[w][hq] : x.l[w][hq] * __builtin_amdgcn_exp2f(mw - best);
              v += *reinterpret_cast<const v4f *>(&x.o[w][hq][d]);
            }
            const uint64_t to = (uint64_t)(2 * wg * kWaves) * slot_heads(TILES) + 16 * r + hq;
            const uint32_t t0 = v0 - (uint32_t)(wave * per) * kUnit;
            put(to, d, v, total, t0, min(t0 + (uint32_t)per_wg * kUnit, e.n));
            if (d == 0) {
              a.part_ml[2 * to] = best;
              a.part_ml[2 * to + 1] = total;
            }
          }
          continue;
        }
        if (h >= heads) continue;
        // a whole one's place is its row's and head's, in the half for shared or own tokens
        const uint64_t mine = (uint64_t)(e.q_row + h / a.group) * a.q_heads + kvh * a.group + h % a.group;
        const uint64_t to = whole ? a.whole0 + (index < a.rows ? 0 : (uint64_t)a.rows * a.q_heads) + mine
                                  : (uint64_t)slot * slot_heads(TILES) + 16 * r + en;
        if (eg == 0) {
          a.part_ml[2 * to] = mx[r];
          a.part_ml[2 * to + 1] = sum[r];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < L::kMfmaV; j += 4)
            put(to, dim_of<D, KIND>(j, 4 * eg + i), v4f{o[r][j][i], o[r][j + 1][i], o[r][j + 2][i], o[r][j + 3][i]}, sum[r], v0, v1);
      }
      left -= take;
      first_segment = false;
    }
  };
#pragma unroll 1
  while (left) {
    if (TILES == 2 && e.q_rows * a.group > 16)
      entry(std::integral_constant<int, TILES>{});
    else
      entry(std::integral_constant<int, 1>{});
    at = 0;
    if (left) {
      do e = scalar(entries[++index]);
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

typedef float v2f __attribute__((ext_vector_type(2)));
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
__device__ __forceinline__ void walk_many(const SharedArgs &a, const SharedEntry *entries, uint32_t wg, uint32_t n_wg,
                                          uint8_t *lds0, uint8_t *lds1) {
  using M = Many<D, KIND>;
  constexpr int kDims = D / 32;   // blocks of dims
  constexpr int kSteps = D / 16;  // of a score
  __shared__ __align__(8) uint16_t lds_gone[2][kWaves];  // a bit for each token of 16 that is not there
  const uint64_t all = entries[a.groups].unit0, share = (all + n_wg - 1) / n_wg;
  const uint64_t least = min(kManyLeast, (entries[a.groups].n + kManyUnit - 1) / kManyUnit);
  const uint64_t per = share < least ? least : share, from = wg * per;
  if (from >= all) return;
  uint64_t left = min(per, all - from);
  uint32_t index = entry_at(entries, a.groups, from);
  SharedEntry e = scalar(entries[index]);
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
          const uint8_t *zeros = reinterpret_cast<const uint8_t *>(&kZeros);
          const uint8_t *key = there ? kbase + off : zeros, *value = there ? vbase + off : zeros;
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
      // a scale of 0 or NaN is taken before tokens that are not there get -inf, and then any other will do
      const bool flat = !(scale2 > 0.0f);
      const float flat_by = scale2;
      if (flat) scale2 = 1.0f;
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
        if (flat) {
          s[0] *= flat_by;
          s[1] *= flat_by;
        }
        if ((out.x | out.y) != 0) {
#pragma unroll
          for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (out[blk] >> (8 * (i / 4) + 4 * hf + i % 4) & 1) s[blk][i] = -INFINITY;
        }
        // The largest product is the largest score; where it passes the running maximum by kRaise, that moves.
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fmaxf(s[0][i], s[1][i]));
        top *= scale2;
        if (__any(top > mx + kRaise)) {
          top = fmaxf(top, __shfl_xor(top, 32));
          const float raised = fmaxf(mx, top);
          const float f = mx == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx - raised);
          mx = raised;
          sum *= f;
#pragma unroll
          for (int d = 0; d < kDims; ++d) o[d] *= f;
        }
        // Scores above it.  The fused product is not rounded as the maximum was, so the largest is above or below it by that
        // rounding; where it would be much, scores are rounded first.
        const float base = mx == -INFINITY ? 0.0f : mx;
        float by = scale2;
        if (__any(__builtin_fabsf(base) > kRounded)) {
          s[0] *= scale2;
          s[1] *= scale2;
          by = 1.0f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[0][i] = fmaf(s[0][i], by, -base);
          s[1][i] = fmaf(s[1][i], by, -base);
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
        a.parts[e.part0 + inner] = SharedParts{whole ? kWhole : slot, 1 + (uint32_t)((units - take + per - 1) / per), 0};
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
      do e = scalar(entries[++index]);
      while (e.n == 0);  // there is one with tokens as long as units are left
    }
  }
}

// Neighbouring runs on one XCD: its L2 then serves the tokens that the heads of an entry have in common.
// LOCAL: the workgroups make the plan themselves.
template <int D, int KIND, int TILES, bool LOCAL>
__global__ __launch_bounds__(kThreads, (Residence<D, KIND, TILES>::kPerSimd)) void shared_walk_kernel(SharedArgs a) {
  __shared__ WalkLds<D, KIND, TILES, true> lds;
  __shared__ LocalPlan local;
  static_assert(sizeof(PlanLds<kThreads>) <= sizeof(lds), "it fits");
  if (LOCAL) plan_here(a, local, reinterpret_cast<PlanLds<kThreads> &>(lds), [](uint32_t) { return false; });
  const uint32_t wg = blockIdx.x % kXcds * (gridDim.x / kXcds) + blockIdx.x / kXcds;
  if (LOCAL)
    walk<D, KIND, TILES, true>(a, local.list, wg, gridDim.x, lds);
  else
    walk<D, KIND, TILES, true>(a, a.entries, wg, gridDim.x, lds);
}

// Both lists at once, so that one's loads and the other's products share the compute units: of the workgroups
// that are resident, as many take the list of many heads as the plan found, spread evenly over the others.
template <int D, int KIND, int PARTS, bool LOCAL>
__global__ __launch_bounds__(kThreads, (Many<D, KIND>::kPerSimd)) void shared_both_kernel(SharedArgs a) {
  constexpr uint32_t kTile = 2 * Many<D, KIND>::kTileBytes;
  __shared__ __align__(16) uint8_t lds0[kTile < sizeof(WalkLds<D, KIND, 2, (D > 64)>) ? sizeof(WalkLds<D, KIND, 2, (D > 64)>) : kTile];
  __shared__ __align__(16) uint8_t lds1[kTile];
  __shared__ LocalPlan local;
  static_assert(sizeof(PlanLds<kThreads>) <= sizeof(lds0), "it fits");
  const uint32_t xcd = blockIdx.x % kXcds, place = blockIdx.x / kXcds, places = gridDim.x / kXcds;
  uint32_t many, before;  // of an XCD's places, and of those before this one
  auto choose = [&](uint32_t n) {
    many = n;
    before = place * many / places;
    return (place + 1) * many / places > before;
  };
  const bool takes_many = LOCAL ? plan_here(a, local, reinterpret_cast<PlanLds<kThreads> &>(lds0), choose) : choose(*a.many_places);
  if (takes_many)
    walk_many<D, KIND, PARTS>(a, LOCAL ? local.list : a.many, xcd * many + before, kXcds * many, lds0, lds1);
  else  // in this kernel heads of 64 leave each run's part: joined, the walk of many would spill more, and three system prompts
        // take 42.0 + 8.3 us for 37.8 + 7.9
    walk<D, KIND, 2, (D > 64)>(a, LOCAL ? local.list : a.entries, xcd * (places - many) + place - before, kXcds * (places - many),
                     *reinterpret_cast<WalkLds<D, KIND, 2, (D > 64)> *>(lds0));
}

// ------------------------------------------------------------------- join

// kWaves (or one) for each (row, query head): its parts of the shared tokens, then of its own, each scaled to
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
  // The row's own entry and its group's in either list, then what each came to: loads that wait for no more than they must.
  const SharedEntry own = a.entries[row];
  const bool shares = own.group != kNoGroup;
  const uint32_t of_group = shares ? own.group : 0;
  const SharedEntry few = a.entries[a.rows + of_group], many = a.many ? a.many[of_group] : few;
  const bool is_many = shares && few.n == 0;
  const SharedEntry &whose = is_many ? many : few;
  auto tile_for = [&](const SharedEntry &e, bool m) { return m ? kManyHeads : tile_of(e.q_rows * a.group); };
  auto index = [&](const SharedEntry &e) { return (row - e.q_row) * a.group + h; };  // this head's among the entry's
  auto part_of = [&](const SharedEntry &e, uint32_t tile) {
    return e.part0 + kvh * ((e.q_rows * a.group + tile - 1) / tile) + index(e) / tile;
  };
  const uint32_t own_tile = tile_for(own, false), pre_tile = tile_for(whose, is_many);
  const uint32_t own_part = own.n ? part_of(own, own_tile) : 0, pre_part = shares ? part_of(whose, pre_tile) : own_part;
  const SharedParts own_parts = a.parts[own_part], pre_parts = a.parts[pre_part];
  struct Source {
    uint32_t n, lead, wgs;      // parts; those of workgroups as a whole, after the first `lead`
    uint64_t at0, at1, stride;  // places: run 0's; run p's at1 + p * stride
  };
  auto source = [&](const SharedParts &p, bool prefix, bool m, uint32_t in_tile) {
    const uint32_t slot = m ? kManyHeads : a.slot_heads;
    const uint64_t cut0 = (m ? a.many_place0 : 0) + in_tile;
    const uint64_t whole = a.whole0 + (prefix ? (uint64_t)a.rows * a.q_heads : 0) + (uint64_t)row * a.q_heads + head;
    // Run p > 0 began with this.
    return Source{p.n, p.lead, p.wgs, p.slot == kWhole ? whole : cut0 + (uint64_t)p.slot * slot, cut0 + (uint64_t)(p.slot / 2 * 2) * slot, 2 * slot};
  };
  Source pre{}, mine{};
  if (shares) pre = source(pre_parts, true, is_many, index(whose) % pre_tile);
  if (own.n) mine = source(own_parts, false, false, index(own) % own_tile);
  const uint32_t n = pre.n + mine.n;
  auto place = [&](uint32_t p) -> uint64_t {
    const Source &s = p < pre.n ? pre : mine;
    uint32_t k = p < pre.n ? p : p - pre.n;
    k += (kWaves - 1) * min(k - min(k, s.lead), s.wgs);  // a workgroup's one part is its first run's
    return k ? s.at1 + k * s.stride : s.at0;
  };

  // Lane l of wave w has part p0 + l * WAVES + w of every 64 * WAVES.  Its maximum and sum of weights; the first's are kept.
  auto max_sum = [&](uint32_t p0) {
    const uint32_t p = p0 + lane * WAVES + wave;
    return p < n ? *reinterpret_cast<const v2f *>(a.part_ml + 2 * place(p)) : v2f{-INFINITY, 0};
  };
  const v2f first = max_sum(0);
  float top = first.x;
#pragma unroll 1
  for (uint32_t p0 = 64 * WAVES; p0 < n; p0 += 64 * WAVES) top = fmaxf(top, max_sum(p0).x);
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
      const v2f ml = p0 ? max_sum(p0) : first;
      const float m = ml.x, l = ml.y;
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

template <int D, int KIND, bool LOCAL>
hipError_t launch_walk(const SharedArgs &a, uint32_t workgroups, hipStream_t stream) {
  const dim3 grid(workgroups), block(kThreads);
  if (!a.many)
    return a.slot_heads == 16 ? launch(shared_walk_kernel<D, KIND, 1, LOCAL>, grid, block, 0, stream, a)
                              : launch(shared_walk_kernel<D, KIND, 2, LOCAL>, grid, block, 0, stream, a);
  return a.out_mode == XFER_OUT_F32 ? launch(shared_both_kernel<D, KIND, 3, LOCAL>, grid, block, 0, stream, a)
                                    : launch(shared_both_kernel<D, KIND, 2, LOCAL>, grid, block, 0, stream, a);
}
template <int D, bool LOCAL>
hipError_t launch_kind(const SharedArgs &a, int kind, uint32_t workgroups, hipStream_t stream) {
  return kind == XFER_KV_BF16 ? launch_walk<D, XFER_KV_BF16, LOCAL>(a, workgroups, stream)
                              : launch_walk<D, XFER_KV_E4M3, LOCAL>(a, workgroups, stream);
}
template <int D>
hipError_t launch_dim(const SharedArgs &a, int kind, uint32_t workgroups, hipStream_t stream) {
  const bool local = a.rows <= kThreads && a.rows + a.groups < kThreads;
  hipError_t e = local ? hipSuccess : launch(shared_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
  if (e != hipSuccess) return e;
  e = local ? launch_kind<D, true>(a, kind, workgroups, stream) : launch_kind<D, false>(a, kind, workgroups, stream);
  if (e != hipSuccess) return e;
  const uint32_t items = a.rows * a.q_heads;
  if (items >= kJoinHeads)
    return launch(shared_join_kernel<D, 1>, dim3((items + kWaves - 1) / kWaves), dim3(kThreads), 0, stream, a);
  return launch(shared_join_kernel<D, kWaves>, dim3(items), dim3(kThreads), 0, stream, a);
}

struct Shape {
  uint32_t slot_heads, workgroups;
  bool many;
  uint64_t parts, many_part0;             // (entry, kv head, tile)s at most, and where those of many heads begin
  uint64_t places, many_place0, whole0;   // query heads of all parts, and where those of many heads and whole ones begin
};
template <int D, int KIND>
uint32_t per_simd(int tiles) {
  return tiles == 1 ? Residence<D, KIND, 1>::kPerSimd : Residence<D, KIND, 2>::kPerSimd;
}
template <int KIND>
uint32_t per_simd(uint32_t head_dim, int tiles) {
  return head_dim == 64 ? per_simd<64, KIND>(tiles) : head_dim == 128 ? per_simd<128, KIND>(tiles) : per_simd<256, KIND>(tiles);
}
Shape shape_of(uint32_t rows, uint32_t groups, uint32_t kv_heads, uint32_t group, uint32_t head_dim, int kind) {
  Shape s{};
  const int tiles = (groups ? (uint64_t)rows * group : group) > 16 ? 2 : 1;  // that an entry of few heads may have
  s.many = groups && (uint64_t)rows * group > kFewHeads;                     // some group may be that large
  s.slot_heads = slot_heads(tiles);
  s.workgroups = kComputeUnits * (s.many ? (head_dim == 256 ? 1 : head_dim == 128 ? 2 : 3)
                                         : kind == XFER_KV_BF16 ? per_simd<XFER_KV_BF16>(head_dim, tiles)
                                                                : per_simd<XFER_KV_E4M3>(head_dim, tiles));
  const uint64_t row_tiles = (group + 15) / 16;
  s.many_part0 = kv_heads * (rows * row_tiles + (uint64_t)rows * group / 16 + groups);
  s.parts = s.many_part0;
  s.many_place0 = 2ull * s.workgroups * kWaves * s.slot_heads;
  s.whole0 = s.many_place0;
  if (s.many) {
    s.parts += kv_heads * ((uint64_t)rows * group / kManyHeads + groups);
    s.whole0 += 2ull * s.workgroups * kManyHeads;
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

// Layout: the entries, the parts of each (entry, kv head, tile), (max, sum) of each part, the weighted sums.  For every run
// of a full grid, whatever max_len is: a caller's workspace then serves all lengths.
uint64_t shared_workspace_bytes(uint32_t rows, uint32_t groups, uint32_t kv_heads, uint32_t group, uint32_t head_dim,
                                int kind) {
  const Shape s = shape_of(rows, groups, kv_heads, group, head_dim, kind);
  return 16 + up16(((uint64_t)rows + 2ull * groups + 2) * sizeof(SharedEntry)) + up16(s.parts * sizeof(SharedParts)) + up16(s.places * 8) +
         s.places * head_dim * 4;
}

hipError_t launch_shared(const SharedArgs &in, int kind, void *workspace, hipStream_t stream) {
  SharedArgs a = in;
  const Shape s = shape_of(a.rows, a.groups, a.cache.kv_heads, a.group, a.cache.head_dim, kind);
  a.slot_heads = s.slot_heads;
  a.whole0 = s.whole0;
  uint8_t *at = static_cast<uint8_t *>(workspace);
  a.many_places = reinterpret_cast<uint32_t *>(at);
  a.places_of_xcd = s.workgroups / kXcds;
  // What a unit of either list costs, one to the other: bytes of keys and values, or products with keys and each part of the
  // weights.  64 answers 44.8 us, three system prompts 39.3, 300 rows in 20 groups 64; with the second 0.6 times that 53.4, 42
  // and 85, 1.6 times 51.0, 44.5 and 52: no one ratio serves all.
  a.unit_cost = kUnit * 2 * a.cache.head_dim * (kind == XFER_KV_BF16 ? 2 : 1) / 64;
  a.many_unit_cost = a.cache.head_dim * (a.out_mode == XFER_OUT_F32 ? 4 : 3) * 2;

  a.entries = reinterpret_cast<SharedEntry *>(at += 16);
  a.parts = reinterpret_cast<SharedParts *>(at += up16(((uint64_t)a.rows + 2ull * a.groups + 2) * sizeof(SharedEntry)));
  if (s.many) a.many = a.entries + a.rows + a.groups + 1;
  a.many_part0 = (uint32_t)s.many_part0;
  a.many_place0 = s.many_place0;
  a.part_ml = reinterpret_cast<float *>(at += up16(s.parts * sizeof(SharedParts)));
  a.part_o = reinterpret_cast<float *>(at + up16(s.places * 8));
  if (a.cache.head_dim == 64) return launch_dim<64>(a, kind, s.workgroups, stream);
  if (a.cache.head_dim == 128) return launch_dim<128>(a, kind, s.workgroups, stream);
  return launch_dim<256>(a, kind, s.workgroups, stream);
}

}  // namespace xfer
