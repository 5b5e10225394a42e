// Attention of one new token of every request over a paged cache of keys and
// values, split over the cache's length and joined.
//
// Every visible key and value is read once and little is done with it: 4 *
// group operations for each element, so HBM bandwidth bounds the call, and
// the layout serves the loads:
//   - the work is one line of units, 128 visible tokens of a (row, kv head)
//     each, row after row; every workgroup adds up the rows' lengths for itself
//     and takes an equal run of it.  So rows of any mixture of lengths keep all
//     compute units busy for the same time, and all workgroups that start are
//     resident at once.  A (row, kv head) that falls to several workgroups leaves
//     (max, sum, weighted sum) of each part in the workspace, at most two for a
//     workgroup, and a second launch joins them;
//   - a workgroup takes all query heads of a kv head, so a key is read from
//     memory once for all of them.  Its waves take tiles of 32 tokens in turn,
//     each with a running maximum and sum of its own, and meet once for each
//     (row, kv head), in LDS.  Heads beyond 16 take more registers of these
//     waves (up to 32 heads; the next 32 are a kv head of their own);
//   - scores are products K Q^T on matrix cores (16x16x32): K's operand is 16
//     bytes of a token's row for each lane, straight from global memory, and
//     a lane ends with four tokens' scores of one query head in each of two
//     such tiles.  With the value rows of exactly these eight tokens loaded
//     by the same group of 16 lanes, the weights are V^T P^T's operand as
//     they stand: nothing crosses lanes, and neither K nor V goes through
//     LDS.  A lane's eight value rows are turned into the operand's order
//     (eight tokens of one dim) by one byte permute for each pair;
//   - which dim a register stands for is free as long as both operands agree,
//     so each load takes the widest contiguous run: a lane group's 16 lanes
//     read whole value rows of head_dim elements.
// The visible tokens of a window with first tokens are numbered through, so
// tiles of a window are as full as any others; a token's place is looked up
// by one lane and handed to the lanes that read it.
//
// Two rows of 131071 tokens (8 kv heads of 128, BF16, 1074 MB) take 164 us, 6.5
// TB/s, and 4.6 us to be joined; 48 rows of up to 8192 tokens 94 us, 6.0 TB/s.
// Where a workgroup has a few units only, the rounds of one after the other
// bound it: 96 windows of 1028 tokens (64, E4M3) 23.2 us, 3.7 TB/s, the last
// of nine rounds for four tokens.
//
// The running maximum is raised only when a score passes it by more than 2^8
// (weights stay below 256, far from binary32's limits), which leaves out most
// of the rescaling and of the exchanges between lanes.
#include "attn_tile.h"

namespace xfer {
namespace {

constexpr int kWaves = 4;                        // that share the tokens of a run
constexpr int kThreads = 64 * kWaves;
constexpr uint32_t kStep = kTile * kWaves;       // tokens of a unit
constexpr uint32_t kJoinUnits = 3;               // that the join is worth
constexpr int kManyWaves = 8;                    // that share the tokens of a row with a compute unit to itself
constexpr uint32_t kAloneBytes = 2048;           // of such a row's units, one row of each, at most
// Keys and values are read past the caches where a call may read more than
// they hold (two rows of 131071 tokens 169 us, 188 through them); fewer may be
// there still, from the call before or from rows that share pages (128 (row, kv
// head)s of 1000 tokens, 65 MB, called in turn: 17.9 us, 19 past them).
constexpr uint64_t kCachedBytes = 96ull << 20;
// Bytes of a key that is read beside the next heads', at most.
constexpr int side_bytes(int heads, int tiles) { return heads == 4 && tiles == 1 ? 256 : 128; }
constexpr uint32_t kComputeUnits = 256;
constexpr uint32_t kMaxWorkgroups = 4 * kComputeUnits;
constexpr uint32_t kXcds = 8;

// The tokens that a row sees.
__device__ __forceinline__ Visible visible_of(const AttnArgs &a, uint32_t row) {
  const uint32_t n = min(a.lens[row], a.max_len);
  const uint32_t before = n - min(n, a.window);  // tokens in front of the window
  Visible v;
  v.first = min(a.sinks, before);
  v.gap = before - v.first;
  v.n = n - v.gap;
  return v;
}

// What a (row, kv head) that fell to several workgroups leaves: its first
// part's slot (kWhole: one workgroup did it all), and how many parts.
struct Parts {
  uint32_t slot, n;
};
constexpr uint32_t kWhole = 0xFFFFFFFFu;

template <uint32_t UNIT>
__device__ __forceinline__ uint32_t units_of(const Visible &v) {
  return v.n ? (v.n + UNIT - 1) / UNIT : 1;
}

// A workgroup's run of units: where it starts, and how long it is.
struct Run {
  uint64_t per, length;  // of any workgroup, and of this one (0: nothing to do)
  uint32_t row;
  uint64_t at;           // the first unit within the row
};

// Adds up the rows' units (a row has units_of() for each of `inner_n` heads)
// and cuts them into equal runs; by all threads.
template <uint32_t UNIT>
__device__ __forceinline__ Run run_of(const AttnArgs &a, uint32_t inner_n, uint32_t wg, uint32_t n_wg) {
  __shared__ uint64_t totals[kWaves];
  __shared__ uint64_t start[2];
  const uint32_t tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const uint32_t each = (a.rows + kThreads - 1) / kThreads;
  const uint32_t r0 = min(tid * each, a.rows), r1 = min(r0 + each, a.rows);
  uint64_t mine = 0;
  for (uint32_t r = r0; r < r1; ++r) mine += (uint64_t)units_of<UNIT>(visible_of(a, r)) * inner_n;
  uint64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint64_t x = __shfl_up(incl, d);
    if ((int)lane >= d) incl += x;
  }
  if (lane == 63) totals[wave] = incl;
  __syncthreads();
  uint64_t all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < (int)wave) incl += totals[w];
    all += totals[w];
  }
  Run run;
  run.per = (all + n_wg - 1) / n_wg;
  const uint64_t from = wg * run.per;
  // No guarded subtraction here: hipcc 7.2 compiles
  //   from < all ? min(per, all - from) : 0
  // to min(per, all - from) without the guard (also alone, in a kernel of its
  // own), since it may assume that what min() is called with is defined.
  run.length = min(run.per, all - min(from, all));
  if (incl - mine <= from && from < incl) {
    uint64_t before = incl - mine;
    uint32_t r = r0;
    for (; r + 1 < r1; ++r) {
      const uint64_t u = (uint64_t)units_of<UNIT>(visible_of(a, r)) * inner_n;
      if (from < before + u) break;
      before += u;
    }
    start[0] = r;
    start[1] = from - before;
  }
  __syncthreads();
  run.row = __builtin_amdgcn_readfirstlane((uint32_t)start[0]);
  run.at = start[1];
  return run;
}

// HEADS kv heads side by side, WAVES waves for each: kWaves together, or
// kManyWaves without runs.
template <int D, int KIND, int TILES, int PARTS, int WAVES, bool STREAM, int HEADS>
__global__ __launch_bounds__(64 * WAVES * HEADS, (Residence<D, KIND, TILES>::kPerSimd)) void attn_kernel(
    AttnArgs a, uint32_t m_groups, uint32_t deal) {
  using L = Layout<D, KIND>;
  using R = Residence<D, KIND, TILES>;
  constexpr int MR = TILES;
  constexpr bool kRuns = WAVES * HEADS == kWaves;
  constexpr uint32_t kRound = kTile * WAVES;         // tokens of a round
  constexpr uint32_t kUnit = kRuns ? kRound : kStep;  // and of a unit
  constexpr int kPad = 4;  // floats between rows of the exchange, so that 16 rows' stores fall on all banks
  __shared__ float lds_heads_o[HEADS][WAVES][16][D + kPad];
  __shared__ float lds_heads_m[HEADS][MR][WAVES][16], lds_heads_l[HEADS][MR][WAVES][16];
  const uint32_t side = HEADS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * WAVES));
  auto &lds_o = lds_heads_o[side];
  auto &lds_all_m = lds_heads_m[side];
  auto &lds_all_l = lds_heads_l[side];

  const uint32_t inner_n = a.cache.kv_heads / HEADS * m_groups;
  const uint32_t xcd = blockIdx.x % kXcds, rest = blockIdx.x / kXcds;
  const bool runs = kRuns && a.parts;
  uint32_t wg = 0, item = 0;
  Run run;
  if (runs) {
    // Neighbouring runs on one XCD: its L2 then serves the lines that two
    // heads share.
    wg = xcd * (gridDim.x / kXcds) + rest;
    if constexpr (kRuns) run = run_of<kUnit>(a, inner_n, wg, gridDim.x);
    if (run.length == 0) return;
  } else {
    // A workgroup for each (row, kv head) and group of its query heads, `deal`
    // of them to each XCD in turn.
    item = (rest / deal * kXcds + xcd) * deal + rest % deal;
    if (item >= a.rows * inner_n) return;
    run.row = item / inner_n;
  }

  const uint32_t tid = threadIdx.x % (64 * WAVES), wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64,
                 n = lane % 16, g = lane / 16;
  // The queries, in the lanes' order, where the exchange lies later.
  v4u *const lds_q = reinterpret_cast<v4u *>(&lds_o[0][0][0]);
  static_assert(!R::kQInLds || MR * L::kMfmaK * 64 * 16 <= (int)sizeof(lds_o), "they fit");
  uint32_t row = run.row;
  Visible vis = visible_of(a, row);
  uint32_t units = units_of<kUnit>(vis);
  uint32_t inner = item % inner_n, unit = 0;
  uint64_t left = units;
  if (runs) {
    inner = __builtin_amdgcn_readfirstlane((uint32_t)(run.at / units));
    unit = __builtin_amdgcn_readfirstlane((uint32_t)(run.at % units));
    left = run.length;
  }
  bool first_segment = true;

#pragma unroll 1
  while (left) {
  const uint32_t take = (uint32_t)min(left, (uint64_t)(units - unit));
  const uint32_t kvh = inner / m_groups * HEADS + side, h0 = inner % m_groups * (16 * MR);  // first query head within the group
  const uint32_t v0 = unit * kUnit, v1 = min((unit + take) * kUnit, vis.n);

  // Q: query head h0 + 16 * r + n, the dims that this lane's K loads hold.
  v4u q[R::kQInLds ? 1 : MR][L::kMfmaK];
  auto load_q = [&](int r, int k) {
    const uint32_t h = h0 + 16 * r + n;
    const uint32_t d = KIND == XFER_KV_BF16 ? k * 32 + g * 8 : (k / 2) * 64 + g * 16 + (k % 2) * 8;
    return h < a.group ? *reinterpret_cast<const v4u *>(a.q + row * a.q_ld + (uint64_t)(kvh * a.group + h) * D + d)
                       : v4u{0, 0, 0, 0};
  };
  if constexpr (R::kQInLds) {
    for (int k = wave; k < MR * L::kMfmaK; k += WAVES) lds_q[k * 64 + lane] = load_q(k / L::kMfmaK, k % L::kMfmaK);
    __syncthreads();
  } else {
#pragma unroll
    for (int r = 0; r < MR; ++r)
#pragma unroll
      for (int k = 0; k < L::kMfmaK; ++k) q[r][k] = load_q(r, k);
  }
  float scale2 = a.scale * 1.4426950408889634f;
  if (KIND == XFER_KV_E4M3 && a.cache.k_scale) scale2 *= a.cache.k_scale[kvh];

  const uint32_t *table = a.page_table + row * a.table_ld;
  v4f o[MR][L::kMfmaV];
  float mx[MR], sum[MR];
  attn_walk<D, KIND, MR, PARTS, kRound, STREAM>(a.cache, kvh, table, vis, v0 + wave * kTile, v1, scale2, n, g, lane, q, lds_q,
                                                o, mx, sum);

  // The waves' results, joined in LDS.
  const bool whole = take == units;
  const uint32_t slot = 2 * wg + (first_segment ? 0 : 1);
  if (unit == 0 && tid == 0 && runs)
    reinterpret_cast<Parts *>(a.parts)[((uint64_t)row * a.cache.kv_heads + kvh) * m_groups + inner % m_groups] =
        whole ? Parts{kWhole, 1} : Parts{slot, 1 + (uint32_t)((units - take + run.per - 1) / run.per)};
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
  const float v_scale = KIND == XFER_KV_E4M3 && a.cache.v_scale ? a.cache.v_scale[kvh] : 1.0f;
#pragma unroll
  for (int r = 0; r < MR; ++r) {
    auto &lds_m = lds_all_m[r];
    auto &lds_l = lds_all_l[r];
    if (r) __syncthreads();
    {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = fmaxf(top, lds_m[w][n]);
      const float f = mx[r] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[r] - top);
#pragma unroll
      for (int j = 0; j < L::kMfmaV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) lds_o[wave][n][dim_of<D, KIND>(j, 4 * g + i)] = o[r][j][i] * f;
    }
    __syncthreads();
#pragma unroll
    for (uint32_t at = tid; at < 4 * D; at += 64 * WAVES) {
      const uint32_t hq = at / (D / 4), d = at % (D / 4) * 4;
      const uint32_t h = h0 + 16 * r + hq;
      if (h >= a.group) continue;
      float top = -INFINITY, total = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = fmaxf(top, lds_m[w][hq]);
      v4f v = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float mw = lds_m[w][hq];
        total += mw == -INFINITY ? lds_l[w][hq] : lds_l[w][hq] * __builtin_amdgcn_exp2f(mw - top);
        v += *reinterpret_cast<const v4f *>(&lds_o[w][hq][d]);
      }
      if constexpr (KIND == XFER_KV_BF16) {
        if (isnan(v.x + v.y + v.z + v.w)) v = with_infinities<KIND>(a.cache, kvh, table, vis, v0, v1, v, d);
      }
      if (whole) {
        v = total == 0.0f ? v4f{0, 0, 0, 0} : v * (v_scale / total);
        const uint64_t at_out = row * a.out_ld + (uint64_t)(kvh * a.group + h) * D + d;
        if (a.out_mode == XFER_OUT_F32)
          *reinterpret_cast<v4f *>(static_cast<float *>(a.out) + at_out) = v;
        else
          *reinterpret_cast<v2u *>(static_cast<uint16_t *>(a.out) + at_out) = v2u{bf16x2(v.x, v.y), bf16x2(v.z, v.w)};
      } else {
        const uint64_t part = ((uint64_t)slot * HEADS + side) * min(a.group, (uint32_t)TILES * 16) + 16 * r + hq;
        *reinterpret_cast<v4f *>(a.part_o + part * D + d) = v;
        if (d == 0) {
          a.part_ml[2 * part] = top;
          a.part_ml[2 * part + 1] = total;
        }
      }
    }
  }

  // The next (row, kv head).
  left -= take;
  first_segment = false;
  unit = 0;
  if (++inner == inner_n) {
    inner = 0;
    if (++row == a.rows) break;
    vis = visible_of(a, row);
    units = units_of<kUnit>(vis);
  }
  if (left) __syncthreads();  // LDS is written again
  }
}

// One workgroup for each (row, query head): the weighted sums of its parts, each
// scaled to the largest maximum, in the parts' order.
template <int D>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnArgs a, uint32_t m_tile, uint32_t m_groups,
                                                               uint32_t heads) {
  constexpr uint32_t kLanes = D / 4, kAtOnce = kThreads / kLanes;
  constexpr int kEach = kMaxWorkgroups / kThreads;  // parts of a thread
  __shared__ float lds_w[kMaxWorkgroups];
  __shared__ float lds_red[2][kWaves];
  __shared__ v4f lds_o[kAtOnce][kLanes];
  const uint32_t row = blockIdx.x / a.q_heads, head = blockIdx.x % a.q_heads;
  const uint32_t kvh = head / a.group, h = head % a.group, tid = threadIdx.x;
  const Parts parts = reinterpret_cast<const Parts *>(a.parts)[((uint64_t)row * a.cache.kv_heads + kvh) * m_groups + h / m_tile];
  if (parts.slot == kWhole) return;
  // Part p > 0 is the first thing that the workgroup p further on did.
  auto place = [&](uint32_t p) {
    return ((uint64_t)(p ? (parts.slot / 2 + p) * 2 : parts.slot) * heads + kvh % heads) * min(a.group, m_tile) + h % m_tile;
  };

  float m[kEach], l[kEach], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t p = i * kThreads + tid;
    m[i] = -INFINITY;
    l[i] = 0;
    if (p < parts.n) {
      m[i] = a.part_ml[2 * place(p)];
      l[i] = a.part_ml[2 * place(p) + 1];
    }
    top = fmaxf(top, m[i]);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
  if (tid % 64 == 0) lds_red[0][tid / 64] = top;
  __syncthreads();
  top = fmaxf(fmaxf(lds_red[0][0], lds_red[0][1]), fmaxf(lds_red[0][2], lds_red[0][3]));
  float total = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t p = i * kThreads + tid;
    const float f = m[i] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[i] - top);
    // not 0: a part's infinity stays one, however small its weights
    if (p < parts.n) lds_w[p] = f == 0.0f ? __uint_as_float(1) : f;
    total += m[i] == -INFINITY ? l[i] : l[i] * f;
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d);
  if (tid % 64 == 0) lds_red[1][tid / 64] = total;
  __syncthreads();
  const uint32_t d4 = tid % kLanes, p0 = tid / kLanes;
  v4f r = {0, 0, 0, 0};
#pragma unroll 4
  for (uint32_t p = p0; p < parts.n; p += kAtOnce)
    r += lds_w[p] * *reinterpret_cast<const v4f *>(a.part_o + place(p) * D + 4 * d4);
  lds_o[p0][d4] = r;
  __syncthreads();
  if (p0 != 0) return;
#pragma unroll
  for (uint32_t s = 1; s < kAtOnce; ++s) r += lds_o[s][d4];
  total = (lds_red[1][0] + lds_red[1][1]) + (lds_red[1][2] + lds_red[1][3]);
  const float v_scale = a.cache.v_scale ? a.cache.v_scale[kvh] : 1.0f;
  r = total == 0.0f ? v4f{0, 0, 0, 0} : r * (v_scale / total);
  const uint64_t at = row * a.out_ld + (uint64_t)head * D + 4 * d4;
  if (a.out_mode == XFER_OUT_F32)
    *reinterpret_cast<v4f *>(static_cast<float *>(a.out) + at) = r;
  else
    *reinterpret_cast<v2u *>(static_cast<uint16_t *>(a.out) + at) = v2u{bf16x2(r.x, r.y), bf16x2(r.z, r.w)};
}

// Workgroups of four waves that the runs are cut for.
template <int D, int KIND>
uint32_t resident(uint32_t tiles) {
  return kComputeUnits * (tiles == 1 ? Residence<D, KIND, 1>::kPerSimd : Residence<D, KIND, 2>::kPerSimd);
}
template <int KIND>
uint32_t resident(uint32_t head_dim, uint32_t tiles) {
  return head_dim == 64    ? resident<64, KIND>(tiles)
         : head_dim == 128 ? resident<128, KIND>(tiles)
                           : resident<256, KIND>(tiles);
}

template <int D, int KIND, int TILES, int PARTS>
hipError_t launch_waves(const AttnArgs &a, const AttnShape &s, hipStream_t stream) {
  const dim3 grid((uint32_t)s.workgroups);
  // a line holds the rows of two heads where they are shorter than it
  constexpr bool kLines = D * Layout<D, KIND>::kBytes >= 128;
  if constexpr (Residence<D, KIND, TILES>::kPerSimd > 1) {
    if (s.waves == kManyWaves)
      return launch(attn_kernel<D, KIND, TILES, PARTS, kManyWaves, false, 1>, grid, dim3(64 * kManyWaves), 0, stream, a,
                    s.m_groups, s.deal);
    if constexpr (D * Layout<D, KIND>::kBytes <= side_bytes(4, TILES)) {
      if (s.heads == 4)
        return launch(attn_kernel<D, KIND, TILES, PARTS, 1, kLines, 4>, grid, dim3(kThreads), 0, stream, a, s.m_groups,
                      s.deal);
    }
    if constexpr (D * Layout<D, KIND>::kBytes <= side_bytes(2, TILES)) {
      if (s.heads == 2)
        return launch(attn_kernel<D, KIND, TILES, PARTS, 2, kLines, 2>, grid, dim3(kThreads), 0, stream, a, s.m_groups,
                      s.deal);
    }
  }
  if constexpr (kLines) {
    if (s.stream)
      return launch(attn_kernel<D, KIND, TILES, PARTS, kWaves, true, 1>, grid, dim3(kThreads), 0, stream, a, s.m_groups,
                    s.deal);
  }
  return launch(attn_kernel<D, KIND, TILES, PARTS, kWaves, false, 1>, grid, dim3(kThreads), 0, stream, a, s.m_groups,
                s.deal);
}

template <int D, int KIND, int TILES>
hipError_t launch_parts(const AttnArgs &a, const AttnShape &s, hipStream_t stream) {
  return a.out_mode == XFER_OUT_F32 ? launch_waves<D, KIND, TILES, 3>(a, s, stream)
                                    : launch_waves<D, KIND, TILES, 2>(a, s, stream);
}

template <int D, int KIND>
hipError_t launch_tiles(const AttnArgs &a, const AttnShape &s, hipStream_t stream) {
  return s.m_tiles == 1 ? launch_parts<D, KIND, 1>(a, s, stream) : launch_parts<D, KIND, 2>(a, s, stream);
}

template <int D>
hipError_t launch_dim(const AttnArgs &a, int kind, const AttnShape &s, hipStream_t stream) {
  const hipError_t e =
      kind == XFER_KV_BF16 ? launch_tiles<D, XFER_KV_BF16>(a, s, stream) : launch_tiles<D, XFER_KV_E4M3>(a, s, stream);
  if (e != hipSuccess || !s.joined) return e;
  return launch(attn_join_kernel<D>, dim3(a.rows * a.q_heads), dim3(kThreads), 0, stream, a, 16 * s.m_tiles,
                s.m_groups, s.heads);
}

uint64_t up16(uint64_t x) { return (x + 15) / 16 * 16; }
// Query heads of all the workgroups' parts: two parts for each.
uint64_t parts_of(const AttnShape &s) { return 2ull * s.workgroups * s.heads * s.part_heads; }

}  // namespace

AttnShape attn_shape(uint32_t rows, uint32_t kv_heads, uint32_t group, uint32_t head_dim, int kind,
                     uint64_t vis_max, uint64_t head_stride) {
  AttnShape s{};
  if (rows == 0) return s;
  s.m_tiles = group <= 16 ? 1 : 2;
  const uint32_t tile = 16 * s.m_tiles;
  s.m_groups = group / tile + (group % tile != 0);
  s.part_heads = group < tile ? group : tile;
  const uint64_t inner = (uint64_t)kv_heads * s.m_groups, steps = (vis_max + kStep - 1) / kStep;
  const uint64_t most =
      kind == XFER_KV_BF16 ? resident<XFER_KV_BF16>(head_dim, s.m_tiles) : resident<XFER_KV_E4M3>(head_dim, s.m_tiles);
  const uint32_t row_bytes = head_dim * (kind == XFER_KV_BF16 ? 2 : 1);
  s.stream = vis_max > kCachedBytes / (2 * row_bytes) / ((uint64_t)rows * kv_heads);
  // Where a token's heads lie one after the other, short rows are read four
  // heads (or two) at a time, a wave or two for each: scattered by the tokens'
  // distance they cost more than their bytes (256,000 tokens of 8 heads of 128
  // bytes: 94 us, 121 one head at a time; of 256 bytes 92, 101).  Not where a wave
  // has enough to do with 32 query heads (256 bytes: 68 us, 61), or with two
  // heads of 256 bytes (36 us, 33).
  const uint32_t heads = kv_heads % 4 == 0 ? 4 : 2;
  const bool beside = s.stream && most > kComputeUnits && kv_heads % 2 == 0 && head_stride == row_bytes &&
                      row_bytes <= (uint32_t)side_bytes(heads, s.m_tiles);
  // Whole (row, kv head)s where none is long, and cutting them up would spare a
  // workgroup no more units than the second launch costs; else equal runs.  What
  // is long depends on what the runs are worth: 768 (row, kv head)s of up to 2800
  // tokens, 64 bytes, take 31 us whole and 45 in runs (128 bytes: 55, 56; 256
  // bytes: 90, 74), with heads side by side 36 and 39 (of up to 1400, 256 bytes:
  // 55, 44).
  const uint32_t whole = beside ? (row_bytes <= 64 ? 24 : row_bytes <= 128 ? 16 : 8) : row_bytes <= 64 ? 32 : 16;
  s.waves = kWaves;
  s.heads = 1;
  s.joined = steps > whole || steps > rows * inner * steps / most + kJoinUnits;
  // Where there are no more (row, kv head)s than compute units, twice the waves
  // take a whole one, in half the rounds.  A compute unit takes in only so much
  // at once, so the longer the rows of a key, the fewer units it may hold up the
  // others for: beyond what an equal share would be, `wait` of them cost as
  // much as the join (1.2, 2.3 and 3.5 us for each two units of 64, 128 and 256
  // bytes a key; 5 us).  256 rows of 1000 tokens, 64 bytes: 9.5 us, 14.5 with
  // four waves and 13.3 joined (128 bytes: 15.0, 20.3).
  const uint32_t wait = row_bytes <= 64 ? 10 : row_bytes <= 128 ? 6 : 3;
  if (most > kComputeUnits && rows * inner <= kComputeUnits && steps > 1 && steps * row_bytes <= kAloneBytes &&
      steps <= 2 * rows * inner * steps / most + wait) {
    s.waves = kManyWaves;
    s.joined = false;
  }
  if (!s.joined) {
    const uint64_t items = rows * inner;
    // What reads the same lines stays on one XCD: a kv head's groups, and two heads
    // of 64 bytes (77 rows of 8 such heads: 20 us, 27 apart).  With whole rows dealt
    // out, few of them left XCDs without work (one row of 40 kv heads of 128 bytes,
    // 350 tokens: 6.1 us, 10.8 so; 9 rows of 28, 256 bytes, 900 tokens: 24 us, 36).
    s.deal = s.m_groups * (row_bytes < 128 && kv_heads % 2 == 0 ? 2 : 1);
    s.workgroups = ((items + s.deal - 1) / s.deal + kXcds - 1) / kXcds * kXcds * s.deal;
    return s;
  }
  if (beside) s.heads = heads;
  uint64_t n;
  if (__builtin_mul_overflow(rows * inner, steps, &n)) n = UINT64_MAX;
  s.workgroups = n < most ? (n + kXcds - 1) / kXcds * kXcds : most;
  return s;
}

// Layout: (max, sum) of each part, the weighted sums, the parts of each (row, kv head).
uint64_t attn_workspace_bytes(const AttnShape &s, uint32_t rows, uint32_t kv_heads, uint32_t head_dim) {
  if (!s.joined) return 0;
  const uint64_t parts = parts_of(s);
  return parts * 8 + parts * head_dim * 4 + up16((uint64_t)rows * kv_heads * s.m_groups * sizeof(Parts));
}

hipError_t launch_attn(const AttnArgs &in, int kind, const AttnShape &s, hipStream_t stream) {
  AttnArgs a = in;
  if (s.joined) {
    const uint64_t parts = parts_of(s);
    a.part_o = a.part_ml + 2 * parts;
    a.parts = a.part_o + parts * a.cache.head_dim;
  } else {
    a.part_ml = nullptr;  // the workgroups take whole (row, kv head)s
  }
  if (a.cache.head_dim == 64) return launch_dim<64>(a, kind, s, stream);
  if (a.cache.head_dim == 128) return launch_dim<128>(a, kind, s, stream);
  return launch_dim<256>(a, kind, s, stream);
}

}  // namespace xfer
