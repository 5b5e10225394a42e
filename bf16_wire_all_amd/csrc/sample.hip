// Sampling with temperature, top-k, top-p and min-p from BF16 logits in two
// column shards.
//
// A BF16 logit has at most 65,280 values that count (NaN and -inf do not), so
// a row is counted by value: how often each occurs, in the row's order
// (larger first), is a list of a few thousand (value, count) entries.  On that
// list every filter is a cut of a prefix and the draw a search in running
// sums; one exponential in binary64 serves all equal logits, and counts are
// whole numbers, so no sum depends on the order of atomics.
//
// Two launches:
//   1. count: a workgroup counts a slice of one shard in LDS (16 bits for each
//      pattern, so a slice has fewer than 65,536 columns) and writes the values
//      that occur, in order, with their counts;
//   2. draw: a workgroup for each row adds up its slices' lists in LDS the
//      same way, finds the cuts and the drawn element (its value and how many
//      equal ones come before it), then looks that one up in the slice that
//      holds it.
// Rows of at most 32,768 columns in all take one launch, which counts both
// shards in one workgroup.
// The kernel boundary orders the two steps, as in the argmax.
//
// The bins fill a compute unit's LDS, so 16 waves share it and instructions
// bound the work (a wave's instruction holds its SIMD for four clocks, and
// four waves share one): a pattern's bin is its magnitude, with the counts of
// the two signs in one word, which takes four operations for each logit, and
// the order is made once, when the bins are read; empty runs of 256 bins are
// passed over; one wave does the searches, 64 probes at a time, without
// barriers between them.
#include "decode.h"

namespace xfer {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr uint32_t kPieceCols = 32768;           // columns that a workgroup holds at a time
// Columns of a slice: a piece where that leaves compute units without a slice,
// else as many as 16 bits count, since a list costs as much as a piece.
constexpr uint32_t kSliceCols = kPieceCols, kWideSliceCols = 65528;
constexpr uint32_t kInf = 0x7F80u;               // the pattern of +inf; -inf has the sign bit too
// Values in the row's order, +inf first: positive patterns count down, zero
// (of either sign) is bin kInf, negative ones count up.
constexpr uint32_t kBins = 2 * kInf;
constexpr uint32_t kWords = 32768;               // one for each magnitude: +count in the low half, -count in the high
constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr uint32_t kLdsEntries = 7168;           // lists up to this long stay in LDS, beside the bins
constexpr uint32_t kMaxSlices = 128;
constexpr uint32_t kCountWorkgroups = 256;       // one on each compute unit: the bins fill its LDS

typedef unsigned int v4u __attribute__((ext_vector_type(4)));

// The BF16 pattern of a bin (+0 for zero).
__device__ __forceinline__ uint32_t pattern_of(uint32_t bin) {
  return bin <= kInf ? kInf - bin : 0x8000u | (bin - kInf);
}
__device__ __forceinline__ double value_of(uint32_t bin) { return (double)__uint_as_float(pattern_of(bin) << 16); }

// A barrier that orders LDS alone: loads from global memory stay in flight
// across it, and stores need not have arrived.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

struct Shards {
  const uint16_t *ptr[2];  // in the order of their ids
  uint64_t ld[2];
  uint32_t ncols[2];
  uint32_t off[2];
  uint32_t slices[2];      // slices of each shard
  uint32_t width[2];       // columns of a slice, a multiple of 8
};

struct Slice {
  const uint16_t *ptr;
  uint32_t cols, gid;
};
__device__ __forceinline__ Slice slice_of(const Shards &sh, uint32_t row, uint32_t k) {
  const uint32_t s = k >= sh.slices[0];
  const uint32_t c0 = min((s ? k - sh.slices[0] : k) * sh.width[s], sh.ncols[s]);
  return {sh.ptr[s] + row * sh.ld[s] + c0, min(sh.width[s], sh.ncols[s] - c0), sh.off[s] + c0};
}

// Piece i of a slice.
__device__ __forceinline__ Slice piece_of(const Slice &s, uint32_t i) {
  const uint32_t c0 = min(i * kPieceCols, s.cols);
  return {s.ptr + c0, min(kPieceCols, s.cols - c0), s.gid + c0};
}

// This thread's elements of a piece, all loads in flight at once.
constexpr int kRounds = kPieceCols / 8 / kThreads;
constexpr uint32_t kMasked = 0xFF80FF80u;        // two of -inf
struct Held {
  v4u w[kRounds];
  uint32_t last;  // one element of an incomplete last vector, above another of -inf
};
__device__ __forceinline__ Held load_piece(const Slice &s) {
  Held h;
  const v4u *vp = reinterpret_cast<const v4u *>(s.ptr);
  const uint32_t n_vec = s.cols / 8;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const uint32_t v = r * kThreads + threadIdx.x;
    h.w[r] = v4u{kMasked, kMasked, kMasked, kMasked};
    if (v < n_vec) h.w[r] = vp[v];
  }
  h.last = kMasked;
  if (threadIdx.x < s.cols % 8) h.last = (uint32_t)s.ptr[n_vec * 8 + threadIdx.x] << 16 | 0xFF80u;
  return h;
}

__device__ __forceinline__ void count_low(uint32_t *hist, uint32_t x) {
  atomicAdd(&hist[x & 0x7FFFu], (x >> 15 & 1u) * 0xFFFFu + 1u);
}
__device__ __forceinline__ void count_high(uint32_t *hist, uint32_t x) {
  atomicAdd(&hist[x >> 16 & 0x7FFFu], (x >> 31) * 0xFFFFu + 1u);
}
// The same for elements that may be masked: a wave's atomics on one address
// take their turns, and a mask would send most of them to that of -inf.
__device__ __forceinline__ void count_two_unmasked(uint32_t *hist, uint32_t x) {
  if ((x & 0xFFFFu) != 0xFF80u) count_low(hist, x);
  if (x >> 16 != 0xFF80u) count_high(hist, x);
}

// Counts of a piece added to hist.  Whether the elements are looked at one by
// one for masked ones goes by the first of each vector.
__device__ __forceinline__ void count_piece(uint32_t *hist, const Held &h) {
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (__any((h.w[r].x & 0xFFFFu) == 0xFF80u)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) count_two_unmasked(hist, h.w[r][i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        count_low(hist, h.w[r][i]);
        count_high(hist, h.w[r][i]);
      }
    }
  }
  count_two_unmasked(hist, h.last);
}

__device__ __forceinline__ uint32_t lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// Running sums over the lanes of a wave, by DPP moves (lanes that a move does
// not reach add 0).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  const uint64_t r = ((uint64_t)dpp<CTRL, ROWS>((uint32_t)(b >> 32)) << 32) | dpp<CTRL, ROWS>((uint32_t)b);
  return __longlong_as_double((long long)r);
}
template <typename T>
__device__ __forceinline__ T scan(T x) {
  x += dpp<0x111, 0xF>(x);  // row_shr:1
  x += dpp<0x112, 0xF>(x);
  x += dpp<0x114, 0xF>(x);
  x += dpp<0x118, 0xF>(x);
  x += dpp<0x142, 0xA>(x);  // row_bcast:15 into rows 1 and 3
  x += dpp<0x143, 0xC>(x);  // row_bcast:31 into rows 2 and 3
  return x;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max(x, dpp<0x111, 0xF>(x));
  x = max(x, dpp<0x112, 0xF>(x));
  x = max(x, dpp<0x114, 0xF>(x));
  x = max(x, dpp<0x118, 0xF>(x));
  x = max(x, dpp<0x142, 0xA>(x));
  x = max(x, dpp<0x143, 0xC>(x));
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
__device__ __forceinline__ double read_lane(double x, uint32_t lane) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, (int)lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), (int)lane);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ uint32_t read_lane(uint32_t x, uint32_t lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)x, (int)lane);
}

// The values that occur in hist, in order.  The words go in groups of 256, a
// lane four in a row, group after group round the waves; the constructor
// returns once every group's numbers are known.
constexpr int kGroups = kWords / 256;
struct GroupCounts {
  uint32_t pos[kGroups], neg[kGroups];
};
struct Compact {
  static constexpr int kOwn = kGroups / kWaves;  // groups of a wave
  v4u x[kOwn];
  uint32_t pos_total, total;   // entries above zero, and in all
  uint32_t pos_incl[2], neg_incl[2];  // of lane l: running numbers up to groups 2l and 2l + 1

  __device__ __forceinline__ Compact(const uint32_t *hist, GroupCounts *counts) {
    const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const v4u *words = reinterpret_cast<const v4u *>(hist);
#pragma unroll
    for (int r = 0; r < kOwn; ++r) x[r] = words[(r * kWaves + wave) * 64 + lane];
    if (wave == 0 && lane == 0) {
      // zero of either sign: the first of the values not above it
      const uint32_t z = x[0].x;
      x[0].x = ((z & 0xFFFFu) + (z >> 16)) << 16;
    }
    if (wave == kWaves - 1) {
      // -inf and NaN count nowhere
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t mag = (kGroups - 1) * 256 + lane * 4 + i;
        const uint32_t w = x[kOwn - 1][i];
        x[kOwn - 1][i] = mag > kInf ? 0 : mag == kInf ? w & 0xFFFFu : w;
      }
    }
#pragma unroll
    for (int r = 0; r < kOwn; ++r) {
      uint32_t p = 0, n = 0;
      if (__any((x[r].x | x[r].y | x[r].z | x[r].w) != 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p += __popcll(__ballot((x[r][i] & 0xFFFFu) != 0));
          n += __popcll(__ballot(x[r][i] >> 16 != 0));
        }
      }
      if (lane == 0) {
        counts->pos[r * kWaves + wave] = p;
        counts->neg[r * kWaves + wave] = n;
      }
    }
    lds_barrier();
    const uint32_t p0 = counts->pos[2 * lane], n0 = counts->neg[2 * lane];
    pos_incl[1] = scan(p0 + counts->pos[2 * lane + 1]);
    neg_incl[1] = scan(n0 + counts->neg[2 * lane + 1]);
    pos_incl[0] = pos_incl[1] - counts->pos[2 * lane + 1];
    neg_incl[0] = neg_incl[1] - counts->neg[2 * lane + 1];
    pos_total = read_lane(pos_incl[1], 63);
    total = pos_total + read_lane(neg_incl[1], 63);
  }

  // out(index, bin, count) for each.
  template <typename Emit>
  __device__ __forceinline__ void emit(const Emit &out) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
#pragma unroll
    for (int r = 0; r < kOwn; ++r) {
      if (!__any((x[r].x | x[r].y | x[r].z | x[r].w) != 0)) continue;
      const uint32_t g = r * kWaves + wave, mag0 = g * 256 + lane * 4;
      uint32_t p_below = 0, p_own = 0, p_all = 0, n_below = 0, n_all = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool own = (x[r][i] & 0xFFFFu) != 0;
        const uint64_t a = __ballot(own);
        p_below += lanes_below(a);
        p_own += own;
        p_all += __popcll(a);
        const uint64_t b = __ballot(x[r][i] >> 16 != 0);
        n_below += lanes_below(b);
        n_all += __popcll(b);
      }
      const uint32_t p_incl = read_lane(g % 2 ? pos_incl[1] : pos_incl[0], g / 2);
      const uint32_t n_incl = read_lane(g % 2 ? neg_incl[1] : neg_incl[0], g / 2);
      // above zero the order goes down the magnitudes: later groups, later
      // lanes and a lane's later words come first
      uint32_t at = pos_total - p_incl + (p_all - p_below - p_own);
#pragma unroll
      for (int i = 3; i >= 0; --i)
        if (const uint32_t c = x[r][i] & 0xFFFFu) out(at++, kInf - (mag0 + i), c);
      at = pos_total + n_incl - n_all + n_below;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (const uint32_t c = x[r][i] >> 16) out(at++, kInf + mag0 + i, c);
    }
  }
};

// The same of kInf words that hold one 32-bit count each: the values of counts
// that 16 bits may not hold.  A wave takes a run of words; returns the number
// of entries, after a barrier.
template <typename Emit>
__device__ __forceinline__ uint32_t compact_wide(const uint32_t *words, uint32_t *scratch, const Emit &out) {
  constexpr uint32_t kRun = kWords / kWaves;
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  uint32_t mine = 0;
  for (uint32_t w = wave * kRun + lane; w < (wave + 1) * kRun; w += 64) mine += __popcll(__ballot(w < kInf && words[w]));
  if (lane == 0) scratch[wave] = mine;
  __syncthreads();
  uint32_t next = 0, total = 0;
  for (uint32_t i = 0; i < kWaves; ++i) {
    if (i < wave) next += scratch[i];
    total += scratch[i];
  }
  for (uint32_t w = wave * kRun + lane; w < (wave + 1) * kRun; w += 64) {
    const uint32_t c = w < kInf ? words[w] : 0;
    const uint64_t b = __ballot(c != 0);
    if (c) out(next + lanes_below(b), w, c);
    next += __popcll(b);
  }
  __syncthreads();
  return total;
}

__device__ __forceinline__ void clear(uint32_t *hist) {
  v4u *p = reinterpret_cast<v4u *>(hist);
#pragma unroll
  for (uint32_t i = 0; i < kWords / 4 / kThreads; ++i) p[i * kThreads + threadIdx.x] = v4u{0, 0, 0, 0};
}

// What the count leaves of a slice besides its list (bin << 16 | count).
struct SliceInfo {
  uint32_t length, most;  // entries, and the largest count
};

// A workgroup goes from slice to slice, and loads the next piece's elements
// before it sorts out the counts of the one at hand.
__global__ __launch_bounds__(kThreads) void sample_count_kernel(Shards sh, uint32_t n_slices, uint32_t jobs,
                                                                uint64_t row_cap, uint32_t *lists, SliceInfo *infos) {
  __shared__ __attribute__((aligned(16))) uint32_t hist[kWords];
  __shared__ GroupCounts counts;
  __shared__ uint32_t most[kWaves];
  uint32_t job = blockIdx.x;
  Slice slice = slice_of(sh, job / n_slices, job % n_slices);
  Held held = load_piece(piece_of(slice, 0));
  for (; job < jobs; job += gridDim.x) {
    clear(hist);
    lds_barrier();
    count_piece(hist, held);
    if (slice.cols > kPieceCols) count_piece(hist, load_piece(piece_of(slice, 1)));
    const uint32_t next = job + gridDim.x;
    if (next < jobs) {
      slice = slice_of(sh, next / n_slices, next % n_slices);
      held = load_piece(piece_of(slice, 0));
    }
    lds_barrier();
    Compact c(hist, &counts);
    const uint32_t row = job / n_slices, k = job % n_slices, s = k >= sh.slices[0];
    uint32_t *list = lists + row * row_cap + (s ? (uint64_t)sh.slices[0] * sh.width[0] : 0) +
                     (uint64_t)(s ? k - sh.slices[0] : k) * sh.width[s];
    uint32_t largest = 0;
    c.emit([&](uint32_t i, uint32_t bin, uint32_t count) {
      list[i] = bin << 16 | count;
      largest = max(largest, count);
    });
    largest = wave_max(largest);
    if (threadIdx.x % 64 == 0) most[threadIdx.x / 64] = largest;
    lds_barrier();  // hist and counts are written again
    if (threadIdx.x == 0) {
#pragma unroll
      for (int w = 1; w < kWaves; ++w) largest = max(largest, most[w]);
      infos[job] = SliceInfo{c.total, largest};
    }
  }
}

struct Scratch {
  uint32_t slice_length[kMaxSlices], slice_count[kMaxSlices];
  double mass[kWaves];
  uint32_t count[kWaves];
  uint32_t below;          // the first entry whose weight is below min_p's limit
  uint32_t place[4];
  uint32_t at, rank;       // the drawn entry, and the drawn element's place among its equals
  float prob;
};

// Smallest r in [1, most] with before + r * w >= target (OVER: > target).
template <bool OVER>
__device__ __forceinline__ uint32_t rank_of(double before, double w, uint32_t most, double target) {
  const double q = (target - before) / w;
  uint32_t r = q > 1.0 ? (q < (double)most ? (uint32_t)q : most) : 1;
  auto reached = [&](uint32_t k) {
    const double c = before + k * w;
    return OVER ? c > target : c >= target;
  };
  // the quotient is off by one step at most
  if (r > 1 && reached(r - 1)) --r;
  if (!reached(r) && r < most) ++r;
  if (!reached(r) && r < most) ++r;
  return r;
}

// First of n (at most 64 * 16) values for which reached(value index) holds, by
// one wave; n if none does.  reached is monotone.
template <typename Reached>
__device__ __forceinline__ uint32_t first_of_1024(const Reached &reached) {
  const uint32_t lane = threadIdx.x % 64;
  const uint64_t coarse = __ballot(reached(lane * 16 + 15));
  if (!coarse) return kThreads;
  const uint32_t base = (uint32_t)__builtin_ctzll(coarse) * 16;
  const uint64_t fine = __ballot(lane < 16 && reached(base + lane % 16));
  return base + (fine ? (uint32_t)__builtin_ctzll(fine) : 15);
}

// The cuts and the draw on a list of n > 0 entries: first(i, &count, &weight)
// once for each entry, then entry(i, &count, &weight).
// Thread t sums up entries [t * per, (t + 1) * per); `masses` and `counts`
// (LDS, one for each thread) become the running sums up to each thread's
// last.  One wave then finds each border: the thread first, then the entry
// among its own.
template <typename First, typename Entry>
__device__ void search(const First &first, const Entry &entry, uint32_t n, const xfer_sample_params &p, float u, double *masses,
                       uint32_t *counts, Scratch *sc) {
  const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  const uint32_t per = (n + kThreads - 1) / kThreads;
  const uint32_t i0 = min(tid * per, n), i1 = min(i0 + per, n);
  const double least = p.min_p > 1.0f ? 1.0 : (double)p.min_p;
  if (tid == 0) sc->below = kNone;
  uint32_t count = 0, below = kNone;
  double mass = 0;
  for (uint32_t i = i0; i < i1; ++i) {
    uint32_t c;
    double w;
    first(i, &c, &w);
    count += c;
    mass += c * w;
    if (w < least && below == kNone) below = i;
  }
  count = scan(count);
  mass = scan(mass);
  if (lane == 63) {
    sc->count[wave] = count;
    sc->mass[wave] = mass;
  }
  __syncthreads();
  const uint64_t any_below = __ballot(below != kNone);
  if (any_below && lane == (uint32_t)__builtin_ctzll(any_below)) atomicMin(&sc->below, below);
  {
    // the waves before this one, in order
    const uint32_t wc = scan(lane < kWaves ? sc->count[lane % kWaves] : 0);
    const double wm = scan(lane < kWaves ? sc->mass[lane % kWaves] : 0.0);
    if (wave) {
      count += read_lane(wc, __builtin_amdgcn_readfirstlane(wave - 1));
      mass += read_lane(wm, __builtin_amdgcn_readfirstlane(wave - 1));
    }
  }
  counts[tid] = count;
  masses[tid] = mass;
  __syncthreads();
  if (wave != 0) return;

  struct Border {
    uint32_t at, count;  // an entry and its elements
    uint32_t rank;       // how many of them come up to the border: at first, all
    uint32_t n_before;   // elements before the entry
    double before, w;    // the weights before the entry, and of each of its elements
  };
  // Among the entries of thread t up to entry `last`, of which `last_count`
  // elements count at most, the first that reached(running count, running
  // mass) holds for; the last of them if it holds for none (*none).
  bool none;
  auto among = [&](uint32_t t, uint32_t last, uint32_t last_count, const auto &reached) {
    const uint32_t i = t * per + lane;
    const bool there = lane < per && i < n && i <= last;
    uint32_t c = 0;
    double w = 0;
    if (there) {
      entry(i, &c, &w);
      if (i == last) c = min(c, last_count);
    }
    const uint32_t n_run = scan(c) + (t ? counts[t - 1] : 0);
    const double m_run = scan(c * w) + (t ? masses[t - 1] : 0.0);
    const uint64_t hit = __ballot(there && reached(n_run, m_run)), all = __ballot(there);
    none = !hit;
    const uint32_t l = hit ? (uint32_t)__builtin_ctzll(hit) : 63 - (uint32_t)__builtin_clzll(all);
    Border b;
    b.at = t * per + l;
    b.count = b.rank = read_lane(c, l);
    b.w = read_lane(w, l);
    b.n_before = read_lane(n_run, l) - b.count;
    b.before = l ? read_lane(m_run, l - 1) : t ? masses[t - 1] : 0.0;
    return b;
  };

  // top_k
  const uint32_t total = counts[kThreads - 1];
  const bool greedy = !(p.temperature > 0.0f);
  const uint32_t keep = greedy ? 1 : p.top_k == 0 ? total : min(p.top_k, total);
  uint32_t t = keep == total ? (n - 1) / per : first_of_1024([&](uint32_t s) { return counts[s] >= keep; });
  Border f = among(t, n - 1, kNone, [&](uint32_t running, double) { return running >= keep; });
  f.rank = keep - f.n_before;
  double z = f.before + f.rank * f.w;

  // top_p
  if (p.top_p < 1.0f) {
    const double target = (double)p.top_p * z;
    t = first_of_1024([&](uint32_t s) { return masses[s] >= target; });
    if (t < kThreads && t * per <= f.at) {
      const Border b = among(t, f.at, f.rank, [&](uint32_t, double running) { return running >= target; });
      if (!none || b.at < f.at) {
        f = b;
        f.rank = rank_of<false>(b.before, b.w, b.count, target);
      }
    }
  }
  // min_p: the first entry's weight is 1, so an entry below it has one before it
  const uint32_t m_at = sc->below;
  if (m_at <= f.at) f = among((m_at - 1) / per, m_at - 1, kNone, [](uint32_t, double) { return false; });
  z = f.before + f.rank * f.w;

  // The draw.
  const double target = u > 0.0f ? (double)u * z : 0.0;
  t = first_of_1024([&](uint32_t s) { return masses[s] > target; });
  if (t * per > f.at) t = f.at / per;
  const Border d = among(t, f.at, f.rank, [&](uint32_t, double running) { return running > target; });
  if (lane == 0) {
    sc->at = d.at;
    sc->rank = (none ? d.count : rank_of<true>(d.before, d.w, d.count, target)) - 1;
    sc->prob = (float)(d.w / z);
  }
}

// Whether one of two patterns is 0 (it may also say so of a pattern of 1 above
// one of 0).
__device__ __forceinline__ uint32_t zero_half(uint32_t x) { return (x - 0x00010001u) & ~x & 0x80008000u; }

// Column of the rank-th element (from 0) of `bin` in a slice, kNone (to every
// thread) if it holds no more than rank; *held becomes how many it holds.
__device__ uint32_t locate(const Slice &s, uint32_t bin, uint32_t rank, uint32_t *held, uint32_t *totals,
                           uint32_t *place) {
  const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  const Held h = load_piece(s);
  // zero has two patterns: without its sign it has one
  const uint32_t keep = bin == kInf ? 0x7FFF7FFFu : 0xFFFFFFFFu, two = pattern_of(bin) * 0x10001u;
  uint32_t match[kRounds];  // bit e: element e of this thread's vector is of the bin
  if (tid == 0) place[0] = kNone;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    match[r] = 0;
    uint32_t x[4], some = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = (h.w[r][i] & keep) ^ two;
      some |= zero_half(x[i]);
    }
    uint32_t c = 0;
    if (__any(some != 0)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) match[r] |= ((x[i] & 0xFFFFu) == 0) << (2 * i) | (x[i] >> 16 == 0) << (2 * i + 1);
      c = read_lane(scan((uint32_t)__popc(match[r])), 63);
    }
    if (lane == 0) totals[r * kWaves + wave] = c;
  }
  // the elements of an incomplete last vector, held by the first threads, come last
  const bool last = ((h.last & keep) ^ two) >> 16 == 0;
  const uint64_t lasts = __ballot(last);
  __syncthreads();
  if (wave == 0) {
    static_assert(kRounds * kWaves == 64, "one lane for each round of a wave");
    const uint32_t c = totals[lane];
    const uint32_t incl = scan(c);
    if (incl - c <= rank && rank < incl) {
      place[0] = lane;
      place[1] = rank - (incl - c);
    }
    const uint32_t vectors = read_lane(incl, 63);
    if (last && vectors + lanes_below(lasts) == rank) {
      place[0] = 64;
      place[3] = s.cols / 8 * 8 + lane;
    }
    if (lane == 0) place[2] = vectors + __popcll(lasts);
  }
  __syncthreads();
  *held = place[2];
  const uint32_t at = place[0];
  if (at == kNone) return kNone;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (at != r * kWaves + wave) continue;
    const uint32_t c = __popc(match[r]);
    const uint32_t incl = scan(c);
    uint32_t left = place[1];
    if (incl - c <= left && left < incl) {
      left -= incl - c;
      uint32_t m = match[r];
      for (; left; --left) m &= m - 1;
      place[3] = (r * kThreads + tid) * 8 + (uint32_t)__builtin_ctz(m);
    }
  }
  __syncthreads();
  return place[3];
}

struct DrawArgs {
  Shards sh;
  const xfer_sample_params *params;
  const float *u;
  xfer_sampled *out;
  const uint32_t *lists;    // per slice (two launches)
  const SliceInfo *infos;
  uint2 *merged;            // a row's list where LDS does not hold it: (bin, count)
  uint64_t row_cap, merged_cap;
  uint32_t n_slices;
};

__device__ __forceinline__ const uint32_t *list_of(const DrawArgs &a, uint32_t row, uint32_t k) {
  const uint32_t s = k >= a.sh.slices[0];
  return a.lists + row * a.row_cap + (s ? (uint64_t)a.sh.slices[0] * a.sh.width[0] : 0) +
         (uint64_t)(s ? k - a.sh.slices[0] : k) * a.sh.width[s];
}

// The count of `bin` in a list of n entries in the bins' order (0 if it has
// none), by one wave: 64 probes at a time.
__device__ __forceinline__ uint32_t count_in_list(const uint32_t *list, uint32_t n, uint32_t bin) {
  const uint32_t lane = threadIdx.x % 64;
  uint32_t lo = 0, hi = n;  // the entry lies in [lo, hi) if there is one
  while (hi - lo > 64) {
    const uint32_t step = (hi - lo + 63) / 64, i = min(lo + (lane + 1) * step - 1, hi - 1);
    const uint64_t up = __ballot(list[i] >> 16 >= bin);
    if (!up) return 0;
    const uint32_t first = (uint32_t)__builtin_ctzll(up);
    hi = min(lo + (first + 1) * step, hi);
    lo = min(lo + first * step, hi);
  }
  const uint32_t e = lane < hi - lo ? list[lo + lane] : 0;
  const uint64_t is = __ballot(e != 0 && e >> 16 == bin);
  return is ? read_lane(e, (uint32_t)__builtin_ctzll(is)) & 0xFFFFu : 0;
}

// How the waves share a row's lists: a slice to each, or several waves to a
// slice, with kAtOnce loads of each lane in flight.
constexpr int kAtOnce = 8;
struct Share {
  uint32_t k0, groups;  // the wave's first slice, and the step to its next
  uint32_t i0, step;    // the lane's first entry, and the step to its next
};
__device__ __forceinline__ Share share_of(uint32_t n_slices) {
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const uint32_t ways = n_slices < kWaves ? kWaves / n_slices : 1, groups = kWaves / ways;
  return {wave / ways, groups, wave % ways * 64 + lane, ways * 64};
}

// The first entries of this lane's share, before it is known how many there are.
struct Ahead {
  uint32_t e[kAtOnce];
};
__device__ __forceinline__ Ahead load_ahead(const DrawArgs &a, uint32_t row, const Share &h) {
  Ahead r;
  const uint32_t k = min(h.k0, a.n_slices - 1), width = a.sh.width[k >= a.sh.slices[0]];
  const uint32_t *list = list_of(a, row, k);
#pragma unroll
  for (int j = 0; j < kAtOnce; ++j) r.e[j] = list[min(h.i0 + j * h.step, width - 1)];
  return r;
}

// visit(entry) of every entry of a row's lists.
template <typename Visit>
__device__ __forceinline__ void for_lists(const DrawArgs &a, uint32_t row, const uint32_t *lengths, const Share &h,
                                          const Ahead &ahead, const Visit &visit) {
  for (uint32_t k = h.k0; k < a.n_slices; k += h.groups) {
    const uint32_t *list = list_of(a, row, k);
    const uint32_t n = lengths[k];
    for (uint32_t i = h.i0; i < n; i += kAtOnce * h.step) {
      Ahead r = ahead;
      if (k != h.k0 || i != h.i0) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
          if (i + j * h.step < n) r.e[j] = list[i + j * h.step];
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (i + j * h.step < n) visit(r.e[j]);
    }
  }
}

// ONE: the row is counted here (both shards hold at most kPieceCols columns
// together); else its slices' lists are added up.
template <bool ONE>
__global__ __launch_bounds__(kThreads) void sample_draw_kernel(DrawArgs a) {
  __shared__ __attribute__((aligned(16))) uint32_t lds[kWords];
  __shared__ uint32_t list[kLdsEntries];  // bin << 16 | count
  __shared__ GroupCounts counts;
  __shared__ uint32_t totals[64];
  __shared__ Scratch sc;
  const uint32_t row = blockIdx.x, tid = threadIdx.x;
  uint2 *merged = a.merged + row * a.merged_cap;
  const xfer_sample_params p = a.params[row];
  const float u = a.u[row];

  // The row's list: in LDS if counts fit 16 bits and it is no longer than
  // kLdsEntries, else in the workspace.
  uint32_t n = 0;
  bool packed = true;
  const Share share = share_of(ONE ? 1 : a.n_slices);
  Ahead ahead{};
  if (ONE) {
    const Held h0 = load_piece(slice_of(a.sh, row, 0)), h1 = load_piece(slice_of(a.sh, row, 1));
    clear(lds);
    lds_barrier();
    count_piece(lds, h0);
    count_piece(lds, h1);
    lds_barrier();
  } else {
    SliceInfo info{0, 0};
    if (tid < a.n_slices) info = a.infos[row * a.n_slices + tid];
    ahead = load_ahead(a, row, share);
    clear(lds);
    if (tid < kMaxSlices) {  // the first two waves
      sc.slice_length[tid] = info.length;
      const uint32_t most = scan(info.most);
      if (tid % 64 == 63) sc.count[tid / 64] = most;
    }
    lds_barrier();
    packed = sc.count[0] + sc.count[1] <= 0xFFFFu;  // no value can occur more often than that
    if (packed) {
      for_lists(a, row, sc.slice_length, share, ahead, [&](uint32_t e) {
        const uint32_t b = e >> 16, c = e & 0xFFFFu;
        if (b < kInf)
          atomicAdd(&lds[kInf - b], c);
        else
          atomicAdd(&lds[b - kInf], c << 16);
      });
      lds_barrier();
    }
  }
  if (packed) {
    Compact c(lds, &counts);
    n = c.total;
    if (n <= kLdsEntries)
      c.emit([&](uint32_t i, uint32_t bin, uint32_t count) { list[i] = bin << 16 | count; });
    else
      c.emit([&](uint32_t i, uint32_t bin, uint32_t count) { merged[i] = make_uint2(bin, count); });
    __syncthreads();
  } else {
    // One half of the values at a time, 32 bits for each (lds is clear for the first).
#pragma unroll 1
    for (uint32_t half = 0; half < 2; ++half) {
      for_lists(a, row, sc.slice_length, share, ahead, [&](uint32_t e) {
        const uint32_t b = (e >> 16) - half * kInf;
        if (b < kInf) atomicAdd(&lds[b], e & 0xFFFFu);
      });
      __syncthreads();
      n += compact_wide(lds, totals, [&](uint32_t i, uint32_t bin, uint32_t count) {
        merged[n + i] = make_uint2(half * kInf + bin, count);
      });
      clear(lds);
      __syncthreads();
    }
  }
  if (n == 0) {
    if (tid == 0) a.out[row] = xfer_sampled{0.0f, -1};
    return;
  }

  const bool in_lds = packed && n <= kLdsEntries;
  const double per_t = p.temperature > 0.0f ? 1.0 / (double)p.temperature : 1.0;
  const double top = value_of(in_lds ? list[0] >> 16 : merged[0].x);
  const bool top_inf = isinf(top);
  auto weight = [&](uint32_t i, uint32_t bin) -> double {
    if (i == 0) return 1.0;
    return top_inf ? 0.0 : exp((value_of(bin) - top) * per_t);
  };
  // The bins are done with: weights and running sums take their place.
  double *weights = reinterpret_cast<double *>(lds), *masses = weights + kLdsEntries;
  uint32_t *sums = reinterpret_cast<uint32_t *>(masses + kThreads);
  static_assert(kLdsEntries * 8 + kThreads * 12 <= kWords * 4, "they fit");
  if (in_lds) {
    auto entry = [&](uint32_t i, uint32_t *c, double *w) { *c = list[i] & 0xFFFFu, *w = weights[i]; };
    auto first = [&](uint32_t i, uint32_t *c, double *w) {
      const uint32_t e = list[i];
      *c = e & 0xFFFFu;
      weights[i] = *w = weight(i, e >> 16);
    };
    search(first, entry, n, p, u, masses, sums, &sc);
  } else {
    auto entry = [&](uint32_t i, uint32_t *c, double *w) {
      const uint2 e = merged[i];
      *c = e.y, *w = weight(i, e.x);
    };
    search(entry, entry, n, p, u, masses, sums, &sc);
  }
  __syncthreads();
  const uint32_t bin = in_lds ? list[sc.at] >> 16 : merged[sc.at].x;
  uint32_t rank = sc.rank, k = 0;
  if (!ONE) {
    // How many of the value each slice holds: its list is in order.
    for (uint32_t s = tid / 64; s < a.n_slices; s += kWaves) {
      const uint32_t c = count_in_list(list_of(a, row, s), sc.slice_length[s], bin);
      if (tid % 64 == 0) sc.slice_count[s] = c;
    }
    __syncthreads();
    while (k + 1 < a.n_slices && rank >= sc.slice_count[k]) rank -= sc.slice_count[k++];
  }
  // In one of two pieces: the slice's, or the row's two shards.
  uint32_t held;
  Slice s = ONE ? slice_of(a.sh, row, 0) : piece_of(slice_of(a.sh, row, k), 0);
  uint32_t col = locate(s, bin, rank, &held, totals, sc.place);
  if (col == kNone) {
    lds_barrier();  // place is written again
    s = ONE ? slice_of(a.sh, row, 1) : piece_of(slice_of(a.sh, row, k), 1);
    col = locate(s, bin, rank - held, &held, totals, sc.place);
  }
  if (tid == 0) a.out[row] = xfer_sampled{sc.prob, (int32_t)(s.gid + col)};
}

uint32_t round_up8(uint32_t x) { return (x + 7u) & ~7u; }

}  // namespace

// Slices of the narrower kind that a row is cut into, at most.
uint32_t sample_slices(uint32_t ncols0, uint32_t ncols1) {
  if ((uint64_t)ncols0 + ncols1 <= kPieceCols) return 1;
  return (ncols0 + kSliceCols - 1) / kSliceCols + (ncols1 + kSliceCols - 1) / kSliceCols;
}

namespace {

struct Sizes {
  bool one;
  uint32_t slices[2], width[2];
  uint64_t row_cap, merged_cap;
};
Sizes sizes_of(uint32_t rows, uint32_t ncols0, uint32_t ncols1) {
  Sizes z{};
  z.one = (uint64_t)ncols0 + ncols1 <= kPieceCols;
  const uint32_t n[2] = {ncols0, ncols1};
  const uint32_t most = (uint64_t)rows * sample_slices(n[0], n[1]) <= kCountWorkgroups ? kSliceCols : kWideSliceCols;
  for (int i = 0; i < 2; ++i) {
    z.slices[i] = (n[i] + most - 1) / most;
    z.width[i] = round_up8((n[i] + z.slices[i] - 1) / z.slices[i]);
    z.row_cap += (uint64_t)z.slices[i] * z.width[i];
  }
  z.merged_cap = z.row_cap < kBins ? z.row_cap : kBins;
  if (z.one) z.row_cap = 0;
  return z;
}
uint64_t up16(uint64_t x) { return (x + 15) / 16 * 16; }

}  // namespace

// Layout: the rows' merged lists, the slices' lengths, the slices' lists.
uint64_t sample_workspace_bytes(uint32_t rows, uint32_t ncols0, uint32_t ncols1) {
  const Sizes z = sizes_of(rows, ncols0, ncols1);
  uint64_t n = rows * z.merged_cap * 8;
  if (!z.one) n += up16((uint64_t)rows * (z.slices[0] + z.slices[1]) * sizeof(SliceInfo)) + rows * z.row_cap * 4;
  return up16(n);
}

hipError_t launch_sample(const SampleArgs &in, hipStream_t stream) {
  // the shard with the lower ids first
  const int order[2] = {in.s[0].col_offset < in.s[1].col_offset ? 0 : 1, in.s[0].col_offset < in.s[1].col_offset ? 1 : 0};
  const Sizes z = sizes_of(in.rows, in.s[order[0]].ncols, in.s[order[1]].ncols);
  DrawArgs a{};
  for (int i = 0; i < 2; ++i) {
    const ArgmaxShard &s = in.s[order[i]];
    a.sh.ptr[i] = s.ptr;
    a.sh.ld[i] = s.ld;
    a.sh.ncols[i] = s.ncols;
    a.sh.off[i] = s.col_offset;
    a.sh.slices[i] = z.slices[i];
    a.sh.width[i] = z.width[i];
  }
  uint8_t *ws = static_cast<uint8_t *>(in.workspace);
  a.params = in.params;
  a.u = in.u;
  a.out = in.out;
  a.merged = reinterpret_cast<uint2 *>(ws);
  a.merged_cap = z.merged_cap;
  if (z.one) return launch(sample_draw_kernel<true>, dim3(in.rows), dim3(kThreads), 0, stream, a);
  a.n_slices = z.slices[0] + z.slices[1];
  a.row_cap = z.row_cap;
  const uint32_t jobs = in.rows * a.n_slices;
  SliceInfo *infos = reinterpret_cast<SliceInfo *>(ws + (uint64_t)in.rows * z.merged_cap * 8);
  uint32_t *lists = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(infos) + up16((uint64_t)jobs * sizeof(SliceInfo)));
  a.infos = infos;
  a.lists = lists;
  const hipError_t e = launch(sample_count_kernel, dim3(jobs < kCountWorkgroups ? jobs : kCountWorkgroups),
                              dim3(kThreads), 0, stream, a.sh, a.n_slices, jobs, a.row_cap, lists, infos);
  if (e != hipSuccess) return e;
  return launch(sample_draw_kernel<false>, dim3(in.rows), dim3(kThreads), 0, stream, a);
}

}  // namespace xfer
