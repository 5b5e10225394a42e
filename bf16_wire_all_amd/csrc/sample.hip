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
//   1. count: a workgroup counts a slice of at most 32,768 columns of one
//      shard in LDS (16 bits for each value: a slice cannot overflow them) and
//      writes the values that occur, in order, with their counts;
//   2. draw: a workgroup for each row adds up its slices' lists in LDS, one
//      half of the values at a time, finds the cuts and the drawn element (its
//      value and how many equal ones come before it), then looks that one up
//      in the slice that holds it.
// Rows of at most 32,768 columns in all take one launch, which counts both
// shards in one workgroup.
// The kernel boundary orders the two steps, as in the argmax.
#include "decode.h"

namespace xfer {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr uint32_t kSliceCols = 32768;
// Values in the row's order, +inf first: bin = 0xFF80 - ord(value), where ord
// maps BF16 patterns to integers in numeric order with -0 and +0 equal.
constexpr uint32_t kBins = 65280;
constexpr uint32_t kHalf = kBins / 2;            // bins of positive values; zero is the first of the others
constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr uint32_t kLdsEntries = 8192;           // lists up to this long stay in LDS
constexpr uint32_t kMaxSlices = 128;

typedef unsigned int v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t bin_of(uint32_t v) {
  const uint32_t mag = v & 0x7FFFu;
  const uint32_t ord = (v & 0x8000u) ? 0x8000u - mag : 0x8000u + mag;
  return 0xFF80u - ord;  // at least kBins for -inf and NaN (which wraps around)
}

__device__ __forceinline__ double value_of(uint32_t bin) {
  const uint32_t ord = 0xFF80u - bin;
  const uint32_t bits = ord >= 0x8000u ? ord - 0x8000u : 0x8000u | (0x8000u - ord);
  return (double)__uint_as_float(bits << 16);
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

__device__ __forceinline__ void count_one(uint32_t *hist, uint32_t v) {
  const uint32_t b = bin_of(v);
  if (b < kBins) atomicAdd(&hist[b / 2], b % 2 ? 0x10000u : 1u);
}

// Counts of a slice added to hist: two bins of 16 bits in a word.
__device__ __forceinline__ void count_slice(uint32_t *hist, const Slice &s) {
  const v4u *vp = reinterpret_cast<const v4u *>(s.ptr);
  const uint32_t n_vec = s.cols / 8;
  for (uint32_t v = threadIdx.x; v < n_vec; v += kThreads) {
    const v4u w = vp[v];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      count_one(hist, w[i] & 0xFFFFu);
      count_one(hist, w[i] >> 16);
    }
  }
  if (threadIdx.x < s.cols % 8) count_one(hist, s.ptr[n_vec * 8 + threadIdx.x]);
}

__device__ __forceinline__ uint32_t lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// The bins of `words` words of hist that occur, in order: emit(index, bin,
// count) for each, indices from `first` on; returns the number of them.
// PACKED: two bins in a word, else one.  A wave takes a run of words, 64 at a time.
template <bool PACKED, typename Emit>
__device__ __forceinline__ uint32_t compact(const uint32_t *hist, uint32_t words, uint32_t bin0, uint32_t first,
                                            uint32_t *scratch, Emit &&emit) {
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const uint32_t per_wave = (words + kThreads - 1) / kThreads * 64;
  const uint32_t w0 = wave * per_wave, w1 = min(w0 + per_wave, words);
  uint32_t mine = 0;
  for (uint32_t w = w0 + lane; w < w1; w += 64) {
    const uint32_t x = hist[w];
    mine += PACKED ? ((x & 0xFFFFu) != 0) + (x >> 16 != 0) : x != 0;
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) mine += __shfl_xor(mine, d);
  if (lane == 0) scratch[wave] = mine;
  __syncthreads();
  uint32_t at = first, total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i < (int)wave) at += scratch[i];
    total += scratch[i];
  }
  for (uint32_t base = w0; base < w1; base += 64) {
    const uint32_t w = base + lane;
    const uint32_t x = w < w1 ? hist[w] : 0;
    if (PACKED) {
      const uint32_t lo = x & 0xFFFFu, hi = x >> 16;
      const uint64_t blo = __ballot(lo != 0), bhi = __ballot(hi != 0);
      if (!(blo | bhi)) continue;
      uint32_t i = at + lanes_below(blo) + lanes_below(bhi);
      if (lo) emit(i++, bin0 + 2 * w, lo);
      if (hi) emit(i, bin0 + 2 * w + 1, hi);
      at += __popcll(blo) + __popcll(bhi);
    } else {
      const uint64_t b = __ballot(x != 0);
      if (!b) continue;
      if (x) emit(at + lanes_below(b), bin0 + w, x);
      at += __popcll(b);
    }
  }
  __syncthreads();  // scratch and hist may be written again
  return total;
}

__device__ __forceinline__ void clear(uint32_t *hist, uint32_t words) {
  v4u *p = reinterpret_cast<v4u *>(hist);
  for (uint32_t i = threadIdx.x; i < words / 4; i += kThreads) p[i] = v4u{0, 0, 0, 0};
}

// Slice k of a row -> its list (bin << 16 | count) and the list's length.
__global__ __launch_bounds__(kThreads) void sample_count_kernel(Shards sh, uint32_t n_slices, uint64_t row_cap,
                                                                uint32_t *lists, uint32_t *lengths) {
  __shared__ __attribute__((aligned(16))) uint32_t hist[kHalf];
  __shared__ uint32_t scratch[kWaves];
  const uint32_t row = blockIdx.x / n_slices, k = blockIdx.x % n_slices;
  clear(hist, kHalf);
  __syncthreads();
  count_slice(hist, slice_of(sh, row, k));
  __syncthreads();
  const uint32_t s = k >= sh.slices[0];
  uint32_t *list = lists + row * row_cap + (s ? (uint64_t)sh.slices[0] * sh.width[0] : 0) +
                   (uint64_t)(s ? k - sh.slices[0] : k) * sh.width[s];
  const uint32_t n = compact<true>(hist, kHalf, 0, 0, scratch,
                                   [&](uint32_t i, uint32_t bin, uint32_t count) { list[i] = bin << 16 | count; });
  if (threadIdx.x == 0) lengths[blockIdx.x] = n;
}

// What the search leaves for every thread to read.
struct Found {
  uint32_t k_at, k_rank;  // the last entry that top_k keeps, and how many of its elements
  double z_k;             // the weights that top_k keeps
  uint32_t p_at, m_at;    // the first entry that reaches top_p, and that falls below min_p
  uint32_t f_at, f_rank;  // the last entry kept in the end
  double z;
  uint32_t d_first;       // the first entry whose running sum passes the drawn number
  uint32_t d_at, d_rank;  // the drawn entry, and the drawn element's place among its equals
  float prob;
};

struct Scratch {
  double mass[kWaves];
  uint32_t count[kWaves];
  uint32_t slice_count[kMaxSlices];
  uint32_t place[4];
  Found f;
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

// The cuts and the draw on a list of n > 0 entries: entry(i, &count, &weight).
// Thread t holds entries [t * per, ...): its running sums start from a scan
// over the threads in order.
template <typename Entry>
__device__ void search(const Entry &entry, uint32_t n, const xfer_sample_params &p, float u, Scratch *sc) {
  const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  const uint32_t per = (n + kThreads - 1) / kThreads;
  const uint32_t i0 = min(tid * per, n), i1 = min(i0 + per, n);
  uint32_t count = 0;
  double mass = 0;
  for (uint32_t i = i0; i < i1; ++i) {
    uint32_t c;
    double w;
    entry(i, &c, &w);
    count += c;
    mass += c * w;
  }
  uint32_t n_incl = count;
  double m_incl = mass;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t nc = __shfl_up(n_incl, d);
    const double nm = __shfl_up(m_incl, d);
    if ((int)lane >= d) {
      n_incl += nc;
      m_incl += nm;
    }
  }
  if (lane == 63) {
    sc->count[wave] = n_incl;
    sc->mass[wave] = m_incl;
  }
  if (tid == 0) sc->f = Found{kNone, 0, 0, kNone, kNone, 0, 0, 0, kNone, 0, 0, 0};
  __syncthreads();
  uint32_t n_before = 0, total = 0;
  double m_before = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i < (int)wave) {
      n_before += sc->count[i];
      m_before += sc->mass[i];
    }
    total += sc->count[i];
  }
  n_before += n_incl - count;
  const double up = __shfl_up(m_incl, 1);
  if (lane) m_before += up;

  // top_k: counts are exact, so one thread finds it.
  const bool greedy = !(p.temperature > 0.0f);
  const uint32_t keep = greedy ? 1 : p.top_k == 0 ? total : min(p.top_k, total);
  if (n_before < keep && keep <= n_before + count) {
    uint32_t nb = n_before;
    double mb = m_before;
    for (uint32_t i = i0; i < i1; ++i) {
      uint32_t c;
      double w;
      entry(i, &c, &w);
      if (keep <= nb + c) {
        sc->f.k_at = i;
        sc->f.k_rank = keep - nb;
        sc->f.z_k = mb + (keep - nb) * w;
        break;
      }
      nb += c;
      mb += c * w;
    }
  }
  __syncthreads();

  // The first entries that reach top_p of that, and that fall below min_p.
  const uint32_t k_at = sc->f.k_at, k_rank = sc->f.k_rank;
  const bool by_p = p.top_p < 1.0f;
  const double p_target = (double)p.top_p * sc->f.z_k;
  const double least = p.min_p > 1.0f ? 1.0 : (double)p.min_p;
  {
    double mb = m_before;
    bool reached = !by_p, below = false;
    for (uint32_t i = i0; i < i1 && i <= k_at && !(reached && below); ++i) {
      uint32_t c;
      double w;
      entry(i, &c, &w);
      const double end = mb + (i == k_at ? k_rank : c) * w;
      if (!reached && end >= p_target) {
        atomicMin(&sc->f.p_at, i);
        reached = true;
      }
      if (!below && w < least) {
        atomicMin(&sc->f.m_at, i);
        below = true;
      }
      mb += c * w;
    }
  }
  __syncthreads();

  // The last entry kept (the first entry's weight is 1, so m_at > 0).
  const uint32_t p_at = sc->f.p_at, m_at = sc->f.m_at;
  uint32_t f_at = by_p && p_at < k_at ? p_at : k_at;
  const bool cut_by_p = by_p && p_at <= k_at;
  const bool cut_by_m = m_at <= f_at;
  if (cut_by_m) f_at = m_at - 1;
  if (i0 <= f_at && f_at < i1) {
    double mb = m_before;
    uint32_t c;
    double w;
    for (uint32_t i = i0; i < f_at; ++i) {
      entry(i, &c, &w);
      mb += c * w;
    }
    entry(f_at, &c, &w);
    const uint32_t most = f_at == k_at ? k_rank : c;
    const uint32_t rank = cut_by_p && !cut_by_m ? rank_of<false>(mb, w, most, p_target) : most;
    sc->f.f_rank = rank;
    sc->f.z = mb + rank * w;
  }
  __syncthreads();

  // The draw.
  const uint32_t f_rank = sc->f.f_rank;
  const double z = sc->f.z, target = u > 0.0f ? (double)u * z : 0.0;
  {
    double mb = m_before;
    for (uint32_t i = i0; i < i1 && i <= f_at; ++i) {
      uint32_t c;
      double w;
      entry(i, &c, &w);
      if (mb + (i == f_at ? f_rank : c) * w > target) {
        atomicMin(&sc->f.d_first, i);
        break;
      }
      mb += c * w;
    }
  }
  __syncthreads();
  const bool past = sc->f.d_first == kNone;
  const uint32_t d_at = past ? f_at : sc->f.d_first;
  if (i0 <= d_at && d_at < i1) {
    double mb = m_before;
    uint32_t c;
    double w;
    for (uint32_t i = i0; i < d_at; ++i) {
      entry(i, &c, &w);
      mb += c * w;
    }
    entry(d_at, &c, &w);
    const uint32_t most = d_at == f_at ? f_rank : c;
    sc->f.d_rank = (past ? most : rank_of<true>(mb, w, most, target)) - 1;
    sc->f.prob = (float)(w / z);
    sc->f.d_at = d_at;
  }
  __syncthreads();
}

// Column of the rank-th element (from 0) of `bin` in a slice, kNone (to every
// thread) if it holds no more than rank; *held becomes how many it holds.
__device__ uint32_t locate(const Slice &s, uint32_t bin, uint32_t rank, uint32_t *held, uint32_t *totals,
                           uint32_t *place) {
  constexpr int kRounds = kSliceCols / 8 / kThreads;
  const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  const v4u *vp = reinterpret_cast<const v4u *>(s.ptr);
  const uint32_t n_vec = s.cols / 8, n_all = (s.cols + 7) / 8;
  uint32_t match[kRounds];  // bit e: element e of this thread's vector is of the bin
  if (tid == 0) place[0] = kNone;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const uint32_t v = r * kThreads + tid;
    match[r] = 0;
    if (v < n_vec) {
      const v4u w = vp[v];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        match[r] |= (bin_of(w[i] & 0xFFFFu) == bin) << (2 * i);
        match[r] |= (bin_of(w[i] >> 16) == bin) << (2 * i + 1);
      }
    } else if (v < n_all) {
      for (uint32_t e = 0; e < s.cols % 8; ++e) match[r] |= (bin_of(s.ptr[v * 8 + e]) == bin) << e;
    }
    uint32_t c = __popc(match[r]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) c += __shfl_xor(c, d);
    if (lane == 0) totals[r * kWaves + wave] = c;
  }
  __syncthreads();
  if (wave == 0) {
    static_assert(kRounds * kWaves == 64, "one lane for each round of a wave");
    const uint32_t c = totals[lane];
    uint32_t incl = c;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t x = __shfl_up(incl, d);
      if ((int)lane >= d) incl += x;
    }
    if (incl - c <= rank && rank < incl) {
      place[0] = lane;
      place[1] = rank - (incl - c);
    }
    if (lane == 63) place[2] = incl;
  }
  __syncthreads();
  *held = place[2];
  const uint32_t at = place[0];
  if (at == kNone) return kNone;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (at != r * kWaves + wave) continue;
    const uint32_t c = __popc(match[r]);
    uint32_t incl = c;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t x = __shfl_up(incl, d);
      if ((int)lane >= d) incl += x;
    }
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
  const uint32_t *lists, *lengths;  // per slice (two launches)
  uint2 *merged;                    // a row's list: (bin, count)
  uint64_t row_cap, merged_cap;
  uint32_t n_slices;
};

// ONE: the row is counted here (both shards hold at most kSliceCols columns
// together); else its slices' lists are added up.
template <bool ONE>
__global__ __launch_bounds__(kThreads) void sample_draw_kernel(DrawArgs a) {
  __shared__ __attribute__((aligned(16))) uint32_t lds[kHalf];
  __shared__ uint32_t totals[64];
  __shared__ Scratch sc;
  const uint32_t row = blockIdx.x, tid = threadIdx.x;
  uint2 *merged = a.merged + row * a.merged_cap;
  auto emit = [&](uint32_t i, uint32_t bin, uint32_t count) { merged[i] = make_uint2(bin, count); };

  uint32_t n;
  if (ONE) {
    clear(lds, kHalf);
    __syncthreads();
    for (uint32_t k = 0; k < 2; ++k) count_slice(lds, slice_of(a.sh, row, k));
    __syncthreads();
    n = compact<true>(lds, kHalf, 0, 0, totals, emit);
  } else {
    n = 0;
#pragma unroll 1
    for (uint32_t half = 0; half < 2; ++half) {
      clear(lds, kHalf);
      __syncthreads();
      uint64_t at = row * a.row_cap;
      for (uint32_t k = 0; k < a.n_slices; ++k) {
        const uint32_t len = a.lengths[row * a.n_slices + k];
        for (uint32_t i = tid; i < len; i += kThreads) {
          const uint32_t e = a.lists[at + i], b = (e >> 16) - half * kHalf;
          if (b < kHalf) atomicAdd(&lds[b], e & 0xFFFFu);
        }
        at += a.sh.width[k >= a.sh.slices[0]];
      }
      __syncthreads();
      n += compact<false>(lds, kHalf, half * kHalf, n, totals, emit);
    }
  }
  if (n == 0) {
    if (tid == 0) a.out[row] = xfer_sampled{0.0f, -1};
    return;
  }

  const xfer_sample_params p = a.params[row];
  const float u = a.u[row];
  const double t = p.temperature > 0.0f ? (double)p.temperature : 1.0;
  const double top = value_of(merged[0].x);
  const bool top_inf = isinf(top);
  auto weight = [&](uint32_t i, uint32_t bin) -> double {
    if (i == 0) return 1.0;
    return top_inf ? 0.0 : exp((value_of(bin) - top) / t);
  };
  if (n <= kLdsEntries) {
    double *lw = reinterpret_cast<double *>(lds);
    uint32_t *lc = lds + 2 * kLdsEntries;
    for (uint32_t i = tid; i < n; i += kThreads) {
      const uint2 e = merged[i];
      lw[i] = weight(i, e.x);
      lc[i] = e.y;
    }
    __syncthreads();
    search([&](uint32_t i, uint32_t *c, double *w) { *c = lc[i], *w = lw[i]; }, n, p, u, &sc);
  } else {
    search(
        [&](uint32_t i, uint32_t *c, double *w) {
          const uint2 e = merged[i];
          *c = e.y, *w = weight(i, e.x);
        },
        n, p, u, &sc);
  }

  const uint32_t bin = merged[sc.f.d_at].x;
  uint32_t rank = sc.f.d_rank, k = 0;
  if (!ONE) {
    // How many of the value each slice holds, from the lists.
    for (uint32_t i = tid; i < a.n_slices; i += kThreads) sc.slice_count[i] = 0;
    __syncthreads();
    uint64_t at = row * a.row_cap;
    for (uint32_t s = 0; s < a.n_slices; ++s) {
      const uint32_t len = a.lengths[row * a.n_slices + s];
      for (uint32_t i = tid; i < len; i += kThreads) {
        const uint32_t e = a.lists[at + i];
        if (e >> 16 == bin) sc.slice_count[s] = e & 0xFFFFu;
      }
      at += a.sh.width[s >= a.sh.slices[0]];
    }
    __syncthreads();
    while (k + 1 < a.n_slices && rank >= sc.slice_count[k]) rank -= sc.slice_count[k++];
  }
  uint32_t held;
  Slice s = slice_of(a.sh, row, k);
  uint32_t col = locate(s, bin, rank, &held, totals, sc.place);
  if (ONE && col == kNone) {
    __syncthreads();  // place is written again
    s = slice_of(a.sh, row, 1);
    col = locate(s, bin, rank - held, &held, totals, sc.place);
  }
  if (tid == 0) a.out[row] = xfer_sampled{sc.f.prob, (int32_t)(s.gid + col)};
}

uint32_t round_up8(uint32_t x) { return (x + 7u) & ~7u; }

struct Sizes {
  bool one;
  uint32_t slices[2], width[2];
  uint64_t row_cap, merged_cap;
};
Sizes sizes_of(uint32_t ncols0, uint32_t ncols1) {
  Sizes z{};
  z.one = (uint64_t)ncols0 + ncols1 <= kSliceCols;
  const uint32_t n[2] = {ncols0, ncols1};
  for (int i = 0; i < 2; ++i) {
    z.slices[i] = (n[i] + kSliceCols - 1) / kSliceCols;
    z.width[i] = round_up8((n[i] + z.slices[i] - 1) / z.slices[i]);
    z.row_cap += (uint64_t)z.slices[i] * z.width[i];
  }
  z.merged_cap = z.row_cap < kBins ? z.row_cap : kBins;
  if (z.one) z.row_cap = 0;
  return z;
}
uint64_t up16(uint64_t x) { return (x + 15) / 16 * 16; }

}  // namespace

uint32_t sample_slices(uint32_t ncols0, uint32_t ncols1) {
  const Sizes z = sizes_of(ncols0, ncols1);
  return z.one ? 1 : z.slices[0] + z.slices[1];
}

// Layout: the rows' merged lists, the slices' lengths, the slices' lists.
uint64_t sample_workspace_bytes(uint32_t rows, uint32_t ncols0, uint32_t ncols1) {
  const Sizes z = sizes_of(ncols0, ncols1);
  uint64_t n = rows * z.merged_cap * 8;
  if (!z.one) n += up16((uint64_t)rows * (z.slices[0] + z.slices[1]) * 4) + rows * z.row_cap * 4;
  return up16(n);
}

hipError_t launch_sample(const SampleArgs &in, hipStream_t stream) {
  // the shard with the lower ids first
  const int order[2] = {in.s[0].col_offset < in.s[1].col_offset ? 0 : 1, in.s[0].col_offset < in.s[1].col_offset ? 1 : 0};
  const Sizes z = sizes_of(in.s[order[0]].ncols, in.s[order[1]].ncols);
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
  uint32_t *lengths = reinterpret_cast<uint32_t *>(ws + (uint64_t)in.rows * z.merged_cap * 8);
  uint32_t *lists = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(lengths) + up16((uint64_t)in.rows * a.n_slices * 4));
  a.lengths = lengths;
  a.lists = lists;
  const hipError_t e = launch(sample_count_kernel, dim3(in.rows * a.n_slices), dim3(kThreads), 0, stream, a.sh,
                              a.n_slices, a.row_cap, lists, lengths);
  if (e != hipSuccess) return e;
  return launch(sample_draw_kernel<false>, dim3(in.rows), dim3(kThreads), 0, stream, a);
}

}  // namespace xfer
