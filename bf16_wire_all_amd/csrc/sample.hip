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
//      value; a slice has at most 40,960 columns) and writes the values that
//      occur, in order, with their counts;
//   2. draw: a workgroup for each row adds up its slices' lists in LDS the
//      same way, finds the cuts and the drawn element (its value and how many
//      equal ones come before it), then looks that one up in the slice that
//      holds it.
// Rows of at most 32,768 columns in all take one launch, which counts both
// shards in one workgroup.
// The kernel boundary orders the two steps, as in the argmax.
//
// A workgroup holds its slice in registers, so that all its loads are in
// flight at once and nothing is read twice (256 rows of 151,936: the count is
// 22 us, 3.5 TB/s; with pieces of 16,384 columns one after the other, read
// again to be counted, it was 27).  The slice's range of magnitudes is found
// before it is counted, and 8,192 bins (64 powers of two, both signs' counts
// in one word) hold it in 32 KiB of LDS: two workgroups share a compute unit,
// and clearing and reading the bins costs little.  Ranges that are wider, and
// sums of counts past 16 bits, take a path of eight passes.
//
// What a row's settings leave out whatever the other slices hold is not
// counted: where top_p does not ask for the sum of all weights, what min_p
// would drop beside the slice's own first element; and what lies below top_k
// elements that the slice is known to have.  That needs a largest value above
// zero: slices all below it are counted whole.  The list then has a few entries,
// and up to 64 of a row are searched by one wave in its registers (rows of
// 129,280 with all filters: the draw is 8.9 us, with whole lists it was 14.1).
//
// What bounds the rest, at one row as at 256, is the chain of steps in a
// workgroup, each some hundreds of clocks: a load, a barrier, a search.  So the
// order is made once, when the bins are read, one wave does the searches, 64
// probes at a time, without barriers between them, and loops of rare cases are
// left as loops, for a workgroup runs through most of the code once and waits
// for it to be fetched.
#include "decode.h"

namespace xfer {
namespace {

constexpr uint32_t kInf = 0x7F80u;               // the pattern of +inf; -inf has the sign bit too
// Values in the row's order, +inf first: positive patterns count down, zero
// (of either sign) is bin kInf, negative ones count up.
constexpr uint32_t kBins = 2 * kInf;
constexpr uint32_t kWords = 8192;                // bins in LDS: +count in the low half, -count in the high
constexpr uint32_t kNone = 0xFFFFFFFFu;
// Columns of a slice, which a workgroup holds in registers: as few as the first
// where that gives compute units work that would have none, up to the second.
constexpr uint32_t kSliceCols = 16384, kWideSliceCols = 40960;
constexpr uint32_t kOneCols = 32768;             // of a row that one launch counts
constexpr uint32_t kMaxSlices = 128;
constexpr uint32_t kComputeUnits = 256;
constexpr uint32_t kCountWorkgroups = 2 * kComputeUnits;

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned short v2us __attribute__((ext_vector_type(2)));
typedef short v2s __attribute__((ext_vector_type(2)));

// The BF16 pattern of a bin (+0 for zero).
__device__ __forceinline__ uint32_t pattern_of(uint32_t bin) {
  return bin <= kInf ? kInf - bin : 0x8000u | (bin - kInf);
}
__device__ __forceinline__ double value_of(uint32_t bin) { return (double)__uint_as_float(pattern_of(bin) << 16); }
// The bin of a pattern that counts.
__device__ __forceinline__ uint32_t bin_of(uint32_t v) {
  const uint32_t mag = v & 0x7FFFu;
  return v & 0x8000u ? kInf + mag : kInf - mag;
}
// Whether a pattern counts: neither NaN nor -inf.
__device__ __forceinline__ bool counts(uint32_t v) { return (v & 0x7FFFu) <= kInf && v != 0xFF80u; }

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

__device__ __forceinline__ uint32_t lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}
__device__ __forceinline__ uint32_t wave_number() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

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


// What the count leaves of a slice besides its list (bin << 16 | count):
// entries, the largest count, and the span of magnitudes.
struct SliceInfo {
  uint32_t length, most, lo, hi;
};

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

// A workgroup of kThreads: 16 waves where a compute unit has one workgroup to
// run, 8 where it has more and two share it.
template <int kThreads>
struct Team {
static constexpr int kWaves = kThreads / 64;
static constexpr uint32_t kLdsEntries = kThreads == 512 ? 5888 : 8192;  // lists up to this long stay in LDS

// ------------------------------------------------------ a slice in registers

// Elements of N parts, each from a round of vectors of its own on; all loads in
// flight at once.  What lies past a part's end is -inf, which counts nowhere.
static constexpr uint32_t kMasked = 0xFF80FF80u;
static constexpr uint32_t kRounds = kWideSliceCols / 8 / kThreads;
// The first round of the second part (kOneCols in two parts never take more
// than kRounds).
__device__ __forceinline__ static uint32_t second_round(const Slice &first) {
  return (first.cols + 8 * kThreads - 1) / (8 * kThreads);
}
struct Held {
  v4u w[kRounds];
  uint32_t own;   // bit r: this wave has vectors of round r
  uint32_t busy;  // waves that have any

  template <int N>
  __device__ __forceinline__ void load(const Slice (&part)[N]) {
    const uint32_t tid = threadIdx.x, wave = wave_number(), r1 = N == 2 ? second_round(part[0]) : kRounds;
    own = 0;
#pragma unroll
    for (uint32_t r = 0; r < kRounds; ++r) {
      const bool second = N == 2 && r >= r1;
      const Slice &s = part[second ? N - 1 : 0];
      const uint32_t v0 = (second ? r - r1 : r) * kThreads;
      w[r] = v4u{kMasked, kMasked, kMasked, kMasked};
      if (v0 + tid < s.cols / 8) w[r] = reinterpret_cast<const v4u *>(s.ptr)[v0 + tid];
      own |= (v0 + wave * 64 < (s.cols + 7) / 8 ? 1u : 0u) << r;
    }
    busy = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const Slice &s = part[i];
      busy = max(busy, min((uint32_t)kWaves, (s.cols + 511) / 512));
      // an incomplete last vector, element by element
      const uint32_t last = s.cols / 8, rest = s.cols % 8;
      if (rest && tid == last % kThreads) {
        v4u x{kMasked, kMasked, kMasked, kMasked};
#pragma unroll
        for (uint32_t e = 0; e < 7; ++e)
          if (e < rest) {
            const uint32_t v = s.ptr[last * 8 + e];
            x[e / 2] = e % 2 ? (x[e / 2] & 0xFFFFu) | v << 16 : (x[e / 2] & 0xFFFF0000u) | v;
          }
#pragma unroll
        for (uint32_t r = 0; r < kRounds; ++r)
          w[r] ^= (w[r] ^ x) & (r == (i ? r1 : 0) + last / kThreads ? ~0u : 0u);
      }
    }
  }
  // visit(round, vector) of this wave's vectors.
  template <typename Visit>
  __device__ __forceinline__ void each(const Visit &visit) const {
#pragma unroll
    for (uint32_t r = 0; r < kRounds; ++r)
      if (own >> r & 1) visit(r, w[r]);
  }
  // The vector of a round that is known at run time.
  __device__ __forceinline__ v4u of_round(uint32_t round) const {
    // by masks: the compiler would index memory for a choice
    v4u x{};
#pragma unroll
    for (uint32_t r = 0; r < kRounds; ++r) x |= w[r] & (r == round ? ~0u : 0u);
    return x;
  }
  // one(element) of every element: a loop, to keep the code of rare cases short.
  template <typename One>
  __device__ __forceinline__ void each_one(const One &one) const {
#pragma unroll 1
    for (uint32_t r = 0; r < kRounds; ++r) {
      if (!(own >> r & 1)) continue;
      const v4u x = of_round(r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        one(x[i] & 0xFFFFu);
        one(x[i] >> 16);
      }
    }
  }
};

// Magnitudes from lo to hi (hi 0: none), zero left out; the largest pattern
// above zero (0: none); a pattern above zero that enough elements reach (0:
// none known).
struct Span {
  uint32_t lo, hi, top, reached;
};
// This lane's span; whether the wave has a zero or +inf (or a NaN that would
// pass for it).
__device__ __forceinline__ static bool span_of(const Held &h, Span *s) {
  v2us low = {0xFFFF, 0xFFFF}, high = {0, 0};
  v2s first = {0, 0};
  h.each([&](uint32_t, const v4u &x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v2us m = __builtin_bit_cast(v2us, x[i] & 0x7FFF7FFFu);
      low = __builtin_elementwise_min(low, m);
      // finite magnitudes wrap round to 0x8080 and more, others to less
      high = __builtin_elementwise_max(high, m - (unsigned short)kInf);
      first = __builtin_elementwise_max(first, __builtin_bit_cast(v2s, (uint32_t)x[i]));
    }
  });
  const uint32_t l = min((uint32_t)low.x, (uint32_t)low.y), t = max((uint32_t)high.x, (uint32_t)high.y);
  const uint32_t f = (uint32_t)max((int)first.x, (int)first.y);
  *s = Span{kNone, 0, 0, 0};
  if (!__any(l == 0 || f >= kInf)) {
    if (t >= 0x10000u - kInf) *s = Span{l, t + kInf - 0x10000u, f, 0};
    return false;
  }
  h.each_one([&](uint32_t v) {
    const uint32_t m = v & 0x7FFFu;
    if (counts(v) && m) {
      s->lo = min(s->lo, m);
      s->hi = max(s->hi, m);
      if (v == m) s->top = max(s->top, m);
    }
  });
  return true;
}

// ------------------------------------------------------------------ counting

// The words behind the bins, one for each lane, take what does not count.
struct Bins {
  uint32_t word[kWords + 64];
};

__device__ __forceinline__ static void clear(Bins *bins) {
  v4u *p = reinterpret_cast<v4u *>(bins->word);
#pragma unroll
  for (uint32_t i = 0; i < kWords / 4 / kThreads; ++i) p[i * kThreads + threadIdx.x] = v4u{0, 0, 0, 0};
}

// Counts a wave's elements in the bins of magnitudes base .. base + kWords - 1,
// which have to hold all of them but zero; *zeros takes the zeros.  `careful`
// if there may be zeros or infinite ones.
__device__ __forceinline__ static void count_all(Bins *bins, const Held &h, bool careful, uint32_t base, uint32_t *zeros) {
  uint32_t *word = bins->word;
  if (!careful) {
    // NaN and -inf lie past the bins' last magnitude
    const uint32_t none = kWords + threadIdx.x % 64;
    h.each([&](uint32_t, const v4u &x) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        atomicAdd(&word[min((x[i] & 0x7FFFu) - base, none)], (x[i] >> 15 & 1u) * 0xFFFFu + 1u);
        atomicAdd(&word[min((x[i] >> 16 & 0x7FFFu) - base, none)], (x[i] >> 31) * 0xFFFFu + 1u);
      }
    });
    return;
  }
  uint32_t n = 0;
  h.each_one([&](uint32_t v) {
    const uint32_t m = v & 0x7FFFu;
    n += m == 0;
    // a mask's elements would all wait for one address
    if (counts(v) && m) atomicAdd(&word[m - base], (v >> 15) * 0xFFFFu + 1u);
  });
  n = read_lane(scan(n), 63);
  if (n && threadIdx.x % 64 == 0) atomicAdd(zeros, n);
}

// The same of the elements from pattern lo (above zero) to hi, in the bins from
// lo on.
__device__ __forceinline__ static void count_top(Bins *bins, const Held &h, uint32_t lo, uint32_t hi) {
  uint32_t *word = bins->word;
  auto one = [&](int v) {
    if ((uint32_t)v - lo <= hi - lo) atomicAdd(&word[(uint32_t)v - lo], 1u);
  };
  h.each([&](uint32_t, const v4u &x) {
    v2s m = __builtin_bit_cast(v2s, (uint32_t)x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(v2s, (uint32_t)x[i]));
    if (!__any(max((int)m.x, (int)m.y) >= (int)lo)) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      one((int)(x[i] << 16) >> 16);
      one((int)x[i] >> 16);
    }
  });
}

// The entries of the bins, in order.  The words go in groups of 256, a lane
// four in a row, group after group round the waves; the constructor returns
// once every group's numbers are known.
static constexpr int kGroups = kWords / 256;
struct GroupCounts {
  uint32_t pos[kGroups], neg[kGroups];
};
struct Compact {
  static constexpr int kOwn = kGroups / kWaves;  // groups of a wave
  v4u x[kOwn];
  uint32_t zeros, pos_total, total;  // elements that are zero; entries above zero, and in all
  uint32_t pos_incl, neg_incl;       // of lane l: running numbers up to group l

  // visit(group, words) of this wave's groups that are not empty.
  template <typename Visit>
  __device__ __forceinline__ void each(const Visit &visit) const {
    v4u y[kOwn];
#pragma unroll
    for (int r = 0; r < kOwn; ++r) y[r] = x[r];
#pragma unroll 1
    for (uint32_t r = 0; r < kOwn; ++r) {
      if (__any((y[0].x | y[0].y | y[0].z | y[0].w) != 0)) visit(r * kWaves + wave_number(), y[0]);
#pragma unroll
      for (int i = 1; i < kOwn; ++i) y[i - 1] = y[i];
    }
  }

  __device__ __forceinline__ Compact(const Bins *bins, uint32_t n_zeros, GroupCounts *groups) {
    const uint32_t lane = threadIdx.x % 64;
    const v4u *words = reinterpret_cast<const v4u *>(bins->word);
#pragma unroll
    for (int r = 0; r < kOwn; ++r) x[r] = words[(r * kWaves + wave_number()) * 64 + lane];
    if (lane < kOwn) groups->pos[lane * kWaves + wave_number()] = groups->neg[lane * kWaves + wave_number()] = 0;
    each([&](uint32_t g, const v4u &y) {
      uint32_t p = 0, n = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p += __popcll(__ballot((y[i] & 0xFFFFu) != 0));
        n += __popcll(__ballot(y[i] >> 16 != 0));
      }
      if (lane == 0) {
        groups->pos[g] = p;
        groups->neg[g] = n;
      }
    });
    lds_barrier();
    static_assert(kGroups <= 64, "a lane for each group");
    pos_incl = scan(lane < kGroups ? groups->pos[lane % kGroups] : 0);
    neg_incl = scan(lane < kGroups ? groups->neg[lane % kGroups] : 0);
    zeros = n_zeros;
    pos_total = read_lane(pos_incl, 63);
    total = pos_total + (zeros != 0) + read_lane(neg_incl, 63);
  }

  // out(index, bin, count) for each; word 0 stands for magnitude `base`.
  template <typename Emit>
  __device__ __forceinline__ void emit(uint32_t base, const Emit &out) const {
    const uint32_t lane = threadIdx.x % 64;
    if (zeros && threadIdx.x == 0) out(pos_total, kInf, zeros);
    each([&](uint32_t g, const v4u &y) {
      const uint32_t mag0 = base + g * 256 + lane * 4;
      uint32_t p_below = 0, p_own = 0, p_all = 0, n_below = 0, n_all = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool own = (y[i] & 0xFFFFu) != 0;
        const uint64_t a = __ballot(own);
        p_below += lanes_below(a);
        p_own += own;
        p_all += __popcll(a);
        const uint64_t b = __ballot(y[i] >> 16 != 0);
        n_below += lanes_below(b);
        n_all += __popcll(b);
      }
      // above zero the order goes down the magnitudes: later groups, later
      // lanes and a lane's later words come first
      uint32_t at = pos_total - read_lane(pos_incl, g) + (p_all - p_below - p_own);
#pragma unroll
      for (int i = 3; i >= 0; --i)
        if (const uint32_t c = y[i] & 0xFFFFu) out(at++, kInf - (mag0 + i), c);
      at = pos_total + (zeros != 0) + read_lane(neg_incl, g) - n_all + n_below;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (const uint32_t c = y[i] >> 16) out(at++, kInf + mag0 + i, c);
    });
  }
};

// The list of any elements, kWords bins at a time with 32 bits for each:
// count(first bin) adds up those from that one on in bins->word, and
// out(index, bin, count) gets the entries.  Returns their number, after a barrier.
template <typename Count, typename Emit>
__device__ __forceinline__ static uint32_t list_in_passes(Bins *bins, uint32_t *scratch, const Count &count, const Emit &out) {
  constexpr uint32_t kRun = kWords / kWaves;
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  uint32_t n = 0;
#pragma unroll 1
  for (uint32_t bin0 = 0; bin0 < kBins; bin0 += kWords) {
    clear(bins);
    lds_barrier();
    count(bin0);
    lds_barrier();
    uint32_t mine = 0;
    for (uint32_t w = wave * kRun + lane; w < (wave + 1) * kRun; w += 64) mine += __popcll(__ballot(bins->word[w] != 0));
    if (lane == 0) scratch[wave] = mine;
    lds_barrier();
    uint32_t next = n;
    for (uint32_t i = 0; i < kWaves; ++i) {
      if (i < wave) next += scratch[i];
      n += scratch[i];
    }
    for (uint32_t w = wave * kRun + lane; w < (wave + 1) * kRun; w += 64) {
      const uint32_t c = bins->word[w];
      const uint64_t b = __ballot(c != 0);
      if (c) out(next + lanes_below(b), bin0 + w, c);
      next += __popcll(b);
    }
    __syncthreads();
  }
  return n;
}
__device__ __forceinline__ static void count_pass(Bins *bins, const Held &h, uint32_t bin0) {
  h.each_one([&](uint32_t v) {
    const uint32_t b = bin_of(v) - bin0;
    if (counts(v) && b < kWords) atomicAdd(&bins->word[b], 1u);
  });
}

// The waves' spans, and the elements that are zero.
struct Spans {
  uint32_t lo[kWaves], hi[kWaves], top[kWaves], reached[kWaves], zeros;
};
// This wave's span for the others, before a barrier; from all lanes' spans.
// With enough > 0 also the largest pattern that the tops of `enough` lanes
// reach.
__device__ __forceinline__ static void share_span(Spans *s, const Span &mine, uint32_t enough) {
  const uint32_t hi = wave_max(mine.hi), lo = ~wave_max(~mine.lo), top = wave_max(mine.top);
  uint32_t reached = 0;
  if (enough) {
#pragma unroll 1
    for (uint32_t bit = 1u << 14; bit; bit >>= 1)
      if (__popcll(__ballot(mine.top >= (reached | bit))) >= enough) reached |= bit;
  }
  if (threadIdx.x % 64 == 0) {
    s->lo[wave_number()] = lo;
    s->hi[wave_number()] = hi;
    s->top[wave_number()] = top;
    s->reached[wave_number()] = reached;
  }
  if (threadIdx.x == 0) s->zeros = 0;
}
// All waves' together; `reached` of the first `busy` ones.
__device__ __forceinline__ static Span join_spans(const Spans &s, uint32_t busy) {
  const uint32_t lane = threadIdx.x % 64, w = lane % kWaves;
  const uint32_t lo = s.lo[w], hi = s.hi[w], top = s.top[w], reached = w < busy ? s.reached[w] : kNone;
  return {~wave_max(~lo), wave_max(hi), wave_max(top), ~wave_max(~reached)};
}
// The lowest magnitude, not zero, of kWords bins that reach hi.
__device__ __forceinline__ static uint32_t base_of(uint32_t hi) { return hi - min(hi, kWords) + 1; }
__device__ __forceinline__ static bool fits(const Span &s) { return s.hi - min(s.lo, s.hi) < kWords; }

// How many elements of a row matter: top_k, or one to a greedy row.
__device__ __forceinline__ static uint32_t keep_of(const xfer_sample_params &p) {
  return !(p.temperature > 0.0f) ? 1 : p.top_k == 0 ? kNone : p.top_k;
}
// A pattern above zero below which nothing that min_p keeps lies, `top` being
// the largest; 0 if there is none, or where top_p asks for every weight.
__device__ __forceinline__ static uint32_t min_p_cut(const xfer_sample_params &p, uint32_t top) {
  if (!(p.temperature > 0.0f) || p.top_p < 1.0f || !(p.min_p > 0.0f)) return 0;
  const float x = __uint_as_float(top << 16);
  // lowered by more than binary32 loses here, and by what an exponential in
  // binary64 still rounds to 1; the pattern is cut off downwards
  const float exponent = logf(fminf(p.min_p, 1.0f)) * (1.0f + 0x1p-18f) - 0x1p-40f;
  const float least = x * (1.0f - 0x1p-18f) + p.temperature * exponent;
  return least > 0.0f ? __float_as_uint(least) >> 16 : 0;
}

// The span of a slice, and then its counts in bins from magnitude *base on.
// Elements that the row's settings leave out, whatever other slices hold, are
// not counted: those below what min_p leaves of the slice's first, and with at
// most `keep` wanted those below a pattern that the tops of as many lanes
// reach.  True if the bins hold the counts, after a barrier; false if the span
// is too wide.
__device__ __forceinline__ static bool count_slice(Bins *bins, Spans *spans, const Held &h, const xfer_sample_params &p,
                                            Span *all, uint32_t *base) {
  clear(bins);
  Span mine;
  const bool careful = span_of(h, &mine);
  const uint32_t keep = keep_of(p);
  const uint32_t enough = keep > 1 && keep <= h.busy * 64 ? (keep + h.busy - 1) / h.busy : 0;
  share_span(spans, mine, enough);
  lds_barrier();
  *all = join_spans(*spans, h.busy);
  uint32_t cut = 0;
  if (all->top) {
    cut = max(min_p_cut(p, all->top), all->reached);
    if (keep == 1) cut = all->top;
  }
  if (cut) {
    all->lo = cut;
    all->hi = all->top;
  }
  if (!fits(*all)) return false;
  *base = cut ? cut : base_of(all->hi);
  if (cut)
    count_top(bins, h, cut, all->top);
  else
    count_all(bins, h, careful || all->hi == kInf, *base, &spans->zeros);
  lds_barrier();
  return true;
}

// A workgroup goes from slice to slice, and loads the next one before it sorts
// out the counts of the one at hand.
__device__ __forceinline__ static void count(const Shards &sh, uint32_t n_slices, uint32_t jobs, uint64_t row_cap,
                                      const xfer_sample_params *params, uint32_t *lists, SliceInfo *infos) {
  __shared__ __attribute__((aligned(16))) Bins bins;
  __shared__ GroupCounts groups;
  __shared__ Spans spans;
  __shared__ uint32_t most[kWaves];
  const uint32_t lane = threadIdx.x % 64;
  Held held;
  auto load = [&](uint32_t job) {
    const Slice part[1] = {slice_of(sh, job / n_slices, job % n_slices)};
    held.load(part);
  };
  uint32_t job = blockIdx.x;
  load(job);
#pragma unroll 1
  for (; job < jobs; job += gridDim.x) {
    const uint32_t row = job / n_slices, k = job % n_slices, s = k >= sh.slices[0], next = job + gridDim.x;
    const xfer_sample_params p = params[row];
    const uint32_t keep = keep_of(p);  // as many entries are enough
    Span all;
    uint32_t base = 0;
    const bool fit = count_slice(&bins, &spans, held, p, &all, &base);
    uint32_t *list = lists + row * row_cap + (s ? (uint64_t)sh.slices[0] * sh.width[0] : 0) +
                     (uint64_t)(s ? k - sh.slices[0] : k) * sh.width[s];
    uint32_t largest = 0, n;
    auto put = [&](uint32_t i, uint32_t bin, uint32_t count) {
      if (i < keep) list[i] = bin << 16 | count;
      largest = max(largest, count);
    };
    if (!fit) {
      lds_barrier();  // the bins are cleared again
      n = list_in_passes(&bins, groups.pos, [&](uint32_t bin0) { count_pass(&bins, held, bin0); }, put);
    }
    if (next < jobs) load(next);
    if (fit) {
      Compact c(&bins, spans.zeros, &groups);
      c.emit(base, put);
      n = c.total;
    }
    largest = wave_max(largest);
    if (lane == 0) most[wave_number()] = largest;
    lds_barrier();  // bins, groups and spans are written again
    if (threadIdx.x == 0) {
#pragma unroll
      for (int w = 1; w < kWaves; ++w) largest = max(largest, most[w]);
      infos[job] = SliceInfo{min(n, keep), largest, all.lo, all.hi};
    }
  }
}

// ----------------------------------------------------------------- searching

struct Scratch {
  SliceInfo info[kMaxSlices];
  uint32_t slice_count[kMaxSlices];
  double mass[kWaves];
  uint32_t count[kWaves];
  uint32_t below[kWaves];  // a wave's first entry whose weight is below min_p's limit
  uint32_t at, rank;       // the drawn entry, and the drawn element's place among its equals
  float prob;
};

// The smallest weight that min_p keeps.
__device__ __forceinline__ static double least_of(const xfer_sample_params &p) {
  return p.min_p > 1.0f ? 1.0 : (double)p.min_p;
}

// Smallest r in [1, most] with before + r * w >= target (over: > target), or
// most.
__device__ __forceinline__ static uint32_t rank_of(double before, double w, uint32_t most, double target, bool over) {
  const double q = (target - before) / w;
  const uint32_t r = q > 1.0 ? (q < (double)most ? (uint32_t)q : most) : 1;
  // the quotient is off by one step at most: a lane for each number about it
  const uint32_t k = min(max(r, 2u) - 1 + threadIdx.x % 4, most);
  const double c = before + k * w;
  const uint64_t reached = __ballot(over ? c > target : c >= target) & 0xF;
  return reached ? read_lane(k, (uint32_t)__builtin_ctzll(reached)) : most;
}

// The cuts and the draw on a list of up to 64 entries by one wave, an entry
// (count, weight) to each lane; `keep` elements are left by top_k.
__device__ __forceinline__ static void search_in_wave(uint32_t count, double weight, uint32_t n, uint32_t keep,
                                               const xfer_sample_params &p, float u, Scratch *sc) {
  const uint32_t lane = threadIdx.x % 64;
  const bool there = lane < n;
  const uint32_t n_run = scan(there ? count : 0);
  const double m_run = scan(there ? count * weight : 0.0);
  const uint64_t below = __ballot(there && weight < least_of(p));
  struct {
    uint32_t at, rank;
    double z;  // weights up to there
  } f = {n - 1, kNone, read_lane(m_run, 63)};
#pragma unroll 1
  for (int border = keep < read_lane(n_run, 63) ? 0 : 1; border < 4; ++border) {  // as in search() below
    double target = 0;
    uint32_t last = f.at, last_count = f.rank;
    if (border == 1) {
      if (!(p.top_p < 1.0f)) continue;
      target = (double)p.top_p * f.z;
    } else if (border == 2) {
      const uint32_t m_at = below ? (uint32_t)__builtin_ctzll(below) : kNone;
      if (m_at > f.at) continue;
      last = m_at - 1;
      last_count = kNone;
    } else if (border == 3) {
      target = u > 0.0f ? (double)u * f.z : 0.0;
    }
    const uint64_t hit = __ballot(there && (border == 0   ? n_run >= keep
                                            : border == 1 ? m_run >= target
                                                          : border == 3 && m_run > target));
    const uint32_t at = min(hit ? (uint32_t)__builtin_ctzll(hit) : last, last);
    const uint32_t c_all = read_lane(count, at), c = at == last ? min(c_all, last_count) : c_all;
    const double w = read_lane(weight, at), before = at ? read_lane(m_run, at - 1) : 0.0, end = before + c * w;
    const bool reached = at < last || (border == 1 ? end >= target : end > target);
    uint32_t rank = c;
    if (border == 0)
      rank = keep - (read_lane(n_run, at) - c_all);
    else if (border == 1 && !reached)
      continue;  // no cut
    else if (border != 2 && reached)
      rank = rank_of(before, w, c, target, border == 3);
    if (border == 3) {
      if (lane == 0) {
        sc->at = at;
        sc->rank = rank - 1;
        sc->prob = (float)(w / f.z);
      }
    } else {
      f.at = at;
      f.rank = rank;
      f.z = before + rank * w;
    }
  }
}

// The cuts and the draw on a list of n > 0 entries: first(i, &count, &weight)
// once for each entry, then entry(i, &count, &weight); `keep` elements are left
// by top_k.  Thread t sums up entries [t * per, (t + 1) * per); `masses` and
// `counts` (LDS, one for each thread) become the running sums of each wave.
// One wave then finds each border: the wave first, then the thread, then the
// entry among its own.
template <typename First, typename Entry>
__device__ __forceinline__ static void search(const First &first, const Entry &entry, uint32_t n, uint32_t keep,
                                       const xfer_sample_params &p, float u, double *masses, uint32_t *counts,
                                       Scratch *sc) {
  const uint32_t tid = threadIdx.x, wave = wave_number(), lane = tid % 64;
  if (n <= 64) {
    if (wave) return;
    uint32_t c = 0;
    double w = 0;
    if (lane < n) first(lane, &c, &w);
    search_in_wave(c, w, n, keep, p, u, sc);
    return;
  }
  const uint32_t per = (n + kThreads - 1) / kThreads;
  const uint32_t i0 = min(tid * per, n), i1 = min(i0 + per, n);
  const double least = least_of(p);
  uint32_t count = 0, below = kNone;
  double mass = 0;
#pragma unroll 1
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
  counts[tid] = count;
  masses[tid] = mass;
  const uint64_t any_below = __ballot(below != kNone);
  if (any_below) below = read_lane(below, (uint32_t)__builtin_ctzll(any_below));
  if (lane == 63) {
    sc->count[wave] = count;
    sc->mass[wave] = mass;
    sc->below[wave] = below;
  }
  __syncthreads();
  if (wave != 0) return;

  // Of lane w: the running sums up to wave w's end, and the first entry whose
  // weight is below min_p's limit.
  const bool is_wave = lane < kWaves;
  const uint32_t wave_counts = scan(is_wave ? sc->count[lane % kWaves] : 0);
  const double wave_masses = scan(is_wave ? sc->mass[lane % kWaves] : 0.0);
  const uint32_t m_at = ~wave_max(~(is_wave ? sc->below[lane % kWaves] : kNone));

  // Four borders, one after the other: the last element that top_k keeps (if
  // it does not keep all), the first that reaches top_p, the last before
  // min_p's limit, and the drawn one.  f is the last entry kept so far, with
  // `rank` of its elements.
  struct {
    uint32_t at, rank;
    double z;  // weights up to there
  } f = {n - 1, kNone, read_lane(wave_masses, 63)};
#pragma unroll 1
  for (int border = keep < read_lane(wave_counts, 63) ? 0 : 1; border < 4; ++border) {
    double target = 0;
    uint32_t t, last = f.at, last_count = f.rank;
    if (border == 1) {
      if (!(p.top_p < 1.0f)) continue;
      target = (double)p.top_p * f.z;
    } else if (border == 2) {
      // the first entry's weight is 1, so an entry below the limit has one before it
      if (m_at > f.at) continue;
      last = m_at - 1;
      last_count = kNone;
    } else if (border == 3) {
      target = u > 0.0f ? (double)u * f.z : 0.0;
    }
    // The wave and the thread whose running sums reach the border.
    auto reached = [&](uint32_t c, double m) {
      return border == 0 ? c >= keep : border == 1 ? m >= target : border == 3 && m > target;
    };
    const uint64_t waves = __ballot(is_wave && reached(wave_counts, wave_masses));
    uint32_t n_base = 0;
    double m_base = 0;
    t = kThreads;
    if (waves) {
      const uint32_t w = (uint32_t)__builtin_ctzll(waves);
      const uint32_t n_wave = w ? read_lane(wave_counts, w - 1) : 0;
      const double m_wave = w ? read_lane(wave_masses, w - 1) : 0.0;
      const uint32_t n_run = counts[w * 64 + lane] + n_wave;
      const double m_run = masses[w * 64 + lane] + m_wave;
      const uint64_t threads = __ballot(reached(n_run, m_run));
      const uint32_t l = threads ? (uint32_t)__builtin_ctzll(threads) : 63;
      t = w * 64 + l;
      n_base = l ? read_lane(n_run, l - 1) : n_wave;
      m_base = l ? read_lane(m_run, l - 1) : m_wave;
    }
    if (t * per > last) {
      if (border == 1) continue;  // all of them are kept
      t = last / per;
      const uint32_t w = t / 64, l = t % 64;
      n_base = (w ? read_lane(wave_counts, w - 1) : 0) + (l ? counts[t - 1] : 0);
      m_base = (w ? read_lane(wave_masses, w - 1) : 0.0) + (l ? masses[t - 1] : 0.0);
    }
    // The entry: the first of the thread's, up to `last` with at most
    // last_count elements, that reaches it, or the last of them.
    uint32_t at = 0, c_at = 0, n_before = 0;
    double before = 0, w_at = 0;
    bool none = true;
#pragma unroll 1
    for (uint32_t c0 = 0; c0 < per && none; c0 += 64) {
      const uint32_t i = t * per + c0 + lane;
      const bool there = c0 + lane < per && i < n && i <= last;
      const uint64_t all = __ballot(there);
      if (!all) break;
      uint32_t c = 0;
      double w = 0;
      if (there) {
        entry(i, &c, &w);
        if (i == last) c = min(c, last_count);
      }
      const uint32_t n_run = scan(c) + n_base;
      const double m_run = scan(c * w) + m_base;
      const uint64_t hit = __ballot(there && reached(n_run, m_run));
      none = !hit;
      const uint32_t l = hit ? (uint32_t)__builtin_ctzll(hit) : 63 - (uint32_t)__builtin_clzll(all);
      at = t * per + c0 + l;
      c_at = read_lane(c, l);
      w_at = read_lane(w, l);
      n_before = read_lane(n_run, l) - c_at;
      before = l ? read_lane(m_run, l - 1) : m_base;
      n_base = read_lane(n_run, 63);
      m_base = read_lane(m_run, 63);
    }
    uint32_t rank = c_at;
    if (border == 0)
      rank = keep - n_before;
    else if (border == 1 && none && at == f.at)
      continue;  // no cut
    else if (border != 2 && !none)
      rank = rank_of(before, w_at, c_at, target, border == 3);
    if (border == 3) {
      if (lane == 0) {
        sc->at = at;
        sc->rank = rank - 1;
        sc->prob = (float)(w_at / f.z);
      }
    } else {
      f.at = at;
      f.rank = rank;
      f.z = before + rank * w_at;
    }
  }
}

// Where the rank-th (from 0) of things lies that are counted in up to 128
// numbers, of which this lane has the 2l-th and the next: the number's index
// (kNone: nowhere), and how many lie before it.
struct Place {
  uint32_t at, before;
};
__device__ __forceinline__ static Place place_of(uint32_t c0, uint32_t c1, uint32_t rank) {
  const uint32_t incl = scan(c0 + c1), excl = incl - c0 - c1;
  const uint64_t holds = __ballot(excl <= rank && rank < incl);
  if (!holds) return {kNone, 0};
  const uint32_t l = (uint32_t)__builtin_ctzll(holds), before = read_lane(excl, l), first = read_lane(c0, l);
  const bool second = rank - before >= first;
  return {2 * l + second, before + (second ? first : 0)};
}

// Calls found(id) in the lane that holds the rank-th element (from 0) of `bin`
// in the parts, which hold one; id is its global one.  `totals` (LDS): a number
// for each round of a wave.
template <int N, typename Found>
__device__ __forceinline__ static void locate(const Held &h, const Slice (&part)[N], uint32_t bin, uint32_t rank,
                                       uint32_t *totals, const Found &found) {
  const uint32_t tid = threadIdx.x, wave = wave_number(), lane = tid % 64;
  // zero has two patterns: without its sign it has one
  const uint32_t keep = bin == kInf ? 0x7FFF7FFFu : 0xFFFFFFFFu, two = pattern_of(bin) * 0x10001u;
  uint32_t own[2] = {0, 0};  // four bits for each round: its elements in this lane
  static_assert(kRounds <= 16, "two registers of rounds");
  h.each([&](uint32_t r, const v4u &x) {
    uint32_t others = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t d = (x[j] & keep) ^ two;
      others += __popc((((d & 0x7FFF7FFFu) + 0x7FFF7FFFu) | d) & 0x80008000u);  // a bit where a half is not 0
    }
    own[r / 8] |= (8 - others) << (r % 8 * 4);
  });
  uint32_t mine = 0;  // of lane r: round r's
#pragma unroll 1
  for (uint32_t r = 0; r < kRounds; ++r) {
    const uint32_t c = (r < 8 ? own[0] : own[1]) >> (r % 8 * 4) & 15u;
    if (!__any(c != 0)) continue;
    const uint32_t all = read_lane(scan(c), 63);
    if (lane == r) mine = all;
  }
  if (lane < kRounds) totals[lane * kWaves + wave] = mine;
  lds_barrier();
  static_assert(kRounds * kWaves <= 128, "a lane for two of them");
  const uint32_t i0 = 2 * lane;
  const uint32_t c0 = i0 < kRounds * kWaves ? totals[i0] : 0, c1 = i0 + 1 < kRounds * kWaves ? totals[i0 + 1] : 0;
  const Place place = place_of(c0, c1, rank);
  if (place.at % kWaves != wave || place.at == kNone) return;  // kNone does not happen
  const uint32_t round = place.at / kWaves;
  const v4u x = h.of_round(round);
  uint32_t m = 0;  // bit e: element e of this lane's vector is of the bin
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t d = (x[j] & keep) ^ two;
    m |= ((d & 0xFFFFu) == 0) << (2 * j) | (d >> 16 == 0) << (2 * j + 1);
  }
  uint32_t left = rank - place.before;
  const uint32_t c = __popc(m), up_to = scan(c);
  if (up_to - c <= left && left < up_to) {
    left -= up_to - c;
    for (; left; --left) m &= m - 1;
    const uint32_t r1 = N == 2 ? second_round(part[0]) : kRounds;
    const bool b = N == 2 && round >= r1;
    found(part[b ? N - 1 : 0].gid + ((b ? round - r1 : round) * kThreads + tid) * 8 + (uint32_t)__builtin_ctz(m));
  }
}

__device__ __forceinline__ static const uint32_t *list_of(const DrawArgs &a, uint32_t row, uint32_t k) {
  const uint32_t s = k >= a.sh.slices[0];
  return a.lists + row * a.row_cap + (s ? (uint64_t)a.sh.slices[0] * a.sh.width[0] : 0) +
         (uint64_t)(s ? k - a.sh.slices[0] : k) * a.sh.width[s];
}

// The count of `bin` in a list of n entries in the bins' order (0 if it has
// none), by one wave: 64 probes at a time.
__device__ __forceinline__ static uint32_t count_in_list(const uint32_t *list, uint32_t n, uint32_t bin) {
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
static constexpr int kAtOnce = 10;
struct Share {
  uint32_t k0, groups;  // the wave's first slice, and the step to its next
  uint32_t i0, step;    // the lane's first entry, and the step to its next
};
__device__ __forceinline__ static Share share_of(uint32_t n_slices) {
  const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const uint32_t ways = n_slices < kWaves ? kWaves / n_slices : 1, groups = kWaves / ways;
  return {wave / ways, groups, wave % ways * 64 + lane, ways * 64};
}

// The first entries of this lane's share, before it is known how many there are.
struct Ahead {
  uint32_t e[kAtOnce];
};
__device__ __forceinline__ static Ahead load_ahead(const DrawArgs &a, uint32_t row, const Share &h) {
  Ahead r;
  const uint32_t k = min(h.k0, a.n_slices - 1), width = a.sh.width[k >= a.sh.slices[0]];
  const uint32_t *list = list_of(a, row, k);
#pragma unroll
  for (int j = 0; j < kAtOnce; ++j) r.e[j] = list[min(h.i0 + j * h.step, width - 1)];
  return r;
}

// visit(entry) of every entry of a row's lists.
template <typename Visit>
__device__ __forceinline__ static void for_lists(const DrawArgs &a, uint32_t row, const SliceInfo *info, const Share &h,
                                          const Ahead &ahead, const Visit &visit) {
  const uint32_t lane = threadIdx.x % 64;
  for (uint32_t k = h.k0; k < a.n_slices; k += h.groups) {
    const uint32_t *list = list_of(a, row, k);
    const uint32_t n = info[k].length;
    for (uint32_t i = h.i0; i < n; i += kAtOnce * h.step) {
      Ahead r = ahead;
      if (k != h.k0 || i != h.i0) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
          if (i + j * h.step < n) r.e[j] = list[i + j * h.step];
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (i - lane + j * h.step >= n) break;  // the whole wave
        if (i + j * h.step < n) visit(r.e[j]);
      }
    }
  }
}

// ONE: the row is counted here (both shards hold at most kOneCols columns
// together); else its slices' lists are added up.
template <bool ONE>
__device__ __forceinline__ static void draw(const DrawArgs &a) {
  // Weights take the place of the bins.
  __shared__ __attribute__((aligned(16))) union {
    Bins bins;
    double weights[kLdsEntries];
  } lds;
  __shared__ uint32_t list[kLdsEntries];  // bin << 16 | count
  __shared__ double masses[kThreads];
  __shared__ uint32_t sums[kThreads];
  __shared__ GroupCounts groups;
  __shared__ Spans spans;
  __shared__ uint32_t totals[kRounds * kWaves];
  __shared__ Scratch sc;
  const uint32_t row = blockIdx.x, tid = threadIdx.x, lane = tid % 64;
  uint2 *merged = a.merged + row * a.merged_cap;
  const xfer_sample_params p = a.params[row];
  const float u = a.u[row];

  // The row's counts: in the bins if they fit 16 bits and the bins hold their
  // span (`packed`).
  const Share share = share_of(ONE ? 1 : a.n_slices);
  Ahead ahead{};
  Held held;
  Slice part[ONE ? 2 : 1];
  Span all;
  uint32_t base = 0;
  bool packed;
  if constexpr (ONE) {
    part[0] = slice_of(a.sh, row, 0);
    part[1] = slice_of(a.sh, row, 1);
    held.load(part);
    packed = count_slice(&lds.bins, &spans, held, p, &all, &base);
  } else {
    SliceInfo info{0, 0, kNone, 0};
    if (tid < a.n_slices) info = a.infos[row * a.n_slices + tid];
    ahead = load_ahead(a, row, share);
    clear(&lds.bins);
    if (tid < kMaxSlices) {
      sc.info[tid] = info;
      sc.slice_count[tid] = 0;
    }
    const uint32_t most = scan(info.most);
    if (lane == 63) sc.count[wave_number()] = most;
    share_span(&spans, Span{info.lo, info.hi, 0, 0}, 0);
    lds_barrier();
    all = join_spans(spans, 0);
    const uint32_t sum = read_lane(scan(lane < kWaves ? sc.count[lane] : 0), 63);
    packed = sum <= 0xFFFFu && fits(all);  // no value can occur more often than that
    if (packed) {
      base = base_of(all.hi);
      for_lists(a, row, sc.info, share, ahead, [&](uint32_t e) {
        const uint32_t b = e >> 16, c = e & 0xFFFFu;
        uint32_t *to = b == kInf ? &spans.zeros : &lds.bins.word[(b < kInf ? kInf - b : b - kInf) - base];
        atomicAdd(to, b > kInf ? c << 16 : c);
      });
      lds_barrier();
    }
  }

  // The row's list: in LDS if it is no longer than kLdsEntries, else in the
  // workspace.
  const uint32_t keep = keep_of(p);  // as many entries are enough
  uint32_t n;
  bool near = false;
  auto put = [&](uint32_t i, uint32_t bin, uint32_t count) {
    if (i >= keep) return;
    if (near)
      list[i] = bin << 16 | count;
    else
      merged[i] = make_uint2(bin, count);
  };
  if (packed) {
    Compact c(&lds.bins, spans.zeros, &groups);
    n = min(c.total, keep);
    near = n <= kLdsEntries;
    c.emit(base, put);
  } else {
    lds_barrier();  // the bins are cleared again
    n = list_in_passes(&lds.bins, groups.pos, [&](uint32_t bin0) {
      if constexpr (ONE) {
        count_pass(&lds.bins, held, bin0);
      } else {
        for_lists(a, row, sc.info, share, ahead, [&](uint32_t e) {
          const uint32_t b = (e >> 16) - bin0;
          if (b < kWords) atomicAdd(&lds.bins.word[b], e & 0xFFFFu);
        });
      }
    }, put);
    n = min(n, keep);
  }
  __syncthreads();
  if (n == 0) {
    if (tid == 0) a.out[row] = xfer_sampled{0.0f, -1};
    return;
  }

  const double per_t = p.temperature > 0.0f ? 1.0 / (double)p.temperature : 1.0;
  auto bin_at = [&](uint32_t i) { return near ? list[i] >> 16 : merged[i].x; };
  const double top = value_of(bin_at(0));
  const bool top_inf = isinf(top);
  auto weight = [&](uint32_t i) { return i == 0 ? 1.0 : top_inf ? 0.0 : exp((value_of(bin_at(i)) - top) * per_t); };
  auto first = [&](uint32_t i, uint32_t *c, double *w) {
    *c = near ? list[i] & 0xFFFFu : merged[i].y;
    *w = weight(i);
    if (near) lds.weights[i] = *w;
  };
  auto entry = [&](uint32_t i, uint32_t *c, double *w) {
    *c = near ? list[i] & 0xFFFFu : merged[i].y;
    *w = near ? lds.weights[i] : weight(i);
  };
  search(first, entry, n, keep, p, u, masses, sums, &sc);
  __syncthreads();
  const uint32_t bin = bin_at(sc.at);
  uint32_t rank = sc.rank;
  if constexpr (!ONE) {
    // How many of the value each slice holds.
    const uint32_t k0 = share.k0;
    if (a.n_slices <= kWaves && (k0 >= a.n_slices || sc.info[k0].length <= kAtOnce * share.step)) {
      // the list of the wave's slice is still at hand
      const uint32_t length = k0 < a.n_slices ? sc.info[k0].length : 0;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (share.i0 + j * share.step < length && ahead.e[j] >> 16 == bin) sc.slice_count[k0] = ahead.e[j] & 0xFFFFu;
    } else {
      // it is in order
#pragma unroll 1
      for (uint32_t j = k0; j < a.n_slices; j += share.groups) {
        const uint32_t c = count_in_list(list_of(a, row, j), sc.info[j].length, bin);
        if (lane == 0) sc.slice_count[j] = c;
      }
    }
    lds_barrier();
    const Place place = place_of(sc.slice_count[2 * lane], sc.slice_count[2 * lane + 1], rank);
    const uint32_t k = min(place.at, a.n_slices - 1);
    rank -= place.before;
    part[0] = slice_of(a.sh, row, k);
    held.load(part);
  }
  locate(held, part, bin, rank, totals, [&](uint32_t id) { a.out[row] = xfer_sampled{sc.prob, (int32_t)id}; });
}

};  // struct Team

template <int THREADS>
__global__ __launch_bounds__(THREADS, 4) void sample_count_kernel(Shards sh, uint32_t n_slices, uint32_t jobs,
                                                                  uint64_t row_cap, const xfer_sample_params *params,
                                                                  uint32_t *lists, SliceInfo *infos) {
  Team<THREADS>::count(sh, n_slices, jobs, row_cap, params, lists, infos);
}
template <int THREADS, bool ONE>
__global__ __launch_bounds__(THREADS, 4) void sample_draw_kernel(DrawArgs a) {
  Team<THREADS>::template draw<ONE>(a);
}
// Whether workgroups are the only ones on their compute units.
bool alone(uint32_t workgroups) { return workgroups <= kComputeUnits; }

template <bool ONE>
hipError_t launch_draw(const DrawArgs &a, uint32_t rows, hipStream_t stream) {
  if (alone(rows)) return launch(sample_draw_kernel<1024, ONE>, dim3(rows), dim3(1024), 0, stream, a);
  return launch(sample_draw_kernel<512, ONE>, dim3(rows), dim3(512), 0, stream, a);
}

uint32_t round_up8(uint32_t x) { return (x + 7u) & ~7u; }
uint32_t cut(uint32_t cols, uint32_t most) { return cols / most + (cols % most != 0); }

}  // namespace

// Slices of the narrower kind that a row is cut into, at most.
uint32_t sample_slices(uint32_t ncols0, uint32_t ncols1) {
  if ((uint64_t)ncols0 + ncols1 <= kOneCols) return 1;
  return cut(ncols0, kSliceCols) + cut(ncols1, kSliceCols);
}

namespace {

struct Sizes {
  bool one;
  uint32_t slices[2], width[2];
  uint64_t row_cap, merged_cap;
};
Sizes sizes_of(uint32_t rows, uint32_t ncols0, uint32_t ncols1) {
  Sizes z{};
  z.one = (uint64_t)ncols0 + ncols1 <= kOneCols;
  const uint32_t n[2] = {ncols0, ncols1};
  uint32_t most = z.one ? kOneCols : kSliceCols;
  auto slices = [&] { return cut(n[0], most) + cut(n[1], most); };
  while (!z.one && most < kWideSliceCols && (slices() > kMaxSlices || (uint64_t)rows * slices() > kCountWorkgroups))
    most = most * 2 < kWideSliceCols ? most * 2 : kWideSliceCols;
  for (int i = 0; i < 2; ++i) {
    z.slices[i] = cut(n[i], most);
    z.width[i] = round_up8(cut(n[i], z.slices[i]));
    z.row_cap += (uint64_t)z.slices[i] * z.width[i];
  }
  z.merged_cap = z.row_cap < kBins ? z.row_cap : kBins;
  if (z.one) z.row_cap = 0;
  return z;
}
uint64_t up16(uint64_t x) { return (x + 15) / 16 * 16; }

}  // namespace

// Layout: the rows' lists that LDS does not hold, what the count leaves of each
// slice, the slices' lists.
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
  if (z.one) return launch_draw<true>(a, in.rows, stream);
  a.n_slices = z.slices[0] + z.slices[1];
  a.row_cap = z.row_cap;
  const uint32_t jobs = in.rows * a.n_slices;
  SliceInfo *infos = reinterpret_cast<SliceInfo *>(ws + (uint64_t)in.rows * z.merged_cap * 8);
  uint32_t *lists = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(infos) + up16((uint64_t)jobs * sizeof(SliceInfo)));
  a.infos = infos;
  a.lists = lists;
  const dim3 grid(jobs < kCountWorkgroups ? jobs : kCountWorkgroups);
  const hipError_t e = alone(jobs) ? launch(sample_count_kernel<1024>, grid, dim3(1024), 0, stream, a.sh, a.n_slices,
                                            jobs, a.row_cap, in.params, lists, infos)
                                   : launch(sample_count_kernel<512>, grid, dim3(512), 0, stream, a.sh, a.n_slices,
                                            jobs, a.row_cap, in.params, lists, infos);
  if (e != hipSuccess) return e;
  return launch_draw<false>(a, in.rows, stream);
}

}  // namespace xfer
