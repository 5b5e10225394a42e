// Log probabilities of given tokens with their ranks, the best elements and the
// entropy of rows of BF16 logits in two column shards.
//
// With m the row's largest logit, x_i = (l_i - m) / T <= 0 and w_i = exp(x_i):
//   Z = 1 + R, R the weights of all elements but the first of the row's order,
//   logprob_i = x_i - log1p(R), entropy = log1p(R) - sum w_i x_i / Z.
// Keeping the largest element out of the sum leaves R's own digits where it is
// small (a token of probability 1 - 1e-9 has a log probability of -1e-9, not
// 0), and both terms of the entropy are positive, so neither cancels.
//
// The logits are read once.  A workgroup holds a slice of a row in registers
// and makes its passes there:
//   1. the largest: packed 16-bit maxima of the patterns as they stand (as
//      whole numbers positive BF16 numbers are in order, negative ones below
//      them; rows without a positive element, or with NaN, are looked at again);
//   2. the best elements: each lane's own largest gives a bound that enough
//      elements reach (the n-th largest of a wave's 64 lanes), and the few
//      elements that reach it go to a list in LDS, where their places are
//      counted;
//   3. the ranks: comparisons, counted a wave at a time;
//   4. the weights: 2^(l c - m c), c = log2(e) / T, by one fused multiply-add
//      and the hardware's power.  m c is rounded to binary32; what that moves
//      all weights by is a factor that is put right afterwards.
// Thread sums are binary32 (of up to 64 elements), everything above binary64.
// The sums of a row's slices are kept relative to the largest so far.
//
// Where rows are few, each is cut into several workgroups' parts, which a
// second launch folds: (largest, R, sum w x) scaled to the row's largest.
//
// 2048 rows of 151,936 with one token's rank each (622 MB): 155-168
// us, 4 TB/s.  The vector unit bounds it, at some 12 instructions for each
// element, half of them the weights': with the sums of slices kept apart and
// joined at the end it took 182 us, with ranks compared as floats and each
// weight clamped by itself 313.  More waves on a SIMD spill (226 us and more).
// 16 rows of 129,280: 10.5 + 5.8 us, chains of dependent steps.
#include "decode.h"

namespace xfer {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRounds = 8;                                // vectors of 8 elements that a thread holds
constexpr uint32_t kSliceCols = kThreads * 8 * kRounds;   // 16,384
// How rows are cut into parts: for so many workgroups (1024: 500 rows of 32,000 29.3 us for 25.2, 512: 16 rows of 129,280
// 15.1 for 10.5), of so many columns at least (2048: 100 rows of 32,000 20.6 us for 12.4, 16 rows 11.9 + 6.7 for 10.5 + 5.8,
// one row 8.5 + 6.8 for 9.3 + 5.9; 8192: one row with 20 alternatives 14.0 + 13.4 for 12.5 + 6.8).
constexpr uint32_t kWorkgroups = 1536;
constexpr uint32_t kMinCols = 4096;
constexpr uint32_t kMaxParts = 128;                       // of a row
constexpr uint32_t kList = 1024;                          // elements that reach the bound, at most
static_assert(kMaxParts % 8 == 0 && kList % 8 == 0 && kList >= kMaxTop * kMaxTop, "the fold's, of as many parts as elements asked for");
constexpr uint32_t kMasked = 0xFF80FF80u;
constexpr unsigned short kFar = 0xF149;                   // -1e30

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef short v2s __attribute__((ext_vector_type(2)));
typedef unsigned short v2us __attribute__((ext_vector_type(2)));

// A place in the row's order: 0 for what is not in it (NaN, -inf), larger for
// larger values, -0 as +0.
__device__ __forceinline__ uint32_t ord(uint32_t v) {
  const uint32_t mag = v & 0x7FFFu;
  if (mag > 0x7F80u || v == 0xFF80u) return 0;
  return v & 0x8000u ? 0x8000u - mag : 0x8000u + mag;
}
// The value of a place that is not 0.
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o >= 0x8000u ? o - 0x8000u : 0x8000u | (0x8000u - o)) << 16);
}
// An element: its place, then its id, the lower first.
__device__ __forceinline__ uint64_t key_of(uint32_t o, uint32_t id) { return o ? (uint64_t)o << 32 | (0xFFFFFFFFu - id) : 0; }
__device__ __forceinline__ uint32_t ord_of(uint64_t key) { return (uint32_t)(key >> 32); }
__device__ __forceinline__ uint32_t id_of(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }

__device__ __forceinline__ uint32_t half(uint32_t w, int h) { return h ? w >> 16 : w & 0xFFFFu; }
__device__ __forceinline__ float as_float(uint32_t w, int h) {
  return __uint_as_float(h ? w & 0xFFFF0000u : w << 16);
}

// Over the lanes of a wave, by DPP moves; lanes that a move does not reach give `old`.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp(int x, int old) {
  return __builtin_amdgcn_update_dpp(old, x, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp(uint64_t x) {
  return (uint64_t)(uint32_t)dpp<CTRL, ROWS>((int)(x >> 32), 0) << 32 | (uint32_t)dpp<CTRL, ROWS>((int)(uint32_t)x, 0);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double x) {
  return __longlong_as_double((long long)dpp<CTRL, ROWS>((uint64_t)__double_as_longlong(x)));
}
__device__ __forceinline__ int wave_max(int x) {
  constexpr int kLow = -0x7FFFFFFF - 1;
  x = max(x, dpp<0x111, 0xF>(x, kLow));
  x = max(x, dpp<0x112, 0xF>(x, kLow));
  x = max(x, dpp<0x114, 0xF>(x, kLow));
  x = max(x, dpp<0x118, 0xF>(x, kLow));
  x = max(x, dpp<0x142, 0xA>(x, kLow));
  x = max(x, dpp<0x143, 0xC>(x, kLow));
  return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ uint64_t read_lane(uint64_t x, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t x) {
  x = max(x, dpp<0x111, 0xF>(x));
  x = max(x, dpp<0x112, 0xF>(x));
  x = max(x, dpp<0x114, 0xF>(x));
  x = max(x, dpp<0x118, 0xF>(x));
  x = max(x, dpp<0x142, 0xA>(x));
  x = max(x, dpp<0x143, 0xC>(x));
  return read_lane(x, 63);
}
__device__ __forceinline__ double wave_sum(double x) {
  x += dpp<0x111, 0xF>(x);
  x += dpp<0x112, 0xF>(x);
  x += dpp<0x114, 0xF>(x);
  x += dpp<0x118, 0xF>(x);
  x += dpp<0x142, 0xA>(x);
  x += dpp<0x143, 0xC>(x);
  return __longlong_as_double((long long)read_lane((uint64_t)__double_as_longlong(x), 63));
}

// What a set of elements comes to: its first element, and of all others the sum
// of weights and of weights times x, relative to that first one.
struct Sum {
  double rest, wx;
  uint64_t top;
};
// (l - m) / T of a row, in binary64.
__device__ __forceinline__ double scaled(float l, float m, float T) {
  if (l == m) return 0.0;
  return __builtin_isinf(m) ? -INFINITY : ((double)l - (double)m) / (double)T;
}
// The sum of all lanes' two sets, by a whole wave.  (Greedy: the first element alone.)
__device__ __forceinline__ Sum join(const Sum &s0, const Sum &s1, float T) {
  Sum all = {0, 0, wave_max(max(s0.top, s1.top))};
  if (!all.top || !(T > 0.0f)) return all;
  const float m = value_of(ord_of(all.top));
  double rest = 0, wx = 0;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const Sum s = i ? s1 : s0;
    if (!s.top) continue;
    const double x = scaled(value_of(ord_of(s.top)), m, T), f = exp(x), own = s.top == all.top ? 0.0 : 1.0;
    if (f > 0) {  // not so where x is -inf
      rest += f * (own + s.rest);
      wx += f * (s.wx + (own + s.rest) * x);
    }
  }
  all.rest = wave_sum(rest);
  all.wx = wave_sum(wx);
  return all;
}

// The next BF16 number above v (NaN above +inf, which nothing reaches).
__device__ __forceinline__ float above(float v) {
  const uint32_t u = __float_as_uint(v);
  return __uint_as_float(v == 0.0f ? 0x10000u : u & 0x80000000u ? u - 0x10000u : u + 0x10000u);
}

struct Slice {
  const uint16_t *ptr;
  uint32_t cols, gid;
};
__device__ __forceinline__ Slice slice_of(const LogprobArgs &a, uint32_t row, uint32_t k) {
  const uint32_t s = k >= a.slices[0];
  const uint32_t c0 = min((s ? k - a.slices[0] : k) * a.width[s], a.s[s].ncols);
  return {a.s[s].ptr + row * a.s[s].ld + c0, min(a.width[s], a.s[s].ncols - c0), a.s[s].col_offset + c0};
}

// A given token's place in the order (0: it has none).
__device__ __forceinline__ uint64_t token_key(const LogprobArgs &a, uint32_t row, int32_t id) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const uint32_t c = (uint32_t)id - a.s[s].col_offset;
    if (id >= 0 && (uint32_t)id >= a.s[s].col_offset && c < a.s[s].ncols)
      return key_of(ord(a.s[s].ptr[row * a.s[s].ld + c]), (uint32_t)id);
  }
  return 0;
}

// The row's results from its sum, its tokens' ranks and its best elements, by a
// whole wave.
__device__ __forceinline__ void finish(const LogprobArgs &a, uint32_t row, const Sum &sum, float T,
                                       const uint32_t *ranks, const uint64_t *best) {
  const uint32_t tid = threadIdx.x;
  const bool greedy = !(T > 0.0f);
  const double log_z = greedy ? 0.0 : log1p(sum.rest);
  const float m = sum.top ? value_of(ord_of(sum.top)) : 0.0f;
  auto logprob = [&](uint64_t key) -> float {
    if (!key) return -INFINITY;
    if (greedy) return key == sum.top ? 0.0f : -INFINITY;
    return (float)(scaled(value_of(ord_of(key)), m, T) - log_z);
  };
  if (tid == 0 && a.entropy) a.entropy[row] = !sum.top || greedy ? 0.0f : (float)(log_z - sum.wx / (1.0 + sum.rest));
  if (tid < a.n_tokens) {
    const uint64_t at = (uint64_t)row * a.n_tokens + tid, key = token_key(a, row, a.tokens[at]);
    a.token_out[at] = xfer_token_logprob{logprob(key), key ? (int32_t)ranks[tid] : -1};
  }
  if (tid < a.n_top) {
    const uint64_t key = best[tid];
    a.top_out[(uint64_t)row * a.n_top + tid] = xfer_top_logprob{logprob(key), key ? (int32_t)id_of(key) : -1};
  }
}

// The n_top best of what is listed (one element once), in order; what lies past their end is left.  By all threads; the
// list's places up to the next multiple of kBlock are written.
constexpr uint32_t kBlock = 8;  // keys that are on their way together
__device__ __forceinline__ void best_of(uint64_t *list, uint32_t n, uint32_t n_top, uint64_t *best) {
  const uint32_t up = (n + kBlock - 1) / kBlock * kBlock;
  if (n + threadIdx.x < up) list[n + threadIdx.x] = 0;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t key = list[i];
    uint32_t before = 0;
#pragma unroll 1
    for (uint32_t j = 0; j < up; j += kBlock)
#pragma unroll
      for (uint32_t k = 0; k < kBlock; ++k) before += list[j + k] > key;
    if (key && before < n_top) best[before] = key;
  }
}

struct Shared {
  uint64_t list[kList];           // what reaches the bound
  uint64_t best[kMaxTop];         // the best so far, in order
  uint64_t token[kMaxTokens];
  uint32_t rank[kMaxTokens];
  int32_t wave_top[kWaves], wave_bound[kWaves];
  double wave_rest[kWaves], wave_wx[kWaves];
  uint64_t wave_key[kWaves];
  uint32_t listed;
  uint32_t equal[2], first[2];  // elements equal to the largest so far, and the lowest id; of the one before it no longer
};

// What reaches `bound` and is in the row's order.
__device__ __forceinline__ float bound_value(int32_t o) {
  return o > 0 ? value_of((uint32_t)o) : __uint_as_float(0xFF7F0000u);  // or the lowest finite number
}

__global__ __launch_bounds__(kThreads, 4) void logprobs_kernel(LogprobArgs a) {
  __shared__ Shared sh;
  const uint32_t tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const uint32_t row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const uint32_t n_slices = a.slices[0] + a.slices[1];
  const uint32_t k0 = (uint32_t)((uint64_t)n_slices * part / a.parts), k1 = (uint32_t)((uint64_t)n_slices * (part + 1) / a.parts);
  const float T = a.temperature ? a.temperature[row] : 1.0f;
  const float c = T > 0.0f ? 1.4426950408889634f / T : 0.0f;
  const int32_t token = tid < a.n_tokens ? a.tokens[(uint64_t)row * a.n_tokens + tid] : -1;
  if (tid < a.n_tokens) sh.rank[tid] = 0;
  if (tid < a.n_top) sh.best[tid] = 0;
  if (tid < 2) sh.equal[tid] = 0, sh.first[tid] = 0xFFFFFFFFu;
  // The largest so far, and of all others this thread's sums relative to it.
  uint32_t o = 0, which = 0;
  float m = 0;
  double rest = 0, wx = 0;

#pragma unroll 1
  for (uint32_t k = k0; k < k1; ++k) {
    const Slice s = slice_of(a, row, k);
    v4u w[kRounds];
    {
      // The vector that the slice ends in, by the thread that holds it.
      const uint32_t end = s.cols / 8;
      v4u last = v4u{kMasked, kMasked, kMasked, kMasked};
      if (s.cols % 8 && tid == end % kThreads) {
#pragma unroll 1
        for (uint32_t i = 0; i < s.cols % 8; ++i) {
          const uint32_t v = s.ptr[8 * end + i], low = 16 * (i % 2);
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q)
            if (i / 2 == q) last[q] = (last[q] & ~(0xFFFFu << low)) | v << low;
        }
      }
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const uint32_t at = r * kThreads + tid;
        w[r] = at == end ? last : v4u{kMasked, kMasked, kMasked, kMasked};
        if (at < end) w[r] = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(s.ptr) + at);
      }
    }
    if (k == k0 && tid < a.n_tokens) sh.token[tid] = token_key(a, row, token);  // on its way with the first slice
    // f(round) for each that the slice has
    auto rounds = [&](auto &&f) {
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        if ((uint32_t)r * kThreads * 8 < s.cols) f(r);
        __builtin_amdgcn_sched_barrier(0);  // or what all rounds leave would be held at once
      }
    };
    // f(word, half, columns from this thread's first one on) for each element of a round
    auto of_round = [&](int r, auto &&f) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t x = w[r][q];
        f(x, 0, 8 * r * kThreads + 2 * q);
        f(x, 1, 8 * r * kThreads + 2 * q + 1);
      }
    };
    // A number made anew for each use: what follows from it for every element, ready in registers for all passes, would
    // not fit.
    auto anew = [](uint32_t x) {
      asm volatile("" : "+v"(x));
      return x;
    };
    // f(pattern, column) for each element that this thread holds, read again: for what is rare
    auto again = [&](auto &&f) {
#pragma unroll 1
      for (uint32_t c = 8 * tid; c < s.cols; c += c % 8 == 7 ? 8 * kThreads - 7 : 1) f((uint32_t)s.ptr[c], c);
    };

    // 1. The largest, and a bound that n_top elements of a wave reach.
    v2s round_top[kRounds], two = {-0x8000, -0x8000};
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const uint32_t x0 = w[r][0], x1 = w[r][1], x2 = w[r][2], x3 = w[r][3];
      round_top[r] = __builtin_elementwise_max(
          __builtin_elementwise_max(__builtin_bit_cast(v2s, x0), __builtin_bit_cast(v2s, x1)),
          __builtin_elementwise_max(__builtin_bit_cast(v2s, x2), __builtin_bit_cast(v2s, x3)));
      two = __builtin_elementwise_max(two, round_top[r]);
    }
    const int mine = max((int)two.x, (int)two.y);
    int top = wave_max(mine);
    int own = mine >= 0 ? 0x8000 + mine : 0;  // this lane's largest in the order; 0: not known
    const uint32_t known = (uint32_t)__popcll(__ballot(mine >= 0));
    const bool plain = top > 0 && top <= 0x7F80 && known >= a.n_top;
    if (!plain) {
      own = 0;
      rounds([&](int r) {
        of_round(r, [&](uint32_t x, int h, uint32_t) { own = max(own, (int)ord(half(anew(x), h))); });
      });
      top = wave_max(own) - 0x8000;
    }
    int bound = 0;
    if (a.n_top) {
#pragma unroll
      for (int b = 0x8000; b; b >>= 1)
        if ((uint32_t)__popcll(__ballot(own >= bound + b)) >= a.n_top) bound += b;
    }
    __syncthreads();  // the slice before this one is done with LDS
    if (lane == 0) {
      sh.wave_top[wave] = top + 0x8000;
      sh.wave_bound[wave] = bound;
    }
    if (tid == 0) sh.listed = a.n_top;
    if (tid < a.n_top) sh.list[tid] = sh.best[tid];
    __syncthreads();
    uint32_t largest = o;
    int32_t reach = a.n_top ? (int32_t)ord_of(sh.best[a.n_top - 1]) : 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      largest = max(largest, (uint32_t)sh.wave_top[i]);
      reach = max(reach, sh.wave_bound[i]);
    }
    largest = __builtin_amdgcn_readfirstlane(largest);
    reach = __builtin_amdgcn_readfirstlane(reach);
    if (largest == 0) continue;  // nothing so far is in the order
    if (largest != o) {
      const float before = m;
      m = value_of(largest);
      if (o) {
        const double x = scaled(before, m, T), f = T > 0.0f ? exp(x) : 0.0;
        const double n = tid == 0 ? sh.equal[which] : 0;
        wx = f > 0 ? f * (wx + x * (rest + n)) : 0.0;  // not so where x is -inf
        rest = f * (rest + n);
        if (tid == 0) sh.equal[which] = 0, sh.first[which] = 0xFFFFFFFFu;
        which ^= 1;
      }
      o = largest;
    }

    // 2. What reaches the bound.
    if (a.n_top) {
      const float at_least = bound_value(reach);
      const int pattern = reach > 0x8000 && plain ? reach - 0x8000 : -0x8000;  // as a round's largest
      rounds([&](int r) {
        if (!__any(max((int)round_top[r].x, (int)round_top[r].y) >= pattern)) return;
        of_round(r, [&](uint32_t x, int h, uint32_t col) {
          const bool in = as_float(x, h) >= at_least;
          const uint64_t mask = __ballot(in);
          if (!mask) return;
          uint32_t base = 0;
          if (lane == 0) base = atomicAdd(&sh.listed, (uint32_t)__popcll(mask));
          base = __builtin_amdgcn_readfirstlane(base);
          const uint32_t at = base + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
          if (in && at < kList) sh.list[at] = key_of(ord(half(x, h)), s.gid + 8 * anew(tid) + col);
        });
      });
    }

    // 3. The elements before each token.
#pragma unroll 1
    for (uint32_t i = 0; i < a.n_tokens; ++i) {
      const uint64_t key = read_lane(sh.token[i], 0);
      if (!key) continue;
      const uint32_t id = id_of(key);
      const float g = value_of(ord_of(key));
      uint32_t n = 0;
      if (id > s.gid && id < s.gid + s.cols) {
        rounds([&](int r) {
          of_round(r, [&](uint32_t x, int h, uint32_t col) {
            const float l = as_float(anew(x), h);
            n += (uint32_t)__popcll(__ballot(l > g || (l == g && (int)(8 * tid) < (int)(id - s.gid - col))));
          });
        });
      } else {
        // equal ones come before it where their ids do
        const float from = id > s.gid ? g : above(g);
        if (plain && from > 0) {
          // as whole numbers, straight from where they lie
          const int at_least = (int)(__float_as_uint(from) >> 16);
          rounds([&](int r) {
            of_round(r, [&](uint32_t x, int h, uint32_t) {
              n += (uint32_t)__popcll(h ? __ballot((int)x >= at_least << 16) : __ballot((short)x >= (short)at_least));
            });
          });
        } else {
          rounds([&](int r) {
            of_round(r, [&](uint32_t x, int h, uint32_t) { n += (uint32_t)__popcll(__ballot(as_float(anew(x), h) >= from)); });
          });
        }
      }
      if (lane == 0 && n) atomicAdd(&sh.rank[i], n);
    }

    // 4. The weights.  Elements equal to the largest are taken out and counted.
    if (own == (int)o || !plain) {
      uint32_t n = 0, first = 0xFFFFFFFFu;
      const short pattern = (short)(o - 0x8000);
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        if (plain && round_top[r].x != pattern && round_top[r].y != pattern) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t x = w[r][q];
          const bool lo = as_float(x, 0) == m, hi = as_float(x, 1) == m;
          n += lo + hi;
          if (lo || hi) first = min(first, 8 * anew(tid) + 8 * r * kThreads + 2 * q + (lo ? 0 : 1));
          const bool lo_out = lo || __builtin_isnan(as_float(x, 0)), hi_out = hi || __builtin_isnan(as_float(x, 1));
          x = lo_out ? (x & 0xFFFF0000u) | (kMasked & 0xFFFFu) : x;
          w[r][q] = hi_out ? (x & 0xFFFFu) | (kMasked & 0xFFFF0000u) : x;
        }
      }
      if (n) {
        atomicAdd(&sh.equal[which], n);
        atomicMin(&sh.first[which], s.gid + first);
      }
    }
    if (!(T > 0.0f) || __builtin_isinf(m)) {
      // all weight is the largest elements'
    } else if (__builtin_fabsf(m) * c <= 0x1p20f && c <= 0x1p20f && c >= 0x1p-60f) {
      const float mc = m * c;
      float sum_w = 0, sum_wt = 0;
      rounds([&](int r) {
        // What is masked or a negative NaN becomes a large negative number, like what is below it: all have weight 0.
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t x = w[r][q];
          w[r][q] = __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(v2us, x), v2us{kFar, kFar}));
        }
        of_round(r, [&](uint32_t x, int h, uint32_t) {
          const float t = fmaf(as_float(x, h), c, -mc);
          const float e = __builtin_amdgcn_exp2f(t);
          sum_w += e;
          sum_wt = fmaf(e, t, sum_wt);
        });
      });
      // Every power is too small by off, at most 2^-4: 2^off - 1 by its series, to 2^-45.
      constexpr double kLn2 = 0.6931471805599453;
      const double off = (double)mc - (double)m * (double)c, y = off * kLn2;
      const double f = 1 + y * (1 + y / 2 * (1 + y / 3 * (1 + y / 4 * (1 + y / 5 * (1 + y / 6 * (1 + y / 7 * (1 + y / 8)))))));
      rest += f * sum_w;
      wx += f * kLn2 * (sum_wt + off * sum_w);
    } else {
      again([&](uint32_t v, uint32_t) {
        if (!ord(v) || as_float(v, 0) == m) return;
        const double t = scaled(as_float(v, 0), m, T), e = exp(t);
        if (e > 0) rest += e, wx += e * t;
      });
    }
    // The best of what is listed.
    if (a.n_top) {
      __syncthreads();
      const uint32_t n = sh.listed;
      if (n <= kList) {
        best_of(sh.list, n, a.n_top, sh.best);
      } else {
        // Very many equal elements, or few lanes with all of them: one after
        // the other, the largest below the one before.
        uint64_t below = ~0ull;
#pragma unroll 1
        for (uint32_t i = 0; i < a.n_top; ++i) {
          uint64_t key = tid < a.n_top && sh.list[tid] < below ? sh.list[tid] : 0;
          again([&](uint32_t v, uint32_t col) {
            const uint64_t y = key_of(ord(v), s.gid + col);
            if (y < below && y > key) key = y;
          });
          key = wave_max(key);
          __syncthreads();
          if (lane == 0) sh.wave_key[wave] = key;
          __syncthreads();
          for (int j = 0; j < kWaves; ++j) key = max(key, sh.wave_key[j]);
          below = key;
          if (tid == 0) sh.best[i] = key;
        }
      }
    }
  }
  rest = wave_sum(rest);
  wx = wave_sum(wx);
  if (lane == 0) sh.wave_rest[wave] = rest, sh.wave_wx[wave] = wx;
  __syncthreads();
  Sum sum = {(double)sh.equal[which] - 1.0, 0, key_of(o, sh.first[which])};
#pragma unroll
  for (int i = 0; i < kWaves; ++i) sum.rest += sh.wave_rest[i], sum.wx += sh.wave_wx[i];
  if (a.parts > 1) {
    const uint64_t at = (uint64_t)row * a.parts + part;
    if (tid == 0) static_cast<Sum *>(a.sums)[at] = sum;
    if (tid < a.n_tokens) a.ranks[at * a.n_tokens + tid] = sh.rank[tid];
    if (tid < a.n_top) a.keys[at * a.n_top + tid] = sh.best[tid];
    return;
  }
  if (wave == 0) finish(a, row, sum, T, sh.rank, sh.best);
}

// One workgroup for each row, whose first wave joins the sums while the others look for the best.
__global__ __launch_bounds__(kThreads) void logprobs_fold_kernel(LogprobArgs a) {
  __shared__ uint32_t rank[kMaxTokens];
  __shared__ uint64_t head[kMaxParts], list[kList], best[kMaxTop];
  __shared__ uint64_t least;
  __shared__ uint32_t listed;
  const uint32_t row = blockIdx.x, tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const float T = a.temperature ? a.temperature[row] : 1.0f;
  const uint64_t at = (uint64_t)row * a.parts;
  const uint64_t *keys = a.keys + at * a.n_top;
  // Two parts to a lane.  All loads that depend on nothing first.
  const Sum *sums = static_cast<const Sum *>(a.sums) + at;
  const Sum none = {0, 0, 0};
  const Sum s0 = lane < a.parts ? sums[lane] : none, s1 = lane + 64 < a.parts ? sums[lane + 64] : none;
  for (uint32_t i = wave; i < a.n_tokens; i += kWaves) {
    uint32_t n = lane < a.parts ? a.ranks[(at + lane) * a.n_tokens + i] : 0;
    n += lane + 64 < a.parts ? a.ranks[(at + lane + 64) * a.n_tokens + i] : 0;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) n += __shfl_xor(n, d);
    if (lane == 0) rank[i] = n;
  }
  if (a.n_top) {
    // The parts' lists are in order.  Where there are as many parts as elements asked for, none that is below
    // that many of their first ones is among the best.
    if (tid < kMaxParts) head[tid] = tid < a.parts ? keys[(uint64_t)tid * a.n_top] : 0;
    if (tid < a.n_top) best[tid] = 0;
    if (tid == 0) least = 1, listed = 0;
    __syncthreads();
    if (tid < a.parts && a.parts >= a.n_top) {
      uint32_t before = 0;
#pragma unroll 1
      for (uint32_t j = 0; j < a.parts; j += kBlock)
#pragma unroll
        for (uint32_t k = 0; k < kBlock; ++k) before += head[j + k] > head[tid] || (head[j + k] == head[tid] && j + k < tid);
      if (before == a.n_top - 1 && head[tid]) least = head[tid];
    }
    __syncthreads();
    for (uint32_t i = tid; i < a.parts * a.n_top; i += kThreads) {
      const uint64_t key = keys[i];
      if (key >= least) {
        const uint32_t to = atomicAdd(&listed, 1u);
        if (to < kList) list[to] = key;
      }
    }
    __syncthreads();
    best_of(list, listed, a.n_top, best);
  }
  __syncthreads();
  if (wave == 0) finish(a, row, join(s0, s1, T), T, rank, best);
}

struct Shape {
  uint32_t parts, slices[2], width[2];
};
Shape shape_of(uint32_t rows, uint32_t ncols0, uint32_t ncols1) {
  // As many parts as give kWorkgroups, of at least kMinCols.
  const uint64_t cols = (uint64_t)ncols0 + ncols1;
  uint64_t want = rows < kWorkgroups ? (kWorkgroups + rows - 1) / rows : 1;
  want = want < kMaxParts - 1 ? want : kMaxParts - 1;
  uint64_t width = (cols + want - 1) / want;
  width = width < kMinCols ? kMinCols : width > kSliceCols ? kSliceCols : (width + 7) / 8 * 8;
  Shape s{};
  const uint32_t n[2] = {ncols0, ncols1};
  for (int i = 0; i < 2; ++i) {
    s.slices[i] = (uint32_t)((n[i] + width - 1) / width);
    s.width[i] = (uint32_t)(((n[i] + s.slices[i] - 1) / s.slices[i] + 7) / 8 * 8);
  }
  const uint64_t slices = (uint64_t)s.slices[0] + s.slices[1];
  s.parts = (uint32_t)(want < slices ? want : slices);
  return s;
}

uint64_t up16(uint64_t x) { return (x + 15) / 16 * 16; }

}  // namespace

uint64_t logprobs_workgroups(uint32_t rows, uint32_t ncols0, uint32_t ncols1) {
  return (uint64_t)rows * shape_of(rows, ncols0, ncols1).parts;
}

// Layout: the parts' sums, their best elements, their ranks.
uint64_t logprobs_workspace_bytes(uint32_t rows, uint32_t ncols0, uint32_t ncols1, uint32_t n_tokens, uint32_t n_top) {
  const Shape s = shape_of(rows, ncols0, ncols1);
  if (s.parts == 1) return 0;
  const uint64_t n = (uint64_t)rows * s.parts;
  return up16(n * sizeof(Sum)) + up16(n * n_top * 8) + up16(n * n_tokens * 4);
}

hipError_t launch_logprobs(const LogprobArgs &in, void *workspace, hipStream_t stream) {
  LogprobArgs a = in;
  const Shape s = shape_of(a.rows, a.s[0].ncols, a.s[1].ncols);
  a.parts = s.parts;
  for (int i = 0; i < 2; ++i) a.slices[i] = s.slices[i], a.width[i] = s.width[i];
  if (s.parts > 1) {
    const uint64_t n = (uint64_t)a.rows * s.parts;
    uint8_t *at = static_cast<uint8_t *>(workspace);
    a.sums = at;
    a.keys = reinterpret_cast<uint64_t *>(at += up16(n * sizeof(Sum)));
    a.ranks = reinterpret_cast<uint32_t *>(at + up16(n * a.n_top * 8));
  }
  const hipError_t e = launch(logprobs_kernel, dim3(a.rows * s.parts), dim3(kThreads), 0, stream, a);
  if (e != hipSuccess || s.parts == 1) return e;
  return launch(logprobs_fold_kernel, dim3(a.rows), dim3(kThreads), 0, stream, a);
}

}  // namespace xfer
