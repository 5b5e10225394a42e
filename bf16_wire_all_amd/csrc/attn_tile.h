// A wave's walk over visible tokens of a paged cache, which the attention of
// one token (attn_paged.hip) and that of rows with a shared prefix
// (attn_shared.hip) have in common: tiles of 32 tokens, the products and the
// running softmax, all in registers.
#pragma once

#include "decode.h"

namespace xfer {
namespace {

constexpr uint32_t kTile = 32;                   // tokens of a wave's tile
constexpr float kRaise = 8.0f;                   // of the running maximum, in powers of two

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const v2bf r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}

// Two E4M3 numbers (half HI of w) as two BF16: every E4M3 value is one.
template <bool HI>
__device__ __forceinline__ uint32_t e4m3x2_to_bf16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// Lane E of this lane's row of 16 lanes.
template <int E>
__device__ __forceinline__ uint32_t row_lane(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x150 + E, 0xF, 0xF, true);
}

// Visible tokens, numbered from 0: the first `first` tokens, then from token
// first + gap on.
struct Visible {
  uint32_t n, first, gap;
};

template <int D, int KIND>
struct Layout {
  static constexpr int kBytes = KIND == XFER_KV_BF16 ? 2 : 1;
  static constexpr int kLoadsK = D * kBytes / 64;      // 16-byte loads of a token's key for each lane
  static constexpr int kDwordsV = D * kBytes / 64;     // dwords of a token's value row for each lane
  static constexpr int kMfmaK = D / 32;
  static constexpr int kMfmaV = D / 16;
};

// Waves that the runs give a SIMD: two, where registers allow.  Three or four
// would fit for heads of 64 with up to 16 of them, three for E4M3 of 128; they
// wait on more places of the memory at once, which serves some calls and costs
// others (heads of 64, E4M3, four for two: 48 rows of up to 8192 tokens 45 us, 58,
// but two rows of 100,000, tokens first, 55, 51, and 768 (row, kv head)s of up to
// 2800 39, 37; heads of 128, BF16, three for two, two rows of 131071: 187, 169).
// Heads of 256 leave no registers for the queries beside two waves' or 32
// heads' results: they are read from LDS for each tile, one step ahead of the
// products (32 heads, E4M3, 8 rows of up to 20001 tokens: 35 us with them in
// registers, 32 so; 32 heads of BF16 keep them, at one wave for a SIMD).
template <int D, int KIND, int TILES>
struct Residence {
  static constexpr bool kQInLds = D == 256 && (TILES == 1 || KIND == XFER_KV_E4M3);
  static constexpr int kPerSimd = D == 256 && (KIND == XFER_KV_BF16 || TILES == 2) ? 1 : 2;
};

// Dims that product j of V^T P^T gives for row n of its result (n < 16).
template <int D, int KIND>
__device__ __forceinline__ uint32_t dim_of(uint32_t j, uint32_t n) {
  // BF16 rows of 512 bytes are read as two runs of 16 bytes for each lane.
  if (D == 256 && KIND == XFER_KV_BF16) return (j / 8) * 128 + n * 8 + j % 8;
  return n * (D / 16) + j;
}

// STREAM: past the caches.
template <bool STREAM, typename T>
__device__ __forceinline__ T load(const uint8_t *p) {
  if (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const T *>(p));
  return *reinterpret_cast<const T *>(p);
}

template <int D, int KIND, bool STREAM>
__device__ __forceinline__ void load_v(uint32_t *dst, const uint8_t *row, uint32_t n) {
  constexpr int W = Layout<D, KIND>::kDwordsV;
  if constexpr (W == 1) {
    dst[0] = load<STREAM, uint32_t>(row + 4 * n);
  } else if constexpr (W == 2) {
    const v2u w = load<STREAM, v2u>(row + 8 * n);
    dst[0] = w.x, dst[1] = w.y;
  } else {
#pragma unroll
    for (int c = 0; c < W / 4; ++c) {
      const v4u w = load<STREAM, v4u>(row + 256 * c + 16 * n);
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[4 * c + i] = w[i];
    }
  }
}

// Weights of eight tokens as PARTS BF16 numbers each.  The first is off by up to
// 2^-8 of the weight, and each rounds what is left: two come to 2^-17 of it, far
// below a BF16 result's own 2^-8, and three hold all 24 bits.
template <int PARTS>
struct Weights {
  v4u part[PARTS];
};

// Tokens v0 .. v1 - 1 of the visible ones, for the query heads in q (or, where
// registers do not hold them, in lds_q): this wave's tiles, from token `first`
// on, ROUND tokens from one to the next.  Leaves the running maxima, the
// sums of weights and the weighted sums.
template <int D, int KIND, int MR, int PARTS, uint32_t ROUND, bool STREAM, int QR>
__device__ __forceinline__ void attn_walk(const CacheView &cache, uint32_t kvh, const uint32_t *table, const Visible &vis,
                                          uint32_t first, uint32_t v1, float scale2, uint32_t n, uint32_t g, uint32_t lane,
                                          const v4u (&q)[QR][Layout<D, KIND>::kMfmaK], const v4u *lds_q,
                                          v4f (&o)[MR][Layout<D, KIND>::kMfmaV], float (&mx)[MR], float (&sum)[MR]) {
  using L = Layout<D, KIND>;
  using R = Residence<D, KIND, MR>;
#pragma unroll
  for (int r = 0; r < MR; ++r) {
    mx[r] = -INFINITY;
    sum[r] = 0;
#pragma unroll
    for (int j = 0; j < L::kMfmaV; ++j) o[r][j] = v4f{0, 0, 0, 0};
  }

  const uint8_t *kbase = cache.k + kvh * cache.head_stride + 16 * g;
  const uint8_t *vbase = cache.v + kvh * cache.head_stride;
  const uint32_t slot_mask = (1u << cache.page_log2) - 1;

  // Lane (n, g) looks up the token whose value row its group reads as row n
  // (n < 8): tokens 4g + n, and 16 + 4g + n - 4.
  const uint32_t my_token = ((n & 4) ? 16 : 0) + 4 * g + (n & 3);
  // Tokens n and 16 + n are looked up by these lanes.
  const uint32_t from_a = 16 * (n >> 2) + (n & 3), from_b = from_a + 4;

  struct Place {
    uint32_t page, token;
    bool there;
  };
  auto look_up = [&](uint32_t t) {
    Place p;
    const uint32_t v = t + my_token;
    p.there = v < v1;
    p.token = p.there ? (v < vis.first ? v : v + vis.gap) : 0;
    p.page = p.there ? table[p.token >> cache.page_log2] : 0;
    return p;
  };
  // Byte offset of a token's slot, or -1 where there is none.
  auto offset_of = [&](const Place &p) -> int64_t {
    if (!p.there || p.page >= cache.n_pages) return -1;
    return (int64_t)(p.page * cache.page_stride + (p.token & slot_mask) * cache.token_stride);
  };
  v4u k[2][L::kLoadsK];
  auto load_k = [&](int64_t off) {
    const uint32_t lo = (uint32_t)off, hi = (uint32_t)((uint64_t)off >> 32);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t from = s ? from_b : from_a;
      const uint64_t o = ((uint64_t)(uint32_t)__shfl((int)hi, from) << 32) | (uint32_t)__shfl((int)lo, from);
      const uint8_t *p = kbase + ((int64_t)o < 0 ? 0 : o);  // a hole's scores are replaced: any row will do
#pragma unroll
      for (int i = 0; i < L::kLoadsK; ++i) k[s][i] = load<STREAM, v4u>(p + 64 * i);
    }
  };

  // The value rows of this lane group's eight tokens; bit e of the result:
  // token e is not there (then the cache's first slot is read).
  auto load_values = [&](uint32_t (&vr)[8][L::kDwordsV], int64_t off) -> uint32_t {
    const uint32_t lo = (uint32_t)off, hi = (uint32_t)((uint64_t)off >> 32);
    uint32_t gone = 0;
#define XFER_ROW(E)                                                                        \
  {                                                                                        \
    const uint32_t h = row_lane<E>(hi);                                                    \
    const bool no = (int32_t)h < 0;                                                        \
    gone |= no ? 1u << E : 0;                                                              \
    load_v<D, KIND, STREAM>(vr[E], vbase + (no ? 0 : ((uint64_t)h << 32) | row_lane<E>(lo)), n);   \
  }
    XFER_ROW(0) XFER_ROW(1) XFER_ROW(2) XFER_ROW(3) XFER_ROW(4) XFER_ROW(5) XFER_ROW(6) XFER_ROW(7)
#undef XFER_ROW
    return gone;
  };

  uint32_t t = first;
  int64_t off = -1;
  Place next{};
  if (t < v1) {
    off = offset_of(look_up(t));
    load_k(off);
    next = look_up(t + ROUND);
  }
  for (; t < v1; t += ROUND) {
    // keep the queries where they are: read anew from LDS for each tile
    if constexpr (R::kQInLds) asm volatile("" ::: "memory");
    uint32_t vr[8][L::kDwordsV];
    const uint32_t absent = load_values(vr, off);
    const bool full = __all(off >= 0);

    // Scores: lane (n, g) gets query head n's of tokens 4g + i and 16 + 4g + i.
    v4f s[MR][2];
#pragma unroll
    for (int r = 0; r < MR; ++r) s[r][0] = s[r][1] = v4f{0, 0, 0, 0};
    // The 16 tokens of a half, dims of step kk.
    auto keys = [&](int half, int kk) {
      if constexpr (KIND == XFER_KV_BF16) {
        return k[half][kk];
      } else {
        const v4u w = k[half][kk / 2];
        const uint32_t w0 = kk % 2 ? w.z : w.x, w1 = kk % 2 ? w.w : w.y;
        return v4u{e4m3x2_to_bf16<false>(w0), e4m3x2_to_bf16<true>(w0), e4m3x2_to_bf16<false>(w1),
                   e4m3x2_to_bf16<true>(w1)};
      }
    };
    if constexpr (R::kQInLds) {
      v4u held[2][MR];
#pragma unroll
      for (int r = 0; r < MR; ++r) held[0][r] = lds_q[r * L::kMfmaK * 64 + lane];
#pragma unroll
      for (int kk = 0; kk < L::kMfmaK; ++kk) {
        if (kk + 1 < L::kMfmaK) {
#pragma unroll
          for (int r = 0; r < MR; ++r) held[(kk + 1) % 2][r] = lds_q[(r * L::kMfmaK + kk + 1) * 64 + lane];
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const v4u op = keys(half, kk);
#pragma unroll
          for (int r = 0; r < MR; ++r) s[r][half] = mfma(op, held[kk % 2][r], s[r][half]);
        }
        __builtin_amdgcn_sched_barrier(0);  // or all reads would be made first, and held
      }
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int kk = 0; kk < L::kMfmaK; ++kk) {
          const v4u op = keys(half, kk);
#pragma unroll
          for (int r = 0; r < MR; ++r) s[r][half] = mfma(op, q[r][kk], s[r][half]);
        }
      }
    }

    // The next tile's keys, while this one's weights are computed.
    const int64_t off_next = offset_of(next);
    if (t + ROUND < v1) {
      load_k(off_next);
      next = look_up(t + 2 * ROUND);
    }

    Weights<PARTS> w[MR];
#pragma unroll
    for (int r = 0; r < MR; ++r) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = s[r][e / 4][e % 4] * scale2;
      if (!full) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (absent >> e) & 1 ? -INFINITY : x[e];
      }
      float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      if (__any(top > mx[r] + kRaise)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float raised = fmaxf(mx[r], top);
        // a head that has seen nothing yet has nothing to rescale
        const float f = mx[r] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[r] - raised);
        mx[r] = raised;
        sum[r] *= f;
#pragma unroll
        for (int j = 0; j < L::kMfmaV; ++j) o[r][j] *= f;
      }
      const float base = mx[r] == -INFINITY ? 0.0f : mx[r];
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(x[e] - base);
        sum[r] += p[e];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x0 = p[2 * i], x1 = p[2 * i + 1];
#pragma unroll
        for (int c = 0; c < PARTS; ++c) {
          const uint32_t two = bf16x2(x0, x1);
          w[r].part[c][i] = two;
          x0 -= __uint_as_float(two << 16);
          x1 -= __uint_as_float(two & 0xFFFF0000u);
        }
      }
    }

    // A row that is not there was read from the cache's first slot: its
    // weight is 0, and 0 times a NaN or an infinity is not.
    if (!full) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int i = 0; i < L::kDwordsV; ++i) vr[e][i] = (absent >> e) & 1 ? 0 : vr[e][i];
    }

    // Weighted sums: product j takes its dim's eight tokens.
#pragma unroll
    for (int i = 0; i < L::kMfmaV / 2; ++i) {
      v4u even, odd;  // dims 2i and 2i + 1, two tokens in a register
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (KIND == XFER_KV_BF16) {
          even[e] = __builtin_amdgcn_perm(vr[2 * e + 1][i], vr[2 * e][i], 0x05040100);
          odd[e] = __builtin_amdgcn_perm(vr[2 * e + 1][i], vr[2 * e][i], 0x07060302);
        } else {
          const uint32_t pairs = __builtin_amdgcn_perm(vr[2 * e + 1][i / 2], vr[2 * e][i / 2], i % 2 ? 0x07030602 : 0x05010400);
          even[e] = e4m3x2_to_bf16<false>(pairs);
          odd[e] = e4m3x2_to_bf16<true>(pairs);
        }
      }
#pragma unroll
      for (int r = 0; r < MR; ++r) {
#pragma unroll
        for (int c = 0; c < PARTS; ++c) o[r][2 * i] = mfma(even, w[r].part[c], o[r][2 * i]);
#pragma unroll
        for (int c = 0; c < PARTS; ++c) o[r][2 * i + 1] = mfma(odd, w[r].part[c], o[r][2 * i + 1]);
      }
    }
    off = off_next;
  }
}

// Four sums from dim d on, some of them NaN.  Where no value is NaN but one is
// infinite, the products made it so: a part of a weight is often 0 or negative.
// The sum is that infinity then, unless there are both.  A loop over all of the
// run's values: calls without an infinity never take it.
template <int KIND>
__device__ __forceinline__ v4f with_infinities(const CacheView &cache, uint32_t kvh, const uint32_t *table,
                                               const Visible &vis, uint32_t v0, uint32_t v1, v4f v, uint32_t d) {
  static_assert(KIND == XFER_KV_BF16, "E4M3 has no infinities");
  const uint8_t *vbase = cache.v + kvh * cache.head_stride;
  const uint32_t slot_mask = (1u << cache.page_log2) - 1;
  uint32_t nan = 0, up = 0, down = 0;  // a bit for each dim
#pragma unroll 1
  for (uint32_t at = v0; at < v1; ++at) {
    const uint32_t token = at < vis.first ? at : at + vis.gap, page = table[token >> cache.page_log2];
    if (page >= cache.n_pages) continue;
    const v2u w = *reinterpret_cast<const v2u *>(vbase + page * cache.page_stride +
                                                 (token & slot_mask) * cache.token_stride + 2 * d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = i % 2 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
      nan |= ((x & 0x7FFFu) > 0x7F80u) << i;
      up |= (x == 0x7F80u) << i;
      down |= (x == 0xFF80u) << i;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (isnan(v[i]) && !(nan >> i & 1) && (up >> i & 1) != (down >> i & 1)) v[i] = up >> i & 1 ? INFINITY : -INFINITY;
  return v;
}

}  // namespace
}  // namespace xfer
