// Attention of one new token of every request over a paged cache of keys and
// values, split over the cache's length and joined.
//
// Every visible key and value is read once and little is done with it: 4 *
// group operations for each element, so HBM bandwidth bounds the call, and
// the layout serves the loads:
//   - a workgroup takes (row, kv head, piece of the row's visible tokens) and
//     all query heads of that kv head (16 or 32 at a time), so a key is read
//     once for all of them.  Its four waves take tiles of 32 tokens in turn,
//     each with a running maximum and sum of its own, and meet once at the
//     end, in LDS.  Rows that are cut into pieces leave (max, sum, weighted
//     sum) in the workspace, and a second launch joins them;
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
// The running maximum is raised only when a score passes it by more than 2^8
// (weights stay below 256, far from binary32's limits), which leaves out most
// of the rescaling and of the exchanges between lanes.
#include "decode.h"

namespace xfer {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr uint32_t kTile = 32;                   // tokens of a wave's tile
constexpr uint32_t kStep = kTile * kWaves;       // tokens of a workgroup's round
constexpr uint32_t kMinChunkSteps = 2;
constexpr uint32_t kTargetWorkgroups = 2048;
constexpr uint32_t kMaxSplits = 256;             // one thread of the join for each
constexpr float kRaise = 8.0f;                   // in powers of two
constexpr uint32_t kXcds = 8;

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

// The rows' visible tokens, numbered from 0: the first `first` tokens, then
// from token first + gap on.
struct Visible {
  uint32_t n, first, gap;
};
__device__ __forceinline__ Visible visible_of(const AttnArgs &a, uint32_t row) {
  Visible v;
  v.n = min(a.lens[row], a.max_len);
  v.first = v.gap = 0;
  if (a.window && v.n > a.window) {
    v.first = min(a.sinks, v.n - a.window);
    v.gap = v.n - a.window - v.first;
    v.n = a.window + v.first;
  }
  return v;
}

template <int D, int KIND>
struct Layout {
  static constexpr int kBytes = KIND == XFER_KV_BF16 ? 2 : 1;
  static constexpr int kLoadsK = D * kBytes / 64;      // 16-byte loads of a token's key for each lane
  static constexpr int kDwordsV = D * kBytes / 64;     // dwords of a token's value row for each lane
  static constexpr int kMfmaK = D / 32;
  static constexpr int kMfmaV = D / 16;
};

// Dims that product j of V^T P^T gives for row n of its result (n < 16).
template <int D, int KIND>
__device__ __forceinline__ uint32_t dim_of(uint32_t j, uint32_t n) {
  // BF16 rows of 512 bytes are read as two runs of 16 bytes for each lane.
  if (D == 256 && KIND == XFER_KV_BF16) return (j / 8) * 128 + n * 8 + j % 8;
  return n * (D / 16) + j;
}

template <int D, int KIND>
__device__ __forceinline__ void load_v(uint32_t *dst, const uint8_t *row, uint32_t n) {
  constexpr int W = Layout<D, KIND>::kDwordsV;
  if constexpr (W == 1) {
    dst[0] = *reinterpret_cast<const uint32_t *>(row + 4 * n);
  } else if constexpr (W == 2) {
    const v2u w = *reinterpret_cast<const v2u *>(row + 8 * n);
    dst[0] = w.x, dst[1] = w.y;
  } else {
#pragma unroll
    for (int c = 0; c < W / 4; ++c) {
      const v4u w = *reinterpret_cast<const v4u *>(row + 256 * c + 16 * n);
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[4 * c + i] = w[i];
    }
  }
}

// Weights of eight tokens as two BF16 numbers each, high and low.
struct Weights {
  v4u hi, lo;
};

template <int D, int KIND, int MT>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attn_kernel(AttnArgs a, uint32_t chunk, uint32_t n_splits,
                                                           uint32_t m_groups) {
  using L = Layout<D, KIND>;
  constexpr int kPad = 4;  // floats between rows of the exchange, so that 16 rows' stores fall on all banks
  __shared__ float lds_o[kWaves][16][D + kPad];
  __shared__ float lds_m[kWaves][MT * 16], lds_l[kWaves][MT * 16];

  // Workgroups of one (piece, row) follow one another on one XCD, whose L2
  // then serves the lines that two heads share; (piece, row) go round the XCDs.
  const uint32_t inner_n = a.cache.kv_heads * m_groups;
  const uint32_t xcd = blockIdx.x % kXcds, rest = blockIdx.x / kXcds;
  const uint32_t inner = rest % inner_n, pair = rest / inner_n * kXcds + xcd;
  const uint32_t split = pair / a.rows, row = pair % a.rows;
  if (split >= n_splits) return;
  const uint32_t kvh = inner / m_groups, mg = inner % m_groups;

  const Visible vis = visible_of(a, row);
  const uint32_t v0 = split * chunk;
  if (v0 >= vis.n && !(n_splits == 1)) return;  // the join does not ask for this piece
  const uint32_t v1 = min(v0 + chunk, vis.n);

  const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid % 64, n = lane % 16, g = lane / 16;
  const uint32_t h0 = mg * (MT * 16);  // first query head of this tile within the group

  // Q: query head h0 + 16 * m + n, the dims that this lane's K loads hold.
  v4u q[MT][L::kMfmaK];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const uint32_t h = h0 + 16 * m + n;
#pragma unroll
    for (int k = 0; k < L::kMfmaK; ++k) {
      const uint32_t d = KIND == XFER_KV_BF16 ? k * 32 + g * 8 : (k / 2) * 64 + g * 16 + (k % 2) * 8;
      q[m][k] = v4u{0, 0, 0, 0};
      if (h < a.group)
        q[m][k] = *reinterpret_cast<const v4u *>(a.q + row * a.q_ld + (uint64_t)(kvh * a.group + h) * D + d);
    }
  }
  float scale2 = a.scale * 1.4426950408889634f;
  if (KIND == XFER_KV_E4M3 && a.cache.k_scale) scale2 *= a.cache.k_scale[kvh];

  const uint8_t *kbase = a.cache.k + kvh * a.cache.head_stride + 16 * g;
  const uint8_t *vbase = a.cache.v + kvh * a.cache.head_stride;
  const uint32_t *table = a.page_table + row * a.table_ld;
  const uint32_t slot_mask = (1u << a.cache.page_log2) - 1;

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
    p.page = p.there ? table[p.token >> a.cache.page_log2] : 0;
    return p;
  };
  // Byte offset of a token's slot, or -1 where there is none.
  auto offset_of = [&](const Place &p) -> int64_t {
    if (!p.there || p.page >= a.cache.n_pages) return -1;
    return (int64_t)(p.page * a.cache.page_stride + (p.token & slot_mask) * a.cache.token_stride);
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
      for (int i = 0; i < L::kLoadsK; ++i) k[s][i] = *reinterpret_cast<const v4u *>(p + 64 * i);
    }
  };

  v4f o[MT][L::kMfmaV];
  float mx[MT], sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mx[m] = -INFINITY;
    sum[m] = 0;
#pragma unroll
    for (int j = 0; j < L::kMfmaV; ++j) o[m][j] = v4f{0, 0, 0, 0};
  }

  uint32_t t = v0 + wave * kTile;
  int64_t off = -1;
  Place next{};
  if (t < v1) {
    off = offset_of(look_up(t));
    load_k(off);
    next = look_up(t + kStep);
  }
  for (; t < v1; t += kStep) {
    // Value rows of this lane group's eight tokens.
    uint32_t vr[8][L::kDwordsV];
    const uint32_t lo = (uint32_t)off, hi = (uint32_t)((uint64_t)off >> 32);
    uint32_t absent = 0;  // bit e: token e of this group is not there
    const bool full = __all(off >= 0);
#define XFER_ROW(E)                                                            \
  {                                                                            \
    const uint32_t h = row_lane<E>(hi);                                        \
    const bool gone = (int32_t)h < 0;                                          \
    const uint64_t at = gone ? 0 : ((uint64_t)h << 32) | row_lane<E>(lo);      \
    absent |= gone ? 1u << E : 0;                                              \
    load_v<D, KIND>(vr[E], vbase + at, n);                                     \
  }
    XFER_ROW(0) XFER_ROW(1) XFER_ROW(2) XFER_ROW(3) XFER_ROW(4) XFER_ROW(5) XFER_ROW(6) XFER_ROW(7)
#undef XFER_ROW

    // Scores: lane (n, g) gets query head n's of tokens 4g + i and 16 + 4g + i.
    v4f s[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) s[m][0] = s[m][1] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int kk = 0; kk < L::kMfmaK; ++kk) {
        v4u op;
        if constexpr (KIND == XFER_KV_BF16) {
          op = k[half][kk];
        } else {
          const v4u w = k[half][kk / 2];
          const uint32_t w0 = kk % 2 ? w.z : w.x, w1 = kk % 2 ? w.w : w.y;
          op = v4u{e4m3x2_to_bf16<false>(w0), e4m3x2_to_bf16<true>(w0), e4m3x2_to_bf16<false>(w1),
                   e4m3x2_to_bf16<true>(w1)};
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) s[m][half] = mfma(op, q[m][kk], s[m][half]);
      }
    }

    // The next tile's keys, while this one's weights are computed.
    const int64_t off_next = offset_of(next);
    if (t + kStep < v1) {
      load_k(off_next);
      next = look_up(t + 2 * kStep);
    }

    Weights w[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = s[m][e / 4][e % 4] * scale2;
      if (!full) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (absent >> e) & 1 ? -INFINITY : x[e];
      }
      float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      if (__any(top > mx[m] + kRaise)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float raised = fmaxf(mx[m], top);
        // a head that has seen nothing yet has nothing to rescale
        const float f = mx[m] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[m] - raised);
        mx[m] = raised;
        sum[m] *= f;
#pragma unroll
        for (int j = 0; j < L::kMfmaV; ++j) o[m][j] *= f;
      }
      const float base = mx[m] == -INFINITY ? 0.0f : mx[m];
      float p[8], low[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(x[e] - base);
        sum[m] += p[e];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[m].hi[i] = bf16x2(p[2 * i], p[2 * i + 1]);
        low[2 * i] = p[2 * i] - __uint_as_float(w[m].hi[i] << 16);
        low[2 * i + 1] = p[2 * i + 1] - __uint_as_float(w[m].hi[i] & 0xFFFF0000u);
        w[m].lo[i] = bf16x2(low[2 * i], low[2 * i + 1]);
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
      uint32_t two[8];  // dims 2i and 2i + 1 of each token
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (KIND == XFER_KV_BF16)
          two[e] = vr[e][i];
        else
          two[e] = i % 2 ? e4m3x2_to_bf16<true>(vr[e][i / 2]) : e4m3x2_to_bf16<false>(vr[e][i / 2]);
      }
      v4u even, odd;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        even[e] = __builtin_amdgcn_perm(two[2 * e + 1], two[2 * e], 0x05040100);
        odd[e] = __builtin_amdgcn_perm(two[2 * e + 1], two[2 * e], 0x07060302);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        o[m][2 * i] = mfma(even, w[m].hi, o[m][2 * i]);
        o[m][2 * i] = mfma(even, w[m].lo, o[m][2 * i]);
        o[m][2 * i + 1] = mfma(odd, w[m].hi, o[m][2 * i + 1]);
        o[m][2 * i + 1] = mfma(odd, w[m].lo, o[m][2 * i + 1]);
      }
    }
    off = off_next;
  }

  // The four waves' results, joined in LDS.
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    sum[m] += __shfl_xor(sum[m], 16);
    sum[m] += __shfl_xor(sum[m], 32);
    if (g == 0) {
      lds_m[wave][16 * m + n] = mx[m];
      lds_l[wave][16 * m + n] = sum[m];
    }
  }
  __syncthreads();
  const float v_scale = KIND == XFER_KV_E4M3 && a.cache.v_scale ? a.cache.v_scale[kvh] : 1.0f;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (m) __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, lds_m[w][16 * m + n]);
    const float f = mx[m] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[m] - top);
#pragma unroll
    for (int j = 0; j < L::kMfmaV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) lds_o[wave][n][dim_of<D, KIND>(j, 4 * g + i)] = o[m][j][i] * f;
    __syncthreads();
#pragma unroll
    for (int it = 0; it < D / 64; ++it) {
      const uint32_t at = it * kThreads + tid, hq = at / (D / 4), d = at % (D / 4) * 4;
      const uint32_t h = h0 + 16 * m + hq;
      if (h >= a.group) continue;
      float all = -INFINITY, total = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) all = fmaxf(all, lds_m[w][16 * m + hq]);
      v4f r = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float mw = lds_m[w][16 * m + hq];
        total += mw == -INFINITY ? lds_l[w][16 * m + hq] : lds_l[w][16 * m + hq] * __builtin_amdgcn_exp2f(mw - all);
        r += *reinterpret_cast<const v4f *>(&lds_o[w][hq][d]);
      }
      if (n_splits == 1) {
        const float inv = total == 0.0f ? 0.0f : v_scale / total;
        r *= inv;
        const uint64_t at_out = row * a.out_ld + (uint64_t)(kvh * a.group + h) * D + d;
        if (a.out_mode == XFER_OUT_F32)
          *reinterpret_cast<v4f *>(static_cast<float *>(a.out) + at_out) = r;
        else
          *reinterpret_cast<v2u *>(static_cast<uint16_t *>(a.out) + at_out) = v2u{bf16x2(r.x, r.y), bf16x2(r.z, r.w)};
      } else {
        const uint64_t part = (((uint64_t)row * a.cache.kv_heads + kvh) * n_splits + split) * a.group + h;
        *reinterpret_cast<v4f *>(a.part_o + part * D + d) = r;
        if (d == 0) {
          a.part_ml[2 * part] = all;
          a.part_ml[2 * part + 1] = total;
        }
      }
    }
  }
}

// One workgroup for each (row, query head): the pieces' weighted sums, each
// scaled to the largest maximum, in the pieces' order.
template <int D>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnArgs a, uint32_t chunk, uint32_t n_splits) {
  constexpr uint32_t kLanes = D / 4, kAtOnce = kThreads / kLanes;
  __shared__ float lds_w[kMaxSplits];
  __shared__ float lds_red[kWaves];
  __shared__ v4f lds_o[kAtOnce][kLanes];
  const uint32_t row = blockIdx.x / a.q_heads, head = blockIdx.x % a.q_heads;
  const uint32_t kvh = head / a.group, h = head % a.group, tid = threadIdx.x;
  const Visible vis = visible_of(a, row);
  const uint32_t pieces = (vis.n + chunk - 1) / chunk;
  const uint64_t part0 = ((uint64_t)row * a.cache.kv_heads + kvh) * n_splits;

  float m = -INFINITY, l = 0;
  if (tid < pieces) {
    m = a.part_ml[2 * ((part0 + tid) * a.group + h)];
    l = a.part_ml[2 * ((part0 + tid) * a.group + h) + 1];
  }
  float top = m;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
  if (tid % 64 == 0) lds_red[tid / 64] = top;
  __syncthreads();
  top = fmaxf(fmaxf(lds_red[0], lds_red[1]), fmaxf(lds_red[2], lds_red[3]));
  const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
  if (tid < pieces) lds_w[tid] = f;
  float total = m == -INFINITY ? l : l * f;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d);
  __syncthreads();
  if (tid % 64 == 0) lds_red[tid / 64] = total;
  const uint32_t d4 = tid % kLanes, s0 = tid / kLanes;
  v4f r = {0, 0, 0, 0};
  for (uint32_t s = s0; s < pieces; s += kAtOnce)
    r += lds_w[s] * *reinterpret_cast<const v4f *>(a.part_o + ((part0 + s) * a.group + h) * D + 4 * d4);
  lds_o[s0][d4] = r;
  __syncthreads();
  if (s0 != 0) return;
#pragma unroll
  for (uint32_t s = 1; s < kAtOnce; ++s) r += lds_o[s][d4];
  total = (lds_red[0] + lds_red[1]) + (lds_red[2] + lds_red[3]);
  const float v_scale = a.cache.v_scale ? a.cache.v_scale[kvh] : 1.0f;
  r *= total == 0.0f ? 0.0f : v_scale / total;
  const uint64_t at = row * a.out_ld + (uint64_t)head * D + 4 * d4;
  if (a.out_mode == XFER_OUT_F32)
    *reinterpret_cast<v4f *>(static_cast<float *>(a.out) + at) = r;
  else
    *reinterpret_cast<v2u *>(static_cast<uint16_t *>(a.out) + at) = v2u{bf16x2(r.x, r.y), bf16x2(r.z, r.w)};
}

template <int D, int KIND>
hipError_t launch_tiles(const AttnArgs &a, const AttnShape &s, hipStream_t stream) {
  const dim3 grid((uint32_t)s.workgroups);
  if (s.m_tiles == 1)
    return launch(attn_kernel<D, KIND, 1>, grid, dim3(kThreads), 0, stream, a, s.chunk, s.n_splits, s.m_groups);
  return launch(attn_kernel<D, KIND, 2>, grid, dim3(kThreads), 0, stream, a, s.chunk, s.n_splits, s.m_groups);
}

template <int D>
hipError_t launch_dim(const AttnArgs &a, int kind, const AttnShape &s, hipStream_t stream) {
  const hipError_t e =
      kind == XFER_KV_BF16 ? launch_tiles<D, XFER_KV_BF16>(a, s, stream) : launch_tiles<D, XFER_KV_E4M3>(a, s, stream);
  if (e != hipSuccess || s.n_splits == 1) return e;
  return launch(attn_join_kernel<D>, dim3(a.rows * a.q_heads), dim3(kThreads), 0, stream, a, s.chunk, s.n_splits);
}

}  // namespace

AttnShape attn_shape(uint32_t rows, uint32_t kv_heads, uint32_t group, uint64_t vis_max) {
  AttnShape s{};
  s.m_tiles = group <= 16 ? 1 : 2;
  const uint32_t tile = 16 * s.m_tiles;
  s.m_groups = group / tile + (group % tile != 0);
  const uint64_t inner = (uint64_t)kv_heads * s.m_groups, pairs = rows * inner;
  const uint64_t steps = (vis_max + kStep - 1) / kStep;
  uint64_t chunk = kMinChunkSteps;
  chunk = chunk * kTargetWorkgroups < pairs * steps ? (pairs * steps + kTargetWorkgroups - 1) / kTargetWorkgroups : chunk;
  if (chunk * kMaxSplits < steps) chunk = (steps + kMaxSplits - 1) / kMaxSplits;
  if (chunk > steps) chunk = steps;
  s.chunk = (uint32_t)(chunk * kStep);
  s.n_splits = (uint32_t)((steps + chunk - 1) / chunk);
  s.workgroups = ((uint64_t)rows * s.n_splits + kXcds - 1) / kXcds * kXcds * inner;
  return s;
}

uint64_t attn_workspace_bytes(const AttnShape &s, uint32_t rows, uint32_t q_heads, uint32_t head_dim) {
  if (s.n_splits == 1) return 0;
  const uint64_t parts = (uint64_t)rows * q_heads * s.n_splits;
  return (parts * 8 + 15) / 16 * 16 + parts * head_dim * 4;
}

hipError_t launch_attn(const AttnArgs &in, int kind, const AttnShape &s, hipStream_t stream) {
  AttnArgs a = in;
  const uint64_t parts = (uint64_t)a.rows * a.q_heads * s.n_splits;
  if (s.n_splits > 1) a.part_o = a.part_ml + (parts * 8 + 15) / 16 * 4;
  if (a.cache.head_dim == 64) return launch_dim<64>(a, kind, s, stream);
  if (a.cache.head_dim == 128) return launch_dim<128>(a, kind, s, stream);
  return launch_dim<256>(a, kind, s, stream);
}

}  // namespace xfer
