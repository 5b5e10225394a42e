// Norms of queries and keys for each head, the position rotation, and the new
// keys' and values' rows of a paged cache, in one pass.
//
// The pass reads q, k and v once and writes q_out and the cache rows once;
// nothing is a contraction, so HBM bandwidth bounds it and the layout serves
// the memory side:
//   - a head's head_dim elements belong to head_dim / 8 lanes of one wave.  A
//     lane holds two runs of four elements, 8 bytes each, which are the two
//     sides of four rotation pairs (halves: dims i.. and i + rot_dim / 2..;
//     pairs: eight neighbours), so the rotation needs no exchange between
//     lanes and a lane needs four cosines and four sines, not eight of each;
//   - the lanes of a workgroup keep their place in the head and go from head
//     to head of one token, so the cosines, sines and weights are read once
//     per lane and not once per head;
//   - the sum of squares goes over the head's 8, 16 or 32 lanes by DPP moves
//     within a row of 16 lanes (and one lane permute for 32).
// Everything is held in binary32 and rounded once, at the store.
//
// 16384 tokens of 56 heads of 128 (BF16) take 73 us, 6.6 TB/s read and written;
// one token 2.4 us, a launch.
#include "decode.h"

namespace xfer {
namespace {

constexpr int kThreads = 256;
// Heads that a lane takes one after the other: with many tokens four, whose
// loads are in flight together (16384 tokens of 56 heads of 128: one 126 us,
// two 88, four 78, eight 78, all with streaming stores); with few tokens one,
// so that the heads of a token spread over more compute units.
constexpr int kHeadsPerLane = 4;
constexpr uint64_t kManyWorkgroups = 1024;
// The queries are stored past the caches (88 us became 71; cache rows the same
// way: 78; of calls that follow one another).  Projections are read past them
// where the call moves more than they hold (80 us became 71); smaller ones have
// just been written and are still there (2000 tokens: 10.5 us, 12.5 past the
// caches).
constexpr uint64_t kCachedBytes = 128ull << 20;

typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two values rounded to BF16, to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const v2bf r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}

// The largest E4M3 is 448; the conversion gives NaN above it, so values are
// limited first (the comparisons leave NaN as it is).
__device__ __forceinline__ float e4m3_limit(float x) { return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x; }

__device__ __forceinline__ uint32_t e4m3x4(const float *x) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_limit(x[0]), e4m3_limit(x[1]), w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_limit(x[2]), e4m3_limit(x[3]), w, true);
  return (uint32_t)w;
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}

// Sum over the LANES lanes of a head; every lane ends with it.
template <int LANES>
__device__ __forceinline__ float head_sum(float x) {
  x = dpp_add<0xB1>(x);   // quad_perm [1,0,3,2]
  x = dpp_add<0x4E>(x);   // quad_perm [2,3,0,1]
  x = dpp_add<0x141>(x);  // row_half_mirror: the other quad of 8 lanes
  if (LANES >= 16) x = dpp_add<0x140>(x);  // row_mirror: the other half of 16 lanes
  if (LANES >= 32) x += __shfl_xor(x, 16);
  return x;
}

template <bool STREAM, typename T>
__device__ __forceinline__ T load(const uint16_t *p) {
  if (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const T *>(p));
  return *reinterpret_cast<const T *>(p);
}
template <bool STREAM, typename T>
__device__ __forceinline__ void store(uint16_t *p, T v) {
  if (STREAM)
    __builtin_nontemporal_store(v, reinterpret_cast<T *>(p));
  else
    *reinterpret_cast<T *>(p) = v;
}

template <int D, int KIND, int STYLE, int HEADS, bool STREAM>
__global__ __launch_bounds__(kThreads) void rope_store_kernel(RopeStoreArgs a, uint32_t wg_per_token) {
  constexpr uint32_t kLanes = D / 8;
  constexpr uint32_t kSlots = kThreads / kLanes;  // heads side by side in a workgroup
  const uint32_t token = blockIdx.x / wg_per_token;
  const uint32_t part = blockIdx.x % wg_per_token;
  const uint32_t place = threadIdx.x % kLanes;
  const uint32_t first = part * (kSlots * HEADS) + threadIdx.x / kLanes;
  const uint32_t hq = a.q_heads, hkv = a.cache.kv_heads, n_heads = hq + 2 * hkv;

  // This lane's two runs of four dims, and whether they are rotated.
  const uint32_t r = a.rot_dim;
  const bool turned = place < r / 8;
  uint32_t d0, d1;
  if (STYLE == XFER_ROPE_HALVES && turned) {
    d0 = 4 * place;
    d1 = r / 2 + 4 * place;
  } else {
    d0 = 8 * place;
    d1 = 8 * place + 4;
  }

  // All loads that depend on nothing first.
  v2u x0[HEADS], x1[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const uint32_t h = first + i * kSlots;
    x0[i] = x1[i] = v2u{0, 0};
    if (h < n_heads) {
      const uint16_t *row = h < hq         ? a.q + token * a.q_ld + (uint64_t)h * D
                            : h < hq + hkv ? a.k + token * a.k_ld + (uint64_t)(h - hq) * D
                                           : a.v + token * a.v_ld + (uint64_t)(h - hq - hkv) * D;
      x0[i] = load<STREAM, v2u>(row + d0);
      x1[i] = load<STREAM, v2u>(row + d1);
    }
  }
  const int64_t slot = a.slots[token];
  const int32_t pos = r ? a.positions[token] : 0;
  const bool pos_ok = !r || (pos >= 0 && (uint32_t)pos < a.max_pos);
  float c[4] = {1, 1, 1, 1}, s[4] = {0, 0, 0, 0};
  if (turned && pos_ok) {
    const float *row = a.cos_sin + (uint64_t)pos * r + 4 * place;
    const v4f cv = *reinterpret_cast<const v4f *>(row), sv = *reinterpret_cast<const v4f *>(row + r / 2);
#pragma unroll
    for (int p = 0; p < 4; ++p) c[p] = cv[p], s[p] = sv[p];
  }
  v2u wq0 = {0, 0}, wq1 = {0, 0}, wk0 = {0, 0}, wk1 = {0, 0};
  if (a.q_weight) {
    wq0 = *reinterpret_cast<const v2u *>(a.q_weight + d0);
    wq1 = *reinterpret_cast<const v2u *>(a.q_weight + d1);
  }
  if (a.k_weight) {
    wk0 = *reinterpret_cast<const v2u *>(a.k_weight + d0);
    wk1 = *reinterpret_cast<const v2u *>(a.k_weight + d1);
  }
  // In bounds of the cache: a slot number from outside cannot be checked on the host.
  const uint64_t n_slots = (uint64_t)a.cache.n_pages << a.cache.page_log2;
  const bool stored = pos_ok && slot >= 0 && (uint64_t)slot < n_slots;
  const uint64_t page = (uint64_t)slot >> a.cache.page_log2;
  const uint64_t at = (uint64_t)slot & ((1ull << a.cache.page_log2) - 1);
  const uint64_t slot_bytes = page * a.cache.page_stride + at * a.cache.token_stride;

#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const uint32_t h = first + i * kSlots;
    if (h >= n_heads) break;  // lanes of one head leave together
    const bool is_q = h < hq, is_v = h >= hq + hkv;
    float y[8] = {bf_lo(x0[i].x), bf_hi(x0[i].x), bf_lo(x0[i].y), bf_hi(x0[i].y),
                  bf_lo(x1[i].x), bf_hi(x1[i].x), bf_lo(x1[i].y), bf_hi(x1[i].y)};
    if (is_q ? a.q_weight != nullptr : !is_v && a.k_weight != nullptr) {
      const v2u w0 = is_q ? wq0 : wk0, w1 = is_q ? wq1 : wk1;
      float sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(y[e], y[e], sum);
      sum = head_sum<kLanes>(sum);
      const float rms = rsqrtf(sum * (1.0f / D) + a.eps);
      const float w[8] = {bf_lo(w0.x), bf_hi(w0.x), bf_lo(w0.y), bf_hi(w0.y),
                          bf_lo(w1.x), bf_hi(w1.x), bf_lo(w1.y), bf_hi(w1.y)};
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * rms * w[e];
    }
    if (turned && !is_v) {
      // the sides of pair p: y[p] and y[4 + p], or neighbours
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int ia = STYLE == XFER_ROPE_HALVES ? p : 2 * p, ib = STYLE == XFER_ROPE_HALVES ? 4 + p : 2 * p + 1;
        const float ya = y[ia], yb = y[ib];
        y[ia] = ya * c[p] - yb * s[p];
        y[ib] = yb * c[p] + ya * s[p];
      }
    }
    if (is_q) {
      uint16_t *row = a.q_out + token * a.q_out_ld + (uint64_t)h * D;
      v2u o0 = {bf16x2(y[0], y[1]), bf16x2(y[2], y[3])}, o1 = {bf16x2(y[4], y[5]), bf16x2(y[6], y[7])};
      if (!pos_ok) o0 = o1 = v2u{0x7FC07FC0u, 0x7FC07FC0u};
      store<(HEADS > 1)>(row + d0, o0);
      store<(HEADS > 1)>(row + d1, o1);
    } else if (stored) {
      const uint32_t hk = is_v ? h - hq - hkv : h - hq;
      uint8_t *row = (is_v ? a.cache.v : a.cache.k) + slot_bytes + hk * a.cache.head_stride;
      if (KIND == XFER_KV_BF16) {
        *reinterpret_cast<v2u *>(row + 2 * d0) = v2u{bf16x2(y[0], y[1]), bf16x2(y[2], y[3])};
        *reinterpret_cast<v2u *>(row + 2 * d1) = v2u{bf16x2(y[4], y[5]), bf16x2(y[6], y[7])};
      } else {
        const float *scales = is_v ? a.cache.v_scale : a.cache.k_scale;
        const float scale = scales ? scales[hk] : 1.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] / scale;
        *reinterpret_cast<uint32_t *>(row + d0) = e4m3x4(y);
        *reinterpret_cast<uint32_t *>(row + d1) = e4m3x4(y + 4);
      }
    }
  }
}

struct Shape {
  int heads_per_lane;
  uint32_t wg_per_token;
};

Shape shape_of(uint32_t tokens, uint32_t heads, uint32_t head_dim) {
  const uint32_t slots = kThreads / (head_dim / 8);
  const uint32_t one = heads / slots + (heads % slots != 0);
  if ((uint64_t)tokens * one < kManyWorkgroups) return {1, one};
  const uint32_t many = slots * kHeadsPerLane;
  return {kHeadsPerLane, heads / many + (heads % many != 0)};
}

template <int D, int KIND, int STYLE>
hipError_t launch_shape(const RopeStoreArgs &a, const Shape &s, hipStream_t stream) {
  const dim3 grid(a.tokens * s.wg_per_token);
  if (s.heads_per_lane == 1)
    return launch(rope_store_kernel<D, KIND, STYLE, 1, false>, grid, dim3(kThreads), 0, stream, a, s.wg_per_token);
  const uint64_t heads = a.q_heads + a.cache.kv_heads * 2ull;
  if (a.tokens * heads * D * 4 <= kCachedBytes)
    return launch(rope_store_kernel<D, KIND, STYLE, kHeadsPerLane, false>, grid, dim3(kThreads), 0, stream, a,
                  s.wg_per_token);
  return launch(rope_store_kernel<D, KIND, STYLE, kHeadsPerLane, true>, grid, dim3(kThreads), 0, stream, a,
                s.wg_per_token);
}

template <int D, int KIND>
hipError_t launch_style(const RopeStoreArgs &a, int style, const Shape &s, hipStream_t stream) {
  if (style == XFER_ROPE_HALVES) return launch_shape<D, KIND, XFER_ROPE_HALVES>(a, s, stream);
  return launch_shape<D, KIND, XFER_ROPE_PAIRS>(a, s, stream);
}

template <int D>
hipError_t launch_dim(const RopeStoreArgs &a, int kind, int style, const Shape &s, hipStream_t stream) {
  if (kind == XFER_KV_BF16) return launch_style<D, XFER_KV_BF16>(a, style, s, stream);
  return launch_style<D, XFER_KV_E4M3>(a, style, s, stream);
}

}  // namespace

uint64_t rope_store_workgroups(uint32_t tokens, uint32_t heads, uint32_t head_dim) {
  return (uint64_t)tokens * shape_of(tokens, heads, head_dim).wg_per_token;
}

hipError_t launch_rope_store(const RopeStoreArgs &a, int kind, int style, hipStream_t stream) {
  const Shape s = shape_of(a.tokens, a.q_heads + 2 * a.cache.kv_heads, a.cache.head_dim);
  if (a.cache.head_dim == 64) return launch_dim<64>(a, kind, style, s, stream);
  if (a.cache.head_dim == 128) return launch_dim<128>(a, kind, style, s, stream);
  return launch_dim<256>(a, kind, style, s, stream);
}

}  // namespace xfer
