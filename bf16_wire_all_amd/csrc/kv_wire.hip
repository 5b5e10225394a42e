// A cache's slots as records of 8 or 4 bits an element for the wire, and back.
//
// A block of 32 elements of a head shares a scale 2^e, e the smallest whole
// number that brings its largest magnitude to L = 448 (E4M3) or 6 (E2M1) at
// most.  A power of two costs a float of either width nothing but range, so x
// / 2^e is exact and an element is rounded once; element * 2^e is a BF16
// number, so what comes back is exactly what was kept.  From the bits u of the
// largest magnitude e needs no logarithm: L = (1 + m) * 2^x, and adding 1 - m
// less the last bit to the mantissa carries into the exponent where the
// magnitude passes (1 + m) of its own power.
//
// Nothing is a contraction: a token's rows are read once and its record is
// written once (or the other way), so the memory bounds both directions, as
// long as few instructions go into an element.  A lane takes neighbouring
// elements of a row, a block falls to two or four lanes, which share its
// maximum by DPP moves, and a workgroup takes neighbouring rows of neighbouring
// tokens, kEach of them a lane, whose loads are in flight together.  Where a
// token's rows fill whole waves, its slot is looked up once for the wave.
//
// Kernel times on three sets of inputs in turn (two would stay in the last cache
// in part): 16,384 tokens of 8 heads of 128 from BF16 to 8 bits (102 MB) 21 us,
// 4.9 TB/s; 65,521 tokens of E4M3 to 8 bits (273 MB) 50 us, 5.4 TB/s; as many
// records of 8 bits to an E4M3 cache 51 us, 5.3 TB/s, to a BF16 one (408 MB)
// 75 us, 5.4 TB/s; 24,001 tokens of 8 heads of 64 from E4M3 to 4 bits (38 MB) 12
// us, and from there to BF16 (63 MB) 11.6 us.
#include "decode.h"

namespace xfer {
namespace {

constexpr int kThreads = 256;
// Elements of a lane, 16 bytes of the cache: 65,521 records to an E4M3 cache 51
// us, and as many tokens from one 50 (8 elements: 65 and 60).  A lane of E4M3 to
// or from 4 bits has 8.
constexpr int elements_of(int kind, int bits) { return kind == XFER_KV_E4M3 && bits == 8 ? 16 : 8; }
// Rows of a lane: one page of 16 tokens 3.0 us, 16,384 tokens 21.6, 24,001 to 4
// bits 13.7, 65,521 restored 51.7 (4 rows: 3.4, 21.3, 13.7, 53.6; one: 2.6, 22.5,
// 15.1, 50.1).
constexpr int kEach = 2;
static_assert(kThreads * kEach * 16 / 64 <= 128, "rows of a workgroup");

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

template <int BYTES>
struct Word;
template <>
struct Word<16> {
  typedef v4u type;
};
template <>
struct Word<8> {
  typedef v2u type;
};
template <>
struct Word<4> {
  typedef uint32_t type;
};

template <int BYTES, bool STREAM>
__device__ __forceinline__ void load(uint32_t *w, const uint8_t *p) {
  typedef typename Word<BYTES>::type T;
  const T v = STREAM ? __builtin_nontemporal_load(reinterpret_cast<const T *>(p)) : *reinterpret_cast<const T *>(p);
  __builtin_memcpy(w, &v, BYTES);
}
template <int BYTES, bool STREAM>
__device__ __forceinline__ void store(uint8_t *p, const uint32_t *w) {
  typedef typename Word<BYTES>::type T;
  T v;
  __builtin_memcpy(&v, w, BYTES);
  if (STREAM)
    __builtin_nontemporal_store(v, reinterpret_cast<T *>(p));
  else
    *reinterpret_cast<T *>(p) = v;
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const v2bf r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}
// The largest E4M3 is 448; the conversion gives NaN above it, so values are
// limited first (the comparisons leave NaN as it is).
__device__ __forceinline__ float e4m3_limit(float x) { return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x; }
__device__ __forceinline__ uint32_t e4m3x4(const float *x) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
}
__device__ __forceinline__ void from_e4m3x4(float *x, uint32_t w) {
  const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
// Eight E2M1 numbers, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float *x) {
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, x[0], x[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], 1.0f, 3);
}
__device__ __forceinline__ void from_e2m1x8(float *x, uint32_t w) {
  const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true));
}

// Where a lane's elements lie: head `head` of keys or values of a token.
struct Place {
  uint32_t token, head, in_record, lane;  // in_record: row of the record, keys before values
  bool there, values, last;
};
// WHOLE: all of a wave's rows are one token's, so what depends on the token is
// the scalar unit's work (16,384 tokens 21.6 us; by every lane for itself 24.6).
template <bool WHOLE>
__device__ __forceinline__ Place place_of(const WireArgs &a, uint32_t i) {
  const uint32_t kv = a.cache.kv_heads, at = i * kThreads + threadIdx.x;
  const uint32_t first = blockIdx.x * ((kThreads * kEach) >> a.lanes_log2);
  const uint32_t row = first + (at >> a.lanes_log2);
  const uint32_t any = WHOLE ? __builtin_amdgcn_readfirstlane(row) : row;
  Place p;
  p.token = __umulhi(any, a.magic) >> a.magic_shift;
  p.in_record = row - p.token * (2 * kv);
  p.values = p.in_record >= kv;
  p.head = p.values ? p.in_record - kv : p.in_record;
  p.lane = at & ((1u << a.lanes_log2) - 1);
  p.there = p.token < a.tokens;
  p.last = p.in_record == 2 * kv - 1 && p.lane == (1u << a.lanes_log2) - 1;
  return p;
}
// Byte of a slot in the cache, or -1: a slot number from outside cannot be
// checked on the host.
__device__ __forceinline__ int64_t slot_byte(const WireArgs &a, uint32_t token) {
  const int64_t slot = a.slots[token];
  const uint64_t n = (uint64_t)a.cache.n_pages << a.cache.page_log2;
  if (slot < 0 || (uint64_t)slot >= n) return -1;
  const uint64_t page = (uint64_t)slot >> a.cache.page_log2, at = (uint64_t)slot & ((1ull << a.cache.page_log2) - 1);
  return (int64_t)(page * a.cache.page_stride + at * a.cache.token_stride);
}

template <int KIND, int BITS, bool WHOLE, bool STREAM>
__global__ __launch_bounds__(kThreads) void quantize_kernel(WireArgs a) {
  constexpr int kElements = elements_of(KIND, BITS);
  constexpr int kIn = kElements * (KIND == XFER_KV_BF16 ? 2 : 1), kOut = kElements * BITS / 8;
  constexpr uint32_t kShift = BITS == 8 ? 8 : 2, kCarry = BITS == 8 ? 0x1FFFFF : 0x3FFFFF;  // of L = 1.75 * 2^8, 1.5 * 2^2
  const uint32_t data_bytes = (2 * a.cache.kv_heads << a.lanes_log2) * kOut;
  Place p[kEach];
  uint32_t w[kEach][kIn / 4];
  bool missing[kEach];  // its zeros are no head's: the sign, infinity or NaN of a scale is not theirs
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    p[i] = place_of<WHOLE>(a, i);
    missing[i] = true;
#pragma unroll
    for (int j = 0; j < kIn / 4; ++j) w[i][j] = 0;
    if (!p[i].there) continue;
    const int64_t at = slot_byte(a, p[i].token);
    missing[i] = at < 0;
    if (at >= 0)
      load<kIn, STREAM>(w[i], (p[i].values ? a.cache.v : a.cache.k) + at + p[i].head * a.cache.head_stride + p[i].lane * kIn);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    float x[kElements];
    if (KIND == XFER_KV_BF16) {
#pragma unroll
      for (int j = 0; j < kElements / 2; ++j) {
        x[2 * j] = __uint_as_float(w[i][j] << 16);
        x[2 * j + 1] = __uint_as_float(w[i][j] & 0xFFFF0000u);
      }
    } else {
      const float *scales = p[i].values ? a.cache.v_scale : a.cache.k_scale;
      const float scale = scales && !missing[i] ? scales[p[i].head] : 1.0f;
#pragma unroll
      for (int j = 0; j < kElements / 4; ++j) from_e4m3x4(x + 4 * j, w[i][j]);
#pragma unroll
      for (int j = 0; j < kElements; ++j) x[j] *= scale;
    }
    uint32_t top = 0;  // infinities and NaN are above all others
#pragma unroll
    for (int j = 0; j < kElements; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    top = dpp_max<0xB1>(top);  // quad_perm [1,0,3,2]
    if (kElements == 8) top = dpp_max<0x4E>(top);  // quad_perm [2,3,0,1]
    const bool finite = top < 0x7F800000u;
    const uint32_t carried = (top + kCarry) >> 23;
    const uint32_t e = finite ? (carried > kShift ? carried - kShift : 0) : 255;  // e + 127, at least 0
    const float inverse = finite ? __uint_as_float((254 - e) << 23) : 0.0f;       // 2^-e, a normal number for all of them
#pragma unroll
    for (int j = 0; j < kElements; ++j) x[j] = finite ? x[j] * inverse : 0.0f;
    uint32_t out[kElements / 4];
    if (BITS == 8) {
#pragma unroll
      for (int j = 0; j < kElements / 4; ++j) out[j] = e4m3x4(x + 4 * j);
    } else {
#pragma unroll
      for (int j = 0; j < kElements / 8; ++j) out[j] = e2m1x8(x + 8 * j);
    }
    if (!p[i].there) continue;
    uint8_t *record = a.records + p[i].token * a.record_ld;
    store<kOut, STREAM>(record + ((p[i].in_record << a.lanes_log2) + p[i].lane) * kOut, out);
    const uint32_t block = ((p[i].in_record << a.lanes_log2) + p[i].lane) / (32 / kElements);
    if (p[i].lane % (32 / kElements) == 0) record[data_bytes + block] = (uint8_t)e;
    if (p[i].last)
      for (uint32_t at = data_bytes + block + 1; at % 16; ++at) record[at] = 0;
  }
}

// 2^(e - 127): the lowest is subnormal, 255 stands for NaN.
__device__ __forceinline__ float scale_of(uint32_t e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
}

// x = limit(x * 2^(e - 127) / head), x a record's elements w.
//
// A division's dozen of instructions for each element would bound the kernel
// (65,521 records 101 us, with it taken by reciprocals 57).
// With h = head / 2^(e - 127) and r = 1 / h, both rounded correctly, q = x r is
// next to the quotient, and q - (q h - x) r, its remainder fused, is the
// quotient rounded correctly: so for every x of four bits and every h, tried
// all, as long as x r is finite (below 2^-126 it may be off, and is 0 in E4M3
// all the same).  h is at least 2^-119, for e up to 186 and a head's scale from
// 2^-60 on, so 448 r is 1.75 * 2^127 at most; one power less and it would be
// infinite.  What lies outside, and NaN, which the limit by a median would lose,
// is divided.
template <int BITS, int kElements>
__device__ __forceinline__ void divide(float *x, const uint32_t *w, uint32_t e, float head) {
  const uint32_t biased = __float_as_uint(head) >> 23;  // with a sign: too large
  bool usual = e - 67 <= 119 && biased - 67 <= 120;
  if (BITS == 8) {
    uint32_t nan = 0;
#pragma unroll
    for (int j = 0; j < kElements / 4; ++j) nan |= (w[j] & 0x7F7F7F7Fu) + 0x01010101u;
    usual = usual && !(nan & 0x80808080u);
  }
  if (usual) {
    const float h = __uint_as_float(__float_as_uint(head) + ((127 - e) << 23)), r = 1.0f / h;
#pragma unroll
    for (int j = 0; j < kElements; ++j) {
      const float q = x[j] * r;
      x[j] = __builtin_amdgcn_fmed3f(fmaf(-fmaf(q, h, -x[j]), r, q), -448.0f, 448.0f);
    }
  } else {
    const float scale = scale_of(e);
#pragma unroll
    for (int j = 0; j < kElements; ++j) x[j] = e4m3_limit(x[j] * scale / head);
  }
}

template <int KIND, int BITS, bool WHOLE, bool STREAM>
__global__ __launch_bounds__(kThreads) void restore_kernel(WireArgs a) {
  constexpr int kElements = elements_of(KIND, BITS);
  constexpr int kOut = kElements * (KIND == XFER_KV_BF16 ? 2 : 1), kIn = kElements * BITS / 8;
  const uint32_t data_bytes = (2 * a.cache.kv_heads << a.lanes_log2) * kIn;
  Place p[kEach];
  uint32_t w[kEach][kElements / 4], e[kEach];
  int64_t at[kEach];
  float head[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    p[i] = place_of<WHOLE>(a, i);
    at[i] = -1;
    e[i] = 0;
    head[i] = 1.0f;
#pragma unroll
    for (int j = 0; j < kElements / 4; ++j) w[i][j] = 0;
    if (!p[i].there) continue;
    at[i] = slot_byte(a, p[i].token);
    const uint8_t *record = a.records + p[i].token * a.record_ld;
    const uint32_t piece = (p[i].in_record << a.lanes_log2) + p[i].lane;
    load<kIn, STREAM>(w[i], record + piece * kIn);
    e[i] = record[data_bytes + piece / (32 / kElements)];
    if (KIND == XFER_KV_E4M3) {
      const float *scales = p[i].values ? a.cache.v_scale : a.cache.k_scale;
      if (scales) head[i] = scales[p[i].head];
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (at[i] < 0) continue;
    float x[kElements];
    if (BITS == 8) {
#pragma unroll
      for (int j = 0; j < kElements / 4; ++j) from_e4m3x4(x + 4 * j, w[i][j]);
    } else {
#pragma unroll
      for (int j = 0; j < kElements / 8; ++j) from_e2m1x8(x + 8 * j, w[i][j]);
    }
    uint32_t out[kOut / 4];
    if (KIND == XFER_KV_BF16) {
#pragma unroll
      for (int j = 0; j < kElements; ++j) x[j] *= scale_of(e[i]);
#pragma unroll
      for (int j = 0; j < kElements / 2; ++j) out[j] = bf16x2(x[2 * j], x[2 * j + 1]);
    } else {
      divide<BITS, kElements>(x, w[i], e[i], head[i]);
#pragma unroll
      for (int j = 0; j < kElements / 4; ++j) out[j] = e4m3x4(x + 4 * j);
    }
    store<kOut, STREAM>((p[i].values ? a.cache.v : a.cache.k) + at[i] + p[i].head * a.cache.head_stride + p[i].lane * kOut, out);
  }
}

// Bytes that a call moves, above which they pass the caches by: 65,521 tokens
// of 8 heads restored (273 MB) 50.4 us, 55 through them; 24,001 tokens of 4
// bits (124 MB), which were quantized just before, 14.2 us, 11.5 through them.
constexpr uint64_t kCachedBytes = 128ull << 20;

template <int KIND, int BITS, bool WHOLE, bool STREAM>
hipError_t launch_as(const WireArgs &a, bool restore, uint32_t grid, hipStream_t stream) {
  return restore ? launch(restore_kernel<KIND, BITS, WHOLE, STREAM>, dim3(grid), dim3(kThreads), 0, stream, a)
                 : launch(quantize_kernel<KIND, BITS, WHOLE, STREAM>, dim3(grid), dim3(kThreads), 0, stream, a);
}
template <int KIND, int BITS>
hipError_t launch_kind(const WireArgs &a, bool restore, uint32_t grid, bool whole, bool past, hipStream_t stream) {
  if (whole)
    return past ? launch_as<KIND, BITS, true, true>(a, restore, grid, stream)
                : launch_as<KIND, BITS, true, false>(a, restore, grid, stream);
  return past ? launch_as<KIND, BITS, false, true>(a, restore, grid, stream)
              : launch_as<KIND, BITS, false, false>(a, restore, grid, stream);
}

}  // namespace

uint64_t wire_workgroups(uint32_t tokens, uint32_t kv_heads, uint32_t head_dim, int kind, int bits) {
  const uint64_t rows = (uint64_t)tokens * kv_heads * 2, of_one = kThreads * kEach / (head_dim / elements_of(kind, bits));
  return rows / of_one + (rows % of_one != 0);
}

hipError_t launch_wire(const WireArgs &in, int kind, int bits, bool restore, hipStream_t stream) {
  WireArgs a = in;
  a.lanes_log2 = (uint32_t)__builtin_ctz(a.cache.head_dim / elements_of(kind, bits));
  const uint32_t grid = (uint32_t)wire_workgroups(a.tokens, a.cache.kv_heads, a.cache.head_dim, kind, bits);
  const uint64_t elements = (uint64_t)a.tokens * a.cache.kv_heads * 2 * a.cache.head_dim;
  const bool past = elements * (kind == XFER_KV_BF16 ? 2 : 1) + elements * bits / 8 > kCachedBytes;
  const bool whole = (2 * a.cache.kv_heads << a.lanes_log2) % 64 == 0;
  // row / (2 kv_heads) is the high half of row * magic, shifted: exact for rows
  // below 2^31, and the largest grid of 2^24 - 1 workgroups has at most 128 each.
  const uint32_t per = 2 * a.cache.kv_heads, log2 = 32 - (uint32_t)__builtin_clz(per - 1);
  a.magic = (uint32_t)(((1ull << (31 + log2)) / per) + 1);
  a.magic_shift = log2 - 1;
  if (kind == XFER_KV_BF16)
    return bits == 8 ? launch_kind<XFER_KV_BF16, 8>(a, restore, grid, whole, past, stream)
                     : launch_kind<XFER_KV_BF16, 4>(a, restore, grid, whole, past, stream);
  return bits == 8 ? launch_kind<XFER_KV_E4M3, 8>(a, restore, grid, whole, past, stream)
                   : launch_kind<XFER_KV_E4M3, 4>(a, restore, grid, whole, past, stream);
}

}  // namespace xfer
