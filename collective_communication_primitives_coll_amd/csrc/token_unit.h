// Device-side building blocks of the token-wise operators (layer norm,
// 8-bit checkpoints, gated activation, vocabulary log probabilities).
//
// A row of `hidden` elements is cut into units of 16 bytes, 8 elements of
// bf16 or 4 of fp32, one to a lane: the lanes of a wave then load and store
// 1 KiB runs.  (With 8 elements of fp32 to a lane, each access leaves out
// every other 16 bytes of its run: layer norm of fp32 rows ran at 4.4 TB/s
// so, and at 4.9-5.3 TB/s with 4.)  A lane owns the same columns of the rows, of
// the weights, of their gradients and of the checkpoint, so that a unit of E
// elements may also be E fp32 weights or E one-byte codes.  Rows of an odd
// width leave most units off a 16-byte boundary; gfx950 loads and stores 16
// bytes at any element's address, so these take the same instructions.
#pragma once

#include <type_traits>

#include "device_common.h"
#include "token_args.h"

namespace coll {

// A checkpoint row as the source of a unit (beside kF32 and kBF16).
constexpr int kE4M3 = 16;

// 16 bytes at the address of an element.
typedef u32x4 u32x4_e __attribute__((aligned(2)));

// Elements of a 16-byte unit.
template <int DT>
constexpr int kElems = 16 / Traits<DT>::B;

// E elements of a type, as loaded.
template <int SRC, int E> struct RawUnit {
  u32x4 v[E * Traits<SRC>::B / 16];
};
template <int E> struct RawUnit<kE4M3, E> {
  uint32_t c[E / 4];  // codes
  float s;            // their group's scale
};

template <int SRC, int E> __device__ __forceinline__ RawUnit<SRC, E> zero_unit() {
  RawUnit<SRC, E> r;
  if constexpr (SRC == kE4M3) {
#pragma unroll
    for (auto& c : r.c) c = 0;
    r.s = 0.0f;
  } else {
#pragma unroll
    for (auto& v : r.v) v = u32x4{0, 0, 0, 0};
  }
  return r;
}

// E elements from element `at` of a row (bf16 or fp32).
template <int DT, int E, bool NT>
__device__ __forceinline__ RawUnit<DT, E> load_unit(const void* row, uint64_t at) {
  const u32x4_e* s = reinterpret_cast<const u32x4_e*>(as_global(static_cast<const uint8_t*>(row)) + at * Traits<DT>::B);
  RawUnit<DT, E> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.v) / 16); ++i) {
    if constexpr (NT) r.v[i] = __builtin_nontemporal_load(s + i);
    else r.v[i] = s[i];
  }
  return r;
}
template <int DT, int E, bool NT>
__device__ __forceinline__ void store_unit(void* row, uint64_t at, const RawUnit<DT, E>& r) {
  u32x4_e* d = reinterpret_cast<u32x4_e*>(as_global(static_cast<uint8_t*>(row)) + at * Traits<DT>::B);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.v) / 16); ++i) {
    if constexpr (NT) __builtin_nontemporal_store(r.v[i], d + i);
    else d[i] = r.v[i];
  }
}

// A row as a bounded buffer: elements past its end read as zero and their
// stores are dropped by the hardware's range check, so that no lane needs a
// branch (a branch around a store makes the compiler wait for every store
// before the next row's loads can be used).  The base is the same on every
// lane of the wave; bytes: a multiple of a unit's.
struct RowBuffer {
  __amdgpu_buffer_rsrc_t rsrc;
  __device__ __forceinline__ RowBuffer(const void* base, uint32_t bytes)
      : rsrc(__builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(wave_value((uint64_t)base)), 0, (int)bytes,
                                               kBufferWord3)) {}
};
constexpr int kCachePolicyNt = 2;

template <int DT, int E, bool NT>
__device__ __forceinline__ RawUnit<DT, E> load_unit(const RowBuffer& b, uint32_t at) {
  RawUnit<DT, E> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.v) / 16); ++i)
    r.v[i] = __builtin_amdgcn_raw_buffer_load_b128(b.rsrc, (int)(at * Traits<DT>::B + i * 16), 0, NT ? kCachePolicyNt : 0);
  return r;
}
template <int DT, int E, bool NT>
__device__ __forceinline__ void store_unit(const RowBuffer& b, uint32_t at, const RawUnit<DT, E>& r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.v) / 16); ++i)
    __builtin_amdgcn_raw_buffer_store_b128(r.v[i], b.rsrc, (int)(at * Traits<DT>::B + i * 16), 0, NT ? kCachePolicyNt : 0);
}
// E codes from element `at` of a checkpoint row, codes and scales in a
// buffer each; groups of 1 << glog elements.
template <int E, bool NT>
__device__ __forceinline__ RawUnit<kE4M3, E> load_codes(const RowBuffer& codes, const RowBuffer& scales, uint32_t at, uint32_t glog) {
  RawUnit<kE4M3, E> q;
  constexpr int CP = NT ? kCachePolicyNt : 0;
  if constexpr (E == 4) {
    q.c[0] = __builtin_amdgcn_raw_buffer_load_b32(codes.rsrc, (int)at, 0, CP);
  } else {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 c = __builtin_amdgcn_raw_buffer_load_b64(codes.rsrc, (int)at, 0, CP);
    q.c[0] = c[0];
    q.c[1] = c[1];
  }
  q.s = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(scales.rsrc, (int)((at >> glog) * 4), 0, 0));
  return q;
}

// The first cnt (1..E-1) elements from element `at`; the others read as zero.
template <int DT, int E>
__device__ __forceinline__ RawUnit<DT, E> load_part(const void* row, uint64_t at, uint32_t cnt) {
  using S = typename Traits<DT>::S;
  const S* s = as_global(static_cast<const S*>(row)) + at;
  uint32_t w[E];
#pragma unroll
  for (uint32_t e = 0; e < E; ++e) {
    w[e] = 0;
    if (e < cnt) {
      if constexpr (DT == kBF16) w[e] = s[e];
      else w[e] = __float_as_uint(s[e]);
    }
  }
  RawUnit<DT, E> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.v) / 4); ++i)
    r.v[i / 4][i % 4] = DT == kBF16 ? w[2 * i] | (w[2 * i + 1] << 16) : w[i];
  return r;
}
template <int DT, int E>
__device__ __forceinline__ void store_part(void* row, uint64_t at, uint32_t cnt, const float (&f)[E]) {
  using S = typename Traits<DT>::S;
  S* d = as_global(static_cast<S*>(row)) + at;
#pragma unroll
  for (uint32_t e = 0; e < E; ++e)
    if (e < cnt) d[e] = narrow1<DT>(f[e]);
}

// E codes from element `at` of a checkpoint row: `hidden` codes, then one
// fp32 scale for each group of 1 << glog elements.
template <int E, bool NT>
__device__ __forceinline__ RawUnit<kE4M3, E> load_codes(const uint8_t* row, uint64_t hidden, uint64_t at, uint32_t glog) {
  const uint8_t* r = as_global(row);
  RawUnit<kE4M3, E> q;
  using W = std::conditional_t<E == 4, uint32_t, uint64_t>;
  const W* c = reinterpret_cast<const W*>(r + at);
  const uint64_t w = NT ? __builtin_nontemporal_load(c) : *c;
  q.c[0] = (uint32_t)w;
  if constexpr (E == 8) q.c[1] = (uint32_t)(w >> 32);
  q.s = reinterpret_cast<const float*>(r + hidden)[at >> glog];
  return q;
}

template <int E>
__device__ __forceinline__ void widen_unit(const RawUnit<kBF16, E>& r, float (&f)[E]) {
  widen<kBF16>(r.v[0], f);
}
template <int E>
__device__ __forceinline__ void widen_unit(const RawUnit<kF32, E>& r, float (&f)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = __uint_as_float(r.v[e / 4][e % 4]);
}
// The format's value of a code is the fp32 product of its e4m3 number and
// the group's scale, rounded on its own (never fused into a later sum).
template <int E>
__device__ __forceinline__ void widen_unit(const RawUnit<kE4M3, E>& r, float (&f)[E]) {
#pragma clang fp contract(off)
#pragma unroll
  for (int h = 0; h < E / 4; ++h) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.c[h], false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.c[h], true);
    f[4 * h] = a[0] * r.s;
    f[4 * h + 1] = a[1] * r.s;
    f[4 * h + 2] = b[0] * r.s;
    f[4 * h + 3] = b[1] * r.s;
  }
}
template <int DT, int E>
__device__ __forceinline__ RawUnit<DT, E> narrow_unit(const float (&f)[E]) {
  RawUnit<DT, E> r;
  if constexpr (DT == kBF16) {
    r.v[0] = narrow<kBF16>(f);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) r.v[e / 4][e % 4] = __float_as_uint(f[e]);
  }
  return r;
}

// ---------------------------------------------------------------------------
// Encoding of a unit: the group's largest magnitude over its lanes (a group
// never leaves its wave: its lanes are adjacent and aligned, at most 64),
// then the format's three fp32 steps.
// Magnitudes are compared as integers, which orders NaN above infinity
// above every finite value; a group that holds either gets a NaN scale and
// so decodes to NaN as a whole.
// ---------------------------------------------------------------------------
template <int DT, int E>
__device__ __forceinline__ uint32_t unit_amax(const RawUnit<DT, E>& r) {
  if constexpr (DT == kBF16) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, r.v[0][i] & 0x7fff7fffu));
    return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) m = max(m, r.v[e / 4][e % 4] & 0x7fffffffu);
    return m;
  }
}

// Scaled values exceed 448 by a rounding at most, which encodes as 448 (the
// conversion makes NaN only from 464 up), so they need no clamp.
__device__ __forceinline__ uint32_t e4m3_pack(float a, float b, float c, float d) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false));
}
// The largest value over each aligned run of 1 << sh lanes, on all of them.
__device__ __forceinline__ uint32_t run_max(uint32_t v, uint32_t sh) {
  if (sh >= 1) v = dpp_max<0xB1>(v);   // quad_perm 1,0,3,2
  if (sh >= 2) v = dpp_max<0x4E>(v);   // quad_perm 2,3,0,1
  if (sh >= 3) v = dpp_max<0x141>(v);  // row_half_mirror
  if (sh >= 4) v = dpp_max<0x140>(v);  // row_mirror
  if (sh >= 5) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((uint32_t)a[0], (uint32_t)a[1]);
  }
  if (sh >= 6) {
    const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max((uint32_t)a[0], (uint32_t)a[1]);
  }
  return v;
}

// amax / 448, rounded to nearest: the product with the rounded reciprocal,
// corrected once by its exact remainder.  Equal to the IEEE quotient for
// every mantissa and every exponent that a floored amax can have (checked
// on the CPU), at 3 operations instead of 10.
__device__ __forceinline__ float over_448(float a) {
  const float y = 1.0f / 448.0f, q = a * y;
  return __builtin_fmaf(__builtin_fmaf(-q, 448.0f, a), y, q);
}

// Every lane of the wave calls it (lanes without a unit with zeros).
template <int DT, int E>
__device__ __forceinline__ RawUnit<kE4M3, E> encode_unit(const RawUnit<DT, E>& r, const float (&f)[E], uint32_t glog) {
#pragma clang fp contract(off)
  constexpr uint32_t ELOG = E == 8 ? 3 : 2;
  const uint32_t m = run_max(unit_amax<DT, E>(r), glog - ELOG);
  const float amax = fmaxf(__uint_as_float(m), 0x1p-110f);
  const float inv = 448.0f / amax;
  RawUnit<kE4M3, E> q;
#pragma unroll
  for (int h = 0; h < E / 4; ++h) q.c[h] = e4m3_pack(f[4 * h] * inv, f[4 * h + 1] * inv, f[4 * h + 2] * inv, f[4 * h + 3] * inv);
  q.s = m < 0x7f800000u ? over_448(amax) : __uint_as_float(0x7fc00000u);
  return q;
}

// Stores the codes from element `at`, their group's scale (the group's first
// unit) and, with the row's first unit, the zero bytes that pad the row.
template <int E, bool NT>
__device__ __forceinline__ void store_codes(uint8_t* row, uint64_t hidden, uint64_t row_bytes, uint64_t at, uint32_t glog,
                                            const RawUnit<kE4M3, E>& q) {
  uint8_t* r = as_global(row);
  using W = std::conditional_t<E == 4, uint32_t, uint64_t>;
  W w = q.c[0];
  if constexpr (E == 8) w |= (uint64_t)q.c[1] << 32;
  W* d = reinterpret_cast<W*>(r + at);
  if constexpr (NT) __builtin_nontemporal_store(w, d);
  else *d = w;
  if ((at & ((1u << glog) - 1)) == 0) reinterpret_cast<float*>(r + hidden)[at >> glog] = q.s;
  if (at == 0)
    for (uint64_t b = hidden + 4 * (hidden >> glog); b < row_bytes; b += 4) *reinterpret_cast<float*>(r + b) = 0.0f;
}

// The same without a branch, of a row's codes and scales in a buffer each;
// pad_codes writes the zeros, once a row.
template <int E, bool NT>
__device__ __forceinline__ void store_codes(const RowBuffer& codes, const RowBuffer& scales, uint32_t at, uint32_t glog,
                                            const RawUnit<kE4M3, E>& q) {
  constexpr int CP = NT ? kCachePolicyNt : 0;
  if constexpr (E == 4) {
    __builtin_amdgcn_raw_buffer_store_b32(q.c[0], codes.rsrc, (int)at, 0, CP);
  } else {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{q.c[0], q.c[1]}, codes.rsrc, (int)at, 0, CP);
  }
  const uint32_t off = (at & ((1u << glog) - 1)) == 0 ? (at >> glog) * 4 : 0x7ffffff0u;  // past any end: not stored
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(q.s), scales.rsrc, (int)off, 0, 0);
}
__device__ __forceinline__ void pad_codes(uint8_t* row, uint64_t hidden, uint64_t row_bytes, uint32_t glog, uint32_t lane) {
  const uint64_t b = hidden + 4 * (hidden >> glog) + 4 * lane;
  if (b < row_bytes) *reinterpret_cast<float*>(as_global(row) + b) = 0.0f;
}

// ---------------------------------------------------------------------------
// Sums and maxima over a wave (or its runs of 8 or 16 lanes), on every lane, in
// one fixed order: 16 lanes by DPP, then across these with the gfx950 lane
// swaps, so that no step goes through LDS.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, false));
}
template <int LANES = kWave, class F>
__device__ __forceinline__ float wave_fold(float v, F f) {
  v = f(v, dpp_move<0xB1>(v));   // quad_perm 1,0,3,2
  v = f(v, dpp_move<0x4E>(v));   // quad_perm 2,3,0,1
  v = f(v, dpp_move<0x141>(v));  // row_half_mirror
  if constexpr (LANES == 8) return v;
  v = f(v, dpp_move<0x140>(v));  // row_mirror
  if constexpr (LANES == 16) return v;
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
template <int LANES = kWave>
__device__ __forceinline__ float wave_sum(float v) {
  return wave_fold<LANES>(v, [](float a, float b) { return a + b; });
}
template <int LANES = kWave>
__device__ __forceinline__ float wave_max(float v) {
  return wave_fold<LANES>(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace coll
