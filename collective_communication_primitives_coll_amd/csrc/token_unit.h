// Device-side building blocks of the token-wise operators (layer norm,
// 8-bit checkpoints, gated activation, vocabulary log probabilities).
//
// A row of `hidden` elements is cut into units of 8 consecutive elements:
// one 16-byte vector of bf16, two of fp32, or 8 bytes of e4m3 codes.  One
// unit size for every type lets a lane own the same columns of the rows,
// the weights, their gradients and the checkpoint.  Rows of an odd width
// leave most units off a 16-byte boundary; gfx950 loads and stores 16
// bytes at any element's address, so these take the same instructions, and
// only a row's last partial unit goes element by element.
#pragma once

#include "device_common.h"

namespace coll {

// A checkpoint row as the source of a unit (beside kF32 and kBF16).
constexpr int kE4M3 = 16;

// 16 bytes at the address of an element.
typedef u32x4 u32x4_e __attribute__((aligned(2)));

template <int SRC> struct RawUnit;
template <> struct RawUnit<kBF16> { u32x4 v[1]; };
template <> struct RawUnit<kF32> { u32x4 v[2]; };
template <> struct RawUnit<kE4M3> {
  uint2 c;  // 8 codes
  float s;  // their group's scale
};

template <int SRC> __device__ __forceinline__ RawUnit<SRC> zero_unit() {
  RawUnit<SRC> r;
  if constexpr (SRC == kE4M3) {
    r.c = make_uint2(0, 0);
    r.s = 0.0f;
  } else {
#pragma unroll
    for (auto& v : r.v) v = u32x4{0, 0, 0, 0};
  }
  return r;
}

// Unit u of a row at `row` (bf16 or fp32).
template <int DT, bool NT>
__device__ __forceinline__ RawUnit<DT> load_unit(const void* row, uint64_t u) {
  const u32x4_e* s = reinterpret_cast<const u32x4_e*>(as_global(static_cast<const uint8_t*>(row)) + u * (8 * Traits<DT>::B));
  RawUnit<DT> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.v) / 16); ++i) {
    if constexpr (NT) r.v[i] = __builtin_nontemporal_load(s + i);
    else r.v[i] = s[i];
  }
  return r;
}
template <int DT, bool NT>
__device__ __forceinline__ void store_unit(void* row, uint64_t u, const RawUnit<DT>& r) {
  u32x4_e* d = reinterpret_cast<u32x4_e*>(as_global(static_cast<uint8_t*>(row)) + u * (8 * Traits<DT>::B));
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.v) / 16); ++i) {
    if constexpr (NT) __builtin_nontemporal_store(r.v[i], d + i);
    else d[i] = r.v[i];
  }
}

// The first cnt (1..7) elements of unit u; the others read as zero.
template <int DT>
__device__ __forceinline__ RawUnit<DT> load_part(const void* row, uint64_t u, uint32_t cnt) {
  using S = typename Traits<DT>::S;
  const S* s = as_global(static_cast<const S*>(row)) + u * 8;
  uint32_t w[8];
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e) {
    w[e] = 0;
    if (e < cnt) {
      if constexpr (DT == kBF16) w[e] = s[e];
      else w[e] = __float_as_uint(s[e]);
    }
  }
  RawUnit<DT> r;
  if constexpr (DT == kBF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[0][i] = w[2 * i] | (w[2 * i + 1] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i / 4][i % 4] = w[i];
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void store_part(void* row, uint64_t u, uint32_t cnt, const float (&f)[8]) {
  using S = typename Traits<DT>::S;
  S* d = as_global(static_cast<S*>(row)) + u * 8;
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e)
    if (e < cnt) d[e] = narrow1<DT>(f[e]);
}

// Unit u of a checkpoint row: `hidden` codes, then one fp32 scale for each
// group of 1 << gsh units.
template <bool NT>
__device__ __forceinline__ RawUnit<kE4M3> load_codes(const uint8_t* row, uint64_t hidden, uint64_t u, uint32_t gsh) {
  const uint8_t* r = as_global(row);
  RawUnit<kE4M3> q;
  const uint64_t* c = reinterpret_cast<const uint64_t*>(r) + u;
  const uint64_t w = NT ? __builtin_nontemporal_load(c) : *c;
  q.c = make_uint2((uint32_t)w, (uint32_t)(w >> 32));
  q.s = reinterpret_cast<const float*>(r + hidden)[u >> gsh];
  return q;
}

__device__ __forceinline__ void widen_unit(const RawUnit<kBF16>& r, float (&f)[8]) { widen<kBF16>(r.v[0], f); }
__device__ __forceinline__ void widen_unit(const RawUnit<kF32>& r, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(r.v[e / 4][e % 4]);
}
// The format's value of a code is the fp32 product of its e4m3 number and
// the group's scale, rounded on its own (never fused into a later sum).
__device__ __forceinline__ void widen_unit(const RawUnit<kE4M3>& r, float (&f)[8]) {
#pragma clang fp contract(off)
  const uint32_t w[2] = {r.c.x, r.c.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
    f[4 * h] = a[0] * r.s;
    f[4 * h + 1] = a[1] * r.s;
    f[4 * h + 2] = b[0] * r.s;
    f[4 * h + 3] = b[1] * r.s;
  }
}
template <int DT>
__device__ __forceinline__ RawUnit<DT> narrow_unit(const float (&f)[8]) {
  RawUnit<DT> r;
  if constexpr (DT == kBF16) {
    r.v[0] = narrow<kBF16>(f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e / 4][e % 4] = __float_as_uint(f[e]);
  }
  return r;
}

// ---------------------------------------------------------------------------
// Encoding of a unit: the group's largest magnitude over its 1 << gsh lanes
// (a group never leaves its wave: at most 512 elements, and the lanes of a
// group are adjacent and aligned), then the format's three fp32 steps.
// Magnitudes are compared as integers, which orders NaN above infinity
// above every finite value; a group that holds either gets a NaN scale and
// so decodes to NaN as a whole.
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ uint32_t unit_amax(const RawUnit<DT>& r) {
  if constexpr (DT == kBF16) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, r.v[0][i] & 0x7fff7fffu));
    return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, r.v[e / 4][e % 4] & 0x7fffffffu);
    return m;
  }
}

__device__ __forceinline__ uint32_t e4m3_pack(float a, float b, float c, float d) {
  a = __builtin_amdgcn_fmed3f(a, -448.0f, 448.0f);
  b = __builtin_amdgcn_fmed3f(b, -448.0f, 448.0f);
  c = __builtin_amdgcn_fmed3f(c, -448.0f, 448.0f);
  d = __builtin_amdgcn_fmed3f(d, -448.0f, 448.0f);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Every lane of the wave calls it (lanes without a unit with zeros).
template <int DT>
__device__ __forceinline__ RawUnit<kE4M3> encode_unit(const RawUnit<DT>& r, const float (&f)[8], uint32_t gsh) {
#pragma clang fp contract(off)
  uint32_t m = unit_amax<DT>(r);
  for (uint32_t off = 1; off < (1u << gsh); off <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, (int)off));
  const float amax = fmaxf(__uint_as_float(m), 0x1p-110f);
  const float inv = 448.0f / amax;
  RawUnit<kE4M3> q;
  q.c.x = e4m3_pack(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
  q.c.y = e4m3_pack(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
  q.s = m < 0x7f800000u ? amax / 448.0f : __uint_as_float(0x7fc00000u);
  return q;
}

// Stores unit u's codes, its group's scale (first unit of the group) and,
// with the row's first unit, the zero bytes that pad the row.
template <bool NT>
__device__ __forceinline__ void store_codes(uint8_t* row, uint64_t hidden, uint64_t row_bytes, uint64_t u, uint32_t gsh,
                                            const RawUnit<kE4M3>& q) {
  uint8_t* r = as_global(row);
  const uint64_t w = (uint64_t)q.c.x | ((uint64_t)q.c.y << 32);
  if constexpr (NT) __builtin_nontemporal_store(w, reinterpret_cast<uint64_t*>(r) + u);
  else reinterpret_cast<uint64_t*>(r)[u] = w;
  if ((u & ((1u << gsh) - 1)) == 0) reinterpret_cast<float*>(r + hidden)[u >> gsh] = q.s;
  if (u == 0) {
    const uint64_t used = hidden + 4 * (hidden >> (gsh + 3));
    for (uint64_t b = used; b < row_bytes; b += 4) *reinterpret_cast<float*>(r + b) = 0.0f;
  }
}

// ---------------------------------------------------------------------------
// Sums and maxima over a wave, on every lane, in one fixed order: rows of 16
// lanes by DPP, then across rows with the gfx950 lane swaps, so that no
// step goes through LDS.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, false));
}
template <class F>
__device__ __forceinline__ float wave_fold(float v, F f) {
  v = f(v, dpp_move<0xB1>(v));   // quad_perm 1,0,3,2
  v = f(v, dpp_move<0x4E>(v));   // quad_perm 2,3,0,1
  v = f(v, dpp_move<0x141>(v));  // row_half_mirror
  v = f(v, dpp_move<0x140>(v));  // row_mirror
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_fold(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_fold(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace coll
