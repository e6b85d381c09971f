// Rows of `hidden` elements that stay in the registers of TPR lanes, and the
// wider ones that are gone over in memory: what the norms' kernels share.
#pragma once

#include <algorithm>
#include <type_traits>

#include "token_unit.h"

namespace coll {

namespace {

constexpr int block_of(int tpr) { return tpr < kBlock && kBlock % tpr == 0 ? kBlock : tpr; }
constexpr int waves_of(int tpr) { return tpr < kWave ? 1 : tpr / kWave; }

// Sums over the TPR lanes of a row, R at once.  red: LDS.  One barrier: a
// caller alternates between two arrays, so that a wave that writes an array
// again has passed a barrier that every wave reached after reading it.
template <int TPR, int R>
__device__ __forceinline__ void row_sums(float (&v)[R], float (&red)[R][waves_of(TPR)]) {
#pragma unroll
  for (int k = 0; k < R; ++k) v[k] = wave_sum<std::min(TPR, kWave)>(v[k]);
  if constexpr (TPR > kWave) {
    if (threadIdx.x % kWave == 0) {
#pragma unroll
      for (int k = 0; k < R; ++k) red[k][threadIdx.x / kWave] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < R; ++k) {
      v[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < TPR / kWave; ++w) v[k] += red[k][w];
    }
  }
}

// A row of the register-resident kernels, E elements to a unit.  Without a
// tail (hidden a multiple of E) it is a bounded buffer.  With one, or where
// a wave holds several rows and no one buffer, a lane
// whose unit reaches past the end takes the row's last E elements instead:
// every lane then loads and stores whole units (the elements it shares with
// a neighbour get the same values from both), and only the sums leave out
// the first skip_of() elements, which are not its own.
template <int SRC, int E, bool TAIL>
struct Row;
template <int DT, int E>
struct Row<DT, E, false> {
  RowBuffer b;
  __device__ __forceinline__ Row(const void* base, uint32_t hidden, uint32_t = 0) : b(base, hidden * Traits<DT>::B) {}
  template <bool NT>
  __device__ __forceinline__ RawUnit<DT, E> get(uint32_t u) const { return load_unit<DT, E, NT>(b, u * E); }
  template <bool NT>
  __device__ __forceinline__ void put(uint32_t u, const RawUnit<DT, E>& r) const { store_unit<DT, E, NT>(b, u * E, r); }
};
template <int DT, int E>
struct Row<DT, E, true> {
  uint8_t* base;
  uint32_t last;  // first element of the row's last E
  __device__ __forceinline__ Row(const void* p, uint32_t hidden, uint32_t = 0) : base((uint8_t*)p), last(hidden - E) {}
  template <bool NT>
  __device__ __forceinline__ RawUnit<DT, E> get(uint32_t u) const {
    return load_unit<DT, E, NT>((const void*)base, min(E * u, last));
  }
  template <bool NT>
  __device__ __forceinline__ void put(uint32_t u, const RawUnit<DT, E>& r) const {
    store_unit<DT, E, NT>((void*)base, min(E * u, last), r);
  }
};
template <int E>
struct Row<kE4M3, E, false> {
  RowBuffer codes, scales;
  uint32_t glog;
  __device__ __forceinline__ Row(const void* base, uint32_t hidden, uint32_t g)
      : codes(base, hidden), scales((const uint8_t*)base + hidden, (hidden >> g) * 4), glog(g) {}
  template <bool NT>
  __device__ __forceinline__ RawUnit<kE4M3, E> get(uint32_t u) const { return load_codes<E, NT>(codes, scales, u * E, glog); }
};

template <int E>
struct Row<kE4M3, E, true> {
  const uint8_t* base;
  uint32_t hidden, glog;
  __device__ __forceinline__ Row(const void* p, uint32_t h, uint32_t g) : base((const uint8_t*)p), hidden(h), glog(g) {}
  template <bool NT>
  __device__ __forceinline__ RawUnit<kE4M3, E> get(uint32_t u) const {
    return load_codes<E, NT>(base, hidden, min(E * u, hidden - E), glog);
  }
};

// Elements of unit u that a row with a tail leaves out of its sums (E: all).
template <int E>
__device__ __forceinline__ uint32_t skip_of(uint32_t u, uint32_t hidden) {
  return E * u > hidden - E ? min(E * u - (hidden - E), (uint32_t)E) : 0;
}
// Whether the i-th of a lane's NU units can reach past the end: row_shape
// fills at least half of the lanes' units, except in its narrow classes.
template <int TPR, int NU>
constexpr bool may_end(int i) { return TPR <= kWave || NU == 1 || 2 * i >= NU; }

// A weight vector's units of this lane (ones or zeros where it is absent).
template <int WT, int E, bool TAIL, int NU, int TPR>
__device__ __forceinline__ void load_weights(const void* w, float absent, uint32_t lane, uint32_t hidden,
                                             RawUnit<WT, E> (&out)[NU]) {
  if (w) {
    const Row<WT, E, TAIL> row(w, hidden);
#pragma unroll
    for (int i = 0; i < NU; ++i) out[i] = row.template get<false>(i * TPR + lane);
  } else {
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = absent;
#pragma unroll
    for (int i = 0; i < NU; ++i) out[i] = narrow_unit<WT, E>(f);
  }
}

// The row of this lane's group: workgroups take block_of(TPR) / TPR rows at
// a time.
template <int TPR>
__device__ __forceinline__ uint64_t own_row(uint64_t block) {
  if constexpr (block_of(TPR) == TPR) return block;
  if constexpr (TPR < kWave) return block * (kBlock / TPR) + threadIdx.x / TPR;
  return block * (kBlock / TPR) + __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
}

// ---------------------------------------------------------------------------
// Rows too wide for the registers.
// ---------------------------------------------------------------------------

// Unit u of a row in memory, zeros past its end.  full: whole units of the
// row; part: elements of its last, partial unit.
template <int SRC>
__device__ __forceinline__ RawUnit<SRC, 8> row_unit(const void* row, uint64_t u, uint64_t full, uint32_t part, uint64_t hidden = 0,
                                                    uint32_t glog = 0) {
  if constexpr (SRC == kE4M3) {
    if (u < full) return load_codes<8, false>(static_cast<const uint8_t*>(row), hidden, u * 8, glog);
  } else {
    if (u < full) return load_unit<SRC, 8, false>(row, u * 8);
    if (u == full) return load_part<SRC, 8>(row, u * 8, part);
  }
  return zero_unit<SRC, 8>();
}
template <int DT>
__device__ __forceinline__ void put_unit(void* row, uint64_t u, uint64_t full, uint32_t part, const float (&f)[8]) {
  if (u < full) store_unit<DT, 8, false>(row, u * 8, narrow_unit<DT, 8>(f));
  else if (u == full) store_part<DT, 8>(row, u * 8, part, f);
}
template <int WT>
__device__ __forceinline__ void weight_unit(const void* w, float absent, uint64_t u, uint64_t full, uint32_t part, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = absent;
  if (w) widen_unit(row_unit<WT>(w, u, full, part), f);
}

// Rows whose loads are issued ahead of the row in work: a workgroup of 1024
// lanes has no registers left for one.  Two ahead, with as many registers
// more, were not faster.
template <int TPR>
constexpr int kAhead = TPR < 1024 ? 1 : 0;

// Lanes per row and 8-element units per lane (two 16-byte units of fp32
// each) for a width, 0 lanes: the wide kernels' (or narrower than a unit).
// At least half of the lanes' units lie in the row, except in the narrow
// classes of 16 and 64 lanes.  (8 x 16384 rows of 128 bf16 took 15 us forward
// and 37 us backward with 16 lanes to a row, 32 and 64 us with 64.  8 x 4096
// rows of 2560: 80 and 91 us with checkpoints with 192 lanes, 88 and 94 with
// 256.)
void row_shape(uint64_t hidden, int* tpr, int* nu) {
  const uint64_t units = (hidden + 7) / 8;
  *tpr = hidden < 8      ? 0
         : units <= 32   ? 16
         : units <= 128  ? 64
         : units <= 256  ? 256
         : units <= 384  ? 192
         : units <= 512  ? 256
         : units <= 768  ? 384
         : units <= 1024 ? 512
         : units <= 1536 ? 768
         : units <= 2048 ? 1024
                         : 0;
  *nu = *tpr && units <= (uint64_t)*tpr ? 1 : 2;
}

// Calls f with the shape as compile-time constants.
template <class F>
int with_shape(int tpr, int nu, F f) {
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  if (tpr == 16) return nu == 1 ? f(std::integral_constant<int, 16>(), one) : f(std::integral_constant<int, 16>(), two);
  if (tpr == 64) return nu == 1 ? f(std::integral_constant<int, 64>(), one) : f(std::integral_constant<int, 64>(), two);
  if (tpr == 192) return f(std::integral_constant<int, 192>(), two);
  if (tpr == 256) return nu == 1 ? f(std::integral_constant<int, 256>(), one) : f(std::integral_constant<int, 256>(), two);
  if (tpr == 384) return f(std::integral_constant<int, 384>(), two);
  if (tpr == 512) return f(std::integral_constant<int, 512>(), two);
  if (tpr == 768) return f(std::integral_constant<int, 768>(), two);
  return f(std::integral_constant<int, 1024>(), two);
}

template <class F>
int with_shape(uint64_t hidden, F f) {
  int tpr, nu;
  row_shape(hidden, &tpr, &nu);
  return with_shape(tpr, nu, f);
}

// Workgroups that share a row's columns in the wide backward pass.
uint64_t wide_chunks(uint64_t hidden) { return ((hidden + 7) / 8 + kBlock - 1) / kBlock; }

}  // namespace

}  // namespace coll
