// RMS norm over every rank's token rows, with the residual's addition before
// it and an output in the rows' type or in 8 bits, and its backward pass with
// the weights' gradient summed over all rows and all ranks.
//
//   forward   h = x + residual (rounded to the rows' type: the next layer and
//             the backward pass see the same h),
//             r = 1 / sqrt(mean h^2 + eps),  y = h r gamma
//   backward  n = h r,  w = dy gamma,
//             dx = r (w - n mean(w n)) + dh,
//             dgamma = sum dy n   (over rows and ranks)
//
// Bound by HBM: 8 bytes an element either way in bf16 with a residual,
// against some 10 fp32 operations.  As in layer norm, a row is read once and
// stays in the registers of TPR lanes between its sum and its result, and the
// backward pass keeps a lane on the same columns for all rows of its
// workgroup; the partial sums of the weights' gradient are added in a fixed
// order by the norms' common join.
//
// Sums are fp32; bf16 results are narrowed once, 8-bit codes come from the
// fp32 values.  Squares leave fp32's range long before the values do: a row
// whose sum of squares is out of it (or, with eps next to nothing, far below
// it) is summed again with its values scaled by a power of two.
#include "token_rows.h"

namespace coll {

namespace {

// Sums of squares that are taken as they are; others again, scaled: by 2^-80,
// which brings values below 2^48 and 2^31 of their squares below 2^127, or by
// 2^100, which brings the smallest denormal to 2^-49.  eps above 2^-80
// outweighs any sum below kLeast, and is not scaled out of range below it.
constexpr float kMost = 0x1p120f, kLeast = 0x1p-90f, kDown = 0x1p-80f, kUp = 0x1p100f, kEpsLeast = 0x1p-80f;
__device__ __forceinline__ float square_scale(float q, float eps) {
  return !(q < kMost) ? kDown : q < kLeast && eps < kEpsLeast ? kUp : 1.0f;
}
// 1 / sqrt(mean h^2 + eps) from the sum of (h k)^2, as the product of two
// factors: the root of the scaled sum, and k.  Their product may leave fp32's
// range where values times it do not (rows below 2^-128, whose values are all
// denormal), so a value takes one after the other, in the order that stays in
// range: by 2^100 before the root, by 2^-80 after it.  1 is exact either way.
struct Rstd {
  float first, second;
  __device__ __forceinline__ Rstd(float q, float k, float hidden, float eps) {
    const float root = rsqrtf(q / hidden + eps * k * k);
    first = k > 1.0f ? k : root;
    second = k > 1.0f ? root : k;
  }
  __device__ __forceinline__ float times(float v) const { return v * first * second; }
  __device__ __forceinline__ float value() const { return first * second; }
};

template <int DT, int E>
__device__ __forceinline__ RawUnit<DT, E> add_units(const RawUnit<DT, E>& a, const RawUnit<DT, E>& b) {
  float f[E], g[E];
  widen_unit(a, f);
  widen_unit(b, g);
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] += g[e];
  return narrow_unit<DT, E>(f);
}

// ---------------------------------------------------------------------------
// Forward.  Grid (runs of rows, ranks), no walk, and the weights asked for
// after the sums, as in layer norm.  h is stored after the sums too: it may
// replace x or the residual, whose rows of an odd width have lanes that share
// elements.  8 x 4096 x 7168 bf16 with a residual: 308 us (6.1 TB/s; 1:1 streams
// reach 6.24), without 151 us; to 8 bits 270 and 123 us.
// ---------------------------------------------------------------------------
// Rows to a lane: one where a row with its residual, or half a workgroup's lanes
// and more, keep enough loads in flight.  us with one row and with two, bf16
// with a residual: 8 x 4096 x 8192 353 and 370, 4096 174 and 176, 2560 114 and
// 111, 8 x 131072 x 64 96 and 80; fp32 8 x 2048 x 7168 329 and 336, 4096 176 and
// 185; without: bf16 8 x 4096 x 8192 170 and 178, 5120 110 and 107, in 8 bits
// 7168 131 and 123.
template <int DT, int TPR, bool RES, bool FP8>
constexpr int rows_of() {
  if (TPR == 1024 && DT == kBF16) return 1;
  return (RES ? TPR >= (DT == kF32 ? 192 : 256) : TPR >= 512 && !FP8) ? 1 : 2;
}

template <int DT, int WT, int TPR, int NU, bool TAIL, bool RES, bool FP8, int E = kElems<DT>>
__global__ __launch_bounds__(block_of(TPR)) void rms_forward_kernel(RmsArgs a) {
  constexpr int kRows = rows_of<DT, TPR, RES, FP8>();
  __shared__ float red[2][kRows][waves_of(TPR)];
  const int rank = blockIdx.y;
  const uint32_t lane = threadIdx.x % TPR, H = (uint32_t)a.hidden;
  const uint64_t row_bytes = (uint64_t)H * Traits<DT>::B;
  const uint64_t row0 = own_row<TPR>(blockIdx.x) * kRows;
  if (row0 >= a.rows) return;
  RawUnit<DT, E> raw[kRows][NU], res[kRows][NU];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    // past the last row: row0 again (its results are not stored)
    const uint64_t off = (row0 + (row0 + k < a.rows ? k : 0)) * row_bytes;
    const Row<DT, E, TAIL> x(static_cast<const uint8_t*>(a.x[rank]) + off, H);
#pragma unroll
    for (int i = 0; i < NU; ++i) raw[k][i] = x.template get<true>(i * TPR + lane);
    if constexpr (RES) {
      const Row<DT, E, TAIL> r(static_cast<const uint8_t*>(a.res[rank]) + off, H);
#pragma unroll
      for (int i = 0; i < NU; ++i) res[k][i] = r.template get<true>(i * TPR + lane);
    }
  }
  // sum of squares of row k, the values times `by`
  auto squares = [&](int k, float by) {
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t skip = TAIL && may_end<TPR, NU>(i) ? skip_of<E>(i * TPR + lane, H) : 0;
      float f[E];
      widen_unit(raw[k][i], f);
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) {
        const float v = f[e] * by;
        q = TAIL && may_end<TPR, NU>(i) && e < skip ? q : __builtin_fmaf(v, v, q);
      }
    }
    return q;
  };
  float q[kRows], by[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if constexpr (RES) {
#pragma unroll
      for (int i = 0; i < NU; ++i) raw[k][i] = add_units<DT, E>(raw[k][i], res[k][i]);
    }
    q[k] = squares(k, 1.0f);
  }
  row_sums<TPR, kRows>(q, red[0]);
  bool scaled = false;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    by[k] = square_scale(q[k], a.eps);
    scaled = scaled || by[k] != 1.0f;
  }
  if (scaled) {  // the same on all lanes of the rows
#pragma unroll
    for (int k = 0; k < kRows; ++k) q[k] = squares(k, by[k]);
    row_sums<TPR, kRows>(q, red[1]);
  }
  RawUnit<WT, E> gamma[NU];
  load_weights<WT, E, TAIL, NU, TPR>(a.gamma[rank], 1.0f, lane, H, gamma);
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const uint64_t row = row0 + k;
    if (row >= a.rows) break;
    const Rstd rstd(q[k], by[k], (float)H, a.eps);
    if (RES && a.h[rank]) {
      const Row<DT, E, TAIL> h(static_cast<uint8_t*>(a.h[rank]) + row * row_bytes, H);
#pragma unroll
      for (int i = 0; i < NU; ++i) h.template put<true>(i * TPR + lane, raw[k][i]);
    }
    uint8_t* y8 = FP8 ? a.y8[rank] + row * a.row_bytes : nullptr;
    // (of a row to itself; where a wave holds several, by their addresses)
    const RowBuffer codes(y8, FP8 ? H : 0), scales(FP8 ? y8 + H : nullptr, FP8 ? (H >> a.glog) * 4 : 0);
    const bool plain = !FP8 || a.y[rank];
    const Row<DT, E, TAIL> y(static_cast<uint8_t*>(a.y[rank]) + row * row_bytes, H);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float f[E], g[E];
      widen_unit(raw[k][i], f);
      widen_unit(gamma[i], g);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = rstd.times(f[e]) * g[e];
      if (plain) y.template put<true>(i * TPR + lane, narrow_unit<DT, E>(f));
      if constexpr (FP8) {
        const uint32_t u = i * TPR + lane;
        const RawUnit<kE4M3, E> code = encode_values<E>(f, a.glog);
        if constexpr (TPR >= kWave) store_codes<E, true>(codes, scales, E * u, a.glog, code);
        else if (E * u < H) store_codes<E, true>(y8, H, a.row_bytes, E * u, a.glog, code);
      }
    }
    if constexpr (FP8 && TPR >= kWave) pad_codes(y8, H, a.row_bytes, a.glog, lane);
    if (lane == 0 && a.rstd[rank]) as_global(a.rstd[rank])[row] = rstd.value();
  }
}

// Rows too wide for the registers (or narrower than one unit): units of 8
// elements in every type, each row gone over twice; the second time it comes
// from the caches.
template <int DT, int WT, bool RES, bool FP8>
__global__ __launch_bounds__(1024) void rms_forward_wide_kernel(RmsArgs a) {
  constexpr int TPR = 1024;
  __shared__ float red[2][1][TPR / kWave];
  const int rank = blockIdx.y;
  const uint64_t H = a.hidden, full = H / 8, units = (H + 7) / 8;
  const uint32_t part = (uint32_t)(H % 8);
  // every lane takes part in every step (the encoding exchanges lanes)
  const uint64_t steps = (units + TPR - 1) / TPR;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint64_t off = row * H * Traits<DT>::B;
    const uint8_t* x = static_cast<const uint8_t*>(a.x[rank]) + off;
    const uint8_t* res = RES ? static_cast<const uint8_t*>(a.res[rank]) + off : nullptr;
    uint8_t* h = RES && a.h[rank] ? static_cast<uint8_t*>(a.h[rank]) + off : nullptr;
    uint8_t* y = !FP8 || a.y[rank] ? static_cast<uint8_t*>(a.y[rank]) + off : nullptr;
    uint8_t* y8 = FP8 ? a.y8[rank] + row * a.row_bytes : nullptr;
    float f[8], q[1] = {0.0f};
    // a unit of h: from x and the residual, or, once it is stored, read back
    // (x may have been replaced by it)
    auto unit = [&](uint64_t u, bool again) {
      if (RES && again && h) {
        widen_unit(row_unit<DT>(h, u, full, part), f);
        return;
      }
      RawUnit<DT, 8> v = row_unit<DT>(x, u, full, part);
      if constexpr (RES) v = add_units<DT, 8>(v, row_unit<DT>(res, u, full, part));
      widen_unit(v, f);
    };
    for (uint64_t k = 0; k < steps; ++k) {
      const uint64_t u = k * TPR + threadIdx.x;
      unit(u, false);
      if (RES && h) put_unit<DT>(h, u, full, part, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) q[0] = __builtin_fmaf(f[e], f[e], q[0]);
    }
    row_sums<TPR, 1>(q, red[0]);
    const float by = square_scale(q[0], a.eps);
    if (by != 1.0f) {
      q[0] = 0.0f;
      for (uint64_t k = 0; k < steps; ++k) {
        unit(k * TPR + threadIdx.x, true);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[0] = __builtin_fmaf(f[e] * by, f[e] * by, q[0]);
      }
    }
    // a barrier either way: a wave that writes red[0] for the next row has
    // passed one that every wave reached after reading it
    float s[1] = {q[0]};
    if (by != 1.0f) row_sums<TPR, 1>(s, red[1]);
    else __syncthreads();
    const Rstd rstd(s[0], by, (float)H, a.eps);
    for (uint64_t k = 0; k < steps; ++k) {
      const uint64_t u = k * TPR + threadIdx.x;
      unit(u, true);
      float g[8];
      weight_unit<WT>(a.gamma[rank], 1.0f, u, full, part, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = rstd.times(f[e]) * g[e];
      if (y) put_unit<DT>(y, u, full, part, f);
      if constexpr (FP8) {
        const RawUnit<kE4M3, 8> code = encode_values<8>(f, a.glog);
        if (u < full) store_codes<8, true>(y8, H, a.row_bytes, u * 8, a.glog, code);
      }
    }
    if (threadIdx.x == 0 && a.rstd[rank]) as_global(a.rstd[rank])[row] = rstd.value();
  }
}

// ---------------------------------------------------------------------------
// Backward.  A workgroup takes every gridDim.x-th run of rows, through all
// ranks of the launch, and writes its partial sums to ws[blockIdx.x][hidden].
// h and dy are asked for one row ahead; dh, which is needed last, with its own
// row: the card works best in a narrow window of memory (8 x 4096 x 7168 bf16:
// 307 us, 6.1 TB/s, and 321 with dh a row ahead as well; two rows ahead 321).
// ---------------------------------------------------------------------------
// Whether dx is written through the L2 at once (device scope) rather than past
// it (non-temporal).  By lanes to a row, us of either with a residual, bf16:
// 256 lanes (4096 columns) 171 and 186, 384 (5120) 114 and 119, 512 (7168) 319
// and 307, 768 (12288) 289 and 281, 1024 (16384) 371 and 367.
template <int TPR>
constexpr bool kWriteThrough = TPR >= kWave && TPR <= 384;

// Units of dx.  The base is the same on every lane that shares a buffer.
template <int DT, int E, int TPR, bool TAIL>
struct DxRow {
  RowBuffer b;
  Row<DT, E, TAIL> row;
  uint32_t last;  // first element of the row's last E
  __device__ __forceinline__ DxRow(void* base, uint32_t hidden)
      : b(base, kWriteThrough<TPR> ? hidden * Traits<DT>::B : 0), row(base, hidden), last(hidden - E) {}
  __device__ __forceinline__ void put(uint32_t u, const RawUnit<DT, E>& r) const {
    if constexpr (kWriteThrough<TPR>) {
      const uint32_t at = TAIL ? min(E * u, last) : E * u;
      __builtin_amdgcn_raw_buffer_store_b128(r.v[0], b.rsrc, (int)(at * Traits<DT>::B), 0, kCachePolicySc1);
    } else {
      row.template put<true>(u, r);
    }
  }
};

// Sum over a wave's four rows of 16 lanes, on every lane.
__device__ __forceinline__ float rows_sum(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int DT, int WT, int TPR, int NU, bool TAIL, bool DH>
__global__ __launch_bounds__(block_of(TPR)) void rms_backward_kernel(RmsArgs a) {
  constexpr int E = kElems<DT>, RPB = block_of(TPR) / TPR, AHEAD = kAhead<TPR>;
  __shared__ float red[2][1][waves_of(TPR)];
  __shared__ float fold[RPB > 1 ? kBlock / kWave : 1][RPB > 1 ? NU * E * TPR : 1];
  const uint32_t lane = threadIdx.x % TPR, H = (uint32_t)a.hidden;
  const uint64_t row_bytes = (uint64_t)H * Traits<DT>::B;
  const uint64_t stride = (uint64_t)gridDim.x * RPB;
  // a place in the ranks' rows, one rank after the other
  struct Place {
    uint64_t row;
    int rank;
    __device__ __forceinline__ void settle(const RmsArgs& a) {
      while (row >= a.rows && rank < a.ranks) {
        row -= a.rows;
        ++rank;
      }
    }
  };
  Place at{own_row<TPR>(blockIdx.x), 0};
  at.settle(a);
  float dg[NU][E] = {};
  if (at.rank < a.ranks) {
    // AHEAD + 1 buffers; the loop is unrolled over them, since moving a
    // loaded register to another waits for its load
    RawUnit<DT, E> bh[AHEAD + 1][NU], bd[AHEAD + 1][NU], br[DH ? NU : 1];
    float bs[AHEAD + 1];
    auto fetch = [&](const Place& r, auto K) {
      constexpr int k = decltype(K)::value;
      const uint64_t off = r.row * row_bytes;
      const Row<DT, E, TAIL> rh(static_cast<const uint8_t*>(a.h[r.rank]) + off, H);
      const Row<DT, E, TAIL> rd(static_cast<const uint8_t*>(a.x[r.rank]) + off, H);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        bh[k][i] = rh.template get<true>(i * TPR + lane);
        bd[k][i] = rd.template get<true>(i * TPR + lane);
      }
      bs[k] = ld_const(a.rstd[r.rank] + r.row);
    };
    fetch(at, std::integral_constant<int, 0>());
    RawUnit<WT, E> gamma[NU];
    int held = -1, turn = 0;
    // one row from buffer K; whether there is another
    auto step = [&](auto K) {
      constexpr int k = decltype(K)::value;
      if (at.rank != held) {
        held = at.rank;
        load_weights<WT, E, TAIL, NU, TPR>(a.gamma[held], 1.0f, lane, H, gamma);
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (auto& v : gamma[i].v) asm volatile("" : "+v"(v));  // waited for here, not in every step
      }
      // after the last row: that row again, so that every step issues the
      // same and the compiler can count what it waits for
      Place next{at.row + stride, at.rank};
      next.settle(a);
      const bool more = next.rank < a.ranks;
      if (!more) next = at;
      if constexpr (DH) {
        const Row<DT, E, TAIL> rr(static_cast<const uint8_t*>(a.res[at.rank]) + at.row * row_bytes, H);
#pragma unroll
        for (int i = 0; i < NU; ++i) br[i] = rr.template get<true>(i * TPR + lane);
      }
      if constexpr (AHEAD > 0) fetch(next, std::integral_constant<int, (k + 1) % (AHEAD + 1)>());
      const float rstd = bs[k];
      float n[NU][E], w[NU][E], s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const uint32_t skip = TAIL && may_end<TPR, NU>(i) ? skip_of<E>(i * TPR + lane, H) : 0;
        float d[E], g[E];
        widen_unit(bh[k][i], n[i]);
        widen_unit(bd[k][i], d);
        widen_unit(gamma[i], g);
#pragma unroll
        for (uint32_t e = 0; e < E; ++e) {
          n[i][e] *= rstd;
          w[i][e] = d[e] * g[e];
          const bool own = !(TAIL && may_end<TPR, NU>(i) && e < skip);
          dg[i][e] += own ? d[e] * n[i][e] : 0.0f;
          s[0] += own ? w[i][e] * n[i][e] : 0.0f;
        }
      }
      if (DH && TAIL && H % E) {
        // dx may take dh's place, and lanes of a row of an odd width share
        // elements: dh has arrived on every wave before any of them stores
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (auto& v : br[i].v) asm volatile("" : "+v"(v));
      }
      row_sums<TPR, 1>(s, red[turn]);
      turn ^= 1;
      const float c = s[0] / (float)H;
      const DxRow<DT, E, TPR, TAIL> dx(static_cast<uint8_t*>(a.y[at.rank]) + at.row * row_bytes, H);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        float r[E];
        if constexpr (DH) widen_unit(br[i], r);
#pragma unroll
        for (int e = 0; e < E; ++e) w[i][e] = rstd * (w[i][e] - n[i][e] * c) + (DH ? r[e] : 0.0f);
        dx.put(i * TPR + lane, narrow_unit<DT, E>(w[i]));
      }
      if constexpr (AHEAD == 0) fetch(next, K);
      at = next;
      return more;
    };
    while (true) {
      if (!step(std::integral_constant<int, 0>())) break;
      if constexpr (AHEAD > 0)
        if (!step(std::integral_constant<int, 1>())) break;
    }
  }
  float* ws = a.ws + (uint64_t)blockIdx.x * H;
  if constexpr (RPB > 1) {
    // a wave's groups of lanes add their sums, then the first group those of
    // the workgroup's waves, in their order (one group after the other: 8 x
    // 500 x 256 bf16 15.0 us for 13.1)
    const uint32_t mine = threadIdx.x / TPR, wave = threadIdx.x / kWave;
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if constexpr (TPR < kWave) dg[i][e] = rows_sum(dg[i][e]);
        if (mine % (RPB * kWave / kBlock) == 0) fold[wave][(i * E + e) * TPR + lane] = dg[i][e];
      }
    __syncthreads();
    if (mine) return;
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = 1; k < kBlock / kWave; ++k) dg[i][e] += fold[k][(i * E + e) * TPR + lane];
  }
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const uint32_t u = i * TPR + lane;
    if (E * u + E <= H) {
      store_unit<kF32, E, false>((void*)ws, E * u, narrow_unit<kF32, E>(dg[i]));
    } else if (TAIL && E * u < H) {
      // the row's last E elements, of which the last H % E are this unit's
      const uint32_t skip = skip_of<E>(u, H);
#pragma unroll
      for (uint32_t e = 0; e < E; ++e)
        if (e >= skip) as_global(ws)[H - E + e] = dg[i][e];
    }
  }
}

// Rows too wide for the registers, in two kernels: the weights' gradient by
// columns (a lane keeps its 8 columns over the workgroup's rows), then the
// rows, each gone over twice.  The columns come first, so that dx may be
// dy's own buffer.
template <int DT>
__global__ __launch_bounds__(kBlock) void rms_backward_wide_columns_kernel(RmsArgs a, uint32_t splits) {
  const uint64_t H = a.hidden, full = H / 8, row_bytes = H * Traits<DT>::B;
  const uint32_t part = (uint32_t)(H % 8), split = blockIdx.x % splits;
  const uint64_t u = (uint64_t)(blockIdx.x / splits) * kBlock + threadIdx.x;
  float dg[8] = {};
  for (int rank = 0; rank < a.ranks; ++rank)
    for (uint64_t row = split; row < a.rows; row += splits) {
      float fh[8], fd[8];
      widen_unit(row_unit<DT>(static_cast<const uint8_t*>(a.h[rank]) + row * row_bytes, u, full, part), fh);
      widen_unit(row_unit<DT>(static_cast<const uint8_t*>(a.x[rank]) + row * row_bytes, u, full, part), fd);
      const float rstd = as_global(a.rstd[rank])[row];
#pragma unroll
      for (int e = 0; e < 8; ++e) dg[e] += fd[e] * (fh[e] * rstd);
    }
  put_unit<kF32>(a.ws + (uint64_t)split * H, u, full, part, dg);
}

template <int DT, int WT, bool DH>
__global__ __launch_bounds__(1024) void rms_backward_wide_rows_kernel(RmsArgs a) {
  constexpr int TPR = 1024;
  __shared__ float red[2][1][TPR / kWave];
  const int rank = blockIdx.y;
  const uint64_t H = a.hidden, full = H / 8, units = (H + 7) / 8;
  const uint32_t part = (uint32_t)(H % 8);
  int turn = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint64_t off = row * H * Traits<DT>::B;
    const uint8_t* h = static_cast<const uint8_t*>(a.h[rank]) + off;
    const uint8_t* dy = static_cast<const uint8_t*>(a.x[rank]) + off;
    const float rstd = as_global(a.rstd[rank])[row];
    float n[8], w[8], g[8], s[1] = {0.0f};
    auto unit = [&](uint64_t u) {
      widen_unit(row_unit<DT>(h, u, full, part), n);
      widen_unit(row_unit<DT>(dy, u, full, part), w);
      weight_unit<WT>(a.gamma[rank], 1.0f, u, full, part, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] *= rstd;
        w[e] *= g[e];
      }
    };
    for (uint64_t u = threadIdx.x; u < units; u += TPR) {
      unit(u);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += w[e] * n[e];
    }
    row_sums<TPR, 1>(s, red[turn]);
    turn ^= 1;
    const float c = s[0] / (float)H;
    for (uint64_t u = threadIdx.x; u < units; u += TPR) {
      unit(u);
      float r[8] = {};
      if constexpr (DH) widen_unit(row_unit<DT>(static_cast<const uint8_t*>(a.res[rank]) + off, u, full, part), r);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = rstd * (w[e] - n[e] * c) + r[e];
      put_unit<DT>(static_cast<uint8_t*>(a.y[rank]) + off, u, full, part, w);
    }
  }
}

// The kernel that takes rows of a width: lanes to a row and units of 8 elements
// to a lane (0: the wide ones).  Codes want a group's lanes in one run of a
// row's, at most a wave: rows of 16 lanes take 64 for wider groups, and fp32
// rows of groups of 512 have 8 elements to a lane (5 x 11770 x 512: 30 us, and
// 468 in the wide kernel).
constexpr uint64_t kLanesGroup4 = 4 * kWave;  // widest group of lanes with 4 elements
void rms_shape(int dtype, uint64_t hidden, uint64_t group, int* tpr, int* nu) {
  row_shape(hidden, tpr, nu);
  const uint64_t elems = dtype == kF32 && group <= kLanesGroup4 ? 4 : 8;
  if (*tpr == 16 && group > 16 * elems) {
    *tpr = 64;
    *nu = 1;
  }
}

// The forward pass's arguments n rows on.
void skip_rows(RmsArgs& a, uint64_t n, uint64_t row_bytes) {
  for (int r = 0; r < a.ranks; ++r) {
    a.x[r] = (const uint8_t*)a.x[r] + n * row_bytes;
    if (a.res[r]) a.res[r] = (const uint8_t*)a.res[r] + n * row_bytes;
    if (a.h[r]) a.h[r] = (uint8_t*)a.h[r] + n * row_bytes;
    if (a.y[r]) a.y[r] = (uint8_t*)a.y[r] + n * row_bytes;
    if (a.rstd[r]) a.rstd[r] += n;
    if (a.y8[r]) a.y8[r] += n * a.row_bytes;
  }
}

template <int DT, int WT, bool RES, bool FP8>
int forward_t(const RmsArgs& a, hipStream_t s) {
  int tpr, nu;
  const uint64_t group = FP8 ? uint64_t{1} << a.glog : 0;
  rms_shape(DT, a.hidden, group, &tpr, &nu);
  if (!tpr) {
    const dim3 grid((uint32_t)std::min<uint64_t>(a.rows, 65536), a.ranks);
    hipLaunchKernelGGL((rms_forward_wide_kernel<DT, WT, RES, FP8>), grid, dim3(1024), 0, s, a);
    return (int)hipGetLastError();
  }
  return with_shape(tpr, nu, [&](auto T, auto N) {
    constexpr int TPR = decltype(T)::value, NU = decltype(N)::value * 8 / kElems<DT>, RPB = block_of(TPR) / TPR;
    constexpr bool PACKED = TPR < kWave;  // several rows to a wave
    const uint64_t run = RPB * rows_of<DT, TPR, RES, FP8>();
    const dim3 block(block_of(TPR));
    const uint64_t most = most_blocks(block.x) * run;
    RmsArgs part = a;
    for (uint64_t left = a.rows; left; skip_rows(part, part.rows, a.hidden * Traits<DT>::B)) {
      part.rows = std::min(left, most);
      left -= part.rows;
      const dim3 grid((uint32_t)((part.rows + run - 1) / run), a.ranks);
      if constexpr (FP8) {  // whole groups, so whole units
        if constexpr (DT == kF32 && !PACKED) {
          if (group > kLanesGroup4) hipLaunchKernelGGL((rms_forward_kernel<DT, WT, TPR, NU / 2, false, RES, true, 8>), grid, block, 0, s, part);
          else hipLaunchKernelGGL((rms_forward_kernel<DT, WT, TPR, NU, false, RES, true>), grid, block, 0, s, part);
        } else {
          hipLaunchKernelGGL((rms_forward_kernel<DT, WT, TPR, NU, PACKED, RES, true>), grid, block, 0, s, part);
        }
      } else {
        if (PACKED || a.hidden % kElems<DT>) hipLaunchKernelGGL((rms_forward_kernel<DT, WT, TPR, NU, true, RES, false>), grid, block, 0, s, part);
        else hipLaunchKernelGGL((rms_forward_kernel<DT, WT, TPR, NU, PACKED, RES, false>), grid, block, 0, s, part);
      }
      if (const int e = (int)hipGetLastError()) return e;
    }
    return 0;
  });
}

template <int DT, int WT, bool DH>
int backward_t(const RmsArgs& a, uint32_t groups, hipStream_t s) {
  int tpr, nu;
  row_shape(a.hidden, &tpr, &nu);
  if (!tpr) {
    const dim3 cols((uint32_t)(wide_chunks(a.hidden) * groups)), rows((uint32_t)std::min<uint64_t>(a.rows, 65536), a.ranks);
    hipLaunchKernelGGL((rms_backward_wide_columns_kernel<DT>), cols, dim3(kBlock), 0, s, a, groups);
    hipLaunchKernelGGL((rms_backward_wide_rows_kernel<DT, WT, DH>), rows, dim3(1024), 0, s, a);
    return (int)hipGetLastError();
  }
  return with_shape(tpr, nu, [&](auto T, auto N) {
    constexpr int TPR = decltype(T)::value, NU = decltype(N)::value * 8 / kElems<DT>;
    const dim3 grid(groups), block(block_of(TPR));
    constexpr bool PACKED = TPR < kWave;
    if (PACKED || a.hidden % kElems<DT>) hipLaunchKernelGGL((rms_backward_kernel<DT, WT, TPR, NU, true, DH>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((rms_backward_kernel<DT, WT, TPR, NU, PACKED, DH>), grid, block, 0, s, a);
    return (int)hipGetLastError();
  });
}

template <int DT, int WT>
int forward_w(const RmsArgs& a, bool residual, bool fp8, hipStream_t s) {
  if (residual) return fp8 ? forward_t<DT, WT, true, true>(a, s) : forward_t<DT, WT, true, false>(a, s);
  return fp8 ? forward_t<DT, WT, false, true>(a, s) : forward_t<DT, WT, false, false>(a, s);
}
template <int DT, int WT>
int backward_w(const RmsArgs& a, bool dh, uint32_t groups, hipStream_t s) {
  return dh ? backward_t<DT, WT, true>(a, groups, s) : backward_t<DT, WT, false>(a, groups, s);
}

}  // namespace

// Workgroups of a launch of the backward pass: by the shape alone (results
// and workspace must not depend on the device or on the grid limit).  As in
// layer norm, but for rows of 128 columns and fewer, whose steps are short:
// with 1024 and 512 workgroups 8 x 65536 x 128 bf16 took 102 and 132 us (fp32
// 185 and 184), 8 x 131072 x 64 150 and 216 (fp32 215 and 251).
constexpr uint64_t kNarrowGroups = 1024;
uint32_t rms_backward_groups(int p, uint64_t rows, uint64_t hidden) {
  int tpr, nu;
  row_shape(hidden, &tpr, &nu);
  if (tpr != 16 || nu != 1) return ln_backward_groups(p, rows, hidden);
  const uint64_t rpb = kBlock / 16, need = (rows * (uint64_t)std::min(p, kArgRanks) + rpb - 1) / rpb;
  return (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(need, kNarrowGroups));
}

int launch_rms_forward(int dtype, int wdtype, const RmsArgs& a, bool residual, bool fp8, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  if (dtype == kF32) return forward_w<kF32, kF32>(a, residual, fp8, s);
  return wdtype == kF32 ? forward_w<kBF16, kF32>(a, residual, fp8, s) : forward_w<kBF16, kBF16>(a, residual, fp8, s);
}

int launch_rms_backward(int dtype, int wdtype, const RmsArgs& a, bool dh, uint32_t groups, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  if (dtype == kF32) return backward_w<kF32, kF32>(a, dh, groups, s);
  return wdtype == kF32 ? backward_w<kBF16, kF32>(a, dh, groups, s) : backward_w<kBF16, kBF16>(a, dh, groups, s);
}

}  // namespace coll
