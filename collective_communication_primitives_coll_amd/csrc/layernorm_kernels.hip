// Layer norm over every rank's token rows, forward and backward, with the
// weights' gradients summed over all rows and all ranks.
//
//   forward   m = mean x,  r = 1 / sqrt(mean (x - m)^2 + eps),
//             y = (x - m) r gamma + beta
//   backward  n = (x - m) r,  w = dy gamma,
//             dx = r (w - mean w - n mean(w n)),
//             dgamma = sum dy n,  dbeta = sum dy   (over rows and ranks)
//
// Bound by HBM: 4 bytes an element forward and 6 backward in bf16, against
// some 10 fp32 operations.  So every row is read once: it stays in
// registers between its statistics and its result, TPR lanes to a row, each
// with one or two units of 8 elements.
//
// The backward pass keeps a lane on the same columns for all rows of its
// workgroup, so that the weights' gradients build up in its registers.  At
// the end each workgroup writes one row of partial sums, and the join
// kernel adds these in a fixed order and stores the total to every rank:
// the AllReduce of the two gradients costs one more read of the partials.
// Both the rows a workgroup takes and the number of workgroups depend on
// the shape alone, so results never change from run to run.
//
// All sums are fp32 (a lane's partial sums run over at most a few hundred
// rows before the join); bf16 results are narrowed once.
#include <type_traits>

#include "token_unit.h"

namespace coll {

namespace {

constexpr int block_of(int tpr) { return tpr < kBlock ? kBlock : tpr; }

// Sum over the TPR lanes of a row.  red: TPR / 64 floats of LDS.  One
// barrier: a caller alternates between two arrays, so that a wave that
// writes an array again has passed a barrier that every wave reached after
// reading it.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (TPR > kWave) {
    constexpr int NW = TPR / kWave;
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w];
  }
  return v;
}

// Unit u of a row, zeros past its end.  full: whole units of the row.
template <int SRC, bool TAIL, bool NT>
__device__ __forceinline__ RawUnit<SRC> row_unit(const void* row, uint64_t u, uint64_t full, uint32_t part, uint64_t hidden,
                                                 uint32_t gsh) {
  if (u < full) {
    if constexpr (SRC == kE4M3) return load_codes<NT>(static_cast<const uint8_t*>(row), hidden, u, gsh);
    else return load_unit<SRC, NT>(row, u);
  }
  if constexpr (TAIL && SRC != kE4M3)
    if (u == full) return load_part<SRC>(row, u, part);
  return zero_unit<SRC>();
}
template <int DT, bool TAIL, bool NT>
__device__ __forceinline__ void put_unit(void* row, uint64_t u, uint64_t full, uint32_t part, const float (&f)[8]) {
  if (u < full) store_unit<DT, NT>(row, u, narrow_unit<DT>(f));
  else if constexpr (TAIL)
    if (u == full) store_part<DT>(row, u, part, f);
}

// A weight vector's units of this lane (ones or zeros where it is absent).
template <int WT, bool TAIL, int NU, int TPR>
__device__ __forceinline__ void load_weights(const void* w, float absent, uint32_t lane, uint32_t full, uint32_t part,
                                             RawUnit<WT> (&out)[NU]) {
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = absent;
#pragma unroll
  for (int i = 0; i < NU; ++i)
    out[i] = w ? row_unit<WT, TAIL, false>(w, i * TPR + lane, full, part, 0, 0) : narrow_unit<WT>(f);
}

// Whether a row's loads are issued before the sums of the row before it: a
// workgroup of 1024 lanes has no registers left for them.
template <int TPR>
constexpr bool kAhead = TPR < 1024;

// ---------------------------------------------------------------------------
// Forward.  Grid (workgroups, ranks); a workgroup takes every gridDim.x-th
// run of its rows, the next row's loads issued before this row's sums.
// ---------------------------------------------------------------------------
template <int DT, int WT, int TPR, int NU, bool TAIL, bool CKPT>
__global__ __launch_bounds__(block_of(TPR)) void ln_forward_kernel(LnArgs a) {
  constexpr int RPB = block_of(TPR) / TPR;
  __shared__ float red[2][TPR / kWave];
  const int rank = blockIdx.y;
  const uint32_t lane = threadIdx.x % TPR;
  const uint32_t H = (uint32_t)a.hidden, full = H / 8, part = H % 8;
  const uint64_t stride = (uint64_t)gridDim.x * RPB, row_bytes = (uint64_t)H * Traits<DT>::B;
  const uint8_t* x = static_cast<const uint8_t*>(a.x[rank]);
  uint64_t row = (uint64_t)blockIdx.x * RPB + (RPB > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0);
  if (row >= a.rows) return;
  RawUnit<DT> cur[NU], nxt[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) cur[i] = row_unit<DT, TAIL, true>(x + row * row_bytes, i * TPR + lane, full, part, 0, 0);
  RawUnit<WT> gamma[NU], beta[NU];
  load_weights<WT, TAIL, NU, TPR>(a.gamma[rank], 1.0f, lane, full, part, gamma);
  load_weights<WT, TAIL, NU, TPR>(a.beta[rank], 0.0f, lane, full, part, beta);
  while (true) {
    const uint64_t next = row + stride;
    const bool more = next < a.rows;
    auto fetch = [&] {
#pragma unroll
      for (int i = 0; i < NU; ++i)
        nxt[i] = row_unit<DT, TAIL, true>(x + next * row_bytes, i * TPR + lane, full, part, 0, 0);
    };
    if (kAhead<TPR> && more) fetch();
    float f[NU][8], s = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      widen_unit(cur[i], f[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += f[i][e];
    }
    const float mean = row_sum<TPR>(s, red[0]) / (float)H;
    // the deviations' squares, not the squares' mean less the mean's
    // square, which cancels where the mean is large
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t u = i * TPR + lane;
      const uint32_t cnt = u < full ? 8u : (TAIL && u == full) ? part : 0u;
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) {
        const float d = f[i][e] - mean;
        if (TAIL ? e < cnt : cnt != 0) q += d * d;
      }
    }
    const float rstd = rsqrtf(row_sum<TPR>(q, red[1]) / (float)H + a.eps);
    uint8_t* y = static_cast<uint8_t*>(a.y[rank]) + row * row_bytes;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t u = i * TPR + lane;
      if constexpr (CKPT) {
        const RawUnit<kE4M3> code = encode_unit<DT>(cur[i], f[i], a.gsh);
        if (u < full) store_codes<true>(a.ckpt[rank] + row * a.row_bytes, H, a.row_bytes, u, a.gsh, code);
      }
      float g[8], b[8];
      widen_unit(gamma[i], g);
      widen_unit(beta[i], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = (f[i][e] - mean) * rstd * g[e] + b[e];
      put_unit<DT, TAIL, true>(y, u, full, part, f[i]);
    }
    if (lane == 0) {
      if (a.mean[rank]) as_global(a.mean[rank])[row] = mean;
      if (a.rstd[rank]) as_global(a.rstd[rank])[row] = rstd;
    }
    if (!more) break;
    if (!kAhead<TPR>) fetch();
    row = next;
#pragma unroll
    for (int i = 0; i < NU; ++i) cur[i] = nxt[i];
  }
}

// Rows too wide for the registers: a workgroup of 1024 goes over the row
// three times (sum, deviations, result); the later two find it in the
// caches.
template <int DT, int WT, bool CKPT>
__global__ __launch_bounds__(1024) void ln_forward_wide_kernel(LnArgs a) {
  constexpr int TPR = 1024;
  __shared__ float red[2][TPR / kWave];
  const int rank = blockIdx.y;
  const uint64_t H = a.hidden, full = H / 8, units = (H + 7) / 8;
  const uint32_t part = (uint32_t)(H % 8);
  // every lane takes part in every step (the encoding exchanges lanes)
  const uint64_t steps = (units + TPR - 1) / TPR;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint8_t* x = static_cast<const uint8_t*>(a.x[rank]) + row * H * Traits<DT>::B;
    uint8_t* y = static_cast<uint8_t*>(a.y[rank]) + row * H * Traits<DT>::B;
    float f[8], s = 0.0f;
    for (uint64_t k = 0; k < steps; ++k) {
      widen_unit(row_unit<DT, true, false>(x, k * TPR + threadIdx.x, full, part, 0, 0), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += f[e];
    }
    const float mean = row_sum<TPR>(s, red[0]) / (float)H;
    float q = 0.0f;
    for (uint64_t k = 0; k < steps; ++k) {
      const uint64_t u = k * TPR + threadIdx.x;
      const uint32_t cnt = u < full ? 8u : u == full ? part : 0u;
      widen_unit(row_unit<DT, true, false>(x, u, full, part, 0, 0), f);
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e)
        if (e < cnt) q += (f[e] - mean) * (f[e] - mean);
    }
    const float rstd = rsqrtf(row_sum<TPR>(q, red[1]) / (float)H + a.eps);
    for (uint64_t k = 0; k < steps; ++k) {
      const uint64_t u = k * TPR + threadIdx.x;
      const RawUnit<DT> raw = row_unit<DT, true, false>(x, u, full, part, 0, 0);
      widen_unit(raw, f);
      if constexpr (CKPT) {
        const RawUnit<kE4M3> code = encode_unit<DT>(raw, f, a.gsh);
        if (u < full) store_codes<true>(a.ckpt[rank] + row * a.row_bytes, H, a.row_bytes, u, a.gsh, code);
      }
      float g[8], b[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        g[e] = 1.0f;
        b[e] = 0.0f;
      }
      if (a.gamma[rank]) widen_unit(row_unit<WT, true, false>(a.gamma[rank], u, full, part, 0, 0), g);
      if (a.beta[rank]) widen_unit(row_unit<WT, true, false>(a.beta[rank], u, full, part, 0, 0), b);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (f[e] - mean) * rstd * g[e] + b[e];
      put_unit<DT, true, false>(y, u, full, part, f);
    }
    if (threadIdx.x == 0) {
      if (a.mean[rank]) as_global(a.mean[rank])[row] = mean;
      if (a.rstd[rank]) as_global(a.rstd[rank])[row] = rstd;
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  Partial sums of workgroup (b, rank) go to
// ws[rank0 + rank][b][0: dgamma, 1: dbeta][hidden].
// ---------------------------------------------------------------------------
template <int TAILS>
__device__ __forceinline__ void put_partial(float* ws, uint64_t u, uint64_t full, uint32_t part, const float (&f)[8]) {
  put_unit<kF32, TAILS != 0, false>(ws, u, full, part, f);
}

template <int SRC, int DT, int WT, int TPR, int NU, bool TAIL>
__global__ __launch_bounds__(block_of(TPR)) void ln_backward_kernel(LnArgs a) {
  constexpr bool AHEAD = kAhead<TPR>;
  constexpr int RPB = block_of(TPR) / TPR;
  __shared__ float red[2][2][TPR / kWave];
  __shared__ float fold[RPB > 1 ? 2 * NU * TPR * 8 : 1];
  const int rank = blockIdx.y;
  const uint32_t lane = threadIdx.x % TPR;
  const uint32_t H = (uint32_t)a.hidden, full = H / 8, part = H % 8;
  const uint64_t stride = (uint64_t)gridDim.x * RPB, row_bytes = (uint64_t)H * Traits<DT>::B;
  const uint64_t src_bytes = SRC == kE4M3 ? a.row_bytes : row_bytes;
  const uint8_t* x = static_cast<const uint8_t*>(a.x[rank]);
  const uint8_t* dy = static_cast<const uint8_t*>(a.dy[rank]);
  const int mine = RPB > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0;
  uint64_t row = (uint64_t)blockIdx.x * RPB + mine;
  float dg[NU][8] = {}, db[NU][8] = {};
  if (row < a.rows) {
    RawUnit<SRC> cx[NU], nx[NU];
    RawUnit<DT> cd[NU], nd[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      cx[i] = row_unit<SRC, TAIL, true>(x + row * src_bytes, i * TPR + lane, full, part, H, a.gsh);
      cd[i] = row_unit<DT, TAIL, true>(dy + row * row_bytes, i * TPR + lane, full, part, 0, 0);
    }
    float mean = as_global(a.mean[rank])[row], rstd = as_global(a.rstd[rank])[row];
    RawUnit<WT> gamma[NU];
    load_weights<WT, TAIL, NU, TPR>(a.gamma[rank], 1.0f, lane, full, part, gamma);
    int turn = 0;
    while (true) {
      const uint64_t next = row + stride;
      const bool more = next < a.rows;
      float nmean = 0.0f, nrstd = 0.0f;
      auto fetch = [&] {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          nx[i] = row_unit<SRC, TAIL, true>(x + next * src_bytes, i * TPR + lane, full, part, H, a.gsh);
          nd[i] = row_unit<DT, TAIL, true>(dy + next * row_bytes, i * TPR + lane, full, part, 0, 0);
        }
        nmean = as_global(a.mean[rank])[next];
        nrstd = as_global(a.rstd[rank])[next];
      };
      if (AHEAD && more) fetch();
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        float fx[8], fd[8], g[8];
        widen_unit(cx[i], fx);
        widen_unit(cd[i], fd);
        widen_unit(gamma[i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // past the row's end dy is zero, and so is all that it enters
          const float n = (fx[e] - mean) * rstd, w = fd[e] * g[e];
          dg[i][e] += fd[e] * n;
          db[i][e] += fd[e];
          s1 += w;
          s2 += w * n;
        }
      }
      s1 = wave_sum(s1);
      s2 = wave_sum(s2);
      if constexpr (TPR > kWave) {
        constexpr int NW = TPR / kWave;
        if (threadIdx.x % kWave == 0) {
          red[turn][0][threadIdx.x / kWave] = s1;
          red[turn][1][threadIdx.x / kWave] = s2;
        }
        __syncthreads();
        s1 = s2 = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          s1 += red[turn][0][w];
          s2 += red[turn][1][w];
        }
        turn ^= 1;
      }
      const float c1 = s1 / (float)H, c2 = s2 / (float)H;
      uint8_t* dx = static_cast<uint8_t*>(a.dx[rank]) + row * row_bytes;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const uint32_t u = i * TPR + lane;
        float fx[8], fd[8], g[8];
        widen_unit(cx[i], fx);
        widen_unit(cd[i], fd);
        widen_unit(gamma[i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = (fx[e] - mean) * rstd;
          fd[e] = rstd * (fd[e] * g[e] - c1 - n * c2);
          fx[e] = n;
        }
        put_unit<DT, TAIL, true>(dx, u, full, part, fd);
        if constexpr (SRC == kE4M3) {
          // the output again, for the weight gradient of the product it fed
          if (a.y[rank]) {
            RawUnit<WT> bu[1];
            float b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = 0.0f;
            if (a.beta[rank]) {
              bu[0] = row_unit<WT, TAIL, false>(a.beta[rank], u, full, part, 0, 0);
              widen_unit(bu[0], b);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) fx[e] = fx[e] * g[e] + b[e];
            put_unit<DT, TAIL, true>(static_cast<uint8_t*>(a.y[rank]) + row * row_bytes, u, full, part, fx);
          }
        }
      }
      if (!more) break;
      if (!AHEAD) fetch();
      row = next;
      mean = nmean;
      rstd = nrstd;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        cx[i] = nx[i];
        cd[i] = nd[i];
      }
    }
  }
  float* ws = a.ws + ((uint64_t)(a.rank0 + rank) * gridDim.x + blockIdx.x) * 2 * H;
  if constexpr (RPB > 1) {
    // the workgroup's waves add their sums in turn
    for (int w = 0; w < RPB; ++w) {
      if (mine == w) {
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* at = fold + (i * 8 + e) * TPR + lane;
            dg[i][e] += w ? at[0] : 0.0f;
            db[i][e] += w ? at[NU * 8 * TPR] : 0.0f;
            at[0] = dg[i][e];
            at[NU * 8 * TPR] = db[i][e];
          }
      }
      __syncthreads();
    }
    if (mine != RPB - 1) return;
  }
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    put_partial<TAIL>(ws, i * TPR + lane, full, part, dg[i]);
    put_partial<TAIL>(ws + H, i * TPR + lane, full, part, db[i]);
  }
}

// Rows too wide for the registers, in two kernels: the weights' gradients by
// columns (a lane keeps its 8 columns over the workgroup's rows), then the
// rows, each gone over twice.  The columns come first, so that dx may be
// dy's own buffer.
template <int SRC, int DT>
__global__ __launch_bounds__(kBlock) void ln_backward_wide_columns_kernel(LnArgs a, uint32_t splits) {
  const int rank = blockIdx.y;
  const uint64_t H = a.hidden, full = H / 8, row_bytes = H * Traits<DT>::B;
  const uint64_t src_bytes = SRC == kE4M3 ? a.row_bytes : row_bytes;
  const uint32_t part = (uint32_t)(H % 8), split = blockIdx.x % splits;
  const uint64_t u = (uint64_t)(blockIdx.x / splits) * kBlock + threadIdx.x;
  float dg[8] = {}, db[8] = {};
  for (uint64_t row = split; row < a.rows; row += splits) {
    float fx[8], fd[8];
    widen_unit(row_unit<SRC, true, false>(static_cast<const uint8_t*>(a.x[rank]) + row * src_bytes, u, full, part, H, a.gsh), fx);
    widen_unit(row_unit<DT, true, false>(static_cast<const uint8_t*>(a.dy[rank]) + row * row_bytes, u, full, part, 0, 0), fd);
    const float mean = as_global(a.mean[rank])[row], rstd = as_global(a.rstd[rank])[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dg[e] += fd[e] * ((fx[e] - mean) * rstd);
      db[e] += fd[e];
    }
  }
  float* ws = a.ws + ((uint64_t)(a.rank0 + rank) * splits + split) * 2 * H;
  put_partial<1>(ws, u, full, part, dg);
  put_partial<1>(ws + H, u, full, part, db);
}

template <int SRC, int DT, int WT>
__global__ __launch_bounds__(1024) void ln_backward_wide_rows_kernel(LnArgs a) {
  constexpr int TPR = 1024;
  __shared__ float red[2][TPR / kWave];
  const int rank = blockIdx.y;
  const uint64_t H = a.hidden, full = H / 8, units = (H + 7) / 8, row_bytes = H * Traits<DT>::B;
  const uint64_t src_bytes = SRC == kE4M3 ? a.row_bytes : row_bytes;
  const uint32_t part = (uint32_t)(H % 8);
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint8_t* x = static_cast<const uint8_t*>(a.x[rank]) + row * src_bytes;
    const uint8_t* dy = static_cast<const uint8_t*>(a.dy[rank]) + row * row_bytes;
    const float mean = as_global(a.mean[rank])[row], rstd = as_global(a.rstd[rank])[row];
    float n[8], w[8], g[8], s1 = 0.0f, s2 = 0.0f;
    auto unit = [&](uint64_t u) {
      widen_unit(row_unit<SRC, true, false>(x, u, full, part, H, a.gsh), n);
      widen_unit(row_unit<DT, true, false>(dy, u, full, part, 0, 0), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = 1.0f;
      if (a.gamma[rank]) widen_unit(row_unit<WT, true, false>(a.gamma[rank], u, full, part, 0, 0), g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] = (n[e] - mean) * rstd;
        w[e] *= g[e];
      }
    };
    for (uint64_t u = threadIdx.x; u < units; u += TPR) {
      unit(u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s1 += w[e];
        s2 += w[e] * n[e];
      }
    }
    const float c1 = row_sum<TPR>(s1, red[0]) / (float)H;
    const float c2 = row_sum<TPR>(s2, red[1]) / (float)H;
    for (uint64_t u = threadIdx.x; u < units; u += TPR) {
      unit(u);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = rstd * (w[e] - c1 - n[e] * c2);
      put_unit<DT, true, false>(static_cast<uint8_t*>(a.dx[rank]) + row * row_bytes, u, full, part, w);
      if constexpr (SRC == kE4M3) {
        if (a.y[rank]) {
          float b[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) b[e] = 0.0f;
          if (a.beta[rank]) widen_unit(row_unit<WT, true, false>(a.beta[rank], u, full, part, 0, 0), b);
#pragma unroll
          for (int e = 0; e < 8; ++e) n[e] = n[e] * g[e] + b[e];
          put_unit<DT, true, false>(static_cast<uint8_t*>(a.y[rank]) + row * row_bytes, u, full, part, n);
        }
      }
    }
  }
}

// The weights' gradients: column j of the `parts` partial rows, added by 16
// waves (each every 16th row, then one after the other in LDS), divided by
// p for an average, and stored to every rank.
template <int WT>
__global__ __launch_bounds__(1024) void ln_join_kernel(LnJoinArgs a) {
  constexpr int NW = 1024 / kWave;
  __shared__ float sums[NW][kWave];
  const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const uint64_t cols = 2 * a.hidden, j = (uint64_t)blockIdx.x * kWave + lane;
  float s = 0.0f;
  if (j < cols) {
    const float* w = as_global(a.ws) + j;
#pragma unroll 8
    for (uint32_t k = wave; k < a.parts; k += NW) s += w[(uint64_t)k * cols];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || j >= cols) return;
#pragma unroll
  for (int w = 1; w < NW; ++w) s += sums[w][lane];
  if (a.avg) s /= (float)a.p;
  const bool beta = j >= a.hidden;
  const uint64_t c = beta ? j - a.hidden : j;
  for (int r = 0; r < a.p; ++r) {
    void* to = beta ? a.dbeta[r] : a.dgamma[r];
    if (to) as_global(static_cast<typename Traits<WT>::S*>(to))[c] = narrow1<WT>(s);
  }
}

// Lanes per row and units per lane for a width, 0 lanes: too wide.  Two
// units a lane keep the backward pass (16 sums of weight gradients a unit,
// this row and the next in registers) within half of a SIMD's registers.
void row_shape(uint64_t hidden, int* tpr, int* nu) {
  const uint64_t units = (hidden + 7) / 8;
  *tpr = units <= 128 ? 64 : units <= 512 ? 256 : units <= 1024 ? 512 : units <= 2048 ? 1024 : 0;
  *nu = *tpr && units <= (uint64_t)*tpr ? 1 : 2;
}

// Calls f with the shape as compile-time constants.
template <class F>
int with_shape(uint64_t hidden, F f) {
  int tpr, nu;
  row_shape(hidden, &tpr, &nu);
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  if (tpr == 64) return nu == 1 ? f(std::integral_constant<int, 64>(), one) : f(std::integral_constant<int, 64>(), two);
  if (tpr == 256) return nu == 1 ? f(std::integral_constant<int, 256>(), one) : f(std::integral_constant<int, 256>(), two);
  if (tpr == 512) return f(std::integral_constant<int, 512>(), two);
  return f(std::integral_constant<int, 1024>(), two);
}

template <int DT, int WT>
int forward_t(const LnArgs& a, int ranks, bool ckpt, hipStream_t s) {
  int tpr, nu;
  row_shape(a.hidden, &tpr, &nu);
  const bool tail = a.hidden % 8 != 0;
  if (!tpr) {
    const uint32_t gx = (uint32_t)(a.rows < 65536 ? a.rows : 65536);
    if (ckpt) hipLaunchKernelGGL((ln_forward_wide_kernel<DT, WT, true>), dim3(gx, ranks), dim3(1024), 0, s, a);
    else hipLaunchKernelGGL((ln_forward_wide_kernel<DT, WT, false>), dim3(gx, ranks), dim3(1024), 0, s, a);
    return (int)hipGetLastError();
  }
  return with_shape(a.hidden, [&](auto T, auto N) {
    constexpr int TPR = decltype(T)::value, NU = decltype(N)::value, RPB = block_of(TPR) / TPR;
    const uint64_t need = (a.rows + RPB - 1) / RPB;
    const uint64_t cap = ln_forward_groups(ranks, TPR);
    const dim3 grid((uint32_t)(need < cap ? need : cap), ranks), block(block_of(TPR));
    if (ckpt) hipLaunchKernelGGL((ln_forward_kernel<DT, WT, TPR, NU, false, true>), grid, block, 0, s, a);
    else if (tail) hipLaunchKernelGGL((ln_forward_kernel<DT, WT, TPR, NU, true, false>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((ln_forward_kernel<DT, WT, TPR, NU, false, false>), grid, block, 0, s, a);
    return (int)hipGetLastError();
  });
}

template <int DT, int WT>
int backward_t(const LnArgs& a, int ranks, uint32_t groups, bool ckpt, hipStream_t s) {
  int tpr, nu;
  row_shape(a.hidden, &tpr, &nu);
  const bool tail = a.hidden % 8 != 0;
  if (!tpr) {
    const uint64_t chunks = ((a.hidden + 7) / 8 + kBlock - 1) / kBlock;
    if (chunks * groups > 0x7fffffffull) return (int)hipErrorInvalidConfiguration;
    const dim3 cols((uint32_t)(chunks * groups), ranks), rows((uint32_t)(a.rows < 65536 ? a.rows : 65536), ranks);
    if (ckpt) {
      hipLaunchKernelGGL((ln_backward_wide_columns_kernel<kE4M3, DT>), cols, dim3(kBlock), 0, s, a, groups);
      hipLaunchKernelGGL((ln_backward_wide_rows_kernel<kE4M3, DT, WT>), rows, dim3(1024), 0, s, a);
    } else {
      hipLaunchKernelGGL((ln_backward_wide_columns_kernel<DT, DT>), cols, dim3(kBlock), 0, s, a, groups);
      hipLaunchKernelGGL((ln_backward_wide_rows_kernel<DT, DT, WT>), rows, dim3(1024), 0, s, a);
    }
    return (int)hipGetLastError();
  }
  return with_shape(a.hidden, [&](auto T, auto N) {
    constexpr int TPR = decltype(T)::value, NU = decltype(N)::value;
    const dim3 grid(groups, ranks), block(block_of(TPR));
    if (ckpt) hipLaunchKernelGGL((ln_backward_kernel<kE4M3, DT, WT, TPR, NU, false>), grid, block, 0, s, a);
    else if (tail) hipLaunchKernelGGL((ln_backward_kernel<DT, DT, WT, TPR, NU, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((ln_backward_kernel<DT, DT, WT, TPR, NU, false>), grid, block, 0, s, a);
    return (int)hipGetLastError();
  });
}

}  // namespace

// Workgroups per rank of the forward pass.
uint32_t ln_forward_groups(int ranks, int tpr) {
  const uint32_t total = tpr == 1024 ? 512 : 2048;
  const uint32_t g = total / (uint32_t)ranks;
  return g ? g : 1;
}

// Workgroups per rank of the backward pass: by the shape alone (results and
// workspace must not depend on the device or on the grid limit).  Two
// 256-lane workgroups fit a CU's registers, one of 1024 lanes.
uint32_t ln_backward_groups(int p, uint64_t rows, uint64_t hidden) {
  int tpr, nu;
  row_shape(hidden, &tpr, &nu);
  const uint64_t rpb = tpr == 64 ? 4 : 1, need = (rows + rpb - 1) / rpb;
  uint64_t g = (tpr == 1024 || tpr == 0 ? 256 : 512) / (uint64_t)p;
  if (g < 1) g = 1;
  return (uint32_t)(need < g ? (need ? need : 1) : g);
}

int launch_ln_forward(int dtype, int wdtype, const LnArgs& a, int ranks, bool ckpt, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  if (dtype == kF32) return forward_t<kF32, kF32>(a, ranks, ckpt, s);
  return wdtype == kF32 ? forward_t<kBF16, kF32>(a, ranks, ckpt, s) : forward_t<kBF16, kBF16>(a, ranks, ckpt, s);
}

int launch_ln_backward(int dtype, int wdtype, const LnArgs& a, int ranks, uint32_t groups, bool ckpt, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  if (dtype == kF32) return backward_t<kF32, kF32>(a, ranks, groups, ckpt, s);
  return wdtype == kF32 ? backward_t<kBF16, kF32>(a, ranks, groups, ckpt, s)
                        : backward_t<kBF16, kBF16>(a, ranks, groups, ckpt, s);
}

int launch_ln_join(int wdtype, const LnJoinArgs& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  const uint64_t blocks = (2 * a.hidden + kWave - 1) / kWave;
  if (wdtype == kF32) hipLaunchKernelGGL((ln_join_kernel<kF32>), dim3((uint32_t)blocks), dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((ln_join_kernel<kBF16>), dim3((uint32_t)blocks), dim3(1024), 0, s, a);
  return (int)hipGetLastError();
}

}  // namespace coll
