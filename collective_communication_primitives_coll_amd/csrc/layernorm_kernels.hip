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
// with 8 or 16 elements of it.
//
// The backward pass keeps a lane on the same columns for all rows of its
// workgroup, so that the weights' gradients build up in its registers.  At
// the end each workgroup writes one row of partial sums, and the join
// kernel adds these in a fixed order and stores the total to every rank:
// the AllReduce of the two gradients costs one more read of the partials.
// Both the rows a workgroup takes and the number of workgroups depend on
// the shape alone, so results never change from run to run.
//
// All sums are fp32 (a lane's partial sum runs over its workgroup's rows, one
// in 256 or 512 of a large call's, before the join); bf16 results are
// narrowed once.
#include "token_rows.h"

namespace coll {

namespace {

// ---------------------------------------------------------------------------
// Forward.  Grid (runs of rows, ranks), and no walk: the workgroups that
// share a CU hide each other's waits, and a workgroup that ends waits for no
// store.  A lane holds the same columns of kRows rows, so that the weights
// are loaded once for them, and it asks for the weights only after the first
// sums: loads return in order, and the weights, though they come from L2,
// queue behind other waves' rows.
// 8 x 4096 x 7168 bf16: 152 us (6.2 TB/s; the card's 1:1 streams reach 6.3).
// One row at a time 158 us, and 173 us with the weights asked for first;
// three rows 155, four 159.  Persistent workgroups, with the weights in
// registers and the next row's loads ahead, 166-175 us; rows claimed from
// counters 158-164 us.
// With the checkpoint, 8 x 2048 x 7168 bf16 and fp32 weights: 109 us
// (5.4 TB/s), bound by how many rows the registers hold.  The codes are
// stored in the first pass: 116-119 us after it, 115 us with the results.
// ---------------------------------------------------------------------------
// Rows to a lane: one where two workgroups of 1024 lanes then fit a CU, which
// bf16 without checkpoints does.  8 x 2048 x 16384, one row and two, in us: 179
// and 213; with checkpoints and fp32 weights 269 and 249 (bf16 weights 242 and
// 249); fp32 391 and 348, with checkpoints 417 and 404.
template <int DT, int TPR, bool CKPT>
constexpr int rows_of() { return TPR == 1024 && DT == kBF16 && !CKPT ? 1 : 2; }

// Whether the registers keep a bf16 row as it was loaded, to be widened again
// in every pass, or its fp32 values, which take twice the room: where one
// more workgroup then fits a CU.  16384 rows in 8 shards, us as loaded and
// widened: 7168 with fp32 weights and checkpoints 109 and 117, 12288 plain
// 134 and 156 (with fp32 weights 136 and 162); where no more fit, widening
// costs: 7168 plain 77 and 76, 4096 with checkpoints 62 and 59, 12288 with
// both 194 and 187.
template <int DT, int WT, int TPR, bool CKPT>
constexpr bool as_loaded() {
  constexpr int more = (WT == kF32) + CKPT;
  return DT == kBF16 && (TPR == 384 || TPR == 512 ? more >= 1 : TPR == 768 ? more <= 1 : TPR == 1024 && !CKPT);
}
// The same unit, but not known to be.
template <bool HIDE, int DT, int E>
__device__ __forceinline__ RawUnit<DT, E>& again(RawUnit<DT, E>& r) {
  if constexpr (HIDE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(r.v[0][i]));
  }
  return r;
}

template <int DT, int WT, int TPR, int NU, bool TAIL, bool CKPT>
__global__ __launch_bounds__(block_of(TPR)) void ln_forward_kernel(LnArgs a) {
  constexpr int E = kElems<DT>;
  constexpr int kRows = rows_of<DT, TPR, CKPT>();
  __shared__ float red[2][kRows][waves_of(TPR)];
  const int rank = blockIdx.y;
  const uint32_t lane = threadIdx.x % TPR, H = (uint32_t)a.hidden;
  const uint64_t row_bytes = (uint64_t)H * Traits<DT>::B;
  const uint64_t row0 = own_row<TPR>(blockIdx.x) * kRows;
  if (row0 >= a.rows) return;
  const uint8_t* x0 = static_cast<const uint8_t*>(a.x[rank]) + row0 * row_bytes;
  RawUnit<DT, E> raw[kRows][NU];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    // past the last row: row0 again (its results are not stored)
    const Row<DT, E, TAIL> x(x0 + (row0 + k < a.rows ? k : 0) * row_bytes, H);
#pragma unroll
    for (int i = 0; i < NU; ++i) raw[k][i] = x.template get<true>(i * TPR + lane);
  }
  float s[kRows], q[kRows];
  constexpr bool kHide = as_loaded<DT, WT, TPR, CKPT>();
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    s[k] = 0.0f;
    uint8_t* ckpt = CKPT ? a.ckpt[rank] + (row0 + k) * a.row_bytes : nullptr;
    const bool live = row0 + k < a.rows;
    // (of a row to itself; where a wave holds several, by their addresses)
    const RowBuffer codes(ckpt, live ? H : 0), scales(CKPT ? ckpt + H : nullptr, live ? (H >> a.glog) * 4 : 0);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t u = i * TPR + lane, skip = TAIL && may_end<TPR, NU>(i) ? skip_of<E>(u, H) : 0;
      float f[E];
      widen_unit(raw[k][i], f);
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) s[k] += TAIL && may_end<TPR, NU>(i) && e < skip ? 0.0f : f[e];
      if constexpr (CKPT) {
        const RawUnit<kE4M3, E> code = encode_unit<DT, E>(raw[k][i], f, a.glog);
        if constexpr (TPR >= kWave) store_codes<E, true>(codes, scales, E * u, a.glog, code);
        else if (E * u < H && live) store_codes<E, true>(ckpt, H, a.row_bytes, E * u, a.glog, code);
      }
    }
  }
  row_sums<TPR, kRows>(s, red[0]);
  RawUnit<WT, E> gamma[NU], beta[NU];
  load_weights<WT, E, TAIL, NU, TPR>(a.gamma[rank], 1.0f, lane, H, gamma);
  load_weights<WT, E, TAIL, NU, TPR>(a.beta[rank], 0.0f, lane, H, beta);
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    s[k] /= (float)H;
    // the deviations' squares, not the squares' mean less the mean's
    // square, which cancels where the mean is large
    q[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t u = i * TPR + lane, skip = TAIL && may_end<TPR, NU>(i) ? skip_of<E>(u, H) : 0;
      float sq = 0.0f, f[E];
      widen_unit(again<kHide>(raw[k][i]), f);
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) {
        const float d = f[e] - s[k];
        sq = TAIL && may_end<TPR, NU>(i) && e < skip ? sq : __builtin_fmaf(d, d, sq);
      }
      q[k] += !TAIL && E * u >= H ? 0.0f : sq;
    }
  }
  row_sums<TPR, kRows>(q, red[1]);
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (row0 + k >= a.rows) break;
    const float rstd = rsqrtf(q[k] / (float)H + a.eps);
    const Row<DT, E, TAIL> y(static_cast<uint8_t*>(a.y[rank]) + (row0 + k) * row_bytes, H);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float f[E], g[E], b[E];
      widen_unit(again<kHide>(raw[k][i]), f);
      widen_unit(gamma[i], g);
      widen_unit(beta[i], b);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = (f[e] - s[k]) * rstd * g[e] + b[e];
      y.template put<true>(i * TPR + lane, narrow_unit<DT, E>(f));
    }
    if constexpr (CKPT && TPR >= kWave) pad_codes(a.ckpt[rank] + (row0 + k) * a.row_bytes, H, a.row_bytes, a.glog, lane);
    if (lane == 0) {
      if (a.mean[rank]) as_global(a.mean[rank])[row0 + k] = s[k];
      if (a.rstd[rank]) as_global(a.rstd[rank])[row0 + k] = rstd;
    }
  }
}

// ---------------------------------------------------------------------------
// Rows too wide for the registers (or narrower than one unit): units of 8
// elements in every type, each row gone over several times; all passes but
// the first find it in the caches.
// ---------------------------------------------------------------------------

template <int DT, int WT, bool CKPT>
__global__ __launch_bounds__(1024) void ln_forward_wide_kernel(LnArgs a) {
  constexpr int TPR = 1024;
  __shared__ float red[2][1][TPR / kWave];
  const int rank = blockIdx.y;
  const uint64_t H = a.hidden, full = H / 8, units = (H + 7) / 8;
  const uint32_t part = (uint32_t)(H % 8);
  // every lane takes part in every step (the encoding exchanges lanes)
  const uint64_t steps = (units + TPR - 1) / TPR;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint8_t* x = static_cast<const uint8_t*>(a.x[rank]) + row * H * Traits<DT>::B;
    uint8_t* y = static_cast<uint8_t*>(a.y[rank]) + row * H * Traits<DT>::B;
    float f[8], s[1] = {0.0f}, q[1] = {0.0f};
    for (uint64_t k = 0; k < steps; ++k) {
      widen_unit(row_unit<DT>(x, k * TPR + threadIdx.x, full, part), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += f[e];
    }
    row_sums<TPR, 1>(s, red[0]);
    const float mean = s[0] / (float)H;
    for (uint64_t k = 0; k < steps; ++k) {
      const uint64_t u = k * TPR + threadIdx.x;
      const uint32_t cnt = u < full ? 8u : u == full ? part : 0u;
      widen_unit(row_unit<DT>(x, u, full, part), f);
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e)
        if (e < cnt) q[0] += (f[e] - mean) * (f[e] - mean);
    }
    row_sums<TPR, 1>(q, red[1]);
    const float rstd = rsqrtf(q[0] / (float)H + a.eps);
    for (uint64_t k = 0; k < steps; ++k) {
      const uint64_t u = k * TPR + threadIdx.x;
      const RawUnit<DT, 8> raw = row_unit<DT>(x, u, full, part);
      widen_unit(raw, f);
      if constexpr (CKPT) {
        const RawUnit<kE4M3, 8> code = encode_unit<DT, 8>(raw, f, a.glog);
        if (u < full) store_codes<8, true>(a.ckpt[rank] + row * a.row_bytes, H, a.row_bytes, u * 8, a.glog, code);
      }
      float g[8], b[8];
      weight_unit<WT>(a.gamma[rank], 1.0f, u, full, part, g);
      weight_unit<WT>(a.beta[rank], 0.0f, u, full, part, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (f[e] - mean) * rstd * g[e] + b[e];
      put_unit<DT>(y, u, full, part, f);
    }
    if (threadIdx.x == 0) {
      if (a.mean[rank]) as_global(a.mean[rank])[row] = mean;
      if (a.rstd[rank]) as_global(a.rstd[rank])[row] = rstd;
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  A workgroup takes every gridDim.x-th run of rows, through all
// ranks of the launch: the rows in work at any time lie close together.
// Partial sums of workgroup b go to ws[b][0: dgamma, 1: dbeta][hidden].
// ---------------------------------------------------------------------------

template <int SRC, int DT, int WT, int TPR, int NU, bool TAIL>
__global__ __launch_bounds__(block_of(TPR)) void ln_backward_kernel(LnArgs a) {
  constexpr int E = kElems<DT>, RPB = block_of(TPR) / TPR, AHEAD = kAhead<TPR>;
  __shared__ float red[2][2][waves_of(TPR)];
  __shared__ float fold[RPB > 1 ? 2 * NU * E * TPR : 1];
  const uint32_t lane = threadIdx.x % TPR, H = (uint32_t)a.hidden;
  const uint64_t row_bytes = (uint64_t)H * Traits<DT>::B, src_bytes = SRC == kE4M3 ? a.row_bytes : row_bytes;
  const uint64_t stride = (uint64_t)gridDim.x * RPB;
  // a place in the ranks' rows, one rank after the other
  struct Place {
    uint64_t row;
    int rank;
    __device__ __forceinline__ void settle(const LnArgs& a) {
      while (row >= a.rows && rank < a.ranks) {
        row -= a.rows;
        ++rank;
      }
    }
  };
  Place at{own_row<TPR>(blockIdx.x), 0};
  at.settle(a);
  float dg[NU][E] = {}, db[NU][E] = {};
  if (at.rank < a.ranks) {
    // AHEAD + 1 buffers; the loop is unrolled over them, since moving a
    // loaded register to another waits for its load
    RawUnit<SRC, E> bx[AHEAD + 1][NU];
    RawUnit<DT, E> bd[AHEAD + 1][NU];
    float bm[AHEAD + 1], bs[AHEAD + 1];
    auto fetch = [&](const Place& r, auto K) {
      constexpr int k = decltype(K)::value;
      const Row<SRC, E, TAIL> rx(static_cast<const uint8_t*>(a.x[r.rank]) + r.row * src_bytes, H, a.glog);
      const Row<DT, E, TAIL> rd(static_cast<const uint8_t*>(a.dy[r.rank]) + r.row * row_bytes, H);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        bx[k][i] = rx.template get<true>(i * TPR + lane);
        bd[k][i] = rd.template get<true>(i * TPR + lane);
      }
      bm[k] = ld_const(a.mean[r.rank] + r.row);
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
      if constexpr (AHEAD > 0) fetch(next, std::integral_constant<int, (k + 1) % (AHEAD + 1)>());
      const float mean = bm[k], rstd = bs[k];
      float n[NU][E], w[NU][E], s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const uint32_t skip = TAIL && may_end<TPR, NU>(i) ? skip_of<E>(i * TPR + lane, H) : 0;
        // Past the row's end x and dy are zero, and so is all that dy enters,
        // as long as n is finite there: without the mean, whose product with
        // rstd may not be (a constant row of large values).
        const float m = !TAIL && may_end<TPR, NU>(i) && E * (i * TPR + lane) >= H ? 0.0f : mean;
        float d[E], g[E];
        widen_unit(bx[k][i], n[i]);
        widen_unit(bd[k][i], d);
        widen_unit(gamma[i], g);
#pragma unroll
        for (uint32_t e = 0; e < E; ++e) {
          n[i][e] = (n[i][e] - m) * rstd;
          w[i][e] = d[e] * g[e];
          const bool own = !(TAIL && may_end<TPR, NU>(i) && e < skip);
          const float de = own ? d[e] : 0.0f, we = own ? w[i][e] : 0.0f;
          dg[i][e] += own ? de * n[i][e] : 0.0f;
          db[i][e] += de;
          s[0] += we;
          s[1] += own ? we * n[i][e] : 0.0f;
        }
      }
      row_sums<TPR, 2>(s, red[turn]);
      turn ^= 1;
      const float c1 = s[0] / (float)H, c2 = s[1] / (float)H;
      const Row<DT, E, TAIL> dx(static_cast<uint8_t*>(a.dx[at.rank]) + at.row * row_bytes, H);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
#pragma unroll
        for (int e = 0; e < E; ++e) w[i][e] = rstd * (w[i][e] - c1 - n[i][e] * c2);
        dx.template put<true>(i * TPR + lane, narrow_unit<DT, E>(w[i]));
      }
      if constexpr (SRC == kE4M3) {
        // the output again, for the weight gradient of the product it fed
        if (a.y[at.rank]) {
          const Row<DT, E, TAIL> y(static_cast<uint8_t*>(a.y[at.rank]) + at.row * row_bytes, H);
          RawUnit<WT, E> beta[NU];
          load_weights<WT, E, TAIL, NU, TPR>(a.beta[at.rank], 0.0f, lane, H, beta);
#pragma unroll
          for (int i = 0; i < NU; ++i) {
            float g[E], b[E];
            widen_unit(gamma[i], g);
            widen_unit(beta[i], b);
#pragma unroll
            for (int e = 0; e < E; ++e) n[i][e] = n[i][e] * g[e] + b[e];
            y.template put<true>(i * TPR + lane, narrow_unit<DT, E>(n[i]));
          }
        }
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
  float* ws = a.ws + (uint64_t)blockIdx.x * 2 * H;
  if constexpr (RPB > 1) {
    // the workgroup's groups of lanes add their sums in turn
    const int mine = (int)own_row<TPR>(0);
    for (int k = 0; k < RPB; ++k) {
      if (mine == k) {
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float* to = fold + (i * E + e) * TPR + lane;
            dg[i][e] += k ? to[0] : 0.0f;
            db[i][e] += k ? to[NU * E * TPR] : 0.0f;
            to[0] = dg[i][e];
            to[NU * E * TPR] = db[i][e];
          }
      }
      __syncthreads();
    }
    if (mine != RPB - 1) return;
  }
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const uint32_t u = i * TPR + lane;
    if (E * u + E <= H) {
      store_unit<kF32, E, false>((void*)ws, E * u, narrow_unit<kF32, E>(dg[i]));
      store_unit<kF32, E, false>((void*)(ws + H), E * u, narrow_unit<kF32, E>(db[i]));
    } else if (TAIL && E * u < H) {
      // the row's last E elements, of which the last H % E are this unit's
      const uint32_t skip = skip_of<E>(u, H);
#pragma unroll
      for (uint32_t e = 0; e < E; ++e)
        if (e >= skip) {
          as_global(ws)[H - E + e] = dg[i][e];
          as_global(ws)[2 * (uint64_t)H - E + e] = db[i][e];
        }
    }
  }
}

// Rows too wide for the registers, in two kernels: the weights' gradients by
// columns (a lane keeps its 8 columns over the workgroup's rows), then the
// rows, each gone over twice.  The columns come first, so that dx may be
// dy's own buffer.
template <int SRC, int DT>
__global__ __launch_bounds__(kBlock) void ln_backward_wide_columns_kernel(LnArgs a, uint32_t splits) {
  const uint64_t H = a.hidden, full = H / 8, row_bytes = H * Traits<DT>::B;
  const uint64_t src_bytes = SRC == kE4M3 ? a.row_bytes : row_bytes;
  const uint32_t part = (uint32_t)(H % 8), split = blockIdx.x % splits;
  const uint64_t u = (uint64_t)(blockIdx.x / splits) * kBlock + threadIdx.x;
  float dg[8] = {}, db[8] = {};
  for (int rank = 0; rank < a.ranks; ++rank)
    for (uint64_t row = split; row < a.rows; row += splits) {
      float fx[8], fd[8];
      widen_unit(row_unit<SRC>(static_cast<const uint8_t*>(a.x[rank]) + row * src_bytes, u, full, part, H, a.glog), fx);
      widen_unit(row_unit<DT>(static_cast<const uint8_t*>(a.dy[rank]) + row * row_bytes, u, full, part), fd);
      const float mean = as_global(a.mean[rank])[row], rstd = as_global(a.rstd[rank])[row];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dg[e] += fd[e] * ((fx[e] - mean) * rstd);
        db[e] += fd[e];
      }
    }
  float* ws = a.ws + (uint64_t)split * 2 * H;
  put_unit<kF32>(ws, u, full, part, dg);
  put_unit<kF32>(ws + H, u, full, part, db);
}

template <int SRC, int DT, int WT>
__global__ __launch_bounds__(1024) void ln_backward_wide_rows_kernel(LnArgs a) {
  constexpr int TPR = 1024;
  __shared__ float red[2][2][TPR / kWave];
  const int rank = blockIdx.y;
  const uint64_t H = a.hidden, full = H / 8, units = (H + 7) / 8, row_bytes = H * Traits<DT>::B;
  const uint64_t src_bytes = SRC == kE4M3 ? a.row_bytes : row_bytes;
  const uint32_t part = (uint32_t)(H % 8);
  int turn = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint8_t* x = static_cast<const uint8_t*>(a.x[rank]) + row * src_bytes;
    const uint8_t* dy = static_cast<const uint8_t*>(a.dy[rank]) + row * row_bytes;
    const float mean = as_global(a.mean[rank])[row], rstd = as_global(a.rstd[rank])[row];
    float n[8], w[8], g[8], s[2] = {0.0f, 0.0f};
    auto unit = [&](uint64_t u) {
      widen_unit(row_unit<SRC>(x, u, full, part, H, a.glog), n);
      widen_unit(row_unit<DT>(dy, u, full, part), w);
      weight_unit<WT>(a.gamma[rank], 1.0f, u, full, part, g);
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) {
        // past the row's end zero, not -mean rstd, which may be infinite
        // (checkpoint rows are whole units)
        n[e] = SRC == kE4M3 || u < full || e < part ? (n[e] - mean) * rstd : 0.0f;
        w[e] *= g[e];
      }
    };
    for (uint64_t u = threadIdx.x; u < units; u += TPR) {
      unit(u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[0] += w[e];
        s[1] += w[e] * n[e];
      }
    }
    row_sums<TPR, 2>(s, red[turn]);
    turn ^= 1;
    const float c1 = s[0] / (float)H, c2 = s[1] / (float)H;
    for (uint64_t u = threadIdx.x; u < units; u += TPR) {
      unit(u);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = rstd * (w[e] - c1 - n[e] * c2);
      put_unit<DT>(static_cast<uint8_t*>(a.dx[rank]) + row * row_bytes, u, full, part, w);
      if constexpr (SRC == kE4M3) {
        if (a.y[rank]) {
          float b[8];
          weight_unit<WT>(a.beta[rank], 0.0f, u, full, part, b);
#pragma unroll
          for (int e = 0; e < 8; ++e) n[e] = n[e] * g[e] + b[e];
          put_unit<DT>(static_cast<uint8_t*>(a.y[rank]) + row * row_bytes, u, full, part, n);
        }
      }
    }
  }
}

// The weights' gradients: 64 columns to a workgroup, each column's `parts`
// partial sums added by 16 waves (each every 16th, 16 loads in flight) and
// these in order, divided by p for an average, and stored to every rank.
// 4.9 us for 256 x 2 x 7168 (6.5 us with the loads in a plain loop, 8.5 with
// 32 columns to a workgroup).
constexpr int kJoinBlock = 1024, kJoinWays = kJoinBlock / kWave, kJoinLoads = 16;

template <int WT>
__global__ __launch_bounds__(kJoinBlock) void ln_join_kernel(LnJoinArgs a) {
  __shared__ float sums[kJoinWays][kWave];
  const uint32_t col = threadIdx.x % kWave, way = threadIdx.x / kWave;
  const uint64_t cols = a.sums * a.hidden, j = a.first + (uint64_t)blockIdx.x * kWave + col;
  float s = 0.0f;
  if (j < cols) {
    const float* w = as_global(a.ws) + j;
    uint32_t k = way;
    for (; k + (kJoinLoads - 1) * kJoinWays < a.parts; k += kJoinLoads * kJoinWays) {
      float v[kJoinLoads];
#pragma unroll
      for (int i = 0; i < kJoinLoads; ++i) v[i] = w[(uint64_t)(k + i * kJoinWays) * cols];
#pragma unroll
      for (int i = 0; i < kJoinLoads; ++i) s += v[i];
    }
    for (; k < a.parts; k += kJoinWays) s += w[(uint64_t)k * cols];
  }
  sums[way][col] = s;
  __syncthreads();
  if (way != 0 || j >= cols) return;
#pragma unroll
  for (int k = 1; k < kJoinWays; ++k) s += sums[k][col];
  if (a.avg) s /= (float)a.p;
  const bool beta = j >= a.hidden;
  const uint64_t c = beta ? j - a.hidden : j;
  for (int r = 0; r < a.p; ++r) {
    void* to = beta ? a.dbeta[r] : a.dgamma[r];
    if (to) as_global(static_cast<typename Traits<WT>::S*>(to))[c] = narrow1<WT>(s);
  }
}

bool is_wide(const LnArgs& a) {
  int tpr, nu;
  row_shape(a.hidden, &tpr, &nu);
  return !tpr;
}

// The forward pass's arguments n rows on.
void skip_rows(LnArgs& a, uint64_t n, uint64_t row_bytes) {
  for (int r = 0; r < a.ranks; ++r) {
    a.x[r] = (const uint8_t*)a.x[r] + n * row_bytes;
    a.y[r] = (uint8_t*)a.y[r] + n * row_bytes;
    if (a.mean[r]) a.mean[r] += n;
    if (a.rstd[r]) a.rstd[r] += n;
    if (a.ckpt[r]) a.ckpt[r] += n * a.row_bytes;
  }
}

template <int DT, int WT>
int forward_t(const LnArgs& a, bool ckpt, hipStream_t s) {
  if (is_wide(a)) {
    const dim3 grid((uint32_t)std::min<uint64_t>(a.rows, 65536), a.ranks), block(1024);
    if (ckpt) hipLaunchKernelGGL((ln_forward_wide_kernel<DT, WT, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((ln_forward_wide_kernel<DT, WT, false>), grid, block, 0, s, a);
    return (int)hipGetLastError();
  }
  return with_shape(a.hidden, [&](auto T, auto N) {
    constexpr int TPR = decltype(T)::value, NU = decltype(N)::value * 8 / kElems<DT>, RPB = block_of(TPR) / TPR;
    const uint64_t run = RPB * (ckpt ? rows_of<DT, TPR, true>() : rows_of<DT, TPR, false>());
    const dim3 block(block_of(TPR));
    constexpr bool PACKED = TPR < kWave;  // several rows to a wave
    const uint64_t most = most_blocks(block.x) * run;
    LnArgs part = a;
    for (uint64_t left = a.rows; left; skip_rows(part, part.rows, a.hidden * Traits<DT>::B)) {
      part.rows = std::min(left, most);
      left -= part.rows;
      const dim3 grid((uint32_t)((part.rows + run - 1) / run), a.ranks);
      if (ckpt) hipLaunchKernelGGL((ln_forward_kernel<DT, WT, TPR, NU, PACKED, true>), grid, block, 0, s, part);
      else if (PACKED || a.hidden % kElems<DT>) hipLaunchKernelGGL((ln_forward_kernel<DT, WT, TPR, NU, true, false>), grid, block, 0, s, part);
      else hipLaunchKernelGGL((ln_forward_kernel<DT, WT, TPR, NU, PACKED, false>), grid, block, 0, s, part);
      if (const int e = (int)hipGetLastError()) return e;
    }
    return 0;
  });
}

template <int DT, int WT>
int backward_t(const LnArgs& a, uint32_t groups, bool ckpt, hipStream_t s) {
  if (is_wide(a)) {
    const dim3 cols((uint32_t)(wide_chunks(a.hidden) * groups)), rows((uint32_t)std::min<uint64_t>(a.rows, 65536), a.ranks);
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
    constexpr int TPR = decltype(T)::value, NU = decltype(N)::value * 8 / kElems<DT>;
    const dim3 grid(groups), block(block_of(TPR));
    constexpr bool PACKED = TPR < kWave;
    if (ckpt) hipLaunchKernelGGL((ln_backward_kernel<kE4M3, DT, WT, TPR, NU, PACKED>), grid, block, 0, s, a);
    else if (PACKED || a.hidden % kElems<DT>) hipLaunchKernelGGL((ln_backward_kernel<DT, DT, WT, TPR, NU, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((ln_backward_kernel<DT, DT, WT, TPR, NU, PACKED>), grid, block, 0, s, a);
    return (int)hipGetLastError();
  });
}

}  // namespace

// Workgroups of a launch of the backward pass: by the shape alone (results
// and workspace must not depend on the device or on the grid limit).  One
// workgroup of 512 lanes to a CU: 8 x 4096 x 7168 bf16 took 238 us with 256,
// 252 with 512 and 279 with 384, whose second round is short.  Two of 256
// lanes or less: 3 x 1777 x 2565 fp32 took 39 us with 512, 42 with 768, which
// write more partial sums, and 43.5 with 384.  In the wide form as many as one
// launch over all columns may hold (fewer than 256 from 2^27 columns on).
uint32_t ln_backward_groups(int p, uint64_t rows, uint64_t hidden) {
  int tpr, nu;
  row_shape(hidden, &tpr, &nu);
  const uint64_t rpb = tpr ? block_of(tpr) / tpr : 1, all = rows * (uint64_t)std::min(p, kArgRanks), need = (all + rpb - 1) / rpb;
  const uint64_t most = tpr && tpr <= kBlock ? 512 : tpr ? 256 : std::min<uint64_t>(256, most_blocks(kBlock) / wide_chunks(hidden));
  return (uint32_t)std::max<uint64_t>(1, std::min(need, most));
}

// Whether the forward kernel of a width writes checkpoints of such groups:
// a group's lanes must lie in one run of a row's.
bool ln_forward_keeps(int dtype, uint64_t hidden, uint64_t group) {
  int tpr, nu;
  row_shape(hidden, &tpr, &nu);
  return group <= (uint64_t)(tpr == 0 ? 512 : std::min(tpr, kWave) * (dtype == kF32 ? 4 : 8));
}

int launch_ln_forward(int dtype, int wdtype, const LnArgs& a, bool ckpt, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  if (dtype == kF32) return forward_t<kF32, kF32>(a, ckpt, s);
  return wdtype == kF32 ? forward_t<kBF16, kF32>(a, ckpt, s) : forward_t<kBF16, kBF16>(a, ckpt, s);
}

int launch_ln_backward(int dtype, int wdtype, const LnArgs& a, uint32_t groups, bool ckpt, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  if (dtype == kF32) return backward_t<kF32, kF32>(a, groups, ckpt, s);
  return wdtype == kF32 ? backward_t<kBF16, kF32>(a, groups, ckpt, s) : backward_t<kBF16, kBF16>(a, groups, ckpt, s);
}

int launch_ln_join(int wdtype, const LnJoinArgs& args, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  LnJoinArgs a = args;
  const uint64_t blocks = (a.sums * a.hidden + kWave - 1) / kWave, most = most_blocks(kJoinBlock);
  for (uint64_t b = 0; b < blocks; b += most) {
    a.first = b * kWave;
    const dim3 grid((uint32_t)std::min(blocks - b, most)), block(kJoinBlock);
    if (wdtype == kF32) hipLaunchKernelGGL((ln_join_kernel<kF32>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((ln_join_kernel<kBF16>), grid, block, 0, s, a);
    if (const int e = (int)hipGetLastError()) return e;
  }
  return 0;
}

}  // namespace coll
