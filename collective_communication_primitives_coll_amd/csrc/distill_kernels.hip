// The loss of a student, whose logits lie in p shards, against a teacher's top
// entries, and the logits' gradient.
//
// With t the inverse temperature, m = max z, d_j = (z_j - m) t and
// L = log sum e^d_j, so that log p_j = d_j - L; the teacher's entries i have
// log probabilities l_i.
//   renormalised   q_i = e^(l_i - log sum e^l),
//                  loss = sum q_i (log q_i - log p_i),
//                  dz_j = t g (p_j - q_j)             (q_j = 0 off the entries)
//   with a tail    q_i = e^l_i, q_0 = 1 - sum q_i the teacher's mass elsewhere,
//                  p_0 the student's there:
//                  loss = sum q_i (log q_i - log p_i) + q_0 (log q_0 - log p_0),
//                  dz_j = t g (p_j - q_j)             at an entry,
//                         t g (p_0 - q_0) p_j / p_0   elsewhere
// (times max(1, sum q) for the p's, should the q's exceed 1; where no entry
// but the teacher's is allowed, q_0 is the rounding of the others' sum, and
// its class is left out: then the p's are times sum q).  A tail below e^kNone
// of the largest logit holds masks of the type's lowest value alone, and
// counts as none: no difference of such values is left in fp32.
//
// Bound by reading the logits once forward, and by reading and writing them
// backward, with one exponential an element.  The passes are those of the
// log probabilities: a wave to a piece of a row's shard, and a wave that
// joins a row's pieces.
//
// With a tail its sum is not the difference of two sums, which is nothing but
// rounding where the student has learned the teacher's entries: the pieces
// leave the entries out as they pass them, with the tail's own maximum, and
// write down each entry's logit.  An entry's place in its piece is the same
// for the whole wave, so leaving it out takes a lane's one register.
//
// The loss is a small difference of what the two models have: what the join
// computes once a row (the entries' exponentials and logarithms, all sums over
// them) is in 64 bits.  The gradient takes its differences, p_0 - q_0 and the
// entries' p - q, in fp32 from the rounded statistics, as each wave computes
// them: with a = log of the tail's sum, p_0 = e^(a - L) is off by the rounding
// of a and L, up to (|a| + |L| + 12) 2^-24 of it (some 4e-7 for normal logits
// over 50257 entries), and the tail's gradient by as much of t g p_j.
//
// 2048 x 131072 bf16 in 8 shards, 32 entries and a tail: 84-87 us for the
// pieces (537 MB at 6.2-6.4 TB/s), 6 for the join, 168-174 for the gradient
// (6.2-6.4 TB/s).  4 such rows of 20 entries: 9.4 us, of which the pieces take
// 5.1 and the join 3.9, a wave's one chain of loads, sums and stores.
// 777 x 50257 fp32 in 4 shards of odd widths, renormalised: 27, 5 and 53 us.
#include "vocab_pieces.h"

namespace coll {

namespace {

typedef float f32x32 __attribute__((ext_vector_type(32)));
constexpr double kNone = -1e4;
constexpr int kEntryLanes = kMaxDistill / kWave;  // entries to a lane, at most

// A lane's running maximum m (raw) and S = sum 2^d about it.
struct RunningSum {
  float m = -FLT_MAX, s = 0.0f;
  // The product is rounded on its own: fused with one addend of a sum over
  // lanes, it would make that sum another one on every lane.
  __device__ __forceinline__ void rebase(float to, float c) {
#pragma clang fp contract(off)
    s *= __builtin_amdgcn_exp2f((m - to) * c);
    m = to;
  }
};

// A lane's entries of a row (the lane-th, and the 64th after it), as places in
// a run of n elements that starts at vocabulary index `first`; ~0: not there.
template <int NT>
struct Entries {
  uint32_t at[NT];
  __device__ __forceinline__ Entries(const int32_t* idx, int top, uint32_t lane, int64_t first, uint32_t n) {
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const int e = (int)lane + k * kWave;
      const int64_t off = (e < top ? (int64_t)idx[e] : -1) - first;
      at[k] = off >= 0 && off < (int64_t)n ? (uint32_t)off : ~0u;
    }
  }
};

template <int DT, bool TAIL, int NT>
__global__ __launch_bounds__(kBlock) void distill_pieces_kernel(DistillArgs a) {
  constexpr int B = Traits<DT>::B, E = kElems<DT>, kChunk = kStep / E;
  constexpr uint32_t kChunkUnits = kChunk * kWave;
  using S = typename Traits<DT>::S;
  const uint32_t lane = threadIdx.x % kWave;
  const float c = a.scale * kLog2e;
  const Item it(a.plan, a.rows, a.first_row, a.p);
  if (!it.any) return;
  const uint64_t row = it.row, item = row * (uint64_t)a.plan.pieces + (uint64_t)it.piece;
  const int r = it.r;
  const int64_t vocab = a.first_index[r + 1] - a.first_index[r];
  const uint8_t* base = as_global(static_cast<const uint8_t*>(a.logits[r])) + (int64_t)row * a.ld[r] * B;
  const Piece pc = piece_of<DT>(base, vocab, a.plan.len[r], it.piece - a.plan.first[r]);
  const uint8_t* units = base + (pc.begin + pc.head) * B;
  RawUnit<DT, E> cur[kChunk], nxt[kChunk];
  auto load = [&](RawUnit<DT, E> (&to)[kChunk], uint32_t u0) {
    const RowBuffer b(units + (uint64_t)u0 * 16, u0 < pc.units ? min(pc.units - u0, kChunkUnits) * 16 : 0);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) to[i] = load_unit<DT, E, true>(b, (i * kWave + lane) * E);
  };
  const Entries<NT> en(as_global(a.idx) + row * (uint64_t)a.top, a.top, lane, a.first_index[r] + pc.begin, pc.units * E + pc.head + pc.tail);
  load(cur, 0);
  // the elements of both ends, one per lane (head on lanes 0..7, tail on
  // 8..15), and the entries' logits, where they lie in this piece; the others
  // load the shard's first element, so that nothing waits here
  const S* elems = reinterpret_cast<const S*>(base);
  uint32_t end_at = ~0u - 1;  // from the piece's first element
  if (lane < pc.head) end_at = lane;
  else if (lane >= 8 && lane - 8 < pc.tail) end_at = pc.head + pc.units * E + lane - 8;
  const S end_raw = elems[end_at < ~0u - 1 ? pc.begin + end_at : 0];
  S z_raw[NT];
#pragma unroll
  for (int k = 0; k < NT; ++k) z_raw[k] = elems[en.at[k] != ~0u ? pc.begin + en.at[k] : 0];

  RunningSum run;
  for (uint32_t u0 = 0; u0 < pc.units; u0 += kChunkUnits) {
    load(nxt, u0 + kChunkUnits);
    if (pc.units - u0 < kChunkUnits) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (u0 + i * kWave + lane >= pc.units) cur[i] = masked_unit<DT>();
    }
    f32x32 f;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      float v[E];
      widen_unit(cur[i], v);
#pragma unroll
      for (int e = 0; e < E; ++e) f[i * E + e] = v[e];
    }
    if constexpr (TAIL) {
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        const uint32_t o = en.at[k] - pc.head - u0 * E;  // (huge where it is in no unit, or in an earlier one)
        unsigned long long hits = __ballot(en.at[k] != ~0u && o < (uint32_t)kLogprobStep);
        for (; hits; hits &= hits - 1) {
          const uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)o, __builtin_ctzll(hits));
          const uint32_t pos = w / (E * kWave) * E + w % E;
          f[pos] = w / E % kWave == lane ? -__builtin_inff() : f[pos];
        }
      }
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kStep; ++i) top = fmaxf(top, f[i]);
    run.rebase(fmaxf(run.m, top), c);
    float s[4] = {};
#pragma unroll
    for (int i = 0; i < kStep; ++i) s[i % 4] += __builtin_amdgcn_exp2f((f[i] - run.m) * c);
    run.s += sum_of(s);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) cur[i] = nxt[i];
  }
  if (pc.head + pc.tail) {
    float end = end_at < ~0u - 1 ? widen1<DT>(end_raw) : -__builtin_inff();
    if constexpr (TAIL) {
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        unsigned long long hits = __ballot(en.at[k] != ~0u && (en.at[k] < pc.head || en.at[k] - pc.head >= pc.units * E));
        for (; hits; hits &= hits - 1)
          if ((uint32_t)__builtin_amdgcn_readlane((int)en.at[k], __builtin_ctzll(hits)) == end_at) end = -__builtin_inff();
      }
    }
    run.rebase(fmaxf(run.m, end), c);
    run.s += __builtin_amdgcn_exp2f((end - run.m) * c);
  }
  run.rebase(wave_max(run.m), c);
  run.s = wave_sum(run.s);
  if (lane == 0) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    reinterpret_cast<f32x2*>(as_global(a.part))[item] = f32x2{run.m, run.s};
  }
#pragma unroll
  for (int k = 0; k < NT; ++k)
    if (en.at[k] != ~0u) as_global(a.zs)[row * (uint64_t)a.top + k * kWave + lane] = widen1<DT>(z_raw[k]);
}

// Sums of 64-bit values over a wave, on every lane, in wave_fold's order; N at
// once, whose steps hide each other's latency.
__device__ __forceinline__ double halves(uint32_t lo, uint32_t hi) { return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo); }
template <int CTRL>
__device__ __forceinline__ double dpp_move(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return halves((uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, false),
                (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, false));
}
template <int N>
__device__ __forceinline__ void wave_sums64(double (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] += dpp_move<0xB1>(v[k]);   // quad_perm 1,0,3,2
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] += dpp_move<0x4E>(v[k]);   // quad_perm 2,3,0,1
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] += dpp_move<0x141>(v[k]);  // row_half_mirror
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] += dpp_move<0x140>(v[k]);  // row_mirror
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v[k]);
    const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    v[k] = halves(lo[0], hi[0]) + halves(lo[1], hi[1]);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v[k]);
    const auto lo = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    v[k] = halves(lo[0], hi[0]) + halves(lo[1], hi[1]);
  }
}

// A wave to a row, a lane to a piece and to one or two entries.
template <int NT>
__global__ __launch_bounds__(kBlock) void distill_join_kernel(DistillJoinArgs a) {
  const int lane = (int)(threadIdx.x % kWave);
  const float c = a.scale * kLog2e, inf = __builtin_inff(), nan = __uint_as_float(0x7fc00000u);
  const uint32_t in = blockIdx.x * (kBlock / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (in >= a.rows) return;
  const uint64_t row = a.first_row + in;
  // (asked for first: needed last)
  float *stats = a.stats[min(lane, a.p - 1)], *losses = a.loss[min(lane, a.p - 1)];
  RunningSum run;
  if (lane < a.pieces) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 rec = reinterpret_cast<const f32x2*>(as_global(a.part))[row * (uint64_t)a.pieces + lane];
    run.m = rec[0];
    run.s = rec[1];
  }
  int32_t id[NT];
  float l[NT], z[NT];
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    const int e = lane + k * kWave;
    const uint64_t at = row * (uint64_t)a.top + (e < a.top ? e : 0);
    id[k] = e < a.top ? as_global(a.idx)[at] : -1;
    l[k] = as_global(a.logp)[at];
    if (l[k] == inf) l[k] = nan;
    const bool ok = id[k] >= 0 && id[k] < a.vocab;
    if (!ok) id[k] = -1;
    const float zi = as_global(a.zs)[at];  // (not written where the entry is in no shard)
    z[k] = ok ? zi : -inf;
  }
  // An index's first entry counts: later ones' lanes as bits, eight entries at
  // a time to compare with (those past the last have no index, and nothing to
  // lose).
  uint64_t again[NT] = {};
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int most = min(a.top - j * kWave, kWave);
    for (int b0 = 0; b0 < most; b0 += 8) {
#pragma unroll
      for (int b = b0; b < b0 + 8; ++b) {
        const int32_t other = __builtin_amdgcn_readlane(id[j], b);
#pragma unroll
        for (int k = j; k < NT; ++k) again[k] |= __ballot(id[k] == other) & (k > j ? ~0ull : ~1ull << b);
      }
    }
  }
  bool counts[NT];
  bool any = false;
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    counts[k] = id[k] >= 0 && !(again[k] >> lane & 1) && (a.tail || l[k] != -inf);
    any = any || counts[k];
  }
  any = __any(any);
  const float mt = wave_max(run.m);
  run.rebase(mt, c);
  const float st = wave_sum(run.s);
  const double scale = a.scale;
  // Over the entries, with e their masses (about the largest where they are to
  // be normalised) and d the student's exponents: sum e, sum e (l - d), and with
  // a tail sum e^d.  The loss then only wants the logarithms of sums.
  float m = mt, lm = -inf;
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    if (a.tail) m = fmaxf(m, counts[k] ? z[k] : -inf);
    else lm = fmaxf(lm, counts[k] ? l[k] : -inf);
  }
  m = wave_max(m);
  lm = a.tail ? 0.0f : wave_max(lm);
  double s[3] = {0.0, 0.0, 0.0};
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    const double d = ((double)z[k] - m) * scale, e = counts[k] ? exp((double)l[k] - lm) : 0.0;
    s[0] += e;
    s[1] += e == 0.0 ? 0.0 : e * (l[k] - d);
    s[2] += counts[k] ? exp(d) : 0.0;
  }
  const double far = ((double)mt - m) * scale;
  double third = log((double)st) + far, fourth = 0.0, sum = st == 0.0f ? 0.0 : st * exp(far);
  wave_sums64(s);
  if (a.tail) {
    sum += s[2];
    if (third < kNone) third = -inf;  // (also of an empty sum)
    fourth = 1.0 - s[0];
  } else {
    third = log(s[0]) + lm;
  }
  // (comparisons that a NaN fails)
  const bool poison = !(sum >= 0.0), empty = sum == 0.0;
  const double log_s = log(sum);
  double loss = a.tail ? s[1] + (s[0] == 0.0 ? 0.0 : s[0] * log_s) : s[1] / s[0] - third + log_s;
  if (a.tail && !(fourth <= 0.0) && third != -inf) loss += fourth * (log(fourth) - (third - log_s));
  if (lane < a.p) {
    typedef float f32x4_e __attribute__((ext_vector_type(4), aligned(4)));
    f32x4_e out;
    out[0] = poison ? nan : empty ? -inf : m;
    out[1] = poison ? nan : empty ? -inf : (float)log_s;
    // one NaN on every rank, whatever lane it comes from
    out[2] = !any ? inf : poison || third != third ? nan : (float)third;
    out[3] = !any ? 0.0f : poison || fourth != fourth ? nan : (float)fourth;
    *reinterpret_cast<f32x4_e*>(as_global(stats) + row * 4) = out;
    as_global(losses)[row] = !any ? 0.0f : poison ? nan : empty ? inf : loss != loss ? nan : (float)loss;
  }
}

// Gradient.  Waves and pieces as in the log probabilities' gradient.
constexpr int kGradUnits = 2;

// A row's gradient off the entries: dz = A 2^d, d = log2 e ((z - m) t - shift).
struct DistillRow {
  float c, m, shift, a;
  // d as written
  __device__ __forceinline__ float far(float z) const { return a * __builtin_amdgcn_exp2f((z - m) * c - shift); }
  // d as one fma, z c - K for the rounded K = m c + shift.  It is off by the
  // exactly known eps, which went into a.
  __device__ __forceinline__ float near(float z) const { return a * __builtin_amdgcn_exp2f(__builtin_fmaf(z, c, -shift)); }
  __device__ __forceinline__ bool make_near() {
#pragma clang fp contract(off)
    if (!(fabsf(m) < 1e4f && c < 100.0f && fabsf(shift) < 1e6f)) return false;
    const float mc = m * c, k = mc + shift, back = k - mc;  // rounded each
    a *= __builtin_amdgcn_exp2f(-(__builtin_fmaf(m, c, -mc) + ((mc - (k - back)) + (shift - back))));
    shift = k;
    return true;
  }
};

template <int DT, int NT>
__global__ __launch_bounds__(kBlock) void distill_grad_kernel(DistillGradArgs a, LogprobPlan plan) {
  constexpr int B = Traits<DT>::B, E = kElems<DT>, N = kGradUnits * E;
  typedef float Held __attribute__((ext_vector_type(N)));
  using S = typename Traits<DT>::S;
  const uint32_t lane = threadIdx.x % kWave;
  const Item it(plan, a.rows, a.first_row, a.p);
  if (!it.any) return;
  const uint64_t row = it.row;
  const int r = it.r;
  const int64_t vocab = a.first_index[r + 1] - a.first_index[r];
  const uint8_t* base = as_global(static_cast<const uint8_t*>(a.logits[r])) + (int64_t)row * a.ld[r] * B;
  uint8_t* out = as_global(static_cast<uint8_t*>(a.dlogits[r])) + (int64_t)row * a.dld[r] * B;
  const Piece pc = piece_of<DT>(base, vocab, kGradUnits * kWave * E, it.piece - plan.first[r]);
  const RowBuffer units(base + (pc.begin + pc.head) * B, pc.units * 16);
  const RowBuffer outs(out + (pc.begin + pc.head) * B, pc.units * 16);
  RawUnit<DT, E> x[kGradUnits];
#pragma unroll
  for (int i = 0; i < kGradUnits; ++i) x[i] = load_unit<DT, E, true>(units, (i * kWave + lane) * E);
  const Entries<NT> en(as_global(a.idx) + row * (uint64_t)a.top, a.top, lane, a.first_index[r] + pc.begin, pc.units * E + pc.head + pc.tail);

  const float third = ld_const(a.stats + 4 * row + 2), fourth = ld_const(a.stats + 4 * row + 3);
  const float log_s = ld_const(a.stats + 4 * row + 1), g = ld_const(a.dloss + row) * a.scale;
  DistillRow d;
  d.c = a.scale * kLog2e;
  d.m = ld_const(a.stats + 4 * row);
  // nothing to learn from, or nothing allowed: no gradient, whatever the logits hold
  const bool none = third == __builtin_inff() || d.m == -__builtin_inff();
  float whole = 1.0f;
  if (a.tail) {
    // (comparisons that let a NaN through)
    const float rest = !(fourth <= 0.0f) ? fourth : 0.0f;
    const bool no_tail = third == -__builtin_inff();
    whole = !(fourth >= 0.0f) || no_tail ? 1.0f - fourth : 1.0f;
    d.a = no_tail ? 0.0f : g * (whole * __builtin_amdgcn_exp2f((third - log_s) * kLog2e) - rest);
    d.shift = no_tail ? 0.0f : third * kLog2e;
  } else {
    d.a = g + (third - third);
    d.shift = log_s * kLog2e;
  }
  const float m = d.m;
  const bool near = d.make_near();
  Held f;
  {
    float v[kGradUnits][E];
#pragma unroll
    for (int i = 0; i < kGradUnits; ++i) widen_unit(x[i], v[i]);
    if (near) {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = d.near(v[i / E][i % E]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = d.far(v[i / E][i % E]);
    }
  }
  const S* elems = reinterpret_cast<const S*>(base);
  uint32_t end_at = ~0u - 1;  // from the piece's first element
  if (lane < pc.head) end_at = lane;
  else if (lane >= 8 && lane - 8 < pc.tail) end_at = pc.head + pc.units * E + lane - 8;
  float end = 0.0f;
  if (end_at < ~0u - 1) {
    const float z = widen1<DT>(elems[pc.begin + end_at]);
    end = near ? d.near(z) : d.far(z);
  }
  // The entries take the place of what was computed there, from the last to
  // the first, so that an index's first entry stays.
#pragma unroll
  for (int k = NT - 1; k >= 0; --k) {
    float v = 0.0f;
    if (en.at[k] != ~0u) {
      const float z = widen1<DT>(elems[pc.begin + en.at[k]]);
      const float l = as_global(a.logp)[row * (uint64_t)a.top + k * kWave + lane];
      const float q = __builtin_amdgcn_exp2f((a.tail ? l : l - third) * kLog2e);
      v = g * (whole * __builtin_amdgcn_exp2f(((z - m) * a.scale - log_s) * kLog2e) - q);
    }
    for (unsigned long long hits = __ballot(en.at[k] != ~0u); hits;) {
      const int b = 63 - __builtin_clzll(hits);
      hits &= ~(1ull << b);
      const uint32_t at = (uint32_t)__builtin_amdgcn_readlane((int)en.at[k], b), w = at - pc.head;
      const float to = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), b));
      if (at >= pc.head && w < pc.units * E) {
        const uint32_t pos = w / (E * kWave) * E + w % E;
        f[pos] = w / E % kWave == lane ? to : f[pos];
      } else if (at == end_at) {
        end = to;
      }
    }
  }
  if (none) {
    f = 0.0f;
    end = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kGradUnits; ++i) {
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = f[i * E + e];
    store_unit<DT, E, true>(outs, (i * kWave + lane) * E, narrow_unit<DT, E>(v));
  }
  if (end_at < ~0u - 1) reinterpret_cast<S*>(out)[pc.begin + end_at] = narrow1<DT>(end);
}

}  // namespace

int launch_distill(int dtype, const DistillArgs& args, const DistillJoinArgs& join, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  DistillArgs a = args;
  const dim3 block(kBlock);
  const int e = over_rows(args.rows, (uint64_t)a.plan.pieces, [&](uint64_t first, uint64_t rows, dim3 grid) {
    a.first_row = first;
    a.rows = rows;
    auto go = [&](auto D, auto T, auto N) {
      hipLaunchKernelGGL((distill_pieces_kernel<decltype(D)::value, decltype(T)::value, decltype(N)::value>), grid, block, 0, s, a);
    };
    auto by_top = [&](auto D, auto T) {
      if (a.top <= kWave) go(D, T, std::integral_constant<int, 1>());
      else go(D, T, std::integral_constant<int, kEntryLanes>());
    };
    auto by_kind = [&](auto D) {
      if (join.tail) by_top(D, std::true_type());
      else by_top(D, std::false_type());
    };
    if (dtype == kF32) by_kind(std::integral_constant<int, kF32>());
    else by_kind(std::integral_constant<int, kBF16>());
  });
  if (e) return e;
  DistillJoinArgs j = join;
  return over_rows(args.rows, 1, [&](uint64_t first, uint64_t rows, dim3 grid) {
    j.first_row = first;
    j.rows = rows;
    if (j.top <= kWave) hipLaunchKernelGGL((distill_join_kernel<1>), grid, block, 0, s, j);
    else hipLaunchKernelGGL((distill_join_kernel<kEntryLanes>), grid, block, 0, s, j);
  });
}

int launch_distill_backward(int dtype, const DistillGradArgs& args, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  DistillGradArgs a = args;
  const int64_t B = dtype == kF32 ? 4 : 2, len = kGradUnits * kWave * 16 / B;
  LogprobPlan plan{};
  for (int r = 0; r < a.p; ++r) {
    const int64_t before = a.ld[r] * B % kLine ? kLine / B - 1 : (int64_t)((uintptr_t)a.logits[r] % kLine) / B;
    plan.first[r + 1] = plan.first[r] + pieces_of(a.first_index[r + 1] - a.first_index[r], before, len);
  }
  finish_plan(&plan, a.p);
  return over_rows(args.rows, (uint64_t)plan.pieces, [&](uint64_t first, uint64_t rows, dim3 grid) {
    a.first_row = first;
    a.rows = rows;
    const dim3 block(kBlock);
    const bool few = a.top <= kWave;
    if (dtype == kF32) {
      if (few) hipLaunchKernelGGL((distill_grad_kernel<kF32, 1>), grid, block, 0, s, a, plan);
      else hipLaunchKernelGGL((distill_grad_kernel<kF32, kEntryLanes>), grid, block, 0, s, a, plan);
    } else {
      if (few) hipLaunchKernelGGL((distill_grad_kernel<kBF16, 1>), grid, block, 0, s, a, plan);
      else hipLaunchKernelGGL((distill_grad_kernel<kBF16, kEntryLanes>), grid, block, 0, s, a, plan);
    }
  });
}

}  // namespace coll
