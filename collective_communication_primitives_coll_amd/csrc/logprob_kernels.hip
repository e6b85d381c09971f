// Log probabilities of given tokens, entropy and top alternatives over a
// vocabulary whose logits lie in p shards, and the logits' gradient.
//
// With T the temperature, per row over the whole vocabulary:
//   m = max z,  d_j = (z_j - m) / T,  S = sum e^d_j,
//   log p_j = d_j - log S,   H = log S - (sum e^d_j d_j) / S,
//   dz_j = (gl (1[j = target] - p_j) - gh p_j (log p_j + H)) / T
// (gl, gh: the gradients of the target's log probability and of H).
//
// Forward is bound by reading the logits once: 2 bytes an element in bf16
// against some 10 fp32 operations, one of them an exponential (quarter
// rate), which is near the balance of the card.  A row's shards are cut
// into pieces, one wave to a piece: as many as keep the card busy when
// there are few rows, one or two per shard when there are many.  A lane
// keeps its own running maximum and its sums about it (one rescale per
// chunk of 32 elements), and the lanes meet once, at the piece's end.
// The join kernel, a wave to a row and a lane to a piece, does what
// the AllReduce of maxima and sums over the ranks would, finds the
// alternatives, and stores the results to every rank.
//
// Alternatives.  A piece also writes down the largest element of each group
// of eight lanes and a step (or a few, so that a row has 1024 groups at
// most), which costs little beside the running maximum.  64 lanes' shares of
// a row's groups bound its k best elements from below by the k-th largest of
// theirs, and few groups reach the bound: the join wave reads those again,
// whole 128-byte lines, and ranks the elements that reach it by counting.
// 2048 rows of 131072 bf16: 88 us without alternatives, 102 us with 8, of
// which the join takes 4 and 10: one wave's chain of loads, searches and
// stores, as long for 4 rows (15 us in all) as for 2048.
// A row of fewer than k groups has no such bound (8 groups to 2048 entries of
// a shard where there are many rows: up to 4096 entries with 20 alternatives,
// up to 6144 with 32).  Every unmasked element then counts as reaching it, and
// from 257 of them on the row is searched again, by insertion.  8192 rows of
// 4000 bf16 in one shard: 21 us without alternatives, 37 with 8, 80 with 20.
// (Insertion into a sorted list while the chunks came took 120 us; a search
// in each piece, whose end no other work hides, 127 us; groups of one lane's
// elements over a whole piece, each in a line of its own, 110 us.)
//
// Sums run in base 2 (v_exp_f32), in fp32.  A difference to the maximum is
// one fma, whose known rounding is taken back out of the sums; where the
// maximum or the scale is large, or an entry masked, it is taken before the
// scaling, so that large logits lose nothing, and held at -16384 or more
// where it multiplies a sum, so that no 0 * inf arises.  The
// running maximum starts at the lowest finite value: a masked entry
// (-infinity) then always contributes zero, and a row with nothing else
// has S = 0.  A NaN or +infinity makes S a NaN.
//
// Gradient: 4 bytes an element in bf16, read once and written once.  4096 x
// 65536 bf16 in 8 shards: 171 us, 6.28 TB/s, what a stream read and written
// one to one reaches on this card.
#include "vocab_pieces.h"

namespace coll {

namespace {

// Where the sums take one fma an element for its difference to the maximum:
// eps, at most 2^-24 of |m c|, is then at most 2^-5 (|m c| stays below 2^20),
// small enough to be taken back out with a factor near 1.
constexpr float kPlainMax = 1e4f, kPlainScale = 100.0f;

// The order of fp32 values as unsigned integers (both zeros alike).
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

constexpr uint32_t kMaskedOrder = 0x007fffffu;  // of -infinity

// Keys of alternatives: the order of the value above the complement of the
// index, so that the larger key is the better entry and the lower index wins
// a tie.
__device__ __forceinline__ unsigned long long key_of(float v, uint32_t index) {
  return ((unsigned long long)order_of(v) << 32) | (uint32_t)~index;
}

// The `top` largest unmasked elements of a wave, one per lane in descending
// order, built by insertion.  An empty place is 0, below every key.  bar: no
// key at or below it can enter.
struct TopList {
  unsigned long long key = 0, bar = ((unsigned long long)kMaskedOrder << 32) | 0xffffffffu;

  __device__ __forceinline__ void insert(unsigned long long k, int top) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(-1, (int)(uint32_t)key, 0x138 /* wave_shr:1 */, 0xf, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(-1, (int)(uint32_t)(key >> 32), 0x138, 0xf, 0xf, false);
    const unsigned long long before = ((unsigned long long)hi << 32) | lo;
    key = key > k ? key : before > k ? k : before;
    const unsigned long long last = lane_value(key, top - 1);
    if (last > bar) bar = last;
  }

  // A lane's E elements, the first at vocabulary index `index` (`in`: the
  // lane has any), and the largest of them: each round offers every lane's
  // best and takes it out (NaN, which no comparison finds), until none can
  // enter.
  template <int E>
  __device__ __forceinline__ void consider(float (&f)[E], float best, uint32_t index, bool in, int top) {
    while (true) {
      uint32_t e0 = 0;
#pragma unroll
      for (int e = E - 1; e >= 0; --e) e0 = f[e] == best ? (uint32_t)e : e0;
      const unsigned long long k = in && best == best ? key_of(best, index + e0) : 0;
      if (!__any(k > bar)) break;
      offer(k, top);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = e0 == (uint32_t)e ? __uint_as_float(0x7fc00000u) : f[e];
      best = f[0];
#pragma unroll
      for (int e = 1; e < E; ++e) best = fmaxf(best, f[e]);
    }
  }

  // Every lane offers one key (0: none).
  __device__ __forceinline__ void offer(unsigned long long k, int top) {
    unsigned long long want = __ballot(k > bar);
    while (want) {
      const int l = __builtin_ctzll(want);
      insert(lane_value(k, l), top);
      want = __ballot(k > bar) & ~((2ull << l) - 1);
    }
  }

  static __device__ __forceinline__ unsigned long long lane_value(unsigned long long v, int l) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), l);
    return ((unsigned long long)hi << 32) | lo;
  }
};

// A lane's running maximum m (raw), S = sum 2^d and A = sum 2^d d about it.
struct Running {
  float m = -FLT_MAX, s = 0.0f, a = 0.0f;

  __device__ __forceinline__ void rebase(float to, float c) {
    const float d = fmaxf((m - to) * c, kFar), k = __builtin_amdgcn_exp2f(d);
    a = (a + s * d) * k;
    s *= k;
    m = to;
  }
  __device__ __forceinline__ void wave_join(float c) {
    rebase(wave_max(m), c);
    // The products are rounded here: fused with one addend of the sums, they
    // would make these sums other ones on every lane, and so on every rank.
    asm volatile("" : "+v"(s), "+v"(a));
    s = wave_sum(s);
    a = wave_sum(a);
  }
};

// How many of a row's 16 values, each lane's row of 16, reach `mine`.
template <int N = 0>
__device__ __forceinline__ int reached_by(float y, float mine) {
  const int one = dpp_move<N ? 0x120 + N : 0xE4>(y) >= mine;  // row_ror:N (0: as it is)
  if constexpr (N < 15) return one + reached_by<N + 1>(y, mine);
  return one;
}
// A bound that at least `top` lanes reach (or that all unmasked elements do,
// where fewer lanes have a group with any).
__device__ __forceinline__ float bar_of(float mine, int top) {
  // the wave's four rows of 16 lanes, each on all rows
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(mine), __float_as_uint(mine), false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(a[0], a[0], false, false);
  const auto c = __builtin_amdgcn_permlane32_swap(a[1], a[1], false, false);
  uint32_t y[4] = {b[0], b[1], c[0], c[1]};
  int reached = 0;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    reached += reached_by(__uint_as_float(y[0]), mine);
    y[0] = y[1];
    y[1] = y[2];
    y[2] = y[3];
  }
  return fmaxf(wave_max(reached >= top ? mine : -FLT_MAX), -FLT_MAX);
}

// Entries that a wave collects in LDS; n counts also those past its end.
template <class T, uint32_t MOST>
struct Bag {
  T* at;
  uint32_t n = 0;
  __device__ __forceinline__ void push(T v, bool in) {
    const unsigned long long mask = __ballot(in);
    if (!mask) return;
    const uint32_t i = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
    if (in && i < MOST) at[i] = v;
    n += (uint32_t)__popcll(mask);
  }
  __device__ __forceinline__ bool full() const { return n > MOST; }
};
constexpr uint32_t kBagMost = 256;
struct JoinStore {
  u32x4 groups[kBagMost];
  unsigned long long keys[kBagMost];
  unsigned long long sorted[kMaxTop];
};

template <int DT, bool TOP>
__global__ __launch_bounds__(kBlock) void logprob_pieces_kernel(LogprobArgs a) {
  constexpr int B = Traits<DT>::B, E = kElems<DT>, kChunk = kStep / E;
  constexpr uint32_t kChunkUnits = kChunk * kWave;
  const uint32_t lane = threadIdx.x % kWave;
  const float c = a.scale * kLog2e;
  const Item it(a.plan, a.rows, a.first_row, a.p);
  if (!it.any) return;
  const uint64_t row = it.row, item = row * (uint64_t)a.plan.pieces + (uint64_t)it.piece;
  const int piece = it.piece, r = it.r;
  const int64_t vocab = a.first_index[r + 1] - a.first_index[r];
  const uint8_t* base = as_global(static_cast<const uint8_t*>(a.logits[r])) + (int64_t)row * a.ld[r] * B;
  const Piece pc = piece_of<DT>(base, vocab, a.plan.len[r], piece - a.plan.first[r]);
  const uint8_t* units = base + (pc.begin + pc.head) * B;
  const uint32_t index0 = (uint32_t)(a.first_index[r] + pc.begin);  // vocabulary index of the piece's first element

  Running run;
  // the largest of the lane's elements in this segment
  float best = -__builtin_inff();
  float* bests = as_global(a.bests) + item * (uint64_t)(a.plan.segs * kSegGroups) + lane / kGroupLanes;
  int seg = 0, left = a.plan.seg_steps;
  auto note = [&] {
    best = wave_max<kGroupLanes>(best);
    if (lane % kGroupLanes == 0) bests[seg * kSegGroups] = best;
    best = -__builtin_inff();
    ++seg;
    left = a.plan.seg_steps;
  };
  // whether the cheap form of the sums holds so far: no masked entries
  bool plain = c < kPlainScale;
  // Loads without a branch: past the end they return zeros, which the last
  // step replaces.
  RawUnit<DT, E> cur[kChunk], nxt[kChunk];
  auto load = [&](RawUnit<DT, E> (&to)[kChunk], uint32_t u0) {
    const RowBuffer b(units + (uint64_t)u0 * 16, u0 < pc.units ? min(pc.units - u0, kChunkUnits) * 16 : 0);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) to[i] = load_unit<DT, E, true>(b, (i * kWave + lane) * E);
  };
  load(cur, 0);
  // the elements of both ends, one per lane (head on lanes 0..7, tail on
  // 8..15), and the target's logit, where they lie in this piece; the
  // others load the shard's first element, so that nothing waits here
  using S = typename Traits<DT>::S;
  const S* elems = reinterpret_cast<const S*>(base);
  int64_t end_off = -1;
  if (lane < pc.head) end_off = pc.begin + lane;
  else if (lane >= 8 && lane - 8 < pc.tail) end_off = pc.begin + pc.head + (int64_t)pc.units * E + lane - 8;
  const S end_raw = elems[max(end_off, (int64_t)0)];
  const int64_t t_off = ld_const(a.targets + row) - a.first_index[r] - pc.begin;
  const bool t_in = t_off >= 0 && t_off < (int64_t)pc.units * E + pc.head + pc.tail;
  const S t_raw = elems[t_in ? pc.begin + t_off : 0];
  for (uint32_t u0 = 0; u0 < pc.units; u0 += kChunkUnits) {
    const bool more = u0 + kChunkUnits < pc.units;
    load(nxt, u0 + kChunkUnits);
    if (pc.units - u0 < kChunkUnits) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (u0 + i * kWave + lane >= pc.units) cur[i] = masked_unit<DT>();
    }
    float f[kChunk][E], top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      widen_unit(cur[i], f[i]);
      top = fmaxf(top, largest(f[i]));
    }
    run.rebase(fmaxf(run.m, top), c);
    float s[kChunk] = {}, w[kChunk] = {}, ds, dw;
    if (plain && __all(fabsf(run.m) < kPlainMax)) {
      // one fma an element: d = z c - M for the rounded M = m c, which is
      // off the true difference by the exactly known eps
      const float M = run.m * c, eps = __builtin_fmaf(run.m, c, -M);
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float d = __builtin_fmaf(f[i][e], c, -M), x = __builtin_amdgcn_exp2f(d);
          s[i] += x;
          w[i] = __builtin_fmaf(x, d, w[i]);
        }
      const float k = __builtin_amdgcn_exp2f(-eps);
      ds = sum_of(s) * k;
      dw = sum_of(w) * k - eps * ds;
      // a masked entry (0 * inf) or a NaN shows here
      plain = __all(dw == dw);
    } else {
      plain = false;
    }
    if (!plain) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        s[i] = w[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float d = (f[i][e] - run.m) * c, x = __builtin_amdgcn_exp2f(d);
          s[i] += x;
          w[i] += x * fmaxf(d, kFar);
        }
      }
      ds = sum_of(s);
      dw = sum_of(w);
    }
    run.s += ds;
    run.a += dw;
    if constexpr (TOP) {
      best = fmaxf(best, top);
      if (--left == 0 || !more) note();
    }
#pragma unroll
    for (int i = 0; i < kChunk; ++i) cur[i] = nxt[i];
  }
  if (pc.head + pc.tail) {
    const float end = end_off >= 0 ? widen1<DT>(end_raw) : -__builtin_inff();
    run.rebase(fmaxf(run.m, end), c);
    const float d = (end - run.m) * c, x = __builtin_amdgcn_exp2f(d);
    run.s += x;
    run.a += x * fmaxf(d, kFar);
  }
  run.wave_join(c);
  if (lane == 0) {
    const float z = t_in ? widen1<DT>(t_raw) : -__builtin_inff();
    const u32x4 rec = {__float_as_uint(run.m), __float_as_uint(run.s), __float_as_uint(run.a), __float_as_uint(z)};
    reinterpret_cast<u32x4*>(as_global(a.part))[item] = rec;
    if constexpr (TOP) {
      // where the piece lies: address of its units (and, above it, the
      // elements before and after them), their number, first index
      const uint64_t where = (uint64_t)(uintptr_t)units | (uint64_t)pc.head << 56 | (uint64_t)pc.tail << 60;
      const u32x4 place = {(uint32_t)where, (uint32_t)(where >> 32), pc.units, index0 + pc.head};
      reinterpret_cast<u32x4*>(as_global(a.places))[item] = place;
    }
  }
  if constexpr (TOP) {
    while (seg < a.plan.segs) note();
  }
}

// What the join needs beside its output pointers.
struct JoinInput {
  const float* part;
  const uint32_t* places;
  const float* bests;
  const int64_t* targets;
  uint64_t rows, first_row;
  int64_t vocab;
  float scale;
  int p, top, pieces, segs, seg_steps;
};

// The largest elements of a row's groups, kLoads to a lane, in one go.
constexpr int kLoads = kMaxGroups / kWave;
__device__ __forceinline__ void load_bests(const JoinInput& a, uint64_t row, int lane, float (&v)[kLoads]) {
  const int n = a.pieces * a.segs * kSegGroups;
  const float* bests = as_global(a.bests) + row * (uint64_t)n;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) v[i] = i * kWave + lane < n ? bests[i * kWave + lane] : -__builtin_inff();
}

// A piece as its wave wrote it down: the address of its units, the elements
// before and after them, their number, the vocabulary index of their first.
struct Place {
  const uint8_t* units;
  uint32_t head, tail, n, index;
  __device__ __forceinline__ Place(u32x4 v)
      : units(as_global((const uint8_t*)(uintptr_t)((((uint64_t)v[1] << 32) | v[0]) & 0xffffffffffffffull))),
        head(v[1] >> 24 & 15), tail(v[1] >> 28), n(v[2]), index(v[3]) {}
};
__device__ __forceinline__ u32x4 lane_place(u32x4 place, int lane) {
  u32x4 v;
#pragma unroll
  for (int d = 0; d < 4; ++d) v[d] = (uint32_t)__shfl((int)place[d], lane);
  return v;
}

// The k best elements of a row, one per lane in descending order (0: fewer).
// place: this lane's piece; v: load_bests.  One wave runs through this code
// once, so it is short rather than unrolled.
template <int DT>
__device__ __forceinline__ unsigned long long row_best(const JoinInput& a, uint64_t row, u32x4 place, const float (&v)[kLoads], int lane,
                                                       JoinStore& st) {
  using S = typename Traits<DT>::S;
  constexpr int E = kElems<DT>;
  const float bar = bar_of(largest(v), a.top);
  // The groups whose elements reach the bar, as the address of their first
  // unit, the units from there to the piece's end, the first's index.
  Bag<u32x4, kBagMost> groups{st.groups};
  uint32_t hits = 0;
#pragma unroll
  for (int i = kLoads - 1; i >= 0; --i) hits = hits + hits + (v[i] >= bar);  // bit i
  for (; __any(hits != 0); hits &= hits - 1) {
    const uint32_t id = (uint32_t)__builtin_ctz(hits | 1u << 31) * kWave + lane, seg = id / kSegGroups;
    const uint32_t piece = seg / (uint32_t)a.segs, round = (seg - piece * a.segs) * (uint32_t)a.seg_steps * (kStep / E);
    const Place pl(lane_place(place, (int)(piece % kWave)));
    const uint32_t u = round * kWave + id % kSegGroups * kGroupLanes;
    const uint64_t at = (uint64_t)(uintptr_t)pl.units + (uint64_t)u * 16;
    groups.push(u32x4{(uint32_t)at, (uint32_t)(at >> 32), pl.n - u, pl.index + u * E}, hits != 0);
  }
  wave_fence();
  // Their units, a power of two of lanes to a group, four units to a lane,
  // loaded without a branch (what lies past an end from the row's own `part`, and masked).
  constexpr int kBatch = 4, kWords = 4 * kBatch;
  Bag<unsigned long long, kBagMost> keys{st.keys};
  const uint32_t units_of = (uint32_t)a.seg_steps * (kStep / E) * kGroupLanes, wide = min(units_of, (uint32_t)kWave), per = kWave / wide;
  const uint32_t lane_g = wide == kWave ? 0 : lane / 32, lane_m = wide == kWave ? lane : lane % 32;
  const uint32_t count = groups.full() ? 0 : groups.n;
  const uint64_t other = (uint64_t)(uintptr_t)a.part + row * (uint64_t)a.pieces * 16;
  for (uint32_t g0 = 0; g0 < count; g0 += kBatch * per)
    for (uint32_t m1 = 0; m1 < units_of && !keys.full(); m1 += wide) {
      const uint32_t m = m1 + lane_m, u = m / kGroupLanes * kWave + m % kGroupLanes;
      u32x4 group[kBatch], raw[kBatch];
      uint32_t word[kWords], index[kBatch];
      bool in[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) group[k] = st.groups[min(g0 + k * per + lane_g, count - 1)];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        in[k] = g0 + k * per + lane_g < count && m < units_of && u < group[k][2];
        index[k] = group[k][3] + u * E;
        const uint64_t at = (((uint64_t)group[k][1] << 32) | group[k][0]) + (uint64_t)u * 16;
        raw[k] = *as_global((const u32x4*)(uintptr_t)(in[k] ? at : other));
      }
#pragma unroll
      for (int w = 0; w < kWords; ++w) word[w] = in[w / 4] ? raw[w / 4][w % 4] : masked_unit<DT>().v[0][w % 4];
      uint64_t hits = 0;  // bit b: element b of the lane's
#pragma unroll
      for (int w = kWords - 1; w >= 0; --w) {
        if constexpr (DT == kBF16) {
          hits = hits + hits + (__uint_as_float(word[w] & 0xffff0000u) >= bar);
          hits = hits + hits + (__uint_as_float(word[w] << 16) >= bar);
        } else {
          hits = hits + hits + (__uint_as_float(word[w]) >= bar);
        }
      }
      for (; __any(hits != 0); hits &= hits - 1) {
        const uint32_t b = (uint32_t)__builtin_ctzll(hits | 1ull << 63), w = b / (E / 4);
        uint32_t x = word[0], first = index[0];
#pragma unroll
        for (int i = 1; i < kWords; ++i) x = w == (uint32_t)i ? word[i] : x;
#pragma unroll
        for (int k = 1; k < kBatch; ++k) first = b / E == (uint32_t)k ? index[k] : first;
        if constexpr (DT == kBF16) x = b % 2 ? x & 0xffff0000u : x << 16;
        keys.push(key_of(__uint_as_float(x), first + b % E), hits != 0);
      }
    }
  // the elements before and after the pieces' units
  if (__any(place[1] >> 24)) {
    for (int i = 0; i < a.pieces * 16; i += kWave) {
      const uint32_t piece = (uint32_t)(i + lane) / 16, l = (uint32_t)lane % 16;
      const Place pl(lane_place(place, (int)(piece % kWave)));
      const bool before = l < pl.head, after = l >= 8 && l - 8 < pl.tail;
      const int64_t off = before ? (int64_t)l - pl.head : (int64_t)pl.n * E + l - 8;
      float f = -__builtin_inff();
      if ((before || after) && piece < (uint32_t)a.pieces) f = widen1<DT>(reinterpret_cast<const S*>(pl.units)[off]);
      keys.push(key_of(f, pl.index + (uint32_t)off), f >= bar);
    }
  }
  unsigned long long mine = 0;
  if (!groups.full() && !keys.full()) {
    const uint32_t n = keys.n;
    if (lane < a.top) st.sorted[lane] = 0;
    wave_fence();
    for (uint32_t i = lane; i < n; i += kWave) {
      const unsigned long long k = st.keys[i];
      uint32_t rank = 0;
#pragma unroll 8
      for (uint32_t j = 0; j < n; ++j) rank += st.keys[j] > k;
      if (rank < (uint32_t)a.top) st.sorted[rank] = k;
    }
    wave_fence();
    if (lane < a.top) mine = st.sorted[lane];
    wave_fence();
  } else {
    // more ties with the bar, or more of the best in few lanes, than there
    // is room for, or no bar in too few groups: the whole row again, by
    // insertion
    TopList list;
    for (int i = 0; i < a.pieces; ++i) {
      u32x4 at;
#pragma unroll
      for (int d = 0; d < 4; ++d) at[d] = (uint32_t)__builtin_amdgcn_readlane((int)place[d], i);
      const Place pl(at);
      const bool before = (uint32_t)lane < pl.head, after = lane >= 8 && (uint32_t)lane - 8 < pl.tail;
      const int64_t off = before ? (int64_t)lane - pl.head : (int64_t)pl.n * E + lane - 8;
      list.offer(before || after ? key_of(widen1<DT>(reinterpret_cast<const S*>(pl.units)[off]), pl.index + (uint32_t)off) : 0, a.top);
      for (uint32_t u0 = 0; u0 < pl.n; u0 += kBatch * kWave) {
        RawUnit<DT, E> raw[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const uint32_t u = u0 + k * kWave + lane;
          raw[k] = u < pl.n ? load_unit<DT, E, false>(pl.units, (uint64_t)u * E) : masked_unit<DT>();
        }
#pragma unroll 1
        for (int k = 0; k < kBatch; ++k) {
          float f[E];
          widen_unit(raw[0], f);
#pragma unroll
          for (int j = 0; j + 1 < kBatch; ++j) raw[j] = raw[j + 1];
          const float top = largest(f);
          const uint32_t u = u0 + k * kWave + lane;
          if (__any(order_of(top) >= (uint32_t)(list.bar >> 32))) list.consider(f, top, pl.index + u * E, u < pl.n, a.top);
        }
      }
    }
    mine = list.key;
  }
  return lane < a.top ? mine : 0;
}

template <int DT, bool TOP>
__global__ __launch_bounds__(kBlock) void logprob_join_kernel(JoinInput a, LogprobJoinArgs j) {
  __shared__ JoinStore store[TOP ? kBlock / kWave : 1];
  const int lane = (int)(threadIdx.x % kWave), pieces = a.pieces;
  const float c = a.scale * kLog2e, inf = __builtin_inff(), nan = __uint_as_float(0x7fc00000u);
  const uint32_t in = blockIdx.x * (kBlock / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint64_t row = a.first_row + in;
  if (in < a.rows) {
    Running run;
    float z = -inf, bests[kLoads];
    if constexpr (TOP) load_bests(a, row, lane, bests);
    u32x4 place = {0, 0, 0, 0};
    if (lane < pieces) {
      const u32x4 rec = reinterpret_cast<const u32x4*>(as_global(a.part))[row * (uint64_t)pieces + lane];
      run.m = __uint_as_float(rec[0]);
      run.s = __uint_as_float(rec[1]);
      run.a = __uint_as_float(rec[2]);
      z = __uint_as_float(rec[3]);
      if constexpr (TOP) place = reinterpret_cast<const u32x4*>(as_global(a.places))[row * (uint64_t)pieces + lane];
    }
    z = wave_max(z);
    const int64_t target = as_global(a.targets)[row];
    const bool counts = target >= 0 && target < a.vocab;
    run.wave_join(c);
    const bool poison = !(run.s >= 0.0f), empty = run.s == 0.0f;
    const float m = poison ? nan : empty ? -inf : run.m;
    const float log_s = poison ? nan : empty ? -inf : logf(run.s);
    if (lane < a.p) {
      float* st = as_global(j.stats[lane]) + row * 2;
      st[0] = m;
      st[1] = log_s;
      as_global(j.logp[lane])[row] = !counts ? 0.0f : empty ? -inf : (z - m) * a.scale - log_s;
      if (j.entropy[lane]) as_global(j.entropy[lane])[row] = empty ? 0.0f : log_s - run.a * kLn2 / run.s;
    }
    if constexpr (TOP) {
      const unsigned long long best = poison || empty ? 0 : row_best<DT>(a, row, place, bests, lane, store[threadIdx.x / kWave]);
      const int have = __popcll(__ballot(best != 0));
      float lp = poison ? nan : best ? (value_of((uint32_t)(best >> 32)) - m) * a.scale - log_s : -inf;
      int32_t idx = poison || !best ? -1 : (int32_t)~(uint32_t)best;
      if (have < a.top && !poison) {
        // fewer unmasked entries than asked for: then the masked ones, lowest
        // index first (at most 31 of the first 64 are listed)
        bool free = lane < a.vocab;
        for (int k = 0; k < have; ++k) free = free && __builtin_amdgcn_readlane(idx, k) != lane;
        unsigned long long left = __ballot(free);
        for (int k = have; k < a.top && left; ++k, left &= left - 1)
          if (lane == k) idx = __builtin_ctzll(left);
      }
      if (lane < a.top)
  #pragma unroll 4
        for (int r = 0; r < a.p; ++r) {
          as_global(j.top_logp[r])[row * (uint64_t)a.top + lane] = lp;
          as_global(j.top_idx[r])[row * (uint64_t)a.top + lane] = idx;
        }
    }
  }
}

// Gradient.  A wave takes two 16-byte units a lane of one row's shard, 2 KiB
// cut as the forward pass's pieces.  The card then works in a narrow window of
// memory: four units of bf16 took 181 us instead of 171 for 4096 x 65536, and
// four and eight of fp32 179 and 181 instead of 173 for 4096 x 32000.
constexpr int kGradUnits = 2;

// A row's gradient.  With d = log2 p_j, dz = 2^d (A + B d), but for the
// target's own term.
struct GradRow {
  float c, m, shift, a, b;

  // d = (z - m) c - shift as written
  __device__ __forceinline__ float far(float z) const {
    const float d = (z - m) * c - shift;
    return __builtin_amdgcn_exp2f(d) * __builtin_fmaf(fmaxf(d, kFar), b, a);
  }
  // d as one fma, z c - K for the rounded K = m c + shift.  It is off by
  // the exactly known eps, which went into a and b.
  __device__ __forceinline__ float near(float z) const {
    const float d = __builtin_fmaf(z, c, -shift);
    return __builtin_amdgcn_exp2f(d) * __builtin_fmaf(fmaxf(d, kFar), b, a);
  }
  __device__ __forceinline__ bool make_near() {
#pragma clang fp contract(off)
    if (!(fabsf(m) < kPlainMax && c < kPlainScale)) return false;
    const float mc = m * c, k = mc + shift, back = k - mc;  // rounded each
    const float eps = __builtin_fmaf(m, c, -mc) + ((mc - (k - back)) + (shift - back));  // m c + shift - K
    const float f = __builtin_amdgcn_exp2f(-eps);
    a = (a - eps * b) * f;
    b *= f;
    shift = k;
    return true;
  }
};

template <int DT>
__global__ __launch_bounds__(kBlock) void logprob_grad_kernel(LogprobGradArgs a, LogprobPlan plan) {
  constexpr int B = Traits<DT>::B, E = kElems<DT>;
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

  const int64_t target = ld_const(a.targets + row);
  const bool counts = target >= 0 && target < a.first_index[a.p];
  GradRow g;
  g.c = a.scale * kLog2e;
  g.m = ld_const(a.stats + 2 * row);
  g.shift = ld_const(a.stats + 2 * row + 1) * kLog2e;
  float gl = ld_const(a.dlogp + row), gh = 0.0f, h = 0.0f;
  if (a.dentropy) {
    gh = ld_const(a.dentropy + row);
    h = ld_const(a.entropy + row);
  }
  if (!counts) gl = 0.0f;
  if (g.m == -__builtin_inff()) g.m = g.shift = gl = gh = h = 0.0f;  // nothing was allowed: no gradient
  g.a = -(gl + gh * h) * a.scale;
  g.b = -gh * kLn2 * a.scale;
  const float own = gl * a.scale;
  const bool near = g.make_near();
  // the target's place from the first unit's first element, if it is here
  const int64_t t_off = counts ? target - a.first_index[r] - pc.begin - pc.head : -1;
  const uint32_t t_unit = t_off >= 0 && t_off < (int64_t)pc.units * E ? (uint32_t)t_off / E : ~0u;
  auto finish = [&](int i, float (&f)[E]) {
    if (i * kWave + lane == t_unit) {
#pragma unroll
      for (uint32_t e = 0; e < E; ++e)
        if (e == (uint32_t)t_off % E) f[e] += own;
    }
    store_unit<DT, E, true>(outs, (i * kWave + lane) * E, narrow_unit<DT, E>(f));
  };
  if (near) {
#pragma unroll
    for (int i = 0; i < kGradUnits; ++i) {
      float f[E];
      widen_unit(x[i], f);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = g.near(f[e]);
      finish(i, f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kGradUnits; ++i) {
      float f[E];
      widen_unit(x[i], f);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = g.far(f[e]);
      finish(i, f);
    }
  }
  // the elements before and after the units
  if (pc.head + pc.tail) {
    int64_t off = -1;  // from the shard's row's start
    if (lane < pc.head) off = pc.begin + lane;
    else if (lane >= 8 && lane - 8 < pc.tail) off = pc.begin + pc.head + (int64_t)pc.units * E + lane - 8;
    if (off >= 0) {
      const float z = widen1<DT>(reinterpret_cast<const S*>(base)[off]);
      float v = near ? g.near(z) : g.far(z);
      if (counts && target - a.first_index[r] == off) v += own;
      reinterpret_cast<S*>(out)[off] = narrow1<DT>(v);
    }
  }
}

}  // namespace

// Pieces of a wave's step or more: as many as wanted, and none over 32768
// elements, as far as a row's 64 pieces allow.
void logprob_plan(int p, uint64_t rows, const int64_t* vocab, LogprobPlan* plan) {
  const int64_t unit = kLogprobStep, most = kMaxPieces / p, most_before = kLine / 2 - 1, want = (int64_t)logprob_want(p, rows);
  plan->first[0] = 0;
  for (int r = 0; r < p; ++r) {
    const int64_t v = vocab[r] + most_before;
    int64_t s = std::min<int64_t>(most, std::max<int64_t>(want, (v + 32767) / 32768));
    s = std::max<int64_t>(1, std::min<int64_t>(s, (v + unit - 1) / unit));
    const int64_t len = ((v + s - 1) / s + 511) / 512 * 512;
    plan->len[r] = len;
    plan->first[r + 1] = plan->first[r] + pieces_of(vocab[r], most_before, len);
  }
  finish_plan(plan, p);
  // as many groups as there may be, of whole steps
  int64_t steps = 1;
  for (int r = 0; r < p; ++r) steps = std::max(steps, (std::min(plan->len[r], vocab[r]) + unit - 1) / unit);
  const int64_t segs = std::min<int64_t>(steps, kMaxGroups / kSegGroups / std::max(plan->pieces, 1));
  plan->seg_steps = (int)((steps + segs - 1) / segs);
  plan->segs = (int)((steps + plan->seg_steps - 1) / plan->seg_steps);
}

int launch_logprob(int dtype, const LogprobArgs& args, const LogprobJoinArgs& j, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  LogprobArgs a = args;
  const dim3 block(kBlock);
  const int e = over_rows(args.rows, (uint64_t)a.plan.pieces, [&](uint64_t first, uint64_t rows, dim3 grid) {
    a.first_row = first;
    a.rows = rows;
    if (dtype == kF32) {
      if (a.top) hipLaunchKernelGGL((logprob_pieces_kernel<kF32, true>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((logprob_pieces_kernel<kF32, false>), grid, block, 0, s, a);
    } else {
      if (a.top) hipLaunchKernelGGL((logprob_pieces_kernel<kBF16, true>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((logprob_pieces_kernel<kBF16, false>), grid, block, 0, s, a);
    }
  });
  if (e) return e;
  JoinInput in{a.part, a.places, a.bests, a.targets, 0, 0, a.first_index[a.p], a.scale, a.p, a.top, a.plan.pieces,
               a.plan.segs, a.plan.seg_steps};
  return over_rows(args.rows, 1, [&](uint64_t first, uint64_t rows, dim3 grid) {
    in.first_row = first;
    in.rows = rows;
    if (!a.top) hipLaunchKernelGGL((logprob_join_kernel<kF32, false>), grid, block, 0, s, in, j);
    else if (dtype == kF32) hipLaunchKernelGGL((logprob_join_kernel<kF32, true>), grid, block, 0, s, in, j);
    else hipLaunchKernelGGL((logprob_join_kernel<kBF16, true>), grid, block, 0, s, in, j);
  });
}

int launch_logprob_backward(int dtype, const LogprobGradArgs& args, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  LogprobGradArgs a = args;
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
    if (dtype == kF32) hipLaunchKernelGGL((logprob_grad_kernel<kF32>), grid, dim3(kBlock), 0, s, a, plan);
    else hipLaunchKernelGGL((logprob_grad_kernel<kBF16>), grid, dim3(kBlock), 0, s, a, plan);
  });
}

}  // namespace coll
