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
// the AllReduce of maxima and sums over the ranks would, and stores the
// results to every rank.
//
// Sums run in base 2 (v_exp_f32), in fp32.  Differences to the maximum are
// taken before the scaling, so large logits lose nothing, and are held at
// -16384 or more where they multiply a sum, so that no 0 * inf arises.  The
// running maximum starts at the lowest finite value: a masked entry
// (-infinity) then always contributes zero, and a row with nothing else
// has S = 0.  A NaN or +infinity makes S a NaN.
//
// Gradient: 4 bytes an element in bf16, read once and written once.
#include <float.h>

#include <algorithm>

#include "token_unit.h"

namespace coll {

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
constexpr float kFar = -16384.0f;
constexpr int kStep = 32;                          // elements per lane and step
constexpr int64_t kWaveStep = (int64_t)kStep * kWave;

// The order of fp32 values as unsigned integers (both zeros alike).
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// The `top` largest of a wave's elements, one per lane in descending order:
// key = order of the value above the complement of the index, so that the
// lower index wins a tie.  An empty place is 0, below every key.  bar: no key
// at or below it can enter.
struct TopList {
  unsigned long long key = 0, bar = 0;

  // A starting bar that at least `top` of the lanes' largest elements pass:
  // the largest order with that many lanes at or above it, found bit by bit.
  __device__ __forceinline__ void raise(uint32_t lane_best, int top) {
    uint32_t t = 0;
    for (int b = 31; b >= 0; --b) {
      const uint32_t c = t | (1u << b);
      const int n = __popcll(__ballot(lane_best >= c));
      if (n >= top) {
        t = c;
        if (n == top) break;
      }
    }
    if (t) bar = ((unsigned long long)t << 32) - 1;
  }

  __device__ __forceinline__ void insert(unsigned long long k, int top) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(-1, (int)(uint32_t)key, 0x138 /* wave_shr:1 */, 0xf, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(-1, (int)(uint32_t)(key >> 32), 0x138, 0xf, 0xf, false);
    const unsigned long long before = ((unsigned long long)hi << 32) | lo;
    key = key > k ? key : before > k ? k : before;
    const unsigned long long last = lane_value(key, top - 1);
    if (last > bar) bar = last;
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

__device__ __forceinline__ unsigned long long key_of(float v, uint32_t index) {
  return ((unsigned long long)order_of(v) << 32) | (uint32_t)~index;
}

// A piece of a row's shard: its elements before the first 16-byte boundary,
// its whole units and the rest.  Pieces after the first start on such a
// boundary, so only a shard's two ends go element by element.
struct Piece {
  int64_t begin;       // first element
  uint32_t head, tail; // elements
  uint32_t units;      // of 16 bytes
};
template <int DT>
__device__ __forceinline__ Piece piece_of(const uint8_t* row, int64_t vocab, int64_t len, int k) {
  constexpr int B = Traits<DT>::B, E = kElems<DT>;
  const int64_t mis = (int64_t)((uintptr_t)row & 15) / B;
  Piece c;
  c.begin = k ? (int64_t)k * len - mis : 0;
  int64_t end = (int64_t)(k + 1) * len - mis;
  if (c.begin > vocab) c.begin = vocab;
  if (end > vocab) end = vocab;
  const uint32_t n = (uint32_t)(end - c.begin);
  const uint32_t h = (uint32_t)(((16 - (((uintptr_t)row + c.begin * B) & 15)) & 15) / B);
  c.head = h < n ? h : n;
  c.units = (n - c.head) / E;
  c.tail = n - c.head - c.units * E;
  return c;
}

template <int DT>
__device__ __forceinline__ RawUnit<DT, kElems<DT>> masked_unit() {
  const uint32_t w = DT == kBF16 ? 0xff80ff80u : 0xff800000u;
  return RawUnit<DT, kElems<DT>>{{u32x4{w, w, w, w}}};
}

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
    s = wave_sum(s);
    a = wave_sum(a);
  }
};

template <int DT, bool TOP>
__global__ __launch_bounds__(kBlock) void logprob_pieces_kernel(LogprobArgs a) {
  constexpr int B = Traits<DT>::B, E = kElems<DT>, kChunk = kStep / E;
  constexpr uint32_t kChunkUnits = kChunk * kWave;
  const uint32_t lane = threadIdx.x % kWave;
  const float c = a.scale * kLog2e;
  const uint64_t items = a.rows * (uint64_t)a.plan.pieces, step = (uint64_t)gridDim.x * (kBlock / kWave);
  uint64_t item = (uint64_t)blockIdx.x * (kBlock / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  for (; item < items; item += step) {
    const uint64_t row = item / (uint64_t)a.plan.pieces;
    const int piece = (int)(item - row * (uint64_t)a.plan.pieces);
    int r = 0;
    while (a.plan.first[r + 1] <= piece) ++r;
    const int64_t vocab = a.first_index[r + 1] - a.first_index[r];
    const uint8_t* base = as_global(static_cast<const uint8_t*>(a.logits[r])) + (int64_t)row * a.ld[r] * B;
    const Piece pc = piece_of<DT>(base, vocab, a.plan.len[r], piece - a.plan.first[r]);
    const uint8_t* units = base + (pc.begin + pc.head) * B;
    const uint32_t index0 = (uint32_t)(a.first_index[r] + pc.begin);  // vocabulary index of the piece's first element

    Running run;
    TopList list;
    RawUnit<DT, E> cur[kChunk], nxt[kChunk];
    auto load = [&](RawUnit<DT, E> (&to)[kChunk], uint32_t u0) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        const uint32_t u = u0 + i * kWave + lane;
        to[i] = u < pc.units ? load_unit<DT, E, true>(units, u * E) : masked_unit<DT>();
      }
    };
    if (pc.units) load(cur, 0);
    // the elements of both ends, one per lane: head on lanes 0..7, tail on 8..15
    float end = -__builtin_inff();
    uint32_t end_off = ~0u;
    if (lane < pc.head) end_off = lane;
    else if (lane >= 8 && lane - 8 < pc.tail) end_off = pc.head + pc.units * E + lane - 8;
    using S = typename Traits<DT>::S;
    if (end_off != ~0u) end = widen1<DT>(reinterpret_cast<const S*>(base)[pc.begin + end_off]);
    // the target's logit, where it lies in this piece
    const int64_t t_off = as_global(a.targets)[row] - a.first_index[r] - pc.begin;
    float z = -__builtin_inff();
    if (t_off >= 0 && t_off < (int64_t)(pc.head + pc.units * E + pc.tail))
      z = widen1<DT>(reinterpret_cast<const S*>(base)[pc.begin + t_off]);
    for (uint32_t u0 = 0; u0 < pc.units; u0 += kChunkUnits) {
      const bool more = u0 + kChunkUnits < pc.units;
      if (more) load(nxt, u0 + kChunkUnits);
      float f[kChunk][E], um[kChunk], top = -FLT_MAX;
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        widen_unit(cur[i], f[i]);
        um[i] = f[i][0];
#pragma unroll
        for (int e = 1; e < E; ++e) um[i] = fmaxf(um[i], f[i][e]);
        top = fmaxf(top, um[i]);
      }
      run.rebase(fmaxf(run.m, top), c);
      float s[kChunk] = {}, w[kChunk] = {};
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float d = (f[i][e] - run.m) * c, x = __builtin_amdgcn_exp2f(d);
          s[i] += x;
          w[i] += x * fmaxf(d, kFar);
        }
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        run.s += s[i];
        run.a += w[i];
      }
      if constexpr (TOP) {
        if (u0 == 0) {
          float best = um[0];
#pragma unroll
          for (int i = 1; i < kChunk; ++i) best = fmaxf(best, um[i]);
          list.raise(order_of(best), a.top);
        }
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          // later units hold higher indices, so a tie with the bar loses
          if (!__any(order_of(um[i]) > (uint32_t)(list.bar >> 32))) continue;
          const uint32_t u = u0 + i * kWave + lane;
#pragma unroll
          for (int e = 0; e < E; ++e)
            list.offer(u < pc.units ? key_of(f[i][e], index0 + pc.head + u * E + e) : 0, a.top);
        }
      }
      if (more) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) cur[i] = nxt[i];
      }
    }
    if (pc.head + pc.tail) {
      run.rebase(fmaxf(run.m, end), c);
      const float d = (end - run.m) * c, x = __builtin_amdgcn_exp2f(d);
      run.s += x;
      run.a += x * fmaxf(d, kFar);
      if constexpr (TOP) list.offer(end_off != ~0u ? key_of(end, index0 + end_off) : 0, a.top);
    }
    run.wave_join(c);
    if (lane == 0) {
      const u32x4 rec = {__float_as_uint(run.m), __float_as_uint(run.s), __float_as_uint(run.a), __float_as_uint(z)};
      reinterpret_cast<u32x4*>(as_global(a.part))[item] = rec;
    }
    if constexpr (TOP)
      if ((int)lane < a.top) as_global(a.keys)[item * (uint64_t)a.top + lane] = list.key;
  }
}

// The largest of the lanes' keys, on every lane: by the upper words, and by
// the lower ones only where these tie.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off));
  return v;
}
__device__ __forceinline__ unsigned long long wave_max_key(unsigned long long k) {
  const uint32_t hi = (uint32_t)(k >> 32), top = wave_max_u32(hi);
  const unsigned long long tie = __ballot(hi == top);
  if ((tie & (tie - 1)) == 0) return TopList::lane_value(k, __builtin_ctzll(tie));
  return ((unsigned long long)top << 32) | wave_max_u32(hi == top ? (uint32_t)k : 0u);
}

// What the join needs beside its output pointers.
struct JoinInput {
  const float* part;
  const unsigned long long* keys;
  const int64_t* targets;
  uint64_t rows;
  int64_t vocab;
  float scale;
  int p, top, pieces;
};

__global__ __launch_bounds__(kBlock) void logprob_join_kernel(JoinInput a, LogprobJoinArgs j) {
  const int lane = (int)(threadIdx.x % kWave), pieces = a.pieces;
  const float c = a.scale * kLog2e, inf = __builtin_inff(), nan = __uint_as_float(0x7fc00000u);
  const uint64_t step = (uint64_t)gridDim.x * (kBlock / kWave);
  uint64_t row = (uint64_t)blockIdx.x * (kBlock / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  for (; row < a.rows; row += step) {
    Running run;
    float z = -inf;
    if (lane < pieces) {
      const u32x4 rec = reinterpret_cast<const u32x4*>(as_global(a.part))[row * (uint64_t)pieces + lane];
      run.m = __uint_as_float(rec[0]);
      run.s = __uint_as_float(rec[1]);
      run.a = __uint_as_float(rec[2]);
      z = __uint_as_float(rec[3]);
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
    if (a.top == 0) continue;
    // merge the pieces' descending lists: a lane holds its list's next two
    const unsigned long long* list = as_global(a.keys) + (row * (uint64_t)pieces + lane) * a.top;
    unsigned long long head = lane < pieces ? list[0] : 0, next = lane < pieces && a.top > 1 ? list[1] : 0, best = 0;
    int at = 2;
    for (int k = 0; k < a.top; ++k) {
      const unsigned long long w = wave_max_key(head);
      if (lane == k) best = w;
      if (head == w && w) {
        head = next;
        next = at < a.top ? list[at] : 0;
        ++at;
      }
    }
    const bool have = best != 0 && !poison;
    const float v = value_of((uint32_t)(best >> 32));
    const float lp = poison ? nan : !have || empty ? -inf : (v - m) * a.scale - log_s;
    const int32_t idx = have ? (int32_t)~(uint32_t)best : -1;
    if (lane < a.top)
      for (int r = 0; r < a.p; ++r) {
        as_global(j.top_logp[r])[row * (uint64_t)a.top + lane] = lp;
        as_global(j.top_idx[r])[row * (uint64_t)a.top + lane] = idx;
      }
  }
}

// Gradient.  A wave takes kGradLen elements of one row's shard, cut as the
// forward pass's pieces.
constexpr int64_t kGradLen = kWaveStep;

struct GradRow {
  float m, shift, gl, gh, h, scale, c;

  // dz of an element, without the target's own term
  __device__ __forceinline__ float operator()(float z) const {
    const float d = (z - m) * c - shift;  // log2 of the probability
    const float p = __builtin_amdgcn_exp2f(d);
    return -p * (gl + gh * (fmaxf(d, kFar) * kLn2 + h)) * scale;
  }
};

template <int DT>
__global__ __launch_bounds__(kBlock) void logprob_grad_kernel(LogprobGradArgs a, LogprobPlan plan) {
  constexpr int B = Traits<DT>::B, E = kElems<DT>, kChunk = kStep / E;
  const uint32_t lane = threadIdx.x % kWave;
  const uint64_t items = a.rows * (uint64_t)plan.pieces, step = (uint64_t)gridDim.x * (kBlock / kWave);
  uint64_t item = (uint64_t)blockIdx.x * (kBlock / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  for (; item < items; item += step) {
    const uint64_t row = item / (uint64_t)plan.pieces;
    const int piece = (int)(item - row * (uint64_t)plan.pieces);
    int r = 0;
    while (plan.first[r + 1] <= piece) ++r;
    const int64_t vocab = a.first_index[r + 1] - a.first_index[r];
    const uint8_t* base = as_global(static_cast<const uint8_t*>(a.logits[r])) + (int64_t)row * a.ld[r] * B;
    uint8_t* out = as_global(static_cast<uint8_t*>(a.dlogits[r])) + (int64_t)row * a.dld[r] * B;
    const Piece pc = piece_of<DT>(base, vocab, kGradLen, piece - plan.first[r]);
    const uint8_t* units = base + (pc.begin + pc.head) * B;
    uint8_t* outs = out + (pc.begin + pc.head) * B;
    RawUnit<DT, E> x[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const uint32_t u = i * kWave + lane;
      x[i] = u < pc.units ? load_unit<DT, E, true>(units, u * E) : masked_unit<DT>();
    }
    uint32_t end_off = ~0u;
    if (lane < pc.head) end_off = lane;
    else if (lane >= 8 && lane - 8 < pc.tail) end_off = pc.head + pc.units * E + lane - 8;
    float end = 0.0f;
    if (end_off != ~0u)
      end = widen1<DT>(reinterpret_cast<const typename Traits<DT>::S*>(base)[pc.begin + end_off]);

    const int64_t target = as_global(a.targets)[row];
    const bool counts = target >= 0 && target < a.first_index[a.p];
    GradRow g;
    g.m = as_global(a.stats)[2 * row];
    const float log_s = as_global(a.stats)[2 * row + 1];
    const bool empty = g.m == -__builtin_inff();
    g.c = a.scale * kLog2e;
    g.scale = a.scale;
    g.shift = log_s * kLog2e;
    g.gl = counts ? as_global(a.dlogp)[row] : 0.0f;
    g.gh = a.dentropy ? as_global(a.dentropy)[row] : 0.0f;
    g.h = a.dentropy ? as_global(a.entropy)[row] : 0.0f;
    if (empty) {  // nothing was allowed: no gradient
      g.m = 0.0f;
      g.shift = 0.0f;
      g.gl = 0.0f;
      g.gh = 0.0f;
      g.h = 0.0f;
    }
    const float own = g.gl * a.scale;
    // the target's place from the piece's first element, if it is here
    const int64_t t_off = counts ? target - a.first_index[r] - pc.begin : -1;
    const uint32_t n = pc.head + pc.units * E + pc.tail;
    const uint32_t t = t_off >= 0 && t_off < (int64_t)n ? (uint32_t)t_off : ~0u;
    const uint32_t t_unit = t == ~0u || t < pc.head ? ~0u : (t - pc.head) / E;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const uint32_t u = i * kWave + lane;
      if (u >= pc.units) continue;
      float f[E];
      widen_unit(x[i], f);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = g(f[e]);
      if (u == t_unit) {
        const uint32_t te = (t - pc.head) % E;
#pragma unroll
        for (uint32_t e = 0; e < E; ++e)
          if (e == te) f[e] += own;
      }
      store_unit<DT, E, true>(outs, u * E, narrow_unit<DT, E>(f));
    }
    if (end_off != ~0u) {
      float v = g(end);
      if (end_off == t) v += own;
      reinterpret_cast<typename Traits<DT>::S*>(out)[pc.begin + end_off] = narrow1<DT>(v);
    }
  }
}

uint32_t wave_grid(uint64_t waves) {
  const uint64_t g = (waves + kBlock / kWave - 1) / (kBlock / kWave);
  return (uint32_t)(g < 0x1000000 ? g : 0x1000000);
}

// Pieces of `len` elements that cover a shard whatever its rows' offset from
// a 16-byte boundary (at most 7 elements).
int pieces_of(int64_t vocab, int64_t len) { return vocab ? (int)((vocab + 7 + len - 1) / len) : 0; }

}  // namespace

// Pieces of a wave's step or more: enough for some 8192 waves
// over all rows, and none over 32768 elements, as far as a row's 64 pieces
// allow.
void logprob_plan(int p, uint64_t rows, const int64_t* vocab, LogprobPlan* plan) {
  const int64_t unit = kWaveStep, most = kMaxPieces / p;
  const uint64_t want = rows ? (8192 + rows * (uint64_t)p - 1) / (rows * (uint64_t)p) : 1;
  plan->first[0] = 0;
  for (int r = 0; r < p; ++r) {
    const int64_t v = vocab[r] + 7;
    int64_t s = std::min<int64_t>(most, std::max<int64_t>((int64_t)std::min<uint64_t>(want, 64), (v + 32767) / 32768));
    s = std::max<int64_t>(1, std::min<int64_t>(s, (v + unit - 1) / unit));
    const int64_t len = ((v + s - 1) / s + 511) / 512 * 512;
    plan->len[r] = len;
    plan->first[r + 1] = plan->first[r] + pieces_of(vocab[r], len);
  }
  plan->pieces = plan->first[p];
}

int launch_logprob(int dtype, const LogprobArgs& a, const LogprobJoinArgs& j, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  const dim3 grid(wave_grid(a.rows * (uint64_t)a.plan.pieces)), join(wave_grid(a.rows)), block(kBlock);
  if (dtype == kF32) {
    if (a.top) hipLaunchKernelGGL((logprob_pieces_kernel<kF32, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((logprob_pieces_kernel<kF32, false>), grid, block, 0, s, a);
  } else {
    if (a.top) hipLaunchKernelGGL((logprob_pieces_kernel<kBF16, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((logprob_pieces_kernel<kBF16, false>), grid, block, 0, s, a);
  }
  const int e = (int)hipGetLastError();
  if (e) return e;
  const JoinInput in{a.part, a.keys, a.targets, a.rows, a.first_index[a.p], a.scale, a.p, a.top, a.plan.pieces};
  hipLaunchKernelGGL(logprob_join_kernel, join, block, 0, s, in, j);
  return (int)hipGetLastError();
}

int launch_logprob_backward(int dtype, const LogprobGradArgs& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  LogprobPlan plan;
  plan.first[0] = 0;
  for (int r = 0; r < a.p; ++r) {
    plan.len[r] = kGradLen;
    plan.first[r + 1] = plan.first[r] + pieces_of(a.first_index[r + 1] - a.first_index[r], kGradLen);
  }
  plan.pieces = plan.first[a.p];
  const dim3 grid(wave_grid(a.rows * (uint64_t)plan.pieces)), block(kBlock);
  if (dtype == kF32) hipLaunchKernelGGL((logprob_grad_kernel<kF32>), grid, block, 0, s, a, plan);
  else hipLaunchKernelGGL((logprob_grad_kernel<kBF16>), grid, block, 0, s, a, plan);
  return (int)hipGetLastError();
}

}  // namespace coll
