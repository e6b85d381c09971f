// Penalties for repeated tokens, biases and masks on logits that lie in p
// shards.  Per row, with c_j how often token j is among the answer's tokens:
//   v = z > 0 ? z (1 / repetition) : z repetition   where the history has token j,
//   v -= c_j frequency + presence               where c_j > 0,
//   v += bias                                   where a bias lists entry j,
//   v = -inf                                    where the mask's bit j is 0
// in fp32, rounded once.
//
// Bound by reading and writing the logits.  A workgroup takes a run of a
// row's shard.  It asks for the run's logits, which stay in registers, and
// marks the row's history and biases in a table of the run's entries in LDS
// while they come.  Every workgroup of a row goes over the whole history and
// keeps what falls into its run: the longer the run the less often, and the
// fewer workgroups share a CU (of 2048 units two, in bf16 by their tables, in
// fp32 by their registers; of 1024 four in bf16, by their tables, and five in
// fp32).  A row's runs follow each other on one XCD, whose L2 then serves the
// history to all but the first.  Few units have a mark: a wave collects its own
// from its lanes and adjusts them at once, before the mask, which needs no
// arithmetic.
// 512 x 131072 bf16 in 8 shards, masks, 100 biases and histories of 4000 tokens
// on average (most shorter, some of 30000 and more): 70-75 us, and 80 with one
// of 50000; 67 with 4000 in every row, 62 without masks and biases, 47 with
// nothing to mark (5.7 TB/s): what marks cost is the instructions of going over
// the history and of the units to adjust (570 a wave, 330 without masks and
// biases), not waiting: asking for the next tokens while these are looked at
// changed nothing.  For the 75, 82 where a row's runs went to all XCDs and 85
// with every lane adjusting its own units.  4 rows of 131072, 400 tokens: 5.2
// us; 333 x 50257 fp32 in 4 shards, 1500 tokens: 32-33 us.
//
// Counts are whole numbers and a bias's first entry wins by its place in the
// list, so results do not depend on the order of the atomics.
#include "vocab_pieces.h"

namespace coll {

namespace {

// A table word of an entry: in its upper bits n - k for the first place k of
// its bias in the row's list of n (0: none), as many bits as n has, below them
// whether the prompt has it, then its count among the answer's tokens.  Rows
// whose two lists are too long for that (2047 biases and 2^20 tokens, 16383
// and 2^17) take two words an entry, and the run in two halves: 85 us for the
// 75 above with one such row (3740 biases, where they were 2047 at most).
struct Word {
  uint32_t shift, prompt;
  __device__ __forceinline__ explicit Word(uint32_t biases) : shift(min(31u, (uint32_t)__builtin_clz(biases | 1))), prompt(1u << (shift - 1)) {}
  __device__ __forceinline__ uint32_t count(uint32_t w) const { return w & (prompt - 1); }
  __device__ __forceinline__ uint32_t seen(uint32_t w) const { return w & (2 * prompt - 1); }
  __device__ __forceinline__ uint32_t bias(uint32_t w) const { return w >> shift; }
};
constexpr uint32_t kLongPrompt = 0x80000000u;

// A row's part of a list, as offsets within it that are in bounds whatever
// the row's offsets are.
struct Span {
  uint64_t begin;
  uint32_t n;
  __device__ __forceinline__ Span(const int64_t* offsets, uint64_t row, uint64_t most) : begin(0), n(0) {
    if (!offsets) return;
    const int64_t a = ld_const(offsets + row), b = ld_const(offsets + row + 1);
    const uint64_t lo = a < 0 ? 0 : min((uint64_t)a, most), hi = b < 0 ? 0 : min((uint64_t)b, most);
    begin = lo;
    n = hi > lo ? (uint32_t)(hi - lo) : 0;
  }
};

// Tokens that a lane asks for at a time.  Four, and 24 registers fewer, let one
// more workgroup of 1024 fp32 units share a CU (333 x 50256 in 4 shards, ~1500
// tokens: 34 us for 36).  In bf16 the tables of these leave room for four
// workgroups either way, and four tokens are fewer instructions where a round
// of them holds the history (512 x 65536 in 8 shards, 1000 tokens: 31.3 for
// 32.3; 4000: 39.6 for 38.4; 20000: 82 for 76).
template <int THREADS, int UNITS>
constexpr int kAhead = THREADS < 512 && UNITS > 1 ? 4 : 8;

template <int DT, int THREADS, int UNITS>
__global__ __launch_bounds__(THREADS) void adjust_kernel(AdjustArgs a) {
  constexpr int B = Traits<DT>::B, E = kElems<DT>;
  constexpr uint32_t kRun = UNITS * THREADS * E;
  constexpr int kTokensAhead = kAhead<THREADS, UNITS>;
  using S = typename Traits<DT>::S;
  __shared__ __attribute__((aligned(16))) uint32_t table[kRun];
  __shared__ u32x4 held[THREADS];           // a wave's units to adjust
  __shared__ uint16_t held_unit[THREADS];
  __shared__ float first_values[THREADS];   // of the biases, those of the list's first places
  const uint32_t lane = threadIdx.x, turn = blockIdx.x / (uint32_t)a.spread, group = turn / (uint32_t)a.chunks;
  const uint32_t chunk = turn - group * (uint32_t)a.chunks;
  const uint32_t in_row = group * (uint32_t)a.spread + (blockIdx.x - turn * (uint32_t)a.spread);
  if (in_row >= a.rows) return;
  const uint64_t row = a.first_row + in_row;
  int r = min((int)((2 * (uint64_t)chunk + 1) * a.ranks_q32 >> 33), a.p - 1);
  while (a.first[r] > (int)chunk) --r;
  while (a.first[r + 1] <= (int)chunk) ++r;
  const int64_t vocab = a.first_index[r + 1] - a.first_index[r], at = (int64_t)(chunk - (uint32_t)a.first[r]) * kRun;
  const uint32_t len = (uint32_t)min((int64_t)kRun, vocab - at), full = len / E, part = len % E;
  const int64_t first = a.first_index[r] + at;  // vocabulary index of the run's first entry
  const uint8_t* src = as_global(static_cast<const uint8_t*>(a.logits[r])) + ((int64_t)row * a.ld[r] + at) * B;
  uint8_t* dst = as_global(static_cast<uint8_t*>(a.out[r])) + ((int64_t)row * a.old[r] + at) * B;
  const Span hist(a.offsets, row, a.ntokens), bias(a.bias_offsets, row, a.nbias);
  const int64_t* tokens = as_global(a.tokens) + hist.begin;
  const int64_t* places = as_global(a.bias_idx) + bias.begin;
  const float* values = as_global(a.bias) + bias.begin;
  // A list of n places in the vocabulary, from place i0 on, a lane's in t.  The
  // first of both lists are asked for before the logits: loads return in
  // order, and these are needed first.
  auto ask = [&](auto& t, const int64_t* all, uint32_t n, uint32_t i0) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < (int)(sizeof(t) / 8); ++k)
      if (i0 + k * THREADS < n) t[k] = (uint64_t)all[min(i0 + k * THREADS + lane, n - 1)];
  };
  uint64_t t[kTokensAhead], p[1];
  float value = 0.0f;
  ask(p, places, bias.n, 0);
  if (bias.n) value = values[min(lane, bias.n - 1)];
  ask(t, tokens, hist.n, 0);
  const RowBuffer from(src, full * 16), to(dst, full * 16);
  RawUnit<DT, E> z[UNITS];
#pragma unroll
  for (int i = 0; i < UNITS; ++i) z[i] = load_unit<DT, E, true>(from, (i * THREADS + lane) * E);
  // the elements behind the last unit, one to a lane (the others load the
  // run's first, so that nothing waits here)
  const uint32_t end = lane < part ? full * E + lane : 0;
  S end_raw = reinterpret_cast<const S*>(src)[end];
  // The mask's bits of `n` entries from entry `entry` of the run on, as loaded.
  const uint64_t mask_last = (uint64_t)(a.first_index[a.p] - 1) / 32;
  const uint32_t* words = as_global(a.mask) + row * (uint64_t)a.mask_ld;
  auto mask_words = [&](uint32_t entry, uint32_t n, uint32_t (&w)[2]) __attribute__((always_inline)) {
    const uint64_t bit = (uint64_t)first + entry;
    // (past the vocabulary: its last word, whose bits are not looked at)
    w[0] = words[min(bit / 32, mask_last)];
    w[1] = words[min((bit + n - 1) / 32, mask_last)];
  };
  auto mask_bits = [&](uint32_t entry, const uint32_t (&w)[2]) {
    return (uint32_t)((((uint64_t)w[1] << 32) | w[0]) >> (((uint32_t)first + entry) % 32));
  };
  uint32_t mw[UNITS][2], end_mw[2] = {~0u, ~0u};
  if (a.mask) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) mask_words((i * THREADS + lane) * E, E, mw[i]);
    mask_words(end, 1, end_mw);
  } else {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) mw[i][0] = mw[i][1] = ~0u;
  }

  const int64_t prompt = a.prompt ? ld_const(a.prompt + row) : 0;
  const uint32_t answer = prompt < 0 ? 0 : (uint32_t)min(prompt, (int64_t)hist.n);  // where the answer starts
  const float repetition = a.repetition ? ld_const(a.repetition + row) : 1.0f, inverse = 1.0f / repetition;
  const float presence = a.presence ? ld_const(a.presence + row) : 0.0f;
  const float frequency = a.frequency ? ld_const(a.frequency + row) : 0.0f;

  const Word word(bias.n);
  auto penalize = [&](float v, bool seen, uint32_t count) {
    v *= !seen ? 1.0f : v > 0.0f ? inverse : repetition;
    return v - (count ? (float)count * frequency + presence : 0.0f);
  };
  auto value_at = [&](uint32_t i) { return i < THREADS ? first_values[i] : values[i]; };
  auto adjust = [&](float v, uint32_t w) {
    v = penalize(v, word.seen(w), word.count(w));
    if (const uint32_t k = word.bias(w)) v += value_at(bias.n - k);
    return v;
  };
  // a unit, by its entries' words
  auto adjust_unit = [&](const RawUnit<DT, E>& raw, uint32_t u) __attribute__((always_inline)) {
    uint32_t w[E], any = 0;
    float f[E];
    widen_unit(raw, f);
#pragma unroll
    for (int e = 0; e < E; ++e) any |= w[e] = table[u * E + e];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = penalize(f[e], word.seen(w[e]), word.count(w[e]));
    if (word.bias(any)) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (const uint32_t k = word.bias(w[e])) f[e] += value_at(bias.n - k);
    }
    return narrow_unit<DT, E>(f);
  };
  // Those of a list's places in this run (of `most` entries from vocabulary
  // index `begin` on): f(entry's place in the run, place in the list).
  auto look = [&](const auto& t, uint32_t n, uint32_t i0, int64_t begin, uint32_t most, auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < (int)(sizeof(t) / 8); ++k) {
      const uint32_t i = i0 + k * THREADS + lane;
      const uint64_t j = t[k] - (uint64_t)begin;
      if (i < n && j < most) f((uint32_t)j, i);
    }
  };
  // t: the history's first places, as asked for
  auto mark_tokens = [&](uint64_t (&t)[kTokensAhead], int64_t begin, uint32_t most, uint32_t prompt_bit) __attribute__((always_inline)) {
    for (uint32_t i0 = 0; i0 < hist.n;) {
      look(t, hist.n, i0, begin, most, [&](uint32_t j, uint32_t i) {
        if (i >= answer) atomicAdd(&table[j], 1u);
        else atomicOr(&table[j], prompt_bit);
      });
      i0 += kTokensAhead * THREADS;
      ask(t, tokens, hist.n, i0);
    }
  };
  auto store = [&]() __attribute__((always_inline)) {
    // the mask on the elements as they are: a -infinity where a bit is 0
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const uint32_t u = i * THREADS + lane, allow = mask_bits(u * E, mw[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        auto all_of = [&](int bit) { return (uint32_t)((int32_t)(allow << (31 - bit)) >> 31); };
        const uint32_t keep = DT == kF32 ? all_of(k) : (all_of(2 * k) & 0xffffu) | (all_of(2 * k + 1) & 0xffff0000u);
        z[i].v[0][k] = (z[i].v[0][k] & keep) | ((DT == kF32 ? 0xff800000u : 0xff80ff80u) & ~keep);
      }
      store_unit<DT, E, true>(to, u * E, z[i]);
    }
    if (lane < part) reinterpret_cast<S*>(dst)[end] = mask_bits(end, end_mw) & 1 ? end_raw : narrow1<DT>(-__builtin_inff());
  };

  if (!hist.n && !bias.n) {
    store();
  } else if (hist.n < word.prompt) {
    u32x4* cleared = reinterpret_cast<u32x4*>(table);  // as far as the run goes, at least
#pragma unroll
    for (int i = 0; i < (int)(kRun / 4 / THREADS); ++i)
      if ((uint32_t)i * THREADS * 4 < len) cleared[i * THREADS + lane] = u32x4{0, 0, 0, 0};
    __syncthreads();
    for (uint32_t i0 = 0; i0 < bias.n;) {
      look(p, bias.n, i0, first, len, [&](uint32_t j, uint32_t i) {
        // the first place's bits, whatever else the word holds
        const uint32_t bits = bias.n - i;
        for (uint32_t had = table[j]; word.bias(had) < bits;) {
          const uint32_t now = atomicCAS(&table[j], had, bits << word.shift | word.seen(had));
          if (now == had) break;
          had = now;
        }
      });
      i0 += THREADS;
      ask(p, places, bias.n, i0);
    }
    first_values[lane] = value;
    mark_tokens(t, first, len, word.prompt);
    __syncthreads();
    // Few units have an entry to adjust: a wave collects its own, and goes
    // over them at once.
    const uint32_t wave0 = lane / kWave * kWave;
    uint32_t place[UNITS], n = 0;
    bool hit[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      uint32_t any = 0;
      // (behind the run's end the table is not cleared)
      if (i * THREADS + lane < full) {
#pragma unroll
        for (int e = 0; e < E; ++e) any |= table[(i * THREADS + lane) * E + e];
      }
      hit[i] = any != 0;
      const unsigned long long m = __ballot(hit[i]);
      place[i] = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
      n += (uint32_t)__popcll(m);
    }
    if (n > kWave) {
#pragma unroll
      for (int i = 0; i < UNITS; ++i)
        if (hit[i]) z[i] = adjust_unit(z[i], i * THREADS + lane);
    } else if (n) {
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        if (hit[i]) {
          held[wave0 + place[i]] = z[i].v[0];
          held_unit[wave0 + place[i]] = (uint16_t)(i * THREADS + lane);
        }
      }
      wave_fence();
      if (lane - wave0 < n) {
        const RawUnit<DT, E> raw = {{held[lane]}};
        held[lane] = adjust_unit(raw, held_unit[lane]).v[0];
      }
      wave_fence();
#pragma unroll
      for (int i = 0; i < UNITS; ++i)
        if (hit[i]) z[i].v[0] = held[wave0 + place[i]];
    }
    if (lane < part) {
      if (const uint32_t w = table[end]) end_raw = narrow1<DT>(adjust(widen1<DT>(end_raw), w));
    }
    store();
  } else {
    // two words an entry: count and prompt, place of the bias; entry by entry
    // (going over so long a list takes longer)
    constexpr uint32_t kHalf = kRun / 2;
    uint32_t* where = table + kHalf;
    for (uint32_t begin = 0; begin < len; begin += kHalf) {
      for (uint32_t i = lane; i < kHalf; i += THREADS) {
        table[i] = 0;
        where[i] = ~0u;
      }
      __syncthreads();
      for (uint32_t i0 = 0; i0 < bias.n; i0 += THREADS) {
        ask(p, places, bias.n, i0);
        look(p, bias.n, i0, first + begin, kHalf, [&](uint32_t j, uint32_t i) { atomicMin(&where[j], i); });
      }
      ask(t, tokens, hist.n, 0);
      mark_tokens(t, first + begin, kHalf, kLongPrompt);
      __syncthreads();
      for (uint32_t i = begin + lane; i < min(begin + kHalf, len); i += THREADS) {
        const uint32_t w = table[i - begin], k = where[i - begin];
        float v = penalize(widen1<DT>(reinterpret_cast<const S*>(src)[i]), w, w & ~kLongPrompt);
        if (k != ~0u) v += values[k];
        uint32_t m[2] = {~0u, ~0u};
        if (a.mask) mask_words(i, 1, m);
        reinterpret_cast<S*>(dst)[i] = narrow1<DT>(mask_bits(i, m) & 1 ? v : -__builtin_inff());
      }
      __syncthreads();
    }
  }
}

// Workgroups go to the XCDs in turn: with enough rows the runs of one are kept
// on one XCD, whose L2 then serves the row's history to all but the first.
constexpr int kXcds = 8;
constexpr uint64_t kSpreadRows = 64;

template <int DT, int THREADS, int UNITS>
int adjust_t(AdjustArgs a, hipStream_t s) {
  constexpr int64_t kRun = (int64_t)UNITS * THREADS * kElems<DT>;
  a.first[0] = 0;
  for (int r = 0; r < a.p; ++r) a.first[r + 1] = a.first[r] + (int)((a.first_index[r + 1] - a.first_index[r] + kRun - 1) / kRun);
  a.chunks = a.first[a.p];
  a.ranks_q32 = ((uint64_t)a.p << 32) / (uint64_t)a.chunks;
  // (a row has 2^21 + 63 runs at most, so that a launch holds one)
  const uint64_t all = a.rows, rows = most_blocks(THREADS) / (uint64_t)a.chunks;
  a.spread = a.offsets && std::min(all, rows) >= kSpreadRows ? kXcds : 1;
  const uint64_t most = rows / (uint64_t)a.spread * (uint64_t)a.spread;
  for (a.first_row = 0; a.first_row < all; a.first_row += most) {
    a.rows = std::min(most, all - a.first_row);
    const uint64_t groups = (a.rows + a.spread - 1) / a.spread;
    hipLaunchKernelGGL((adjust_kernel<DT, THREADS, UNITS>), dim3((uint32_t)(groups * a.spread * a.chunks)), dim3(THREADS), 0, s, a);
    if (const int e = (int)hipGetLastError()) return e;
  }
  return 0;
}

// Runs: of one unit to a lane where few rows leave CUs without work; else of 1024
// units to 256 lanes, but where shards are shorter of 256 units to 128,
// since a workgroup's lanes without entries and its table keep others out.
// Long histories want the longest runs, which go over them the least often,
// and more lanes.  us with runs of 256 units (256 lanes, and 128), 512, 1024 and
// 2048 (512 lanes), bf16, masks and 16 biases, calls replayed from a graph, by
// shards and tokens (~: on average, most less, some ten times as many):
//   4 rows of 8 x 16384, 400 tokens           5.2   5.1   5.2   6.1   6.3
//   the same, 20000 tokens                   11.3  19.6   8.5  13.6  10.8
//   16 rows of 8 x 16384, ~4000              12.0  19.7   8.6  13.5  11.0
//   64 rows of 8 x 4096, ~400                 7.5   7.5   6.8   6.7   7.9
//   the same, ~20000                         57.5   115  34.0  61.8  35.3
//   480 rows of 8 x 526, none                12.4   9.1  27.4  17.5  32.9
//   266 rows of 16 x 412, ~5700              39.5  64.5  47.1  44.2  56.4
//   1024 rows of 5 x 3319, 1000              40.7  28.3  49.7  33.3  58.8
//   512 rows of 8 x 8192, 1000               58.2  34.9  72.7  31.2  48.6
//   512 rows of 8 x 16384, none              82.3  49.4   104  49.7  54.0
//   the same, 4000                            141   108   147  71.7  67.0
//   the same, 20000                           358   329   283   149   110
//   the same, ~4000                           178   158   175  93.8  80.2
//   512 rows of 8 x 18992, ~4000              208   171   206   111   132
// The rule's choice is the least of a line or within a seventh of it, but where
// shards are somewhat longer than a run (3319 and 18992 entries: 33.3 and 132).
// The histories' lengths are on the device: the rule looks at the size of the
// list that holds them.
constexpr uint64_t kFewRuns = 512, kManyRuns = 1024, kLongHistory = 2000;

template <int DT>
int adjust_d(const AdjustArgs& a, hipStream_t s) {
  constexpr int E = kElems<DT>;
  int64_t runs = 0, longest = 0;
  for (int r = 0; r < a.p; ++r) {
    const int64_t n = a.first_index[r + 1] - a.first_index[r];
    runs += (n + 1024 * E - 1) / (1024 * E);
    longest = std::max(longest, n);
  }
  auto fewer = [&](uint64_t than) { return a.rows < (than + (uint64_t)runs - 1) / (uint64_t)runs; };
  const bool history = a.ntokens / a.rows >= kLongHistory;
  if (fewer(kFewRuns)) return history ? adjust_t<DT, 512, 1>(a, s) : adjust_t<DT, 256, 1>(a, s);
  if (history && (longest > 1024 * E || fewer(kManyRuns))) return adjust_t<DT, 512, 4>(a, s);
  if (!history && longest <= 256 * E) return adjust_t<DT, 128, 2>(a, s);
  return adjust_t<DT, 256, 4>(a, s);
}

}  // namespace

int launch_adjust(int dtype, const AdjustArgs& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  return dtype == kF32 ? adjust_d<kF32>(a, s) : adjust_d<kBF16>(a, s);
}

}  // namespace coll
