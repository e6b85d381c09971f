// Penalties for repeated tokens, biases and masks on logits that lie in p
// shards.  Per row, with c_j how often token j is among the answer's tokens:
//   v = z > 0 ? z / repetition : z repetition   where the history has token j,
//   v -= c_j frequency + presence               where c_j > 0,
//   v += bias                                   where a bias lists entry j,
//   v = -inf                                    where the mask's bit j is 0
// in fp32, rounded once.
//
// Bound by reading and writing the logits.  A workgroup takes a run of a
// row's shard.  It asks for the run's logits, counts the row's history in a
// table of its entries in LDS while they come (every workgroup of a row goes
// over the whole history, which comes from L2, and keeps what falls into its
// run), and then goes once over the run.  Counts are whole numbers and a
// bias's first entry wins by its place in the list, so results do not depend
// on the order of the atomics.
#include "vocab_pieces.h"

namespace coll {

namespace {

// A table word of an entry: its count among the answer's tokens (bits 0..14),
// whether the prompt has it (bit 15), and kBiasPlaces less the place of its
// bias in the row's list (bits 16..31; 0: none).  Longer histories and lists
// take two words an entry, and the run in two halves.
constexpr uint32_t kPrompt = 0x8000u, kCountMost = 0x7fffu, kBiasPlaces = 0xffffu;
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

template <int DT, int UNITS>
__global__ __launch_bounds__(kBlock) void adjust_kernel(AdjustArgs a) {
  constexpr int B = Traits<DT>::B, E = kElems<DT>;
  constexpr uint32_t kRun = UNITS * kBlock * E;
  __shared__ __attribute__((aligned(16))) uint32_t table[kRun];
  const uint32_t in = blockIdx.x / (uint32_t)a.chunks, chunk = blockIdx.x - in * (uint32_t)a.chunks;
  const uint64_t row = a.first_row + in;
  int r = min((int)((2 * (uint64_t)chunk + 1) * a.ranks_q32 >> 33), a.p - 1);
  while (a.first[r] > (int)chunk) --r;
  while (a.first[r + 1] <= (int)chunk) ++r;
  const int64_t vocab = a.first_index[r + 1] - a.first_index[r], at = (int64_t)(chunk - (uint32_t)a.first[r]) * kRun;
  const uint32_t len = (uint32_t)min((int64_t)kRun, vocab - at), full = len / E, part = len % E;
  const int64_t first = a.first_index[r] + at;  // vocabulary index of the run's first entry
  const uint8_t* src = as_global(static_cast<const uint8_t*>(a.logits[r])) + ((int64_t)row * a.ld[r] + at) * B;
  uint8_t* dst = as_global(static_cast<uint8_t*>(a.out[r])) + ((int64_t)row * a.old[r] + at) * B;
  const RowBuffer from(src, full * 16), to(dst, full * 16);
  RawUnit<DT, E> z[UNITS];
#pragma unroll
  for (int i = 0; i < UNITS; ++i) z[i] = load_unit<DT, E, true>(from, (i * kBlock + threadIdx.x) * E);
  RawUnit<DT, E> last = zero_unit<DT, E>();
  const bool ends = part && full % kBlock == threadIdx.x;  // this lane has the run's last elements
  if (ends) last = load_part<DT, E>(src, full * E, part);

  const Span hist(a.offsets, row, a.ntokens), bias(a.bias_offsets, row, a.nbias);
  const int64_t prompt = a.prompt ? ld_const(a.prompt + row) : 0;
  const uint32_t answer = prompt < 0 ? 0 : (uint32_t)min(prompt, (int64_t)hist.n);  // where the answer starts
  const int64_t* tokens = as_global(a.tokens) + hist.begin;
  const int64_t* places = as_global(a.bias_idx) + bias.begin;
  const float* values = as_global(a.bias) + bias.begin;
  const float repetition = a.repetition ? ld_const(a.repetition + row) : 1.0f;
  const float presence = a.presence ? ld_const(a.presence + row) : 0.0f;
  const float frequency = a.frequency ? ld_const(a.frequency + row) : 0.0f;

  auto penalize = [&](float v, bool seen, uint32_t count) {
    if (seen) v = v > 0.0f ? v / repetition : v * repetition;
    if (count) v -= (float)count * frequency + presence;
    return v;
  };
  // the mask's bits of unit u
  auto mask_out = [&](uint32_t u, float (&f)[E]) {
    if (!a.mask) return;
    const uint64_t bit = (uint64_t)first + (uint64_t)u * E;
    const uint32_t* words = as_global(a.mask) + row * (uint64_t)a.mask_ld;
    // (where both words are the row's last one, the bits past it are not looked at)
    const uint64_t w0 = bit / 32, w1 = min((bit + E - 1) / 32, (uint64_t)(a.first_index[a.p] - 1) / 32);
    const uint32_t allow = (uint32_t)((((uint64_t)words[w1] << 32) | words[w0]) >> (bit % 32));
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (!(allow >> e & 1)) f[e] = -__builtin_inff();
  };
  // every unit of the run that `mine` takes, marked by mark(unit, values)
  auto finish = [&](auto mine, auto mark) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const uint32_t u = i * kBlock + threadIdx.x;
      if (u < full && mine(u)) {
        float f[E];
        widen_unit(z[i], f);
        mark(u, f);
        mask_out(u, f);
        store_unit<DT, E, true>(to, u * E, narrow_unit<DT, E>(f));
      }
    }
    if (ends && mine(full)) {
      float f[E];
      widen_unit(last, f);
      mark(full, f);
      mask_out(full, f);
      store_part<DT, E>(dst, full * E, part, f);
    }
  };
  // Each entry of a list of n places in this run (of `most` entries from
  // vocabulary index `begin` on): f(entry's place in the run, place in the list).
  auto each = [&](const int64_t* list, uint32_t n, int64_t begin, uint32_t most, auto f) {
    for (uint32_t i = threadIdx.x; i < n; i += kBlock) {
      const uint64_t j = (uint64_t)list[i] - (uint64_t)begin;
      if (j < most) f((uint32_t)j, i);
    }
  };

  if (!hist.n && !bias.n) {
    finish([](uint32_t) { return true; }, [](uint32_t, float (&)[E]) {});
  } else if (hist.n <= kCountMost && bias.n <= kBiasPlaces) {
    u32x4* t = reinterpret_cast<u32x4*>(table);
#pragma unroll
    for (int i = 0; i < (int)(kRun / 4 / kBlock); ++i) t[i * kBlock + threadIdx.x] = u32x4{0, 0, 0, 0};
    __syncthreads();
    if (bias.n) {
      each(places, bias.n, first, len, [&](uint32_t j, uint32_t i) { atomicMax(&table[j], (kBiasPlaces - i) << 16); });
      __syncthreads();
    }
    each(tokens, hist.n, first, len, [&](uint32_t j, uint32_t i) {
      if (i >= answer) atomicAdd(&table[j], 1u);
      else atomicOr(&table[j], kPrompt);
    });
    __syncthreads();
    finish([](uint32_t) { return true; }, [&](uint32_t u, float (&f)[E]) {
      uint32_t w[E], any = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) any |= w[e] = table[u * E + e];
      if (any) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          f[e] = penalize(f[e], w[e] & 0xffffu, w[e] & kCountMost);
          if (w[e] >> 16) f[e] += values[kBiasPlaces - (w[e] >> 16)];
        }
      }
    });
  } else {
    // two words an entry: count and prompt, place of the bias
    constexpr uint32_t kHalf = kRun / 2;
    uint32_t* where = table + kHalf;
    for (uint32_t half = 0; half < 2; ++half) {
      const int64_t begin = first + half * kHalf;
      for (uint32_t i = threadIdx.x; i < kHalf; i += kBlock) {
        table[i] = 0;
        where[i] = ~0u;
      }
      __syncthreads();
      each(places, bias.n, begin, kHalf, [&](uint32_t j, uint32_t i) { atomicMin(&where[j], i); });
      each(tokens, hist.n, begin, kHalf, [&](uint32_t j, uint32_t i) {
        if (i >= answer) atomicAdd(&table[j], 1u);
        else atomicOr(&table[j], kLongPrompt);
      });
      __syncthreads();
      finish([&](uint32_t u) { return u * E / kHalf == half; }, [&](uint32_t u, float (&f)[E]) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t j = u * E - half * kHalf + e, w = table[j], k = where[j];
          f[e] = penalize(f[e], w, w & ~kLongPrompt);
          if (k != ~0u) f[e] += values[k];
        }
      });
      __syncthreads();
    }
  }
}

// Units to a lane: four where that still gives the card's CUs some workgroups
// each, which then go over a row's history the fewest times.
constexpr uint64_t kManyRuns = 2048;

template <int DT, int UNITS>
int adjust_t(AdjustArgs a, hipStream_t s) {
  constexpr int64_t kRun = (int64_t)UNITS * kBlock * kElems<DT>;
  a.first[0] = 0;
  for (int r = 0; r < a.p; ++r) a.first[r + 1] = a.first[r] + (int)((a.first_index[r + 1] - a.first_index[r] + kRun - 1) / kRun);
  a.chunks = a.first[a.p];
  a.ranks_q32 = ((uint64_t)a.p << 32) / (uint64_t)a.chunks;
  const uint64_t all = a.rows;
  return over_rows(all, (uint64_t)a.chunks * (kBlock / kWave), [&](uint64_t first, uint64_t rows, dim3 grid) {
    a.first_row = first;
    a.rows = rows;
    hipLaunchKernelGGL((adjust_kernel<DT, UNITS>), grid, dim3(kBlock), 0, s, a);
  });
}

template <int DT>
int adjust_d(const AdjustArgs& a, hipStream_t s) {
  constexpr uint64_t kLong = 4 * kBlock * kElems<DT>;
  uint64_t runs = 0;
  for (int r = 0; r < a.p; ++r) runs += ((uint64_t)(a.first_index[r + 1] - a.first_index[r]) + kLong - 1) / kLong;
  return a.rows >= (kManyRuns + runs - 1) / runs ? adjust_t<DT, 4>(a, s) : adjust_t<DT, 1>(a, s);
}

}  // namespace

int launch_adjust(int dtype, const AdjustArgs& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  return dtype == kF32 ? adjust_d<kF32>(a, s) : adjust_d<kBF16>(a, s);
}

}  // namespace coll
