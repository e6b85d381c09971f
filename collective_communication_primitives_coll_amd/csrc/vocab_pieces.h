// Rows of a vocabulary that lies in p shards, cut into pieces of one wave each:
// what the kernels over sharded logits share (log probabilities,
// distillation, and of the small parts a sampler's adjustments).
#pragma once

#include <float.h>

#include <algorithm>

#include "token_unit.h"

namespace coll {

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
constexpr float kFar = -16384.0f;
constexpr int kStep = kLogprobStep / kWave;  // elements per lane and step

// A piece of a row's shard: its elements before the first 16-byte boundary,
// its whole units and the rest.  Pieces after the first start on a 128-byte
// line, so that no two waves share one and only a shard's two ends go element
// by element.
constexpr int kLine = 128;
struct Piece {
  int64_t begin;       // first element
  uint32_t head, tail; // elements
  uint32_t units;      // of 16 bytes
};
template <int DT>
__device__ __forceinline__ Piece piece_of(const uint8_t* row, int64_t vocab, int64_t len, int k) {
  constexpr int B = Traits<DT>::B, E = kElems<DT>;
  const int64_t mis = (int64_t)((uintptr_t)row % kLine) / B;
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

// A launch's item: a piece of a row.  No loop over items, so that nothing is
// hoisted out of it, and 32-bit numbers within a launch.
struct Item {
  uint64_t row;
  int piece, r;  // of the row, rank that holds it
  bool any;
  __device__ __forceinline__ Item(const LogprobPlan& plan, uint64_t rows, uint64_t first_row, int p) {
    const uint32_t i = blockIdx.x * (kBlock / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t in = i / (uint32_t)plan.pieces;
    row = first_row + in;
    any = in < rows;
    piece = (int)(i - in * (uint32_t)plan.pieces);
    r = min((int)((2 * (uint64_t)piece + 1) * plan.ranks_q32 >> 33), p - 1);
    while (plan.first[r] > piece) --r;
    while (plan.first[r + 1] <= piece) ++r;
  }
};

template <int DT>
__device__ __forceinline__ RawUnit<DT, kElems<DT>> masked_unit() {
  const uint32_t w = DT == kBF16 ? 0xff80ff80u : 0xff800000u;
  return RawUnit<DT, kElems<DT>>{{u32x4{w, w, w, w}}};
}

// LDS is written and read by one wave alone.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int N>
__device__ __forceinline__ float largest(const float (&f)[N]) {
  float v = f[0];
#pragma unroll
  for (int e = 1; e < N; ++e) v = fmaxf(v, f[e]);
  return v;
}

template <int N>
__device__ __forceinline__ float sum_of(const float (&v)[N]) {
  float s = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) s += v[i];
  return s;
}

uint32_t wave_grid(uint64_t waves) { return (uint32_t)((waves + kBlock / kWave - 1) / (kBlock / kWave)); }

// Calls f(first row, rows, blocks) for launches of as many rows as one may
// have, `waves` waves to a row (2^22 at most, so that a row always fits).
template <class F>
int over_rows(uint64_t rows, uint64_t waves, F f) {
  const uint64_t most = most_blocks(kBlock) * (kBlock / kWave) / waves;
  for (uint64_t first = 0; first < rows; first += most) {
    const uint64_t n = std::min(most, rows - first);
    f(first, n, dim3(wave_grid(n * waves)));
    if (const int e = (int)hipGetLastError()) return e;
  }
  return 0;
}

void finish_plan(LogprobPlan* plan, int p) {
  plan->pieces = plan->first[p];
  plan->ranks_q32 = ((uint64_t)p << 32) / (uint64_t)std::max(plan->pieces, 1);
}

// Pieces of `len` elements that cover a shard whose rows start at most
// `before` elements after a line's start.
int pieces_of(int64_t vocab, int64_t before, int64_t len) { return vocab ? (int)((vocab + before + len - 1) / len) : 0; }

}  // namespace

}  // namespace coll
