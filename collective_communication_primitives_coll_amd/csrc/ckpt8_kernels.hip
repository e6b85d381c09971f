// Activation checkpoints in 8 bits: rows of e4m3 codes with one fp32 scale
// per group (the row format of the FP8 dispatch), written and read whole,
// or by the two passes of the gated activation
//
//   forward   out = silu(g) u,   silu(g) = g s,  s = 1 / (1 + e^-g),
//             from rows [g | u]; the rows themselves are kept in 8 bits
//   backward  dg = dy u s (1 + g (1 - s)),  du = dy g s
//             with g and u from the checkpoint
//
// Bound by HBM: forward moves 8 bytes an element pair in bf16 (4 + 2 + 2),
// backward 10 with the output written again, at about 30 fp32 operations.
// The rows are cut into units of 16 bytes that the lanes take in their
// order through the whole rank, rows one after the other, so narrow rows
// leave no lanes idle.  A group is whole units, its first unit at a
// multiple of the group's lane count, so it lies within one wave and its
// largest magnitude is found with lane exchanges.
#include "token_unit.h"

namespace coll {

namespace {

// Units per lane in flight.
constexpr int kCkptUnits = 2;

struct RowIndex {
  uint64_t row;
  uint32_t unit;
};

// The unit that lies `off` units past unit `u0` of row `row0`.
__device__ __forceinline__ RowIndex row_index(uint64_t row0, uint32_t u0, uint32_t off, const Ckpt8Args& a) {
  const uint32_t n = u0 + off;  // below 2^31 + the tile
  const uint32_t q = (uint32_t)(((uint64_t)n * a.div_mul) >> a.div_shift);
  return RowIndex{row0 + q, n - q * (uint32_t)a.units};
}

// Calls body(row, unit, valid) for each unit of this workgroup's tiles,
// with all lanes of a wave together.  `load` is called for all units of a
// tile before `use` is called for any.
template <class State, class Load, class Use>
__device__ __forceinline__ void walk_units(const Ckpt8Args& a, Load load, Use use) {
  constexpr uint32_t TILE = kBlock * kCkptUnits;
  const uint64_t total = a.rows * a.units, tiles = (total + TILE - 1) / TILE;
  for (uint64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const uint64_t base = t * TILE, row0 = base / a.units;
    const uint32_t u0 = (uint32_t)(base - row0 * a.units);
    State st[kCkptUnits];
    RowIndex at[kCkptUnits];
    bool in[kCkptUnits];
#pragma unroll
    for (int k = 0; k < kCkptUnits; ++k) {
      const uint32_t off = k * kBlock + threadIdx.x;
      at[k] = row_index(row0, u0, off, a);
      in[k] = base + off < total;
      load(st[k], at[k].row, at[k].unit, in[k]);
    }
#pragma unroll
    for (int k = 0; k < kCkptUnits; ++k) use(st[k], at[k].row, at[k].unit, in[k]);
  }
}

__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896340736f));
}

template <int DT, int E>
__global__ __launch_bounds__(kBlock) void ckpt8_save_kernel(Ckpt8Args a) {
  const int rank = blockIdx.y;
  struct State {
    RawUnit<DT, E> x;
  };
  walk_units<State>(
      a,
      [&](State& s, uint64_t row, uint64_t u, bool in) {
        s.x = in ? load_unit<DT, E, true>(static_cast<const uint8_t*>(a.src[rank]) + row * a.hidden * Traits<DT>::B, u * E)
                 : zero_unit<DT, E>();
      },
      [&](State& s, uint64_t row, uint64_t u, bool in) {
        float f[E];
        widen_unit(s.x, f);
        const RawUnit<kE4M3, E> q = encode_unit<DT, E>(s.x, f, a.glog);
        if (in) store_codes<E, true>(a.ckpt[rank] + row * a.row_bytes, a.hidden, a.row_bytes, u * E, a.glog, q);
      });
}

template <int DT, int E>
__global__ __launch_bounds__(kBlock) void ckpt8_load_kernel(Ckpt8Args a) {
  const int rank = blockIdx.y;
  struct State {
    RawUnit<kE4M3, E> q;
  };
  walk_units<State>(
      a,
      [&](State& s, uint64_t row, uint64_t u, bool in) {
        s.q = in ? load_codes<E, true>(a.ckpt[rank] + row * a.row_bytes, a.hidden, u * E, a.glog) : zero_unit<kE4M3, E>();
      },
      [&](State& s, uint64_t row, uint64_t u, bool in) {
        float f[E];
        widen_unit(s.q, f);
        if (in) store_unit<DT, E, true>(static_cast<uint8_t*>(a.dst[rank]) + row * a.hidden * Traits<DT>::B, u * E, narrow_unit<DT, E>(f));
      });
}

// a.hidden: elements of a checkpoint row, 2 * ffn; a.width: ffn.
template <int DT, int E>
__global__ __launch_bounds__(kBlock) void swiglu_forward_kernel(Ckpt8Args a) {
  const int rank = blockIdx.y;
  struct State {
    RawUnit<DT, E> g, u;
  };
  walk_units<State>(
      a,
      [&](State& s, uint64_t row, uint64_t j, bool in) {
        if (in) {
          const uint8_t* x = static_cast<const uint8_t*>(a.src[rank]) + row * a.hidden * Traits<DT>::B;
          s.g = load_unit<DT, E, true>(x, j * E);
          s.u = load_unit<DT, E, true>(x, (a.units + j) * E);
        } else {
          s.g = s.u = zero_unit<DT, E>();
        }
      },
      [&](State& s, uint64_t row, uint64_t j, bool in) {
        float g[E], u[E];
        widen_unit(s.g, g);
        widen_unit(s.u, u);
        const RawUnit<kE4M3, E> qg = encode_unit<DT, E>(s.g, g, a.glog), qu = encode_unit<DT, E>(s.u, u, a.glog);
        if (!in) return;
        uint8_t* c = a.ckpt[rank] + row * a.row_bytes;
        store_codes<E, true>(c, a.hidden, a.row_bytes, j * E, a.glog, qg);
        store_codes<E, true>(c, a.hidden, a.row_bytes, (a.units + j) * E, a.glog, qu);
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] *= g[e] * sigmoid(g[e]);
        store_unit<DT, E, true>(static_cast<uint8_t*>(a.dst[rank]) + row * (a.hidden / 2) * Traits<DT>::B, j * E, narrow_unit<DT, E>(u));
      });
}

template <int DT, int E>
__global__ __launch_bounds__(kBlock) void swiglu_backward_kernel(Ckpt8Args a) {
  const int rank = blockIdx.y;
  struct State {
    RawUnit<kE4M3, E> g, u;
    RawUnit<DT, E> dy;
  };
  walk_units<State>(
      a,
      [&](State& s, uint64_t row, uint64_t j, bool in) {
        if (in) {
          const uint8_t* c = a.ckpt[rank] + row * a.row_bytes;
          s.g = load_codes<E, true>(c, a.hidden, j * E, a.glog);
          s.u = load_codes<E, true>(c, a.hidden, (a.units + j) * E, a.glog);
          s.dy = load_unit<DT, E, true>(static_cast<const uint8_t*>(a.src[rank]) + row * (a.hidden / 2) * Traits<DT>::B, j * E);
        } else {
          s.g = s.u = zero_unit<kE4M3, E>();
          s.dy = zero_unit<DT, E>();
        }
      },
      [&](State& s, uint64_t row, uint64_t j, bool in) {
        if (!in) return;
        float g[E], u[E], dy[E];
        widen_unit(s.g, g);
        widen_unit(s.u, u);
        widen_unit(s.dy, dy);
        float again[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float sg = sigmoid(g[e]), act = g[e] * sg;
          again[e] = act * u[e];
          g[e] = dy[e] * u[e] * sg * (1.0f + g[e] * (1.0f - sg));
          u[e] = dy[e] * act;
        }
        uint8_t* dx = static_cast<uint8_t*>(a.dst[rank]) + row * a.hidden * Traits<DT>::B;
        store_unit<DT, E, true>(dx, j * E, narrow_unit<DT, E>(g));
        store_unit<DT, E, true>(dx, (a.units + j) * E, narrow_unit<DT, E>(u));
        if (a.again[rank])
          store_unit<DT, E, true>(static_cast<uint8_t*>(a.again[rank]) + row * (a.hidden / 2) * Traits<DT>::B, j * E, narrow_unit<DT, E>(again));
      });
}

}  // namespace

int launch_ckpt8(int kind, int dtype, Ckpt8Args a, int ranks, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  // 16-byte units; a group of 512 in fp32 would span two waves of them, and
  // takes units of 8 elements
  const int elems = dtype == kF32 && a.glog < 9 ? 4 : 8;
  a.units = a.width / elems;
  // exact division by the units of a row, for the 31-bit values of
  // row_index: with 2^sh >= d, m = ceil(2^(31+sh) / d) fits 33 bits and
  // (n m) >> (31+sh) = floor(n / d) for n < 2^31
  uint32_t sh = 0;
  while ((uint64_t{1} << sh) < a.units) ++sh;
  a.div_shift = 31 + sh;
  a.div_mul = ((uint64_t{1} << a.div_shift) + a.units - 1) / a.units;
  const uint64_t tile = kBlock * kCkptUnits, tiles = (a.rows * a.units + tile - 1) / tile;
  // (the workgroups walk what one launch cannot hold)
  const dim3 grid((uint32_t)(tiles < most_blocks(kBlock) ? tiles : most_blocks(kBlock)), ranks), block(kBlock);
#define COLL_CKPT8(K)                                                                                \
  if (dtype == kBF16) hipLaunchKernelGGL((K<kBF16, 8>), grid, block, 0, s, a);                       \
  else if (elems == 4) hipLaunchKernelGGL((K<kF32, 4>), grid, block, 0, s, a);                       \
  else hipLaunchKernelGGL((K<kF32, 8>), grid, block, 0, s, a);                                       \
  break;
  switch (kind) {
    case kCkpt8Save: COLL_CKPT8(ckpt8_save_kernel)
    case kCkpt8Load: COLL_CKPT8(ckpt8_load_kernel)
    case kSwigluForward: COLL_CKPT8(swiglu_forward_kernel)
    default: COLL_CKPT8(swiglu_backward_kernel)
  }
#undef COLL_CKPT8
  return (int)hipGetLastError();
}

}  // namespace coll
