// Kernel argument blocks and launcher declarations of the token-wise operators
// (host and device).
#pragma once

#include "kernel_args.h"

namespace coll {

// Token-wise operators.  A launch takes up to kArgRanks ranks (the rank is
// the grid's second dimension), so that its pointer arrays stay well below
// the 4 KiB of a kernel's arguments; more ranks take a second launch.
constexpr int kArgRanks = 32;

// Workgroups of a launch along a grid dimension, `block` work items each: HIP
// takes fewer than 2^32 work items.
constexpr uint64_t most_blocks(uint64_t block) { return 0xffffffffull / block; }

struct LnArgs {
  const void* x[kArgRanks];      // rows; backward from a checkpoint: its rows
  const void* dy[kArgRanks];     // backward
  const void* gamma[kArgRanks];  // or null: ones
  const void* beta[kArgRanks];   // or null: zeros
  float* mean[kArgRanks];        // forward: written unless null; backward: read
  float* rstd[kArgRanks];
  void* y[kArgRanks];            // backward from a checkpoint: or null
  void* dx[kArgRanks];
  uint8_t* ckpt[kArgRanks];      // forward with a checkpoint
  float* ws;                     // backward: partial sums [groups][2][hidden] of this launch
  uint64_t rows;                 // per rank
  uint64_t hidden;
  uint64_t row_bytes;            // of a checkpoint row
  uint32_t glog;                 // log2 of a checkpoint group's elements
  int ranks;                     // of this launch
  float eps;
};

struct LnJoinArgs {
  void* dgamma[kMaxRanks];       // null where absent
  void* dbeta[kMaxRanks];
  const float* ws;               // [parts][sums][hidden]
  uint64_t hidden;
  uint64_t sums;                 // 2: dgamma's, then dbeta's; 1: dgamma's alone
  uint64_t first;                // column of this launch's first sum, of sums * hidden (set by the launcher)
  uint32_t parts;
  int p;
  int avg;
};

// RMS norm, forward and backward.
struct RmsArgs {
  const void* x[kArgRanks];      // forward: rows; backward: dy
  const void* res[kArgRanks];    // the residual; backward: dh (null: none, on every rank)
  const void* gamma[kArgRanks];  // or null: ones
  void* h[kArgRanks];            // forward with a residual: written unless null; backward: read
  float* rstd[kArgRanks];        // forward: written unless null; backward: read
  void* y[kArgRanks];            // forward: written unless null; backward: dx
  uint8_t* y8[kArgRanks];        // forward in 8 bits
  float* ws;                     // backward: partial sums [groups][hidden] of this launch
  uint64_t rows;                 // per rank
  uint64_t hidden;
  uint64_t row_bytes;            // of a row in 8 bits
  uint32_t glog;                 // log2 of its groups' elements
  int ranks;                     // of this launch
  float eps;
};

// 8-bit checkpoints and the gated activation.
enum Ckpt8Kind : int { kCkpt8Save = 0, kCkpt8Load = 1, kSwigluForward = 2, kSwigluBackward = 3 };
struct Ckpt8Args {
  const void* src[kArgRanks];    // rows; backward: dout
  void* dst[kArgRanks];          // load: rows; forward: out; backward: the rows' gradient
  void* again[kArgRanks];        // backward: the output again, or null
  uint8_t* ckpt[kArgRanks];
  uint64_t rows;
  uint64_t hidden;               // elements of a checkpoint row
  uint64_t width;                // elements that the lanes walk per row (ffn in the gated activation)
  uint64_t units;                // units of them (set by the launcher)
  uint64_t row_bytes;
  uint64_t div_mul;              // division by units (set by the launcher)
  uint32_t div_shift;
  uint32_t glog;                 // log2 of a group's elements
};

// Vocabulary log probabilities over p shards.  A row's shards are cut into
// pieces, at most kMaxPieces to a row (a wave's lanes).
constexpr int kMaxPieces = 64;
constexpr int kMaxTop = 32;
// Elements that a wave takes in one step.
constexpr int kLogprobStep = 2048;
// Groups of elements (a row's) whose largest the search for alternatives
// starts from.  Eight lanes, so whole 128-byte lines, share a group.
constexpr int kMaxGroups = 1024, kGroupLanes = 8, kSegGroups = 64 / kGroupLanes;
// Pieces that a shard's row is cut into, as far as its length allows: enough
// for kLogprobWaves waves over all rows.  (Rows past that many want one piece;
// their product with p may not fit.)
constexpr uint64_t kLogprobWaves = 8192;
inline uint64_t logprob_want(int p, uint64_t rows) {
  const uint64_t shards = (rows < kLogprobWaves ? rows : kLogprobWaves) * (uint64_t)p;
  const uint64_t want = shards ? (kLogprobWaves + shards - 1) / shards : 1;
  return want < kMaxPieces ? want : kMaxPieces;
}
// The most rows that want so many (2 or more).
inline uint64_t logprob_most_rows(int p, uint64_t want) { return (kLogprobWaves - 1) / ((want - 1) * (uint64_t)p); }
struct LogprobPlan {
  int pieces;                    // per row, over all ranks
  uint64_t ranks_q32;            // ranks to a piece on average, times 2^32: where a piece's rank is first sought
  int segs, seg_steps;           // a piece's segments, of kSegGroups groups each, and the steps of one
  int first[kMaxRanks + 1];      // first piece of each rank, and the end
  int64_t len[kMaxRanks];        // elements per piece (the rank's last may be shorter)
};
struct LogprobArgs {
  const void* logits[kMaxRanks];
  int64_t ld[kMaxRanks];         // elements from row to row
  int64_t first_index[kMaxRanks + 1];  // first vocabulary index of each shard, and the end
  LogprobPlan plan;
  const int64_t* targets;
  float* part;                   // [rows][pieces][4]: max, sum, entropy sum, target's logit (-inf where elsewhere)
  uint32_t* places;              // with alternatives: [rows][pieces][4], where each piece lies
  float* bests;                  // with alternatives: [rows][pieces][segs][kSegGroups], largest elements
  uint64_t rows, first_row;      // this launch's
  float scale;                   // inverse temperature
  int p;
  int top;
};
struct LogprobJoinArgs {
  float* stats[kMaxRanks];       // [rows][2]
  float* logp[kMaxRanks];
  float* entropy[kMaxRanks];     // null where absent
  float* top_logp[kMaxRanks];    // [rows][top]
  int32_t* top_idx[kMaxRanks];
};
struct LogprobGradArgs {
  const void* logits[kMaxRanks];
  void* dlogits[kMaxRanks];
  int64_t ld[kMaxRanks];
  int64_t dld[kMaxRanks];
  int64_t first_index[kMaxRanks + 1];
  const int64_t* targets;
  const float* stats;            // [rows][2]
  const float* dlogp;
  const float* entropy;          // null without dentropy
  const float* dentropy;
  uint64_t rows, first_row;      // this launch's
  float scale;
  int p;
};

// Distillation from a teacher's entries over the same shards and pieces.
constexpr int kMaxDistill = 128;
struct DistillArgs {
  const void* logits[kMaxRanks];
  int64_t ld[kMaxRanks];         // elements from row to row
  int64_t first_index[kMaxRanks + 1];  // first vocabulary index of each shard, and the end
  LogprobPlan plan;
  const int32_t* idx;            // [rows][top]
  float* part;                   // [rows][pieces][2]: max and sum, without the entries where there is a tail
  float* zs;                     // [rows][top]: the entries' logits
  uint64_t rows, first_row;      // this launch's
  float scale;                   // inverse temperature
  int p;
  int top;
};
struct DistillJoinArgs {
  float* stats[kMaxRanks];       // [rows][4]
  float* loss[kMaxRanks];
  const int32_t* idx;
  const float* logp;             // [rows][top]
  const float* part;
  const float* zs;
  uint64_t rows, first_row;      // this launch's
  int64_t vocab;
  float scale;
  int p, top, pieces;
  int tail;                      // whether all other entries are one more class
};
struct DistillGradArgs {
  const void* logits[kMaxRanks];
  void* dlogits[kMaxRanks];
  int64_t ld[kMaxRanks];
  int64_t dld[kMaxRanks];
  int64_t first_index[kMaxRanks + 1];
  const int32_t* idx;
  const float* logp;
  const float* stats;            // [rows][4]
  const float* dloss;
  uint64_t rows, first_row;      // this launch's
  float scale;
  int p, top, tail;
};

// Penalties, biases and masks on the same shards; null where absent.
struct AdjustArgs {
  const void* logits[kMaxRanks];
  void* out[kMaxRanks];
  int64_t ld[kMaxRanks];         // elements from row to row
  int64_t old[kMaxRanks];
  int64_t first_index[kMaxRanks + 1];  // first vocabulary index of each shard, and the end
  int first[kMaxRanks + 1];      // first run of each shard's rows, and the end (set by the launcher)
  int chunks;                    // runs of a row (set by the launcher)
  int spread;                    // rows whose runs take turns (set by the launcher)
  uint64_t ranks_q32;            // ranks to a run on average, times 2^32
  const int64_t* tokens;         // [ntokens], row r's from offsets[r] to offsets[r + 1]
  const int64_t* offsets;
  const int64_t* prompt;
  const float* repetition;       // [rows]
  const float* presence;
  const float* frequency;
  const int64_t* bias_idx;       // [nbias], row r's from bias_offsets[r] to bias_offsets[r + 1]
  const float* bias;
  const int64_t* bias_offsets;
  const uint32_t* mask;          // [rows], mask_ld words apart
  int64_t mask_ld;
  uint64_t ntokens, nbias;
  uint64_t rows, first_row;      // this launch's
  int p;
};

// Layer norm.  ln_backward_groups: workgroups of each launch of the backward
// pass (they fix its workspace, so they depend on the shape alone).
uint32_t ln_backward_groups(int p, uint64_t rows, uint64_t hidden);
bool ln_forward_keeps(int dtype, uint64_t hidden, uint64_t group);
int launch_ln_forward(int dtype, int wdtype, const LnArgs& a, bool ckpt, void* stream);
int launch_ln_backward(int dtype, int wdtype, const LnArgs& a, uint32_t groups, bool ckpt, void* stream);
int launch_ln_join(int wdtype, const LnJoinArgs& a, void* stream);

// RMS norm.  rms_backward_groups: as ln_backward_groups.  The weights'
// gradients are joined by launch_ln_join.
uint32_t rms_backward_groups(int p, uint64_t rows, uint64_t hidden);
int launch_rms_forward(int dtype, int wdtype, const RmsArgs& a, bool residual, bool fp8, void* stream);
int launch_rms_backward(int dtype, int wdtype, const RmsArgs& a, bool dh, uint32_t groups, void* stream);

// 8-bit checkpoints and the gated activation (kind: Ckpt8Kind).
int launch_ckpt8(int kind, int dtype, Ckpt8Args a, int ranks, void* stream);

// Vocabulary log probabilities: the pieces' pass and the join over them,
// then the logits' gradient.
// Workspace bytes of a piece.
inline size_t logprob_piece_bytes(const LogprobPlan& plan, int top) {
  return top ? 32 + (size_t)plan.segs * kSegGroups * 4 : 16;
}
void logprob_plan(int p, uint64_t rows, const int64_t* vocab, LogprobPlan* plan);
int launch_logprob(int dtype, const LogprobArgs& a, const LogprobJoinArgs& j, void* stream);
int launch_logprob_backward(int dtype, const LogprobGradArgs& a, void* stream);

// Distillation: the pieces' pass (a.plan: logprob_plan's) and the join over
// them, then the logits' gradient.
int launch_distill(int dtype, const DistillArgs& a, const DistillJoinArgs& j, void* stream);
int launch_distill_backward(int dtype, const DistillGradArgs& a, void* stream);

int launch_adjust(int dtype, const AdjustArgs& a, void* stream);

}  // namespace coll
