// Host side of the token-wise operators' entry points: layer norm, 8-bit
// checkpoints, vocabulary log probabilities.  Argument checks, byte ranges
// and the record of the last HIP error are internal to coll_api.cpp, so that
// file is part of this translation unit, and is not compiled by itself.
#include "coll_api.cpp"

#include "token_args.h"

namespace {

// The byte ranges of one call, in a fixed array (a call allocates nothing
// and cannot throw).  The check sorts them by address and keeps the furthest
// end of the outputs, and of all ranges, seen so far.
struct RangeSet {
  static constexpr int kMost = 12 * kMaxRanks + 16;
  Range r[kMost];
  int n = 0;

  void add(const void* p, size_t bytes, bool out) {
    if (p && bytes && n < kMost) r[n++] = rng(p, bytes, out, 0);
  }
  template <typename PtrT>
  void add_all(PtrT const* arr, int p, size_t bytes, bool out) {
    for (int i = 0; arr && i < p; ++i) add(arr[i], bytes, out);
  }
  // An input that may be its rank's output: then one range, an output.
  void add_in_place(const void* const* in, void* const* out, int p, size_t bytes) {
    for (int i = 0; i < p; ++i) {
      if (in[i] != out[i]) add(in[i], bytes, false);
      add(out[i], bytes, true);
    }
  }
  coll_status_t check() {
    std::sort(r, r + n, [](const Range& a, const Range& b) { return a.b < b.b; });
    uintptr_t any = 0, outs = 0;
    for (int i = 0; i < n; ++i) {
      if (r[i].b < (r[i].out ? any : outs)) return COLL_ERR_ALIAS;
      any = std::max(any, r[i].e);
      if (r[i].out) outs = std::max(outs, r[i].e);
    }
    return COLL_OK;
  }
};

// Optional rank arrays: absent as a whole, never in part.
template <typename PtrT>
bool none_or_all(PtrT const* arr, int p) {
  return !arr || all_non_null(arr, p);
}
template <typename PtrT>
bool aligned_or_none(PtrT const* arr, int p, size_t d) {
  return !arr || elem_aligned(arr, p, d);
}

coll_status_t float_dtype(int d) {
  if (!arith_dtype_ok(d)) return COLL_ERR_INVALID_ARG;
  return d == COLL_I32 ? COLL_ERR_UNSUPPORTED : COLL_OK;
}

// A checkpoint's groups must lie within one wave: 64 lanes of 8 elements.
coll_status_t ckpt8_shape(size_t hidden, size_t group) {
  if (hidden == 0 || group == 0 || hidden % group) return COLL_ERR_INVALID_ARG;
  if (group < 16 || group > 512 || (group & (group - 1)) || hidden >= (size_t{1} << 31)) return COLL_ERR_UNSUPPORTED;
  return COLL_OK;
}
uint32_t group_log(size_t group) {
  uint32_t s = 0;
  while ((size_t{1} << s) < group) ++s;
  return s;
}

// Arguments that layer norm's entry points share: shape and types.
coll_status_t check_ln_shape(int p, size_t rows, size_t hidden, size_t group, bool ckpt, int dtype, int wdtype,
                             size_t* bytes, size_t* ckpt_bytes) {
  if (p < 1 || p > kMaxRanks || hidden == 0) return COLL_ERR_INVALID_ARG;
  coll_status_t st = float_dtype(dtype);
  if (st == COLL_OK) st = float_dtype(wdtype);
  if (st != COLL_OK) return st;
  if (wdtype != COLL_F32 && wdtype != dtype) return COLL_ERR_UNSUPPORTED;
  if (hidden >= (size_t{1} << 31)) return COLL_ERR_UNSUPPORTED;
  size_t t;
  if (!mul_ok(rows, hidden, 4 * (size_t)kMaxRanks, &t)) return COLL_ERR_INVALID_ARG;
  *bytes = rows * hidden * dsize(dtype);
  *ckpt_bytes = 0;
  if (ckpt) {
    st = ckpt8_shape(hidden, group);
    if (st != COLL_OK) return st;
    *ckpt_bytes = rows * fp8_row_bytes(hidden, group);
  }
  return COLL_OK;
}

// One of the four checkpoint kernels over all ranks; arguments as Ckpt8Args.
coll_status_t run_ckpt8(int kind, const void* const* src, void* const* dst, void* const* again, void* const* ckpt, int p,
                        size_t rows, size_t hidden, size_t width, size_t group, int dtype, void* stream) {
  for (int r0 = 0; r0 < p; r0 += coll::kArgRanks) {
    const int n = std::min(p - r0, coll::kArgRanks);
    coll::Ckpt8Args a{};
    for (int r = 0; r < n; ++r) {
      if (src) a.src[r] = src[r0 + r];
      if (dst) a.dst[r] = dst[r0 + r];
      if (again) a.again[r] = again[r0 + r];
      a.ckpt[r] = (uint8_t*)ckpt[r0 + r];
    }
    a.rows = rows;
    a.hidden = hidden;
    a.width = width;
    a.row_bytes = fp8_row_bytes(hidden, group);
    a.glog = group_log(group);
    const int e = coll::launch_ckpt8(kind, dtype, a, n, stream);
    if (e) return hip_fail(e);
  }
  return COLL_OK;
}

coll_status_t ln_forward(const void* const* x, const void* const* gamma, const void* const* beta, void* const* y,
                         float* const* mean, float* const* rstd, void* const* ckpt, bool with_ckpt, int p, size_t rows,
                         size_t hidden, size_t group, float eps, int dtype, int wdtype, void* stream) {
  size_t bytes, cbytes;
  coll_status_t st = check_ln_shape(p, rows, hidden, group, with_ckpt, dtype, wdtype, &bytes, &cbytes);
  if (st != COLL_OK) return st;
  if (!(eps >= 0.0f) || eps > 3e38f) return COLL_ERR_INVALID_ARG;
  if (rows == 0) return COLL_OK;
  if (!all_non_null(x, p) || !all_non_null(y, p) || !none_or_all(gamma, p) || !none_or_all(beta, p) ||
      !none_or_all(mean, p) || !none_or_all(rstd, p) || (with_ckpt && !all_non_null(ckpt, p)))
    return COLL_ERR_INVALID_ARG;
  const size_t d = dsize(dtype), w = dsize(wdtype);
  if (!elem_aligned(x, p, d) || !elem_aligned(y, p, d) || !aligned_or_none(gamma, p, w) || !aligned_or_none(beta, p, w) ||
      !aligned_or_none(mean, p, 4) || !aligned_or_none(rstd, p, 4) || (with_ckpt && !elem_aligned(ckpt, p, 16)))
    return COLL_ERR_INVALID_ARG;
  RangeSet rs;
  rs.add_in_place(x, y, p, bytes);
  rs.add_all(gamma, p, hidden * w, false);
  rs.add_all(beta, p, hidden * w, false);
  rs.add_all(mean, p, rows * 4, true);
  rs.add_all(rstd, p, rows * 4, true);
  if (with_ckpt) rs.add_all(ckpt, p, cbytes, true);
  st = rs.check();
  if (st != COLL_OK) return st;
  if (with_ckpt && !coll::ln_forward_keeps(dtype, hidden, group)) {
    // a group wider than the lanes that layer norm gives a row's unit: the
    // checkpoint is written on its own, and first (y may be x)
    st = run_ckpt8(coll::kCkpt8Save, x, nullptr, nullptr, ckpt, p, rows, hidden, hidden, group, dtype, stream);
    if (st != COLL_OK) return st;
    with_ckpt = false;
  }
  for (int r0 = 0; r0 < p; r0 += coll::kArgRanks) {
    const int n = std::min(p - r0, coll::kArgRanks);
    coll::LnArgs a{};
    for (int r = 0; r < n; ++r) {
      a.x[r] = x[r0 + r];
      a.y[r] = y[r0 + r];
      if (gamma) a.gamma[r] = gamma[r0 + r];
      if (beta) a.beta[r] = beta[r0 + r];
      if (mean) a.mean[r] = mean[r0 + r];
      if (rstd) a.rstd[r] = rstd[r0 + r];
      if (with_ckpt) a.ckpt[r] = (uint8_t*)ckpt[r0 + r];
    }
    a.rows = rows;
    a.hidden = hidden;
    a.ranks = n;
    a.eps = eps;
    if (with_ckpt) {
      a.row_bytes = fp8_row_bytes(hidden, group);
      a.glog = group_log(group);
    }
    const int e = coll::launch_ln_forward(dtype, wdtype, a, with_ckpt, stream);
    if (e) return hip_fail(e);
  }
  return COLL_OK;
}

int ln_launches(int p) { return (p + coll::kArgRanks - 1) / coll::kArgRanks; }
size_t ln_workspace(int p, size_t rows, size_t hidden) {
  return (size_t)ln_launches(p) * coll::ln_backward_groups(p, rows, hidden) * 2 * hidden * sizeof(float);
}

coll_status_t ln_backward(const void* const* dy, const void* const* x, bool from_ckpt, const float* const* mean,
                          const float* const* rstd, const void* const* gamma, const void* const* beta, void* const* dx,
                          void* const* y, void* const* dgamma, void* const* dbeta, int p, size_t rows, size_t hidden,
                          size_t group, int op, int dtype, int wdtype, void* workspace, size_t workspace_bytes,
                          void* stream) {
  size_t bytes, cbytes;
  coll_status_t st = check_ln_shape(p, rows, hidden, group, from_ckpt, dtype, wdtype, &bytes, &cbytes);
  if (st != COLL_OK) return st;
  if (!op_ok(op)) return COLL_ERR_INVALID_ARG;
  if (op != COLL_SUM && op != COLL_AVG) return COLL_ERR_UNSUPPORTED;
  const size_t d = dsize(dtype), w = dsize(wdtype);
  if (!none_or_all(dgamma, p) || !none_or_all(dbeta, p) || !aligned_or_none(dgamma, p, w) || !aligned_or_none(dbeta, p, w))
    return COLL_ERR_INVALID_ARG;
  RangeSet rs;
  rs.add_all(dgamma, p, hidden * w, true);
  rs.add_all(dbeta, p, hidden * w, true);
  if (rows > 0) {
    if (!all_non_null(dy, p) || !all_non_null(x, p) || !all_non_null(mean, p) || !all_non_null(rstd, p) ||
        !all_non_null(dx, p) || !none_or_all(gamma, p) || !none_or_all(beta, p) || !none_or_all(y, p))
      return COLL_ERR_INVALID_ARG;
    if (!elem_aligned(dy, p, d) || !elem_aligned(x, p, from_ckpt ? 16 : d) || !elem_aligned(mean, p, 4) ||
        !elem_aligned(rstd, p, 4) || !elem_aligned(dx, p, d) || !aligned_or_none(gamma, p, w) ||
        !aligned_or_none(beta, p, w) || !aligned_or_none(y, p, d))
      return COLL_ERR_INVALID_ARG;
    const size_t need = ln_workspace(p, rows, hidden);
    if (!workspace || !elem_aligned1(workspace, 16) || workspace_bytes < need) return COLL_ERR_INVALID_ARG;
    rs.add(workspace, need, true);
    rs.add_in_place(dy, dx, p, bytes);
    rs.add_all(x, p, from_ckpt ? cbytes : bytes, false);
    rs.add_all(mean, p, rows * 4, false);
    rs.add_all(rstd, p, rows * 4, false);
    rs.add_all(gamma, p, hidden * w, false);
    rs.add_all(beta, p, hidden * w, false);
    rs.add_all(y, p, bytes, true);
  }
  st = rs.check();
  if (st != COLL_OK) return st;
  const uint32_t groups = coll::ln_backward_groups(p, rows, hidden);
  for (int r0 = 0; rows > 0 && r0 < p; r0 += coll::kArgRanks) {
    const int n = std::min(p - r0, coll::kArgRanks);
    coll::LnArgs a{};
    for (int r = 0; r < n; ++r) {
      a.x[r] = x[r0 + r];
      a.dy[r] = dy[r0 + r];
      a.mean[r] = const_cast<float*>(mean[r0 + r]);
      a.rstd[r] = const_cast<float*>(rstd[r0 + r]);
      a.dx[r] = dx[r0 + r];
      if (gamma) a.gamma[r] = gamma[r0 + r];
      if (beta) a.beta[r] = beta[r0 + r];
      if (y) a.y[r] = y[r0 + r];
    }
    a.ws = (float*)workspace + (size_t)(r0 / coll::kArgRanks) * groups * 2 * hidden;
    a.rows = rows;
    a.hidden = hidden;
    a.ranks = n;
    if (from_ckpt) {
      a.row_bytes = fp8_row_bytes(hidden, group);
      a.glog = group_log(group);
    }
    const int e = coll::launch_ln_backward(dtype, wdtype, a, groups, from_ckpt, stream);
    if (e) return hip_fail(e);
  }
  if (!dgamma && !dbeta) return COLL_OK;
  coll::LnJoinArgs j{};
  for (int r = 0; r < p; ++r) {
    if (dgamma) j.dgamma[r] = dgamma[r];
    if (dbeta) j.dbeta[r] = dbeta[r];
  }
  j.ws = (const float*)workspace;
  j.hidden = hidden;
  j.parts = rows ? (uint32_t)ln_launches(p) * groups : 0;  // no rows: the sums are zero
  j.p = p;
  j.avg = op == COLL_AVG;
  return finish(coll::launch_ln_join(wdtype, j, stream));
}

// Shards of a vocabulary: sizes, strides and the first index of each.
coll_status_t check_shards(const void* const* logits, const int64_t* ld, const int64_t* vocab, int p, size_t rows,
                           size_t d, int64_t (&first)[kMaxRanks + 1]) {
  if (!ld || !vocab) return COLL_ERR_INVALID_ARG;
  size_t t;
  if (!mul_ok(rows, 4 * coll::kMaxTop, 1, &t)) return COLL_ERR_INVALID_ARG;  // the widest of the arrays by row
  first[0] = 0;
  for (int r = 0; r < p; ++r) {
    if (vocab[r] < 0 || ld[r] < vocab[r] || vocab[r] > 0x7fffffffll) return COLL_ERR_INVALID_ARG;
    first[r + 1] = first[r] + vocab[r];
    if (!mul_ok((size_t)ld[r], rows, d, &t)) return COLL_ERR_INVALID_ARG;
  }
  if (first[p] < 1) return COLL_ERR_INVALID_ARG;
  if (first[p] > 0x7fffffffll) return COLL_ERR_UNSUPPORTED;  // indices are int32
  if (rows == 0) return COLL_OK;
  if (!logits) return COLL_ERR_INVALID_ARG;
  for (int r = 0; r < p; ++r)
    if (vocab[r] && (!logits[r] || (uintptr_t)logits[r] % d)) return COLL_ERR_INVALID_ARG;
  return COLL_OK;
}
// `rows` runs of `width` bytes, `stride` apart.  Two blocks of one stride
// whose address ranges cross (column slices of one matrix) overlap only if
// their columns do; of unlike strides, they count as overlapping.
struct Block {
  uintptr_t at;
  size_t rows, stride, width;
  uintptr_t end() const { return at + (rows - 1) * stride + width; }
};
bool blocks_overlap(const Block& a, const Block& b) {
  if (!a.width || !b.width || a.at >= b.end() || b.at >= a.end()) return false;
  if (a.stride != b.stride) return true;
  const Block &lo = a.at <= b.at ? a : b, &hi = a.at <= b.at ? b : a;
  const size_t off = (hi.at - lo.at) % lo.stride;
  return off < lo.width || off + hi.width > lo.stride;
}
size_t shard_bytes(size_t rows, int64_t ld, int64_t vocab, size_t d) {
  return vocab ? ((rows - 1) * (size_t)ld + (size_t)vocab) * d : 0;
}

// Workspace bytes of one call with so many rows.
bool logprob_need(int p, size_t rows, const int64_t* vocab, int top_k, size_t* bytes) {
  coll::LogprobPlan plan;
  coll::logprob_plan(p, rows, vocab, &plan);
  return mul_ok(rows, (size_t)plan.pieces, coll::logprob_piece_bytes(plan, top_k), bytes);
}

}  // namespace

COLL_EXPORT coll_status_t coll_layernorm(const void* const* x, const void* const* gamma, const void* const* beta,
                                         void* const* y, float* const* mean, float* const* rstd, int p, size_t rows,
                                         size_t hidden, float eps, coll_dtype_t dtype, coll_dtype_t wdtype, void* stream) {
  return ln_forward(x, gamma, beta, y, mean, rstd, nullptr, false, p, rows, hidden, 0, eps, dtype, wdtype, stream);
}

COLL_EXPORT coll_status_t coll_layernorm_ckpt8(const void* const* x, const void* const* gamma, const void* const* beta,
                                               void* const* y, float* const* mean, float* const* rstd, void* const* ckpt,
                                               int p, size_t rows, size_t hidden, size_t group, float eps,
                                               coll_dtype_t dtype, coll_dtype_t wdtype, void* stream) {
  return ln_forward(x, gamma, beta, y, mean, rstd, ckpt, true, p, rows, hidden, group, eps, dtype, wdtype, stream);
}

COLL_EXPORT size_t coll_layernorm_workspace_bytes(int p, size_t rows, size_t hidden) {
  size_t t;
  if (p < 1 || p > kMaxRanks || hidden == 0 || hidden >= (size_t{1} << 31) || !mul_ok(rows, hidden, 4 * (size_t)kMaxRanks, &t))
    return 0;
  return ln_workspace(p, rows, hidden);
}

COLL_EXPORT coll_status_t coll_layernorm_backward(const void* const* dy, const void* const* x, const float* const* mean,
                                                  const float* const* rstd, const void* const* gamma, void* const* dx,
                                                  void* const* dgamma, void* const* dbeta, int p, size_t rows,
                                                  size_t hidden, coll_op_t op, coll_dtype_t dtype, coll_dtype_t wdtype,
                                                  void* workspace, size_t workspace_bytes, void* stream) {
  return ln_backward(dy, x, false, mean, rstd, gamma, nullptr, dx, nullptr, dgamma, dbeta, p, rows, hidden, 0, op, dtype,
                     wdtype, workspace, workspace_bytes, stream);
}

COLL_EXPORT coll_status_t coll_layernorm_backward_ckpt8(const void* const* dy, const void* const* ckpt,
                                                        const float* const* mean, const float* const* rstd,
                                                        const void* const* gamma, const void* const* beta,
                                                        void* const* dx, void* const* y, void* const* dgamma,
                                                        void* const* dbeta, int p, size_t rows, size_t hidden,
                                                        size_t group, coll_op_t op, coll_dtype_t dtype,
                                                        coll_dtype_t wdtype, void* workspace, size_t workspace_bytes,
                                                        void* stream) {
  return ln_backward(dy, ckpt, true, mean, rstd, gamma, beta, dx, y, dgamma, dbeta, p, rows, hidden, group, op, dtype,
                     wdtype, workspace, workspace_bytes, stream);
}

COLL_EXPORT size_t coll_ckpt8_row_bytes(size_t hidden, size_t group) {
  return ckpt8_shape(hidden, group) == COLL_OK ? fp8_row_bytes(hidden, group) : 0;
}

COLL_EXPORT coll_status_t coll_ckpt8_save(const void* const* x, void* const* ckpt, int p, size_t rows, size_t hidden,
                                          size_t group, coll_dtype_t dtype, void* stream) {
  size_t bytes, cbytes;
  coll_status_t st = check_ln_shape(p, rows, hidden, group, true, dtype, COLL_F32, &bytes, &cbytes);
  if (st != COLL_OK || rows == 0) return st;
  if (!all_non_null(x, p) || !all_non_null(ckpt, p) || !elem_aligned(x, p, dsize(dtype)) || !elem_aligned(ckpt, p, 16))
    return COLL_ERR_INVALID_ARG;
  RangeSet rs;
  rs.add_all(x, p, bytes, false);
  rs.add_all(ckpt, p, cbytes, true);
  st = rs.check();
  if (st != COLL_OK) return st;
  return run_ckpt8(coll::kCkpt8Save, x, nullptr, nullptr, ckpt, p, rows, hidden, hidden, group, dtype, stream);
}

COLL_EXPORT coll_status_t coll_ckpt8_load(const void* const* ckpt, void* const* x, int p, size_t rows, size_t hidden,
                                          size_t group, coll_dtype_t dtype, void* stream) {
  size_t bytes, cbytes;
  coll_status_t st = check_ln_shape(p, rows, hidden, group, true, dtype, COLL_F32, &bytes, &cbytes);
  if (st != COLL_OK || rows == 0) return st;
  if (!all_non_null(x, p) || !all_non_null(ckpt, p) || !elem_aligned(x, p, dsize(dtype)) || !elem_aligned(ckpt, p, 16))
    return COLL_ERR_INVALID_ARG;
  RangeSet rs;
  rs.add_all(ckpt, p, cbytes, false);
  rs.add_all(x, p, bytes, true);
  st = rs.check();
  if (st != COLL_OK) return st;
  return run_ckpt8(coll::kCkpt8Load, nullptr, x, nullptr, const_cast<void* const*>(ckpt), p, rows, hidden, hidden,
                   group, dtype, stream);
}

COLL_EXPORT coll_status_t coll_swiglu_ckpt8(const void* const* gate_up, void* const* out, void* const* ckpt, int p,
                                            size_t rows, size_t ffn, size_t group, coll_dtype_t dtype, void* stream) {
  if (ffn == 0 || group == 0 || ffn % group) return COLL_ERR_INVALID_ARG;
  if (ffn >= (size_t{1} << 30)) return COLL_ERR_UNSUPPORTED;
  size_t bytes, cbytes;
  coll_status_t st = check_ln_shape(p, rows, 2 * ffn, group, true, dtype, COLL_F32, &bytes, &cbytes);
  if (st != COLL_OK || rows == 0) return st;
  const size_t d = dsize(dtype);
  if (!all_non_null(gate_up, p) || !all_non_null(out, p) || !all_non_null(ckpt, p) || !elem_aligned(gate_up, p, d) ||
      !elem_aligned(out, p, d) || !elem_aligned(ckpt, p, 16))
    return COLL_ERR_INVALID_ARG;
  RangeSet rs;
  rs.add_all(gate_up, p, bytes, false);
  rs.add_all(out, p, bytes / 2, true);
  rs.add_all(ckpt, p, cbytes, true);
  st = rs.check();
  if (st != COLL_OK) return st;
  return run_ckpt8(coll::kSwigluForward, gate_up, out, nullptr, ckpt, p, rows, 2 * ffn, ffn, group, dtype, stream);
}

COLL_EXPORT coll_status_t coll_swiglu_backward_ckpt8(const void* const* ckpt, const void* const* dout,
                                                     void* const* dgate_up, void* const* out, int p, size_t rows,
                                                     size_t ffn, size_t group, coll_dtype_t dtype, void* stream) {
  if (ffn == 0 || group == 0 || ffn % group) return COLL_ERR_INVALID_ARG;
  if (ffn >= (size_t{1} << 30)) return COLL_ERR_UNSUPPORTED;
  size_t bytes, cbytes;
  coll_status_t st = check_ln_shape(p, rows, 2 * ffn, group, true, dtype, COLL_F32, &bytes, &cbytes);
  if (st != COLL_OK || rows == 0) return st;
  const size_t d = dsize(dtype);
  if (!all_non_null(ckpt, p) || !all_non_null(dout, p) || !all_non_null(dgate_up, p) || !none_or_all(out, p) ||
      !elem_aligned(ckpt, p, 16) || !elem_aligned(dout, p, d) || !elem_aligned(dgate_up, p, d) || !aligned_or_none(out, p, d))
    return COLL_ERR_INVALID_ARG;
  RangeSet rs;
  rs.add_all(ckpt, p, cbytes, false);
  rs.add_all(dout, p, bytes / 2, false);
  rs.add_all(dgate_up, p, bytes, true);
  rs.add_all(out, p, bytes / 2, true);
  st = rs.check();
  if (st != COLL_OK) return st;
  return run_ckpt8(coll::kSwigluBackward, dout, dgate_up, out, const_cast<void* const*>(ckpt), p, rows, 2 * ffn, ffn,
                   group, dtype, stream);
}

COLL_EXPORT size_t coll_vocab_logprob_workspace_bytes(int p, size_t rows, const int64_t* vocab, int top_k) {
  if (p < 1 || p > kMaxRanks || !vocab || top_k < 0 || top_k > coll::kMaxTop) return 0;
  for (int r = 0; r < p; ++r)
    if (vocab[r] < 0 || vocab[r] > 0x7fffffffll) return 0;
  // Fewer rows are cut into more pieces, which may take more: the most that
  // any number of rows up to this one needs.  It grows with the rows as long
  // as these want one number of pieces, so the last of each such run decides.
  size_t most;
  if (!logprob_need(p, rows, vocab, top_k, &most)) return 0;
  for (uint64_t want = 2; want <= coll::kMaxPieces; ++want) {
    const uint64_t last = coll::logprob_most_rows(p, want);
    size_t bytes;
    if (last < rows && logprob_need(p, last, vocab, top_k, &bytes)) most = std::max(most, bytes);
  }
  return most;
}

COLL_EXPORT coll_status_t coll_vocab_logprob(const void* const* logits, const int64_t* ld, const int64_t* vocab,
                                             const int64_t* targets, float inv_temp, float* const* stats,
                                             float* const* logp, float* const* entropy, int top_k,
                                             float* const* top_logp, int32_t* const* top_idx, int p, size_t rows,
                                             coll_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (p < 1 || p > kMaxRanks || top_k < 0 || !(inv_temp > 0.0f) || inv_temp > 1e30f) return COLL_ERR_INVALID_ARG;
  if (top_k > coll::kMaxTop) return COLL_ERR_UNSUPPORTED;
  coll_status_t st = float_dtype(dtype);
  if (st != COLL_OK) return st;
  const size_t d = dsize(dtype);
  coll::LogprobArgs a{};
  st = check_shards(logits, ld, vocab, p, rows, d, a.first_index);
  if (st != COLL_OK || rows == 0) return st;
  if (!targets || !elem_aligned1(targets, 8) || !all_non_null(stats, p) || !all_non_null(logp, p) ||
      !none_or_all(entropy, p) || !elem_aligned(stats, p, 4) || !elem_aligned(logp, p, 4) || !aligned_or_none(entropy, p, 4))
    return COLL_ERR_INVALID_ARG;
  if (top_k && (!all_non_null(top_logp, p) || !all_non_null(top_idx, p) || !elem_aligned(top_logp, p, 4) ||
                !elem_aligned(top_idx, p, 4)))
    return COLL_ERR_INVALID_ARG;
  coll::logprob_plan(p, rows, vocab, &a.plan);
  size_t need;
  if (!mul_ok(rows, (size_t)a.plan.pieces, coll::logprob_piece_bytes(a.plan, top_k), &need)) return COLL_ERR_INVALID_ARG;
  if (!workspace || !elem_aligned1(workspace, 16) || workspace_bytes < need) return COLL_ERR_INVALID_ARG;
  RangeSet rs;
  for (int r = 0; r < p; ++r) rs.add(logits[r], shard_bytes(rows, ld[r], vocab[r], d), false);
  rs.add(targets, rows * 8, false);
  rs.add(workspace, need, true);
  rs.add_all(stats, p, rows * 8, true);
  rs.add_all(logp, p, rows * 4, true);
  rs.add_all(entropy, p, rows * 4, true);
  if (top_k) {
    rs.add_all(top_logp, p, rows * 4 * (size_t)top_k, true);
    rs.add_all(top_idx, p, rows * 4 * (size_t)top_k, true);
  }
  st = rs.check();
  if (st != COLL_OK) return st;
  coll::LogprobJoinArgs j{};
  for (int r = 0; r < p; ++r) {
    a.logits[r] = logits[r];
    a.ld[r] = ld[r];
    j.stats[r] = stats[r];
    j.logp[r] = logp[r];
    if (entropy) j.entropy[r] = entropy[r];
    if (top_k) {
      j.top_logp[r] = top_logp[r];
      j.top_idx[r] = top_idx[r];
    }
  }
  a.targets = targets;
  a.part = (float*)workspace;
  a.places = (uint32_t*)((char*)workspace + rows * (size_t)a.plan.pieces * 16);
  a.bests = (float*)((char*)workspace + rows * (size_t)a.plan.pieces * 32);
  a.rows = rows;
  a.scale = inv_temp;
  a.p = p;
  a.top = top_k;
  return finish(coll::launch_logprob(dtype, a, j, stream));
}

COLL_EXPORT coll_status_t coll_vocab_logprob_backward(const void* const* logits, const int64_t* ld, const int64_t* vocab,
                                                      const int64_t* targets, float inv_temp, const float* stats,
                                                      const float* dlogp, const float* entropy, const float* dentropy,
                                                      void* const* dlogits, const int64_t* dld, int p, size_t rows,
                                                      coll_dtype_t dtype, void* stream) {
  if (p < 1 || p > kMaxRanks || !(inv_temp > 0.0f) || inv_temp > 1e30f) return COLL_ERR_INVALID_ARG;
  coll_status_t st = float_dtype(dtype);
  if (st != COLL_OK) return st;
  const size_t d = dsize(dtype);
  coll::LogprobGradArgs a{};
  st = check_shards(logits, ld, vocab, p, rows, d, a.first_index);
  if (st == COLL_OK) st = check_shards((const void* const*)dlogits, dld, vocab, p, rows, d, a.first_index);
  if (st != COLL_OK || rows == 0) return st;
  if (!targets || !elem_aligned1(targets, 8) || !stats || !elem_aligned1(stats, 4) || !dlogp || !elem_aligned1(dlogp, 4))
    return COLL_ERR_INVALID_ARG;
  if (dentropy && (!entropy || !elem_aligned1(entropy, 4) || !elem_aligned1(dentropy, 4))) return COLL_ERR_INVALID_ARG;
  const void* small[5] = {targets, stats, dlogp, dentropy ? entropy : nullptr, dentropy};
  const size_t small_bytes[5] = {rows * 8, rows * 8, rows * 4, rows * 4, rows * 4};
  for (int r = 0; r < p; ++r) {
    const Block out{(uintptr_t)dlogits[r], rows, (size_t)dld[r] * d, (size_t)vocab[r] * d};
    for (int k = 0; k < 5; ++k)
      if (small[k] && blocks_overlap(out, Block{(uintptr_t)small[k], 1, small_bytes[k], small_bytes[k]})) return COLL_ERR_ALIAS;
    for (int s = 0; s < p; ++s) {
      const Block in{(uintptr_t)logits[s], rows, (size_t)ld[s] * d, (size_t)vocab[s] * d};
      const bool in_place = s == r && in.at == out.at && in.stride == out.stride;
      if (!in_place && blocks_overlap(out, in)) return COLL_ERR_ALIAS;
      const Block other{(uintptr_t)dlogits[s], rows, (size_t)dld[s] * d, (size_t)vocab[s] * d};
      if (s < r && blocks_overlap(out, other)) return COLL_ERR_ALIAS;
    }
  }
  for (int r = 0; r < p; ++r) {
    a.logits[r] = logits[r];
    a.dlogits[r] = dlogits[r];
    a.ld[r] = ld[r];
    a.dld[r] = dld[r];
  }
  a.targets = targets;
  a.stats = stats;
  a.dlogp = dlogp;
  a.entropy = entropy;
  a.dentropy = dentropy;
  a.rows = rows;
  a.scale = inv_temp;
  a.p = p;
  return finish(coll::launch_logprob_backward(dtype, a, stream));
}
