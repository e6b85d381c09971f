"""Distillation over a sharded vocabulary on the GPU against the float64
oracle.  Tolerances as in test_gpu_token_ops: U is half a step of fp32, HALF of
the result's type."""
import numpy as np
import pytest

from gpu_util import BF16, F32
from oracle import token_ops
from test_gpu_token_ops import HALF, LP_SHAPES, TINY, U, close, coll, dev, f32, host, rng, shards, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


def entries(g, z, k, t, odd=True):
    """A teacher near z (all of whose masked entries it masks too): k entries in any order, fp32 log probabilities;
    where odd, some of them absent, listed twice or of no mass."""
    rows, v = z.shape
    with np.errstate(invalid="ignore", divide="ignore"):
        w = (np.where(np.isfinite(z), z, -np.inf) + g.normal(0, 0.7, z.shape)) * t
        w -= w.max(1, keepdims=True)
        w -= np.log(np.exp(w).sum(1, keepdims=True))
    idx = np.argsort(-w, 1, kind="stable")[:, :k]
    logp = np.take_along_axis(w, idx, 1)
    if idx.shape[1] < k:                                      # a vocabulary of fewer entries
        idx = np.concatenate([idx, np.full((rows, k - v), -1)], 1)
        logp = np.concatenate([logp, np.full((rows, k - v), -np.inf)], 1)
    order = g.permuted(np.tile(np.arange(k), (rows, 1)), axis=1)
    idx, logp = np.take_along_axis(idx, order, 1).astype(np.int32), np.take_along_axis(logp, order, 1).astype(np.float32)
    if odd:
        for i in range(rows):
            if i % 3 == 1 and k > 2:
                idx[i, g.integers(k)] = idx[i, g.integers(k)]     # twice (or itself)
                idx[i, g.integers(k)] = g.choice([-1, v, 0x7fffffff, -2 ** 31])
            if i % 4 == 2 and k > 1:
                logp[i, g.integers(k)] = -np.inf
    return idx, logp


def run(coll, zs, idx, logp, t, tail):
    import torch
    p, (rows, k) = len(zs), idx.shape
    i, l = torch.from_numpy(idx).cuda(), torch.from_numpy(logp).cuda()
    o = {"stats": f32(p, rows, 4), "loss": f32(p, rows)}
    ws = workspace(coll.coll_vocab_distill_workspace_bytes(rows, [z.shape[1] for z in zs], k))
    coll.coll_vocab_distill(zs, i, l, list(o["stats"]), list(o["loss"]), ws, kind=int(tail), inv_temp=t)
    torch.cuda.synchronize()
    return o, i, l


def parts(e, tail):
    """What the tolerances are made of: the exponents' sizes and the probabilities, of rows with finite statistics."""
    d = np.where(np.isfinite(e["d"]), e["d"], 0.0)
    s = np.where(np.isfinite(e["stats"]), e["stats"], 0.0)
    prob = np.where(np.isfinite(e["d"]), np.exp(d - s[:, 1:2]), 0.0)
    # the sum that is taken in fp32: of the entries that are not listed, about their own maximum, or of all
    out = np.where(np.isfinite(e["d"]) & ~(e["among"] & tail), np.exp(d), 0.0)
    top = np.where(out > 0, d, -np.inf).max(1, initial=-np.inf, keepdims=True)
    far = np.where(out > 0, np.abs(d - np.where(np.isfinite(top), top, 0.0)), 0.0)
    size = np.where(out.sum(1) > 0, (out * far).sum(1) / np.maximum(out.sum(1), 1e-300), 0.0)
    # a term's exponent is off by 3 |d| U, the term by 4 U more; chains of at most 16 chunks, 12 in a chunk, 12 over lanes
    return d, s, prob, U * (3 * size + 4 + 64)


def check(o, e, tail):
    d, s, prob, off = parts(e, tail)
    p0 = np.exp(np.where(np.isfinite(e["stats"][:, 2]), s[:, 2] - s[:, 1], -800.0)) if tail else np.ones(len(d))
    whole, rest = np.maximum(1.0, 1.0 - s[:, 3]), np.maximum(s[:, 3], 0.0)
    # by the log of that sum the loss changes by p_0 max(1, sum q) - q_0, or by 1
    by = np.abs(whole * p0 - rest) if tail else 1.0
    same = {n: all((x[0].cpu().numpy().view(np.uint32) == y.cpu().numpy().view(np.uint32)).all() for y in x[1:]) for n, x in o.items()}
    assert same == {n: True for n in o}                       # the same bits on every rank
    for r in range(o["loss"].shape[0]):
        got = host(o["stats"][r])
        close(got[:, 0], e["stats"][:, 0], 0.0, "max")
        close(got[:, 1], e["stats"][:, 1], p0 * off + 2 * U * np.abs(s[:, 1]), "log sum")
        close(got[:, 2], e["stats"][:, 2], (off if tail else 0.0) + 2 * U * np.abs(s[:, 2]) + 1e-13, "third")
        close(got[:, 3], e["stats"][:, 3], 2 * U * np.abs(s[:, 3]) + 1e-13, "fourth")
        # 64-bit sums of at most 128 terms of a size below 1000 (1e-13 each), and the result's rounding
        close(host(o["loss"][r]), e["loss"], by * off + 2 * U * np.abs(np.where(np.isfinite(e["loss"]), e["loss"], 0.0)) + 1e-11, "loss")


def grad_and_check(coll, zs, ze, idx, logp, i, l, t, tail, dtype, seed, place="apart"):
    """Gradient from the oracle's statistics in fp32, written apart, to column slices of one matrix, or in place."""
    import torch
    rows, v = ze.shape
    e = token_ops.distill(ze, idx, logp.astype(np.float64), t, tail)
    st, ste = dev(e["stats"], F32)
    gl, gle = dev(rng(61, seed).normal(0, 1, rows), F32)
    widths = [z.shape[1] for z in zs]
    cuts = np.cumsum([0, *widths])
    if place == "slices":
        full = torch.full((rows, v + 3), float("nan"), dtype=zs[0].dtype, device="cuda")
        dz = [full[:, a:b] for a, b in zip(cuts, cuts[1:])]
    elif place == "in place":
        dz = zs
    else:
        dz = [torch.full((rows, w), float("nan"), dtype=zs[0].dtype, device="cuda") for w in widths]
    coll.coll_vocab_distill_backward(zs, i, l, st, gl, dz, kind=int(tail), inv_temp=t)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore", over="ignore"):
        want = token_ops.distill_backward(ze, e["among"], e["q"], t, ste, gle, tail)
    s = np.where(np.isfinite(ste), ste, 0.0)
    d = np.where(np.isfinite(e["d"]), e["d"], 0.0)
    ls, third, fourth = s[:, 1:2], s[:, 2:3], s[:, 3:4]
    prob = np.where(np.isfinite(e["d"]), np.exp(d - ls), 0.0)
    g = np.abs(gle)[:, None] * t
    q = np.where(np.isfinite(e["q"]), e["q"], 0.0)
    lq = np.abs(np.log(np.maximum(q, 1e-300))) * (q > 0)
    whole = np.maximum(1.0, np.abs(1.0 - fourth)) if tail else 1.0
    # exponents: 3 |d| U and 3 of the shift's, the exponential 4 U, and some products
    lim = whole * prob * (4 * np.abs(d) + 4 * np.abs(ls) + 12) * U + q * (4 * lq + (0 if tail else 6) * np.abs(third) + 12) * U
    if tail:
        have = np.isfinite(ste[:, 2:3])
        p0 = np.where(have, np.exp(np.minimum(third - ls, 0.0)), 0.0)
        share = np.where(have & np.isfinite(e["d"]), np.exp(np.minimum(d - third, 0.0)), 0.0)
        factor = np.abs(whole * p0 - np.maximum(fourth, 0.0))
        others = share * (factor * (4 * np.abs(d) + 4 * np.abs(third) + 12) * U
                          + whole * p0 * (4 * np.abs(third) + 4 * np.abs(ls) + 12) * U + np.abs(fourth) * 2 * U)
        lim = np.where(e["among"], lim, others)
    got = np.concatenate([host(x) for x in dz], 1)
    close(got, want, HALF[dtype] * np.abs(np.where(np.isfinite(want), want, 0.0)) + g * lim + TINY * 10, "dlogits")
    if place == "slices":
        assert torch.isnan(full[:, v:].float()).all()


CASES = [(*s[:6], k) for s in LP_SHAPES for k in (1, 7, 64, 65, 128) if s[0] <= 1000 or k in (7, 128)]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("rows,cuts,dtype,pad,off,t,k", CASES)
def test_distillation_and_gradient(coll, rows, cuts, dtype, pad, off, t, k, tail):
    g = rng(60, rows, len(cuts), cuts[-1], dtype, k, tail)
    zs, ze = shards(g.normal(0, 3, (rows, cuts[-1])), cuts, dtype, pad, off)
    t = float(np.float32(t))
    idx, logp = entries(g, ze, k, t)
    o, i, l = run(coll, zs, idx, logp, t, tail)
    check(o, token_ops.distill(ze, idx, logp.astype(np.float64), t, tail), tail)
    for place in ("apart", "slices", "in place"):
        grad_and_check(coll, zs, ze, idx, logp, i, l, t, tail, dtype, cuts[-1], place)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("v,p", [(40, 1), (3000, 3), (9000, 1), (70000, 2)])
def test_masked_rows_and_edge_values(coll, dtype, v, p, tail):
    g = rng(62, v, p, dtype, tail)
    k, inf = 9, np.inf
    z = g.normal(0, 3, (20, v))
    low = {F32: np.finfo(np.float32).min, BF16: -3.3895313892515355e38}[dtype]
    z[0] = -inf                                               # nothing is allowed
    z[1, 5:] = -inf                                           # fewer are allowed than listed: no others
    z[2, v // 2] = np.nan
    z[3, 1] = inf
    z[4] = np.nan                                             # padding, whatever it holds
    z[5] = -inf
    z[9, g.permutation(v)[:v * 9 // 10]] = -inf
    z[12] = low
    z[13] = low
    z[13, [2, v - 2]] = [1.0, 2.0]                            # masked by the lowest value
    z[14] = 1e4 + np.arange(v) % 7                            # large logits
    z[15, :9] += 300.0                                        # the entries hold it all: p_0 underflows
    z[16] = np.where(np.arange(v) < 9, -300.0, z[16])         # the entries hold nothing
    z[18] = inf                                               # padding
    idx, logp = entries(g, np.where(np.isfinite(z), z, -5.0), k, 1.0, odd=False)
    idx[1], logp[1] = [4, 3, 2, 1, 0, -1, -1, v, -7], np.float32(np.log([0.1, 0.2, 0.3, 0.3, 0.1, 0.5, 0.5, 0.5, 0.5]))
    idx[4], idx[5], idx[18] = -1, v, -2
    logp[6] = -inf                                            # no mass on any entry
    logp[7] += 1.0                                            # masses above 1
    logp[8, 3] = np.nan
    idx[9, 0], logp[9, 0] = int(np.flatnonzero(np.isneginf(z[9]))[0]), -1.0          # mass where the student has none
    idx[10] = idx[10, 0]                                      # one entry, listed nine times
    logp[11, 2] = inf
    idx[15], idx[16] = np.arange(9), np.arange(9)
    logp[16] = np.float32(-30.0)
    idx[17, :8], logp[17, :8] = -1, -inf                      # one entry is left
    cuts = [v * r // p for r in range(p + 1)]
    zs, ze = shards(z, cuts, dtype, 0, 1)
    for t in (1.0, 0.5):
        o, i, l = run(coll, zs, idx, logp, t, tail)
        with np.errstate(invalid="ignore"):
            e = token_ops.distill(ze, idx, logp.astype(np.float64), t, tail)
        assert e["loss"][0] == inf and (e["loss"][[4, 5, 18]] == 0).all() and e["loss"][9] == inf and np.isfinite(e["loss"][1])
        check(o, e, tail)
        grad_and_check(coll, zs, ze, idx, logp, i, l, t, tail, dtype, v)


def test_gradient_by_differences(coll):
    """Against central differences of the kernel's own forward pass (fp32, two shards)."""
    g = rng(63)
    v, rows, t, k = 45, 3, 0.75, 6
    z = g.normal(0, 2, (rows, v)).astype(np.float32)
    gl = g.normal(0, 1, rows).astype(np.float32)
    for tail in (False, True):
        idx, logp = entries(g, z, k, t)
        loss = lambda z: (host(run(coll, shards(z, [0, 21, v], F32)[0], idx, logp, t, tail)[0]["loss"][1]) * gl).sum()  # noqa: E731
        zs, _ = shards(z, [0, 21, v], F32)
        o, i, l = run(coll, zs, idx, logp, t, tail)
        dz = [x.clone() for x in zs]
        coll.coll_vocab_distill_backward(zs, i, l, o["stats"][0], dev(gl, F32)[0], dz, kind=int(tail), inv_temp=t)
        got = np.concatenate([host(x) for x in dz], 1)
        # h^2 / 6 times third derivatives (below 4 for these sizes), and 3 results of up to 8, off by 100 U each
        h = 2.0 ** -6
        lim = h * h * 4 + 3 * 8 * 100 * U / (2 * h)
        for r in range(rows):
            for j in {0, 20, 21, 44, *[int(x) for x in idx[r] if 0 <= x < v]}:
                a, b = z.copy(), z.copy()
                a[r, j] += np.float32(h)
                b[r, j] -= np.float32(h)
                step = float(a[r, j]) - float(b[r, j])
                assert abs((loss(a) - loss(b)) / step - got[r, j]) < lim, (tail, r, j)


def test_a_student_that_is_its_teacher(coll):
    """The teacher's entries from the log probabilities' alternatives over the same shards: no loss but rounding, and no
    gradient but the stats' rounding."""
    import torch
    g = rng(64)
    rows, v, k = 37, 5000, 20
    zs, ze = shards(g.normal(0, 2, (rows, v)), [0, 1300, v], BF16)
    tg = torch.zeros(rows, dtype=torch.int64, device="cuda")
    st, lp, tl = f32(2, rows, 2), f32(2, rows), f32(2, rows, k)
    ti = torch.zeros(2, rows, k, dtype=torch.int32, device="cuda")
    coll.coll_vocab_logprob(zs, tg, list(st), list(lp), workspace(coll.coll_vocab_logprob_workspace_bytes(rows, [1300, v - 1300], k)),
                            top_k=k, top_logp=list(tl), top_idx=list(ti))
    o = {"stats": f32(2, rows, 4), "loss": f32(2, rows)}
    coll.coll_vocab_distill(zs, ti[0], tl[1], list(o["stats"]), list(o["loss"]), workspace(coll.coll_vocab_distill_workspace_bytes(rows, [1300, v - 1300], k)))
    # log probabilities of a size of 10, off by 100 U each: the divergence is of second order in them
    assert np.abs(host(o["loss"])).max() < (1000 * U) ** 2 * 100 + 1e-9
    dz = [torch.zeros_like(z) for z in zs]
    coll.coll_vocab_distill_backward(zs, ti[0], tl[1], o["stats"][0], torch.ones(rows, device="cuda"), dz)
    prob = np.exp(ze - ze.max(1, keepdims=True))
    prob /= prob.sum(1, keepdims=True)
    # and the gradient of first order: of a probability, or of its share of p_0 - q_0
    assert (np.abs(np.concatenate([host(x) for x in dz], 1)) <= 2000 * U * np.maximum(prob, prob / (1 - np.sort(prob, 1)[:, -k:].sum(1, keepdims=True)))).all()


def test_a_workspace_for_more_rows_and_rows_of_a_longer_buffer(coll):
    """4095 rows of 6200 entries, cut into three pieces each, in the workspace of 4096, which need two each; buffers
    that hold more rows keep what is behind the last."""
    import torch
    g = rng(65)
    rows, v, k = 4095, 6200, 4
    zs, ze = shards(g.normal(0, 3, (rows, v)), [0, v], BF16)
    idx, logp = entries(g, ze, k, 1.0)
    i, l = torch.from_numpy(idx).cuda(), torch.from_numpy(logp).cuda()
    o = {"stats": f32(1, rows + 3, 4), "loss": f32(1, rows + 3)}
    ws = workspace(coll.coll_vocab_distill_workspace_bytes(rows + 1, [v], k))
    coll.coll_vocab_distill(zs, i, l, list(o["stats"]), list(o["loss"]), ws, rows=rows)
    torch.cuda.synchronize()
    e = token_ops.distill(ze, idx, logp.astype(np.float64), 1.0, True)
    check({x: y[:, :rows] for x, y in o.items()}, e, True)
    assert torch.isnan(o["stats"][:, rows:]).all() and torch.isnan(o["loss"][:, rows:]).all()


def test_rows_past_2_31_elements(coll):
    import torch
    g = rng(66)
    v, pick, k = 131072, [0, 16383, 16384, 16385, 17000], 5
    rows = pick[-1] + 1
    z = torch.zeros(rows, v, dtype=torch.bfloat16, device="cuda")
    small, ze = dev(g.normal(0, 3, (len(pick), v)), BF16)
    z[pick] = small
    ids, lps = entries(g, ze, k, 1.0)
    i, l = torch.full((rows, k), -1, dtype=torch.int32, device="cuda"), torch.zeros(rows, k, device="cuda")
    i[pick], l[pick] = torch.from_numpy(ids).cuda(), torch.from_numpy(lps).cuda()
    o = {"stats": f32(1, rows, 4), "loss": f32(1, rows)}
    coll.coll_vocab_distill([z], i, l, list(o["stats"]), list(o["loss"]), workspace(coll.coll_vocab_distill_workspace_bytes(rows, [v], k)))
    e = token_ops.distill(ze, ids, lps.astype(np.float64), 1.0, True)
    check({x: y[:, pick] for x, y in o.items()}, e, True)
    coll.coll_vocab_distill_backward([z], i, l, o["stats"][0], torch.ones(rows, device="cuda"), [z])       # in place
    want = token_ops.distill_backward(ze, e["among"], e["q"], 1.0, host(o["stats"][0])[pick], np.ones(5), True)
    s = host(o["stats"][0])[pick]
    d = ze - s[:, :1]
    lim = HALF[BF16] * np.abs(want) + 200 * U * (np.exp(d - s[:, 1:2]) + e["q"] + np.exp(np.minimum(d - s[:, 2:3], 0.0)))
    close(host(z[pick]), want, lim, "dlogits")
    z[pick] = 0
    assert not bool(z.view(torch.int16).any())                # all other rows are padding: zeros
