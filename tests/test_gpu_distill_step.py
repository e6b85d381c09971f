"""RMS norm, distillation and the adjustment of logits together: the example's
step with its gradients against autograd's in fp32 on the CPU, its texts, and
the operators on other streams, in captured graphs and as deferred calls."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

from gpu_util import BF16, F32
from oracle import token_ops
from test_gpu_adjust import Case
from test_gpu_token_ops import coll, dev, f32, new, rng, shards, u8, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "sharded_distillation.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("sharded_distillation", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("p,rows,hidden,vocab,top", [(4, 64, 256, 1000, 16), (1, 33, 128, 517, 5), (3, 7, 384, 2048, 32)])
def test_gradients_of_a_step(ex, p, rows, hidden, vocab, top, fp8):
    m = ex.ShardedDistillation(p=p, rows=rows, hidden=hidden, vocab=vocab, top=top, fp8=fp8, seed=3)
    g = torch.Generator().manual_seed(5)
    for r in range(p):  # weights that differ from ones, the same on every rank
        m.w["gamma"][r].copy_(torch.linspace(0.5, 1.5, hidden))
    tokens = [torch.randint(vocab, (rows,), generator=g) for _ in range(p)]
    loss = float(m.forward_backward([t.cuda() for t in tokens]))

    w = {k: [t.cpu().clone().requires_grad_() for t in (v if k == "out" else v[:1])] for k, v in m.w.items()}
    t = torch.cat(tokens)
    x = m.embedding.cpu().float()[t].requires_grad_()
    y = torch.nn.functional.rms_norm(x + x @ w["w"][0], (hidden,), w["gamma"][0], 1e-6)
    lp = torch.log_softmax(y @ torch.cat(w["out"], 1) / m.temp, 1)
    teacher = torch.cat([a.cpu() for a in m.teacher_logits(t.cuda())], 1).float()
    idx = torch.sort(teacher, dim=1, descending=True, stable=True).indices[:, :top]     # ties (of bf16 logits) by the lower index
    lq = torch.log_softmax(teacher / m.temp, 1).gather(1, idx)
    rest = lambda z: torch.logsumexp(z.scatter(1, idx, -math.inf), 1, keepdim=True)  # noqa: E731
    lq, lp = torch.cat([lq, rest(torch.log_softmax(teacher / m.temp, 1))], 1), torch.cat([lp.gather(1, idx), rest(lp)], 1)
    want = (lq.exp() * (lq - lp)).sum(1)
    (want.mean() * m.temp ** 2).backward()
    # logits are sums of `hidden` products of order 1 / sqrt(hidden), whose factors are off by 2^-8 (2^-4 in 8 bits) at
    # most: by 2^-8 sqrt(2) or 2^-4 of a unit on average over independent roundings
    off = 2.0 ** -4 if fp8 else 2.0 ** -7
    assert abs(loss - float(want.mean().detach())) < 4 * off
    # a gradient's factors: the logits' exponentials, off by as much, and some five values of 2^-8
    for k, grads in m.grad.items():
        ref = [v.grad for v in w[k]] if k == "out" else [w[k][0].grad] * p
        for a, b in zip(grads, ref):
            assert float((a.cpu() - b).norm()) <= (2 * off + 0.03) * float(b.norm()), k
    dx = torch.cat([d.cpu().float() for d in m.dy])
    assert float((dx - x.grad).norm()) <= (2 * off + 0.03) * float(x.grad.norm())


def test_texts_and_steps(ex):
    m, losses = ex.train(3, seed=1, log=None, rows=48, vocab=777, p=3)
    assert all(math.isfinite(v) for v in losses)
    for k in ("gamma", "w"):
        for r in range(1, m.p):
            assert torch.equal(m.w[k][0], m.w[k][r]), k
    allow = torch.rand(777, generator=torch.Generator().manual_seed(2)) < 0.3
    allow[5] = True
    first = torch.tensor([5, 9, 11, 700])
    text = m.write(first.cuda(), 12, allow).cpu()
    assert torch.equal(text[:, 0], first) and bool(allow[text[:, 1:]].all())
    # the same choice from the logits that the oracle adjusts (every other entry is further below than a rounding of bf16)
    for n in range(1, 12):
        z = torch.cat([a.cpu() for a in m.teacher_logits(text[:, n - 1].cuda())], 1).double().numpy()
        one = [1.0] * 4
        want, _ = token_ops.adjust(z, [t[:n].numpy() for t in text], [1] * 4, [np.float32(1.2)] * 4, one, [0.5] * 4, None, np.tile(allow.numpy(), (4, 1)))
        best = want.max(1)
        assert (want[np.arange(4), text[:, n].numpy()] >= best - 2.0 ** -7 * np.abs(best)).all()


# ----------------------------------------------------------------------------
# Streams, graphs, repeats
# ----------------------------------------------------------------------------

def _step(coll, g, stream=None, defer=False):
    """All operators once over two ranks; returns the calls and the outputs."""
    p, rows, hidden, v, top = 2, 37, 640, 1111, 70
    N = lambda *s, d=BF16: dev(g.normal(0, 1, s), d)[0]  # noqa: E731
    x, res, dy, dh = [[N(rows, hidden) for _ in range(p)] for _ in range(4)]
    w = [dev(g.normal(1, 0.2, hidden), F32)[0] for _ in range(p)]
    y, h, dx = [[new((rows, hidden), BF16) for _ in range(p)] for _ in range(3)]
    y8, rstd, dg = u8(p, rows, coll.coll_ckpt8_row_bytes(hidden, 128)), f32(p, rows), f32(p, hidden)
    ws = workspace(coll.coll_rmsnorm_workspace_bytes(p, rows, hidden))
    zs, _ = shards(g.normal(0, 3, (rows, v)), [0, 500, v], F32)
    by = Case(g, rows, v).device()
    out = [torch.zeros_like(z) for z in zs]
    idx = torch.from_numpy(g.integers(-1, v, (rows, top)).astype(np.int32)).cuda()
    logp = torch.log_softmax(N(rows, top, d=F32), 1) - 0.1
    st, lo = [f32(p, rows, 4) for _ in range(2)], [f32(p, rows) for _ in range(2)]
    ws2 = workspace(coll.coll_vocab_distill_workspace_bytes(rows, [500, v - 500], top))
    dz = [[torch.zeros_like(z) for z in zs] for _ in range(2)]
    k = dict(stream=stream, defer=defer)
    calls = [
        lambda: coll.coll_rmsnorm(x, w, y, hidden, residual=res, **k),
        lambda: coll.coll_rmsnorm_fp8(x, w, list(y8), hidden, 128, residual=res, h=h, rstd=list(rstd), **k),
        lambda: coll.coll_rmsnorm_backward(dy, h, list(rstd), w, dx, list(dg), ws, hidden, dh=dh, **k),
        lambda: coll.coll_vocab_adjust(zs, out, **by, **k),
        lambda: coll.coll_vocab_distill(zs, idx, logp, list(st[0]), list(lo[0]), ws2, kind=0, **k),
        lambda: coll.coll_vocab_distill(zs, idx, logp, list(st[1]), list(lo[1]), ws2, kind=1, **k),
        lambda: coll.coll_vocab_distill_backward(zs, idx, logp, st[0][1], lo[0][0], dz[0], kind=0, **k),
        lambda: coll.coll_vocab_distill_backward(zs, idx, logp, st[1][0], lo[1][1], dz[1], kind=1, **k),
    ]
    return calls, [*y, *h, *dx, y8, rstd, dg, *out, *st, *lo, *dz[0], *dz[1]], (x, res, dy, dh, w, zs, by, idx, logp, ws, ws2)


def _bits(t):
    return t.contiguous().view(torch.uint8)


def test_repeats_streams_and_grid_limits_give_the_same_bits(coll):
    calls, outs, keep = _step(coll, rng(90))
    for c in calls:
        c()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    for limit in (0, 1, 7):
        coll.coll_set_grid_limit(limit)
        try:
            calls2, outs2, keep2 = _step(coll, rng(90), stream=side)
            side.wait_stream(torch.cuda.current_stream())
            for c in calls2:
                c()
            side.synchronize()
        finally:
            coll.coll_set_grid_limit(0)
        for a, b in zip(first, outs2):
            assert torch.equal(_bits(a), _bits(b))


def test_graph_replays_match_eager_calls(coll):
    calls, outs, keep = _step(coll, rng(91))
    for c in calls:
        c()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls:
            c()
    for i in range(8):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(_bits(a), _bits(b)), f"replay {i}"
        calls[i % len(calls)]()                               # eager work between the replays
        torch.cuda.synchronize()


def test_graph_replays_follow_their_inputs(coll):
    """Histories, lists, entries and logits that change between replays, lengths among them."""
    calls, outs, (x, res, dy, dh, w, zs, by, idx, logp, ws, ws2) = _step(coll, rng(92))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls:
            c()
    for i in range(3):
        for t in (*x, *res, *zs, logp):
            t.copy_(t.roll(1, 0))
        idx.copy_(idx.flip(1))
        for o in ("offsets", "bias_offsets"):
            n = by[o][1:] - by[o][:-1]
            by[o][1:] = n.roll(1).cumsum(0)
        by["mask"].copy_(by["mask"].roll(1, 0))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for c in calls:
            c()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(_bits(a), _bits(b)), f"replay {i}"


def test_deferred_calls(coll):
    calls, outs, keep = _step(coll, rng(93), defer=True)
    prepared = [c() for c in calls]
    for _ in range(2):
        for f in prepared:
            f()
    torch.cuda.synchronize()
    again, outs2, keep2 = _step(coll, rng(93))
    for c in again:
        c()
    torch.cuda.synchronize()
    for a, b in zip(outs, outs2):
        assert torch.equal(_bits(a), _bits(b))


def test_calls_on_two_streams_at_once(coll):
    """The same inputs, a workspace each: neither call touches the other's results."""
    calls, outs, keep = _step(coll, rng(94))
    for c in calls:
        c()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [_step(coll, rng(94), stream=s) for s in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, b in zip(both[0][0], both[1][0]):
            a()
            b()
    torch.cuda.synchronize()
    for _, got, _ in both:
        for a, b in zip(outs, got):
            assert torch.equal(_bits(a), _bits(b))
