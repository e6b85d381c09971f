"""The token-wise operators together with the collectives: the example's
training step, its gradients against autograd's in fp32 on the CPU, and its
loss over some steps."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "sharded_training_step.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("sharded_training_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("p,rows,hidden,ffn,vocab,group", [(4, 64, 256, 512, 1000, 64), (1, 33, 128, 128, 517, 16), (3, 7, 384, 256, 2048, 128)])
def test_gradients_of_a_step(ex, p, rows, hidden, ffn, vocab, group):
    m = ex.ShardedStep(p=p, rows=rows, hidden=hidden, ffn=ffn, vocab=vocab, group=group, seed=3)
    g = torch.Generator().manual_seed(5)
    for r in range(p):  # weights that differ from ones and zeros, the same on every rank
        m.w["gamma"][r].copy_(torch.linspace(0.5, 1.5, hidden))
        m.w["beta"][r].copy_(torch.linspace(-0.5, 0.5, hidden))
    tokens = [torch.randint(vocab, (rows,), generator=g) for _ in range(p)]
    loss = float(m.forward_backward([t.cuda() for t in tokens]))

    w = {k: [t.cpu().clone().requires_grad_() for t in (v if k == "out" else v[:1])] for k, v in m.w.items()}
    t = torch.cat(tokens)
    x = m.embedding.cpu().float()[t].requires_grad_()
    y = torch.nn.functional.layer_norm(x, (hidden,), w["gamma"][0], w["beta"][0])
    gate, up = (y @ w["gate_up"][0]).chunk(2, 1)
    h = x + (torch.nn.functional.silu(gate) * up) @ w["down"][0]
    want = torch.nn.functional.cross_entropy(h @ torch.cat(w["out"], 1), m.successor.cpu()[t])
    want.backward()

    # rounding to bf16 (2^-9 of each value on average over many) and sums of
    # hidden terms of order 1 in the logits
    assert abs(loss - float(want.detach())) < 0.02
    # a gradient's factors come from two codes, off by 2^-4 each at most, and
    # some six values of 2^-8: so its norm's error is below 0.15 of its norm
    for k, grads in m.grad.items():
        ref = [v.grad for v in w[k]] if k == "out" else [w[k][0].grad] * p
        for a, b in zip(grads, ref):
            assert float((a.cpu() - b).norm()) <= 0.15 * float(b.norm()), k
    dx = torch.cat([d.cpu().float() for d in m.dy])
    assert float((dx - x.grad).norm()) <= 0.15 * float(x.grad.norm())


def test_loss_falls_and_replicas_agree(ex):
    m, losses = ex.train(40, seed=1, log=None)
    # it starts near log(vocab) (logits of unit variance add half), and a
    # sixteenth of the tokens, each seen 160 times, is learned well below it
    assert losses[0] > math.log(m.vocab) - 0.5 and all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.5 * losses[0]
    for k in ("gamma", "beta", "gate_up", "down"):
        for r in range(1, m.p):
            assert torch.equal(m.w[k][0], m.w[k][r]), k
