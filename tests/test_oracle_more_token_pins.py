"""Pins for the oracle of RMS norm, distillation and the adjustment of logits:
torch's CPU library in float64, central differences, and the definitions' edge
values."""
import numpy as np
import pytest
import torch

from oracle import token_ops


def _rng(*seed):
    return np.random.default_rng([9200, *seed])


@pytest.mark.parametrize("rows,hidden", [(1, 1), (3, 5), (4, 64), (2, 257)])
def test_rmsnorm_matches_library_and_autograd(rows, hidden):
    g = _rng(rows, hidden)
    h, gamma, dy, dh = g.normal(1, 2, (rows, hidden)), g.normal(1, 0.3, hidden), g.normal(size=(rows, hidden)), g.normal(size=(rows, hidden))
    y, rstd = token_ops.rmsnorm(h, gamma, 1e-6)
    t, w = torch.from_numpy(h).requires_grad_(), torch.from_numpy(gamma).requires_grad_()
    out = torch.nn.functional.rms_norm(t, (hidden,), w, 1e-6)
    assert np.allclose(y, out.detach().numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(rstd, 1 / np.sqrt(np.square(h).sum(1) / hidden + 1e-6))
    (out * torch.from_numpy(dy) + t * torch.from_numpy(dh)).sum().backward()
    dx, dgamma, n = token_ops.rmsnorm_backward(dy, h, rstd, gamma, dh)
    assert np.allclose(dx, t.grad.numpy(), rtol=1e-10, atol=1e-11) and np.allclose(dgamma, w.grad.numpy(), rtol=1e-11, atol=1e-12)
    assert np.allclose(n, h * rstd[:, None])
    assert np.allclose(token_ops.rmsnorm_backward(dy, h, rstd, gamma)[0] + dh, dx)


def _entries(g, z, k, t):
    """A teacher near z: its k likeliest entries, and its log probabilities."""
    teacher = torch.log_softmax(torch.from_numpy(z + g.normal(0, 0.7, z.shape)) * t, 1)
    logp, idx = teacher.topk(k, 1)
    return idx.numpy(), logp.numpy(), teacher.numpy()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("t", [1.0, 0.5])
def test_distillation_matches_library_and_autograd(tail, t):
    g = _rng(1, tail)
    z = g.normal(0, 3, (6, 23))
    z[2, 5:9] = -np.inf
    idx, logp, _ = _entries(g, z, 4, t)
    r = token_ops.distill(z, idx, logp, t, tail)
    x = torch.from_numpy(z).requires_grad_()
    lp = torch.log_softmax(x * t, 1)
    at = torch.from_numpy(idx)
    top, q = lp.gather(1, at), torch.from_numpy(np.exp(logp))
    if tail:
        rest = torch.logsumexp(lp.scatter(1, at, -np.inf), 1, keepdim=True)
        top, q = torch.cat([top, rest], 1), torch.cat([q, 1 - q.sum(1, keepdim=True)], 1)
    else:
        q = q / q.sum(1, keepdim=True)
    loss = torch.nn.functional.kl_div(top, q, reduction="none").sum(1)
    assert np.allclose(r["loss"], loss.detach().numpy(), rtol=1e-10, atol=1e-12)
    w = g.normal(size=6)
    (loss * torch.from_numpy(w)).sum().backward()
    dz = token_ops.distill_backward(z, r["among"], r["q"], t, r["stats"], w, tail)
    want = np.where(np.isneginf(z), 0.0, x.grad.numpy())
    assert np.allclose(dz, want, rtol=1e-9, atol=1e-12)
    # over all entries both kinds are the whole divergence
    idx, logp, teacher = _entries(g, z, 23, t)
    whole = (np.exp(teacher) * np.where(np.isneginf(teacher), 0.0, teacher - np.where(np.isneginf(z), 0.0, lp.detach().numpy()))).sum(1)
    assert np.allclose(token_ops.distill(z, idx, logp, t, tail)["loss"], whole, atol=1e-10)


@pytest.mark.parametrize("tail", [False, True])
def test_distillation_gradient_by_differences(tail):
    g = _rng(2, tail)
    z, w, t = g.normal(0, 2, (3, 11)), g.normal(size=3), 0.8
    idx, logp, _ = _entries(g, z, 4, t)
    idx[1, 2], idx[2, 3] = -1, idx[2, 0]                  # an absent entry, one listed twice
    if tail:
        logp[0] += 0.4                                    # masses above 1
    r = token_ops.distill(z, idx, logp, t, tail)
    dz = token_ops.distill_backward(z, r["among"], r["q"], t, r["stats"], w, tail)
    loss = lambda z: (token_ops.distill(z, idx, logp, t, tail)["loss"] * w).sum()  # noqa: E731
    for i in range(3):
        for j in range(11):
            e = np.zeros_like(z)
            e[i, j] = 1e-6
            assert abs((loss(z + e) - loss(z - e)) / 2e-6 - dz[i, j]) < 1e-6


def test_distillation_edge_rows():
    z = np.full((6, 5), -np.inf)
    z[1:] = [0.0, 1.0, 2.0, 3.0, np.nan]
    z[2:] = [0.0, 1.0, 2.0, 3.0, -np.inf]
    idx = np.array([[0, 1], [-1, 5], [-1, -1], [3, 4], [3, 3], [2, 3]])
    logp = np.log(np.array([[0.5, 0.25]] * 6))
    logp[5] = -np.inf
    for tail in (False, True):
        r = token_ops.distill(z, idx, logp, 1.0, tail)
        assert r["loss"][0] == np.inf and r["loss"][1] == 0 and r["loss"][2] == 0 and r["loss"][3] == np.inf
        assert (r["stats"][1:3, 2] == np.inf).all() and np.isneginf(r["stats"][0, :2]).all()
        p = np.exp(np.arange(4)) / np.exp(np.arange(4)).sum()
        if tail:
            assert np.allclose(r["loss"][4], 0.5 * np.log(0.5 / p[3]) + 0.5 * np.log(0.5 / (1 - p[3])))
            assert np.allclose(r["loss"][5], -np.log(p[0] + p[1]))
        else:
            assert np.allclose(r["loss"][4], -np.log(p[3])) and r["loss"][5] == 0 and r["stats"][5, 2] == np.inf
        dz = token_ops.distill_backward(z, r["among"], r["q"], 1.0, r["stats"], np.ones(6), tail)
        assert (dz[:3] == 0).all() and np.isfinite(dz).all()


def test_adjustment_by_hand():
    z = np.array([[2.0, -2.0, 0.0, 4.0, -1.0], [1.0, 1.0, 1.0, np.nan, -np.inf]])
    out, _ = token_ops.adjust(z, [[0, 1, 0, 3, 3, 9, -1], [4]], [2, 0], [2.0, 3.0], [0.5, 0.25], [0.125, 0.0],
                              [[(4, 10.0), (4, 20.0), (7, 1.0), (0, -np.inf)], []], np.array([[1, 1, 1, 1, 1], [1, 1, 0, 0, 1]], dtype=bool))
    # row 0: 0 and 1 are the prompt's, then 0 once and 3 twice
    assert np.array_equal(out[0], [-np.inf, -4.0, 0.0, 2.0 - 0.5 - 0.25, 9.0])
    assert np.array_equal(out[1], [1.0, 1.0, -np.inf, -np.inf, -np.inf])
    out, _ = token_ops.adjust(z[:1], [[3, 3, 0]], None, None, None, [1.0])
    assert np.array_equal(out[0], [1.0, -2.0, 0.0, 2.0, -1.0])
    assert np.array_equal(token_ops.adjust(z[:1])[0], z[:1])
