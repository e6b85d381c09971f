"""Pins for the token-wise operators' oracle: torch's CPU library in float64
for the forward values, central differences and torch's autograd in float64
for the gradients, and the definitions' edge values."""
import numpy as np
import pytest
import torch

from oracle import fp8, token_ops


def _rng(*seed):
    return np.random.default_rng([9100, *seed])


@pytest.mark.parametrize("rows,hidden", [(1, 1), (3, 5), (4, 64), (2, 257)])
def test_layernorm_matches_library(rows, hidden):
    g = _rng(rows, hidden)
    x, gamma, beta = g.normal(3, 2, (rows, hidden)), g.normal(1, 0.3, hidden), g.normal(size=hidden)
    y, mean, rstd = token_ops.layernorm(x, gamma, beta, 1e-5)
    t = torch.nn.functional.layer_norm(torch.from_numpy(x), (hidden,), torch.from_numpy(gamma), torch.from_numpy(beta), 1e-5)
    assert np.allclose(y, t.numpy(), rtol=1e-11, atol=1e-11)
    assert np.allclose(mean, x.mean(1)) and np.allclose(rstd, 1 / np.sqrt(x.var(1) + 1e-5))


@pytest.mark.parametrize("rows,hidden", [(1, 2), (3, 5), (4, 33)])
def test_layernorm_gradient_by_differences(rows, hidden):
    g = _rng(1, rows, hidden)
    x, gamma, beta, dy = g.normal(1, 2, (rows, hidden)), g.normal(1, 0.3, hidden), g.normal(size=hidden), g.normal(size=(rows, hidden))
    _, mean, rstd = token_ops.layernorm(x, gamma, beta, 1e-5)
    dx, dgamma, dbeta, _ = token_ops.layernorm_backward(dy, x, mean, rstd, gamma)
    loss = lambda x, ga, be: (token_ops.layernorm(x, ga, be, 1e-5)[0] * dy).sum()  # noqa: E731
    h = 1e-6
    for i in range(rows):
        for j in range(hidden):
            e = np.zeros_like(x)
            e[i, j] = h
            assert abs((loss(x + e, gamma, beta) - loss(x - e, gamma, beta)) / (2 * h) - dx[i, j]) < 1e-6
    for j in range(hidden):
        e = np.zeros(hidden)
        e[j] = h
        assert abs((loss(x, gamma + e, beta) - loss(x, gamma - e, beta)) / (2 * h) - dgamma[j]) < 1e-6
        assert abs((loss(x, gamma, beta + e) - loss(x, gamma, beta - e)) / (2 * h) - dbeta[j]) < 1e-6


def test_swiglu_and_its_gradient():
    g = _rng(2)
    x, dout = g.normal(0, 3, (4, 20)), g.normal(size=(4, 10))
    t = torch.from_numpy(x).requires_grad_()
    out = torch.nn.functional.silu(t[:, :10]) * t[:, 10:]
    out.backward(torch.from_numpy(dout))
    assert np.allclose(token_ops.swiglu(x), out.detach().numpy(), rtol=1e-12)
    dx = token_ops.swiglu_backward(x, dout)
    assert np.allclose(dx, t.grad.numpy(), rtol=1e-11, atol=1e-13)
    h = 1e-6
    for i, j in [(0, 0), (1, 9), (2, 10), (3, 19)]:
        e = np.zeros_like(x)
        e[i, j] = h
        d = ((token_ops.swiglu(x + e) - token_ops.swiglu(x - e)) * dout).sum() / (2 * h)
        assert abs(d - dx[i, j]) < 1e-7


def test_swiglu_far_values():
    x = np.array([[800.0, -800.0, 0.0, 2.0, 3.0, 4.0]])
    assert np.allclose(token_ops.swiglu(x), [[1600.0, 0.0, 0.0]])


def test_checkpoint_values_are_within_half_a_step():
    g = _rng(3)
    x = g.normal(0, 5, (6, 128)).astype(np.float32)
    rows = token_ops.ckpt8_rows(x, 32)
    assert rows.shape == (6, fp8.row_bytes(128, 32))
    v = token_ops.ckpt8_values(rows, 128, 32)
    amax = np.abs(x.reshape(6, 4, 32)).max(-1, keepdims=True)
    # half a step of e4m3: 2^-4 of the value, or half its subnormal 2^-9 times the scale
    lim = np.maximum(np.abs(x).reshape(6, 4, 32) * 2.0 ** -4, amax / 448 * 2.0 ** -10) * (1 + 1e-5)
    assert (np.abs(v - x).reshape(6, 4, 32) <= lim).all()


@pytest.mark.parametrize("t", [1.0, 0.5, 2.5])
def test_logprob_matches_library(t):
    g = _rng(4)
    z = g.normal(0, 4, (5, 37))
    z[1, 3:30] = -np.inf
    targets = np.array([0, 36, 5, -1, 12])
    r = token_ops.logprob(z, targets, t, 6)
    lp = torch.log_softmax(torch.from_numpy(z) * t, 1)
    assert np.allclose(r["logprobs"], lp.numpy(), rtol=1e-12)
    assert r["logp"][3] == 0.0 and np.allclose(np.delete(r["logp"], 3), lp.numpy()[[0, 1, 2, 4], [0, 36, 5, 12]])
    ent = torch.distributions.Categorical(logits=lp).entropy()
    assert np.allclose(np.delete(r["entropy"], 1), np.delete(ent.numpy(), 1))
    assert np.array_equal(r["top_idx"], np.argsort(-z, 1, kind="stable")[:, :6])


def test_logprob_edge_rows():
    z = np.full((4, 5), -np.inf)
    z[1] = 7.0                       # all alike
    z[2] = [0, np.nan, 1, 2, 3]
    z[3] = [0, np.inf, 1, 2, 3]
    r = token_ops.logprob(z, np.array([2, 2, 0, 9]), 1.0, 3)
    assert np.isneginf(r["stats"][0]).all() and np.isneginf(r["logp"][0]) and r["entropy"][0] == 0
    assert list(r["top_idx"][0]) == [0, 1, 2] and np.isneginf(r["top_logp"][0]).all()
    assert np.allclose(r["logp"][1], -np.log(5)) and np.allclose(r["entropy"][1], np.log(5))
    assert list(r["top_idx"][1]) == [0, 1, 2]
    assert np.isnan(r["logp"][2]) and list(r["top_idx"][2]) == [-1, -1, -1]
    assert np.isnan(r["stats"][3]).all() and r["logp"][3] == 0.0
    dz = token_ops.logprob_backward(z[:1], np.array([2]), 1.0, r["stats"][:1], [1.0], [0.0], [1.0])
    assert (dz == 0).all()


@pytest.mark.parametrize("t", [1.0, 0.7])
def test_logprob_gradient_by_differences(t):
    g = _rng(5)
    z = g.normal(0, 2, (3, 11))
    z[1, :4] = -np.inf
    targets, gl, gh = np.array([4, 7, -5]), g.normal(size=3), g.normal(size=3)
    r = token_ops.logprob(z, targets, t)
    dz = token_ops.logprob_backward(z, targets, t, r["stats"], gl, r["entropy"], gh)
    assert (dz[1, :4] == 0).all()

    def loss(z):
        q = token_ops.logprob(z, targets, t)
        return (q["logp"] * gl + q["entropy"] * gh).sum()
    h = 1e-6
    for i in range(3):
        for j in range(11):
            if np.isneginf(z[i, j]):
                continue
            e = np.zeros_like(z)
            e[i, j] = h
            assert abs((loss(z + e) - loss(z - e)) / (2 * h) - dz[i, j]) < 1e-6
