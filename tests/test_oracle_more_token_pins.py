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
