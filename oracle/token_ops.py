"""CPU oracle for the token-wise operators of a training step.

TEST INFRASTRUCTURE ONLY.  Plain NumPy in float64, from the operators'
definitions, sharing no code with the HIP path.  Inputs are float64 arrays of
the exact values the kernels read (bf16 and fp32 values widened); the 8-bit
format's own steps are fp32 by definition and come from oracle/fp8.py.

Every function also returns what the tests' tolerances are made of, where it
is not a result itself.
"""
from __future__ import annotations

import numpy as np

from . import fp8


def layernorm(x, gamma, beta, eps):
    """x [rows, H] -> y, mean, rstd."""
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    return d * rstd[:, None] * gamma + beta, mean, rstd


def layernorm_backward(dy, x, mean, rstd, gamma):
    """One rank's rows -> dx, sum dy n, sum dy, and n (the normalised rows)."""
    n = (x - mean[:, None]) * rstd[:, None]
    w = dy * gamma
    c1 = w.mean(axis=1, keepdims=True)
    c2 = (w * n).mean(axis=1, keepdims=True)
    return rstd[:, None] * (w - c1 - n * c2), (dy * n).sum(axis=0), dy.sum(axis=0), n


def ckpt8_rows(x32, group):
    """Packed checkpoint rows [rows, row_bytes] of float32 rows (finite)."""
    return np.stack([fp8.encode_row(r, group) for r in np.asarray(x32, dtype=np.float32)])


def ckpt8_values(rows, hidden, group):
    """The float32 values of packed rows: code * scale, rounded to fp32."""
    rows = np.asarray(rows, dtype=np.uint8)
    ng = hidden // group
    codes = fp8.e4m3_decode(rows[:, :hidden]).reshape(len(rows), ng, group)
    scales = np.ascontiguousarray(rows[:, hidden:hidden + 4 * ng]).view("<f4").reshape(-1, ng)
    return (codes * scales[:, :, None]).astype(np.float32).reshape(len(rows), hidden)


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def swiglu(x):
    """[rows, 2F] (gate, then up) -> [rows, F]."""
    f = x.shape[1] // 2
    return x[:, :f] * sigmoid(x[:, :f]) * x[:, f:]


def swiglu_backward(x, dout):
    f = x.shape[1] // 2
    g, u, s = x[:, :f], x[:, f:], sigmoid(x[:, :f])
    return np.concatenate([dout * u * s * (1.0 + g * sigmoid(-g)), dout * g * s], axis=1)


def logprob(z, targets, t, top_k=0):
    """z [rows, V] (-inf: masked), t = inverse temperature.  Returns a dict of
    stats [rows, 2], logp, entropy, top_logp, top_idx and, per element,
    d = (z - m) t and logprobs = d - L."""
    rows, v = z.shape
    out = {"stats": np.empty((rows, 2)), "logp": np.zeros(rows), "entropy": np.zeros(rows),
           "top_logp": np.full((rows, top_k), -np.inf), "top_idx": np.full((rows, top_k), -1, dtype=np.int32),
           "d": np.full((rows, v), -np.inf), "logprobs": np.full((rows, v), -np.inf)}
    for i in range(rows):
        if np.isnan(z[i]).any() or np.isposinf(z[i]).any():
            for k in ("stats", "logp", "entropy", "top_logp", "d", "logprobs"):
                out[k][i] = np.nan
            if not 0 <= targets[i] < v:
                out["logp"][i] = 0.0
            continue
        m = z[i].max()
        order = np.argsort(-z[i], kind="stable")[:top_k]
        out["top_idx"][i, :len(order)] = order
        out["stats"][i] = -np.inf
        if m > -np.inf:
            d = (z[i] - m) * t
            e = np.exp(d)
            ls = np.log(e.sum())
            lp = d - ls
            p = e / e.sum()
            out["stats"][i] = m, ls
            out["entropy"][i] = -(p[p > 0] * lp[p > 0]).sum()
            out["d"][i], out["logprobs"][i] = d, lp
        out["top_logp"][i, :len(order)] = out["logprobs"][i][order]
        if 0 <= targets[i] < v:
            out["logp"][i] = out["logprobs"][i][targets[i]]
    return out


def logprob_backward(z, targets, t, stats, dlogp, entropy, dentropy):
    """dz [rows, V] from the forward pass's stats and entropy."""
    rows, v = z.shape
    dz = np.zeros((rows, v))
    for i in range(rows):
        m, ls = stats[i]
        if np.isneginf(m):
            continue
        lp = (z[i] - m) * t - ls
        p = np.exp(lp)
        lp = np.where(p > 0, lp, 0.0)
        counts = 0 <= targets[i] < v
        g = dlogp[i] if counts else 0.0
        dz[i] = -g * p - dentropy[i] * p * (lp + entropy[i])
        if counts:
            dz[i, targets[i]] += g
        dz[i] *= t
    return dz
