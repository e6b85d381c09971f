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


def rmsnorm(h, gamma, eps):
    """h [rows, H] -> y, rstd."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * gamma, rstd


def rmsnorm_backward(dy, h, rstd, gamma, dh=None):
    """One rank's rows -> dx, sum dy n, and n (the normalised rows)."""
    n = h * rstd[:, None]
    w = dy * gamma
    dx = rstd[:, None] * (w - n * (w * n).mean(axis=1, keepdims=True))
    return dx if dh is None else dx + dh, (dy * n).sum(axis=0), n


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


def distill(z, idx, logp, t, tail):
    """z [rows, V] (-inf: masked), the teacher's entries idx and logp [rows, K], t = inverse temperature, tail: all
    other entries are one more class.  Returns a dict of stats [rows, 4], loss, and, for tolerances, among
    [rows, V] (which entries are listed), q [rows, V] and d = (z - m) t."""
    rows, v = z.shape
    out = {"stats": np.full((rows, 4), np.nan), "loss": np.full(rows, np.nan), "among": np.zeros((rows, v), dtype=bool),
           "q": np.zeros((rows, v)), "d": np.full((rows, v), np.nan)}
    for i in range(rows):
        lq = np.full(v, -np.inf)
        among = out["among"][i]
        for j, lj in zip(idx[i], logp[i]):
            if 0 <= j < v and not among[j]:
                among[j], lq[j] = True, lj
        padding = not among.any() if tail else not (among & ~np.isneginf(lq)).any()
        if padding:
            out["loss"][i], out["stats"][i, 2:] = 0.0, (np.inf, 0.0)
        broken = np.isnan(lq).any() or np.isposinf(lq).any()
        if tail:
            q, fourth = np.exp(lq), 1.0 - np.exp(lq).sum()
        elif broken or padding:
            q, fourth = np.full(v, np.nan), 0.0
        else:
            total = np.log(np.exp(lq - lq.max()).sum()) + lq.max()
            q, fourth = np.exp(lq - total), 0.0
        if broken:
            q, fourth = np.full(v, np.nan), np.nan
        out["q"][i] = q
        if np.isnan(z[i]).any() or np.isposinf(z[i]).any():
            continue
        m = z[i].max()
        if m == -np.inf:
            out["stats"][i, :2] = -np.inf
            if not padding:
                out["loss"][i] = np.inf
                out["stats"][i, 2:] = (-np.inf, fourth) if tail else (total if not broken else np.nan, 0.0)
            continue
        d = (z[i] - m) * t
        ls = np.log(np.exp(d).sum())
        out["stats"][i, :2], out["d"][i] = (m, ls), d
        if padding:
            continue
        rest = d[~among]
        far = rest.max() if rest.size else -np.inf
        ltail = np.log(np.exp(rest - far).sum()) + far if far > -np.inf else -np.inf
        if ltail < -1e4:                                    # masks of a type's lowest value: none are allowed
            ltail = -np.inf
        out["stats"][i, 2:] = (ltail, fourth) if tail else (np.nan if broken else total, 0.0)
        if broken:
            continue
        with np.errstate(invalid="ignore"):
            loss = np.where(q > 0, q * ((lq if tail else lq - total) - (d - ls)), 0.0).sum()
        if tail and fourth > 0 and ltail > -np.inf:  # (left out where no other entry is allowed)
            loss += fourth * (np.log(fourth) - (ltail - ls))
        out["loss"][i] = loss
    return out


def distill_backward(z, among, q, t, stats, dloss, tail):
    """dz [rows, V] from the forward pass's stats; among and q as distill gives them."""
    dz = np.zeros(z.shape)
    for i in range(len(z)):
        m, ls, third, fourth = stats[i]
        if third == np.inf or m == -np.inf:
            continue
        d = (z[i] - m) * t
        p = np.exp(d - ls)
        if tail:
            rest, whole = (fourth if not fourth <= 0 else 0.0), (1.0 - fourth if not fourth >= 0 or third == -np.inf else 1.0)
            others = 0.0 * p if third == -np.inf else np.exp(d - third) * (whole * np.exp(third - ls) - rest)
            dz[i] = np.where(among[i], whole * p - q[i], others)
        else:
            dz[i] = np.where(among[i], p - q[i], p + (third - third))
        dz[i] *= dloss[i] * t
    return dz


def adjust(z, history=None, prompt=None, repetition=None, presence=None, frequency=None, biases=None, allow=None):
    """z [rows, V]; history[i]: row i's tokens, the first prompt[i] of them the prompt's; biases[i]: pairs (entry,
    value); allow [rows, V] truth values.  Returns the adjusted logits and the size of the terms in each."""
    out = np.array(z, dtype=np.float64)
    rows, v = out.shape
    size = np.zeros((rows, v))
    for i in range(rows):
        h = np.asarray(history[i] if history else [], dtype=np.int64)
        inside = lambda t: t[(t >= 0) & (t < v)]  # noqa: E731
        start = min(max(int(prompt[i]), 0), len(h)) if prompt is not None else 0
        seen = np.unique(inside(h))
        count = np.bincount(inside(h[start:]), minlength=v)
        if repetition is not None:
            r = float(repetition[i])
            out[i, seen] = np.where(out[i, seen] > 0, out[i, seen] / r, out[i, seen] * r)
        size[i] = np.abs(np.where(np.isfinite(out[i]), out[i], 0.0))
        less = (count * float(frequency[i]) if frequency is not None else 0.0) + (float(presence[i]) if presence is not None else 0.0)
        out[i] -= np.where(count > 0, less, 0.0)
        size[i] += 2 * np.abs(np.where(count > 0, less, 0.0))
        had = set()
        for j, b in biases[i] if biases else []:
            if 0 <= j < v and j not in had:
                had.add(j)
                out[i, j] += b
                size[i, j] += abs(b) if np.isfinite(b) else 0.0
    if allow is not None:
        out[~allow] = -np.inf
    return out, size
