"""Cases, plain forms and 64-bit values of the token-wise training operators over p logical ranks.

Three operators, each with its forward and its backward pass:

* ``layernorm``: layer norm over every rank's token rows; backward sums the weights' gradients over all
  rows and all ranks (data parallelism's AllReduce of them included);
* ``swiglu`` and ``roundtrip``: activation checkpoints in 8 bits (e4m3 codes, one fp32 scale a group), written by
  the gated activation's forward pass and read by its backward pass; layer norm has the same (``ckpt``);
* ``logprob``: log probabilities of given tokens, entropy and top alternatives over a vocabulary whose logits
  are sharded over the ranks, and the gradient of the logits.

``run`` computes them with elementary torch operations in fp32, or, where ``own`` is true, with the library.
"""
import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-5


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one token per rank, as a decoding step sees the layer: latency only
        dict(name="ln_forward_token", op="layernorm", way="forward", ckpt=0, p=4, rows=1, hidden=4096, dtype="bf16", wdtype="bf16", avg=False),
        # a training layer's tokens: 4096 x 7168 on each of 8 ranks
        dict(name="ln_forward_large", op="layernorm", way="forward", ckpt=0, p=8, rows=4096, hidden=7168, dtype="bf16", wdtype="bf16", avg=False),
        # its backward pass, the weights' gradients averaged over the ranks
        dict(name="ln_backward_large", op="layernorm", way="backward", ckpt=0, p=8, rows=4096, hidden=7168, dtype="bf16", wdtype="bf16", avg=True),
        # fp32 rows of an odd width (no row but the first of four is 16-byte aligned), few of them
        dict(name="ln_backward_odd_f32", op="layernorm", way="backward", ckpt=0, p=3, rows=1777, hidden=2565, dtype="f32", wdtype="f32", avg=False),
        # a layer whose input is kept in 8 bits between its two passes, fp32 master weights
        dict(name="ln_step_ckpt8", op="layernorm", way="step", ckpt=128, p=8, rows=2048, hidden=7168, dtype="bf16", wdtype="f32", avg=True),
        # the tokens that a few experts of a small batch get: forward and backward
        dict(name="swiglu_step_small", op="swiglu", way="step", ckpt=128, p=2, rows=17, hidden=1408, dtype="bf16"),
        # the gated activation of a training step, 4096 tokens a rank, forward and backward
        dict(name="swiglu_step_large", op="swiglu", way="step", ckpt=128, p=8, rows=4096, hidden=4096, dtype="bf16"),
        # an fp32 activation kept in 8 bits and brought back, an odd number of rows
        dict(name="ckpt8_roundtrip_f32", op="roundtrip", way="step", ckpt=64, p=4, rows=1021, hidden=5120, dtype="f32"),
        # serving: a few requests' next-token logits on 8 shards, with the 20 likeliest tokens
        dict(name="logprob_few_tokens", op="logprob", way="forward", p=8, rows=4, vocab=131072, dtype="bf16", top=20, temp=0.7, masked=False),
        # scoring a batch of sequences: log probabilities, entropy and the 8 likeliest tokens of 2048 positions
        dict(name="logprob_score_large", op="logprob", way="forward", p=8, rows=2048, vocab=131072, dtype="bf16", top=8, temp=1.0, masked=False),
        # a policy step over an odd vocabulary in fp32: forward, then the gradient through log probability and
        # entropy; some positions allow only part of the vocabulary, some are padding
        dict(name="logprob_step_odd_f32", op="logprob", way="step", p=4, rows=777, vocab=50257, dtype="f32", top=0, temp=1.0, masked=True),
        # the loss's gradient at the largest size: half a GiB of logits in, half a GiB of gradient out
        dict(name="logprob_backward_large", op="logprob", way="backward", p=8, rows=4096, vocab=65536, dtype="bf16", top=0, temp=1.0, masked=False),
    ]


def _log(rng, lo, hi):
    return int(round(float(lo) * (float(hi) / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["layernorm", "layernorm", "swiglu", "roundtrip", "logprob", "logprob"])
    p = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "logprob":
        vocab = _log(rng, 1000, 200000)
        rows = _log(rng, 1, max(1.0, min(8192, 2.6e8 / vocab / (BYTES[dtype] // 2))))
        way = rng.choice(["forward", "backward", "step"])
        top = rng.choice([0, 1, 8, 20, 32]) if way == "forward" else 0
        return dict(op=op, way=way, p=p, rows=rows, vocab=vocab, dtype=dtype, top=top,
                    temp=rng.choice([1.0, 1.0, 0.6, 1.3]), masked=rng.random() < 0.4)
    if op == "layernorm":
        ckpt = rng.choice([0, 0, 0, 32, 128, 256])
        way = "step" if ckpt else rng.choice(["forward", "backward", "step"])
        hidden = _log(rng, 64, 16384)
        if ckpt:
            hidden = max(ckpt, hidden // ckpt * ckpt)
        rows = _log(rng, 1, max(1.0, min(16384, 1.1e8 / p / hidden)))
        return dict(op=op, way=way, ckpt=ckpt, p=p, rows=rows, hidden=hidden, dtype=dtype,
                    wdtype=rng.choice(["f32", dtype]), avg=rng.random() < 0.5)
    group = rng.choice([16, 32, 64, 128, 128, 256, 512])
    hidden = max(group, _log(rng, 64, 16384) // group * group)
    rows = _log(rng, 1, max(1.0, min(16384, 5e7 / p / hidden)))
    return dict(op=op, way="step", ckpt=group, p=p, rows=rows, hidden=hidden, dtype=dtype)


def _row_bytes(hidden, group):
    return hidden + 16 * ((4 * (hidden // group) + 15) // 16)


def work(case):
    p, rows, b = case["p"], case["rows"], BYTES[case["dtype"]]
    if case["op"] == "logprob":
        n = rows * case["vocab"]
        by = fl = 0.0
        if case["way"] in ("forward", "step"):
            by += n * b + rows * 8 + p * rows * (8 + 4 + 4 + 8 * case["top"])
            fl += 8.0 * n
        if case["way"] in ("backward", "step"):
            by += 2 * n * b + rows * (8 + 8 + 4 + 4 + 4)
            fl += 8.0 * n
        return {"bytes": by, "flops": fl}
    n = p * rows * case["hidden"]
    if case["op"] == "roundtrip":
        return {"bytes": 2 * n * b + 2.0 * p * rows * _row_bytes(case["hidden"], case["ckpt"]), "flops": 4.0 * n}
    if case["op"] == "swiglu":  # gate and up in, out; the checkpoint out and in; dout in, both gradients and out again
        return {"bytes": 2 * n * b + n * b + 2.0 * p * rows * _row_bytes(2 * case["hidden"], case["ckpt"]) + n * b + 2 * n * b + n * b,
                "flops": 30.0 * n}
    w = p * case["hidden"] * BYTES[case["wdtype"]]
    kept = float(p * rows * _row_bytes(case["hidden"], case["ckpt"])) if case["ckpt"] else 0.0
    by = fl = 0.0
    if case["way"] in ("forward", "step"):
        by += 2 * n * b + 2 * w + 8 * p * rows + kept
        fl += 8.0 * n
    if case["way"] in ("backward", "step"):
        by += (2 * n * b + kept if case["ckpt"] else 3 * n * b) + 3 * w + 8 * p * rows
        fl += 14.0 * n
    return {"bytes": by, "flops": fl}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, p, rows, hidden, dtype):
    """Rows as a residual stream has them: unlike channels (some far wider than the rest) and unlike tokens."""
    channel = torch.exp(0.5 * _normal(g, hidden))
    shift = 0.2 * _normal(g, hidden)
    token = torch.exp(0.3 * _normal(g, p, rows, 1))
    return ((_normal(g, p, rows, hidden) * channel + shift) * token).to(dtype)


def _shards(case):
    """First vocabulary entry of every rank's shard, and the end: shards differ by one where p does not divide it."""
    p, v = case["p"], case["vocab"]
    return [v * r // p for r in range(p + 1)]


def _inputs(case, seed):
    """What both sides and the 64-bit values start from, from the seed alone."""
    g = _generator(seed)
    p, rows, dt = case["p"], case["rows"], DTYPES[case["dtype"]]
    if case["op"] == "logprob":
        v = case["vocab"]
        z = 2.5 * _normal(g, rows, v)
        targets = torch.randint(0, v, (rows,), generator=g, device="cuda")
        z.scatter_add_(1, targets[:, None], 6.0 + 3.0 * _normal(g, rows, 1))   # mostly likely tokens, as in a text
        if case["masked"]:
            # a third of the positions allow about a tenth of the vocabulary, their target within it;
            # every 16th is padding
            allow = torch.rand(rows, v, generator=g, device="cuda") < 0.1
            allow.scatter_(1, targets[:, None], True)
            allow |= (torch.arange(rows, device="cuda") % 3 != 1)[:, None]
            z.masked_fill_(~allow, float("-inf"))
            targets = torch.where(torch.arange(rows, device="cuda") % 16 == 15, torch.full_like(targets, -100), targets)
        cut = _shards(case)
        z = z.to(dt)
        s = {"logits": [z[:, a:b].contiguous() for a, b in zip(cut, cut[1:])], "targets": targets}
        s["dlogp"] = _normal(g, rows) / rows
        s["dentropy"] = -0.01 * torch.rand(rows, generator=g, device="cuda") / rows
        if case["way"] == "backward":   # what the forward pass left
            m, log_s, h = _softmax_stats(z.float(), 1.0 / case["temp"])
            s["stats"], s["entropy"] = torch.stack([m, log_s], -1), h
        return s
    hidden = case["hidden"]
    if case["op"] == "roundtrip":
        return {"x": _activations(g, p, rows, hidden, dt)}
    if case["op"] == "swiglu":
        return {"x": _activations(g, p, rows, 2 * hidden, dt), "dy": (1e-3 * _normal(g, p, rows, hidden)).to(dt)}
    wt = DTYPES[case["wdtype"]]
    s = {"x": _activations(g, p, rows, hidden, dt),
         # data parallelism: every rank holds the same weights, a copy each
         "gamma": (1 + 0.2 * _normal(g, hidden)).to(wt).repeat(p, 1), "beta": (0.1 * _normal(g, hidden)).to(wt).repeat(p, 1),
         "dy": (1e-3 * _normal(g, p, rows, hidden)).to(dt)}
    if case["way"] == "backward":
        x = s["x"].float()
        s["mean"] = x.mean(-1)
        s["rstd"] = torch.rsqrt((x - s["mean"][..., None]).square().mean(-1) + EPS)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        # the buffers that a user's program keeps for the results, and the calls with their arguments marshalled once
        _prepare_own(s)
    return s


# ----------------------------------------------------------------------------
# The plain forms
# ----------------------------------------------------------------------------

def _encode8(x, group):
    """The value that each element's 8-bit code and its group's scale stand for."""
    g = x.reshape(*x.shape[:-1], -1, group)
    top = torch.full((), 448.0, device=x.device)
    amax = g.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -110)
    codes = (g * torch.div(top.expand_as(amax), amax)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return (codes.float() * torch.div(amax, top.expand_as(amax))).reshape(x.shape)


def _softmax_stats(z, inv_temp):
    """Largest logit, log of the sum of exponentials about it, and entropy of each row; a row that its mask leaves
    nothing of has -inf, -inf and 0."""
    m = z.amax(-1)
    base = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    d = (z - base[:, None]) * inv_temp
    e = torch.exp(d)
    total = e.sum(-1)
    log_s = torch.log(total)
    a = (e * torch.where(e > 0, d, torch.zeros_like(d))).sum(-1)
    h = torch.where(m == float("-inf"), torch.zeros_like(m), log_s - a / total)
    return m, log_s, h


def _plain_layernorm(s):
    c, x, out = s["case"], s["x"].float(), {}
    gamma, beta = s["gamma"].float()[:, None], s["beta"].float()[:, None]
    if c["way"] == "backward":
        mean, rstd = s["mean"][..., None], s["rstd"][..., None]
    else:
        mean = x.mean(-1, keepdim=True)
        rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + EPS)
        out["y"] = ((x - mean) * rstd * gamma + beta).to(s["x"].dtype)
        out["mean"], out["rstd"] = mean[..., 0], rstd[..., 0]
        if c["way"] == "forward":
            return out
    if c["ckpt"]:
        x = _encode8(x, c["ckpt"])
    dy = s["dy"].float()
    xh = (x - mean) * rstd
    g = dy * gamma
    out["dx"] = (rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))).to(s["x"].dtype)
    over = float(c["p"]) if c["avg"] else 1.0
    out["dgamma"] = ((dy * xh).sum((0, 1)) / over).to(s["gamma"].dtype).expand(c["p"], -1).contiguous()
    out["dbeta"] = (dy.sum((0, 1)) / over).to(s["gamma"].dtype).expand(c["p"], -1).contiguous()
    return out


def _plain_swiglu(s):
    c, dt = s["case"], s["x"].dtype
    f = c["hidden"]
    x = s["x"].float()
    gate, up = x[..., :f], x[..., f:]
    out = (gate * torch.sigmoid(gate) * up).to(dt)
    kept = _encode8(x, c["ckpt"])
    gate, up = kept[..., :f], kept[..., f:]
    sig = torch.sigmoid(gate)
    dy = s["dy"].float()
    dx = torch.cat([dy * up * sig * (1 + gate * (1 - sig)), dy * gate * sig], -1).to(dt)
    return {"out": out, "dx": dx, "again": (gate * sig * up).to(dt)}


def _plain_logprob(s):
    c, out = s["case"], {}
    z = torch.cat(s["logits"], -1).float()
    rows, v = z.shape
    inv_temp = 1.0 / c["temp"]
    targets = s["targets"]
    valid = (targets >= 0) & (targets < v)
    at = targets.clamp(0, v - 1)[:, None]
    if c["way"] == "backward":
        m, log_s = s["stats"][:, 0], s["stats"][:, 1]
        h = s["entropy"]
    else:
        m, log_s, h = _softmax_stats(z, inv_temp)
    empty = m == float("-inf")
    base = torch.where(empty, torch.zeros_like(m), m)
    if c["way"] != "backward":
        nothing = torch.full_like(m, float("-inf"))
        lp = torch.where(empty, nothing, (z.gather(1, at)[:, 0] - base) * inv_temp - log_s)
        lp = torch.where(valid, lp, torch.zeros_like(lp))
        each = lambda t: t.expand(c["p"], *t.shape).contiguous()  # noqa: E731  every rank gets the results
        out = {"stats": each(torch.stack([m, log_s], -1)), "logp": each(lp), "entropy": each(h)}
        if c["top"]:
            # by value, ties to the lowest index: the fp32 pattern as an ordered integer above the reversed index
            bits = (z + 0.0).view(torch.int32)
            key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64) * 2 ** 32 + (2 ** 32 - 1 - torch.arange(v, device=z.device))
            idx = (2 ** 32 - 1) - (torch.topk(key, c["top"], -1).values & 0xFFFFFFFF)
            val = (z.gather(1, idx) - base[:, None]) * inv_temp - log_s[:, None]
            out["top_logp"] = each(torch.where(empty[:, None], nothing[:, None], val))
            out["top_idx"] = each(idx.to(torch.int32))
        if c["way"] == "forward":
            return out
    lp = (z - base[:, None]) * inv_temp - log_s[:, None]
    prob = torch.exp(lp)
    g = torch.where(valid, s["dlogp"], torch.zeros_like(s["dlogp"]))[:, None]
    dz = -g * prob - s["dentropy"][:, None] * prob * (torch.where(prob > 0, lp, torch.zeros_like(lp)) + h[:, None])
    dz = dz.scatter_add(1, at, g) * inv_temp
    dz = torch.where(empty[:, None], torch.zeros_like(dz), dz).to(s["logits"][0].dtype)
    out["dlogits"] = [t.contiguous() for t in torch.split(dz, [t.shape[1] for t in s["logits"]], -1)]
    return out


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "layernorm":
        return _plain_layernorm(state)
    if op == "swiglu":
        return _plain_swiglu(state)
    if op == "roundtrip":
        x = state["x"]
        return {"x": _encode8(x.float(), state["case"]["ckpt"]).to(x.dtype)}
    return _plain_logprob(state)


# ----------------------------------------------------------------------------
# The library's operators
# ----------------------------------------------------------------------------

def _prepare_own(s):
    import collective_communication_primitives_coll_amd as coll
    c = s["case"]
    p, rows = c["p"], c["rows"]
    calls, out = [], {}

    def new(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if c["op"] == "logprob":
        inv_temp = 1.0 / c["temp"]
        z = s["logits"]
        if c["way"] != "backward":
            out = {"stats": new(p, rows, 2), "logp": new(p, rows), "entropy": new(p, rows)}
            top = {}
            if c["top"]:
                out["top_logp"], out["top_idx"] = new(p, rows, c["top"]), new(p, rows, c["top"], dtype=torch.int32)
                top = dict(top_k=c["top"], top_logp=list(out["top_logp"]), top_idx=list(out["top_idx"]))
            ws = new(coll.coll_vocab_logprob_workspace_bytes(rows, [t.shape[1] for t in z], c["top"]), dtype=torch.uint8)
            calls.append(coll.coll_vocab_logprob(z, s["targets"], list(out["stats"]), list(out["logp"]), ws,
                                                 entropy=list(out["entropy"]), inv_temp=inv_temp, defer=True, **top))
        if c["way"] != "forward":
            # the gradient's inputs: the forward pass's own results, or what it left before
            stats, h = (out["stats"][0], out["entropy"][0]) if out else (s["stats"], s["entropy"])
            dz = [torch.empty_like(t) for t in z]
            calls.append(coll.coll_vocab_logprob_backward(z, s["targets"], stats, s["dlogp"], dz, entropy=h,
                                                          dentropy=s["dentropy"], inv_temp=inv_temp, defer=True))
            out["dlogits"] = dz
    elif c["op"] == "roundtrip":
        x = s["x"]
        kept = new(p, rows, coll.coll_ckpt8_row_bytes(c["hidden"], c["ckpt"]), dtype=torch.uint8)
        out["x"] = torch.empty_like(x)
        calls.append(coll.coll_ckpt8_save(list(x), list(kept), c["hidden"], c["ckpt"], defer=True))
        calls.append(coll.coll_ckpt8_load(list(kept), list(out["x"]), c["hidden"], c["ckpt"], defer=True))
    elif c["op"] == "swiglu":
        x, dy = s["x"], s["dy"]
        kept = new(p, rows, coll.coll_ckpt8_row_bytes(2 * c["hidden"], c["ckpt"]), dtype=torch.uint8)
        out = {"out": torch.empty_like(dy), "dx": torch.empty_like(x), "again": torch.empty_like(dy)}
        calls.append(coll.coll_swiglu_ckpt8(list(x), list(out["out"]), list(kept), c["hidden"], c["ckpt"], defer=True))
        calls.append(coll.coll_swiglu_backward_ckpt8(list(kept), list(dy), list(out["dx"]), c["hidden"], c["ckpt"],
                                                     out=list(out["again"]), defer=True))
    else:
        x, dy, h, wt = s["x"], s["dy"], c["hidden"], s["gamma"].dtype
        each = lambda t: list(t)  # noqa: E731  a rank's buffers by rank
        kept = new(p, rows, coll.coll_ckpt8_row_bytes(h, c["ckpt"]), dtype=torch.uint8) if c["ckpt"] else None
        mean, rstd = s.get("mean"), s.get("rstd")
        if c["way"] != "backward":
            mean, rstd = new(p, rows), new(p, rows)
            out = {"y": torch.empty_like(x), "mean": mean, "rstd": rstd}
            if c["ckpt"]:
                calls.append(coll.coll_layernorm_ckpt8(each(x), each(s["gamma"]), each(s["beta"]), each(out["y"]), each(mean),
                                                       each(rstd), each(kept), h, c["ckpt"], eps=EPS, defer=True))
            else:
                calls.append(coll.coll_layernorm(each(x), each(s["gamma"]), each(s["beta"]), each(out["y"]), h, eps=EPS,
                                                 mean=each(mean), rstd=each(rstd), defer=True))
        if c["way"] != "forward":
            out |= {"dx": torch.empty_like(x), "dgamma": new(p, h, dtype=wt), "dbeta": new(p, h, dtype=wt)}
            ws = new(coll.coll_layernorm_workspace_bytes(p, rows, h), dtype=torch.uint8)
            tail = (each(mean), each(rstd), each(s["gamma"]), each(out["dx"]), each(out["dgamma"]), each(out["dbeta"]), ws, h)
            op = coll.COLL_AVG if c["avg"] else coll.COLL_SUM
            if c["ckpt"]:
                calls.append(coll.coll_layernorm_backward_ckpt8(each(dy), each(kept), *tail, c["ckpt"], op=op, defer=True))
            else:
                calls.append(coll.coll_layernorm_backward(each(dy), each(x), *tail, op=op, defer=True))
    s["calls"], s["out"] = calls, out


def _run_own(s):
    for call in s["calls"]:
        call()
    return s["out"]


# ----------------------------------------------------------------------------
# The values in 64 bits
# ----------------------------------------------------------------------------

def _kept8(x, group):
    """What a group's 8-bit codes stand for, from the format's definition: scale and its inverse are fp32 quotients,
    the scaled value an fp32 product; its nearest e4m3 number (ties to even, 448 at most) by the spacing of those
    numbers, 2^(e-3) in [2^e, 2^(e+1)) and 2^-9 below 2^-6; the product with the scale in 64 bits."""
    g = x.float().unflatten(-1, (x.shape[-1] // group, group))
    amax = torch.maximum(g.abs().max(-1, keepdim=True).values, torch.tensor(2.0 ** -110, device=x.device))
    a = amax.cpu().numpy()
    inv = torch.from_numpy(np.float32(448) / a).to(x.device)
    scale = torch.from_numpy(a / np.float32(448)).to(x.device)
    v = (g * inv).double()
    e = torch.frexp(v)[1].clamp_min(-5) - 1
    step = torch.ldexp(torch.ones_like(v), e - 3)
    q = (torch.round(v / step) * step).clamp(-448, 448)
    return (q * scale.double()).flatten(-2)


def _exact_layernorm(c, s):
    p, way = c["p"], c["way"]
    got = {k: [] for k in ("y", "mean", "rstd", "dx")}
    dgamma = dbeta = 0.0
    for r in range(p):
        x = s["x"][r].double()
        gamma, beta = s["gamma"][r].double(), s["beta"][r].double()
        if way == "backward":
            mean, rstd = s["mean"][r].double(), s["rstd"][r].double()
        else:
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = (var + EPS) ** -0.5
            got["y"].append(torch.addcmul(beta, (x - mean[:, None]) * rstd[:, None], gamma))
            got["mean"].append(mean)
            got["rstd"].append(rstd)
            if way == "forward":
                continue
        if c["ckpt"]:
            x = _kept8(s["x"][r], c["ckpt"])
        n = (x - mean[:, None]) * rstd[:, None]
        dy = s["dy"][r].double()
        dgamma = dgamma + torch.einsum("ij,ij->j", dy, n)
        dbeta = dbeta + dy.sum(0)
        w = dy * gamma
        h = x.shape[1]
        got["dx"].append((w * h - w.sum(1, keepdim=True) - n * (w * n).sum(1, keepdim=True)) * (rstd / h)[:, None])
    out = {k: torch.stack(v) for k, v in got.items() if v}
    if way != "forward":
        over = p if c["avg"] else 1
        out["dgamma"], out["dbeta"] = (dgamma / over).repeat(p, 1), (dbeta / over).repeat(p, 1)
    return out


def _exact_swiglu(c, s):
    f, got = c["hidden"], {"out": [], "dx": [], "again": []}
    for r in range(c["p"]):
        x, dy = s["x"][r].double(), s["dy"][r].double()
        got["out"].append(x[:, :f] / (1 + torch.exp(-x[:, :f])) * x[:, f:])
        x = _kept8(s["x"][r], c["ckpt"])
        g, u = x[:, :f], x[:, f:]
        t = 1 / (1 + torch.exp(-g))
        got["dx"].append(torch.hstack([dy * u * (t + g * t * (1 - t)), dy * g * t]))
        got["again"].append(g * t * u)
    return {k: torch.stack(v) for k, v in got.items()}


def _exact_logprob(c, s):
    rows, v, p = c["rows"], c["vocab"], c["p"]
    inv = 1.0 / c["temp"]
    step = max(1, int(4e7) // v)
    got = {k: [] for k in ("stats", "logp", "entropy", "top_logp", "top_idx", "dlogits")}
    for a in range(0, rows, step):
        z = torch.hstack([t[a:a + step] for t in s["logits"]]).double()
        n = torch.arange(z.shape[0], device=z.device)
        t = s["targets"][a:a + step]
        counts = (t >= 0) & (t < v)
        t = torch.where(counts, t, 0)
        m = z.max(1).values
        if bool((m == float("-inf")).any()):
            return None
        logp = torch.log_softmax(z * inv, 1)
        prob = logp.exp()
        h = -torch.special.xlogy(prob, prob).sum(1)
        if c["way"] != "backward":
            lse = torch.logsumexp(z * inv, 1)
            got["stats"].append(torch.stack([m, lse - m * inv], 1))
            got["logp"].append(torch.where(counts, logp[n, t], 0.0))
            got["entropy"].append(h)
            if c["top"]:
                idx = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :c["top"]]
                got["top_logp"].append(logp.gather(1, idx))
                got["top_idx"].append(idx.to(torch.int32))
        if c["way"] != "forward":
            d = torch.where(counts, s["dlogp"][a:a + step].double(), 0.0)
            e = s["dentropy"][a:a + step].double()
            one = torch.zeros_like(prob)
            one[n, t] = 1.0
            # of entropy: -p (log p + H), p log p without a 0 * inf
            dh = -(torch.special.xlogy(prob, prob) + prob * h[:, None])
            got["dlogits"].append((d[:, None] * (one - prob) + e[:, None] * dh) * inv)
    out = {k: torch.cat(x) for k, x in got.items() if x}
    for k in out:
        if k == "dlogits":
            cut = _shards(c)
            out[k] = [out[k][:, a:b].contiguous() for a, b in zip(cut, cut[1:])]
        else:
            out[k] = out[k].expand(p, *out[k].shape).contiguous()
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "layernorm":
        return _exact_layernorm(case, s)
    if case["op"] == "swiglu":
        return _exact_swiglu(case, s)
    if case["op"] == "roundtrip":
        return {"x": torch.stack([_kept8(x, case["ckpt"]) for x in s["x"]])}
    return _exact_logprob(case, s)
