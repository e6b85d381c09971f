"""Cases, plain forms and 64-bit values of three more token-wise operators over p logical ranks.

* ``rms``: RMS norm of every rank's token rows with the residual's addition before it, its output in the rows' type
  or in 8 bits (e4m3 codes, one fp32 scale a group), and its backward pass, which sums the weights' gradient over all
  rows and all ranks;
* ``distill``: the loss of a student, whose logits are sharded over the ranks, against a teacher's top entries, and
  the logits' gradient;
* ``adjust``: penalties for repeated tokens, biases and grammar masks on sharded logits.

``run`` computes them with elementary torch operations in fp32, or, where ``own`` is true, with the library.
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-6
NOTHING = float("-inf")


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one token per rank between two layers of a decoding step: latency only
        dict(name="rms_token", op="rms", way="forward", res=True, fp8=0, p=4, rows=1, hidden=4096, dtype="bf16", wdtype="bf16", avg=False),
        # a training layer's tokens: 4096 x 7168 on each of 8 ranks, added to the residual stream and normalised
        dict(name="rms_forward_large", op="rms", way="forward", res=True, fp8=0, p=8, rows=4096, hidden=7168, dtype="bf16", wdtype="bf16", avg=False),
        # its backward pass: the stream's own gradient joins, the weights' gradient is averaged over the ranks
        dict(name="rms_backward_large", op="rms", way="backward", res=True, fp8=0, p=8, rows=4096, hidden=7168, dtype="bf16", wdtype="bf16", avg=True),
        # a layer whose normalised rows travel in 8 bits, and the values that their receiver gets
        dict(name="rms_fp8", op="rms", way="forward", res=True, fp8=128, p=8, rows=2048, hidden=5120, dtype="bf16", wdtype="f32", avg=False),
        # fp32 rows of an odd width without a residual (a norm of queries or of a head's input), both passes
        dict(name="rms_step_odd_f32", op="rms", way="step", res=False, fp8=0, p=3, rows=1777, hidden=2565, dtype="f32", wdtype="f32", avg=False),
        # a few positions of a student with a teacher's 20 likeliest tokens, all others as one class
        dict(name="distill_few_tokens", op="distill", way="forward", tail=True, p=8, rows=4, vocab=131072, top=20, dtype="bf16", temp=1.0, masked=False),
        # a distillation step: 2048 positions, 32 entries each, loss and gradient at a raised temperature
        dict(name="distill_step_large", op="distill", way="step", tail=True, p=8, rows=2048, vocab=131072, top=32, dtype="bf16", temp=2.0, masked=False),
        # an odd vocabulary in fp32, the teacher renormalised over its entries; a third of the positions allow only a
        # part of the vocabulary, some are padding
        dict(name="distill_step_odd_f32", op="distill", way="step", tail=False, p=4, rows=777, vocab=50257, top=8, dtype="f32", temp=1.0, masked=True),
        # serving: a few requests' next-token logits on 8 shards, histories of a few hundred tokens, one grammar each
        dict(name="adjust_few_tokens", op="adjust", p=8, rows=4, vocab=131072, history=400, bias=16, mask=True, dtype="bf16"),
        # a full decoding batch: histories of up to tens of thousands of tokens, biases and grammars
        dict(name="adjust_batch", op="adjust", p=8, rows=512, vocab=131072, history=4000, bias=100, mask=True, dtype="bf16"),
        # an odd vocabulary in fp32, penalties alone
        dict(name="adjust_odd_f32", op="adjust", p=4, rows=333, vocab=50257, history=1500, bias=0, mask=False, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(float(lo) * (float(hi) / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["rms", "rms", "distill", "distill", "adjust"])
    p = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rms":
        fp8 = rng.choice([0, 0, 0, 16, 128, 512])
        way = "forward" if fp8 else rng.choice(["forward", "backward", "step"])
        hidden = _log(rng, 64, 16384)
        if fp8:
            hidden = max(fp8, hidden // fp8 * fp8)
        rows = _log(rng, 1, max(1.0, min(16384, 1.1e8 / p / hidden)))
        return dict(op=op, way=way, res=rng.random() < 0.7, fp8=fp8, p=p, rows=rows, hidden=hidden, dtype=dtype,
                    wdtype=rng.choice(["f32", dtype]), avg=rng.random() < 0.5)
    vocab = _log(rng, 1000, 200000)
    rows = _log(rng, 1, max(1.0, min(8192, 2.2e8 / vocab / (BYTES[dtype] // 2))))
    if op == "distill":
        return dict(op=op, way=rng.choice(["forward", "backward", "step"]), tail=rng.random() < 0.5, p=p, rows=rows, vocab=vocab,
                    top=rng.choice([1, 5, 8, 20, 32, 64, 100, 128]), dtype=dtype, temp=rng.choice([1.0, 1.0, 2.0, 0.7]), masked=rng.random() < 0.4)
    rows = min(rows, 1024)
    return dict(op=op, p=p, rows=rows, vocab=vocab, history=_log(rng, 1, max(1.0, min(20000, 2.5e6 / rows))), bias=rng.choice([0, 1, 30, 300]),
                mask=rng.random() < 0.6, dtype=dtype)


def _row_bytes(hidden, group):
    return hidden + 16 * ((4 * (hidden // group) + 15) // 16)


def work(case):
    p, rows, b = case["p"], case["rows"], BYTES[case["dtype"]]
    if case["op"] == "rms":
        n = p * rows * case["hidden"]
        w = p * case["hidden"] * BYTES[case["wdtype"]]
        by = fl = 0.0
        if case["way"] in ("forward", "step"):
            by += (3 if case["res"] else 1) * n * b + w + 4 * p * rows
            # the result; in 8 bits it is written, read by its receiver and comes out as bf16 values
            by += 2.0 * p * rows * _row_bytes(case["hidden"], case["fp8"]) + 2 * n if case["fp8"] else n * b
            fl += 6.0 * n
        if case["way"] in ("backward", "step"):
            by += (4 if case["res"] else 3) * n * b + 2 * w + 4 * p * rows
            fl += 10.0 * n
        return {"bytes": by, "flops": fl}
    n = rows * case["vocab"]
    if case["op"] == "distill":
        entries = rows * case["top"] * 8.0
        by = fl = 0.0
        if case["way"] in ("forward", "step"):
            by += n * b + entries + p * rows * 20
            fl += 5.0 * n
        if case["way"] in ("backward", "step"):
            by += 2 * n * b + entries + rows * 20
            fl += 5.0 * n
        return {"bytes": by, "flops": fl}
    by = 2.0 * n * b + rows * (case["history"] * 8 + case["bias"] * 12 + 40) + (n / 8.0 if case["mask"] else 0)
    return {"bytes": by, "flops": 3.0 * n}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _activations(g, p, rows, hidden, dtype):
    """Rows as a residual stream has them: unlike channels (some far wider than the rest) and unlike tokens."""
    channel = torch.exp(0.5 * _normal(g, hidden))
    token = torch.exp(0.3 * _normal(g, p, rows, 1))
    return (_normal(g, p, rows, hidden) * channel * token).to(dtype)


def _cuts(case):
    """First vocabulary entry of every rank's shard, and the end: shards differ by one where p does not divide it."""
    p, v = case["p"], case["vocab"]
    return [v * r // p for r in range(p + 1)]


def _split(case, z):
    cut = _cuts(case)
    return [z[:, a:b].contiguous() for a, b in zip(cut, cut[1:])]


def _ragged(g, rows, mean):
    """Lengths from zero up (most short, few long) of about that mean, as offsets."""
    lengths = (mean * torch.exp(_normal(g, rows)) / 1.65).long()
    lengths = torch.where(torch.arange(rows, device="cuda") % 7 == 6, torch.zeros_like(lengths), lengths)
    return torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), lengths.cumsum(0)])


def _inputs(case, seed):
    """What both sides and the 64-bit values start from, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    p, rows, dt = case["p"], case["rows"], DTYPES[case["dtype"]]
    if case["op"] == "rms":
        hidden = case["hidden"]
        s = {"x": _activations(g, p, rows, hidden, dt),
             # data parallelism: every rank holds the same weights, a copy each
             "gamma": (1 + 0.2 * _normal(g, hidden)).to(DTYPES[case["wdtype"]]).repeat(p, 1)}
        if case["res"]:
            s["res"] = (3 * _activations(g, p, rows, hidden, torch.float32)).to(dt)
        if case["way"] != "forward":
            s["dy"] = (1e-3 * _normal(g, p, rows, hidden)).to(dt)
            if case["res"]:
                s["dh"] = (1e-3 * _normal(g, p, rows, hidden)).to(dt)
        if case["way"] == "backward":   # what the forward pass left
            s["h"] = (s.pop("x").float() + s.pop("res").float()).to(dt) if case["res"] else s.pop("x")
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + EPS)
        return s
    v = case["vocab"]
    z = 2.5 * _normal(g, rows, v)
    if case["op"] == "distill":
        k = case["top"]
        # the teacher agrees with the student by and large
        likely = torch.randint(0, v, (rows, 3), generator=g, device="cuda")
        z.scatter_add_(1, likely, 6 + 2 * _normal(g, rows, 3))
        teacher = z + 0.7 * _normal(g, rows, v)
        if case["masked"]:
            # a third of the positions allow about a tenth of the vocabulary, to both models
            deny = (_uniform(g, rows, v) > 0.1) & (torch.arange(rows, device="cuda") % 3 == 1)[:, None]
            deny.scatter_(1, teacher.topk(min(k, v), -1).indices, False)
            z.masked_fill_(deny, NOTHING)
            teacher.masked_fill_(deny, NOTHING)
        value, index = torch.topk(teacher / case["temp"], k, -1)
        logp = value - torch.logsumexp(teacher / case["temp"], -1, keepdim=True)
        del teacher
        if case["masked"]:   # padding has no entries
            index = torch.where((torch.arange(rows, device="cuda") % 16 == 15)[:, None], torch.full_like(index, -1), index)
        s = {"logits": _split(case, z.to(dt)), "idx": index.int(), "logp": logp.contiguous(), "dloss": (0.5 + _uniform(g, rows)) / rows}
        if case["way"] == "backward":
            s["stats"] = _plain_distill(case, s, "forward")["stats"][0].contiguous()
        return s
    offsets = _ragged(g, rows, case["history"])
    n = int(offsets[-1])
    # a text repeats its frequent tokens
    s = {"logits": _split(case, z.to(dt)), "offsets": offsets,
         "tokens": (v * _uniform(g, n) ** 3).long().clamp_max(v - 1),
         "prompt": ((offsets[1:] - offsets[:-1]).float() * _uniform(g, rows)).long(),
         "repetition": 1 + 0.3 * _uniform(g, rows), "presence": 0.5 * _uniform(g, rows), "frequency": 0.2 * _uniform(g, rows)}
    if case["bias"]:
        at = _ragged(g, rows, case["bias"])
        n = int(at[-1])
        s |= {"bias_offsets": at, "bias_idx": torch.randint(0, v, (n,), generator=g, device="cuda"), "bias": 4 * _normal(g, n)}
    if case["mask"]:
        # grammars allow from a handful of tokens to nearly all of them; one in five requests has none
        share = _uniform(g, rows, 1) ** 4
        share[::5] = 1.0
        s["mask"] = _packed(_uniform(g, rows, v) < share)
    return s


def _packed(allow):
    """Truth values as the bits of 32-bit words, the lowest first."""
    rows, v = allow.shape
    words = -(-v // 32)
    bits = torch.zeros(rows, words * 32, dtype=torch.int64, device=allow.device)
    bits[:, :v] = allow
    w = (bits.view(rows, words, 32) << torch.arange(32, device=allow.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


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
    g = x.unflatten(-1, (-1, group))
    top = torch.full((), 448.0, device=x.device)
    amax = g.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -110)
    codes = (g * torch.div(top.expand_as(amax), amax)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return (codes.float() * torch.div(amax, top.expand_as(amax))).flatten(-2)


def _plain_rms(c, s):
    out = {}
    if c["way"] == "backward":
        h, rstd = s["h"].float(), s["rstd"]
    else:
        h = s["x"].float()
        if c["res"]:
            out["h"] = (h + s["res"].float()).to(s["x"].dtype)
            h = out["h"].float()
        rstd = torch.rsqrt(h.square().mean(-1) + EPS)
        y = h * rstd[..., None] * s["gamma"].float()[:, None]
        out["y"] = _encode8(y, c["fp8"]).to(torch.bfloat16) if c["fp8"] else y.to(s["x"].dtype)
        out["rstd"] = rstd
    if c["way"] != "forward":
        dy = s["dy"].float()
        n = h * rstd[..., None]
        w = dy * s["gamma"].float()[:, None]
        dx = rstd[..., None] * (w - n * (w * n).mean(-1, keepdim=True))
        out["dx"] = (dx + s["dh"].float() if c["res"] else dx).to(s["dy"].dtype)
        over = float(c["p"]) if c["avg"] else 1.0
        out["dgamma"] = ((dy * n).sum((0, 1)) / over).to(s["gamma"].dtype).expand(c["p"], -1).contiguous()
    return out


def _counted(idx, v):
    """Which entries count: those in the vocabulary, an index's first one."""
    same = idx[:, :, None] == idx[:, None, :]
    later = torch.ones(same.shape[1:], dtype=torch.bool, device=idx.device).tril(-1)
    return (idx >= 0) & (idx < v) & ~(same & later).any(-1)


def _plain_distill(c, s, way):
    t = 1.0 / c["temp"]
    z = torch.cat(s["logits"], -1).float()
    rows, v = z.shape
    counts = _counted(s["idx"], v)
    # entries that do not count lie in one more column, of nothing
    z = torch.nn.functional.pad(z, (0, 1), value=NOTHING)
    at = torch.where(counts, s["idx"], torch.full_like(s["idx"], v)).long()
    # the loss, and what the teacher leaves to the others, are small differences of what the two models have: the
    # entries and the rows' sums are held in 64 bits
    zi = z.gather(1, at).double()
    lq = torch.where(counts, s["logp"], torch.full_like(s["logp"], NOTHING)).double()
    if way == "backward":
        stats = s["stats"].double()
    else:
        m = z.amax(-1)
        base = torch.where(m == NOTHING, torch.zeros_like(m), m)[:, None]
        inside = torch.exp((zi - base) * t).sum(-1)
        outside = torch.exp((z.scatter(1, at, NOTHING) - base) * t).sum(-1, dtype=torch.float64)
        third, fourth = torch.logsumexp(lq, -1), torch.zeros_like(inside)
        if c["tail"]:
            third, fourth = torch.log(outside), 1 - torch.exp(lq).sum(-1)
        empty = ~counts.any(-1) if c["tail"] else third == NOTHING
        third = torch.where(empty, torch.full_like(third, float("inf")), third)
        fourth = torch.where(empty, torch.zeros_like(fourth), fourth)
        stats = torch.stack([m.double(), torch.log(inside + outside), third, fourth], -1)
    m, log_s, third, fourth = stats[:, 0:1], stats[:, 1:2], stats[:, 2:3], stats[:, 3:4]
    empty = third == float("inf")
    base = torch.where(m == NOTHING, torch.zeros_like(m), m)
    if not c["tail"]:
        lq = lq - third
    q = torch.exp(lq)
    lp = (zi - base) * t - log_s
    out = {}
    if way != "backward":
        loss = torch.where(q > 0, q * (lq - lp), torch.zeros_like(q)).sum(-1, keepdim=True)
        if c["tail"]:
            loss = loss + torch.where(fourth > 0, fourth * (torch.log(fourth) - (third - log_s)), torch.zeros_like(fourth))
        loss = torch.where(empty, torch.zeros_like(loss), loss)[:, 0]
        each = lambda x: x.float().expand(c["p"], *x.shape).contiguous()  # noqa: E731  every rank gets the results
        out = {"stats": each(stats), "loss": each(loss)}
        if way == "forward":
            return out
    if c["tail"]:
        whole = (1 - fourth).clamp_min(1)
        mine = whole * torch.exp(lp) - q
        share, of = third.float(), whole * torch.exp(third - log_s) - fourth.clamp_min(0)
    else:
        mine = torch.exp(lp) - q
        share, of = log_s.float(), torch.ones_like(log_s)
    dz = (torch.exp((z - base.float()) * t - share) * of.float()).scatter(1, at, mine.float())[:, :v] * (s["dloss"][:, None] * t)
    dz = torch.where(empty | (m == NOTHING), torch.zeros_like(dz), dz)
    out["dlogits"] = _split(c, dz.to(s["logits"][0].dtype))
    return out


def _rows_of(offsets, n):
    """The row that each of n entries belongs to."""
    return torch.searchsorted(offsets[1:].contiguous(), torch.arange(n, device=offsets.device), right=True)


def _plain_adjust(c, s):
    z = torch.cat(s["logits"], -1).float()
    rows, v = z.shape
    n = s["tokens"].numel()
    row = _rows_of(s["offsets"], n)
    at = row * v + s["tokens"]
    answer = torch.arange(n, device=z.device) >= (s["offsets"][:-1] + s["prompt"])[row]
    count = torch.zeros(rows * v, device=z.device).index_add_(0, at, answer.float()).view(rows, v)
    seen = torch.zeros(rows * v, dtype=torch.bool, device=z.device).index_fill_(0, at, True).view(rows, v)
    per = lambda k: s[k][:, None]  # noqa: E731
    z = torch.where(seen, torch.where(z > 0, z / per("repetition"), z * per("repetition")), z)
    z = z - count * per("frequency") - (count > 0) * per("presence")
    if c["bias"]:
        n = s["bias"].numel()
        at = _rows_of(s["bias_offsets"], n) * v + s["bias_idx"]
        # an index's first entry counts
        first = torch.full((rows * v,), n, dtype=torch.int64, device=z.device).scatter_reduce_(0, at, torch.arange(n, device=z.device), "amin")
        z = z + torch.nn.functional.pad(s["bias"], (0, 1))[first].view(rows, v)
    if c["mask"]:
        bits = (s["mask"][:, :, None] >> torch.arange(32, dtype=torch.int32, device=z.device)) & 1
        z = torch.where(bits.flatten(1)[:, :v] > 0, z, torch.full_like(z, NOTHING))
    return {"out": _split(c, z.to(s["logits"][0].dtype))}


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "rms":
        return _plain_rms(c, state)
    if c["op"] == "distill":
        return _plain_distill(c, state, c["way"])
    return _plain_adjust(c, state)


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

    each = lambda t: None if t is None else list(t)  # noqa: E731  a rank's buffers by rank
    if c["op"] == "rms":
        hidden, dt, wt = c["hidden"], DTYPES[c["dtype"]], DTYPES[c["wdtype"]]
        h, rstd = s.get("h"), s.get("rstd")
        if c["way"] != "backward":
            rstd = out["rstd"] = new(p, rows)
            h = s["x"]
            if c["res"]:
                h = out["h"] = torch.empty_like(h)
            kept = each(h) if c["res"] else None
            if c["fp8"]:
                rows8 = new(p, rows, coll.coll_ckpt8_row_bytes(hidden, c["fp8"]), dtype=torch.uint8)
                out["y"] = new(p, rows, hidden, dtype=torch.bfloat16)
                calls.append(coll.coll_rmsnorm_fp8(each(s["x"]), each(s["gamma"]), each(rows8), hidden, c["fp8"], eps=EPS,
                                                   residual=each(s.get("res")), h=kept, rstd=each(rstd), defer=True))
                # the receiver's side
                calls.append(coll.coll_ckpt8_load(each(rows8), each(out["y"]), hidden, c["fp8"], defer=True))
            else:
                out["y"] = torch.empty_like(s["x"])
                calls.append(coll.coll_rmsnorm(each(s["x"]), each(s["gamma"]), each(out["y"]), hidden, eps=EPS, residual=each(s.get("res")),
                                               h=kept, rstd=each(rstd), defer=True))
        if c["way"] != "forward":
            out |= {"dx": new(p, rows, hidden, dtype=dt), "dgamma": new(p, hidden, dtype=wt)}
            ws = new(coll.coll_rmsnorm_workspace_bytes(p, rows, hidden), dtype=torch.uint8)
            calls.append(coll.coll_rmsnorm_backward(each(s["dy"]), each(h), each(rstd), each(s["gamma"]), each(out["dx"]), each(out["dgamma"]), ws,
                                                    hidden, op=coll.COLL_AVG if c["avg"] else coll.COLL_SUM, dh=each(s.get("dh")), defer=True))
    elif c["op"] == "distill":
        z, kind = s["logits"], coll.COLL_DISTILL_TAIL if c["tail"] else coll.COLL_DISTILL_RENORM
        stats, t = s.get("stats"), 1.0 / c["temp"]
        if c["way"] != "backward":
            out = {"stats": new(p, rows, 4), "loss": new(p, rows)}
            stats = out["stats"][0]
            ws = new(coll.coll_vocab_distill_workspace_bytes(rows, [x.shape[1] for x in z], c["top"]), dtype=torch.uint8)
            calls.append(coll.coll_vocab_distill(z, s["idx"], s["logp"], each(out["stats"]), each(out["loss"]), ws, kind=kind, inv_temp=t, defer=True))
        if c["way"] != "forward":
            out["dlogits"] = [torch.empty_like(x) for x in z]
            calls.append(coll.coll_vocab_distill_backward(z, s["idx"], s["logp"], stats, s["dloss"], out["dlogits"], kind=kind, inv_temp=t, defer=True))
    else:
        out["out"] = [torch.empty_like(x) for x in s["logits"]]
        calls.append(coll.coll_vocab_adjust(s["logits"], out["out"], tokens=s["tokens"], offsets=s["offsets"], prompt=s["prompt"],
                                            repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                                            bias_idx=s.get("bias_idx"), bias=s.get("bias"), bias_offsets=s.get("bias_offsets"),
                                            mask=s.get("mask"), defer=True))
    s["calls"], s["out"] = calls, out


def _run_own(s):
    [call() for call in s["calls"]]
    return s["out"]


# ----------------------------------------------------------------------------
# The values in 64 bits
# ----------------------------------------------------------------------------

def _kept8(y, group):
    """What a group's 8-bit codes stand for: the nearest e4m3 number (ties to even, 448 at most) of each value over
    its group's scale, by the spacing of those numbers, 2^(e-3) in [2^e, 2^(e+1)) and 2^-9 below 2^-6; the scale is
    an fp32 number."""
    g = y.unflatten(-1, (y.shape[-1] // group, group))
    scale = (g.abs().max(-1, keepdim=True).values.clamp_min(2.0 ** -110) / 448).float().double()
    v = g / scale
    step = torch.ldexp(torch.ones_like(v), torch.frexp(v)[1].clamp_min(-5) - 4)
    return ((torch.round(v / step) * step).clamp(-448, 448) * scale).flatten(-2)


def _exact_rms(c, s):
    def one(r):
        gamma = s["gamma"][r].double()
        got = {}
        if c["way"] == "backward":
            h, rstd = s["h"][r].double(), s["rstd"][r].double()
        else:
            h = s["x"][r].double()
            if c["res"]:
                got["h"] = h + s["res"][r].double()
                h = got["h"].to(s["x"].dtype).double()   # the stream's type is part of the operator
            rstd = (torch.linalg.vector_norm(h, dim=1) ** 2 / h.shape[1] + EPS) ** -0.5
            y = torch.einsum("ij,i,j->ij", h, rstd, gamma)
            got["y"], got["rstd"] = _kept8(y, c["fp8"]) if c["fp8"] else y, rstd
        if c["way"] != "forward":
            dy = s["dy"][r].double()
            w = dy * gamma
            dot = torch.einsum("ij,ij->i", w, h)
            got["dx"] = w * rstd[:, None] - h * (dot * rstd ** 3 / h.shape[1])[:, None]
            if c["res"]:
                got["dx"] += s["dh"][r].double()
            got["dgamma"] = torch.einsum("ij,ij,i->j", dy, h, rstd)
        return got

    ranks = [one(r) for r in range(c["p"])]
    out = {k: torch.stack([g[k] for g in ranks]) for k in ranks[0]}
    if "dgamma" in out:
        out["dgamma"] = (out["dgamma"].sum(0) / (c["p"] if c["avg"] else 1)).repeat(c["p"], 1)
    return out


def _exact_distill(c, s):
    t, v = 1.0 / c["temp"], c["vocab"]
    step = max(1, int(4e7) // v)

    def some(a):
        z = torch.hstack([x[a:a + step] for x in s["logits"]]).double()
        idx, lt = s["idx"][a:a + step].long(), s["logp"][a:a + step].double()
        n, k = idx.shape
        # the teacher's probabilities by vocabulary entry, from the last to the first so that the first one stays
        lq = torch.full((n, v + 1), NOTHING, dtype=torch.float64, device=z.device)
        among = torch.zeros(n, v + 1, dtype=torch.bool, device=z.device)
        line = torch.arange(n, device=z.device)
        for i in reversed(range(k)):
            at = torch.where((idx[:, i] >= 0) & (idx[:, i] < v), idx[:, i], v)
            lq[line, at] = lt[:, i]
            among[line, at] = True
        lq, among = lq[:, :v], among[:, :v]
        logp = torch.log_softmax(z * t, 1)
        m = z.max(1).values
        stats = [m, torch.logsumexp((z - m[:, None]) * t, 1)]
        g = s["dloss"][a:a + step].double()[:, None] * t
        if c["tail"]:
            empty = ~among.any(1)
            q, inside = lq.exp(), torch.where(among, logp.exp(), 0.0).sum(1, keepdim=True)
            rest = 1 - q.sum(1, keepdim=True)
            ltail = torch.logsumexp(torch.where(among, NOTHING, (z - m[:, None]) * t), 1, keepdim=True)
            ltot = stats[1][:, None]
            loss = torch.where(q > 0, q * (lq - logp), 0.0).sum(1) + torch.where(rest > 0, rest * (rest.clamp_min(1e-300).log() - ltail + ltot), 0.0)[:, 0]
            whole = q.sum(1, keepdim=True) + rest.clamp_min(0)
            others = torch.softmax(torch.where(among, NOTHING, z * t), 1)
            dz = torch.where(among, whole * logp.exp() - q, others * (whole * (1 - inside) - rest.clamp_min(0)))
            stats += [ltail[:, 0], rest[:, 0]]
        else:
            total = torch.logsumexp(lq, 1, keepdim=True)
            empty = total[:, 0] == NOTHING
            q = torch.softmax(torch.where(empty[:, None], 0.0, lq), 1)
            loss = torch.where(q > 0, q * (lq - total - logp), 0.0).sum(1)
            dz = logp.exp() - q
            stats += [total[:, 0], torch.zeros_like(m)]
        stats[2] = torch.where(empty, float("inf"), stats[2])
        stats[3] = torch.where(empty, 0.0, stats[3])
        return torch.stack(stats, 1), torch.where(empty, 0.0, loss), torch.where(empty[:, None], 0.0, dz * g)

    parts = [some(a) for a in range(0, c["rows"], step)]
    stats, loss, dz = (torch.cat([q[i] for q in parts]) for i in range(3))
    out = {}
    if c["way"] != "backward":
        out = {"stats": stats.repeat(c["p"], 1, 1), "loss": loss.repeat(c["p"], 1)}
    if c["way"] != "forward":
        out["dlogits"] = _split(c, dz)
    return out


def _exact_adjust(c, s):
    z = torch.hstack(s["logits"]).double()
    rows, v = z.shape
    words = s["mask"].long() if c["mask"] else None
    ends = s["offsets"].tolist()
    for r in range(rows):
        history = s["tokens"][ends[r]:ends[r + 1]]
        count = torch.bincount(history[int(s["prompt"][r]):], minlength=v).double()
        was = torch.bincount(history, minlength=v) > 0
        rho = s["repetition"][r].double()
        z[r] *= torch.where(was, torch.where(z[r] > 0, 1 / rho, rho), 1.0)
        z[r] -= count * s["frequency"][r].double() + torch.sign(count) * s["presence"][r].double()
    if c["bias"]:
        n = s["bias"].numel()
        row = torch.repeat_interleave(torch.arange(rows, device=z.device), s["bias_offsets"].diff())
        order = torch.argsort(row * v + s["bias_idx"], stable=True)
        key = (row * v + s["bias_idx"])[order]
        lead = torch.ones(n, dtype=torch.bool, device=z.device)
        lead[1:] = key[1:] != key[:-1]
        z.view(-1)[key[lead]] += s["bias"][order][lead].double()
    if c["mask"]:
        j = torch.arange(v, device=z.device)
        z[((words[:, j // 32] >> (j % 32)) & 1) == 0] = NOTHING
    return {"out": _split(c, z)}


def exact(case, seed):
    s = _inputs(case, seed)
    return {"rms": _exact_rms, "distill": _exact_distill, "adjust": _exact_adjust}[case["op"]](case, s)
