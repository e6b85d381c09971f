"""Penalties, biases and masks in each of the five run shapes that the launch
chooses from, on the GPU against the float64 oracle: shards of several runs,
marks on the first and the last entries of each.  Which shape a size takes is
checked on the CPU, by recorded launches."""
import numpy as np
import pytest

from gpu_util import BF16, F32
from test_abi_cpu import host_only
from test_gpu_adjust import Case, check
from test_gpu_token_ops import coll, rng, shards  # noqa: F401
from test_token_abi_cpu import recorded

ELEMS = {F32: 4, BF16: 8}
# lanes, units to a lane, rows, tokens to a row (at least, and below), and shards in units of 16 bytes: full runs, a
# second and a third run, one of a unit, none; each of these is one entry longer or shorter in turn
SHAPES = {
    "256x1": (256, 1, 3, (0, 1900), (512, 256, 0, 640, 1)),
    "512x1": (512, 1, 3, (2100, 4000), (1024, 512, 0, 1100, 1)),
    "128x2": (128, 2, 180, (0, 300), (256, 255, 0, 256, 1)),
    "256x4": (256, 4, 110, (0, 300), (2048, 1024, 0, 1500, 1)),
    "512x4": (512, 4, 90, (2100, 2600), (4096, 2048, 0, 2500, 1)),
    # short shards take the longest runs where they are few
    "512x4 short": (512, 4, 140, (2100, 2300), (1024, 1000, 0, 1, 1)),
}
# whether a shape's widths end one entry past a unit, or one before it
ENDS = [0, 1, -1]


def widths_of(name, dtype, end):
    # (a shard may not outgrow the shape's runs where these must hold it whole)
    most = SHAPES[name][4][0] * ELEMS[dtype] if name in ("128x2", "512x4 short") else 1 << 30
    return [min(max(0, u * ELEMS[dtype] + end * (u > 0)), most) for u in SHAPES[name][4]]


@host_only
@pytest.mark.parametrize("name", SHAPES)
def test_sizes_take_their_shape(tmp_path, name):
    lanes, units, rows, (lo, hi), _ = SHAPES[name]
    calls, want = [], []
    for dtype in (F32, BF16):
        for end in ENDS:
            w = widths_of(name, dtype, end)
            run = lanes * units * ELEMS[dtype]
            one = f"_i64(*{w})"
            for tokens in {lo * rows, (hi - 1) * rows}:
                what = f"__import__('test_adjust_abi_cpu').by(tokens=b.one(), ntokens={tokens}, offsets=b.one())"
                calls.append(f"L.coll_vocab_adjust(b({len(w)}), {one}, {one}, {what}, b({len(w)}), {one}, {len(w)}, {rows}, {dtype}, None)")
                spread = 8 if rows >= 64 else 1
                want.append([(-(-rows // spread) * spread * sum(-(-x // run) for x in w), lanes)])
    found = recorded(tmp_path, calls)
    assert [[(g[0], b[0]) for g, b in launched] for launched in found] == want


@pytest.mark.gpu
@pytest.mark.parametrize("end", ENDS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", SHAPES)
def test_marks_on_every_run(coll, name, dtype, end):  # noqa: F811
    import torch
    lanes, units, rows, (lo, hi), _ = SHAPES[name]
    widths = widths_of(name, dtype, end)
    run, g = lanes * units * ELEMS[dtype], rng(86, list(SHAPES).index(name), dtype, end + 1)
    cuts = np.cumsum([0, *widths])
    v = int(cuts[-1])
    zs, ze = shards(g.normal(0, 3, (rows, v)), [int(x) for x in cuts], dtype, 3, 1)
    edges = []                                                # the runs' first and last entries, and units' around them
    for a, b in zip(cuts, cuts[1:]):
        for at in range(int(a), int(b), run):
            last = min(at + run, int(b)) - 1
            edges += [j for j in (at, at + 1, last - ELEMS[dtype], last - 1, last) if a <= j < b]
    edges = np.array(sorted(set(edges)))
    longest = hi - 1 - 2 * len(edges)
    c = Case(g, rows, v, lengths=(max(lo, 0), (max(lo, 0) + longest) // 2, longest) if lo else (0, 1, 30, longest // 2))
    for r in range(rows):
        if r % 4 == 0:                                        # once in the prompt and twice after it
            c.history[r] = np.concatenate([edges, c.history[r], edges, edges])[:hi - 1 if lo else None]
            c.prompt[r] = len(edges)
        elif r % 4 == 1:
            c.history[r] = np.concatenate([c.history[r], edges])
            c.biases[r] = c.biases[r][:50] + [(int(j), np.float32(3.0)) for j in edges]
        elif r % 4 == 2:
            c.history[r], c.biases[r] = (c.history[r] if lo else c.history[r][:0]), [(int(j), np.float32(-2.0)) for j in edges]
        else:
            c.biases[r] = []
    c.allow[1:3] = True
    tokens = sum(len(h) for h in c.history)
    assert lo * rows <= tokens < hi * rows                    # the shape that the CPU test checks
    want, size = c.want(ze)
    by = c.device(1)
    out = [torch.full((rows, w), float("nan"), dtype=zs[0].dtype, device="cuda") for w in widths]
    coll.coll_vocab_adjust(zs, out, **by)
    check(out, want, size, dtype, "apart")
    coll.coll_vocab_adjust(zs, zs, **by)
    assert all(torch.equal(a, b) for a, b in zip(out, zs))
