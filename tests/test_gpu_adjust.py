"""Penalties, biases and masks on sharded logits on the GPU against the float64
oracle.  Tolerances as in test_gpu_token_ops: U is half a step of fp32, HALF of
the result's type."""
import numpy as np
import pytest

from gpu_util import BF16, F32
from oracle import token_ops
from test_gpu_token_ops import HALF, LP_SHAPES, TINY, U, close, coll, dev, f32, host, rng, shards, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


def cuda(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def packed(allow, pad=0):
    """Device words of truth values, `pad` words of ones after each row."""
    rows, v = allow.shape
    words = -(-v // 32)
    bits = np.ones((rows, words * 32), dtype=np.uint8)        # bits past the vocabulary are not looked at
    bits[:, :v] = allow
    w = np.packbits(bits, axis=1, bitorder="little").view("<u4")
    full = np.full((rows, words + pad), 0xFFFFFFFF, dtype=np.uint32)
    full[:, :words] = w
    return cuda(full.view(np.int32), np.int32)[:, :words]


def ragged(lists, dtype):
    return cuda(np.concatenate([np.asarray(x, dtype=dtype) for x in lists]) if len(lists) else np.zeros(0), dtype), \
        cuda(np.cumsum([0, *[len(x) for x in lists]]), np.int64)


class Case:
    """Everything that may be listed, for rows of v entries; lengths: the histories' and the lists'."""

    def __init__(self, g, rows, v, lengths=(0, 1, 3, 40, 700), longest=None):
        tokens = lambda n: np.where(g.random(n) < 0.05, g.choice([-1, v, v + 5, 2 ** 40, -2 ** 63], n), (v * g.random(n) ** 2).astype(np.int64))  # noqa: E731
        self.history = [tokens(int(g.choice(lengths))) for _ in range(rows)]
        if longest:
            self.history[rows // 2] = tokens(longest)
        self.prompt = [int(g.integers(-1, len(h) + 2)) for h in self.history]
        self.repetition, self.presence, self.frequency = [g.uniform(*r, rows).astype(np.float32) for r in ((0.7, 1.5), (-0.5, 1.0), (-0.1, 0.3))]
        self.biases = [[(int(j), np.float32(b)) for j, b in zip(tokens(n), g.normal(0, 5, n))] for n in g.choice(lengths, rows)]
        self.allow = g.random((rows, v)) < g.random((rows, 1))
        self.allow[0] = False                                 # a mask that leaves nothing

    def device(self, pad=0):
        t, to = ragged(self.history, np.int64)
        bi, bo = ragged([[j for j, _ in b] for b in self.biases], np.int64)
        bv, _ = ragged([[x for _, x in b] for b in self.biases], np.float32)
        c = lambda x: cuda(x, np.float32)  # noqa: E731
        return dict(tokens=t, offsets=to, prompt=cuda(self.prompt, np.int64), repetition=c(self.repetition), presence=c(self.presence),
                    frequency=c(self.frequency), bias_idx=bi, bias=bv, bias_offsets=bo, mask=packed(self.allow, pad))

    def want(self, z, only=None):
        k = dict(history=self.history, prompt=self.prompt, repetition=self.repetition, presence=self.presence, frequency=self.frequency,
                 biases=self.biases, allow=self.allow)
        return token_ops.adjust(z, **{n: x for n, x in k.items() if only is None or n in only})


def check(got, want, size, dtype, what):
    # a quotient or product, a fused product and sum, a difference, a sum: each off by U of a term or of their sum
    close(np.concatenate([host(x) for x in got], 1), want, HALF[dtype] * np.abs(np.where(np.isfinite(want), want, 0.0)) + 5 * U * size + TINY, what)


@pytest.mark.parametrize("rows,cuts,dtype,pad,off,t,top", LP_SHAPES)
def test_all_of_it(coll, rows, cuts, dtype, pad, off, t, top):
    import torch
    g = rng(80, rows, len(cuts), cuts[-1], dtype)
    v = cuts[-1]
    zs, ze = shards(g.normal(0, 3, (rows, v)), cuts, dtype, pad, off)
    c = Case(g, rows, v, lengths=(0, 1, 3, 40) if rows > 1000 else (0, 1, 3, 40, 700, 5000))
    want, size = c.want(ze)
    by = c.device(pad)
    out = [torch.full((rows, b - a), float("nan"), dtype=zs[0].dtype, device="cuda") for a, b in zip(cuts, cuts[1:])]
    coll.coll_vocab_adjust(zs, out, **by)
    check(out, want, size, dtype, "apart")
    full = torch.full((rows, v + 3), float("nan"), dtype=zs[0].dtype, device="cuda")
    slices = [full[:, a:b] for a, b in zip(cuts, cuts[1:])]
    coll.coll_vocab_adjust(zs, slices, **by)
    assert all(torch.equal(a, b) for a, b in zip(out, slices)) and torch.isnan(full[:, v:].float()).all()
    coll.coll_vocab_adjust(zs, zs, **by)
    assert all(torch.equal(a, b) for a, b in zip(out, zs))
    if pad:                                                   # what lies between the rows stays
        assert all(torch.isnan(z.as_strided((1,), (1,), z.storage_offset() + z.shape[1]).float()).all() for z in zs)


PARTS = [("history", "repetition"), ("history", "prompt", "repetition"), ("history", "presence"), ("history", "prompt", "frequency"), ("biases",), ("allow",),
         ("biases", "allow"), ("history", "presence", "frequency", "biases"), ("history",), ()]


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_each_part_alone(coll, parts, dtype):
    import torch
    g = rng(81, len(parts), dtype)
    rows, cuts = 6, [0, 1000, 1003, 4001]
    zs, ze = shards(g.normal(0, 3, (rows, 4001)), cuts, dtype, 1, 1)
    c = Case(g, rows, 4001)
    names = {"history": ("tokens", "offsets"), "biases": ("bias_idx", "bias", "bias_offsets"), "allow": ("mask",)}
    by = {k: x for k, x in c.device().items() if any(k in names.get(p, (p,)) for p in parts)}
    out = [torch.full_like(z, float("nan")) for z in zs]
    coll.coll_vocab_adjust(zs, out, **by)
    check(out, *c.want(ze, parts), dtype, parts)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("longest,list_length", [(32767, 3), (32768, 3), (100000, 40), (5, 65535), (5, 65536), (40000, 70000),
                                                  (1048575, 2), (1048576, 2), (5, 2047), (5, 2048)])
@pytest.mark.parametrize("rows", [3, 300])
def test_long_histories_and_lists(coll, longest, list_length, rows, dtype):
    """Either side of what a table of one word an entry holds, in runs of either length."""
    import torch
    g = rng(82, longest, list_length, rows, dtype)
    v = 20011
    zs, ze = shards(g.normal(0, 3, (rows, v)), [0, 9000, v], dtype, 0, 1)
    c = Case(g, rows, v, longest=longest)
    c.history[0] = np.full(longest, 17)                       # one token, all along
    c.biases[rows // 2] = [(int(j), np.float32(b)) for j, b in zip(g.integers(0, v, list_length), g.normal(0, 5, list_length))]
    c.biases[1] = [(5, np.float32(1.0))] + [(5, np.float32(9.0))] * (list_length - 1)
    out = [torch.full_like(z, float("nan")) for z in zs]
    by = c.device()
    coll.coll_vocab_adjust(zs, out, **by)
    want, size = c.want(ze)
    check(out, want, size, dtype, "out")
    coll.coll_vocab_adjust(zs, zs, **by)
    assert all(torch.equal(a, b) for a, b in zip(out, zs))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("longest,list_length", [(131071, 16383), (131072, 16383), (65535, 16384), (65536, 16384), (1048576, 2047)])
def test_one_row_of_a_long_history_and_a_long_list(coll, longest, list_length, dtype):
    """Either side of what a word holds of both: one token all along, in the answer and in prompt and answer, and biased."""
    import torch
    g = rng(83, longest, list_length, dtype)
    rows, v = 3, 2003
    zs, ze = shards(g.normal(0, 3, (rows, v)), [0, 900, v], dtype, 0, 1)
    c = Case(g, rows, v)
    for r in (1, 2):
        c.history[r] = np.full(longest, 17 + 1000 * (r == 2))
        c.prompt[r] = r - 1
        c.biases[r] = [(int(j), np.float32(b)) for j, b in zip(g.integers(0, v, list_length), g.normal(0, 5, list_length))]
        c.biases[r][list_length - 1] = (1900 + r, np.float32(2.0))
    out = [torch.full_like(z, float("nan")) for z in zs]
    coll.coll_vocab_adjust(zs, out, **c.device())
    check(out, *c.want(ze), dtype, "out")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("widths", [(526, 2048, 1), (2047, 1030, 0, 9), (2049, 8192, 3), (4100, 8191), (8193, 700), (16384, 16385, 5)])
def test_shards_and_the_lengths_of_runs(coll, widths, dtype):
    """Shards that end with a run of each length, before or behind one."""
    import torch
    g = rng(84, len(widths), widths[0], dtype)
    widths = [w if dtype == BF16 else w // 2 + w % 2 for w in widths]
    rows, cuts = 140, np.cumsum([0, *widths])
    v = int(cuts[-1])
    zs, ze = shards(g.normal(0, 3, (rows, v)), list(cuts), dtype, 3, 1)
    c = Case(g, rows, v, lengths=(0, 1, 30, 600))
    for r in range(0, rows, 2):                               # every run's last entries
        c.history[r] = np.concatenate([c.history[r], cuts[1:] - 1])
        c.biases[r] = c.biases[r] + [(int(x) - 1, np.float32(3.0)) for x in cuts[1:]]
    out = [torch.full_like(z, float("nan")) for z in zs]
    coll.coll_vocab_adjust(zs, out, **c.device())
    check(out, *c.want(ze), dtype, "out")


def test_edge_values(coll):
    """Masked entries and NaN, infinities, zeros of either sign and infinite biases."""
    import torch
    v = 50
    z = np.zeros((1, v))
    z[0, :8] = [np.nan, np.nan, np.inf, -np.inf, -0.0, 0.0, 3.0, -3.0]
    z[0, 8:16] = z[0, :8]
    zs, ze = shards(z, [0, 20, v], F32)
    allow = np.ones((1, v), dtype=bool)
    allow[0, [0, 40]] = False
    history = [list(range(8)) + [20]]
    biases = [[(9, np.float32(1.0)), (11, np.float32(5.0)), (14, -np.float32(np.inf)), (15, np.float32(np.inf)), (49, np.float32(2.0))]]
    by = dict(zip(("tokens", "offsets"), ragged(history, np.int64))) | dict(zip(("bias_idx", "bias_offsets"), ragged([[j for j, _ in biases[0]]], np.int64)))
    by |= dict(bias=ragged([[b for _, b in biases[0]]], np.float32)[0], mask=packed(allow), repetition=cuda([2.0], np.float32), presence=cuda([0.5], np.float32))
    coll.coll_vocab_adjust(zs, zs, **by)
    got = np.concatenate([host(x) for x in zs], 1)[0]
    want, _ = token_ops.adjust(ze, history, None, [2.0], [0.5], None, biases, allow)
    assert np.array_equal(got, want[0], equal_nan=True)
    assert got[0] == -np.inf and np.isnan(got[1]) and got[2] == np.inf and got[3] == -np.inf and got[6] == 1.0 and got[7] == -6.5 and got[14] == -np.inf


def test_offsets_that_are_none_stay_in_bounds(coll):
    """Negative, falling and too large offsets: nothing outside the lists is read, and the other rows are right."""
    import torch
    g = rng(83)
    rows, v = 6, 3000
    zs, ze = shards(g.normal(0, 3, (rows, v)), [0, v], F32)
    tokens = g.integers(0, v, 100)
    offsets = [0, 10, 5, 2 ** 62, -7, 90, 100]                # rows 0 and 5 are sound
    out = [torch.full_like(zs[0], float("nan"))]
    bias = g.normal(0, 1, 100).astype(np.float32)
    coll.coll_vocab_adjust(zs, out, tokens=cuda(tokens, np.int64), offsets=cuda(offsets, np.int64), frequency=cuda([1.0] * rows, np.float32),
                           bias_idx=cuda(tokens, np.int64), bias=cuda(bias, np.float32), bias_offsets=cuda(offsets, np.int64))
    parts = [tokens[:10], [], tokens[5:], [], tokens[:90], tokens[90:]]
    pairs = [list(zip(tokens[:10], bias[:10])), [], list(zip(tokens[5:], bias[5:])), [], list(zip(tokens[:90], bias[:90])), list(zip(tokens[90:], bias[90:]))]
    check(out, *token_ops.adjust(ze, parts, None, None, None, [1.0] * rows, pairs), F32, "out")


def test_rows_of_no_history_and_empty_lists(coll):
    import torch
    g = rng(84)
    zs, ze = shards(g.normal(0, 3, (4, 100)), [0, 100], BF16)
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    zero = torch.zeros(5, dtype=torch.int64, device="cuda")
    out = [torch.full_like(zs[0], float("nan"))]
    coll.coll_vocab_adjust(zs, out, tokens=none, offsets=zero, repetition=torch.ones(4, device="cuda"), bias_idx=none,
                           bias=torch.zeros(0, device="cuda"), bias_offsets=zero)
    assert torch.equal(out[0], zs[0])


def test_rows_past_2_31_elements(coll):
    import torch
    g = rng(85)
    v, pick = 131072, [0, 16383, 16384, 17000]
    rows = pick[-1] + 1
    z = torch.zeros(rows, v, dtype=torch.bfloat16, device="cuda")
    small, ze = dev(g.normal(0, 3, (4, v)), BF16)
    z[pick] = small
    c = Case(g, 4, v)
    c.allow[:] = g.random((4, v)) < 0.9
    lists, pairs = [[] for _ in range(rows)], [[] for _ in range(rows)]
    per = {k: np.full(rows, d, dtype=np.float32) for k, d in (("repetition", 1.0), ("presence", 0.0), ("frequency", 0.0))}
    prompt = np.zeros(rows, dtype=np.int64)
    for i, r in enumerate(pick):
        lists[r], pairs[r], prompt[r] = c.history[i], c.biases[i], c.prompt[i]
        for k in per:
            per[k][r] = getattr(c, k)[i]
    t, to = ragged(lists, np.int64)
    bi, bo = ragged([[j for j, _ in b] for b in pairs], np.int64)
    bv, _ = ragged([[x for _, x in b] for b in pairs], np.float32)
    mask = torch.full((rows, v // 32), -1, dtype=torch.int32, device="cuda")
    mask[pick] = packed(c.allow)
    coll.coll_vocab_adjust([z], [z], tokens=t, offsets=to, prompt=cuda(prompt, np.int64), bias_idx=bi, bias=bv, bias_offsets=bo, mask=mask,
                           **{k: cuda(x, np.float32) for k, x in per.items()})
    check([z[pick]], *c.want(ze), BF16, "picked rows")
    z[pick] = 0
    assert not bool(z.view(torch.int16).any())
