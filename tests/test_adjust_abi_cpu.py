"""Host-side checks of the entry point of penalties, biases and masks: refusals,
overlaps, empty calls, launches of the largest shapes, none of which reaches the
device."""
import ctypes

import pytest

import collective_communication_primitives_coll_amd as coll
from test_abi_cpu import _arr, host_only
from test_token_abi_cpu import AL, BF16, F32, I32, INV, OK, P, U8, UNS, Bufs, DeviceTensor, _i64, recorded


def by(**k):
    s = coll.coll_adjust_t()
    for name, x in k.items():
        setattr(s, name, x)
    return ctypes.byref(s)


def test_no_rows_is_ok_without_pointers():
    ld = _i64(8, 8, 8, 8)
    assert coll.lib().coll_vocab_adjust(None, ld, ld, by(), None, ld, P, 0, BF16, None) == OK


@host_only
def test_refusals():
    L, b = coll.lib(), Bufs()
    z, out = b(), b()
    t, to, pr, re, ps, fr, bi, bv, bo, m = [b.one() for _ in range(10)]
    vocab, ld = _i64(100, 100, 100, 50), _i64(100, 100, 128, 50)
    whole = dict(tokens=t, ntokens=20, offsets=to, prompt=pr, repetition=re, presence=ps, frequency=fr, bias_idx=bi, bias=bv, nbias=9,
                 bias_offsets=bo, mask=m, mask_ld=11)

    def f(z=z, ld=ld, vocab=vocab, out=out, old=ld, p=P, rows=9, dt=BF16, what=None, **k):
        return L.coll_vocab_adjust(z, ld, vocab, by(**{**whole, **k}) if what is None else what, out, old, p, rows, dt, None)
    hole, _k = _arr([z[0], 0, z[2], z[3]])
    assert f(p=0) == INV and f(p=65) == INV and f(dt=U8) == INV and f(dt=I32) == UNS
    assert L.coll_vocab_adjust(z, ld, vocab, None, out, ld, P, 9, BF16, None) == INV
    assert f(ld=None) == INV and f(vocab=None) == INV and f(old=None) == INV and f(ld=_i64(99, 100, 100, 50)) == INV and f(old=_i64(100, 100, 99, 50)) == INV
    assert f(vocab=_i64(-1, 2, 2, 2)) == INV and f(vocab=_i64(0, 0, 0, 0)) == INV
    big = _i64(1 << 30, 1 << 30, 1 << 30, 1 << 30)
    assert f(vocab=big, ld=big, old=big, mask=None) == UNS
    assert f(z=None) == INV and f(z=hole) == INV and f(out=None) == INV and f(out=hole) == INV and f(z=b(off=1)) == INV and f(out=b(off=1)) == INV
    for rows in (1 << 58, 1 << 60, 1 << 62, (1 << 64) - 1):
        assert f(rows=rows) == INV
    assert f(ntokens=1 << 31) == UNS and f(nbias=1 << 31) == UNS
    assert f(mask_ld=10) == INV and f(mask_ld=-1) == INV and f(mask_ld=1 << 62) == INV
    # penalties want a history, biases their lists, lists their entries
    assert f(offsets=None) == INV and f(bias_offsets=None) == INV and f(tokens=None) == INV and f(bias=None) == INV and f(bias_idx=None) == INV
    for k in ("tokens", "prompt", "repetition", "presence", "frequency"):
        assert f(what=by(**{k: whole[k]})) == INV
    assert f(what=by(ntokens=3)) == INV and f(what=by(nbias=3)) == INV and f(what=by(bias=bv)) == INV
    for k in ("tokens", "offsets", "prompt", "bias_idx", "bias_offsets"):
        assert f(**{k: whole[k] + 4}) == INV, k
    for k in ("repetition", "presence", "frequency", "bias", "mask"):
        assert f(**{k: whole[k] + 2}) == INV, k
    for k in ("tokens", "offsets", "prompt", "repetition", "presence", "frequency", "bias_idx", "bias", "bias_offsets", "mask"):
        assert f(**{k: out[1]}) == AL, k
    near, _k1 = _arr([z[r] + 64 for r in range(P)])
    assert f(out=near) == AL and f(out=z, old=_i64(104, 100, 128, 50)) == AL
    cross, _k2 = _arr([z[1], z[0], out[2], out[3]])
    same, _k3 = _arr([out[0], out[0], out[2], out[3]])
    assert f(out=cross) == AL and f(out=same) == AL


def test_binding_refuses_before_the_call():
    import torch
    T = lambda d: lambda *s: DeviceTensor(d, *s)  # noqa: E731
    f, i, w = T(torch.float32), T(torch.int64), T(torch.int32)
    good = dict(tokens=i(30), offsets=i(6), prompt=i(5), repetition=f(5), presence=f(5), frequency=f(5), bias_idx=i(9), bias=f(9), bias_offsets=i(6), mask=w(5, 4))

    def call(rows=None, out=None, **k):
        return coll.coll_vocab_adjust([f(5, 60), f(5, 40)], out or [f(5, 60), f(5, 40)], rows=rows, defer=True, stream=0, **{**good, **k})
    call()
    call(mask=None)
    call(mask=w(7, 9))
    for k in (dict(tokens=w(30)), dict(tokens=f(30)), dict(offsets=i(5)), dict(prompt=i(4)), dict(repetition=f(4)), dict(presence=i(5)), dict(frequency=f(1)),
              dict(bias_idx=i(8)), dict(bias=i(9)), dict(bias_offsets=i(5)), dict(bias_offsets=w(6)), dict(mask=w(5, 3)), dict(mask=w(4, 4)), dict(mask=f(5, 4)),
              dict(mask=w(20)), dict(ntokens=31), dict(nbias=10), dict(mask_ld=5), dict(rows=6), dict(out=[f(5, 60)]), dict(out=[f(5, 60), f(5, 39)]),
              dict(tokens=None, ntokens=4), dict(mask=DeviceTensor(torch.int32, 5, 4, stride=(8, 2)))):
        with pytest.raises(ValueError):
            call(**k)


@host_only
def test_launches_hold_the_work_items_that_hip_takes(tmp_path):
    shapes = [(64, 1 << 20, 1), (64, (1 << 20) + 3, 16), (1, 1 << 26, 8), (1, (1 << 28) + 1, 100), (8, 1 << 20, 16384), (1, 3, 0x7fffffff), (64, 100, (1 << 25) - 1),
              (1, 1 << 18, 131072)]
    calls = []
    for p, rows, v in shapes:
        one = f"_i64(*[{v}] * {p})"
        for dt in (0, 1):
            calls.append(f"L.coll_vocab_adjust(b({p}), {one}, {one}, __import__('test_adjust_abi_cpu').by(), b({p}), {one}, {p}, {rows}, {dt}, None)")
    for (p, rows, v), *found in zip(shapes, *[iter(recorded(tmp_path, calls))] * 2):
        for launched, elems in zip(found, (4, 8)):
            # a workgroup to a shard's row at least, and a lane to four units of 16 bytes
            assert sum(g[0] for g, b in launched) >= rows * p and sum(4 * elems * g[0] * b[0] for g, b in launched) >= rows * p * v
