"""Host-side checks of the distillation's entry points: refusals, workspaces,
overlaps, empty calls, launches of the largest shapes, none of which reaches
the device."""
import pytest

import collective_communication_primitives_coll_amd as coll
from test_abi_cpu import _arr, host_only
from test_token_abi_cpu import AL, BF16, F32, I32, INV, LOGPROB_VOCABS, OK, P, U8, UNS, Bufs, DeviceTensor, _i64, recorded


def test_workspaces():
    ws = coll.coll_vocab_distill_workspace_bytes
    assert ws(0, [100], 4) == 0 and ws(4, [100] * 65, 4) == 0 and ws(4, [-1, 5], 4) == 0 and ws(4, [10], 0) == 0 and ws(4, [10], 129) == 0
    for vocab in LOGPROB_VOCABS:
        for top in (1, 20, 128):
            had = 0
            for rows in [*range(0, 2100), *range(2100, 9000, 97), 1 << 20, (1 << 20) + 1, 1 << 40]:
                n = ws(rows, vocab, top)
                assert n >= had and (n > 0) == (rows > 0) and n <= rows * (64 * 8 + 4 * top), (vocab, top, rows)
                had = n
    for rows in (1 << 58, 1 << 60, 1 << 63, (1 << 64) - 1):
        assert ws(rows, [1] * 3, 128) == 0


def test_no_rows_is_ok_without_pointers():
    L, ld = coll.lib(), _i64(8, 8, 8, 8)
    assert L.coll_vocab_distill(None, ld, ld, None, None, 3, 1, 1.0, None, None, P, 0, F32, None, 0, None) == OK
    assert L.coll_vocab_distill_backward(None, ld, ld, None, None, 3, 0, 1.0, None, None, None, ld, P, 0, BF16, None) == OK


@host_only
def test_refusals():
    L, b = coll.lib(), Bufs()
    z, st, lo, dz = b(), b(), b(), b()
    i, l, ws, s1, g1 = b.one(), b.one(), b.one(), b.one(), b.one()
    vocab, ld = _i64(100, 100, 100, 50), _i64(100, 100, 128, 50)
    need = coll.coll_vocab_distill_workspace_bytes(9, list(vocab), 4)
    hole, _k = _arr([z[0], 0, z[2], z[3]])

    def fwd(z=z, ld=ld, vocab=vocab, i=i, l=l, k=4, kind=1, temp=1.0, st=st, lo=lo, p=P, rows=9, dt=BF16, ws=ws, n=need):
        return L.coll_vocab_distill(z, ld, vocab, i, l, k, kind, temp, st, lo, p, rows, dt, ws, n, None)

    def bwd(z=z, ld=ld, vocab=vocab, i=i, l=l, k=4, kind=1, temp=1.0, st=s1, g=g1, dz=dz, dld=ld, p=P, rows=9, dt=BF16):
        return L.coll_vocab_distill_backward(z, ld, vocab, i, l, k, kind, temp, st, g, dz, dld, p, rows, dt, None)
    big = _i64(1 << 30, 1 << 30, 1 << 30, 1 << 30)
    for f in (fwd, bwd):
        assert f(p=0) == INV and f(p=65) == INV and f(dt=U8) == INV and f(dt=I32) == UNS and f(k=0) == INV and f(k=-1) == INV and f(k=129) == UNS
        assert f(kind=2) == INV and f(kind=-1) == INV
        for bad in (0.0, -1.0, float("nan"), float("inf")):
            assert f(temp=bad) == INV
        assert f(ld=None) == INV and f(vocab=None) == INV and f(ld=_i64(99, 100, 100, 50)) == INV
        assert f(vocab=_i64(-1, 2, 2, 2)) == INV and f(vocab=_i64(0, 0, 0, 0)) == INV and f(z=None) == INV and f(z=hole) == INV and f(z=b(off=1)) == INV
        assert f(i=None) == INV and f(l=None) == INV and f(i=i + 2) == INV and f(l=l + 2) == INV and f(st=None) == INV
        for rows in (1 << 58, 1 << 60, 1 << 62, (1 << 64) - 1):
            assert f(rows=rows) == INV
    assert fwd(vocab=big, ld=big) == UNS and bwd(vocab=big, ld=big, dld=big) == UNS
    assert fwd(lo=None) == INV and fwd(st=b(off=2)) == INV and fwd(lo=b(off=2)) == INV and fwd(st=hole) == INV
    assert fwd(ws=None) == INV and fwd(n=need - 1) == INV and fwd(ws=ws + 8) == INV
    assert fwd(st=lo) == AL and fwd(st=z) == AL and fwd(ws=z[0]) == AL and fwd(i=st[0]) == AL and fwd(l=lo[2]) == AL and fwd(ws=i) == AL
    assert bwd(dz=None) == INV and bwd(dld=None) == INV and bwd(dld=_i64(100, 100, 99, 50)) == INV and bwd(g=None) == INV and bwd(g=g1 + 1) == INV
    assert bwd(st=s1 + 2) == INV
    assert bwd(st=dz[1]) == AL and bwd(i=dz[3]) == AL and bwd(l=dz[0]) == AL and bwd(g=dz[2]) == AL
    assert bwd(dz=z, dld=_i64(104, 100, 128, 50)) == AL               # in place, but another stride
    cross, _k1 = _arr([z[1], z[0], dz[2], dz[3]])
    assert bwd(dz=cross) == AL
    same, _k2 = _arr([dz[0], dz[0], dz[2], dz[3]])
    assert bwd(dz=same) == AL


def test_binding_refuses_before_the_call():
    import torch
    f, t = (lambda *s: DeviceTensor(torch.float32, *s)), (lambda *s: DeviceTensor(torch.int32, *s))
    ok = dict(defer=True, stream=0)

    def both(i=t(5, 4), l=f(5, 4), st=f(5, 4), lo=f(5), **k):
        ws, out = DeviceTensor(torch.uint8, 1 << 20), []
        out.append(lambda: coll.coll_vocab_distill([f(5, 100)], i, l, [st], [lo], ws, **k, **ok))
        kb = {a: b for a, b in k.items() if a != "workspace_bytes"}
        out.append(lambda: coll.coll_vocab_distill_backward([f(5, 100)], i, l, st, lo, [f(5, 100)], **kb, **ok))
        return out
    for call in both() + both(rows=3) + both(i=t(20), l=f(20), rows=5, top_k=4) + both(workspace_bytes=1 << 20)[:1]:
        call()
    for call in (both(i=f(5, 4)) + both(l=t(5, 4)) + both(l=f(5, 3)) + both(st=f(5, 3)) + both(lo=f(4)) + both(lo=t(5)) + both(rows=6) + both(top_k=3)
                 + both(i=t(20), l=f(20)) + both(l=f(4, 5)) + both(workspace_bytes=(1 << 20) + 1)[:1]):
        with pytest.raises(ValueError):
            call()


@host_only
def test_launches_hold_the_work_items_that_hip_takes(tmp_path):
    shapes = [(64, 1 << 20, 1), (64, (1 << 20) + 3, 16), (1, 1 << 26, 8), (1, (1 << 28) + 1, 100), (8, 1 << 20, 16384), (1, 3, 0x7fffffff)]
    calls = []
    for p, rows, v in shapes:
        one, k = f"_i64(*[{v}] * {p})", 128 if v > 1000 else 5
        calls.append(f"L.coll_vocab_distill(b({p}), {one}, {one}, b.one(), b.one(), {k}, {k & 1}, 1.0, b({p}), b({p}), {p}, {rows}, 1, "
                     f"b.one(), coll.coll_vocab_distill_workspace_bytes({rows}, [{v}] * {p}, {k}), None)")
        calls.append(f"L.coll_vocab_distill_backward(b({p}), {one}, {one}, b.one(), b.one(), {k}, 1, 1.0, b.one(), b.one(), b({p}), {one}, {p}, {rows}, 1, None)")
    found = recorded(tmp_path, calls)
    waves = lambda launched: sum(g[0] * b[0] // 64 for g, b in launched)  # noqa: E731
    for (p, rows, v), fwd, back in zip(shapes, found[::2], found[1::2]):
        assert waves(fwd) >= rows * p + rows and waves(back) >= rows * p * -(-v // 1024)       # pieces, then the join


@host_only
def test_a_workspace_for_more_rows_serves_fewer(tmp_path):
    calls = []
    for vocab in LOGPROB_VOCABS:
        p, ld = len(vocab), [max(v, 1) for v in vocab]
        for rows, most in ((1000, 1024), (1023, 1024), (1, 2), (500, 8192), (63, 200), (129, 130), (4095, 4096)):
            for top in (1, 128):
                calls.append(f"L.coll_vocab_distill(b({p}), _i64(*{ld}), _i64(*{vocab}), b.one(), b.one(), {top}, 1, 1.0, b({p}), b({p}), "
                             f"{p}, {rows}, 1, b.one(), coll.coll_vocab_distill_workspace_bytes({most}, {vocab}, {top}), None)")
    recorded(tmp_path, calls)
