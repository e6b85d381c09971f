"""Host-side checks of the RMS norm's entry points: refusals, overlaps, empty
calls, launches of the largest shapes, none of which reaches the device."""
import pytest

import collective_communication_primitives_coll_amd as coll
from test_abi_cpu import _arr, host_only
from test_token_abi_cpu import AL, BASE, BF16, F32, I32, INV, OK, P, U8, UNS, Bufs, DeviceTensor, recorded


def test_workspace_sizes():
    ws = coll.coll_rmsnorm_workspace_bytes
    assert ws(0, 10, 64) == 0 and ws(65, 10, 64) == 0 and ws(4, 10, 0) == 0 and ws(4, 1 << 60, 64) == 0 and ws(4, 10, 1 << 31) == 0
    for p, hidden in [(1, 1), (1, 7), (8, 64), (3, 2565), (33, 7168), (64, 20000)]:
        sizes = [ws(p, rows, hidden) for rows in range(0, 3000, 7)]
        assert sizes == sorted(sizes) and sizes[0] > 0 and not any(n % (4 * hidden) for n in sizes), (p, hidden)


def test_no_rows_is_ok_without_pointers():
    L = coll.lib()
    assert L.coll_rmsnorm(None, None, None, None, None, None, P, 0, 64, 1e-6, BF16, BF16, None) == OK
    assert L.coll_rmsnorm_fp8(None, None, None, None, None, None, None, P, 0, 64, 16, 1e-6, BF16, F32, None) == OK
    assert L.coll_rmsnorm_backward(None, None, None, None, None, None, None, P, 0, 64, 0, F32, F32, None, 0, None) == OK


@host_only
def test_forward_refusals():
    L, b = coll.lib(), Bufs()
    x, res, g, h, y, s, y8 = b(), b(), b(), b(), b(), b(), b()
    odd, hole, _k = b(off=1), *_arr([BASE, 0, BASE + 64, BASE + 128])

    def fwd(x=x, res=res, g=g, h=h, y=y, s=s, p=P, rows=10, hidden=64, eps=1e-6, dt=BF16, wt=BF16):
        return L.coll_rmsnorm(x, res, g, h, y, s, p, rows, hidden, eps, dt, wt, None)
    assert fwd(p=0) == INV and fwd(p=65) == INV and fwd(hidden=0) == INV and fwd(dt=U8) == INV and fwd(dt=7) == INV
    assert fwd(dt=I32, wt=I32) == UNS and fwd(dt=F32, wt=BF16) == UNS and fwd(wt=I32) == UNS and fwd(hidden=1 << 31) == UNS
    assert fwd(rows=1 << 60) == INV and fwd(eps=-1.0) == INV and fwd(eps=float("nan")) == INV and fwd(eps=float("inf")) == INV
    assert fwd(res=None) == INV                                          # a stream without a residual
    assert fwd(x=None) == INV and fwd(y=None) == INV and fwd(x=hole) == INV and fwd(res=hole) == INV and fwd(g=hole) == INV
    assert fwd(h=hole) == INV and fwd(s=hole) == INV
    assert fwd(x=odd) == INV and fwd(res=odd) == INV and fwd(y=odd) == INV and fwd(g=odd) == INV and fwd(s=odd) == INV and fwd(h=odd) == INV
    assert fwd(h=y) == AL and fwd(y=g) == AL and fwd(h=g) == AL and fwd(s=x) == AL and fwd(s=h) == AL
    near, _k1 = _arr([x[r] + 64 for r in range(P)])                      # half over its input
    assert fwd(y=near) == AL and fwd(h=near) == AL
    swap, _k2 = _arr([res[1], res[0], res[2], res[3]])                   # another rank's
    assert fwd(y=swap) == AL and fwd(h=swap) == AL
    assert fwd(h=x, y=x) == AL and fwd(x=res, h=x, y=x) == AL

    def codes(y8=y8, group=16, hidden=64, y=None, h=h):
        return L.coll_rmsnorm_fp8(x, res, g, h, y, s, y8, P, 10, hidden, group, 1e-6, BF16, BF16, None)
    assert codes(y8=None) == INV and codes(y8=hole) == INV and codes(y8=b(off=8)) == INV and codes(group=0) == INV and codes(y=hole) == INV
    assert codes(group=48, hidden=96) == UNS and codes(group=1024, hidden=1024) == UNS and codes(hidden=72) == INV
    assert codes(y8=x) == AL and codes(y8=h) == AL and codes(y=y8) == AL and codes(y8=s) == AL


@host_only
def test_backward_refusals():
    L, b = coll.lib(), Bufs()
    dy, dh, h, s, g, dx, dg, ws = b(), b(), b(), b(), b(), b(), b(), b.one()
    odd, hole, _k = b(off=1), *_arr([BASE, 0, BASE + 64, BASE + 128])
    need = coll.coll_rmsnorm_workspace_bytes(P, 10, 64)

    def bwd(dy=dy, dh=dh, h=h, s=s, g=g, dx=dx, dg=dg, op=0, ws=ws, n=need, dt=BF16, wt=BF16, rows=10, p=P, hidden=64):
        return L.coll_rmsnorm_backward(dy, dh, h, s, g, dx, dg, p, rows, hidden, op, dt, wt, ws, n, None)
    assert bwd(op=1) == UNS and bwd(op=2) == UNS and bwd(op=9) == INV and bwd(ws=None) == INV and bwd(n=need - 1) == INV
    assert bwd(p=0) == INV and bwd(p=65) == INV and bwd(hidden=0) == INV and bwd(dt=I32) == UNS and bwd(wt=I32) == UNS and bwd(rows=1 << 60) == INV
    assert bwd(ws=ws + 4) == INV and bwd(dy=None) == INV and bwd(h=None) == INV and bwd(s=None) == INV and bwd(dx=None) == INV
    assert bwd(dh=hole) == INV and bwd(s=hole) == INV and bwd(dg=hole) == INV and bwd(g=hole) == INV
    assert bwd(dx=odd) == INV and bwd(dh=odd) == INV and bwd(dg=odd) == INV and bwd(h=odd) == INV
    assert bwd(dx=h) == AL and bwd(dg=g) == AL and bwd(ws=dx[0]) == AL and bwd(ws=h[1]) == AL and bwd(dx=s) == AL and bwd(dg=dx) == AL
    near, _k1 = _arr([dh[r] + 64 for r in range(P)])
    assert bwd(dx=near) == AL
    assert bwd(rows=0, ws=None, n=0, dy=None, dx=None, dg=hole) == INV


def test_binding_refuses_before_the_call():
    import torch
    f, h, u = (lambda t: lambda *s: DeviceTensor(t, *s))(torch.float32), (lambda *s: DeviceTensor(torch.bfloat16, *s)), (lambda *s: DeviceTensor(torch.uint8, *s))
    ok = dict(defer=True, stream=0)
    coll.coll_rmsnorm([f(4, 64)], [f(64)], [f(4, 64)], 64, residual=[f(4, 64)], h=[f(4, 64)], rstd=[f(4)], **ok)
    bad = [dict(residual=[h(4, 64)]), dict(h=[f(4, 63)]), dict(rstd=[f(3)]), dict(rstd=[h(4)]), dict(residual=[f(4, 64)] * 2), dict(gamma=[f(63)]), dict(rows=5)]
    for k in bad:
        k = dict(gamma=[f(64)]) | k
        with pytest.raises(ValueError):
            coll.coll_rmsnorm([f(4, 64)], k.pop("gamma"), [f(4, 64)], 64, **k, **ok)
    for y8 in (None, [u(4 * 64)], [f(4 * 128)]):                        # absent, too small, not bytes
        with pytest.raises(ValueError):
            coll.coll_rmsnorm_fp8([f(4, 64)], None, y8, 64, 32, **ok)
    ws = f(100000)
    coll.coll_rmsnorm_backward([f(4, 64)], [f(4, 64)], [f(4)], None, [f(4, 64)], [f(64)], ws, 64, dh=[f(4, 64)], **ok)
    for k in (dict(dh=[h(4, 64)]), dict(dh=[f(3, 64)]), dict(workspace_bytes=400001), dict(rows=5)):
        with pytest.raises(ValueError):
            coll.coll_rmsnorm_backward([f(4, 64)], [f(4, 64)], [f(4)], None, [f(4, 64)], [f(64)], ws, 64, **k, **ok)


@host_only
def test_launches_hold_the_work_items_that_hip_takes(tmp_path):
    # rows of a few elements that need more than one launch of the forward pass; rows so wide that the backward
    # pass's columns, or the join over them, do
    forward = [(8, (1 << 29) - 32, 1), (8, 1 << 29, 2), (8, (1 << 31) + 7, 1), (300, (1 << 27) + 1, 1), (1024, 1 << 28, 1), (5120, 1 << 25, 2), (1 << 30, 3, 2)]
    calls = []
    for h, rows, p in forward:
        calls.append(f"L.coll_rmsnorm(b({p}), b({p}), None, b({p}), b({p}), b({p}), {p}, {rows}, {h}, 1e-6, 1, 1, None)")
        h = -(-h // 16) * 16
        calls.append(f"L.coll_rmsnorm_fp8(b({p}), None, None, None, None, b({p}), b({p}), {p}, {rows}, {h}, 16, 1e-6, 0, 0, None)")
    for h, rows, p in [(8, 1 << 30, 3), (1 << 27, 1, 1), ((1 << 27) + 9, 256, 2), (1 << 30, 64, 1), ((1 << 31) - 1, 200, 1)]:
        calls.append(f"L.coll_rmsnorm_backward(b({p}), b({p}), b({p}), b({p}), None, b({p}), b({p}), {p}, {rows}, {h}, 0, 1, 0, "
                     f"b.one(), coll.coll_rmsnorm_workspace_bytes({p}, {rows}, {h}), None)")
    found = recorded(tmp_path, calls)
    for (h, rows, p), launched in zip(forward, found[::2]):
        assert h > 8 or sum(g[0] for g, b in launched) * 32 >= rows      # 32 rows to a workgroup
