"""Host-side checks of the token-wise operators' entry points: refusals,
workspaces, overlaps and empty calls, none of which reaches the device."""
import ctypes
import json
import math
import os
import subprocess
import sys
import textwrap

import pytest

import collective_communication_primitives_coll_amd as coll
from conftest import ROOT
from test_abi_cpu import _arr, host_only

OK, INV, UNS, AL = coll.COLL_OK, coll.COLL_ERR_INVALID_ARG, coll.COLL_ERR_UNSUPPORTED, coll.COLL_ERR_ALIAS
F32, BF16, I32, U8 = 0, 1, 2, 3
BASE = 0x7F0000000000
P = 4


class Bufs:
    """Made-up rank arrays, far apart."""

    def __init__(self):
        self.keep, self.next = [], BASE

    def __call__(self, off=0, p=P, step=0x10000000):
        a, k = _arr([self.next + off + step * r for r in range(p)])
        self.next += step * (p + 1)
        self.keep.append(k)
        return a

    def one(self, off=0):
        self.next += 0x10000000
        return self.next - 0x10000000 + off


def _i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def test_shape_functions():
    rb = coll.coll_ckpt8_row_bytes
    assert rb(7168, 128) == 7168 + 56 * 4 and rb(16, 16) == 32 and rb(512, 512) == 528
    for hidden, group in [(0, 16), (100, 16), (64, 0), (64, 8), (96, 48), (1024, 1024), (1 << 31, 512)]:
        assert rb(hidden, group) == 0, (hidden, group)
    ws = coll.coll_layernorm_workspace_bytes
    assert ws(0, 10, 64) == 0 and ws(65, 10, 64) == 0 and ws(4, 10, 0) == 0 and ws(4, 1 << 60, 64) == 0
    for p, rows, hidden in [(1, 1, 1), (8, 4096, 7168), (64, 3, 100), (3, 5, 40000)]:
        n = ws(p, rows, hidden)
        assert n > 0 and n % (2 * hidden * 4) == 0
    lw = coll.coll_vocab_logprob_workspace_bytes
    assert lw(0, [100], 4) == 0 and lw(4, [100] * 65, 4) == 0 and lw(4, [-1, 5], 4) == 0 and lw(4, [10], 33) == 0
    for rows, vocab, top in [(1, [1], 0), (3, [50257], 32), (5, [0, 9, 0], 1), (2048, [16384] * 8, 8), (7, [1000] * 64, 5)]:
        n = lw(rows, vocab, top)
        most = 64 * 32 + 1024 * 4 if top else 64 * 16      # bytes of a row: 64 pieces, and 1024 groups of elements
        assert n > 0 and n % (16 * rows) == 0 and n // rows <= most


def test_no_rows_is_ok_without_pointers():
    L = coll.lib()
    assert L.coll_layernorm(None, None, None, None, None, None, P, 0, 64, 1e-5, BF16, BF16, None) == OK
    assert L.coll_layernorm_ckpt8(None, None, None, None, None, None, None, P, 0, 64, 16, 1e-5, BF16, F32, None) == OK
    assert L.coll_layernorm_backward(None, None, None, None, None, None, None, None, P, 0, 64, 0, F32, F32, None, 0, None) == OK
    assert L.coll_ckpt8_save(None, None, P, 0, 64, 32, F32, None) == OK
    assert L.coll_ckpt8_load(None, None, P, 0, 64, 32, F32, None) == OK
    assert L.coll_swiglu_ckpt8(None, None, None, P, 0, 64, 32, BF16, None) == OK
    assert L.coll_swiglu_backward_ckpt8(None, None, None, None, P, 0, 64, 32, BF16, None) == OK
    ld = _i64(8, 8, 8, 8)
    assert L.coll_vocab_logprob(None, ld, ld, None, 1.0, None, None, None, 0, None, None, P, 0, F32, None, 0, None) == OK
    assert L.coll_vocab_logprob_backward(None, ld, ld, None, 1.0, None, None, None, None, None, ld, P, 0, F32, None) == OK


@host_only
def test_layernorm_refusals():
    L = coll.lib()
    b = Bufs()
    x, g, be, y, m, s, ck = b(), b(), b(), b(), b(), b(), b()
    odd, hole, holek = b(off=1), *_arr([BASE, 0, BASE + 64, BASE + 128])

    def fwd(x=x, g=g, be=be, y=y, m=m, s=s, p=P, rows=10, hidden=64, eps=1e-5, dt=BF16, wt=BF16):
        return L.coll_layernorm(x, g, be, y, m, s, p, rows, hidden, eps, dt, wt, None)
    assert fwd(p=0) == INV and fwd(p=65) == INV and fwd(hidden=0) == INV and fwd(dt=U8) == INV and fwd(dt=7) == INV
    assert fwd(dt=I32, wt=I32) == UNS and fwd(dt=F32, wt=BF16) == UNS and fwd(wt=I32) == UNS and fwd(hidden=1 << 31) == UNS
    assert fwd(rows=1 << 60) == INV and fwd(eps=-1.0) == INV and fwd(eps=float("nan")) == INV and fwd(eps=float("inf")) == INV
    assert fwd(x=None) == INV and fwd(y=None) == INV and fwd(x=hole) == INV and fwd(g=hole) == INV and fwd(m=hole) == INV
    assert fwd(x=odd) == INV and fwd(y=odd) == INV and fwd(g=odd) == INV and fwd(s=odd) == INV
    assert fwd(y=g) == AL and fwd(m=s) == AL and fwd(m=x) == AL and fwd(y=m) == AL
    near, _k = _arr([x[r] + 64 for r in range(P)])       # the output half over its input
    assert fwd(y=near) == AL
    swap, _k2 = _arr([x[1], x[0], x[2], x[3]])           # another rank's input
    assert fwd(y=swap) == AL

    def ckpt(ck=ck, group=16, hidden=64, m=m):
        return L.coll_layernorm_ckpt8(x, g, be, y, m, s, ck, P, 10, hidden, group, 1e-5, BF16, BF16, None)
    assert ckpt(ck=None) == INV and ckpt(ck=hole) == INV and ckpt(ck=b(off=8)) == INV and ckpt(group=0) == INV
    assert ckpt(group=48, hidden=96) == UNS and ckpt(group=1024, hidden=1024) == UNS and ckpt(hidden=72) == INV
    assert ckpt(ck=y) == AL and ckpt(ck=x) == AL

    dy, dx, dg, db, ws = b(), b(), b(), b(), b.one()
    need = coll.coll_layernorm_workspace_bytes(P, 10, 64)

    def bwd(dy=dy, x=x, m=m, s=s, g=g, dx=dx, dg=dg, db=db, op=0, ws=ws, n=need, wt=BF16, rows=10):
        return L.coll_layernorm_backward(dy, x, m, s, g, dx, dg, db, P, rows, 64, op, BF16, wt, ws, n, None)
    assert bwd(op=1) == UNS and bwd(op=2) == UNS and bwd(op=9) == INV and bwd(ws=None) == INV and bwd(n=need - 1) == INV
    assert bwd(ws=ws + 4) == INV and bwd(dy=None) == INV and bwd(m=None) == INV and bwd(s=hole) == INV and bwd(dg=hole) == INV
    assert bwd(dx=odd) == INV and bwd(db=odd) == INV
    assert bwd(dx=x) == AL and bwd(dg=db) == AL and bwd(dg=g) == AL and bwd(ws=dx[0]) == AL and bwd(dx=m) == AL
    assert bwd(rows=0, dg=db) == AL

    def bck(y=None, be=None, group=16, x=ck):
        return L.coll_layernorm_backward_ckpt8(dy, x, m, s, g, be, dx, y, dg, db, P, 10, 64, group, 0, BF16, BF16, ws, need, None)
    assert bck(group=24) == INV and bck(group=8) == UNS and bck(y=hole) == INV and bck(y=dx) == AL and bck(y=ck) == AL
    assert bck(x=b(off=2)) == INV and bck(be=odd) == INV


@host_only
def test_checkpoint_and_gated_activation_refusals():
    L = coll.lib()
    b = Bufs()
    x, ck, out, dx = b(), b(), b(), b()
    odd = b(off=1)
    for f in (lambda a, c, **k: L.coll_ckpt8_save(a, c, k.get("p", P), k.get("rows", 9), k.get("h", 64), k.get("g", 32), k.get("dt", BF16), None),
              lambda a, c, **k: L.coll_ckpt8_load(c, a, k.get("p", P), k.get("rows", 9), k.get("h", 64), k.get("g", 32), k.get("dt", BF16), None)):
        assert f(x, ck, p=0) == INV and f(x, ck, h=65) == INV and f(x, ck, g=8) == UNS and f(x, ck, h=96, g=48) == UNS
        assert f(x, ck, dt=I32) == UNS and f(x, ck, dt=U8) == INV and f(None, ck) == INV and f(x, None) == INV
        assert f(odd, ck) == INV and f(x, odd) == INV and f(x, x) == AL and f(x, ck, rows=1 << 59) == INV

    def fwd(x=x, out=out, ck=ck, ffn=64, g=32, dt=BF16, p=P):
        return L.coll_swiglu_ckpt8(x, out, ck, p, 9, ffn, g, dt, None)
    assert fwd(p=65) == INV and fwd(ffn=0) == INV and fwd(ffn=48) == INV and fwd(g=16, ffn=1 << 30) == UNS and fwd(dt=I32) == UNS
    assert fwd(out=None) == INV and fwd(ck=odd) == INV and fwd(out=x) == AL and fwd(ck=out) == AL and fwd(g=1024, ffn=1024) == UNS

    dout, dgu = b(), b()

    def bwd(ck=ck, dout=dout, dgu=dgu, out=None, ffn=64, g=32):
        return L.coll_swiglu_backward_ckpt8(ck, dout, dgu, out, P, 9, ffn, g, BF16, None)
    assert bwd(ck=None) == INV and bwd(dout=odd) == INV and bwd(out=odd) == INV and bwd(g=0) == INV
    assert bwd(dgu=dout) == AL and bwd(dgu=ck) == AL and bwd(out=dout) == AL and bwd(out=dgu) == AL


@host_only
def test_logprob_refusals():
    L = coll.lib()
    b = Bufs()
    z, st, lp, en, tl, ti, dz = b(), b(), b(), b(), b(), b(), b()
    t, ws = b.one(), b.one()
    vocab, ld = _i64(100, 100, 100, 50), _i64(100, 100, 128, 50)
    need = coll.coll_vocab_logprob_workspace_bytes(9, list(vocab), 4)

    def fwd(z=z, ld=ld, vocab=vocab, t=t, temp=1.0, st=st, lp=lp, en=en, k=4, tl=tl, ti=ti, p=P, dt=BF16, ws=ws, n=need, rows=9):
        return L.coll_vocab_logprob(z, ld, vocab, t, temp, st, lp, en, k, tl, ti, p, rows, dt, ws, n, None)
    assert fwd(p=0) == INV and fwd(p=65) == INV and fwd(dt=U8) == INV and fwd(dt=I32) == UNS and fwd(k=-1) == INV and fwd(k=33) == UNS
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert fwd(temp=bad) == INV
    assert fwd(ld=None) == INV and fwd(vocab=None) == INV and fwd(ld=_i64(99, 100, 100, 50)) == INV
    assert fwd(vocab=_i64(-1, 2, 2, 2)) == INV and fwd(vocab=_i64(0, 0, 0, 0)) == INV
    big = _i64(1 << 30, 1 << 30, 1 << 30, 1 << 30)
    assert fwd(vocab=big, ld=big) == UNS
    assert fwd(t=None) == INV and fwd(t=t + 4) == INV and fwd(st=None) == INV and fwd(lp=None) == INV and fwd(tl=None) == INV
    assert fwd(z=None) == INV and fwd(z=b(off=1)) == INV and fwd(en=b(off=2)) == INV
    assert fwd(ws=None) == INV and fwd(n=need - 1) == INV and fwd(ws=ws + 8) == INV
    assert fwd(st=lp) == AL and fwd(st=z) == AL and fwd(ws=z[0]) == AL and fwd(tl=ti) == AL and fwd(lp=en) == AL
    assert fwd(t=st[0]) == AL

    s1, d1, e1, h1 = b.one(), b.one(), b.one(), b.one()

    def bwd(z=z, dz=dz, dld=ld, st=s1, dlp=d1, en=e1, den=h1, t=t, ld=ld, temp=1.0):
        return L.coll_vocab_logprob_backward(z, ld, vocab, t, temp, st, dlp, en, den, dz, dld, P, 9, BF16, None)
    assert bwd(temp=0.0) == INV and bwd(dz=None) == INV and bwd(dld=None) == INV and bwd(dld=_i64(100, 100, 99, 50)) == INV
    assert bwd(st=None) == INV and bwd(dlp=None) == INV and bwd(en=None) == INV and bwd(den=h1 + 1) == INV
    assert bwd(st=dz[1]) == AL and bwd(t=dz[3]) == AL and bwd(den=dz[0]) == AL
    assert bwd(dz=z, dld=_i64(104, 100, 128, 50)) == AL               # in place, but another stride
    cross, _k = _arr([z[1], z[0], dz[2], dz[3]])
    assert bwd(dz=cross) == AL
    same, _k2 = _arr([dz[0], dz[0], dz[2], dz[3]])
    assert bwd(dz=same) == AL
    # column slices of one matrix may stand side by side, not across each other
    lds = _i64(350, 350, 350, 350)
    cols, _k3 = _arr([dz[0] + 2 * c for c in (0, 90, 200, 300)])      # the first two share ten columns
    assert bwd(dz=cols, dld=lds, z=z) == AL
    wrap, _k4 = _arr([dz[0] + 2 * c for c in (0, 100, 200, 320)])     # the last runs into the next row's first
    assert bwd(dz=wrap, dld=lds) == AL


def test_binding_refuses_before_the_call():
    import torch
    z = torch.zeros(2, 3)
    with pytest.raises(ValueError):
        coll.coll_vocab_logprob([z], torch.zeros(2, dtype=torch.int64), [z], [z], z)        # host tensors
    with pytest.raises(ValueError):
        coll.coll_vocab_logprob([z], torch.zeros(2, dtype=torch.int32), [z], [z], z)        # int32 targets
    with pytest.raises(ValueError):
        coll.coll_layernorm([1, 2], None, None, [1], 8, rows=1, dtype=F32)                  # unlike rank counts
    with pytest.raises(ValueError):
        coll.coll_layernorm_ckpt8([1], None, None, [1], None, None, None, 16, 16, rows=1, dtype=F32)
    with pytest.raises(ValueError):
        coll.coll_vocab_logprob_backward([1], 1, 1, 1, [1], rows=1, dtype=F32)              # raw addresses, no sizes
    with pytest.raises(ValueError):
        coll.coll_layernorm_backward([1], [1], [1], [1], None, [1], None, None, 1, 8, rows=1, dtype=F32)  # no workspace size


class DeviceTensor:
    """As much of a device tensor as the binding looks at, for deferred calls that are never made."""
    is_cuda = True

    def __init__(self, dtype, *shape, stride=None):
        self.dtype, self.shape = dtype, shape
        self.strides = stride or tuple(math.prod(shape[i + 1:]) for i in range(len(shape)))

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    def stride(self, i):
        return self.strides[i]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return BASE


def _logprob_calls(n, targets=None, z=None, dz=None, **k):
    """Deferred forward and backward calls of one rank's n rows of 100 entries."""
    import torch
    f = lambda *s: DeviceTensor(torch.float32, *s)  # noqa: E731
    z, dz = z or f(n, 100), dz or f(n, 100)
    t = DeviceTensor(torch.int64, n if targets is None else targets)
    ws = DeviceTensor(torch.uint8, 1 << 20)
    kf = {a: b for a, b in k.items() if a != "dld"}
    return (lambda: coll.coll_vocab_logprob([z], t, [f(n, 2)], [f(n)], ws, defer=True, stream=0, **kf),
            lambda: coll.coll_vocab_logprob_backward([z], t, f(n, 2), f(n), [dz], defer=True, stream=0, **k))


def test_binding_refuses_targets_shorter_than_the_rows():
    for call in _logprob_calls(5, 5) + _logprob_calls(5, 6, rows=5):
        call()
    for call in _logprob_calls(5, 4, rows=5):
        with pytest.raises(ValueError, match="targets"):
            call()


def test_binding_refuses_workspace_bytes_past_the_tensor():
    import torch
    f = lambda *s: DeviceTensor(torch.float32, *s)  # noqa: E731
    for call in _logprob_calls(5, workspace_bytes=1 << 20)[:1]:
        call()
    for call in _logprob_calls(5, workspace_bytes=(1 << 20) + 1)[:1]:
        with pytest.raises(ValueError, match="workspace_bytes"):
            call()
    ws = DeviceTensor(torch.float32, 1000)
    back = lambda n: coll.coll_layernorm_backward([f(5, 64)], [f(5, 64)], [f(5)], [f(5)], None, [f(5, 64)], None, None, ws, 64,  # noqa: E731
                                                  workspace_bytes=n, defer=True, stream=0)
    back(4000)
    with pytest.raises(ValueError, match="workspace_bytes"):
        back(4001)


def test_binding_refuses_a_row_stride_that_is_not_the_tensors():
    import torch
    z = DeviceTensor(torch.float32, 5, 100, stride=(128, 1))
    for call in _logprob_calls(5, z=z, ld=[128]) + _logprob_calls(5, z=z, dz=z, ld=[128], dld=[128])[1:]:
        call()
    one = DeviceTensor(torch.float32, 1, 100)
    for call in _logprob_calls(1, z=one, ld=[999]):                                     # no second row
        call()
    for call in _logprob_calls(5, z=z, ld=[100]) + _logprob_calls(5, dz=z, dld=[100])[1:]:
        with pytest.raises(ValueError, match="ld is 100"):
            call()


def test_logprob_of_rows_past_the_address_space():
    """Row counts whose products leave 64 bits, in a process of its own: they must not end it."""
    code = textwrap.dedent(f"""
        import sys
        sys.path.insert(0, {ROOT!r})
        sys.path.insert(0, {os.path.join(ROOT, "tests")!r})
        import collective_communication_primitives_coll_amd as coll
        from test_token_abi_cpu import _i64
        L = coll.lib()
        for rows in (1 << 58, 1 << 60, (1 << 61) + 5, 1 << 62, 1 << 63, (1 << 64) - 1):
            for p in (1, 3, 16, 64):
                assert coll.coll_vocab_logprob_workspace_bytes(rows, [1] * p, 0) in (0, rows * p * 16), (rows, p)
                assert coll.coll_vocab_logprob_workspace_bytes(rows, [1] * p, 4) == 0 or rows * p < 1 << 58
                # (every pointer absent: no such call gets past the checks)
                one = _i64(*[1] * p)
                assert L.coll_vocab_logprob(None, one, one, None, 1.0, None, None, None, 0, None, None, p, rows, 1, None, 0, None) == 1
                assert L.coll_vocab_logprob_backward(None, one, one, None, 1.0, None, None, None, None, None, one, p, rows, 1, None) == 1
        print("through")
    """)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "through" in r.stdout, (r.returncode, r.stderr[-2000:])


@host_only
def test_logprob_backward_refuses_rows_past_the_address_space():
    L, b = coll.lib(), Bufs()
    z, dz, t, st, dl, one = b(), b(), b.one(), b.one(), b.one(), _i64(1, 1, 1, 1)
    for rows in (1 << 60, 1 << 61, 1 << 62):                            # 8 bytes a row leave 64 bits, or what an address may be
        assert L.coll_vocab_logprob_backward(z, one, one, t, 1.0, st, dl, None, None, dz, one, P, rows, BF16, None) == INV


# ----------------------------------------------------------------------------
# Launches of the largest shapes.  A stand-in for the runtime's launch calls
# records them, so that the entry points run whole, on made-up addresses,
# without a device.
# ----------------------------------------------------------------------------

RECORDER = r"""
struct Dim { unsigned x, y, z; };
static Dim grids[65536], blocks[65536], grid_now, block_now;
static int n;
extern "C" int __hipPushCallConfiguration(Dim grid, Dim block, unsigned long, void*) {
  grid_now = grid, block_now = block;
  return 0;
}
extern "C" int __hipPopCallConfiguration(Dim* grid, Dim* block, unsigned long* lds, void** stream) {
  *grid = grid_now, *block = block_now, *lds = 0, *stream = nullptr;
  return 0;
}
extern "C" int hipLaunchKernel(const void*, Dim grid, Dim block, void**, unsigned long, void*) {
  if (n < 65536) { grids[n] = grid; blocks[n] = block; }
  ++n;
  return 0;
}
extern "C" int hipGetLastError() { return 0; }
extern "C" int launches(unsigned* out) {
  for (int i = 0; i < n && i < 65536; ++i, out += 6) {
    out[0] = grids[i].x, out[1] = grids[i].y, out[2] = grids[i].z;
    out[3] = blocks[i].x, out[4] = blocks[i].y, out[5] = blocks[i].z;
  }
  const int had = n;
  n = 0;
  return had;
}
"""


class FarBufs(Bufs):
    """Made-up rank arrays, a TiB apart."""

    def __call__(self, p):
        return super().__call__(p=p, step=1 << 40)

    def one(self):
        self.next += 1 << 40
        return self.next - (1 << 40)


def recorded(tmp_path, calls):
    """The launches of each call, [(grid, block), ...] a call: `calls` are expressions of the C library L, the buffer
    maker b and _i64, each giving a status."""
    (tmp_path / "recorder.cpp").write_text(RECORDER)
    so = tmp_path / "recorder.so"
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(so), str(tmp_path / "recorder.cpp")], check=True)
    code = textwrap.dedent(f"""
        import ctypes, json, sys
        R = ctypes.CDLL({str(so)!r}, ctypes.RTLD_GLOBAL)   # ahead of the runtime's own
        sys.path.insert(0, {ROOT!r})
        sys.path.insert(0, {os.path.join(ROOT, "tests")!r})
        import collective_communication_primitives_coll_amd as coll
        from test_token_abi_cpu import FarBufs, _i64
        L, out = coll.lib(), (ctypes.c_uint * (6 * 65536))()
        for call in {calls!r}:
            b = FarBufs()
            status = eval(call)
            assert status == 0, (status, call)
            n = R.launches(out)
            assert 0 < n <= 65536, (n, call)
            print(json.dumps([[out[6 * i:6 * i + 3], out[6 * i + 3:6 * i + 6]] for i in range(n)]))
    """)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    found = [json.loads(line) for line in r.stdout.splitlines() if line.startswith("[[")]
    assert len(found) == len(calls)
    for call, launched in zip(calls, found):
        for grid, block in launched:
            assert all(g > 0 and g * w < 1 << 32 for g, w in zip(grid, block)), (call, grid, block)
    return found


@host_only
def test_logprob_launches_hold_the_work_items_that_hip_takes(tmp_path):
    shapes = [(64, 1 << 20, 1), (64, (1 << 20) + 3, 16), (1, 1 << 26, 8), (1, (1 << 28) + 1, 100), (8, 1 << 20, 16384), (1, 3, 0x7fffffff)]
    calls = []
    for p, rows, v in shapes:
        one = f"_i64(*[{v}] * {p})"
        calls.append(f"L.coll_vocab_logprob(b({p}), {one}, {one}, b.one(), 1.0, b({p}), b({p}), None, 0, None, None, {p}, {rows}, 1, "
                     f"b.one(), coll.coll_vocab_logprob_workspace_bytes({rows}, [{v}] * {p}), None)")
        calls.append(f"L.coll_vocab_logprob_backward(b({p}), {one}, {one}, b.one(), 1.0, b.one(), b.one(), None, None, b({p}), {one}, {p}, {rows}, 1, None)")
    found = recorded(tmp_path, calls)
    waves = lambda launched: sum(g[0] * b[0] // 64 for g, b in launched)  # noqa: E731
    for (p, rows, v), fwd, back in zip(shapes, found[::2], found[1::2]):
        assert waves(fwd) >= rows * p + rows and waves(back) >= rows * p * -(-v // 1024)       # pieces, then the join


@host_only
def test_checkpoint_launches_hold_the_work_items_that_hip_takes(tmp_path):
    calls = []
    for dt, rows in ((0, 1 << 22), (1, 1 << 22), (1, 1 << 23)):          # rows of 16384 elements: 2^24 tiles or more
        calls += [f"L.coll_ckpt8_save(b(2), b(2), 2, {rows}, 16384, 128, {dt}, None)", f"L.coll_ckpt8_load(b(2), b(2), 2, {rows}, 16384, 128, {dt}, None)",
                  f"L.coll_swiglu_ckpt8(b(2), b(2), b(2), 2, {rows}, 16384, 128, {dt}, None)",
                  f"L.coll_swiglu_backward_ckpt8(b(2), b(2), b(2), b(2), 2, {rows}, 16384, 128, {dt}, None)"]
    for launched in recorded(tmp_path, calls):
        assert len(launched) == 1 and launched[0][0][1] == 2             # both ranks; the workgroups walk what the grid leaves


@host_only
def test_layernorm_launches_hold_the_work_items_that_hip_takes(tmp_path):
    # rows of a few elements that need more than one launch of the forward pass; rows so wide that the backward
    # pass's columns, or the join over them, do
    forward = [(8, (1 << 29) - 32, 1), (8, 1 << 29, 2), (8, (1 << 31) + 7, 1), (300, (1 << 27) + 1, 1), (1024, 1 << 28, 1), (5120, 1 << 25, 2)]
    calls = []
    for h, rows, p in forward:
        calls.append(f"L.coll_layernorm(b({p}), None, None, b({p}), b({p}), b({p}), {p}, {rows}, {h}, 1e-5, 1, 1, None)")
        h = -(-h // 16) * 16
        calls.append(f"L.coll_layernorm_ckpt8(b({p}), None, None, b({p}), b({p}), b({p}), b({p}), {p}, {rows}, {h}, 16, 1e-5, 0, 0, None)")
    n_forward = len(calls)
    backward = [(8, 1 << 30, 3), (1 << 27, 1, 1), ((1 << 27) + 9, 256, 2), (1 << 30, 64, 1), ((1 << 31) - 1, 200, 1)]
    for h, rows, p in backward:
        ws = f"b.one(), coll.coll_layernorm_workspace_bytes({p}, {rows}, {h}), None)"
        calls.append(f"L.coll_layernorm_backward(b({p}), b({p}), b({p}), b({p}), None, b({p}), b({p}), b({p}), {p}, {rows}, {h}, 0, 1, 0, {ws}")
        h = h // 16 * 16
        calls.append(f"L.coll_layernorm_backward_ckpt8(b({p}), b({p}), b({p}), b({p}), None, None, b({p}), None, b({p}), b({p}), {p}, {rows}, "
                     f"{max(h, 16)}, 16, 0, 1, 0, b.one(), coll.coll_layernorm_workspace_bytes({p}, {rows}, {max(h, 16)}), None)")
    found = recorded(tmp_path, calls)
    for (h, rows, p), launched in zip(forward, found[:n_forward:2]):
        assert h > 8 or sum(g[0] for g, b in launched) * 32 >= rows      # 32 rows to a workgroup
    for (h, rows, p), launched in zip(backward, found[n_forward::2]):
        joins = launched[2 if h > 16384 else 1:]                         # after the columns and the rows, or both in one
        assert sum(g[0] for g, b in joins) * 64 >= 2 * h, (h, launched)


LOGPROB_VOCABS = [[16384] * 8, [131072], [50257], [1], [2000, 70000, 0], [12564, 12564, 12564, 12565], [1000] * 64, [100000] * 5]


def test_workspaces_never_shrink_as_rows_grow():
    for vocab in LOGPROB_VOCABS:
        for top in (0, 1, 8, 32):
            had = 0
            for rows in [*range(0, 2100), *range(2100, 9000, 97), 1 << 20, (1 << 20) + 1, 1 << 40]:
                n = coll.coll_vocab_logprob_workspace_bytes(rows, vocab, top)
                assert n >= had and (n > 0) == (rows > 0), (vocab, top, rows)
                had = n
    for p, hidden in [(1, 7), (8, 64), (3, 2565), (33, 7168), (64, 20000)]:
        sizes = [coll.coll_layernorm_workspace_bytes(p, rows, hidden) for rows in range(0, 3000, 7)]
        assert sizes == sorted(sizes) and sizes[0] > 0, (p, hidden)


@host_only
def test_a_workspace_for_more_rows_serves_fewer(tmp_path):
    calls = []
    for vocab in LOGPROB_VOCABS:
        p, ld = len(vocab), [max(v, 1) for v in vocab]
        for rows, most in ((1000, 1024), (1023, 1024), (1, 2), (500, 8192), (63, 200), (129, 130), (4095, 4096)):
            for top in (0, 8):
                calls.append(f"L.coll_vocab_logprob(b({p}), _i64(*{ld}), _i64(*{vocab}), b.one(), 1.0, b({p}), b({p}), None, {top}, b({p}), b({p}), "
                             f"{p}, {rows}, 1, b.one(), coll.coll_vocab_logprob_workspace_bytes({most}, {vocab}, {top}), None)")
    recorded(tmp_path, calls)


def test_rows_without_columns_are_refused_by_the_library():
    """The binding counts rows where they are not given; no columns are the library's to refuse."""
    import torch
    f, u = lambda *s: [DeviceTensor(torch.float32, *s)], lambda *s: [DeviceTensor(torch.uint8, *s)]  # noqa: E731
    for call in (lambda: coll.coll_layernorm(f(4, 8), None, None, f(4, 8), 0, stream=0),
                 lambda: coll.coll_layernorm_backward(f(4, 8), f(4, 8), f(4), f(4), None, f(4, 8), None, None, f(64)[0], 0, stream=0),
                 lambda: coll.coll_ckpt8_save(f(4, 8), u(64), 0, 16, stream=0), lambda: coll.coll_ckpt8_load(u(64), f(4, 8), 0, 16, stream=0),
                 lambda: coll.coll_swiglu_ckpt8(f(4, 8), f(4, 4), u(64), 0, 16, stream=0),
                 lambda: coll.coll_swiglu_backward_ckpt8(u(64), f(4, 4), f(4, 8), 0, 16, stream=0)):
        with pytest.raises(coll.CollError) as e:
            call()
        assert e.value.status == INV
