"""RMS norm on the GPU against the float64 oracle.  Tolerances as in
test_gpu_token_ops: U is half a step of fp32, HALF of the result's type, and a
sum of n terms adds n U times the sum of magnitudes along its longest chain."""
import numpy as np
import pytest

from gpu_util import BF16, F32
from oracle import token_ops
from test_gpu_token_ops import HALF, TINY, U, chain, close, coll, dev, f32, host, new, rng, u8, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


def T(xs):
    return [t for t, _ in xs]


def y_tol(y, hidden, dtype):
    # the sum of squares is off by chain + 2 roundings, its root by half of that; a rounding each of the mean, eps,
    # two of the root (1 ulp) and two products
    return (HALF[dtype] + (chain(hidden) / 2 + 8) * U) * np.abs(y) + TINY


def dx_tol(dy, dh, n, rstd, gamma, dx, dtype):
    w = np.abs(dy * gamma)
    size = w + np.abs(n) * (w * np.abs(n)).mean(1, keepdims=True)
    return HALF[dtype] * np.abs(dx) + (chain(dy.shape[1]) + 8) * U * rstd[:, None] * size + 2 * U * np.abs(dh) + TINY


def weight_tol(coll, p, rows, hidden, terms, value, wdtype):
    parts = coll.coll_rmsnorm_workspace_bytes(p, rows, hidden) // (4 * hidden)
    c = -(-p * rows // parts) + 4 + -(-parts // 16) + 16 + 8
    return HALF[wdtype] * np.abs(value) + c * U * terms + TINY


SHAPES = [
    # p, rows, hidden: one element, one lane, tails, every layout's edges, wide rows, ranks past one launch
    (1, 1, 1), (2, 3, 7), (1, 5, 8), (3, 2, 9), (2, 3, 100), (1, 9, 256), (1, 5, 257), (4, 6, 511), (1, 9, 512), (2, 4, 513), (1, 3, 1024), (1, 7, 1025),
    (3, 11, 2049), (2, 700, 2560), (2, 2, 4096), (1, 3, 4097), (3, 5, 6143), (8, 70, 7168), (1, 2, 8193), (1, 4, 8201), (2, 3, 10248), (1, 3, 12289),
    (2, 3, 16384), (1, 2, 16385), (2, 3, 20003), (33, 3, 72), (64, 2, 136), (1, 1500, 64), (5, 333, 100),
]


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("p,rows,hidden", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_forward_and_backward(coll, p, rows, hidden, dtype, wdtype, residual):
    import torch
    g = rng(50, p, rows, hidden, dtype, wdtype, residual)
    off = 1 if hidden % 2 else 0           # odd widths also start off a vector's boundary
    big = lambda: [dev(g.normal(0.3, 2.0, (rows, hidden)) * np.exp(g.normal(0, 1, (rows, 1))), dtype, off) for _ in range(p)]  # noqa: E731
    x, res = big(), big() if residual else None
    dy = [dev(g.normal(0, 1e-2, (rows, hidden)), dtype, off) for _ in range(p)]
    dh = [dev(g.normal(0, 1e-2, (rows, hidden)), dtype, off) for _ in range(p)] if residual else None
    gamma = [dev(g.normal(1, 0.3, hidden), wdtype, off) for _ in range(p)]
    y, h, dx = [[new((rows, hidden), dtype, off) for _ in range(p)] for _ in range(3)]
    rstd = f32(p, rows)
    coll.coll_rmsnorm(T(x), T(gamma), y, hidden, eps=1e-6, residual=T(res) if residual else None, h=h if residual else None, rstd=list(rstd))
    if not residual:
        h = T(x)
    dg = new((p, hidden), wdtype)
    op = coll.COLL_AVG if p % 2 else coll.COLL_SUM
    coll.coll_rmsnorm_backward(T(dy), h, list(rstd), T(gamma), dx, list(dg), workspace(coll.coll_rmsnorm_workspace_bytes(p, rows, hidden)),
                               hidden, op=op, dh=T(dh) if residual else None)
    torch.cuda.synchronize()
    total = terms = 0.0
    for r in range(p):
        he = host(h[r])
        if residual:
            want = x[r][1] + res[r][1]
            close(he, want, HALF[dtype] * np.abs(want) + U * np.abs(want), f"h {r}")
        ye, re = token_ops.rmsnorm(he, gamma[r][1], 1e-6)
        close(host(rstd[r]), re, re * (chain(hidden) / 2 + 6) * U, f"rstd {r}")
        close(host(y[r]), ye, y_tol(ye, hidden, dtype), f"y {r}")
        s = host(rstd[r])
        dhe = dh[r][1] if residual else np.zeros((rows, hidden))
        dxe, dge, n = token_ops.rmsnorm_backward(dy[r][1], he, s, gamma[r][1], dhe)
        close(host(dx[r]), dxe, dx_tol(dy[r][1], dhe, n, s, gamma[r][1], dxe, dtype), f"dx {r}")
        total, terms = total + dge, terms + np.abs(dy[r][1] * n).sum(0)
    over = p if op == coll.COLL_AVG else 1
    for r in range(p):
        close(host(dg[r]), total / over, weight_tol(coll, p, rows, hidden, terms / over, total / over, wdtype), f"dgamma {r}")
    for t in (y, dx, h) if residual else (y, dx):             # nothing past the end
        for v in t:
            assert torch.isnan(v.as_strided((1,), (1,), v.storage_offset() + v.numel()).float()).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hidden", [5, 24, 101, 1001, 5120, 8201, 17001])
def test_in_place_forms_give_the_same_bits(coll, hidden, dtype):
    import torch
    g = rng(51, hidden, dtype)
    p, rows = 2, 5
    x, res, dy, dh = [T([dev(g.normal(0, 1, (rows, hidden)), dtype) for _ in range(p)]) for _ in range(4)]
    gamma = [dev(g.normal(1, 0.2, hidden), F32)[0]] * p

    def copies(ts):
        return [t.clone() for t in ts]
    y, h = [[new((rows, hidden), dtype) for _ in range(p)] for _ in range(2)]
    rstd = f32(p, rows)
    coll.coll_rmsnorm(x, gamma, y, hidden, residual=res, h=h, rstd=list(rstd))
    for hx, yx in (("x", None), ("res", None), (None, "x"), (None, "res"), ("x", "res"), ("res", "x")):
        a, b = copies(x), copies(res)
        at = {"x": a, "res": b}
        h2 = at[hx] if hx else [new((rows, hidden), dtype) for _ in range(p)]
        y2 = at[yx] if yx else [new((rows, hidden), dtype) for _ in range(p)]
        coll.coll_rmsnorm(a, gamma, y2, hidden, residual=b, h=h2)
        assert all(torch.equal(u, v) for u, v in zip(y + h, y2 + h2)), (hx, yx)
    # the stream not kept; the row itself its own residual; no residual, in place
    for yx in (None, "x", "res"):
        a, b = copies(x), copies(res)
        y2 = {"x": a, "res": b, None: [new((rows, hidden), dtype) for _ in range(p)]}[yx]
        coll.coll_rmsnorm(a, gamma, y2, hidden, residual=b)
        assert all(torch.equal(u, v) for u, v in zip(y, y2)), yx
    a, b = copies(x), copies(x)
    y2, y3 = [[new((rows, hidden), dtype) for _ in range(p)] for _ in range(2)]
    coll.coll_rmsnorm(a, gamma, y2, hidden, residual=a, h=a)
    coll.coll_rmsnorm(b, gamma, y3, hidden, residual=copies(b))
    assert all(torch.equal(u, v) for u, v in zip(y2, y3)) and all(torch.equal(u, 2 * v) for u, v in zip(a, b))
    a = copies(x)
    y2 = [new((rows, hidden), dtype) for _ in range(p)]
    coll.coll_rmsnorm(x, gamma, y2, hidden)
    coll.coll_rmsnorm(a, gamma, a, hidden)
    assert all(torch.equal(u, v) for u, v in zip(a, y2))
    ws = workspace(coll.coll_rmsnorm_workspace_bytes(p, rows, hidden))
    dx, dg = [new((rows, hidden), dtype) for _ in range(p)], f32(p, hidden)
    coll.coll_rmsnorm_backward(dy, h, list(rstd), gamma, dx, list(dg), ws, hidden, dh=dh)
    for place in ("dy", "dh"):
        a, b = copies(dy), copies(dh)
        out, dg2 = a if place == "dy" else b, f32(p, hidden)
        coll.coll_rmsnorm_backward(a, h, list(rstd), gamma, out, list(dg2), ws, hidden, dh=b)
        assert all(torch.equal(u, v) for u, v in zip(dx, out)) and torch.equal(dg, dg2), place
    dx2 = [new((rows, hidden), dtype) for _ in range(p)]
    coll.coll_rmsnorm_backward(dy, h, list(rstd), gamma, dx2, None, ws, hidden, dh=dh)
    assert all(torch.equal(u, v) for u, v in zip(dx, dx2))


@pytest.mark.parametrize("dtype,hidden", [(BF16, 2049), (BF16, 4097), (BF16, 6145), (BF16, 137), (F32, 1025), (F32, 2561), (F32, 8193)])
def test_gradient_in_place_of_rows_whose_waves_share_elements(coll, dtype, hidden):
    """The row's last, partial unit begins a wave, whose lane shares elements with the wave before."""
    import torch
    g = rng(57, hidden, dtype)
    p, rows = 2, 2000
    gen = torch.Generator(device="cuda")
    gen.manual_seed(hidden)
    dy, dh, h = [[torch.randn(rows, hidden, generator=gen, device="cuda").to({F32: torch.float32, BF16: torch.bfloat16}[dtype]) for _ in range(p)] for _ in range(3)]
    gamma = [dev(g.normal(1, 0.2, hidden), F32)[0]] * p
    rstd = torch.rand(p, rows, generator=gen, device="cuda") + 0.5
    ws = workspace(coll.coll_rmsnorm_workspace_bytes(p, rows, hidden))
    dx, dg, dg2 = [new((rows, hidden), dtype) for _ in range(p)], f32(p, hidden), f32(p, hidden)
    coll.coll_rmsnorm_backward(dy, h, list(rstd), gamma, dx, list(dg), ws, hidden, dh=dh)
    for place in ("dy", "dh"):
        a, b = [t.clone() for t in dy], [t.clone() for t in dh]
        out = a if place == "dy" else b
        coll.coll_rmsnorm_backward(a, h, list(rstd), gamma, out, list(dg2), ws, hidden, dh=b)
        assert all(torch.equal(u, v) for u, v in zip(dx, out)) and torch.equal(dg, dg2), place


def test_backward_of_no_rows_writes_zeros(coll):
    dg = f32(2, 40)
    coll.coll_rmsnorm_backward([0, 0], [0, 0], [0, 0], None, [0, 0], list(dg), 0, 40, rows=0, dtype=F32, wdtype=F32, workspace_bytes=0)
    assert (host(dg) == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hidden", [7, 40, 100, 1024, 2049, 7168, 9000, 20003])
def test_rows_of_every_magnitude(coll, hidden, dtype):
    """Values whose squares leave fp32's range on either side, with eps next to nothing; a NaN, an infinity or zeros in
    one row stay in that row's results."""
    g = rng(52, hidden, dtype)
    x = g.uniform(0.5, 1.5, (12, hidden)) * np.where(g.random((12, hidden)) < 0.5, -1, 1)
    scale = [1.0, 2.0 ** 120, 2.0 ** 70, 2.0 ** -70, 2.0 ** -110, 2.0 ** 60, 2.0 ** -45, 1.0, 1.0, 1.0, 2.0 ** 126, 2.0 ** -125]
    x *= np.array(scale)[:, None]
    x[7, hidden // 2] = np.nan
    x[8, hidden - 1] = np.inf
    x[9] = 0.0
    t, xe = dev(x, dtype)
    gamma, ge = dev(g.normal(1, 0.2, hidden), F32)
    for eps in (0.0, float(np.float32(1e-30)), float(np.float32(1e-5))):
        y, rstd = new((12, hidden), dtype), f32(12)
        coll.coll_rmsnorm([t], [gamma], [y], hidden, eps=eps, rstd=[rstd])
        got, s = host(y), host(rstd)
        assert np.isnan(got[7]).all() and np.isnan(s[7])
        assert np.isnan(got[8, hidden - 1]) and (got[8, :hidden - 1] == 0).all() and s[8] == 0
        assert np.isnan(got[9]).all() if eps == 0 else (got[9] == 0).all()
        keep = [i for i in range(12) if i not in (7, 8, 9)]
        ye, re = token_ops.rmsnorm(xe[keep], ge, eps)
        close(s[keep], re, re * (chain(hidden) / 2 + 8) * U + 2.0 ** -149, "rstd")
        close(got[keep], ye, y_tol(ye, hidden, dtype), "y")


CODES = [
    # p, rows, hidden, group: every layout, groups wider than a layout's lanes, ranks past one launch
    (1, 1, 16, 16), (2, 9, 64, 32), (1, 5, 128, 128), (3, 4, 256, 256), (2, 3, 256, 64), (3, 5, 1536, 512), (2, 7, 512, 512), (8, 33, 7168, 128), (1, 9, 2560, 64),
    (1, 3, 5120, 256), (2, 2, 12288, 512), (1, 3, 16384, 64), (2, 3, 20480, 512), (34, 2, 512, 16),
]


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("p,rows,hidden,group", CODES)
def test_output_in_8_bits(coll, p, rows, hidden, group, dtype, wdtype):
    import torch
    g = rng(53, p, rows, hidden, group, dtype, wdtype)
    x, res = [[dev(g.normal(0, 2, (rows, hidden)) * np.exp(g.normal(0, 1, hidden)), dtype) for _ in range(p)] for _ in range(2)]
    gamma = [dev(g.normal(1, 0.3, hidden), wdtype) for _ in range(p)]
    rb = coll.coll_ckpt8_row_bytes(hidden, group)
    y8, alone, h, y, rstd = u8(p, rows, rb), u8(p, rows, rb), [new((rows, hidden), dtype) for _ in range(p)], [new((rows, hidden), dtype) for _ in range(p)], f32(p, rows)
    coll.coll_rmsnorm_fp8(T(x), T(gamma), list(y8), hidden, group, residual=T(res), h=h, rstd=list(rstd), y=y)
    coll.coll_rmsnorm_fp8(T(x), T(gamma), list(alone), hidden, group, residual=T(res))
    y2, h2, rstd2 = [new((rows, hidden), dtype) for _ in range(p)], [new((rows, hidden), dtype) for _ in range(p)], f32(p, rows)
    coll.coll_rmsnorm(T(x), T(gamma), y2, hidden, residual=T(res), h=h2, rstd=list(rstd2))
    torch.cuda.synchronize()
    assert torch.equal(y8, alone)
    for r in range(p):
        assert torch.equal(h[r], h2[r])
        he = host(h[r])
        ye, re = token_ops.rmsnorm(he, gamma[r][1], 1e-6)
        for got, s in ((y[r], rstd[r]), (y2[r], rstd2[r])):
            close(host(s), re, re * (chain(hidden) / 2 + 6) * U, f"rstd {r}")
            close(host(got), ye, y_tol(ye, hidden, dtype), f"y {r}")
        rows8 = y8[r].cpu().numpy()
        scales = np.ascontiguousarray(rows8[:, hidden:hidden + 4 * (hidden // group)]).view("<f4").astype(np.float64)
        off = y_tol(ye, hidden, F32)                          # of the value that was encoded
        amax = np.abs(ye).reshape(rows, -1, group).max(2)
        close(scales, np.maximum(amax, 2.0 ** -110) / 448, amax / 448 * ((chain(hidden) / 2 + 8) * U + 2 * U) + TINY, f"scales {r}")
        value = token_ops.ckpt8_values(rows8, hidden, group).astype(np.float64)
        # half a step of e4m3 (or of its subnormals), off by the scaled product's rounding and the scale's
        step = np.maximum(2.0 ** -4 * np.abs(ye), 2.0 ** -10 * np.repeat(scales, group, axis=1))
        close(value, ye, step * (1 + 2.0 ** -18) + 2 * off, f"values {r}")
        assert (rows8[:, hidden + 4 * (hidden // group):] == 0).all()
        if dtype == F32:                                      # then y holds the very values that were encoded
            assert np.array_equal(rows8, token_ops.ckpt8_rows(y[r].cpu().numpy(), group))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("hidden", [7, 48, 100, 512, 1024, 2049, 5120, 7168, 16384, 20003, 20480])
def test_rows_whose_reciprocal_leaves_fp32(coll, hidden, residual, dtype):
    """1 / rms above the largest fp32 value, or among its denormals: y and its 8-bit rows are those of any other row;
    rstd is the nearest fp32 value, an infinity above them."""
    import torch
    g = rng(58, hidden, residual, dtype)
    down = [-129, -130, -131] if dtype == BF16 else [-129, -130, -140, -147]
    scale = 2.0 ** np.array([*down, 0, -127, 126, *down, 20])
    rows = len(scale)
    sign = np.where(g.random((rows, hidden)) < 0.5, -1, 1)
    x, xe = dev(g.uniform(0.5, 1.5, (rows, hidden)) * sign * scale[:, None], dtype)
    if residual:                                              # the values from both: x again, or nothing
        res, he = [x], 2 * xe
        he[5], res[0] = xe[5], x.clone()
        res[0][5] = 0.0
    else:
        res, he = None, xe
    gamma, ge = dev(g.normal(1, 0.2, hidden), F32)
    y, rstd, h = new((rows, hidden), dtype), f32(rows), [new((rows, hidden), dtype)] if residual else None
    coll.coll_rmsnorm([x], [gamma], [y], hidden, eps=0.0, residual=res, h=h, rstd=[rstd])
    if residual:
        close(host(h[0]), he, 0.0, "h")
    ye, re = token_ops.rmsnorm(he, ge, 0.0)
    over = re > 2.0 ** 128
    assert over.any() and np.isposinf(host(rstd)[over]).all()
    close(host(rstd)[~over], re[~over], re[~over] * (chain(hidden) / 2 + 8) * U + 2.0 ** -149, "rstd")
    close(host(y), ye, y_tol(ye, hidden, dtype), "y")
    if hidden % 16 == 0:
        group = 512 if hidden % 512 == 0 else 16
        rb = coll.coll_ckpt8_row_bytes(hidden, group)
        y8, again = u8(rows, rb), new((rows, hidden), dtype)
        coll.coll_rmsnorm_fp8([x], [gamma], [y8], hidden, group, eps=0.0, residual=res, y=[again])
        close(host(again), ye, y_tol(ye, hidden, dtype), "y beside the codes")
        value = token_ops.ckpt8_values(y8.cpu().numpy(), hidden, group).astype(np.float64)
        amax = np.repeat(np.abs(ye).reshape(rows, -1, group).max(2), group, axis=1)
        # half a step of e4m3 (or of its subnormals, 2^-10 of the scale amax / 448), off by roundings far below 2^-12
        close(value, ye, (2.0 ** -4 * np.abs(ye) + 2.0 ** -10 * amax / 448) * (1 + 2.0 ** -12) + 2 * y_tol(ye, hidden, F32), "values")


@pytest.mark.parametrize("dtype,hidden,group", [(BF16, 64, 16), (F32, 256, 256), (BF16, 512, 512), (F32, 2560, 64), (BF16, 7168, 128), (F32, 7168, 512),
                                                (BF16, 16384, 128), (BF16, 20480, 512)])
def test_in_place_forms_with_8_bit_rows(coll, dtype, hidden, group):
    """h and y in the place of x and the residual, either of them or both, in the pass that writes the codes."""
    import torch
    g = rng(59, hidden, group, dtype)
    p, rows = 2, 5
    x, res = [T([dev(g.normal(0, 1, (rows, hidden)), dtype) for _ in range(p)]) for _ in range(2)]
    gamma = [dev(g.normal(1, 0.2, hidden), F32)[0]] * p
    rb = coll.coll_ckpt8_row_bytes(hidden, group)

    def run(hx, yx, x=x, res=res):
        at = {"x": [t.clone() for t in x], "res": [t.clone() for t in res] if res else None, "new": [new((rows, hidden), dtype) for _ in range(p)], None: None}
        y8, rstd = u8(p, rows, rb), f32(p, rows)
        if "new" == hx == yx:
            at["new2"] = [new((rows, hidden), dtype) for _ in range(p)]
            yx = "new2"
        coll.coll_rmsnorm_fp8(at["x"], gamma, list(y8), hidden, group, residual=at["res"], h=at[hx], rstd=list(rstd), y=at[yx])
        return at[hx], at[yx], y8, rstd
    h, y, y8, rstd = run("new", "new")
    for hx in ("x", "res", "new", None):
        for yx in ("x", "res", "new", None):
            if hx == yx:
                continue
            got = run(hx, yx)
            assert hx is None or all(torch.equal(a, b) for a, b in zip(h, got[0])), (hx, yx)
            assert yx is None or all(torch.equal(a, b) for a, b in zip(y, got[1])), (hx, yx)
            assert torch.equal(y8, got[2]) and torch.equal(rstd, got[3]), (hx, yx)
    plain = run(None, "new", res=None)
    for yx in ("x", None):
        got = run(None, yx, res=None)
        assert yx is None or all(torch.equal(a, b) for a, b in zip(plain[1], got[1]))
        assert torch.equal(plain[2], got[2]) and torch.equal(plain[3], got[3])


def test_codes_of_rows_with_a_non_finite_value(coll):
    for hidden, dtype in ((64, F32), (2560, BF16), (20480, BF16)):
        x = rng(54).normal(0, 1, (3, hidden))
        x[1, 5] = np.nan
        t, _ = dev(x, dtype)
        y8 = u8(3, coll.coll_ckpt8_row_bytes(hidden, 32))
        coll.coll_rmsnorm_fp8([t], None, [y8], hidden, 32)
        back = new((3, hidden), F32)
        coll.coll_ckpt8_load([y8], [back], hidden, 32)
        got = host(back)
        assert np.isnan(got[1]).all() and np.isfinite(got[[0, 2]]).all()


def test_gradient_by_differences(coll):
    """dx (of x and of the residual alike) and dgamma against central differences of the kernel's own forward pass."""
    import torch
    g = rng(55)
    p, rows, hidden = 2, 3, 37
    x, res = [[g.normal(0, 1, (rows, hidden)).astype(np.float32) for _ in range(p)] for _ in range(2)]
    gamma = g.normal(1, 0.3, hidden).astype(np.float32)
    dy, dh = [[g.normal(0, 1, (rows, hidden)).astype(np.float32) for _ in range(p)] for _ in range(2)]

    def forward(x, res, gamma):
        y, h = [[new((rows, hidden), F32) for _ in range(p)] for _ in range(2)]
        rstd = f32(p, rows)
        coll.coll_rmsnorm([dev(v, F32)[0] for v in x], [dev(gamma, F32)[0]] * p, y, hidden, residual=[dev(v, F32)[0] for v in res], h=h, rstd=list(rstd))
        return y, h, rstd

    def loss(*a):
        y, h, _ = forward(*a)
        return sum((host(u) * d).sum() for u, d in zip(y + h, dy + dh))
    _, h, rstd = forward(x, res, gamma)
    dx, dg = [new((rows, hidden), F32) for _ in range(p)], f32(p, hidden)
    coll.coll_rmsnorm_backward([dev(v, F32)[0] for v in dy], h, list(rstd), [dev(gamma, F32)[0]] * p, dx, list(dg),
                               workspace(coll.coll_rmsnorm_workspace_bytes(p, rows, hidden)), hidden, dh=[dev(v, F32)[0] for v in dh])
    torch.cuda.synchronize()
    # step 2^-6: the third derivative's h^2 term stays below 2^-12 * 8, and the loss's 444 terms are rounded by 40 U each at most
    e = 2.0 ** -6
    lim = e * e * 8 + 444 * 40 * U * 4 / (2 * e)
    for r, i, j in [(0, 0, 0), (1, 2, 36), (0, 1, 17), (1, 0, 5)]:
        for k in (0, 1):
            a, b = [[v.copy() for v in x], [v.copy() for v in res]], [[v.copy() for v in x], [v.copy() for v in res]]
            a[k][r][i, j] += np.float32(e)
            b[k][r][i, j] -= np.float32(e)
            step = float(a[k][r][i, j]) - float(b[k][r][i, j])
            assert abs((loss(*a, gamma) - loss(*b, gamma)) / step - host(dx[r])[i, j]) < lim
    for j in (0, 20, 36):
        a, b = gamma.copy(), gamma.copy()
        a[j] += np.float32(e)
        b[j] -= np.float32(e)
        assert abs((loss(x, res, a) - loss(x, res, b)) / (float(a[j]) - float(b[j])) - host(dg[0])[j]) < lim


def test_rows_past_2_31_elements(coll):
    import torch
    g = rng(56)
    hidden, rows = 7168, 300001
    pick = [0, 149796, 149797, 300000]
    x, res = [torch.zeros(rows, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    a, ae = dev(g.normal(0, 1, (4, hidden)), BF16)
    b, be = dev(g.normal(0, 1, (4, hidden)), BF16)
    x[pick], res[pick] = a, b
    y8, rstd, y = torch.zeros(rows, coll.coll_ckpt8_row_bytes(hidden, 128), dtype=torch.uint8, device="cuda"), f32(rows), torch.empty_like(x)
    coll.coll_rmsnorm_fp8([x], None, [y8], hidden, 128, residual=[res], h=[x], rstd=[rstd], y=[y])      # h in place
    torch.cuda.synchronize()
    he = host(x[pick])
    close(he, ae + be, (HALF[BF16] + U) * np.abs(ae + be), "h")
    ye, re = token_ops.rmsnorm(he, np.ones(hidden), 1e-6)
    close(host(y[pick]), ye, y_tol(ye, hidden, BF16), "y")
    value = token_ops.ckpt8_values(y8[pick].cpu().numpy(), hidden, 128)
    assert (np.abs(value - ye) <= 2.0 ** -4 * np.abs(ye) * 1.001 + 2.0 ** -10).all()
    dx, dg = torch.empty_like(x), f32(hidden)
    coll.coll_rmsnorm_backward([y], [x], [rstd], None, [dx], [dg], workspace(coll.coll_rmsnorm_workspace_bytes(1, rows, hidden)), hidden)
    yb, s = host(y[pick]), host(rstd[pick])
    dxe, dge, n = token_ops.rmsnorm_backward(yb, he, s, np.ones(hidden))
    close(host(dx[pick]), dxe, dx_tol(yb, 0 * yb, n, s, np.ones(hidden), dxe, BF16), "dx")
    close(host(dg), dge, weight_tol(coll, 1, rows, hidden, np.abs(yb * n).sum(0), dge, F32), "dgamma")
