"""Token-wise operators on the GPU against the float64 oracle.

Tolerances are bounds of the rounding each result can have, from the number
formats and the length of the sums: U is half a step of fp32; a result in
bf16 or fp32 adds half its own step (HALF); a sum of n terms adds n U times
the sum of magnitudes along its longest chain of additions.
"""
import numpy as np
import pytest

from gpu_util import BF16, F32, torch_dtype
from oracle import fp8, ref, token_ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
TINY = 1e-37        # below it, fp32 results may flush to zero


@pytest.fixture(scope="module")
def coll():
    import torch
    import collective_communication_primitives_coll_amd as c
    torch.cuda.set_device(0)
    c.lib()
    return c


def rng(*seed):
    return np.random.default_rng([7300, *[int(s) for s in seed]])


def dev(a, dtype, off=0):
    """Device tensor of the values a rounded to dtype (off: elements past a
    fresh allocation), and the float64 values it holds."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch_dtype(dtype))
    d = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")[off:].view(t.shape)
    d.copy_(t)
    return d, t.double().numpy()


def new(shape, dtype, off=0):
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + off + 16,), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    return buf[off:off + n].view(shape)


def host(t):
    return t.detach().double().cpu().numpy()


def f32(*shape):
    import torch
    return torch.full(shape, float("nan"), dtype=torch.float32, device="cuda")


def u8(*shape):
    import torch
    return torch.full(shape, 0xA5, dtype=torch.uint8, device="cuda")


def workspace(n):
    import torch
    return torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")[:n]     # NaN patterns


def close(got, want, tol, what):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN positions"
    inf = ~fine & ~np.isnan(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities"
    tol = np.broadcast_to(tol, want.shape)
    over = np.abs(got - want)[fine] - tol[fine]
    if over.size and over.max() > 0:
        i = int(np.argmax(over))
        raise AssertionError(f"{what}: off by {np.abs(got - want)[fine][i]:g}, allowed {tol[fine][i]:g}, value {want[fine][i]:g}")


# ----------------------------------------------------------------------------
# Layer norm
# ----------------------------------------------------------------------------

def chain(hidden):
    """Longest chain of additions of a row's sum: a lane's elements, then lanes and waves."""
    return 16 + 6 + 16 if hidden <= 16384 else 8 * -(-hidden // 8192) + 6 + 16


def ln_forward_tol(x, gamma, beta, mean, rstd, y, dtype):
    c = chain(x.shape[1]) + 8
    r, far = rstd[:, None], np.abs(x).mean(1, keepdims=True)
    return HALF[dtype] * np.abs(y) + c * U * (r * np.abs(gamma) * (np.abs(x - mean[:, None]) + far) + np.abs(beta)) * 2 + TINY


def ln_backward_tol(dy, n, rstd, gamma, dx, dtype):
    c = chain(dy.shape[1]) + 8
    w = np.abs(dy * gamma)
    size = w + w.mean(1, keepdims=True) + np.abs(n) * (w * np.abs(n)).mean(1, keepdims=True)
    return HALF[dtype] * np.abs(dx) + c * U * rstd[:, None] * size + TINY


def weight_tol(coll, p, rows, hidden, terms, value, wdtype):
    parts = coll.coll_layernorm_workspace_bytes(p, rows, hidden) // (8 * hidden)
    c = -(-p * rows // parts) + 4 + -(-parts // 16) + 16 + 8
    return HALF[wdtype] * np.abs(value) + c * U * terms + TINY


LN_SHAPES = [
    # p, rows, hidden: one element, one lane, tails, every layout's edges, wide rows, ranks past one launch
    (1, 1, 1), (2, 3, 7), (1, 5, 8), (3, 2, 9), (4, 6, 511), (1, 9, 512), (2, 4, 513), (2, 5, 1000), (1, 3, 1024), (1, 7, 1025),
    (3, 11, 2049), (2, 2, 4096), (1, 3, 4097), (8, 70, 7168), (1, 2, 8192), (1, 2, 8193), (2, 3, 16384), (1, 2, 16385), (2, 3, 20003),
    (33, 3, 72), (64, 2, 136), (1, 1500, 64), (5, 333, 100),
    # the layouts whose lanes are no power of two
    (2, 700, 2560), (1, 3, 3071), (3, 5, 4100), (2, 6, 5120), (1, 5, 6143), (1, 4, 8201), (2, 3, 10248), (1, 3, 12288),
]


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("p,rows,hidden", LN_SHAPES)
def test_layernorm_forward_and_backward(coll, p, rows, hidden, dtype, wdtype):
    import torch
    g = rng(p, rows, hidden, dtype, wdtype)
    off = 1 if hidden % 2 else 0           # odd widths also start off a vector's boundary
    x, dy = [], []
    for r in range(p):
        x.append(dev(g.normal(1.5, 2.0, (rows, hidden)) * np.exp(g.normal(0, 1, (rows, 1))), dtype, off))
        dy.append(dev(g.normal(0, 1e-2, (rows, hidden)), dtype, off))
    gamma = [dev(g.normal(1, 0.3, hidden), wdtype, off) for _ in range(p)]
    beta = [dev(g.normal(0, 0.5, hidden), wdtype) for _ in range(p)]
    T = lambda xs: [t for t, _ in xs]  # noqa: E731
    y, dx = [new((rows, hidden), dtype, off) for _ in range(p)], [new((rows, hidden), dtype) for _ in range(p)]
    mean, rstd = f32(p, rows), f32(p, rows)
    coll.coll_layernorm(T(x), T(gamma), T(beta), y, hidden, eps=1e-5, mean=list(mean), rstd=list(rstd))
    dg, db = new((p, hidden), wdtype), new((p, hidden), wdtype)
    ws = workspace(coll.coll_layernorm_workspace_bytes(p, rows, hidden))
    op = coll.COLL_AVG if p % 2 else coll.COLL_SUM
    coll.coll_layernorm_backward(T(dy), T(x), list(mean), list(rstd), T(gamma), dx, list(dg), list(db), ws, hidden, op=op)
    torch.cuda.synchronize()
    sg = sb = tg = tb = 0.0
    for r in range(p):
        ye, me, re = token_ops.layernorm(x[r][1], gamma[r][1], beta[r][1], 1e-5)
        far = np.abs(x[r][1]).mean(1)
        close(host(mean[r]), me, (chain(hidden) + 4) * U * far + TINY, f"mean {r}")
        # var's rounding, and the mean's square
        close(host(rstd[r]), re, re * ((chain(hidden) + 8) * U + re ** 2 * ((chain(hidden) + 4) * U * far) ** 2), f"rstd {r}")
        close(host(y[r]), ye, ln_forward_tol(x[r][1], gamma[r][1], beta[r][1], me, re, ye, dtype), f"y {r}")
        # backward from the statistics that the kernel was given
        m, s = host(mean[r]), host(rstd[r])
        dxe, dge, dbe, n = token_ops.layernorm_backward(dy[r][1], x[r][1], m, s, gamma[r][1])
        close(host(dx[r]), dxe, ln_backward_tol(dy[r][1], n, s, gamma[r][1], dxe, dtype), f"dx {r}")
        sg, sb, tg, tb = sg + dge, sb + dbe, tg + np.abs(dy[r][1] * n).sum(0), tb + np.abs(dy[r][1]).sum(0)
    over = p if op == coll.COLL_AVG else 1
    for r in range(p):
        close(host(dg[r]), sg / over, weight_tol(coll, p, rows, hidden, tg / over, sg / over, wdtype), f"dgamma {r}")
        close(host(db[r]), sb / over, weight_tol(coll, p, rows, hidden, tb / over, sb / over, wdtype), f"dbeta {r}")
    assert torch.isnan(y[0].view(-1).as_strided((1,), (1,), y[0].storage_offset() + y[0].numel()).float()).all()   # nothing past the end


def test_layernorm_without_weights_or_statistics_and_in_place(coll):
    import torch
    g = rng(1)
    for hidden in (24, 1001, 5120, 17000):
        x, xe = dev(g.normal(0, 1, (5, hidden)), BF16)
        y, y2 = new((5, hidden), BF16), x.clone()
        coll.coll_layernorm([x], None, None, [y], hidden)
        coll.coll_layernorm([y2], None, None, [y2], hidden)
        ye, me, re = token_ops.layernorm(xe, np.ones(hidden), np.zeros(hidden), 1e-5)
        close(host(y), ye, ln_forward_tol(xe, np.ones(hidden), np.zeros(hidden), me, re, ye, BF16), "y")
        assert torch.equal(y, y2)
        dy, dye = dev(g.normal(0, 1, (5, hidden)), BF16)
        mean, rstd = dev(me, F32), dev(re, F32)
        ws = workspace(coll.coll_layernorm_workspace_bytes(1, 5, hidden))
        dx, dx2, dg = new((5, hidden), BF16), dy.clone(), f32(hidden)
        coll.coll_layernorm_backward([dy], [x], [mean[0]], [rstd[0]], None, [dx], None, None, ws, hidden)
        coll.coll_layernorm_backward([dx2], [x], [mean[0]], [rstd[0]], None, [dx2], [dg], None, ws, hidden)
        dxe, dge, _, n = token_ops.layernorm_backward(dye, xe, mean[1], rstd[1], np.ones(hidden))
        close(host(dx), dxe, ln_backward_tol(dye, n, rstd[1], np.ones(hidden), dxe, BF16), "dx")
        assert torch.equal(dx, dx2)
        close(host(dg), dge, weight_tol(coll, 1, 5, hidden, np.abs(dye * n).sum(0), dge, F32), "dgamma")


def test_layernorm_backward_of_no_rows_writes_zeros(coll):
    dg, db = f32(2, 40), f32(2, 40)
    coll.coll_layernorm_backward([0, 0], [0, 0], [0, 0], [0, 0], None, [0, 0], list(dg), list(db), 0, 40, rows=0, dtype=F32,
                                 wdtype=F32, workspace_bytes=0)
    assert (host(dg) == 0).all() and (host(db) == 0).all()


def test_layernorm_rows_apart(coll):
    """A NaN, an infinity or a constant in one row stays in that row's results."""
    g = rng(2)
    for hidden in (64, 4096, 7168, 20000):
        x = g.normal(0, 1, (6, hidden))
        x[1, 3] = np.nan
        x[3, hidden - 1] = np.inf
        x[4] = 3.0                                   # no variance: y = beta
        t, xe = dev(x, F32)
        y, mean, rstd = new((6, hidden), F32), f32(6), f32(6)
        beta, be = dev(g.normal(0, 1, hidden), F32)
        coll.coll_layernorm([t], None, [beta], [y], hidden, mean=[mean], rstd=[rstd])
        got = host(y)
        assert np.isnan(got[1]).all() and np.isnan(got[3]).any() and not np.isfinite(got[3]).all()
        assert np.array_equal(got[4], be) and host(mean)[4] == 3.0
        keep = [0, 2, 5]
        ye, me, re = token_ops.layernorm(xe[keep], np.ones(hidden), be, 1e-5)
        close(got[keep], ye, ln_forward_tol(xe[keep], np.ones(hidden), be, me, re, ye, F32), "other rows")


def test_layernorm_of_a_far_mean(coll):
    """Rows whose mean is 1000 times their spread keep their variance."""
    x, xe = dev(rng(3).normal(1000, 1, (4, 3000)), F32)
    y = new((4, 3000), F32)
    coll.coll_layernorm([x], None, None, [y], 3000)
    ye, me, re = token_ops.layernorm(xe, np.ones(3000), np.zeros(3000), 1e-5)
    close(host(y), ye, ln_forward_tol(xe, np.ones(3000), np.zeros(3000), me, re, ye, F32), "y")


def test_layernorm_gradient_by_differences(coll):
    """dx, dgamma and dbeta against central differences of the kernel's own forward pass (fp32, p = 2)."""
    import torch
    g = rng(4)
    p, rows, hidden = 2, 3, 37
    x = [g.normal(0, 1, (rows, hidden)).astype(np.float32) for _ in range(p)]
    gamma, beta = g.normal(1, 0.3, hidden).astype(np.float32), g.normal(0, 1, hidden).astype(np.float32)
    dy = [g.normal(0, 1, (rows, hidden)).astype(np.float32) for _ in range(p)]

    def forward(x, gamma, beta):
        y = [new((rows, hidden), F32) for _ in range(p)]
        mean, rstd = f32(p, rows), f32(p, rows)
        coll.coll_layernorm([dev(v, F32)[0] for v in x], [dev(gamma, F32)[0]] * p, [dev(beta, F32)[0]] * p, y, hidden,
                            mean=list(mean), rstd=list(rstd))
        return [host(v) for v in y], mean, rstd

    def loss(*a):
        return sum((y * d).sum() for y, d in zip(forward(*a)[0], dy))
    _, mean, rstd = forward(x, gamma, beta)
    dx, dg, db = [new((rows, hidden), F32) for _ in range(p)], f32(p, hidden), f32(p, hidden)
    coll.coll_layernorm_backward([dev(v, F32)[0] for v in dy], [dev(v, F32)[0] for v in x], list(mean), list(rstd),
                                 [dev(gamma, F32)[0]] * p, dx, list(dg), list(db),
                                 workspace(coll.coll_layernorm_workspace_bytes(p, rows, hidden)), hidden)
    torch.cuda.synchronize()
    # step 2^-6 (exact in the sums to 2 U of values of size 4): the third derivative's h^2 term stays below
    # 2^-12 * 8, and the loss, of some 10 units, is rounded by 222 terms of 40 U each at most
    h, lim = 2.0 ** -6, 2.0 ** -12 * 8 + 222 * 40 * U * 4 / (2 * 2.0 ** -6)
    for r, i, j in [(0, 0, 0), (1, 2, 36), (0, 1, 17), (1, 0, 5)]:
        a, b = [v.copy() for v in x], [v.copy() for v in x]
        a[r][i, j] += np.float32(h)
        b[r][i, j] -= np.float32(h)
        step = float(a[r][i, j]) - float(b[r][i, j])
        assert abs((loss(a, gamma, beta) - loss(b, gamma, beta)) / step - host(dx[r])[i, j]) < lim
    for j in (0, 20, 36):
        for k, got in ((0, dg), (1, db)):
            a, b = [gamma.copy(), beta.copy()], [gamma.copy(), beta.copy()]
            a[k][j] += np.float32(h)
            b[k][j] -= np.float32(h)
            step = float(a[k][j]) - float(b[k][j])
            assert abs((loss(x, *a) - loss(x, *b)) / step - host(got[0])[j]) < lim


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("hidden", [8, 64, 320, 1024, 2560, 4096, 7168, 12288, 16384, 16400])
def test_layernorm_of_whole_units_off_their_boundary(coll, hidden, dtype, wdtype):
    """Widths of whole 16-byte units whose every buffer starts at an element's address only: the same bits as from
    aligned buffers."""
    import torch
    g = rng(22, hidden, dtype, wdtype)
    rows, group = 5, 16
    data = [g.normal(0.5, 2, (rows, hidden)), g.normal(0, 1, (rows, hidden)), g.normal(1, 0.3, hidden), g.normal(0, 0.5, hidden)]
    got = []
    for off in (0, 1, 3):
        x, dy, gamma, beta = [dev(a, t, off)[0] for a, t in zip(data, (dtype, dtype, wdtype, wdtype))]
        if off:
            assert all(t.data_ptr() % 16 for t in (x, dy, gamma, beta))
        y, dx, y2, dx2, again = [new((rows, hidden), dtype, off) for _ in range(5)]
        dg, db, dg2, db2 = [new((hidden,), wdtype, off) for _ in range(4)]
        mean, rstd = f32(rows), f32(rows)
        ws = workspace(coll.coll_layernorm_workspace_bytes(1, rows, hidden))
        coll.coll_layernorm([x], [gamma], [beta], [y], hidden, mean=[mean], rstd=[rstd])
        coll.coll_layernorm_backward([dy], [x], [mean], [rstd], [gamma], [dx], [dg], [db], ws, hidden)
        out = [y, mean, rstd, dx, dg, db]
        if hidden % group == 0:
            ck = u8(rows, coll.coll_ckpt8_row_bytes(hidden, group))
            coll.coll_layernorm_ckpt8([x], [gamma], [beta], [y2], [mean], [rstd], [ck], hidden, group)
            coll.coll_layernorm_backward_ckpt8([dy], [ck], [mean], [rstd], [gamma], [dx2], [dg2], [db2], ws, hidden, group, beta=[beta], y=[again])
            out += [y2, ck, dx2, dg2, db2, again]
        torch.cuda.synchronize()
        got.append([t.clone() for t in out])
        for t in (y, dx, dg, db):                              # nothing past the end
            assert torch.isnan(t.view(-1).as_strided((1,), (1,), t.storage_offset() + t.numel()).float()).all()
    assert not torch.isnan(got[0][0].float()).any() and not torch.isnan(got[0][3].float()).any()
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hidden", [7, 9, 136, 320, 1000, 1800, 2560, 3001, 4608, 7168, 9000, 12296, 20003])
def test_layernorm_gradient_of_a_large_constant_row(coll, hidden, dtype):
    """A constant row whose mean times 1 / sqrt(eps) passes fp32's range: its normalised values are 0 and its
    gradient is finite, in every layout, whether the row fills its lanes or not."""
    g = rng(21, hidden, dtype)
    x = g.normal(0, 1, (3, hidden))
    x[1] = 2.0 ** 110                                         # times 1e6: 1.3e39
    x, xe = dev(x, dtype)
    y, mean, rstd = new((3, hidden), dtype), f32(3), f32(3)
    coll.coll_layernorm([x], None, None, [y], hidden, eps=1e-12, mean=[mean], rstd=[rstd])
    assert (host(y)[1] == 0).all() and host(mean)[1] == 2.0 ** 110
    m, s = host(mean), host(rstd)
    assert m[1] * s[1] > 3.5e38
    dy, dye = dev(g.normal(0, 1, (3, hidden)), dtype)
    dx, dg, db = new((3, hidden), dtype), f32(hidden), f32(hidden)
    ws = workspace(coll.coll_layernorm_workspace_bytes(1, 3, hidden))
    dxe, dge, dbe, n = token_ops.layernorm_backward(dye, xe, m, s, np.ones(hidden))

    def check(what):
        close(host(dx), dxe, ln_backward_tol(dye, n, s, np.ones(hidden), dxe, dtype), f"dx {what}")
        close(host(dg), dge, weight_tol(coll, 1, 3, hidden, np.abs(dye * n).sum(0), dge, F32), f"dgamma {what}")
        close(host(db), dbe, weight_tol(coll, 1, 3, hidden, np.abs(dye).sum(0), dbe, F32), f"dbeta {what}")
    coll.coll_layernorm_backward([dy], [x], [mean], [rstd], None, [dx], [dg], [db], ws, hidden, wdtype=F32)
    check("of the rows")
    if hidden % 64 == 0:
        rows_e = token_ops.ckpt8_rows(xe.astype(np.float32), 32)
        xe = token_ops.ckpt8_values(rows_e, hidden, 32).astype(np.float64)
        assert (xe[1] == 2.0 ** 110).all()                    # 448 steps of its scale
        ck = u8(3, coll.coll_ckpt8_row_bytes(hidden, 32))
        coll.coll_ckpt8_save([x], [ck], hidden, 32)
        dxe, dge, dbe, n = token_ops.layernorm_backward(dye, xe, m, s, np.ones(hidden))
        coll.coll_layernorm_backward_ckpt8([dy], [ck], [mean], [rstd], None, [dx], [dg], [db], ws, hidden, 32, wdtype=F32)
        check("of the checkpoint")


# ----------------------------------------------------------------------------
# 8-bit checkpoints
# ----------------------------------------------------------------------------

CK_SHAPES = [(1, 1, 16, 16), (2, 3, 48, 16), (3, 5, 96, 32), (1, 7, 512, 512), (2, 9, 1536, 512), (8, 17, 7168, 128), (1, 260, 64, 64),
             (35, 2, 256, 256), (2, 2, 16384, 64), (1, 3, 20480, 256)]


def narrowed(v32, dtype):
    return ref.bf16_to_f32(ref.f32_to_bf16_rne(v32.reshape(-1))).reshape(v32.shape) if dtype == BF16 else v32


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("p,rows,hidden,group", CK_SHAPES)
def test_checkpoint_is_the_format_bit_for_bit(coll, p, rows, hidden, group, dtype):
    import torch
    g = rng(10, p, rows, hidden, group, dtype)
    off = 3                                        # element-aligned rows, 16-byte aligned checkpoints
    x = [dev(g.normal(0, 1, (rows, hidden)) * np.exp(g.normal(0, 4, (rows, hidden // group)).repeat(group, 1)), dtype, off) for _ in range(p)]
    x[0][0][0, :group] = 0                         # a group of zeros
    x[0][1][0, :group] = 0
    rb = coll.coll_ckpt8_row_bytes(hidden, group)
    ck, back = u8(p, rows, rb), [new((rows, hidden), dtype, 1) for _ in range(p)]
    coll.coll_ckpt8_save([t for t, _ in x], list(ck), hidden, group)
    coll.coll_ckpt8_load(list(ck), back, hidden, group)
    torch.cuda.synchronize()
    for r in range(p):
        rows_e = token_ops.ckpt8_rows(x[r][1].astype(np.float32), group)
        assert np.array_equal(ck[r].cpu().numpy(), rows_e), f"rank {r}"
        v = narrowed(token_ops.ckpt8_values(rows_e, hidden, group), dtype)
        assert np.array_equal(host(back[r]), v.astype(np.float64)), f"rank {r} values"


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_checkpoint_group_with_a_non_finite_value_is_nan(coll, dtype):
    x = rng(11).normal(0, 1, (4, 128))
    for i, (j, v) in enumerate([(0, np.nan), (40, np.inf), (95, -np.inf), (127, -np.nan)]):
        x[i, j] = v
    t, xe = dev(x, dtype)
    ck, back = u8(4, coll.coll_ckpt8_row_bytes(128, 32)), new((4, 128), dtype)
    coll.coll_ckpt8_save([t], [ck], 128, 32)
    coll.coll_ckpt8_load([ck], [back], 128, 32)
    got = host(back).reshape(4, 4, 32)
    for i, k in enumerate([0, 1, 2, 3]):
        assert np.isnan(got[i, k]).all() and np.isfinite(np.delete(got[i], k, 0)).all()


def test_a_dispatched_fp8_row_is_a_checkpoint(coll):
    import torch
    T, hidden, group, p = 5, 256, 64, 2
    x = [dev(rng(12, r).normal(0, 2, (T, hidden)), BF16) for r in range(p)]
    dest = [torch.tensor([0, 1, 1, 0, 1], dtype=torch.int32, device="cuda") for _ in range(p)]
    rb = coll.coll_moe_fp8_row_bytes(hidden, group)
    assert rb == coll.coll_ckpt8_row_bytes(hidden, group)
    recv, loc = [u8(2 * T * rb) for _ in range(p)], [torch.zeros(T, dtype=torch.int64, device="cuda") for _ in range(p)]
    counts = torch.zeros(p * p, dtype=torch.int64, device="cuda")
    coll.coll_moe_dispatch_fp8([t for t, _ in x], dest, recv, loc, counts, 1, hidden, group)
    rows = 4                                       # rank 0 gets tokens 0 and 3 of both ranks
    back = new((rows, hidden), BF16)
    coll.coll_ckpt8_load([recv[0]], [back], hidden, group, rows=rows)
    want = np.concatenate([v[[0, 3]] for _, v in x])
    v = narrowed(token_ops.ckpt8_values(token_ops.ckpt8_rows(want, group), hidden, group), BF16)
    assert np.array_equal(host(back), v.astype(np.float64))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("p,rows,ffn,group", [(1, 1, 16, 16), (2, 3, 48, 16), (3, 17, 1408, 128), (1, 9, 512, 512), (40, 2, 64, 32), (2, 70, 4096, 256)])
def test_gated_activation(coll, p, rows, ffn, group, dtype):
    import torch
    g = rng(13, p, rows, ffn, dtype)
    x = [dev(g.normal(0, 3, (rows, 2 * ffn)), dtype) for _ in range(p)]
    dout = [dev(g.normal(0, 1e-2, (rows, ffn)), dtype) for _ in range(p)]
    rb = coll.coll_ckpt8_row_bytes(2 * ffn, group)
    ck = u8(p, rows, rb)
    out, again = [new((rows, ffn), dtype) for _ in range(p)], [new((rows, ffn), dtype) for _ in range(p)]
    dx, dx2 = [new((rows, 2 * ffn), dtype) for _ in range(p)], [new((rows, 2 * ffn), dtype) for _ in range(p)]
    T = lambda xs: [t for t, _ in xs]  # noqa: E731
    coll.coll_swiglu_ckpt8(T(x), out, list(ck), ffn, group)
    coll.coll_swiglu_backward_ckpt8(list(ck), T(dout), dx, ffn, group, out=again)
    coll.coll_swiglu_backward_ckpt8(list(ck), T(dout), dx2, ffn, group)
    torch.cuda.synchronize()
    for r in range(p):
        rows_e = token_ops.ckpt8_rows(x[r][1].astype(np.float32), group)
        assert np.array_equal(ck[r].cpu().numpy(), rows_e), f"checkpoint {r}"

        def act_tol(xe, ye):
            # the exponent's argument is off by 2 |g| U, the rest by a few U each
            return (HALF[dtype] + (2 * np.abs(xe[:, :ffn]) + 12) * U) * np.abs(ye) + TINY * (1 + np.abs(xe[:, ffn:]))
        ye = token_ops.swiglu(x[r][1])
        close(host(out[r]), ye, act_tol(x[r][1], ye), f"out {r}")
        k = token_ops.ckpt8_values(rows_e, 2 * ffn, group).astype(np.float64)
        ke = token_ops.swiglu(k)
        close(host(again[r]), ke, act_tol(k, ke), f"out again {r}")
        de = token_ops.swiglu_backward(k, dout[r][1])
        gate, up, s = k[:, :ffn], k[:, ffn:], token_ops.sigmoid(k[:, :ffn])
        c = (2 * np.abs(gate) + 14) * U
        lim = np.concatenate([np.abs(dout[r][1] * up) * s * c * (1 + 2 * np.abs(gate)), np.abs(de[:, ffn:]) * c], 1)
        close(host(dx[r]), de, HALF[dtype] * np.abs(de) + lim + TINY * 10, f"dx {r}")
        assert torch.equal(dx[r], dx2[r])


def test_gated_activation_far_gates(coll):
    """Gates from -1000 to 1000, zeros, and both infinities' neighbours."""
    gate = np.array([-1000, -200, -89, -88, -20, -1e-30, 0, 1e-30, 20, 88, 200, 1000, 3e38, -3e38, 1, -1], dtype=np.float64)
    x, xe = dev(np.concatenate([gate, np.full(16, 0.5)])[None], F32)
    out, ck = new((1, 16), F32), u8(1, coll.coll_ckpt8_row_bytes(32, 16))
    coll.coll_swiglu_ckpt8([x], [out], [ck], 16, 16)
    ye = token_ops.swiglu(xe)
    close(host(out), ye, (HALF[F32] + (2 * np.minimum(np.abs(xe[:, :16]), 200) + 12) * U) * np.abs(ye) + TINY * 1e3, "out")


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("p,rows,hidden,group", [(1, 1, 16, 16), (2, 9, 64, 32), (3, 5, 1536, 512), (8, 33, 7168, 128), (1, 3, 16384, 64), (2, 3, 20480, 512), (34, 2, 512, 16),
                                                 (2, 700, 2560, 128), (1, 5, 5120, 64), (2, 3, 4608, 512), (1, 3, 12288, 16)])
def test_layernorm_from_a_checkpoint(coll, p, rows, hidden, group, dtype, wdtype):
    import torch
    g = rng(14, p, rows, hidden, dtype, wdtype)
    x = [dev(g.normal(0.5, 2, (rows, hidden)), dtype) for _ in range(p)]
    dy = [dev(g.normal(0, 1, (rows, hidden)), dtype) for _ in range(p)]
    gamma, beta = [dev(g.normal(1, 0.3, hidden), wdtype) for _ in range(p)], [dev(g.normal(0, 0.5, hidden), wdtype) for _ in range(p)]
    T = lambda xs: [t for t, _ in xs]  # noqa: E731
    ck = u8(p, rows, coll.coll_ckpt8_row_bytes(hidden, group))
    y, y0 = [new((rows, hidden), dtype) for _ in range(p)], [new((rows, hidden), dtype) for _ in range(p)]
    mean, rstd, m0, r0 = f32(p, rows), f32(p, rows), f32(p, rows), f32(p, rows)
    coll.coll_layernorm_ckpt8(T(x), T(gamma), T(beta), y, list(mean), list(rstd), list(ck), hidden, group)
    coll.coll_layernorm(T(x), T(gamma), T(beta), y0, hidden, mean=list(m0), rstd=list(r0))
    dx, again = [new((rows, hidden), dtype) for _ in range(p)], [new((rows, hidden), dtype) for _ in range(p)]
    dg, db = new((p, hidden), wdtype), new((p, hidden), wdtype)
    ws = workspace(coll.coll_layernorm_workspace_bytes(p, rows, hidden))
    coll.coll_layernorm_backward_ckpt8(T(dy), list(ck), list(mean), list(rstd), T(gamma), dx, list(dg), list(db), ws, hidden, group,
                                       beta=T(beta), y=again)
    torch.cuda.synchronize()
    assert torch.equal(mean, m0) and torch.equal(rstd, r0) and all(torch.equal(a, b) for a, b in zip(y, y0))
    sg = sb = tg = tb = 0.0
    for r in range(p):
        rows_e = token_ops.ckpt8_rows(x[r][1].astype(np.float32), group)
        assert np.array_equal(ck[r].cpu().numpy(), rows_e), f"checkpoint {r}"
        k = token_ops.ckpt8_values(rows_e, hidden, group).astype(np.float64)
        m, s = host(mean[r]), host(rstd[r])
        dxe, dge, dbe, n = token_ops.layernorm_backward(dy[r][1], k, m, s, gamma[r][1])
        close(host(dx[r]), dxe, ln_backward_tol(dy[r][1], n, s, gamma[r][1], dxe, dtype), f"dx {r}")
        ae = n * gamma[r][1] + beta[r][1]
        close(host(again[r]), ae, HALF[dtype] * np.abs(ae) + 6 * U * (np.abs(n * gamma[r][1]) + s[:, None] * np.abs(m)[:, None] * np.abs(gamma[r][1]) + np.abs(beta[r][1])), f"y again {r}")
        sg, sb, tg, tb = sg + dge, sb + dbe, tg + np.abs(dy[r][1] * n).sum(0), tb + np.abs(dy[r][1]).sum(0)
    for r in range(p):
        close(host(dg[r]), sg, weight_tol(coll, p, rows, hidden, tg, sg, wdtype), f"dgamma {r}")
        close(host(db[r]), sb, weight_tol(coll, p, rows, hidden, tb, sb, wdtype), f"dbeta {r}")


# ----------------------------------------------------------------------------
# Vocabulary log probabilities
# ----------------------------------------------------------------------------

def shards(z, cuts, dtype, pad=0, off=0):
    """Device shards of the columns between the cuts, `pad` columns of NaN after each row."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(z, dtype=np.float32)).to(torch_dtype(dtype))
    out = []
    for a, b in zip(cuts, cuts[1:]):
        ld = b - a + pad
        buf = torch.full((off + z.shape[0] * ld,), float("nan"), dtype=t.dtype, device="cuda")
        s = buf[off:].view(z.shape[0], ld)[:, :b - a]
        s.copy_(t[:, a:b])
        out.append(s)
    return out, t.double().numpy()


def run_logprob(coll, zs, targets, t, top, entropy=True):
    import torch
    p, rows = len(zs), len(targets)
    tg = torch.tensor(targets, dtype=torch.int64, device="cuda")
    o = {"stats": f32(p, rows, 2), "logp": f32(p, rows), "entropy": f32(p, rows), "top_logp": f32(p, rows, max(top, 1)),
         "top_idx": torch.full((p, rows, max(top, 1)), -7, dtype=torch.int32, device="cuda")}
    ws = workspace(coll.coll_vocab_logprob_workspace_bytes(rows, [z.shape[1] for z in zs], top))
    coll.coll_vocab_logprob(zs, tg, list(o["stats"]), list(o["logp"]), ws, entropy=list(o["entropy"]) if entropy else None, top_k=top,
                            top_logp=list(o["top_logp"]), top_idx=list(o["top_idx"]), inv_temp=t)
    torch.cuda.synchronize()
    return o, tg


def check_logprob(o, e, targets, t, top):
    lp = np.where(np.isfinite(e["logprobs"]), e["logprobs"], 0.0)
    d = np.where(np.isfinite(e["d"]), e["d"], 0.0)
    prob = np.where(np.isfinite(e["logprobs"]), np.exp(lp), 0.0)
    ls = np.abs(np.where(np.isfinite(e["stats"][:, 1]), e["stats"][:, 1], 0.0))
    # a term's exponent is off by 3 |d| U, the term by 4 U more; chains of at most 16 chunks, 12 in a
    # chunk, 12 over lanes
    ls_tol = U * (3 * (prob * np.abs(d)).sum(1) + 4 + 64 + 4 * ls)
    h_tol = 2 * ls_tol + U * ((3 * prob * d * d).sum(1) + 72 * (prob * np.abs(d)).sum(1))
    p = o["stats"].shape[0]
    for r in range(p):
        close(host(o["stats"][r])[:, 0], e["stats"][:, 0], 0.0, "max")
        close(host(o["stats"][r])[:, 1], e["stats"][:, 1], ls_tol, "log sum")
        v = len(e["d"][0])
        at = np.array([x if 0 <= x < v else 0 for x in targets])
        dt = np.abs(d[np.arange(len(targets)), at])
        close(host(o["logp"][r]), e["logp"], ls_tol + U * (4 * dt + 2 * ls), "logp")
        close(host(o["entropy"][r]), e["entropy"], h_tol, "entropy")
        if top:
            assert np.array_equal(o["top_idx"][r].cpu().numpy(), e["top_idx"]), "alternatives"
            dd = np.where(np.isfinite(e["top_logp"]), np.abs(e["top_logp"]), 0.0) + ls[:, None]
            close(host(o["top_logp"][r]), e["top_logp"], ls_tol[:, None] + U * (4 * dd + 2 * ls[:, None]), "alternatives' logp")


def grad_and_check(coll, zs, ze, tg, targets, t, dtype, seed, place="apart"):
    """Gradient from the oracle's statistics in fp32, written to shards of the same width, column slices of one
    matrix, or in place."""
    import torch
    rows, v = ze.shape
    g = rng(20, seed)
    e = token_ops.logprob(ze, targets, t)
    st, ste = dev(e["stats"], F32)
    en, ene = dev(e["entropy"], F32)
    gl, gle = dev(g.normal(0, 1, rows), F32)
    gh, ghe = dev(g.normal(0, 0.1, rows), F32)
    widths = [z.shape[1] for z in zs]
    cuts = np.cumsum([0, *widths])
    if place == "slices":
        full = torch.full((rows, v + 3), float("nan"), dtype=zs[0].dtype, device="cuda")
        dz = [full[:, a:b] for a, b in zip(cuts, cuts[1:])]
    elif place == "in place":
        dz = zs
    else:
        dz = [torch.full((rows, w), float("nan"), dtype=zs[0].dtype, device="cuda") for w in widths]
    coll.coll_vocab_logprob_backward(zs, tg, st, gl, dz, entropy=en, dentropy=gh, inv_temp=t)
    torch.cuda.synchronize()
    want = token_ops.logprob_backward(ze, targets, t, ste, gle, ene, ghe)
    d = np.where(np.isfinite(ze) & np.isfinite(ste[:, :1]), (ze - np.where(np.isfinite(ste[:, :1]), ste[:, :1], 0.0)) * t, 0.0)
    d = np.where(np.isfinite(d), d, 0.0)
    ls = np.abs(np.where(np.isfinite(ste[:, 1:]), ste[:, 1:], 0.0))
    prob = np.where(np.isfinite(ze) & np.isfinite(ste[:, :1]), np.exp(d - np.where(np.isfinite(ste[:, 1:]), ste[:, 1:], 0.0)), 0.0)
    rel = (4 * np.abs(d) + 4 * ls + 10) * U
    size = np.abs(gle)[:, None] + np.abs(ghe)[:, None] * (np.abs(d) + ls + np.abs(ene)[:, None] + 1)
    lim = HALF[dtype] * np.abs(want) + t * (prob * size * rel + np.abs(gle)[:, None] * 4 * U * (prob + (np.arange(v) == np.array(targets)[:, None]))) + TINY * 10
    got = np.concatenate([host(x) for x in dz], 1)
    close(got, want, lim, "dlogits")
    if place == "slices":
        assert torch.isnan(full[:, v:].float()).all()


LP_SHAPES = [
    # rows, cuts of the vocabulary, dtype, pad, off, temperature's inverse, top
    (1, [0, 1], F32, 0, 0, 1.0, 1), (3, [0, 5], BF16, 0, 1, 1.0, 5), (2, [0, 3, 8], F32, 1, 1, 0.5, 12), (5, [0, 0, 9, 9, 30], BF16, 0, 0, 2.0, 3),
    (4, [0, 1000], BF16, 3, 5, 1.0, 8), (7, [0, 129, 257, 600], F32, 0, 2, 1.3, 32), (1, [0, 2048], BF16, 0, 0, 1.0, 20), (2, [0, 2049, 4100], BF16, 1, 0, 1.0, 20),
    (3, [0, 16384, 32768], F32, 0, 0, 0.8, 8), (2, [0, 50257], BF16, 0, 3, 1.0, 0), (1, [0, 40000, 131072], BF16, 0, 0, 1.0, 32), (300, [0, 700, 1401], BF16, 0, 0, 1.0, 4),
    (9000, [0, 37], F32, 0, 0, 1.0, 2), (2, list(range(0, 65 * 31, 31)), BF16, 0, 1, 1.0, 8), (1, [0, 200000], F32, 0, 1, 1.0, 16),
]


@pytest.mark.parametrize("rows,cuts,dtype,pad,off,t,top", LP_SHAPES)
def test_logprob_and_gradient(coll, rows, cuts, dtype, pad, off, t, top):
    g = rng(15, rows, len(cuts), cuts[-1], dtype, top)
    v = cuts[-1]
    z = g.normal(0, 3, (rows, v))
    targets = [int(x) for x in g.integers(0, v, rows)]
    if rows > 2:
        targets[1], targets[-1] = -100, v                     # padding, and one past the end
    zs, ze = shards(z, cuts, dtype, pad, off)
    t = float(np.float32(t))
    o, tg = run_logprob(coll, zs, targets, t, top)
    check_logprob(o, token_ops.logprob(ze, targets, t, top), targets, t, top)
    for place in ("apart", "slices", "in place"):
        grad_and_check(coll, zs, ze, tg, targets, t, dtype, v, place)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("v,p", [(40, 1), (3000, 3), (9000, 1), (70000, 2)])
def test_logprob_masked_rows_ties_and_edge_values(coll, dtype, v, p):
    g = rng(16, v, p, dtype)
    z = g.normal(0, 3, (12, v))
    low = {F32: np.finfo(np.float32).min, BF16: -3.3895313892515355e38}[dtype]
    z[0] = -np.inf                                            # nothing is allowed
    z[1] = -np.inf
    z[1, v - 1] = -5.0                                        # one entry is
    z[2] = low                                                # all at the type's lowest value: alike
    z[3] = low
    z[3, [2, v - 2]] = [1.0, 2.0]                             # masked by the lowest value
    z[4, g.permutation(v)[:v * 9 // 10]] = -np.inf
    z[5] = 4.25                                               # every entry ties
    z[6] = np.round(z[6])                                     # many ties
    z[7, v // 2] = np.nan
    z[8, 1] = np.inf
    z[9] = np.sort(z[9])                                      # ascending: each entry beats those before
    z[10] = np.where(np.arange(v) % 2, -0.0, 0.0)             # both zeros tie
    z[11] = 1e4 + np.arange(v) % 7                            # large logits
    targets = [0, v - 1, v // 3, 2, 5, v - 1, 1, 3, 0, v - 1, 4, 6]
    cuts = [v * r // p for r in range(p + 1)]
    zs, ze = shards(z, cuts, dtype, 0, 1)
    for t, top in ((1.0, 20), (0.5, 32)):
        o, tg = run_logprob(coll, zs, targets, t, top)
        check_logprob(o, token_ops.logprob(ze, targets, t, top), targets, t, top)
        keep = [0, 1, 2, 3, 4, 5, 6, 9, 10, 11]
        grad_and_check(coll, [x[keep] for x in zs], ze[keep], tg[keep], [targets[i] for i in keep], t, dtype, v)


def test_logprob_gradient_without_entropy_and_of_poisoned_rows(coll):
    import torch
    z = rng(17).normal(0, 1, (3, 50))
    z[1, 7] = np.nan
    zs, ze = shards(z, [0, 20, 50], F32)
    targets = [3, 4, 49]
    o, tg = run_logprob(coll, zs, targets, 1.0, 0)
    gl, gle = dev(np.array([1.0, 2.0, -1.0]), F32)
    dz = [torch.zeros_like(x) for x in zs]
    coll.coll_vocab_logprob_backward(zs, tg, o["stats"][0], gl, dz)
    got = np.concatenate([host(x) for x in dz], 1)
    assert np.isnan(got[1]).all()
    e = token_ops.logprob(ze, targets, 1.0)
    for i in (0, 2):
        want = token_ops.logprob_backward(ze[i:i + 1], targets[i:i + 1], 1.0, host(o["stats"][0])[i:i + 1], gle[i:i + 1], e["entropy"][i:i + 1], [0.0])
        close(got[i:i + 1], want, 100 * U * (np.abs(want) + np.exp(e["logprobs"][i])), "dlogits")


def test_logprob_gradient_by_differences(coll):
    """Against central differences of the kernel's own forward pass (fp32, two shards)."""
    g = rng(18)
    v, rows, t = 45, 3, 0.75
    z = g.normal(0, 2, (rows, v)).astype(np.float32)
    targets = [2, 44, -1]
    gl, gh = g.normal(0, 1, rows).astype(np.float32), g.normal(0, 1, rows).astype(np.float32)

    def loss(z):
        o, _ = run_logprob(coll, shards(z, [0, 21, v], F32)[0], targets, t, 0)
        return (host(o["logp"][1]) * gl + host(o["entropy"][0]) * gh).sum()
    zs, _ = shards(z, [0, 21, v], F32)
    o, tg = run_logprob(coll, zs, targets, t, 0)
    dz = [x.clone() for x in zs]
    coll.coll_vocab_logprob_backward(zs, tg, o["stats"][0], dev(gl, F32)[0], dz, entropy=o["entropy"][0], dentropy=dev(gh, F32)[0], inv_temp=t)
    got = np.concatenate([host(x) for x in dz], 1)
    # h^2 / 6 times third derivatives (below 4 for these sizes), and 6 results of up to 8, off by 100 U each
    h = 2.0 ** -6
    lim = h * h * 4 + 6 * 8 * 100 * U / (2 * h)
    for i, j in [(0, 2), (0, 30), (1, 44), (1, 0), (2, 10), (2, 21)]:
        a, b = z.copy(), z.copy()
        a[i, j] += np.float32(h)
        b[i, j] -= np.float32(h)
        step = float(a[i, j]) - float(b[i, j])
        assert abs((loss(a) - loss(b)) / step - got[i, j]) < lim, (i, j)


# ----------------------------------------------------------------------------
# Streams, graphs, repeats, large offsets
# ----------------------------------------------------------------------------

def _step(coll, g, stream=None, defer=False):
    """All operators once over two ranks; returns the calls and the outputs."""
    p, rows, hidden, ffn, v = 2, 37, 640, 256, 1111
    x = [dev(g.normal(0, 1, (rows, hidden)), BF16)[0] for _ in range(p)]
    w = [dev(g.normal(1, 0.2, hidden), F32)[0] for _ in range(p)]
    b = [dev(g.normal(0, 0.2, hidden), F32)[0] for _ in range(p)]
    y, dx = [new((rows, hidden), BF16) for _ in range(p)], [new((rows, hidden), BF16) for _ in range(p)]
    mean, rstd = f32(p, rows), f32(p, rows)
    ck = u8(p, rows, coll.coll_ckpt8_row_bytes(hidden, 128))
    dg, db = f32(p, hidden), f32(p, hidden)
    ws = workspace(coll.coll_layernorm_workspace_bytes(p, rows, hidden))
    gu = [dev(g.normal(0, 1, (rows, 2 * ffn)), BF16)[0] for _ in range(p)]
    out, dgu = [new((rows, ffn), BF16) for _ in range(p)], [new((rows, 2 * ffn), BF16) for _ in range(p)]
    ck2 = u8(p, rows, coll.coll_ckpt8_row_bytes(2 * ffn, 64))
    zs, _ = shards(g.normal(0, 3, (rows, v)), [0, 500, v], F32)
    import torch
    tg = torch.from_numpy(g.integers(0, v, rows)).cuda()
    st, lp, en, tl = f32(p, rows, 2), f32(p, rows), f32(p, rows), f32(p, rows, 5)
    ti = torch.zeros(p, rows, 5, dtype=torch.int32, device="cuda")
    ws2 = workspace(coll.coll_vocab_logprob_workspace_bytes(rows, [500, v - 500], 5))
    dz = [torch.zeros_like(z) for z in zs]
    k = dict(stream=stream, defer=defer)
    calls = [
        lambda: coll.coll_layernorm_ckpt8(x, w, b, y, list(mean), list(rstd), list(ck), hidden, 128, **k),
        lambda: coll.coll_layernorm_backward_ckpt8(y, list(ck), list(mean), list(rstd), w, dx, list(dg), list(db), ws, hidden, 128, **k),
        lambda: coll.coll_swiglu_ckpt8(gu, out, list(ck2), ffn, 64, **k),
        lambda: coll.coll_swiglu_backward_ckpt8(list(ck2), out, dgu, ffn, 64, **k),
        lambda: coll.coll_vocab_logprob(zs, tg, list(st), list(lp), ws2, entropy=list(en), top_k=5, top_logp=list(tl), top_idx=list(ti), **k),
        lambda: coll.coll_vocab_logprob_backward(zs, tg, st[1], lp[0], dz, entropy=en[1], dentropy=lp[1], **k),
    ]
    return calls, [*y, *dx, mean, rstd, ck, dg, db, *out, *dgu, ck2, st, lp, en, tl, ti, *dz]


def test_repeats_streams_and_grid_limits_give_the_same_bits(coll):
    import torch
    calls, outs = _step(coll, rng(30))
    for c in calls:
        c()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for limit in (0, 1, 7):
        coll.coll_set_grid_limit(limit)
        try:
            calls2, outs2 = _step(coll, rng(30), stream=side)
            side.wait_stream(torch.cuda.current_stream())
            for c in calls2:
                c()
            side.synchronize()
        finally:
            coll.coll_set_grid_limit(0)
        for a, b in zip(first, outs2):
            assert torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8))


def test_graph_replays_match_eager_calls(coll):
    import torch
    calls, outs = _step(coll, rng(31))
    for c in calls:
        c()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls:
            c()
    for i in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8)), f"replay {i}"
        calls[i % len(calls)]()                               # eager work between the replays
        torch.cuda.synchronize()


def test_deferred_calls(coll):
    import torch
    calls, outs = _step(coll, rng(32), defer=True)
    prepared = [c() for c in calls]
    for _ in range(2):
        for f in prepared:
            f()
    torch.cuda.synchronize()
    again, outs2 = _step(coll, rng(32))
    for c in again:
        c()
    torch.cuda.synchronize()
    for a, b in zip(outs, outs2):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_rows_past_2_31_elements(coll):
    """Logits, layer-norm rows and checkpoints whose last rows lie past 2^31 elements."""
    import torch
    g = rng(33)
    v, pick = 131072, [0, 16383, 16384, 16385, 17000]
    rows = pick[-1] + 1
    z = torch.zeros(rows, v, dtype=torch.bfloat16, device="cuda")
    small, ze = dev(g.normal(0, 3, (len(pick), v)), BF16)
    z[pick] = small
    targets = [int(x) for x in g.integers(0, v, rows)]
    o, tg = run_logprob(coll, [z], targets, 1.0, 4)
    t5 = [targets[i] for i in pick]
    e = token_ops.logprob(ze, t5, 1.0, 4)
    check_logprob({k: x[:, pick] for k, x in o.items()}, e, t5, 1.0, 4)
    coll.coll_vocab_logprob_backward([z], tg, o["stats"][0], torch.ones(rows, device="cuda"), [z])   # in place
    want = token_ops.logprob_backward(ze, t5, 1.0, host(o["stats"][0])[pick], np.ones(5), e["entropy"], np.zeros(5))
    close(host(z[pick]), want, HALF[BF16] * np.abs(want) + 200 * U * np.abs(want) + 8 * U * (np.arange(v) == np.array(t5)[:, None]) + TINY, "dlogits")
    del z, o
    hidden, rows = 7168, 300001
    pick = [0, 149796, 149797, 300000]
    x = torch.zeros(rows, hidden, dtype=torch.bfloat16, device="cuda")
    small, xe = dev(g.normal(0, 1, (len(pick), hidden)), BF16)
    x[pick] = small
    ck = torch.zeros(rows, coll.coll_ckpt8_row_bytes(hidden, 128), dtype=torch.uint8, device="cuda")
    mean, rstd = f32(rows), f32(rows)
    y = torch.empty_like(x)
    coll.coll_layernorm_ckpt8([x], None, None, [y], [mean], [rstd], [ck], hidden, 128)
    torch.cuda.synchronize()
    ye, me, re = token_ops.layernorm(xe, np.ones(hidden), np.zeros(hidden), 1e-5)
    close(host(y[pick]), ye, ln_forward_tol(xe, np.ones(hidden), np.zeros(hidden), me, re, ye, BF16), "y")
    rows_e = token_ops.ckpt8_rows(xe.astype(np.float32), 128)
    assert np.array_equal(ck[pick].cpu().numpy(), rows_e)
    ck.zero_()
    coll.coll_ckpt8_save([x], [ck], hidden, 128)
    assert np.array_equal(ck[pick].cpu().numpy(), rows_e)
    dx, dg = torch.empty_like(x), f32(hidden)
    ws = workspace(coll.coll_layernorm_workspace_bytes(1, rows, hidden))
    coll.coll_layernorm_backward([y], [x], [mean], [rstd], None, [dx], [dg], None, ws, hidden)
    yb = host(y[pick])
    dxe, dge, _, n = token_ops.layernorm_backward(yb, xe, host(mean)[pick], host(rstd)[pick], np.ones(hidden))
    close(host(dx[pick]), dxe, ln_backward_tol(yb, n, host(rstd)[pick], np.ones(hidden), dxe, BF16), "dx")
    close(host(dg), dge, weight_tol(coll, 1, rows, hidden, np.abs(yb * n).sum(0), dge, F32), "dgamma")


@pytest.mark.parametrize("p,rows", [(64, (1 << 20) + 3), (1, (1 << 26) + 5)])
def test_logprob_of_more_rows_than_a_launch_holds(coll, p, rows):
    """64 entries in 64 shards, and 2 in one: a launch ends 4 waves short of 2^26, so the last rows take another one,
    the second time also in the join."""
    import torch
    v = max(p, 2)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(34)
    z = torch.randn(rows, v, generator=gen, device="cuda").mul_(3).to(torch.bfloat16)
    zs = [z[:, v * r // p:v * (r + 1) // p].contiguous() for r in range(p)]
    tg = torch.randint(0, v, (rows,), generator=gen, device="cuda")
    st, lp = f32(p, rows, 2), f32(p, rows)
    ws = workspace(coll.coll_vocab_logprob_workspace_bytes(rows, [x.shape[1] for x in zs]))
    coll.coll_vocab_logprob(zs, tg, list(st), list(lp), ws)
    gl = torch.randn(rows, generator=gen, device="cuda")
    dz = [torch.full_like(x, float("nan")) for x in zs]
    coll.coll_vocab_logprob_backward(zs, tg, st[0], gl, dz)
    torch.cuda.synchronize()
    for a in range(0, rows, 1 << 24):
        n = slice(a, min(rows, a + (1 << 24)))
        d = z[n].double()
        m = d.amax(1)
        d -= m[:, None]
        ls = d.exp().sum(1).log()
        want = d.gather(1, tg[n, None])[:, 0] - ls
        # differences of up to 40 and sums of up to 64: as check_logprob, no term above 300 U
        for r in {0, p - 1}:
            assert torch.equal(st[r][n, 0].double(), m)
            assert float((st[r][n, 1].double() - ls).abs().max()) <= 300 * U
            assert float((lp[r][n].double() - want).abs().max()) <= 300 * U
        prob = (d - ls[:, None]).exp_()
        ge = prob.neg_().scatter_add_(1, tg[n, None], torch.ones_like(want)[:, None]).mul_(gl[n, None].double())
        got = torch.cat([x[n] for x in dz], 1).double()
        assert bool(((got - ge).abs() <= HALF[BF16] * ge.abs() + 300 * U * gl[n, None].double().abs()).all())


def test_layernorm_of_more_rows_than_a_launch_holds(coll):
    """Rows of 16 elements, 32 to a workgroup: a launch ends 32 rows short of 2^29, so the last rows take another one."""
    import torch
    g = rng(35)
    hidden, rows, cut = 16, (1 << 29) + 5, (1 << 29) - 32
    pick = [0, 1, 12345678, cut - 1, cut, cut + 1, cut + 31, rows - 2, rows - 1]
    x = torch.zeros(rows, hidden, dtype=torch.bfloat16, device="cuda")
    small, xe = dev(g.normal(0.5, 2, (len(pick), hidden)), BF16)
    x[pick] = small
    beta, be = dev(g.normal(0, 1, hidden), BF16)
    gamma, ge = dev(g.normal(1, 0.3, hidden), BF16)
    y = torch.full_like(x, float("nan"))
    mean, rstd = f32(rows), f32(rows)
    ck = u8(rows, coll.coll_ckpt8_row_bytes(hidden, 16))
    coll.coll_layernorm_ckpt8([x], [gamma], [beta], [y], [mean], [rstd], [ck], hidden, 16)
    torch.cuda.synchronize()
    ye, me, re = token_ops.layernorm(xe, ge, be, 1e-5)
    close(host(y[pick]), ye, ln_forward_tol(xe, ge, be, me, re, ye, BF16), "y")
    close(host(mean[pick]), me, (chain(hidden) + 4) * U * np.abs(xe).mean(1), "mean")
    close(host(rstd[pick]), re, re * ((chain(hidden) + 8) * U + re ** 2 * ((chain(hidden) + 4) * U * np.abs(xe).mean(1)) ** 2), "rstd")
    assert np.array_equal(ck[pick].cpu().numpy(), token_ops.ckpt8_rows(xe.astype(np.float32), 16))
    y[pick] = beta                                            # all others: rows of zeros
    mean[pick] = 0.0
    zeros = torch.from_numpy(token_ops.ckpt8_rows(np.zeros((1, hidden), dtype=np.float32), 16)).cuda()
    ck[pick] = zeros
    for a in range(0, rows, 1 << 26):
        assert bool((y[a:a + (1 << 26)] == beta).all()) and bool((ck[a:a + (1 << 26)] == zeros).all()), a
    assert bool((mean == 0).all())


def test_layernorm_gradient_of_more_columns_than_a_launch_joins(coll):
    """A row of 2^27 + 16 columns, whose weight gradients a join of 2^22 workgroups of 64 sums cannot hold."""
    import torch
    hidden = (1 << 27) + 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(36)
    x, dy = [torch.randn(1, hidden, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
    mean, rstd = torch.tensor([0.25], device="cuda"), torch.tensor([0.875], device="cuda")
    dx, dg, db = torch.full_like(x, float("nan")), f32(hidden), f32(hidden)
    ws = workspace(coll.coll_layernorm_workspace_bytes(1, 1, hidden))
    coll.coll_layernorm_backward([dy], [x], [mean], [rstd], None, [dx], [dg], [db], ws, hidden, wdtype=F32)
    torch.cuda.synchronize()
    assert torch.equal(db, dy[0].float())                     # one row: nothing to add
    n = (x[0].double() - 0.25) * 0.875
    want = dy[0].double() * n
    assert bool(((dg.double() - want).abs() <= 3 * U * want.abs() + TINY).all())
    d = dy[0].double()
    dxe = 0.875 * (d - d.mean() - n * want.mean())
    # the two means: sums of 2^27 terms whose magnitudes are below 1 on average, 2^17 of them one after another in a lane
    assert bool(((dx[0].double() - dxe).abs() <= HALF[BF16] * dxe.abs() + (chain(hidden) + 8) * U * (d.abs() + 1 + n.abs())).all())


def test_logprob_in_a_workspace_for_more_rows(coll):
    """4095 rows of 6200 entries, cut into three pieces each, in the workspace of 4096, which need two each."""
    import torch
    g = rng(37)
    rows, v, top = 4095, 6200, 4
    zs, ze = shards(g.normal(0, 3, (rows, v)), [0, v], BF16)
    targets = [int(x) for x in g.integers(0, v, rows)]
    tg = torch.tensor(targets, dtype=torch.int64, device="cuda")
    o = {"stats": f32(1, rows, 2), "logp": f32(1, rows), "entropy": f32(1, rows), "top_logp": f32(1, rows, top),
         "top_idx": torch.full((1, rows, top), -7, dtype=torch.int32, device="cuda")}
    ws = workspace(coll.coll_vocab_logprob_workspace_bytes(rows + 1, [v], top))
    coll.coll_vocab_logprob(zs, tg, list(o["stats"]), list(o["logp"]), ws, entropy=list(o["entropy"]), top_k=top,
                            top_logp=list(o["top_logp"]), top_idx=list(o["top_idx"]))
    torch.cuda.synchronize()
    check_logprob(o, token_ops.logprob(ze, targets, 1.0, top), targets, 1.0, top)
