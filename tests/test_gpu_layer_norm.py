"""Layer norm forward and backward on the GPU against the 64-bit formulas."""
import pytest
import torch

import block_util as bu
from gpu_util import moe_mod

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 1), (5, 7), (2, 31), (4, 33), (9, 128), (7, 1000), (3, 1024), (2, 1537), (5, 4096), (3, 7168),
          (2, 8192), (1, 16384), (2, 16392), (2, 40000), (700, 264), (401, 2049)]
EPS = 1e-5


def inputs(rows, H, dtype, pdtype, seed=0):
    x = (bu.randn(rows, H, seed=seed) * torch.exp(0.5 * bu.randn(H, seed=seed + 1)) + 0.3).to(dtype)
    w = (1.0 + 0.3 * bu.randn(H, seed=seed + 2)).to(pdtype)
    b = bu.randn(H, seed=seed + 3, scale=0.2).to(pdtype)
    return x, w, b


def forward(moe, x, w, b, residual=None, eps=EPS, want_sum=True):
    rows, H = x.shape
    d = lambda t: None if t is None else t.cuda()
    y = torch.full((rows, H), float("nan"), dtype=x.dtype, device="cuda")
    s = torch.full_like(y, float("nan")) if residual is not None and want_sum else None
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    moe.moe_layer_norm(d(x), d(w), d(b), eps, y, residual=d(residual), sum_out=s, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    return y, s, mean, rstd


def check_forward(got, h, w, b, eps, dtype):
    y, _, mean, rstd = got
    ry, rm, rr, _ = bu.norm_forward(h, w, b, eps)
    ty, tm, tr = bu.norm_forward_tol(h, w, b, eps, dtype)
    bu.assert_within(y, ry, ty, "y")
    bu.assert_within(mean, rm, tm, "mean")
    bu.assert_within(rstd, rr, tr, "rstd")


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("rows,H", SHAPES)
def test_forward(rows, H, dtype):
    moe = moe_mod()
    for pdtype in {dtype, torch.float32}:
        x, w, b = inputs(rows, H, dtype, pdtype)
        check_forward(forward(moe, x, w, b), x, w, b, EPS, dtype)


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("rows,H", [(3, 33), (4, 1024), (3, 7168), (2, 20000)])
def test_forward_residual(rows, H, dtype):
    """The norm is that of the stored sum, with and without the sum as an output, and the sum may replace an input."""
    moe = moe_mod()
    x, w, b = inputs(rows, H, dtype, dtype)
    res = bu.randn(rows, H, seed=9, scale=2.0, dtype=dtype)
    h = (x.float() + res.float()).to(dtype)
    a = forward(moe, x, w, b, res)
    assert torch.equal(a[1].cpu(), h)
    check_forward(a, h, w, b, EPS, dtype)
    assert torch.equal(forward(moe, x, w, b, res, want_sum=False)[0], a[0])
    for which in (0, 1):
        xd, rd, y = x.cuda(), res.cuda(), torch.empty_like(a[0])
        into = (xd, rd)[which]
        moe.moe_layer_norm(xd, w.cuda(), b.cuda(), EPS, y, residual=rd, sum_out=into)
        assert torch.equal(y, a[0]) and torch.equal(into.cpu(), h)


@pytest.mark.parametrize("dtype", bu.DTYPES)
def test_forward_without_parameters(dtype):
    moe = moe_mod()
    x, w, b = inputs(6, 513, dtype, dtype)
    for ww, bb in ((None, None), (w, None), (None, b)):
        check_forward(forward(moe, x, ww, bb), x, ww, bb, EPS, dtype)


def test_constant_rows_and_far_means():
    """Zero variance gives the bias; a mean far from zero loses no more than the inputs' own spacing."""
    moe = moe_mod()
    for H in (5, 256, 7168):
        x = torch.full((4, H), 3.0)
        _, w, b = inputs(4, H, torch.float32, torch.float32)
        y, _, mean, rstd = forward(moe, x, w, b)
        assert torch.equal(y.cpu(), b.expand(4, H)) and bool((mean == 3.0).all())
        assert bool((rstd.cpu() - EPS ** -0.5).abs().max() < EPS ** -0.5 * 4 * bu.U * 4)
        x = 1000.0 + bu.randn(4, H, seed=4)
        check_forward(forward(moe, x, w, b), x, w, b, EPS, torch.float32)


@pytest.mark.parametrize("H", [100, 2048])
def test_nonfinite_rows_stay_alone(H):
    moe = moe_mod()
    x, w, b = inputs(5, H, torch.bfloat16, torch.float32)
    ref = forward(moe, x, w, b)[0]
    bad = x.clone()
    bad[1, 3], bad[3, 7] = float("nan"), float("inf")
    y = forward(moe, bad, w, b)[0]
    for r in (0, 2, 4):
        assert torch.equal(y[r], ref[r])
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[3]).any())


def strided(t, pad, shift):
    """A copy of t whose rows lie apart and start `shift` elements into a buffer."""
    buf = torch.full((t.shape[0], t.shape[1] + pad + shift), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return buf, v


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("H,pad,shift", [(1024, 64, 0), (1024, 8, 8), (1024, 1, 0), (1024, 7, 1), (515, 5, 3)])
def test_strides_and_alignment(dtype, H, pad, shift):
    moe = moe_mod()
    rows = 37
    x, w, b = inputs(rows, H, dtype, dtype)
    res = bu.randn(rows, H, seed=5, dtype=dtype)
    gy, gs = bu.randn(rows, H, seed=6, dtype=dtype), bu.randn(rows, H, seed=7, dtype=dtype)
    y, s, mean, rstd = forward(moe, x, w, b, res)
    xb, xv = strided(x, pad, shift)
    rb, rv = strided(res, pad, shift)
    ob, ov = strided(torch.zeros(rows, H, dtype=dtype), pad, shift)
    sb, sv = strided(torch.zeros(rows, H, dtype=dtype), pad, shift)
    moe.moe_layer_norm(xv, w.cuda(), b.cuda(), EPS, ov, residual=rv, sum_out=sv)
    h = (x.float() + res.float()).to(dtype)
    ty, _, _ = bu.norm_forward_tol(h, w, b, EPS, dtype)
    bu.assert_within(ov, bu.norm_forward(h, w, b, EPS)[0], ty)
    assert torch.equal(sv.cpu(), h)
    for buf in (ob, sb):  # nothing outside the view is written
        assert bool(torch.isnan(buf[:, :shift]).all()) and bool(torch.isnan(buf[:, shift + H:]).all())
    gb_, gv = strided(gy, pad, shift)
    _, gsv = strided(gs, pad, shift)
    xob, xo = strided(torch.zeros(rows, H, dtype=dtype), pad, shift)
    ws = torch.empty(moe.moe_layer_norm_workspace_size(rows, H), dtype=torch.uint8, device="cuda")
    gw, gb = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_layer_norm_backward(gv, sv, w.cuda(), mean, rstd, xo, gw, gb, ws, grad_sum=gsv)
    refs = bu.norm_backward(gy, h, w, mean.cpu(), rstd.cpu(), gs)
    tols = bu.norm_backward_tol(gy, h, w, mean.cpu(), rstd.cpu(), gs, dtype)
    for got, ref, tol in zip((xo, gw, gb), refs, tols):
        bu.assert_within(got, ref, tol)
    assert bool(torch.isnan(xob[:, :shift]).all()) and bool(torch.isnan(xob[:, shift + H:]).all())


def backward(moe, gy, h, w, mean, rstd, gsum=None):
    rows, H = h.shape
    d = lambda t: None if t is None else t.cuda()
    gx = torch.full((rows, H), float("nan"), dtype=h.dtype, device="cuda")
    gw, gb = (torch.full((H,), float("nan"), device="cuda") for _ in range(2))
    ws = torch.full((moe.moe_layer_norm_workspace_size(rows, H),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_layer_norm_backward(d(gy), d(h), d(w), d(mean), d(rstd), gx, gw, gb, ws, grad_sum=d(gsum))
    torch.cuda.synchronize()
    return gx, gw, gb


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("rows,H", SHAPES + [(1531, 513), (2000, 1024), (5000, 96), (330, 7168)])
def test_backward(rows, H, dtype):
    moe = moe_mod()
    for pdtype in {dtype, torch.float32}:
        x, w, _ = inputs(rows, H, dtype, pdtype)
        _, mean, rstd, _ = bu.norm_forward(x, None, None, EPS)
        mean, rstd = mean.float(), rstd.float()
        gy, gs = bu.randn(rows, H, seed=11, dtype=dtype), bu.randn(rows, H, seed=12, dtype=dtype)
        for gsum, ww in ((None, w), (gs, w), (gs, None)):
            got = backward(moe, gy, x, ww, mean, rstd, gsum)
            refs = bu.norm_backward(gy, x, ww, mean, rstd, gsum)
            tols = bu.norm_backward_tol(gy, x, ww, mean, rstd, gsum, dtype)
            for name, g, r, t in zip(("gx", "gw", "gb"), got, refs, tols):
                bu.assert_within(g, r, t, name)


@pytest.mark.parametrize("rows,H", [(40, 96), (300, 2048)])
def test_backward_outputs_in_place_and_partial(rows, H):
    """grad_x may replace grad_y or grad_sum; either parameter gradient may be left out; results repeat bit for bit."""
    moe = moe_mod()
    x, w, _ = inputs(rows, H, torch.bfloat16, torch.float32)
    _, mean, rstd, _ = bu.norm_forward(x, None, None, EPS)
    mean, rstd = mean.float(), rstd.float()
    gy, gs = bu.randn(rows, H, seed=1, dtype=x.dtype), bu.randn(rows, H, seed=2, dtype=x.dtype)
    gx, gw, gb = backward(moe, gy, x, w, mean, rstd, gs)
    again = backward(moe, gy, x, w, mean, rstd, gs)
    assert all(torch.equal(a, b) for a, b in zip((gx, gw, gb), again))
    ws = torch.empty(moe.moe_layer_norm_workspace_size(rows, H), dtype=torch.uint8, device="cuda")
    xd, wd, md, rd = x.cuda(), w.cuda(), mean.cuda(), rstd.cuda()
    for which in (0, 1):
        a = [gy.cuda(), gs.cuda()]
        gw2, gb2 = torch.empty_like(gw), torch.empty_like(gb)
        moe.moe_layer_norm_backward(a[0], xd, wd, md, rd, a[which], gw2, gb2, ws, grad_sum=a[1])
        assert torch.equal(a[which], gx) and torch.equal(gw2, gw) and torch.equal(gb2, gb)
    only = torch.empty_like(gw)
    out = torch.empty_like(gx)
    moe.moe_layer_norm_backward(gy.cuda(), xd, wd, md, rd, out, only, None, ws, grad_sum=gs.cuda())
    assert torch.equal(only, gw) and torch.equal(out, gx)
    moe.moe_layer_norm_backward(gy.cuda(), xd, wd, md, rd, out, None, only, ws, grad_sum=gs.cuda())
    assert torch.equal(only, gb) and torch.equal(out, gx)
    moe.moe_layer_norm_backward(gy.cuda(), xd, wd, md, rd, out, grad_sum=gs.cuda())
    assert torch.equal(out, gx)


def test_no_rows():
    moe = moe_mod()
    e = torch.empty(0, 64, device="cuda")
    s = torch.empty(0, device="cuda")
    moe.moe_layer_norm(e, None, None, EPS, torch.empty_like(e), mean=s, rstd=s)
    gx, gw, gb = backward(moe, e, e, torch.ones(64), s, s)
    assert bool((gw == 0).all()) and bool((gb == 0).all())


@pytest.mark.parametrize("H", [48, 1024])
def test_gradient_against_differences(H):
    """The kernel's gradients against central differences of the 64-bit forward pass along random directions."""
    moe = moe_mod()
    rows = 6
    x, w, b = inputs(rows, H, torch.float32, torch.float32)
    gy = bu.randn(rows, H, seed=21)
    _, mean, rstd, _ = bu.norm_forward(x, w, b, EPS)
    gx, gw, gb = backward(moe, gy, x, w, mean.float(), rstd.float())
    loss = lambda xx, ww, bb: float((bu.norm_forward(xx, ww, bb, EPS)[0] * gy.double()).sum())
    tols = bu.norm_backward_tol(gy, x, w, mean.float(), rstd.float(), None, torch.float32)
    step = 1e-4
    xd, wd, bd = x.double(), w.double(), b.double()
    for i, (got, tol) in enumerate(zip((gx, gw, gb), tols)):
        v = bu.randn(*got.shape, seed=30 + i).double()
        d = [torch.zeros_like(t) for t in (xd, wd, bd)]
        d[i] = v * step
        num = (loss(xd + d[0], wd + d[1], bd + d[2]) - loss(xd - d[0], wd - d[1], bd - d[2])) / (2 * step)
        # roundings of the gradient and of the statistics, and the difference's own error (step^2 and 1e-16 / step)
        slack = float((tol * v.abs()).sum()) + 64 * bu.U * float((f64abs(got) * v.abs()).sum())
        slack += step ** 2 * 10 * float((f64abs(got) * v.abs()).sum()) + 1e-9 * rows * H
        assert abs(float((bu.f64(got) * v).sum()) - num) <= slack


def f64abs(t):
    return bu.f64(t).abs()


def test_refusals():
    moe = moe_mod()
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    w, b = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    y = torch.empty_like(x)
    with pytest.raises(ValueError):  # another type
        moe.moe_layer_norm(x, w, b, EPS, y.float())
    with pytest.raises(ValueError):  # half parameters of another kind than the rows
        moe.moe_layer_norm(x, w.half(), b.half(), EPS, y)
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x, w, b.bfloat16(), EPS, y)
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x, w[:32], None, EPS, y)
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x, w, b, EPS, y[:2])
    with pytest.raises(ValueError):  # columns apart
        moe.moe_layer_norm(x.t(), torch.ones(4, device="cuda"), None, EPS, torch.empty_like(x.t()))
    with pytest.raises(ValueError):
        moe.moe_layer_norm(x.cpu(), w, b, EPS, y)
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        with pytest.raises(moe.MoeError):
            moe.moe_layer_norm(x, w, b, bad["eps"], y)
    with pytest.raises(moe.MoeError):  # a sum without a residual
        moe.moe_layer_norm(x, w, b, EPS, y, sum_out=torch.empty_like(x))
    with pytest.raises(moe.MoeError):  # y over an input
        moe.moe_layer_norm(x, w, b, EPS, x)
    buf = torch.zeros(5, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError):  # the sum one row off its input
        moe.moe_layer_norm(buf[:4], w, b, EPS, y, residual=x, sum_out=buf[1:])
    s = torch.ones(4, device="cuda")
    gw = torch.empty(64, device="cuda")
    ws = torch.empty(moe.moe_layer_norm_workspace_size(4, 64), dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_layer_norm_backward(x, y, w, s, s, torch.empty_like(x), gw, None, ws[:16])
    assert ei.value.status == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(moe.MoeError):
        moe.moe_layer_norm_backward(x, y, w, s, s, torch.empty_like(x), gw, None, None)
    with pytest.raises(moe.MoeError):
        moe.moe_layer_norm_backward(x, y, w, s, s, y)
    with pytest.raises(moe.MoeError):
        moe.moe_layer_norm_backward(x, y, w, None, s, torch.empty_like(x))


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("rows,H", [(3, 8193), (200, 16384), (170, 9001), (90, 16383), (100, 12000), (11, 4100)])
def test_backward_of_rows_wider_than_a_block(rows, H, dtype):
    """Rows that clusters share, aligned and not, more of them than clusters and fewer."""
    test_backward(rows, H, dtype)


@pytest.mark.parametrize("rows,H,dtype", [(200000, 8, torch.bfloat16), (100000, 13, torch.float16),
                                          (170000, 264, torch.bfloat16), (80000, 260, torch.float32)])
def test_backward_of_many_rows(rows, H, dtype):
    """More rows a team than the statistics it loads at once, several times over."""
    moe = moe_mod()
    x, w, _ = inputs(rows, H, dtype, torch.float32)
    _, mean, rstd, _ = bu.norm_forward(x, None, None, EPS)
    mean, rstd = mean.float(), rstd.float()
    gy = bu.randn(rows, H, seed=11, dtype=dtype)
    got = backward(moe, gy, x, w, mean, rstd)
    refs = bu.norm_backward(gy, x, w, mean, rstd, None)
    tols = bu.norm_backward_tol(gy, x, w, mean, rstd, None, dtype)
    for name, g, r, t in zip(("gx", "gw", "gb"), got, refs, tols):
        bu.assert_within(g, r, t, name)


@pytest.mark.parametrize("H", [1024, 1001, 5001])
def test_a_row_of_nans_stays_alone(H):
    """Unaligned rows share 16-byte pieces: what is wrong in one does not reach the next."""
    moe = moe_mod()
    x, w, b = inputs(40, H, torch.bfloat16, torch.bfloat16)
    x[7] = float("nan")
    x[20] = float("inf")
    y, _, mean, rstd = forward(moe, x, w, b, None)
    gx, _, _ = backward(moe, x, x, w, mean.cpu(), rstd.cpu())
    bad = torch.zeros(40, dtype=torch.bool)
    bad[7] = bad[20] = True
    for out in (y, gx):
        assert torch.equal(torch.isnan(out).all(1).cpu(), bad)
        assert torch.equal(torch.isnan(out).any(1).cpu(), bad)


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("H", [1, 2, 3, 5, 7, 9])
def test_rows_narrower_than_a_piece(H, dtype):
    """Rows that lie close, so that several share 16 bytes and the last ones' pieces end behind the matrix."""
    moe = moe_mod()
    for rows in (2, 3, 4, 8, 9, 30, 300):
        for pad in (0, 1, 2):
            x, w, b = inputs(rows, H, dtype, dtype)
            res = bu.randn(rows, H, seed=3, dtype=dtype)
            views = []
            for t in (x, res, torch.zeros_like(x)):
                flat = torch.full((rows * (H + pad) - pad,), float("nan"), dtype=dtype, device="cuda")
                v = flat.as_strided((rows, H), (H + pad, 1))
                v.copy_(t)
                views.append(v)
            h = (x.float() + res.float()).to(dtype)
            moe.moe_layer_norm(views[0], w.cuda(), b.cuda(), EPS, views[2], residual=views[1])
            bu.assert_within(views[2], bu.norm_forward(h, w, b, EPS)[0], bu.norm_forward_tol(h, w, b, EPS, dtype)[0])
            moe.moe_layer_norm(views[0], w.cuda(), b.cuda(), EPS, views[2])
            bu.assert_within(views[2], bu.norm_forward(x, w, b, EPS)[0], bu.norm_forward_tol(x, w, b, EPS, dtype)[0])


@pytest.mark.parametrize("rows,H,dtype,residual", [
    (100003, 32, torch.bfloat16, False), (50001, 120, torch.float32, True), (30011, 1000, torch.float16, True),
    (100003, 13, torch.bfloat16, True), (100003, 51, torch.float32, False), (12007, 1001, torch.bfloat16, True),
    (3001, 4096, torch.bfloat16, True), (1500, 2050, torch.float16, False), (1600, 1501, torch.float32, True),
    (1300, 6144, torch.float32, True), (500, 8201, torch.bfloat16, True), (450, 16384, torch.float16, False),
    (400, 16401, torch.bfloat16, True), (300, 4099, torch.float32, False), (330, 8197, torch.float32, True),
    (400, 20000, torch.bfloat16, False)])
def test_forward_of_more_rows_than_run_at_once(rows, H, dtype, residual):
    """Every kernel's loop over rows, several rows a CTA or team, with the next row on its way."""
    moe = moe_mod()
    x, w, b = inputs(rows, H, dtype, torch.float32)
    res = bu.randn(rows, H, seed=9, dtype=dtype) if residual else None
    h = (x.float() + res.float()).to(dtype) if residual else x
    got = forward(moe, x, w, b, res)
    check_forward(got, h, w, b, EPS, dtype)
    assert not residual or torch.equal(got[1].cpu(), h)


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("rows,H", [(3000, 100), (2600, 513)])
def test_many_rows_that_start_differently(rows, H, dtype):
    """Inputs and outputs that share no alignment, element by element, more rows than run at once."""
    moe = moe_mod()
    x, w, b = inputs(rows, H, dtype, dtype)
    gy = bu.randn(rows, H, seed=11, dtype=dtype)
    _, xv = strided(x, 3, 1)
    _, yv = strided(x, 2, 5)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    moe.moe_layer_norm(xv, w.cuda(), b.cuda(), EPS, yv, mean=mean, rstd=rstd)
    check_forward((yv, None, mean, rstd), x, w, b, EPS, dtype)
    _, gv = strided(gy, 1, 2)
    ws = torch.empty(moe.moe_layer_norm_workspace_size(rows, H), dtype=torch.uint8, device="cuda")
    gw, gb = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_layer_norm_backward(gv, xv, w.cuda(), mean, rstd, yv, gw, gb, ws)
    refs = bu.norm_backward(gy, x, w, mean.cpu(), rstd.cpu(), None)
    tols = bu.norm_backward_tol(gy, x, w, mean.cpu(), rstd.cpu(), None, dtype)
    for got, ref, tol in zip((yv, gw, gb), refs, tols):
        bu.assert_within(got, ref, tol)
