"""Root-mean-square norm on the GPU, with its 8-bit output and its backward pass, against the 64-bit formulas."""
import pytest
import torch

import block_util as bu
import train_util as tu
from block_util import U
from gpu_util import moe_mod

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 1), (5, 7), (4, 33), (9, 128), (6, 136), (7, 1000), (3, 1024), (2, 1537), (5, 4096), (3, 7168),
          (2, 8192), (1, 16384), (2, 16392), (2, 40000), (700, 264), (401, 2049), (3000, 64), (1300, 320)]
EPS = 1e-6


def inputs(rows, H, dtype, pdtype, seed=0):
    x = (bu.randn(rows, H, seed=seed) * torch.exp(0.5 * bu.randn(H, seed=seed + 1))).to(dtype)
    return x, (1.0 + 0.3 * bu.randn(H, seed=seed + 2)).to(pdtype)


def forward(moe, x, w, residual=None, eps=EPS, y=True, codes=True, want_sum=True):
    rows, H = x.shape
    d = lambda t: None if t is None else t.cuda()
    out = torch.full((rows, H), float("nan"), dtype=x.dtype, device="cuda") if y else None
    s = torch.full((rows, H), float("nan"), dtype=x.dtype, device="cuda") if residual is not None and want_sum else None
    rstd = torch.full((rows,), float("nan"), device="cuda")
    c = torch.full((rows, H), 0xAA, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) if codes else None
    sc = torch.full((rows, -(-H // 128)), float("nan"), device="cuda") if codes else None
    moe.moe_rms_norm(d(x), d(w), eps, out, residual=d(residual), sum_out=s, rstd=rstd, codes=c, scales=sc)
    torch.cuda.synchronize()
    return out, s, rstd, c, sc


def check_codes(c, sc, v, tv):
    """The scale is amax / 448 of values within their bounds; each code is within half a step of v over its own scale:
    2^-4 of the value, or half of E4M3's smallest step 2^-9, and what v itself may be off."""
    rows, H = v.shape
    pad = -(-H // 128) * 128 - H
    b = lambda t: torch.nn.functional.pad(t, (0, pad)).view(rows, -1, 128)
    amax, ta = b(v.abs()).amax(2), b(tv).amax(2)
    scale = torch.where(amax == 0, 1.0, amax / 448.0)
    bu.assert_within(sc, scale, (ta / 448.0 + 2 * U * scale) * 1.01 + 2.0 ** -149, "scales")
    s = bu.f64(sc).repeat_interleave(128, dim=1)[:, :H]
    got = c.cpu().float().double()
    assert bool(torch.isfinite(got).all())
    q, tq = v / s, tv / s + U * (v / s).abs()
    bu.assert_within(got, q, 2.0 ** -4 * q.abs().clamp(min=2.0 ** -6) + tq, "codes")
    # what lies clear of the border between two codes has the one nearest to it
    near = q.clamp(-448, 448).float().to(torch.float8_e4m3fn).float().double()
    clear = ((q + tq).clamp(-448, 448).float().to(torch.float8_e4m3fn).float() ==
             (q - tq).clamp(-448, 448).float().to(torch.float8_e4m3fn).float())
    assert bool((got == near)[clear].all())


def check(got, h, w, eps=EPS):
    y, _, rstd, c, sc = got
    v, r = tu.rms_forward(h, w, eps)
    tv, tr = tu.rms_forward_tol(h, w, eps)
    bu.assert_within(rstd, r, tr, "rstd")
    if y is not None:
        bu.assert_within(y, v, tv + bu.rounding(v, y.dtype), "y")
    if c is not None:
        check_codes(c, sc, v, tv)


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("rows,H", SHAPES)
def test_forward(rows, H, dtype):
    moe = moe_mod()
    for pdtype in {dtype, torch.float32}:
        x, w = inputs(rows, H, dtype, pdtype)
        both = forward(moe, x, w)
        check(both, x, w)
        alone = forward(moe, x, w, codes=False)
        check(alone, x, w)
        only = forward(moe, x, w, y=False)
        assert only[0] is None and torch.equal(only[3].view(torch.uint8), both[3].view(torch.uint8))
        assert torch.equal(only[4], both[4])


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("rows,H", [(3, 33), (4, 1024), (3, 7168), (2, 20000), (900, 256)])
def test_forward_residual(rows, H, dtype):
    """The norm is that of the stored sum, with and without the sum as an output, and the sum may replace an input."""
    moe = moe_mod()
    x, w = inputs(rows, H, dtype, dtype)
    res = bu.randn(rows, H, seed=9, scale=2.0, dtype=dtype)
    h = (x.float() + res.float()).to(dtype)
    for codes in (False, True):
        a = forward(moe, x, w, res, codes=codes)
        assert torch.equal(a[1].cpu(), h)
        check(a, h, w)
        assert torch.equal(forward(moe, x, w, res, want_sum=False, codes=codes)[0], a[0])
        for which in (0, 1):
            xd, rd, y = x.cuda(), res.cuda(), torch.empty_like(a[0])
            into = (xd, rd)[which]
            moe.moe_rms_norm(xd, w.cuda(), EPS, y, residual=rd, sum_out=into)
            bu.assert_within(y, *(lambda v, t: (v, t + bu.rounding(v, dtype)))(tu.rms_forward(h, w, EPS)[0],
                                                                               tu.rms_forward_tol(h, w, EPS)[0]))
            assert torch.equal(into.cpu(), h)


@pytest.mark.parametrize("H", [5, 64, 192, 1000, 7168])
def test_rows_of_zeros_and_no_weight(H):
    moe = moe_mod()
    for dtype in bu.DTYPES:
        x, _ = inputs(4, H, dtype, dtype)
        x[1] = 0
        x[2, :min(H, 128)] = 0  # a block of zeros beside others
        y, _, rstd, c, sc = got = forward(moe, x, None)
        check(got, x, None)
        assert bool((y[1] == 0).all()) and bool((c[1].float() == 0).all()) and bool((sc[1] == 1).all())
        assert bool((c[2, :128].float() == 0).all()) and float(sc[2, 0]) == 1.0


@pytest.mark.parametrize("H,stride", [(256, 1 << 27), (515, (1 << 27) + 1)])
def test_offsets_beyond_32_bits(H, stride):
    """Rows so far apart that their offsets pass 2^31 elements: as any others."""
    moe = moe_mod()
    rows, dtype = 34, torch.bfloat16
    x, w = inputs(rows, H, dtype, dtype)
    res, gy = (bu.randn(rows, H, seed=s).to(dtype) for s in (7, 8))

    def apart(t):
        v = torch.empty((rows - 1) * stride + H, dtype=dtype, device="cuda").as_strided(t.shape, (stride, 1))
        return v.copy_(t)

    xd, rd, yd, rstd = apart(x), apart(res), apart(x), torch.empty(rows, device="cuda")
    c = torch.empty(rows, H, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sc = torch.empty(rows, -(-H // 128), device="cuda")
    moe.moe_rms_norm(xd, w.cuda(), EPS, yd, residual=rd, sum_out=rd, rstd=rstd, codes=c, scales=sc)
    h = (x.float() + res.float()).to(dtype)
    assert torch.equal(rd.cpu(), h)
    check((yd, None, rstd, c, sc), h, w)
    ws = torch.empty(moe.moe_rms_norm_workspace_size(rows, H), dtype=torch.uint8, device="cuda")
    gw, gxd = torch.empty(H, device="cuda"), yd
    moe.moe_rms_norm_backward(xd.copy_(gy), rd, w.cuda(), rstd, gxd, grad_weight=gw, workspace=ws)
    refs, tols = (f(gy, h, w, rstd.cpu(), None, *a) for f, a in ((tu.rms_backward, ()), (tu.rms_backward_tol, (dtype,))))
    bu.assert_within(gxd, refs[0], tols[0], "gx")
    bu.assert_within(gw, refs[1], tols[1], "gw")


@pytest.mark.parametrize("H", [100, 2048])
def test_nonfinite_rows_stay_alone(H):
    moe = moe_mod()
    x, w = inputs(5, H, torch.bfloat16, torch.float32)
    ref = forward(moe, x, w)
    bad = x.clone()
    bad[1, 3], bad[3, 7] = float("nan"), float("inf")
    got = forward(moe, bad, w)
    for r in (0, 2, 4):
        for a, b in ((got[0], ref[0]), (got[3].view(torch.uint8), ref[3].view(torch.uint8)), (got[4], ref[4])):
            assert torch.equal(a[r], b[r])
    assert bool(torch.isnan(got[0][1]).all()) and bool(torch.isnan(got[0][3]).any())
    assert bool(torch.isnan(got[3].float()[1]).all()) and bool(torch.isnan(got[4][1]).all())


@pytest.mark.parametrize("H", [256, 500, 4096])
def test_a_weight_that_is_not_finite_stays_in_its_column(H):
    """Its own block's scale and codes are lost; other blocks, the end of a short row among them, are as ever."""
    moe = moe_mod()
    x, w = inputs(3, H, torch.bfloat16, torch.float32)
    ref = forward(moe, x, w)
    w2 = w.clone()
    w2[0] = float("inf")
    got = forward(moe, x, w2)
    assert torch.equal(got[0][:, 1:], ref[0][:, 1:])
    assert torch.equal(got[4][:, 1:], ref[4][:, 1:])
    assert torch.equal(got[3].view(torch.uint8)[:, 128:], ref[3].view(torch.uint8)[:, 128:])


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_scales_at_the_ends_of_the_range(scale):
    """Weights that bring v, and with it the scales, to the ends of fp32's range."""
    moe = moe_mod()
    for H in (128, 300, 2048):
        x, w = inputs(4, H, torch.float32, torch.float32)
        w = w * scale * (1e-7 if scale < 1 else 1e6)
        check(forward(moe, x, w), x, w)


def strided(t, pad, shift):
    buf = torch.full((t.shape[0], t.shape[1] + pad + shift), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return buf, v


def backward(moe, gy, h, w, rstd, gsum=None, want_w=True):
    rows, H = h.shape
    d = lambda t: None if t is None else t.cuda()
    gx = torch.full((rows, H), float("nan"), dtype=h.dtype, device="cuda")
    gw = torch.full((H,), float("nan"), device="cuda") if want_w else None
    ws = torch.full((moe.moe_rms_norm_workspace_size(rows, H),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_rms_norm_backward(d(gy), d(h), d(w), d(rstd), gx, gw, ws, grad_sum=d(gsum))
    torch.cuda.synchronize()
    return gx, gw


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("rows,H", SHAPES)
def test_backward(rows, H, dtype):
    moe = moe_mod()
    for pdtype in {dtype, torch.float32}:
        x, w = inputs(rows, H, dtype, pdtype)
        gy, gs = bu.randn(rows, H, seed=6, dtype=dtype), bu.randn(rows, H, seed=7, dtype=dtype)
        rstd = tu.rms_forward(x, w, EPS)[1].float()
        for gsum in (None, gs):
            gx, gw = backward(moe, gy, x, w, rstd, gsum)
            refs, tols = tu.rms_backward(gy, x, w, rstd, gsum), tu.rms_backward_tol(gy, x, w, rstd, gsum, dtype)
            bu.assert_within(gx, refs[0], tols[0], "gx")
            bu.assert_within(gw, refs[1], tols[1], "gw")
        assert torch.equal(backward(moe, gy, x, w, rstd, gs, False)[0], gx)
        assert all(torch.equal(a, b) for a, b in zip(backward(moe, gy, x, w, rstd, gs), (gx, gw)))


def test_gradient_against_differences():
    moe = moe_mod()
    x, w = inputs(3, 40, torch.float32, torch.float32)
    gy = bu.randn(3, 40, seed=6)
    rstd = tu.rms_forward(x, w, EPS)[1].float()
    gx, gw = (t.cpu().double() for t in backward(moe, gy, x, w, rstd))
    loss = lambda a, b: (tu.rms_forward(a, b, EPS)[0] * gy.double()).sum(1)
    h = 1e-5
    for c in (0, 17, 39):
        e = torch.zeros(40, dtype=torch.float64)
        e[c] = h
        diff = (loss(x.double() + e, w) - loss(x.double() - e, w)) / (2 * h)
        assert bool(((gx[:, c] - diff).abs() <= 1e-5 * (1 + diff.abs())).all())
        diff = ((loss(x, w.double() + e) - loss(x, w.double() - e)) / (2 * h)).sum()
        assert abs(gw[c] - diff) <= 1e-5 * (1 + abs(diff))


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("H,pad,shift", [(1024, 64, 0), (1024, 8, 8), (1024, 1, 0), (1024, 7, 1), (515, 5, 3)])
def test_strides_and_alignment(dtype, H, pad, shift):
    moe = moe_mod()
    rows = 37
    x, w = inputs(rows, H, dtype, dtype)
    res = bu.randn(rows, H, seed=5, dtype=dtype)
    gy, gs = bu.randn(rows, H, seed=6, dtype=dtype), bu.randn(rows, H, seed=7, dtype=dtype)
    h = (x.float() + res.float()).to(dtype)
    v, rstd = tu.rms_forward(h, w, EPS)
    tv, _ = tu.rms_forward_tol(h, w, EPS)
    _, xv = strided(x, pad, shift)
    _, rv = strided(res, pad, shift)
    for codes in (False, True):
        ob, ov = strided(torch.zeros(rows, H, dtype=dtype), pad, shift)
        sb, sv = strided(torch.zeros(rows, H, dtype=dtype), pad, shift)
        # codes that begin at any byte
        c = torch.full((rows * H + shift,), 0xAA, dtype=torch.uint8, device="cuda")[shift:].view(rows, H) if codes else None
        sc = torch.empty(rows, -(-H // 128), device="cuda") if codes else None
        moe.moe_rms_norm(xv, w.cuda(), EPS, ov, residual=rv, sum_out=sv, codes=c, scales=sc)
        bu.assert_within(ov, v, tv + bu.rounding(v, dtype))
        assert torch.equal(sv.cpu(), h)
        if codes:
            check_codes(c.clone().view(torch.float8_e4m3fn), sc, v, tv)
        for buf in (ob, sb):  # nothing outside the view is written
            assert bool(torch.isnan(buf[:, :shift]).all()) and bool(torch.isnan(buf[:, shift + H:]).all())
    _, gv = strided(gy, pad, shift)
    _, gsv = strided(gs, pad, shift)
    xob, xo = strided(torch.zeros(rows, H, dtype=dtype), pad, shift)
    ws = torch.empty(moe.moe_rms_norm_workspace_size(rows, H), dtype=torch.uint8, device="cuda")
    gw, rs = torch.empty(H, device="cuda"), rstd.float()
    moe.moe_rms_norm_backward(gv, sv, w.cuda(), rs.cuda(), xo, gw, ws, grad_sum=gsv)
    refs, tols = tu.rms_backward(gy, h, w, rs, gs), tu.rms_backward_tol(gy, h, w, rs, gs, dtype)
    bu.assert_within(xo, refs[0], tols[0])
    bu.assert_within(gw, refs[1], tols[1])
    assert bool(torch.isnan(xob[:, :shift]).all()) and bool(torch.isnan(xob[:, shift + H:]).all())


def test_codes_feed_the_dispatch():
    """Codes and scales of the norm are dispatched as FP8 rows, byte for byte, with zeros in the pad rows."""
    moe = moe_mod()
    T, H, E, K, m = 40, 256, 4, 2, 8
    x, w = inputs(T, H, torch.bfloat16, torch.bfloat16)
    _, _, _, c, sc = forward(moe, x, w)
    r = tu.Routed(moe, T, E, K, m)
    shape = moe.Shape(T, H, E, K)
    rows = torch.full((r.cap, H), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((r.cap, H // 128), 7.0, device="cuda")
    moe.moe_dispatch_permute(r.handle, shape, r.layout, moe.DTYPE_FP8_E4M3_B128, c.view(torch.uint8), sc,
                             moe.Routing(0, torch.zeros(T, K, dtype=torch.int16, device="cuda")), rows, None, scales)
    token = r.handle.token_of.long()
    on = r.routed.cuda()
    assert torch.equal(rows[on], c.view(torch.uint8)[token[on]]) and torch.equal(scales[on], sc[token[on]])


def test_no_rows_and_refusals():
    moe = moe_mod()
    none = torch.empty(0, 64, device="cuda")
    moe.moe_rms_norm(none, None, EPS, none)
    gw = torch.full((64,), float("nan"), device="cuda")
    ws = torch.empty(moe.moe_rms_norm_workspace_size(0, 64), dtype=torch.uint8, device="cuda")
    moe.moe_rms_norm_backward(none, none, None, torch.empty(0, device="cuda"), torch.empty_like(none), gw, ws)
    assert bool((gw == 0).all())
    x, y = torch.zeros(4, 128, device="cuda"), torch.zeros(4, 128, device="cuda")
    c, sc = torch.zeros(4, 128, dtype=torch.uint8, device="cuda"), torch.zeros(4, 1, device="cuda")
    for bad in (dict(y=y[:3]), dict(y=y.half()), dict(y=y, codes=c.int(), scales=sc), dict(y=y, codes=c[:, :64], scales=sc),
                dict(y=y, codes=c, scales=torch.zeros(4, 2, device="cuda")), dict(y=y, rstd=sc)):
        with pytest.raises(ValueError):
            moe.moe_rms_norm(x, None, EPS, **bad)
    for bad in (dict(y=None), dict(y=y, codes=c), dict(y=y, scales=sc), dict(y=x), dict(y=y, sum_out=c.float()),
                dict(y=y, codes=y.view(torch.uint8).view(-1)[:512].view(4, 128), scales=sc),
                dict(y=None, codes=x.view(torch.uint8).view(-1)[:512].view(4, 128), scales=sc)):
        with pytest.raises(moe.MoeError):
            moe.moe_rms_norm(x, None, EPS, **bad)
