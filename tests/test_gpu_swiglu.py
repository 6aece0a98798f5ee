"""SwiGLU of dispatched rows and its gradient on the GPU against the 64-bit formulas."""
import pytest
import torch

import block_util as bu
import train_util as tu
from gpu_util import moe_mod

pytestmark = pytest.mark.gpu

# (T, E, K, m, I): one token, widths of one element to many pieces, few rows and more than run at once
SIZES = [(1, 1, 1, 1, 1), (1, 8, 2, 32, 128), (5, 3, 2, 8, 7), (9, 4, 2, 4, 2048), (40, 6, 3, 32, 100), (3, 2, 1, 1, 5000),
         (700, 5, 2, 8, 264), (1500, 4, 1, 1, 33), (2, 1024, 8, 1, 64)]


def run(moe, r, pre, p, dtype):
    I = pre.shape[1] // 2
    out = torch.full((r.cap, I), 7.0, dtype=dtype, device="cuda")
    moe.moe_swiglu(r.handle, r.shape, r.layout, pre.cuda(), out, None if p is None else p.cuda())
    return out


def run_backward(moe, r, pre, p, ga, want_probs=True):
    gpre = torch.full(pre.shape, 7.0, dtype=pre.dtype, device="cuda")
    gp = torch.full((r.cap,), 7.0, device="cuda") if want_probs else None
    moe.moe_swiglu_backward(r.handle, r.shape, r.layout, pre.cuda(), ga.cuda(), gpre, None if p is None else p.cuda(), gp)
    return gpre, gp


def probs_of(r, seed=5):
    p = torch.rand(r.cap, generator=torch.Generator().manual_seed(seed))
    p[~r.routed] = float("nan")
    return p


def check(r, got, ref, tol):
    got = got.cpu()
    assert bool((got[~r.routed] == 7.0).all()), "rows outside the segments were written"
    bu.assert_within(got[r.routed], ref[r.routed], tol[r.routed])


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("T,E,K,m,I", SIZES)
def test_forward_and_backward(T, E, K, m, I, dtype):
    moe = moe_mod()
    r = tu.Routed(moe, T, E, K, m, empty=(0,) if E > K else ())
    pre, ga = r.rows(2 * I, dtype, 1, 2.0), r.rows(I, dtype, 2)
    for p in (None, probs_of(r)):
        check(r, run(moe, r, pre, p, dtype), tu.swiglu(pre, p), tu.swiglu_tol(pre, p, dtype))
        ref, rp, tol, tp = tu.swiglu_backward(pre, p, ga)
        gpre, gp = run_backward(moe, r, pre, p, ga)
        check(r, gpre, ref, tol + bu.rounding(ref, dtype))
        check(r, gp, rp, tp + bu.rounding(rp, torch.float32))
        assert torch.equal(run_backward(moe, r, pre, p, ga, False)[0], gpre)


@pytest.mark.parametrize("dtype", bu.DTYPES)
@pytest.mark.parametrize("I", [1, 8, 40])
def test_gradient_of_the_probabilities_at_any_gate(I, dtype):
    """fp32 whatever the rows: sums of one term, exact but for it. The term's error does not grow with the gate: the full
    exponential to 2 ulp (4 U), 1 + z to U and z's 2 U, the quotient to 2 ulp (4 U) and its product to U (s to 12 U), then
    three products: 15 U, and U for terms of the second order."""
    moe = moe_mod()
    r = tu.Routed(moe, 3000, 4, 1, 1)
    g = torch.Generator().manual_seed(1)
    pre, ga = torch.zeros(r.cap, 2 * I), torch.rand(r.cap, I, generator=g) + 1
    pre[:, 0] = torch.rand(r.cap, generator=g) + 1
    pre[:, I:] = torch.rand(r.cap, I, generator=g) * 90 - 70
    pre, ga = pre.to(dtype), ga.to(dtype)
    _, ref, _, _ = tu.swiglu_backward(pre, None, ga)
    gp = run_backward(moe, r, pre, None, ga)[1]
    check(r, gp, ref, 16 * bu.U * ref.abs())


@pytest.mark.parametrize("dtype", bu.DTYPES)
def test_gradient_against_differences(dtype):
    """Central differences of the 64-bit forward: the gradient is that of what the forward computes."""
    moe = moe_mod()
    r = tu.Routed(moe, 6, 2, 1, 4)
    pre, ga, p = r.rows(2 * 24, dtype, 1, rest=0.0), r.rows(24, dtype, 2, rest=0.0), probs_of(r)
    p[~r.routed] = 0.0
    gpre, gp = (t.cpu().double() for t in run_backward(moe, r, pre, p, ga))
    loss = lambda a, q: (tu.swiglu(a, q) * ga.double()).sum(1)
    h = 1e-4
    for c in (0, 11, 24, 47):
        up, down = pre.double().clone(), pre.double().clone()
        up[:, c] += h
        down[:, c] -= h
        diff = (loss(up, p) - loss(down, p)) / (2 * h)
        # the third derivative times h^2 / 6 is below 1e-8 * |ga| * 10; then the gradient's own rounding
        tol = 1e-6 * (1 + diff.abs()) + bu.rounding(diff, dtype) * 1.01
        assert bool(((gpre[:, c] - diff).abs() <= tol)[r.routed].all()), c
    diff = (loss(pre.double(), p.double() + h) - loss(pre.double(), p.double() - h)) / (2 * h)
    assert bool(((gp - diff).abs() <= 1e-5 * (1 + diff.abs()))[r.routed].all())


@pytest.mark.parametrize("I,stride", [(64, 1 << 26), (33, (1 << 26) + 1)])
def test_offsets_beyond_32_bits(I, stride):
    """Rows so far apart that their offsets pass 2^31 elements: as rows that are close."""
    moe = moe_mod()
    r = tu.Routed(moe, 40, 2, 2, 2)
    pre, ga, p, dtype = r.rows(2 * I, torch.bfloat16, 1), r.rows(I, torch.bfloat16, 2), probs_of(r), torch.bfloat16
    assert (r.cap - 2) * stride > 1 << 32

    def apart(t):
        v = torch.empty((r.cap - 1) * stride + t.shape[1], dtype=dtype, device="cuda").as_strided(t.shape, (stride, 1))
        return v.copy_(t)

    prd, gad, act = apart(pre), apart(ga), apart(torch.full((r.cap, I), 7.0))
    moe.moe_swiglu(r.handle, r.shape, r.layout, prd, act, p.cuda())
    assert torch.equal(act, run(moe, r, pre, p, dtype))
    gp = torch.full((r.cap,), 7.0, device="cuda")
    moe.moe_swiglu_backward(r.handle, r.shape, r.layout, prd, gad, prd, p.cuda(), gp)
    want, want_p = run_backward(moe, r, pre, p, ga)
    assert torch.equal(prd[r.routed.cuda()], want[r.routed.cuda()]) and torch.equal(gp, want_p)


@pytest.mark.parametrize("dtype", bu.DTYPES)
def test_gates_at_the_ends(dtype):
    """Gates far out: exp neither overflows nor cancels, and the gate's slope there is 0 or 1."""
    moe = moe_mod()
    r = tu.Routed(moe, 1, 1, 1, 1)
    g = torch.tensor([-300.0, -100.0, -88.5, -60.0, -20.0, -0.0, 0.0, 20.0, 60.0, 88.5, 100.0, 300.0], dtype=dtype)
    pre = torch.cat([torch.full_like(g, 1.5), g])[None, :]
    ga = torch.ones(1, g.numel(), dtype=dtype)
    check(r, run(moe, r, pre, None, dtype), tu.swiglu(pre, None), tu.swiglu_tol(pre, None, dtype))
    ref, rp, tol, tp = tu.swiglu_backward(pre, None, ga)
    gpre, gp = run_backward(moe, r, pre, None, ga)
    check(r, gpre, ref, tol + bu.rounding(ref, dtype))
    check(r, gp, rp, tp + bu.rounding(rp, torch.float32))


@pytest.mark.parametrize("I,pad,shift", [(64, 8, 8), (64, 1, 0), (40, 3, 5), (33, 2, 1)])
@pytest.mark.parametrize("dtype", bu.DTYPES)
def test_strides_alignment_and_in_place(dtype, I, pad, shift):
    moe = moe_mod()
    r = tu.Routed(moe, 30, 3, 2, 8)
    pre, ga, p = r.rows(2 * I, dtype, 1), r.rows(I, dtype, 2), probs_of(r)
    ref, gref, pref = run(moe, r, pre, p, dtype), *run_backward(moe, r, pre, p, ga)

    def apart(t):
        buf = torch.full((r.cap, t.shape[1] + pad + shift), 9.0, dtype=dtype, device="cuda")
        v = buf[:, shift:shift + t.shape[1]]
        v.copy_(t)
        return buf, v

    pb, pv = apart(pre)
    ob, ov = apart(torch.full((r.cap, I), 7.0))
    _, gv = apart(ga)
    moe.moe_swiglu(r.handle, r.shape, r.layout, pv, ov, p.cuda())
    assert torch.equal(ov, ref)
    gp = torch.full((r.cap,), 7.0, device="cuda")
    moe.moe_swiglu_backward(r.handle, r.shape, r.layout, pv, gv, pv, p.cuda(), gp)
    assert torch.equal(pv[r.routed.cuda()], gref[r.routed.cuda()])
    bu.assert_within(gp.cpu()[r.routed], bu.f64(pref)[r.routed], 2 * tu.swiglu_backward(pre, p, ga)[3][r.routed])
    for buf, cols in ((pb, 2 * I), (ob, I)):
        assert bool((buf[:, :shift] == 9.0).all()) and bool((buf[:, shift + cols:] == 9.0).all())


@pytest.mark.parametrize("cut", [0, 1, 9, 33])
def test_below_the_capacity(cut):
    moe = moe_mod()
    r = tu.Routed(moe, 25, 4, 2, 8, cap=cut)
    pre, ga = r.rows(64, torch.bfloat16, 1), r.rows(32, torch.bfloat16, 2)
    check(r, run(moe, r, pre, None, torch.bfloat16), tu.swiglu(pre, None), tu.swiglu_tol(pre, None, torch.bfloat16))
    ref, _, tol, _ = tu.swiglu_backward(pre, None, ga)
    check(r, run_backward(moe, r, pre, None, ga)[0], ref, tol + bu.rounding(ref, torch.bfloat16))


def test_no_tokens_and_refusals():
    moe = moe_mod()
    r = tu.Routed(moe, 0, 2, 1, 8)
    pre = torch.zeros(r.cap, 64, dtype=torch.bfloat16, device="cuda")
    act = torch.full((r.cap, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_swiglu(r.handle, r.shape, r.layout, pre, act)
    assert bool((act == 7.0).all())
    call = lambda *a, **k: moe.moe_swiglu(r.handle, r.shape, r.layout, *a, **k)
    for bad in ((pre[:, :62], act), (pre.float(), act), (pre[:3], act), (pre, act[:, 0])):
        with pytest.raises(ValueError):
            call(*bad)
    with pytest.raises(ValueError):
        call(pre, act, probs=torch.zeros(r.cap, dtype=torch.float64, device="cuda"))
    with pytest.raises(moe.MoeError):  # over its input
        call(pre, pre[:, 16:48])
    with pytest.raises(moe.MoeError):  # the gradient over the rows, shifted
        wide = torch.zeros(r.cap, 80, dtype=torch.bfloat16, device="cuda")
        moe.moe_swiglu_backward(r.handle, r.shape, r.layout, wide[:, :64], act, wide[:, 16:80])
