"""Top-k router and its gradient on the GPU against the 64-bit definition."""
import numpy as np
import pytest
import torch

import block_util as bu
import workloads
from gpu_util import moe_mod

pytestmark = pytest.mark.gpu

CASES = [(1, 1, 1), (5, 2, 1), (3, 7, 7), (9, 31, 4), (8, 33, 32), (64, 64, 8), (33, 100, 6), (16, 128, 128),
         (64, 256, 8), (40, 256, 36), (17, 257, 9), (7, 512, 22), (12, 1000, 40), (5, 1024, 128), (3000, 64, 8)]


def topk(moe, logits, K, score=0, renorm=True, scale=1.0, fmt=0, bias=None):
    T, E = logits.shape
    r = moe.Router(E, K, score=score, renormalize=renorm, scale=scale)
    sparse = fmt == moe.ROUTING_SPARSE_BOOL
    m = torch.full(r.map_shape(fmt, T), 77, dtype=torch.uint8 if sparse else torch.int16, device="cuda")
    p = torch.full(m.shape, float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_router_topk(r, logits.cuda(), moe.Routing(fmt, m, p), bias.cuda() if bias is not None else None, status)
    torch.cuda.synchronize()
    return m.cpu().numpy(), p.cpu().numpy(), int(status.item())


def check(moe, logits, K, score, renorm, scale=1.0, bias=None, exact_ids=True):
    l = logits.float().numpy()
    T, E = l.shape
    scores = bu.router_scores(l, score == 1, None if bias is None else bias.numpy())
    on = bu.router_select(scores, K)
    live = scores > -np.inf
    ids, pd, st = topk(moe, logits, K, score, renorm, scale, moe.ROUTING_DENSE_I16, bias)
    m, ps, st2 = topk(moe, logits, K, score, renorm, scale, moe.ROUTING_SPARSE_BOOL, bias)
    got_on, got_w = bu.dense_to_full(ids, pd, E)
    if exact_ids:
        assert np.array_equal(got_on, on)
    else:  # scores within rounding of one another may change places
        s = np.where(live, scores, -1e30)
        for t in range(T):
            assert got_on[t].sum() == on[t].sum() and not (got_on[t] & ~live[t]).any()
            out = live[t] & ~got_on[t]
            if out.any() and got_on[t].any():
                assert s[t][got_on[t]].min() >= s[t][out].max() - 16 * bu.U * (1 + np.abs(s[t][live[t]]).max())
        on = got_on
    for t in range(T):  # ids ascending, then -1 with weight 0
        n = int(on[t].sum())
        assert list(ids[t, :n]) == list(np.nonzero(on[t])[0]) and (ids[t, n:] == -1).all() and (pd[t, n:] == 0).all()
    assert np.array_equal(m, on.astype(np.uint8)) and np.array_equal(ps.astype(np.float64), got_w)
    want = bu.router_weights(l, live, on, score == 1, renorm, scale)
    tol = bu.router_tol(l, live, want, E)
    assert (np.abs(got_w - want) <= tol).all(), float(np.max(np.abs(got_w - want) - tol))
    nan = bool(np.isnan(l).any() or (bias is not None and bool(torch.isnan(bias).any())))
    assert st == st2 == (moe.DEV_ERR_NAN_LOGIT if nan else 0)
    return on


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,K", CASES)
def test_router(T, E, K, score):
    moe = moe_mod()
    for dtype in bu.DTYPES:
        for renorm in (True, False):
            check(moe, bu.randn(T, E, seed=T + E, dtype=dtype), K, score, renorm, 1.0 if renorm else 2.5)


@pytest.mark.parametrize("score", [0, 1])
def test_ties_masks_and_extremes(score):
    """Equal logits go to the lowest expert; -inf is never chosen; the type's lowest value is an ordinary logit."""
    moe = moe_mod()
    E, K = 96, 6
    low = torch.finfo(torch.float32).min
    l = bu.randn(14, E, seed=3)
    l[0] = 0.0
    l[1] = float("-inf")
    l[2] = float("-inf")
    l[2, 50] = -3.0
    l[3, ::2] = float("-inf")
    l[4] = low
    l[5] = low
    l[5, 7] = 1.0
    l[6, 20:60] = 4.0
    l[7, 3], l[7, 80] = 0.0, -0.0
    l[7, 4:80] = -5.0
    l[8] *= 60.0
    l[9] = -200.0 + l[9]
    l[10] = 200.0 + l[10]
    l[11, 90:] = float("-inf")
    l[11, :87] = float("-inf")
    l[12] = torch.round(l[12])
    l[13] = 1e-42 * torch.round(l[13] * 3)
    for renorm in (True, False):
        check(moe, l, K, score, renorm)
    for dtype in (torch.bfloat16, torch.float16):
        check(moe, torch.round(bu.randn(50, 256, seed=2)).to(dtype), 8, score, True)


@pytest.mark.parametrize("score", [0, 1])
def test_infinite_and_nan_logits(score):
    moe = moe_mod()
    l = bu.randn(6, 40, seed=8)
    l[0, 9] = float("inf")
    l[1, 9], l[1, 12] = float("inf"), float("inf")
    for renorm in (True, False):
        check(moe, l, 4, score, renorm)
    l[2, 5] = float("nan")
    l[3] = float("nan")
    l[4, 1:] = float("nan")
    for renorm in (True, False):
        check(moe, l, 4, score, renorm)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,K", [(64, 8), (256, 8), (300, 17)])
def test_selection_bias(score, E, K):
    """The bias moves the choice and not the weights; -inf masks an expert, NaN masks and is reported."""
    moe = moe_mod()
    l = bu.randn(50, E, seed=5)
    bias = bu.randn(E, seed=6, scale=0.5)
    for renorm in (True, False):
        check(moe, l, K, score, renorm, bias=bias, exact_ids=score == 0)
    bias[3], bias[E - 1] = float("-inf"), 30.0
    assert check(moe, l, K, score, True, bias=bias, exact_ids=score == 0)[:, E - 1].all()
    bias[10] = float("nan")
    check(moe, l, K, score, True, bias=bias, exact_ids=score == 0)


def test_strided_logits():
    moe = moe_mod()
    for dtype in bu.DTYPES:
        for off in (0, 1, 5):
            wide = bu.randn(30, 300, seed=1, dtype=dtype).cuda()
            view = wide[:, off:off + 256]
            a = topk(moe, view.contiguous(), 8)
            r = moe.Router(256, 8)
            m = torch.empty(30, 8, dtype=torch.int16, device="cuda")
            p = torch.empty(30, 8, device="cuda")
            moe.moe_router_topk(r, view, moe.Routing(0, m, p))
            assert np.array_equal(m.cpu().numpy(), a[0]) and np.array_equal(p.cpu().numpy(), a[1])
            g = torch.zeros(30, 290, dtype=dtype, device="cuda")
            ref = torch.empty(30, 256, dtype=dtype, device="cuda")
            gp = bu.randn(30, 8, seed=4).cuda()
            moe.moe_router_topk_backward(r, view, moe.Routing(0, m), gp, g[:, off:off + 256])
            moe.moe_router_topk_backward(r, view.contiguous(), moe.Routing(0, m), gp, ref)
            assert torch.equal(g[:, off:off + 256], ref)
            assert bool((g[:, :off] == 0).all()) and bool((g[:, off + 256:] == 0).all())


def backward(moe, logits, K, score, renorm, scale, fmt, m, gp):
    T, E = logits.shape
    r = moe.Router(E, K, score=score, renormalize=renorm, scale=scale)
    gl = torch.full((T, E), float("nan"), dtype=logits.dtype, device="cuda")
    moe.moe_router_topk_backward(r, logits.cuda(), moe.Routing(fmt, torch.from_numpy(m).cuda()),
                                 torch.from_numpy(gp.astype(np.float32)).cuda(), gl)
    return gl


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,K", CASES)
def test_router_backward(T, E, K, score):
    moe = moe_mod()
    for dtype in bu.DTYPES:
        for renorm in (True, False):
            logits = bu.randn(T, E, seed=T * 3 + E, dtype=dtype)
            if E > 4:
                logits[::3, 1] = float("-inf")
            l = logits.float().numpy()
            scale = 1.0 if renorm else 2.5
            ids, _, _ = topk(moe, logits, K, score, renorm, scale)
            gp = bu.randn(T, K, seed=7).numpy()
            on, g = bu.dense_to_full(ids, gp, E)
            want = bu.router_backward(l, on, g, score == 1, renorm, scale)
            # n to (spread + E / 32 + 48) U as the weights; g - dot keeps the terms' magnitudes
            n = bu.router_weights(l, l > -np.inf, on if (score or renorm) else l > -np.inf, score == 1, renorm, 1.0)
            rel = bu.router_tol(l, l > -np.inf, n, E) / np.maximum(n, 1e-300)
            mag = scale * n * (np.abs(g) + (np.abs(g) * n * on).sum(1, keepdims=True))
            tol = mag * (3 * np.where(n > 0, rel, 0).max(1, keepdims=True) + 64 * bu.U) + 2.0 ** -126
            tol = torch.from_numpy(tol) + bu.rounding(torch.from_numpy(want), dtype)
            dense = backward(moe, logits, K, score, renorm, scale, moe.ROUTING_DENSE_I16, ids, gp)
            bu.assert_within(dense, torch.from_numpy(want), tol, "dense")
            gs = np.where(on, g, np.nan)  # entries off the map are ignored
            sparse = backward(moe, logits, K, score, renorm, scale, moe.ROUTING_SPARSE_BOOL, on.astype(np.uint8), gs)
            assert torch.equal(dense, sparse)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_against_differences(score, renorm):
    """The kernel's gradient against central differences of the 64-bit weights with the choice held."""
    moe = moe_mod()
    T, E, K = 6, 48, 5
    logits = bu.randn(T, E, seed=2)
    ids, _, _ = topk(moe, logits, K, score, renorm)
    gp = bu.randn(T, K, seed=3).numpy()
    on, g = bu.dense_to_full(ids, gp, E)
    got = bu.f64(backward(moe, logits, K, score, renorm, 1.0, 0, ids, gp)).numpy()
    l = logits.double().numpy()
    loss = lambda v: (bu.router_weights(v, np.ones(v.shape, bool), on, score == 1, renorm, 1.0) * g).sum()
    step = 1e-5
    for seed in range(4):
        v = bu.randn(T, E, seed=10 + seed).double().numpy()
        num = (loss(l + step * v) - loss(l - step * v)) / (2 * step)
        # fp32 roundings of terms no larger than |g|, and the difference's own error
        assert abs((got * v).sum() - num) <= 100 * bu.U * (np.abs(g).sum() * np.abs(v).max()) + 1e-8


def test_rows_without_routes_have_no_gradient():
    moe = moe_mod()
    logits = bu.randn(4, 64, seed=1)
    ids = np.full((4, 8), -1, np.int16)
    ids[2, :2] = (4, 9)
    ids[3, 0], ids[3, 1] = 3000, -7  # outside the experts: ignored
    gp = bu.randn(4, 8, seed=2).numpy()
    for score in (0, 1):
        for renorm in (True, False):
            g = backward(moe, logits, 8, score, renorm, 1.0, 0, ids, gp)
            assert bool((g[[0, 1, 3]] == 0).all()) and bool((g[2] != 0).any())


def test_zero_tokens_and_routing_feeds_preprocess():
    moe = moe_mod()
    r = moe.Router(16, 4)
    e = torch.empty(0, 16, device="cuda")
    moe.moe_router_topk(r, e, moe.Routing(0, torch.empty(0, 4, dtype=torch.int16, device="cuda"),
                                          torch.empty(0, 4, device="cuda")))
    moe.moe_router_topk_backward(r, e, moe.Routing(0, torch.empty(0, 4, dtype=torch.int16, device="cuda")),
                                 torch.empty(0, 4, device="cuda"), torch.empty_like(e))
    # dense and sparse maps dispatch alike
    logits = bu.randn(200, 16, seed=3)
    logits[5] = float("-inf")
    cap = workloads.unbounded_capacity(200, 4, 16, 32)
    shape, layout = moe.Shape(200, 128, 16, 4), moe.Layout(32, cap)
    handles = []
    for fmt in (moe.ROUTING_DENSE_I16, moe.ROUTING_SPARSE_BOOL):
        m, p, _ = topk(moe, logits, 4, fmt=fmt)
        h = moe.Handle.empty(shape, layout)
        ws = torch.empty(moe.moe_preprocess_workspace_size(shape), dtype=torch.uint8, device="cuda")
        moe.moe_preprocess(moe.Routing(fmt, torch.from_numpy(m).cuda(), torch.from_numpy(p).cuda()), shape, layout, h,
                           ws)
        handles.append(h)
    a, b = handles
    assert torch.equal(a.row_of, b.row_of) and int(a.status.item()) == 0 and int(b.status.item()) == 0
    assert bool((a.row_of[20:24] == -1).all())


def test_refusals():
    moe = moe_mod()
    l = torch.zeros(4, 16, device="cuda")
    m, p = torch.empty(4, 2, dtype=torch.int16, device="cuda"), torch.empty(4, 2, device="cuda")
    good = moe.Router(16, 2)
    for bad in (moe.Router(16, 2, score=2), moe.Router(16, 2, scale=float("inf"))):
        with pytest.raises(moe.MoeError):
            moe.moe_router_topk(bad, l, moe.Routing(0, m, p))
    with pytest.raises(moe.MoeError):  # more routes than experts
        moe.moe_router_topk(moe.Router(1, 2), l[:, :1], moe.Routing(0, m, p))
    with pytest.raises(moe.MoeError):
        moe.moe_router_topk(good, l, moe.Routing(0, m, None))
    with pytest.raises(ValueError):
        moe.moe_router_topk(good, l, moe.Routing(7, m, p))
    with pytest.raises(ValueError):
        moe.moe_router_topk(good, l, moe.Routing(0, m.int(), p))
    with pytest.raises(ValueError):
        moe.moe_router_topk(good, l.double(), moe.Routing(0, m, p))
    with pytest.raises(ValueError):
        moe.moe_router_topk(good, l, moe.Routing(1, m, p))
    with pytest.raises(ValueError):
        moe.moe_router_topk(good, l, moe.Routing(0, m, p), select_bias=torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_router_topk_backward(good, l, moe.Routing(0, m), p[:2], torch.empty_like(l))
    wide = torch.zeros(4, 40, device="cuda")
    with pytest.raises(moe.MoeError):  # the gradient over the logits, shifted
        moe.moe_router_topk_backward(good, wide[:, :16], moe.Routing(0, m), p, wide[:, 8:24])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K", [(9, 5, 2), (33, 64, 8), (20, 256, 8), (6, 300, 17), (4, 1000, 40)])
def test_gradient_with_experts_the_bias_masks(T, E, K, renorm, score, fmt):
    """Weights and gradient are of the same formula whatever the bias does to the choice: a bias of -inf or NaN keeps
    an expert from being chosen and leaves its logit in the softmax; logits of -inf are in neither."""
    moe = moe_mod()
    scale = 1.0 if renorm else 2.5
    for dtype in bu.DTYPES:
        logits = bu.randn(T, E, seed=T + E, dtype=dtype)
        logits[:, 1] += 3.0  # what the bias masks would have been chosen, and weighs in the sum
        logits[::2, 3] = float("-inf")
        bias = bu.randn(E, seed=6, scale=0.5)
        bias[1], bias[0] = float("-inf"), float("nan")
        l = logits.float().numpy()
        m, w, status = topk(moe, logits, K, score, renorm, scale, fmt, bias)
        assert status == moe.DEV_ERR_NAN_LOGIT
        on, got = bu.dense_to_full(m, w, E) if fmt == 0 else (m != 0, w.astype(np.float64))
        assert not on[:, :2].any() and (on.sum(1) == np.minimum(K, (l > -np.inf).sum(1) - 2)).all()
        live = l > -np.inf
        want = bu.router_weights(l, live, on, score == 1, renorm, scale)
        assert (np.abs(got - want) <= bu.router_tol(l, live, want, E)).all()
        gp = np.where(on, bu.randn(T, E, seed=7).numpy(), 0.0)
        g = bu.f64(backward(moe, logits, K, score, renorm, scale, fmt, m,
                            gp if fmt else np.where(m >= 0, np.take_along_axis(gp, np.maximum(m, 0).astype(np.int64),
                                                                               1), 0.0)))
        ref = bu.router_backward(l, on, gp, score == 1, renorm, scale)
        n = bu.router_weights(l, live, on if (score or renorm) else live, score == 1, renorm, 1.0)
        rel = bu.router_tol(l, live, n, E) / np.maximum(n, 1e-300)
        mag = scale * n * (np.abs(gp) + (np.abs(gp) * n * on).sum(1, keepdims=True))
        tol = mag * (3 * np.where(n > 0, rel, 0).max(1, keepdims=True) + 64 * bu.U) + 2.0 ** -126
        tol = torch.from_numpy(tol) + bu.rounding(torch.from_numpy(ref), dtype)
        bu.assert_within(g, torch.from_numpy(ref), tol)
        # the formula of the gradient is the weights': its product with a direction against their differences
        v = np.where(live, bu.randn(T, E, seed=9).double().numpy(), 0.0)
        step = 1e-5
        a, b = (bu.router_weights(np.where(live, l + d * step * v, -np.inf), live, on, score == 1, renorm, scale)
                for d in (1, -1))
        num = ((a - b) * gp).sum() / (2 * step)
        assert abs((ref * v).sum() - num) <= 1e-7 * (1 + np.abs(gp).sum())


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,K,copies", [(7, 2, 400), (64, 8, 100), (100, 6, 60), (256, 8, 31), (256, 36, 31), (300, 17, 30),
                                        (1000, 40, 30)])
def test_more_tokens_than_run_at_once(E, K, copies, score):
    """Every token's routes and gradient are those of the same token in a batch of its own, wherever it lies."""
    moe = moe_mod()
    T = 997
    for dtype, renorm, fmt in ((torch.float32, True, 0), (torch.bfloat16, False, 0), (torch.float16, True, 1),
                               (torch.float32, False, 1)):
        base = bu.randn(T, E, seed=E, dtype=dtype)
        base[5] = float("-inf")
        base[11::17, 2] = float("-inf")
        check(moe, base[:200], K, score, renorm)
        logits = base.repeat(copies, 1)
        m0, p0, _ = topk(moe, base, K, score, renorm, 1.5, fmt)
        m, p, _ = topk(moe, logits, K, score, renorm, 1.5, fmt)
        assert (m.reshape(copies, T, -1) == m0).all() and (p.reshape(copies, T, -1) == p0).all()
        gp = bu.randn(*m0.shape, seed=7).numpy()
        g0 = backward(moe, base, K, score, renorm, 1.5, fmt, m0, gp)
        g = backward(moe, logits, K, score, renorm, 1.5, fmt, m, np.tile(gp, (copies, 1)))
        assert torch.equal(g.view(copies, T, E), g0.expand(copies, T, E))


def test_choice_by_biased_sigmoids_is_that_of_fp32():
    """With a bias the choice goes by 1 / (1 + exp(-logit)) + bias, every step rounded to fp32 once, and equal scores by
    the lowest expert: near ties, of which there are many among so many tokens, come out as in plain fp32."""
    moe = moe_mod()
    for T, E, K in ((60000, 256, 8), (30000, 64, 6), (9000, 1000, 40)):
        l = bu.randn(T, E, seed=E, scale=3.0).cuda()
        l[:50] *= 30.0
        l[T // 2:] = 1e-5 * l[T // 2:] + torch.linspace(-4.0, 4.0, T - T // 2, device="cuda")[:, None]
        bias = bu.randn(E, seed=1, scale=1e-5).cuda()
        score = 1.0 / (1.0 + torch.exp(-l)) + bias
        ids = torch.sort(torch.sort(score, dim=1, descending=True, stable=True).indices[:, :K], dim=1).values
        m, _, _ = topk(moe, l, K, score=1, bias=bias)
        assert int((torch.from_numpy(m) != ids.cpu()).any(1).sum()) == 0
