"""The operators around the layer used together with it: the example's decode and
training blocks against plain 64-bit forms, one CUDA graph, another stream."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import block_util as bu
from gpu_util import moe_mod

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    moe_mod()
    spec = importlib.util.spec_from_file_location("moe_block_example", os.path.join(ROOT, "examples", "moe_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def step_of(v):
    """One bf16 rounding of each value."""
    return bu.rounding(v, torch.bfloat16)


def test_decode_block_matches_64_bits():
    """Every stage against its 64-bit form on the values the stage before it stored."""
    ex = example()
    T, H, E, K, I = 12, 512, 16, 3, 256
    block = ex.DecodeBlock(ex.random_weights(E, H, I, 64), T, K)
    x, res = bu.randn(T, H, seed=1, dtype=torch.bfloat16), bu.randn(T, H, seed=2, dtype=torch.bfloat16)
    y = block.step(x.cuda(), res.cuda())
    torch.cuda.synchronize()
    w = block.w
    h = (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(block.sum.cpu(), h)
    nw, nb = w.norm_w.cpu(), w.norm_b.cpu()
    bu.assert_within(block.h, bu.norm_forward(h, nw, nb, ex.EPS)[0], bu.norm_forward_tol(h, nw, nb, ex.EPS, h.dtype)[0])
    logits = block.logits.float().cpu().numpy()
    on = bu.router_select(bu.router_scores(logits, False, None), K)
    got_on, probs = bu.dense_to_full(block.routing.map.cpu().numpy(), block.routing.probs.cpu().numpy(), E)
    assert np.array_equal(on, got_on)
    want = bu.router_weights(logits, np.ones_like(on), on, False, True, 1.0)
    assert (np.abs(probs - want) <= bu.router_tol(logits, np.ones_like(on), want, E)).all()
    # experts on the stored h, the activations rounded to bf16 between the two products
    deq = lambda q, e: bu.w4_dequant(*(t if t is None else (t if e is None else t[e]).cpu()
                                       for t in (q.codes, q.scales, q.zeros)), q.group)
    hb = block.h.cpu()

    def mlp(rows, w13, w2, e):
        act, ta = bu.w4_product(rows, deq(w13, e), w13.group, swiglu=True)
        W2 = deq(w2, e)
        out, to = bu.w4_product(act.to(torch.bfloat16), W2, w2.group)
        # either side's activations are within ta of one another before their rounding, and a step apart after it
        return out, to + (ta + step_of(act)) @ W2.abs().T

    total, tol = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        t = np.nonzero(on[:, e])[0]
        if len(t):
            out, to = mlp(hb[t], w.w13, w.w2, e)
            p = torch.from_numpy(probs[t, e])[:, None]
            total[t] += p * out
            tol[t] += p * (to + step_of(out))
    shared, ts = mlp(hb, w.shared_w13, w.shared_w2, None)
    ref = total + shared + h.double()
    # roundings: the combined rows, the shared expert's sum and the residual's
    tol = tol + ts + step_of(total) + step_of(total + shared) + step_of(ref) + 1e-6 * ref.abs()
    bu.assert_within(y, ref, 1.05 * tol)


def test_decode_block_in_a_graph_and_on_another_stream():
    ex = example()
    T, H, E, K, I = 5, 256, 8, 2, 128
    block = ex.DecodeBlock(ex.random_weights(E, H, I, 128), T, K)
    x, res = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16,
                                                                                 device="cuda")

    def fill(seed):
        x.copy_(bu.randn(T, H, seed=seed, dtype=torch.bfloat16))
        res.copy_(bu.randn(T, H, seed=seed + 50, dtype=torch.bfloat16))

    refs = {}
    for seed in (1, 2, 3):
        fill(seed)
        refs[seed] = block.step(x, res).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, res)
    for seed in (3, 1, 2):
        fill(seed)
        graph.replay()
        assert torch.equal(y, refs[seed])
    side = torch.cuda.Stream()
    for seed in (2, 3):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fill(seed)
            y2 = block.step(x, res).clone()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y2, refs[seed])


def test_explicit_streams():
    """The stream argument, a torch stream or a raw handle, is the stream the call runs on."""
    moe = moe_mod()
    x = torch.zeros(64, 4096, device="cuda")
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)  # the call has to wait for what its stream holds
            x.fill_(3.0)
            x[:, 0] = 5.0
        moe.moe_layer_norm(x, None, None, 1e-5, y, stream=handle)
        side.synchronize()
        ref = torch.nn.functional.layer_norm(x, (4096,))
        assert bool((y - ref).abs().max() < 1e-3)
        with torch.cuda.stream(side):
            x.zero_()
            y.zero_()
        side.synchronize()


def test_train_block_gradients():
    """The example's gradients against autograd of the block in 64 bits, the choice of experts held."""
    ex = example()
    T, H, E, K = 48, 256, 8, 2
    r = lambda *s, seed: bu.randn(*s, seed=seed)
    nw, nb = (1 + 0.1 * r(H, seed=1)).bfloat16(), (0.1 * r(H, seed=2)).bfloat16()
    router = r(E, H, seed=3) * H ** -0.5
    block = ex.TrainBlock(nw.cuda(), nb.cuda(), router.cuda(), T, K)
    x, res, g = (r(T, H, seed=s).bfloat16() for s in (4, 5, 6))
    out = block.forward(x.cuda(), res.cuda())
    gx, gnw, gnb, gr = block.backward(g.cuda())
    torch.cuda.synchronize()
    ids = block.routing.map.long().cpu()
    h = (x.float() + res.float()).bfloat16().double().requires_grad_(True)
    pw, pb, pr = (t.double().requires_grad_(True) for t in (nw, nb, router))
    n = torch.nn.functional.layer_norm(h, (H,), pw, pb, ex.EPS)
    p = torch.softmax(n @ pr.T, 1).gather(1, ids)
    y = p.sum(1, keepdim=True) * n + h
    y.backward(g.double())
    # bf16 steps of what is stored between the stages: h (the norm's output), the rows' gradients and their sum.
    # A route's gradient is the dot of g with h, of |g| |h| 2^-8 at most and less by the signs, here under 1 % of
    # the sum of |g| over the tokens that a router's row sees.
    bound = lambda ref, steps, scale: steps * 2.0 ** -8 * (ref.abs() + scale)
    assert bool(((bu.f64(out) - y.detach()).abs() <= bound(y.detach(), 3, 1.0)).all())
    assert bool(((bu.f64(gx) - h.grad).abs() <= bound(h.grad, 4, 1.0)).all())
    rows = g.double().abs().sum(0)
    assert bool(((bu.f64(gnw) - pw.grad).abs() <= bound(pw.grad, 3, 0) + 2.0 ** -7 * rows * 4).all())
    assert bool(((bu.f64(gnb) - pb.grad).abs() <= bound(pb.grad, 3, 0) + 2.0 ** -7 * rows).all())
    assert bool(((bu.f64(gr) - pr.grad).abs() <= 1e-2 * g.double().abs().mean() * T).all())


def test_the_example_runs(capsys):
    example().main()
    text = capsys.readouterr().out
    assert "decode block" in text and "train block" in text
