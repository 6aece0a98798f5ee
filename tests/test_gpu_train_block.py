"""The experts' training operators used together, as the example does: every stage against its 64-bit form on the values
that the stage before it stored, two steps that gather the weights' gradients, one CUDA graph, another stream."""
import numpy as np
import pytest
import torch

import block_util as bu
import train_util as tu
from gpu_util import moe_mod
from test_gpu_block import example
from train_util import BF

pytestmark = pytest.mark.gpu


def block_of(T, H, I, E, K, seed=0, m=8):
    ex = example()
    r = lambda *s, k: bu.randn(*s, seed=seed + k)
    w = dict(norm_w=(1 + 0.1 * r(H, k=1)).bfloat16(), router=r(E, H, k=2) * H ** -0.5,
             w13=(r(E, 2 * I, H, k=3) * H ** -0.5).bfloat16(), w2=(r(E, H, I, k=4) * I ** -0.5).bfloat16())
    return ex, w, ex.ExpertTrainBlock(*(t.cuda() for t in w.values()), T, K, m)


def segments_of(block):
    off, cnt = block.handle.padded_offsets.cpu().numpy(), block.handle.tokens_per_expert.cpu().numpy()
    return [(e, int(off[e]), int(off[e] + cnt[e])) for e in range(block.shape.E)]


class _Plan:
    """What train_util's forms read of a routing."""

    def __init__(self, block):
        self.segments, self.cap, self.shape = segments_of(block), block.layout.capacity, block.shape
        self.routed = torch.zeros(self.cap, dtype=torch.bool)
        for _, b, n in self.segments:
            self.routed[b:n] = True


@pytest.mark.parametrize("T,H,I,E,K", [(1, 128, 128, 8, 2), (37, 256, 384, 6, 3), (300, 512, 256, 4, 2)])
def test_every_stage(T, H, I, E, K):
    ex, w, block = block_of(T, H, I, E, K)
    x, res, g = (bu.randn(T, H, seed=s).bfloat16() for s in (11, 12, 13))
    y = block.forward(x.cuda(), res.cuda())
    torch.cuda.synchronize()
    h = (x.float() + res.float()).bfloat16()
    assert torch.equal(block.sum.cpu(), h)
    v, tv = tu.rms_forward(h, w["norm_w"], ex.EPS)[0], tu.rms_forward_tol(h, w["norm_w"], ex.EPS)[0]
    bu.assert_within(block.h, v, tv + bu.rounding(v, BF), "norm")
    r = _Plan(block)
    on = r.routed
    token = block.handle.token_of.cpu().long()
    rows, pre, act, out, probs = (t.cpu().clone() for t in (block.rows, block.pre, block.act, block.out_rows, block.probs))
    assert torch.equal(rows[on], block.h.cpu()[token[on]])

    def stage(got, ref, tol, what):
        bu.assert_within(got[on], ref[on], tol[on], what)

    ref = tu.gemm_forward(r, w["w13"], rows)
    stage(pre, ref, tu.gemm_tol(ref, tu.gemm_forward(r, w["w13"].abs(), rows.abs()), H, BF), "FC1")
    pre[~on], probs[~on] = 0, 0
    stage(act, tu.swiglu(pre, probs), tu.swiglu_tol(pre, probs, BF), "SwiGLU")
    ref = tu.gemm_forward(r, w["w2"], act)
    stage(out, ref, tu.gemm_tol(ref, tu.gemm_forward(r, w["w2"].abs(), act.abs()), I, BF), "FC2")
    total, absolute = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    total.index_add_(0, token[on], out[on].double())
    absolute.index_add_(0, token[on], out[on].double().abs())
    bu.assert_within(block.y, total, K * bu.U * absolute + bu.rounding(total, BF), "combine")

    # two steps: the second adds to the first's gradients of the weights
    g_w13, g_w2 = torch.zeros(w["w13"].shape, dtype=torch.float64), torch.zeros(w["w2"].shape, dtype=torch.float64)
    t13, t2 = g_w13.clone(), g_w2.clone()
    for step in (1, 2):
        if step == 2:
            block.forward(x.cuda(), res.cuda())
        g_x, g_norm_w, g_router = block.backward(g.cuda())
        torch.cuda.synchronize()
        g_rows = torch.zeros(r.cap, H, dtype=BF)
        g_rows[on] = g[token[on]]  # weight 1: the combine is unweighted
        g_act, g_pre, g_probs = block.g_act.cpu(), block.pre.cpu(), block.g_probs_rows.cpu()
        most = max(n - b for _, b, n in r.segments)
        for total, tol, got, a, b in ((g_w2, t2, block.g_w2, g_rows, act), (g_w13, t13, block.g_w13, g_pre, rows)):
            add = tu.gemm_weight(r, a, b)
            total += add
            tol += tu.gemm_tol(total, tu.gemm_weight(r, a.abs(), b.abs()), most, torch.float32)
            bu.assert_within(got, total, tol, "weights")
        ref = tu.gemm_data(r, w["w2"], g_rows)
        stage(g_act, ref, tu.gemm_tol(ref, tu.gemm_data(r, w["w2"].abs(), g_rows.abs()), H, BF), "gradient of act")
        ga = g_act.clone()
        ga[~on] = 0
        ref, rp, tol, tp = tu.swiglu_backward(pre, probs, ga)
        stage(g_pre, ref, tol + bu.rounding(ref, BF), "gradient of pre")
        stage(g_probs, rp, tp + bu.rounding(rp, torch.float32), "gradient of the probabilities")
        ref = tu.gemm_data(r, w["w13"], g_pre)
        stage(block.g_out_rows.cpu(), ref, tu.gemm_tol(ref, tu.gemm_data(r, w["w13"].abs(), g_pre.abs()), 2 * I, BF),
              "gradient of the rows")
        refs = tu.rms_backward(block.g_h.cpu(), h, w["norm_w"], block.rstd.cpu(), g)
        tols = tu.rms_backward_tol(block.g_h.cpu(), h, w["norm_w"], block.rstd.cpu(), g, BF)
        bu.assert_within(g_x, refs[0], tols[0], "gx")
        bu.assert_within(g_norm_w, refs[1], tols[1], "gw")
    assert bool(torch.isfinite(g_router).all())


def test_gradients_against_autograd():
    """All of the block against autograd in 64 bits, the choice of experts held. Each of the about a dozen tensors
    between the stages is rounded to bf16 once, by 2^-8 of its elements at most and half of that in the mean square;
    a chain of a dozen such errors that do not cancel stays below 12 * 2^-9 = 2.4 % in the 2-norm."""
    T, H, I, E, K = 64, 256, 128, 4, 2
    ex, w, block = block_of(T, H, I, E, K, seed=30)
    x, res, g = (bu.randn(T, H, seed=s).bfloat16() for s in (41, 42, 43))
    y = block.forward(x.cuda(), res.cuda())
    gx, gnw, gr = block.backward(g.cuda())
    torch.cuda.synchronize()
    ids = block.routing.map.long().cpu()
    s = (x.float() + res.float()).bfloat16().double().requires_grad_(True)
    p = {k: v.double().requires_grad_(True) for k, v in w.items()}
    h = s * (s.square().mean(1, keepdim=True) + ex.EPS) ** -0.5 * p["norm_w"]
    probs = torch.softmax((h @ p["router"].T).gather(1, ids), 1)
    total = s
    for k in range(K):
        pre = torch.einsum("th,tnh->tn", h, p["w13"][ids[:, k]])
        a = pre[:, :I] * torch.nn.functional.silu(pre[:, I:]) * probs[:, k:k + 1]
        total = total + torch.einsum("ti,thi->th", a, p["w2"][ids[:, k]])
    total.backward(g.double())
    for name, got, ref in (("y", y, total), ("gx", gx, s.grad), ("norm", gnw, p["norm_w"].grad),
                           ("router", gr, p["router"].grad), ("w13", block.g_w13, p["w13"].grad),
                           ("w2", block.g_w2, p["w2"].grad)):
        ref = ref.detach()
        assert float((bu.f64(got) - ref).norm() / ref.norm()) <= 0.024, name


def test_in_a_graph_and_on_another_stream():
    T, H, I, E, K = 50, 128, 256, 5, 2
    ex, w, block = block_of(T, H, I, E, K, seed=60)
    x, res, g = (torch.empty(T, H, dtype=BF, device="cuda") for _ in range(3))

    def fill(seed):
        for i, t in enumerate((x, res, g)):
            t.copy_(bu.randn(T, H, seed=seed + 10 * i).bfloat16())

    def step():
        block.g_w13.zero_()
        block.g_w2.zero_()
        y = block.forward(x, res)
        return (y,) + block.backward(g) + (block.g_w13, block.g_w2)

    refs = {}
    for seed in (1, 2, 3):
        fill(seed)
        refs[seed] = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (3, 1, 2):
        fill(seed)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, refs[seed]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fill(3)
        got = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, refs[3]))


def test_fp8_rows_of_the_norm_through_the_layer():
    """The norm's codes and scales go through the dispatch and the FP8 experts like rows the dispatch quantises: the
    same bytes where the norm's rows are exact in bf16, so that both paths encode the same values."""
    moe = moe_mod()
    T, H, I, E, K, m = 48, 256, 128, 4, 2, 32
    # rows whose mean square is 1 and a power-of-two weight: h * rstd * w is h * w, exact in bf16 (eps 0)
    sign = torch.where(bu.randn(T, H, seed=1) < 0, -1.0, 1.0).bfloat16()
    w = torch.exp2(torch.randint(-2, 3, (H,), generator=torch.Generator().manual_seed(2)).float()).bfloat16()
    y = torch.empty(T, H, dtype=BF, device="cuda")
    codes = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(T, H // 128, device="cuda")
    moe.moe_rms_norm(sign.cuda(), w.cuda(), 0.0, y, codes=codes, scales=scales)
    assert torch.equal(y.cpu(), sign * w)
    r = tu.Routed(moe, T, E, K, m)
    shape = moe.Shape(T, H, E, K, I)
    none = moe.Routing(0, torch.zeros(T, K, dtype=torch.int16, device="cuda"))
    got = [torch.zeros(r.cap, H, dtype=torch.uint8, device="cuda"), torch.zeros(r.cap, H // 128, device="cuda")]
    want = [torch.zeros_like(t) for t in got]
    moe.moe_dispatch_permute(r.handle, shape, r.layout, moe.DTYPE_FP8_E4M3_B128, codes, scales, none, got[0], None, got[1])
    moe.moe_dispatch_permute(r.handle, shape, r.layout, moe.DTYPE_BF16_TO_FP8, y, None, none, want[0], None, want[1])
    on = r.routed.cuda()
    assert torch.equal(got[0][on], want[0][on]) and torch.equal(got[1][on], want[1][on])


def test_the_example_prints_the_expert_block(capsys):
    example().main()
    assert "expert block" in capsys.readouterr().out
