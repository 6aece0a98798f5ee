"""4-bit matrix-vector products on the GPU against their 64-bit definition."""
import numpy as np
import pytest
import torch

import block_util as bu
from gpu_util import moe_mod

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def dev(t):
    return None if t is None else t.cuda()


def product(moe, x, w, swiglu=False, addend=None, group=128):
    codes, scales, zeros = w
    N = codes.shape[0]
    y = torch.full((x.shape[0], N // 2 if swiglu else N), float("nan"), dtype=x.dtype, device="cuda")
    moe.moe_w4_matvec(moe.W4Weight(dev(codes), dev(scales), dev(zeros), group), dev(x), y,
                      moe.W4_SWIGLU if swiglu else moe.W4_NONE, dev(addend))
    torch.cuda.synchronize()
    return y


# (M, N, Kd): one token to several passes; one feature, ragged tiles; one lane of a group, a short last group
SIZES = [(1, 1, 32), (1, 16, 128), (1, 300, 512), (2, 33, 96), (3, 17, 160), (4, 64, 1024), (5, 48, 4128), (7, 130, 224),
         (8, 64, 2048), (9, 50, 256), (13, 515, 1056), (16, 32, 4096), (17, 40, 288), (31, 66, 320), (32, 128, 512),
         (33, 20, 128), (70, 34, 352), (1, 1024, 7168), (2, 64, 14336)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,Kd", SIZES)
def test_product(M, N, Kd, group):
    moe = moe_mod()
    for dtype in (BF, HF):
        for zeros in (False, True):
            w = bu.w4_random(N, Kd, group, dtype, zeros, seed=M + N)
            W = bu.w4_dequant(*w, group)
            x = bu.randn(M, Kd, seed=Kd, dtype=dtype)
            ref, tol = bu.w4_product(x, W, group, dtype=dtype)
            bu.assert_within(product(moe, x, w, group=group), ref, tol, "plain")
            add = bu.randn(M, N, seed=1, dtype=dtype)
            ref, tol = bu.w4_product(x, W, group, addend=add, dtype=dtype)
            bu.assert_within(product(moe, x, w, addend=add, group=group), ref, tol, "addend")
            if N % 2 == 0:
                ref, tol = bu.w4_product(x, W, group, swiglu=True, dtype=dtype)
                bu.assert_within(product(moe, x, w, swiglu=True, group=group), ref, tol, "swiglu")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_code_and_zero_point_is_exact(dtype, group):
    """One-hot tokens read single weights back: (q - z) * scale for all 16 codes and zero points, scales powers of two."""
    moe = moe_mod()
    N, Kd = 32, 512
    codes, scales, zeros = bu.w4_random(N, Kd, group, dtype, True, seed=5)
    scales = torch.exp2(torch.randint(-6, 3, scales.shape, generator=torch.Generator().manual_seed(1)).float()).to(dtype)
    W = bu.w4_dequant(codes, scales, zeros, group)
    x = torch.eye(Kd, dtype=dtype)
    y = product(moe, x, (codes, scales, zeros), group=group)
    assert torch.equal(bu.f64(y), W.T)
    y = product(moe, x, (codes, scales, None), group=group)
    assert torch.equal(bu.f64(y), bu.w4_dequant(codes, scales, None, group).T)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 13, 30])
def test_nothing_is_left_from_an_earlier_call(M, group):
    """A product whose last group and last rows are short, right after one that filled the GPU's shared memory with
    NaN scales and NaN tokens."""
    moe = moe_mod()
    codes, scales, zeros = bu.w4_random(8192, 4096, group, HF, True, seed=1)
    dirty = (codes | 0xFF, torch.full_like(scales, float("nan")), zeros)
    w = bu.w4_random(99, 8224, group, HF, True, seed=2)
    x = bu.randn(M, 8224, seed=3, dtype=HF)
    ref, tol = bu.w4_product(x, bu.w4_dequant(*w, group), group, dtype=HF)
    for _ in range(3):
        assert bool(torch.isnan(product(moe, torch.full((M, 4096), float("nan"), dtype=HF), dirty, group=group)).all())
        bu.assert_within(product(moe, x, w, group=group), ref, tol)


@pytest.mark.parametrize("M", [1, 4, 11, 20])
def test_strided_rows_and_addend_in_place(M):
    moe = moe_mod()
    N, Kd, group = 70, 256, 64
    w = bu.w4_random(N, Kd, group, BF, True, seed=2)
    x, add = bu.randn(M, Kd, seed=3, dtype=BF), bu.randn(M, N, seed=4, dtype=BF)
    ref = product(moe, x, w, addend=add, group=group)
    wide = torch.full((M, Kd + 40), float("nan"), dtype=BF, device="cuda")
    xv = wide[:, 8:8 + Kd]
    xv.copy_(x)
    out = torch.full((M, N + 9), float("nan"), dtype=BF, device="cuda")
    yv = out[:, 5:5 + N]
    yv.copy_(add)
    weight = moe.W4Weight(*(dev(t) for t in w), group)
    moe.moe_w4_matvec(weight, xv, yv, addend=yv)
    assert torch.equal(yv, ref)
    assert bool(torch.isnan(out[:, :5]).all()) and bool(torch.isnan(out[:, 5 + N:]).all())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("scale", [1e38, 3e36, 1e-30, 2e-35])
def test_tokens_at_the_ends_of_the_range(scale, zeros, group):
    """bf16 tokens of one sign whose sum over a group is beyond fp32's range, and tiny ones, where the product is an
    ordinary number."""
    moe = moe_mod()
    for M, N, Kd in ((1, 256, 512), (5, 40, 608), (20, 70, 1024)):
        codes, scales, zp = bu.w4_random(N, Kd, group, BF, zeros, seed=M)
        # the largest product stays below Kd * 15 * 0.015 * 1e-5 * 2e38 = 4.6e35
        w = (codes, (scales.float() * (1e-5 if scale > 1 else 100.0)).to(BF), zp)
        x = ((1.0 + torch.rand(M, Kd, generator=torch.Generator().manual_seed(Kd))) * scale).to(BF)
        if M > 1:
            x[1] = -x[1]
        assert bool(torch.isfinite(x).all())
        ref, tol = bu.w4_product(x, bu.w4_dequant(*w, group), group)
        y = product(moe, x, w, group=group)
        assert bool(torch.isfinite(y).all())
        bu.assert_within(y, ref, tol)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("M,N,Kd", [(1, 257, 7168), (3, 130, 4096), (7, 300, 2048), (11, 70, 7168), (13, 515, 1056),
                                    (37, 33, 8224), (70, 261, 2048)])
def test_outputs_that_do_not_fill_a_round(M, N, Kd, group):
    """Few rows, so that CTAs share K steps, and numbers of outputs that leave some lanes of a warp without one in the
    last round before the CTAs meet; several passes over the weights where M exceeds 32. Results repeat bit for bit."""
    moe = moe_mod()
    w = bu.w4_random(N, Kd, group, BF, True, seed=N)
    x = bu.randn(M, Kd, seed=M, dtype=BF)
    for swiglu in (False, True)[:2 - N % 2]:
        ref, tol = bu.w4_product(x, bu.w4_dequant(*w, group), group, swiglu=swiglu)
        first = product(moe, x, w, swiglu=swiglu, group=group)
        bu.assert_within(first, ref, tol)
        for _ in range(20):
            assert torch.equal(product(moe, x, w, swiglu=swiglu, group=group), first)


def test_nonfinite_tokens_stay_alone():
    moe = moe_mod()
    w = bu.w4_random(40, 256, 128, BF, False, seed=2)
    x = bu.randn(12, 256, seed=3, dtype=BF)
    ref = product(moe, x, w)
    x[4, 100], x[9, 3] = float("nan"), float("inf")
    y = product(moe, x, w)
    keep = [r for r in range(12) if r not in (4, 9)]
    assert torch.equal(y[keep], ref[keep])
    assert bool(torch.isnan(y[4]).all())


def expert_case(moe, T, E, K, m, Kd, N, group, dtype, zeros, cap=None, seed=0, empty=()):
    r = np.random.default_rng(seed)
    score = r.standard_normal((T, E))
    score[:, list(empty)] = -9.0
    ids = np.sort(np.argsort(-score, axis=1)[:, :K], axis=1).astype(np.int16)
    full = T * K + E * (m - 1)
    cap = full if cap is None else cap
    shape, layout = moe.Shape(T, Kd, E, K), moe.Layout(m, cap)
    h = moe.Handle.empty(shape, layout)
    ws = torch.empty(moe.moe_preprocess_workspace_size(shape), dtype=torch.uint8, device="cuda")
    moe.moe_preprocess(moe.Routing(0, torch.from_numpy(ids).cuda()), shape, layout, h, ws)
    codes, scales, zp = bu.w4_random(N, Kd, group, dtype, zeros, seed, (E,))
    x = bu.randn(cap, Kd, seed=seed + 1, dtype=dtype)
    return shape, layout, h, (codes, scales, zp), x


@pytest.mark.parametrize("T,E,K,m,Kd,N,group,swiglu", [
    (1, 8, 2, 32, 128, 64, 128, True), (1, 300, 8, 1, 256, 48, 64, False), (5, 4, 4, 8, 384, 34, 128, True),
    (40, 16, 3, 32, 256, 100, 32, True), (64, 256, 8, 4, 128, 32, 128, False), (100, 3, 2, 1, 160, 50, 64, False),
    (7, 1024, 16, 1, 64, 18, 32, True), (2, 33, 1, 16, 1024, 130, 128, True)])
def test_experts(T, E, K, m, Kd, N, group, swiglu):
    moe = moe_mod()
    for dtype, zeros in ((BF, False), (HF, True)):
        shape, layout, h, w, x = expert_case(moe, T, E, K, m, Kd, N, group, dtype, zeros, empty=(0,) if E > K else ())
        n_out = N // 2 if swiglu else N
        y = torch.full((layout.capacity, n_out), 5.0, dtype=dtype, device="cuda")
        moe.moe_grouped_w4_matvec(h, shape, layout, moe.W4Weight(*(dev(t) for t in w), group), x.cuda(), y,
                                  moe.W4_SWIGLU if swiglu else moe.W4_NONE)
        counts, off = h.tokens_per_expert.cpu().numpy(), h.padded_offsets.cpu().numpy()
        routed = torch.zeros(layout.capacity, dtype=torch.bool)
        for e in range(E):
            if not counts[e]:
                continue
            s = slice(int(off[e]), int(off[e] + counts[e]))
            routed[s] = True
            W = bu.w4_dequant(*(t if t is None else t[e] for t in w), group)
            ref, tol = bu.w4_product(x[s], W, group, swiglu=swiglu, dtype=dtype)
            bu.assert_within(y[s], ref, tol, f"expert {e}")
        assert bool((y.cpu()[~routed] == 5.0).all())  # pad rows and rows beyond the segments are left alone


@pytest.mark.parametrize("cut", [0, 1, 17, 40])
def test_experts_below_the_capacity(cut):
    """Rows at or beyond the capacity are neither read nor written: the capacity cuts a segment, or leaves none."""
    moe = moe_mod()
    T, E, K, m, Kd, N = 30, 4, 2, 8, 128, 40
    shape, layout, h, w, x = expert_case(moe, T, E, K, m, Kd, N, 64, BF, True)
    weight = moe.W4Weight(*(dev(t) for t in w), 64)
    y = torch.zeros(layout.capacity, N, dtype=BF, device="cuda")
    moe.moe_grouped_w4_matvec(h, shape, layout, weight, x.cuda(), y)
    cl = moe.Layout(m, cut)
    short = torch.full((layout.capacity, N), 7.0, dtype=BF, device="cuda")
    moe.moe_grouped_w4_matvec(h, shape, cl, weight, x.cuda()[:cut], short[:cut])
    off = h.padded_offsets.cpu().numpy()
    cnt = h.tokens_per_expert.cpu().numpy()
    routed = np.zeros(layout.capacity, bool)
    for e in range(E):
        routed[off[e]:off[e] + cnt[e]] = True
    routed[cut:] = False
    r = torch.from_numpy(routed).cuda()
    assert torch.equal(short[r], y[r]) and bool((short[~r] == 7.0).all())


@pytest.mark.parametrize("T", [1, 30])
def test_experts_of_a_damaged_handle(T):
    """A segment that begins before the rows, or has no rows, is left out; the other experts' rows are as ever."""
    moe = moe_mod()
    E, K, Kd, N = 40, 2, 128, 40
    shape, layout, h, w, x = expert_case(moe, T, E, K, 8, Kd, N, 64, BF, True)
    weight = moe.W4Weight(*(dev(t) for t in w), 64)
    y = torch.full((layout.capacity, N), 7.0, dtype=BF, device="cuda")
    moe.moe_grouped_w4_matvec(h, shape, layout, weight, x.cuda(), y)
    off, cnt = h.padded_offsets.cpu().numpy(), h.tokens_per_expert.cpu().numpy()
    some = [int(e) for e in np.nonzero(cnt)[0][:2]]
    h.padded_offsets[some[0]] = -3
    h.tokens_per_expert[some[1]] = -(1 << 31)
    got = torch.full_like(y, 7.0)
    moe.moe_grouped_w4_matvec(h, shape, layout, weight, x.cuda(), got)
    for e in some:
        y[off[e]:off[e] + cnt[e]] = 7.0
    assert torch.equal(got, y)


def test_experts_equal_single_matrices():
    """An expert's rows are those of moe_w4_matvec with its matrix: both within the bounds of the definition."""
    moe = moe_mod()
    shape, layout, h, w, x = expert_case(moe, 6, 5, 2, 1, 512, 64, 128, BF, False)
    y = torch.zeros(layout.capacity, 64, dtype=BF, device="cuda")
    moe.moe_grouped_w4_matvec(h, shape, layout, moe.W4Weight(dev(w[0]), dev(w[1]), None, 128), x.cuda(), y)
    off, cnt = h.padded_offsets.cpu().numpy(), h.tokens_per_expert.cpu().numpy()
    for e in range(5):
        if cnt[e]:
            s = slice(int(off[e]), int(off[e] + cnt[e]))
            ref, tol = bu.w4_product(x[s], bu.w4_dequant(w[0][e], w[1][e], None, 128), 128)
            a = product(moe, x[s], (w[0][e], w[1][e], None))
            bu.assert_within(a, ref, tol)
            bu.assert_within(y[s], ref, tol)


def quantize_ref(w, group, zeros):
    """The quantizer's definition in numpy fp32 (rows [R][Kd] of a 16-bit type)."""
    R, Kd = w.shape
    G = -(-Kd // group)
    q, s, z = np.zeros((R, Kd), np.uint8), torch.zeros(R, G, dtype=w.dtype), np.full((R, G), 8, np.uint8)
    f = w.float().numpy()
    for g in range(G):
        v = f[:, g * group:(g + 1) * group]
        lo, hi = np.minimum(v.min(1), 0), np.maximum(v.max(1), 0)
        span = (hi - lo) / np.float32(15) if zeros else np.maximum(hi, -lo) / np.float32(7)
        st = torch.from_numpy(span.astype(np.float32)).to(w.dtype)
        st[st == 0] = 1.0
        s[:, g] = st
        sf = st.float().numpy()
        if zeros:
            z[:, g] = np.clip(np.rint(-lo / sf), 0, 15)
        q[:, g * group:(g + 1) * group] = np.clip(np.rint(v / sf[:, None]) + z[:, g:g + 1], 0, 15)
    codes = q[:, 0::2] | (q[:, 1::2] << 4)
    zp = np.zeros((R, (G + 1) // 2 * 2), np.uint8)
    zp[:, :G] = z
    return codes, s, zp[:, 0::2] | (zp[:, 1::2] << 4)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("R,Kd,group", [(1, 32, 32), (5, 96, 64), (9, 544, 128), (40, 256, 32), (3, 4096, 64)])
def test_quantizer_bit_exact(R, Kd, group, dtype):
    moe = moe_mod()
    w = bu.randn(R, Kd, seed=R, scale=0.02, dtype=dtype)
    w[0, :16] = 0
    if R > 2:
        w[1] = 0
        w[2] = w[2].abs() + 0.01
    G = -(-Kd // group)
    for zeros in (False, True):
        codes = torch.full((R, Kd // 2), 255, dtype=torch.uint8, device="cuda")
        scales = torch.empty(R, G, dtype=dtype, device="cuda")
        zp = torch.full((R, (G + 1) // 2), 255, dtype=torch.uint8, device="cuda") if zeros else None
        moe.moe_quantize_w4_rows(w.cuda(), group, codes, scales, zp)
        rc, rs, rz = quantize_ref(w, group, zeros)
        assert torch.equal(scales.cpu(), rs) and np.array_equal(codes.cpu().numpy(), rc)
        if zeros:
            assert np.array_equal(zp.cpu().numpy(), rz)


def test_zero_tokens():
    moe = moe_mod()
    w = bu.w4_random(16, 64, 32, BF, False, seed=0)
    weight = moe.W4Weight(dev(w[0]), dev(w[1]), None, 32)
    moe.moe_w4_matvec(weight, torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, 16, dtype=BF, device="cuda"))


def test_refusals():
    moe = moe_mod()
    codes, scales, zeros = (dev(t) for t in bu.w4_random(16, 256, 64, BF, True, seed=0))
    x, y = torch.zeros(2, 256, dtype=BF, device="cuda"), torch.empty(2, 16, dtype=BF, device="cuda")
    good = moe.W4Weight(codes, scales, zeros, 64)
    with pytest.raises(ValueError):  # scales of another group size
        moe.moe_w4_matvec(moe.W4Weight(codes, scales, zeros, 32), x, y)
    with pytest.raises(ValueError):
        moe.moe_w4_matvec(moe.W4Weight(codes.int(), scales, zeros, 64), x, y)
    with pytest.raises(ValueError):
        moe.moe_w4_matvec(good, x.half(), y)
    with pytest.raises(ValueError):
        moe.moe_w4_matvec(good, x[:, :128], y)
    with pytest.raises(ValueError):
        moe.moe_w4_matvec(good, x, y, addend=y[:1])
    with pytest.raises(moe.MoeError):  # fp32 scales
        moe.moe_w4_matvec(moe.W4Weight(codes, scales.float(), zeros, 64), x.float(), y.float())
    with pytest.raises(moe.MoeError):  # a group size that is not built
        moe.moe_w4_matvec(moe.W4Weight(codes, scales[:, :1].contiguous(), None, 256), x, y)
    with pytest.raises(moe.MoeError):
        moe.moe_w4_matvec(good, x, y, activation=5)
    with pytest.raises(moe.MoeError):  # an addend after SwiGLU
        moe.moe_w4_matvec(good, x, y[:, :8], moe.W4_SWIGLU, addend=torch.empty(2, 8, dtype=BF, device="cuda"))
    odd = moe.W4Weight(codes[:15], scales[:15], zeros[:15], 64)
    with pytest.raises(moe.MoeError):  # SwiGLU of an odd number of rows
        moe.moe_w4_matvec(odd, x, torch.empty(2, 7, dtype=BF, device="cuda"), moe.W4_SWIGLU)
    wide = torch.zeros(2, 300, dtype=BF, device="cuda")
    with pytest.raises(moe.MoeError):  # rows that are not 16-byte aligned
        moe.moe_w4_matvec(good, wide[:, 1:257], y)
    with pytest.raises(moe.MoeError):
        moe.moe_w4_matvec(good, torch.zeros(2, 257, dtype=BF, device="cuda")[:, :256], y)
    with pytest.raises(moe.MoeError):  # y over x
        moe.moe_w4_matvec(good, x, x[:, :16])
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_w4_rows(x, 48, torch.empty(2, 128, dtype=torch.uint8, device="cuda"),
                                 torch.empty(2, 6, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_quantize_w4_rows(x.float(), 64, codes[:2], scales[:2])
