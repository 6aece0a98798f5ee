"""Products grouped by expert on the GPU (forward, gradient of the rows, gradient of the weights) against their
64-bit definition, and on small whole numbers, whose sums are exact in fp32 in any order, bit for bit."""
import numpy as np
import pytest
import torch

import block_util as bu
import train_util as tu
from gpu_util import moe_mod
from train_util import BF, HF, F32

pytestmark = pytest.mark.gpu

# (T, E, K, m, N, Kd): one token to several tiles of rows; widths of one element, odd, of a tile, of several
SIZES = [(1, 1, 1, 1, 1, 1), (1, 8, 2, 32, 128, 64), (3, 4, 2, 8, 33, 65), (5, 300, 8, 1, 48, 40), (40, 3, 2, 32, 256, 128),
         (7, 16, 4, 1, 264, 72), (64, 2, 1, 8, 512, 256), (130, 5, 3, 4, 136, 1000), (300, 2, 2, 1, 320, 192),
         (100, 7, 3, 16, 1001, 77), (700, 3, 1, 32, 128, 520), (33, 1024, 1, 1, 64, 64), (257, 1, 1, 1, 640, 384),
         (513, 4, 4, 32, 256, 256), (1100, 1, 1, 1, 72, 136)]


def matrices(E, N, Kd, dtype, seed, ints=None):
    g = torch.Generator().manual_seed(seed)
    if ints is not None:
        return torch.randint(-ints, ints + 1, (E, N, Kd), generator=g).to(dtype)
    return (torch.randn(E, N, Kd, generator=g) * Kd ** -0.5).to(dtype)


def forward(moe, r, w, x):
    y = torch.full((r.cap, w.shape[1]), 7.0, dtype=w.dtype, device="cuda")
    moe.moe_grouped_gemm(r.handle, r.shape, r.layout, w.cuda(), x.cuda(), y, tu.workspace(moe, r, *w.shape[1:]))
    torch.cuda.synchronize()
    return y


def data(moe, r, w, gy):
    gx = torch.full((r.cap, w.shape[2]), 7.0, dtype=w.dtype, device="cuda")
    moe.moe_grouped_gemm_backward_data(r.handle, r.shape, r.layout, w.cuda(), gy.cuda(), gx,
                                       tu.workspace(moe, r, *w.shape[1:]))
    torch.cuda.synchronize()
    return gx


def weight(moe, r, gy, x, out_dtype, addend=None):
    N, Kd = gy.shape[1], x.shape[1]
    gw = torch.full((r.shape.E, N, Kd), float("nan"), dtype=out_dtype, device="cuda")
    moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, x.cuda(), gy.cuda(), gw,
                                         tu.workspace(moe, r, N, Kd), None if addend is None else addend.cuda())
    torch.cuda.synchronize()
    return gw


def assert_rows(r, got, ref, tol=None):
    got = got.cpu()
    assert bool((got[~r.routed] == 7.0).all()), "rows outside the segments were written"
    if tol is None:
        assert torch.equal(got[r.routed], ref[r.routed].to(got.dtype))
    else:
        bu.assert_within(got[r.routed], ref[r.routed], tol[r.routed])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,E,K,m,N,Kd", SIZES)
def test_whole_numbers(T, E, K, m, N, Kd, dtype):
    """Sums of products of whole numbers up to 2 stay below 2^24: every result is the exact sum, rounded once."""
    moe = moe_mod()
    r = tu.Routed(moe, T, E, K, m, empty=(0,) if E > K else ())
    w = matrices(E, N, Kd, dtype, 1, ints=2)
    x, gy = r.rows(Kd, dtype, 2, ints=2), r.rows(N, dtype, 3, ints=2)
    assert_rows(r, forward(moe, r, w, x), tu.gemm_forward(r, w, x))
    assert_rows(r, data(moe, r, w, gy), tu.gemm_data(r, w, gy))
    gw = tu.gemm_weight(r, gy, x)
    assert torch.equal(weight(moe, r, gy, x, dtype).cpu(), gw.to(dtype))
    assert torch.equal(weight(moe, r, gy, x, F32).cpu(), gw.float())


@pytest.mark.parametrize("T,E,K,m,N,Kd,skew", [(3000, 16, 4, 32, 1024, 512, 0.0), (2500, 3, 1, 8, 2312, 328, 0.0),
                                               (5000, 40, 2, 1, 520, 264, 1.2)])
def test_more_tiles_than_run_at_once(T, E, K, m, N, Kd, skew):
    moe = moe_mod()
    r = tu.Routed(moe, T, E, K, m, skew=skew)
    w = matrices(E, N, Kd, BF, 1, ints=2)
    x, gy = r.rows(Kd, BF, 2, ints=2), r.rows(N, BF, 3, ints=2)
    assert_rows(r, forward(moe, r, w, x), tu.gemm_forward(r, w, x))
    assert_rows(r, data(moe, r, w, gy), tu.gemm_data(r, w, gy))
    gw = tu.gemm_weight(r, gy, x)
    assert torch.equal(weight(moe, r, gy, x, BF).cpu(), gw.to(BF))
    assert torch.equal(weight(moe, r, gy, x, F32).cpu(), gw.float())


@pytest.mark.parametrize("T,E,K,m,N,Kd,skew,empty", [(3000, 16, 4, 32, 1025, 513, 0.0, (5,)), (2500, 3, 1, 8, 2311, 329, 0.0, ()),
                                                     (5000, 40, 2, 1, 521, 265, 1.2, (0, 39)), (9000, 7, 1, 1, 1537, 1001, 0.0, (3,)),
                                                     (2000, 200, 3, 4, 515, 259, 0.5, (7, 8))])
def test_unaligned_more_tiles_than_run_at_once(T, E, K, m, N, Kd, skew, empty):
    """Operands shifted into place in several tiles of each pair of SMs, some dealt from the counter: odd and even numbers
    of stages a tile, so that every ring goes on in the next tile where it stood, and experts without rows between."""
    moe = moe_mod()
    r = tu.Routed(moe, T, E, K, m, skew=skew, empty=empty)
    w = matrices(E, N, Kd, BF, 1, ints=2)
    x, gy = r.rows(Kd, BF, 2, ints=2), r.rows(N, BF, 3, ints=2)
    assert_rows(r, forward(moe, r, w, x), tu.gemm_forward(r, w, x))
    assert_rows(r, data(moe, r, w, gy), tu.gemm_data(r, w, gy))
    gw = tu.gemm_weight(r, gy, x)
    assert torch.equal(weight(moe, r, gy, x, BF).cpu(), gw.to(BF))
    assert torch.equal(weight(moe, r, gy, x, F32).cpu(), gw.float())
    assert int(r.handle.status.item()) == 0


@pytest.mark.parametrize("N,Kd", [(128, 64), (264, 136), (320, 520), (65, 33)])
def test_every_length_of_an_expert(N, Kd):
    """Experts of 0 to 150 rows, with and without pad rows between (NaN in all of those): every number of rows in the last
    stage along an expert's rows, the buffer's first rows and its last ones among them."""
    moe = moe_mod()
    E = 151
    counts, pads = np.arange(E)[::-1].copy(), np.arange(E) % 3
    counts[0], counts[-1] = 1, 37  # the first rows, and the last ones of the buffer
    pads[-1] = 0
    r = tu.Routed(moe, int(counts.sum()) + 8, E, 1, 2)
    off = np.concatenate([[0], np.cumsum(counts + pads)]).astype(np.int32)
    r.cap = int(off[-1])
    r.layout = moe.Layout(1, r.cap)
    r.handle.padded_offsets.copy_(torch.from_numpy(off))
    r.handle.tokens_per_expert.copy_(torch.from_numpy(counts.astype(np.int32)))
    r.segments = [(e, int(off[e]), int(off[e] + counts[e])) for e in range(E)]
    r.routed = torch.zeros(r.cap, dtype=torch.bool)
    for _, b, n in r.segments:
        r.routed[b:n] = True
    w = matrices(E, N, Kd, BF, 1, ints=2)
    x, gy = r.rows(Kd, BF, 2, ints=2), r.rows(N, BF, 3, ints=2)
    gw = tu.gemm_weight(r, gy, x)
    assert torch.equal(weight(moe, r, gy, x, F32).cpu(), gw.float())
    assert torch.equal(weight(moe, r, gy, x, BF).cpu(), gw.to(BF))
    assert_rows(r, forward(moe, r, w, x), tu.gemm_forward(r, w, x))
    assert_rows(r, data(moe, r, w, gy), tu.gemm_data(r, w, gy))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,E,K,m,N,Kd", [(1, 8, 2, 32, 264, 2048), (50, 6, 2, 8, 384, 512), (333, 4, 2, 1, 129, 257),
                                          (900, 2, 1, 32, 256, 640)])
def test_against_64_bits(T, E, K, m, N, Kd, dtype):
    moe = moe_mod()
    r = tu.Routed(moe, T, E, K, m, seed=4, skew=0.5)
    w = matrices(E, N, Kd, dtype, 5)
    x, gy = r.rows(Kd, dtype, 6), r.rows(N, dtype, 7)
    ref = tu.gemm_forward(r, w, x)
    assert_rows(r, forward(moe, r, w, x), ref, tu.gemm_tol(ref, tu.gemm_forward(r, w.abs(), x.abs()), Kd, dtype))
    ref = tu.gemm_data(r, w, gy)
    assert_rows(r, data(moe, r, w, gy), ref, tu.gemm_tol(ref, tu.gemm_data(r, w.abs(), gy.abs()), N, dtype))
    ref, most = tu.gemm_weight(r, gy, x), tu.gemm_weight(r, gy.abs(), x.abs())
    rows = max(n - b for _, b, n in r.segments)
    for out in (dtype, F32):
        bu.assert_within(weight(moe, r, gy, x, out), ref, tu.gemm_tol(ref, most, rows, out))


@pytest.mark.parametrize("N,Kd", [(256, 192), (65, 130)])
@pytest.mark.parametrize("rows", [700, 769, 6000])
def test_long_sums(rows, N, Kd):
    """fp32 gradients of many rows. An addition inside the tensor cores cuts at most 2^-23 off the sum so far, whose mean
    square grows in proportion to the rows, so that 48 steps of 16 rows are off by 48 * 2/3 * 2^-23 = 3.8e-6 of their sum
    at the most; parts of that length are joined by roundings of 2^-24. One sum of 6000 rows could be 3e-5 off."""
    moe = moe_mod()
    r = tu.Routed(moe, rows, 1, 1, 1)
    x, gy = r.rows(Kd, BF, 1), r.rows(N, BF, 2)
    ref = tu.gemm_weight(r, gy, x)
    got = weight(moe, r, gy, x, F32)
    assert float((bu.f64(got) - ref).norm() / ref.norm()) <= 48 * 2 / 3 * 2.0 ** -23 + 8 * 2.0 ** -24
    add = torch.randn(1, N, Kd, generator=torch.Generator().manual_seed(3)) * 100
    both = weight(moe, r, gy, x, F32, add)
    assert float((bu.f64(both) - ref - add).norm() / ref.norm()) <= 5e-6 + 8 * 2.0 ** -24 * float(add.norm() / ref.norm())
    assert all(torch.equal(weight(moe, r, gy, x, F32, add), both) for _ in range(3))


def one_expert(moe, rows):
    """A routing of `rows` rows of one expert, without the arrays that the products do not read."""
    r = tu.Routed(moe, 8, 1, 1, 1)
    r.cap, r.shape, r.layout = rows, moe.Shape(rows, 128, 1, 1), moe.Layout(1, rows)
    r.handle.padded_offsets.copy_(torch.tensor([0, rows], dtype=torch.int32))
    r.handle.tokens_per_expert.fill_(rows)
    return r


def positive(rows, cols, dtype, seed, long_rows):
    """Numbers between 2^-5 and 2^-3, with a scale of its own for each line that is summed along: sums as wide apart as
    a power of two, so that their roundings to 16 bits are spread evenly."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand(rows, cols, generator=g, device="cuda") * 0.5 + 0.5
    line = torch.exp2(torch.rand(rows if long_rows else cols, generator=g, device="cuda"))
    return (u * (line[:, None] if long_rows else line[None]) * 2.0 ** -4).to(dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,few,cols", [(1 << 20, 24, 40), ((1 << 20) - 1, 19, 33), (40000, 300, 264)])
def test_long_sums_in_16_bits(n, few, cols, dtype):
    """Sums of n numbers of one sign, rounded to 16 bits once: parts of 8192, each addition inside the tensor cores cutting
    at most 2^-23 off the part's sum so far, which is half the part on average, so that 2^-11 of the result may be
    missing; up to 128 parts are joined by roundings of 2^-24, half of which reach the whole sum. The mean over the
    results has that bound without their own rounding, up to four of its standard deviations. (One sum of 2^20 may be
    short by 2^-4 by the same bound, and was by 2^-7.)"""
    moe = moe_mod()
    short = 2.0 ** -11 + 64 * 2.0 ** -24

    def check(got, ref):
        assert bool(((bu.f64(got) - bu.f64(ref)).abs() <= short * bu.f64(ref) + bu.rounding(bu.f64(ref), dtype)).all())
        rel = (got.double() / ref - 1).mean().abs().item()
        assert rel <= short + 4 * torch.finfo(dtype).eps / 2 / 3 ** 0.5 / ref.numel() ** 0.5, rel

    r = one_expert(moe, n)  # the weights' gradient, along n rows
    x, gy = positive(n, cols, dtype, 1, False), positive(n, few, dtype, 2, False)
    gw = torch.empty(1, few, cols, dtype=dtype, device="cuda")
    ws = tu.workspace(moe, r, few, cols)
    moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, x, gy, gw, ws)
    check(gw[0], gy.double().T @ x.double())
    r = one_expert(moe, few)
    x, w = positive(few, n, dtype, 3, True), positive(cols, n, dtype, 4, True)[None]
    y = torch.empty(few, cols, dtype=dtype, device="cuda")
    moe.moe_grouped_gemm(r.handle, r.shape, r.layout, w, x, y, ws)
    check(y, x.double() @ w[0].double().T)
    w = w[0].T.contiguous()[None]
    moe.moe_grouped_gemm_backward_data(r.handle, r.shape, r.layout, w, x, y, ws)
    check(y, x.double() @ w[0].double())


@pytest.mark.parametrize("rows,wide,n", [(600, 8192, 33000), (600, 8191, 33001), (300, 20000, 16385), (40, 19000, 49160)])
def test_long_sums_of_more_tiles_than_run_at_once(rows, wide, n):
    """Sums in three to seven parts, of several tiles a pair of SMs, on whole numbers: parts joined beside the next tile."""
    moe = moe_mod()
    g = torch.Generator(device="cuda").manual_seed(1)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(BF)
    times = lambda a, b: (a.float() @ b.float()).to(BF)  # whole numbers below 2^24: exact in any order
    r = one_expert(moe, rows)
    ws = tu.workspace(moe, r, wide, n)
    w, x, y = ints(1, wide, n), ints(rows, n), torch.empty(rows, wide, dtype=BF, device="cuda")
    moe.moe_grouped_gemm(r.handle, r.shape, r.layout, w, x, y, ws)
    assert torch.equal(y, times(x, w[0].T))
    w = w[0].T.contiguous()[None]
    moe.moe_grouped_gemm_backward_data(r.handle, r.shape, r.layout, w, x, y, ws)
    assert torch.equal(y, times(x, w[0]))
    del w, x, y
    r = one_expert(moe, n)
    x, gy = ints(n, 2056 + wide % 2), ints(n, 2312 + wide % 2)
    gw = torch.empty(1, gy.shape[1], x.shape[1], dtype=BF, device="cuda")
    moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, x, gy, gw, ws)
    assert torch.equal(gw[0], times(gy.T, x))


@pytest.mark.parametrize("N,Kd", [(128, 192), (264, 136), (33, 50)])
def test_addend(N, Kd):
    """The addend joins the fp32 sum; it may be the gradient itself, which then gathers several calls."""
    moe = moe_mod()
    r = tu.Routed(moe, 60, 5, 2, 8, empty=(1,))
    x, gy = r.rows(Kd, BF, 1, ints=2), r.rows(N, BF, 2, ints=2)
    add = torch.randint(-9, 10, (5, N, Kd), generator=torch.Generator().manual_seed(3)).float()
    ref = tu.gemm_weight(r, gy, x)
    assert torch.equal(weight(moe, r, gy, x, F32, add).cpu(), (ref + add).float())
    gw = add.cuda()
    ws = tu.workspace(moe, r, N, Kd)
    for _ in range(3):
        moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, x.cuda(), gy.cuda(), gw, ws, gw)
    assert torch.equal(gw.cpu(), (3 * ref + add).float())


@pytest.mark.parametrize("N,Kd", [(128, 128), (72, 41)])
@pytest.mark.parametrize("cut", [0, 1, 17, 70])
def test_below_the_capacity(cut, N, Kd):
    """Rows at or beyond the capacity are neither read nor written, and take no part in the weights' gradient."""
    moe = moe_mod()
    r = tu.Routed(moe, 50, 4, 2, 8, cap=cut, seed=3)
    w = matrices(4, N, Kd, BF, 1, ints=2)
    x, gy = r.rows(Kd, BF, 2, ints=2), r.rows(N, BF, 3, ints=2)
    assert_rows(r, forward(moe, r, w, x), tu.gemm_forward(r, w, x))
    assert_rows(r, data(moe, r, w, gy), tu.gemm_data(r, w, gy))
    assert torch.equal(weight(moe, r, gy, x, F32).cpu(), tu.gemm_weight(r, gy, x).float())


@pytest.mark.parametrize("N,Kd", [(128, 256), (40, 24)])
def test_no_tokens(N, Kd):
    moe = moe_mod()
    r = tu.Routed(moe, 0, 3, 1, 8)
    w = matrices(3, N, Kd, BF, 1)
    forward(moe, r, w, torch.full((r.cap, Kd), float("nan"), dtype=BF))
    data(moe, r, w, torch.full((r.cap, N), float("nan"), dtype=BF))
    nan = lambda c: torch.full((r.cap, c), float("nan"), dtype=BF)
    assert bool((weight(moe, r, nan(N), nan(Kd), F32) == 0).all())
    add = matrices(3, N, Kd, F32, 2)
    assert torch.equal(weight(moe, r, nan(N), nan(Kd), F32, add).cpu(), add)


@pytest.mark.parametrize("N,Kd,pad,shift", [(128, 192, 8, 8), (128, 192, 64, 0), (128, 192, 1, 0), (136, 72, 3, 5),
                                            (65, 31, 7, 1)])
def test_strides_and_alignment(N, Kd, pad, shift):
    moe = moe_mod()
    r = tu.Routed(moe, 90, 3, 2, 4)
    w = matrices(3, N, Kd, HF, 1, ints=2)
    x, gy = r.rows(Kd, HF, 2, ints=2), r.rows(N, HF, 3, ints=2)

    def apart(t):
        buf = torch.full((r.cap, t.shape[1] + pad + shift), 9.0, dtype=HF, device="cuda")
        v = buf[:, shift:shift + t.shape[1]]
        v.copy_(t)
        return buf, v

    def outside(buf, cols):
        assert bool((buf[:, :shift] == 9.0).all()) and bool((buf[:, shift + cols:] == 9.0).all())

    # the weights one element off their allocation's alignment where rows are off too
    store = torch.zeros(w.numel() + 8, dtype=HF, device="cuda")
    wv = store[shift % 8:][:w.numel()].view_as(w)
    wv.copy_(w)
    xv, gv = apart(x)[1], apart(gy)[1]
    ws = tu.workspace(moe, r, N, Kd)
    yb, yv = apart(torch.full((r.cap, N), 7.0))
    moe.moe_grouped_gemm(r.handle, r.shape, r.layout, wv, xv, yv, ws)
    assert_rows(r, yv, tu.gemm_forward(r, w, x))
    outside(yb, N)
    gb, gxv = apart(torch.full((r.cap, Kd), 7.0))
    moe.moe_grouped_gemm_backward_data(r.handle, r.shape, r.layout, wv, gv, gxv, ws)
    assert_rows(r, gxv, tu.gemm_data(r, w, gy))
    outside(gb, Kd)
    gw = torch.empty(3, N, Kd, device="cuda")
    moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, xv, gv, gw, ws)
    assert torch.equal(gw.cpu(), tu.gemm_weight(r, gy, x).float())


@pytest.mark.parametrize("N,Kd,stride", [(136, 72, 1 << 25), (33, 17, (1 << 25) + 1)])
def test_offsets_beyond_32_bits(N, Kd, stride):
    """Rows so far apart that their offsets pass 2^31 elements, 2^32 bytes."""
    moe = moe_mod()
    r = tu.Routed(moe, 40, 2, 2, 8)
    w, x, gy = matrices(2, N, Kd, BF, 1, ints=2), r.rows(Kd, BF, 2, ints=2), r.rows(N, BF, 3, ints=2)
    assert (r.cap - 8) * stride > 1 << 31

    def apart(t):
        v = torch.empty((r.cap - 1) * stride + t.shape[1], dtype=BF, device="cuda").as_strided(t.shape, (stride, 1))
        return v.copy_(t)

    xd, gd, ws = apart(x), apart(gy), tu.workspace(moe, r, N, Kd)
    y, gw = apart(torch.full((r.cap, N), 7.0)), torch.empty(2, N, Kd, device="cuda")
    moe.moe_grouped_gemm(r.handle, r.shape, r.layout, w.cuda(), xd, y, ws)
    assert_rows(r, y, tu.gemm_forward(r, w, x))
    moe.moe_grouped_gemm_backward_data(r.handle, r.shape, r.layout, w.cuda(), gd, xd.fill_(7.0), ws)
    assert_rows(r, xd, tu.gemm_data(r, w, gy))
    moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, xd.copy_(x), gd, gw, ws)
    assert torch.equal(gw.cpu(), tu.gemm_weight(r, gy, x).float())


@pytest.mark.parametrize("N,Kd", [(256, 128), (77, 50)])
def test_nonfinite_rows_and_weights_stay_alone(N, Kd):
    moe = moe_mod()
    r = tu.Routed(moe, 80, 4, 2, 8, seed=1)
    w, x, gy = matrices(4, N, Kd, BF, 1), r.rows(Kd, BF, 2), r.rows(N, BF, 3)
    seg = [(e, b, n) for e, b, n in r.segments if n - b > 4]
    (e0, b0, _), (e1, b1, n1) = seg[0], seg[1]
    y, gx, gw = forward(moe, r, w, x), data(moe, r, w, gy), weight(moe, r, gy, x, F32)
    bad_x, bad_g, bad_w = x.clone(), gy.clone(), w.clone()
    bad_x[b0 + 2, 1], bad_g[b0 + 2, 3] = float("nan"), float("inf")
    bad_w[e1, N - 1, Kd - 1] = float("nan")
    keep = r.routed.clone()
    keep[b0 + 2] = False
    keep[b1:n1] = False
    keep = keep.cuda()
    ny, ng = forward(moe, r, bad_w, bad_x), data(moe, r, bad_w, bad_g)
    assert torch.equal(ny[keep], y[keep]) and torch.equal(ng[keep], gx[keep])
    assert bool(torch.isnan(ny[b0 + 2]).all()) and bool(torch.isnan(ny[b1:n1, N - 1]).all())
    assert torch.equal(ny[b1:n1, :N - 1], y[b1:n1, :N - 1])
    assert bool(torch.isnan(ng[b1:n1, Kd - 1]).all()) and torch.equal(ng[b1:n1, :Kd - 1], gx[b1:n1, :Kd - 1])
    nw = weight(moe, r, bad_g, bad_x, F32)
    others = [e for e in range(4) if e != e0]
    assert torch.equal(nw[others], gw[others])
    assert bool(torch.isnan(nw[e0][:, 1]).all()) and not bool(torch.isfinite(nw[e0][3]).any())


def test_repeated_calls_agree():
    moe = moe_mod()
    r = tu.Routed(moe, 500, 8, 3, 32, skew=1.0)
    w, x, gy = matrices(8, 384, 320, BF, 1), r.rows(320, BF, 2), r.rows(384, BF, 3)
    first = forward(moe, r, w, x), data(moe, r, w, gy), weight(moe, r, gy, x, F32)
    for _ in range(5):
        again = forward(moe, r, w, x), data(moe, r, w, gy), weight(moe, r, gy, x, F32)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("N,Kd", [(128, 128), (30, 24)])
def test_a_damaged_handle(N, Kd):
    """A segment that begins before the rows, or has no rows, is left out; the other experts are as ever."""
    moe = moe_mod()
    r = tu.Routed(moe, 60, 6, 2, 8)
    w, x, gy = matrices(6, N, Kd, BF, 1), r.rows(Kd, BF, 2), r.rows(N, BF, 3)
    y, gw = forward(moe, r, w, x), weight(moe, r, gy, x, F32)
    some = [e for e, b, n in r.segments if n > b][:2]
    r.handle.padded_offsets[some[0]] = -3
    r.handle.tokens_per_expert[some[1]] = -(1 << 31)
    for e, b, n in r.segments:
        if e in some:
            y[b:n] = 7.0
            gw[e] = 0.0
    assert torch.equal(forward(moe, r, w, x), y)
    assert torch.equal(weight(moe, r, gy, x, F32), gw)


@pytest.mark.parametrize("N,Kd", [(136, 72), (33, 50)])
@pytest.mark.parametrize("T", [1, 20, 150])
def test_a_handle_of_more_tokens_than_the_shape(T, N, Kd):
    """Each expert's rows end after as many as the shape has routes."""
    moe = moe_mod()
    r = tu.Routed(moe, 600, 4, 2, 8)
    w, x, gy = matrices(4, N, Kd, BF, 1, ints=2), r.rows(Kd, BF, 2, ints=2), r.rows(N, BF, 3, ints=2)
    r.shape = moe.Shape(T, 128, 4, 2)
    r.segments = [(e, b, min(n, b + 2 * T)) for e, b, n in r.segments]
    r.routed = torch.zeros(r.cap, dtype=torch.bool)
    for e, b, n in r.segments:
        r.routed[b:n] = True
    assert_rows(r, forward(moe, r, w, x), tu.gemm_forward(r, w, x))
    assert_rows(r, data(moe, r, w, gy), tu.gemm_data(r, w, gy))
    assert torch.equal(weight(moe, r, gy, x, F32).cpu(), tu.gemm_weight(r, gy, x).float())


def test_streams_and_graphs():
    """Captured and replayed with other inputs and another routing, and on a stream of its own."""
    moe = moe_mod()
    T, E, K, m, N, Kd = 120, 6, 2, 8, 256, 192
    a, b = tu.Routed(moe, T, E, K, m, seed=1), tu.Routed(moe, T, E, K, m, seed=2)
    w = matrices(E, N, Kd, BF, 1, ints=2)
    xs, gs = [t.rows(Kd, BF, 3, ints=2) for t in (a, b)], [t.rows(N, BF, 4, ints=2) for t in (a, b)]
    live = tu.Routed(moe, T, E, K, m, seed=1)
    wd, x, gy = w.cuda(), xs[0].cuda(), gs[0].cuda()
    y = torch.zeros(a.cap, N, dtype=BF, device="cuda")
    gx = torch.zeros(a.cap, Kd, dtype=BF, device="cuda")
    gw = torch.zeros(E, N, Kd, device="cuda")
    ws = tu.workspace(moe, a, N, Kd)

    def calls():
        moe.moe_grouped_gemm(live.handle, a.shape, a.layout, wd, x, y, ws)
        moe.moe_grouped_gemm_backward_data(live.handle, a.shape, a.layout, wd, gy, gx, ws)
        moe.moe_grouped_gemm_backward_weight(live.handle, a.shape, a.layout, x, gy, gw, ws)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for r, xv, gv in ((b, xs[1], gs[1]), (a, xs[0], gs[0]), (b, xs[1], gs[1])):
        x.copy_(xv)
        gy.copy_(gv)
        for f in ("padded_offsets", "tokens_per_expert", "token_of"):
            getattr(live.handle, f).copy_(getattr(r.handle, f))
        for t in (y, gx):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert_rows(r, y, tu.gemm_forward(r, w, xv))
        assert_rows(r, gx, tu.gemm_data(r, w, gv))
        assert torch.equal(gw.cpu(), tu.gemm_weight(r, gv, xv).float())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y.fill_(7.0)
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_grouped_gemm(live.handle, a.shape, a.layout, wd, x, y, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert_rows(b, y, tu.gemm_forward(b, w, xs[1]))


@pytest.mark.parametrize("N,Kd", [(512, 256), (257, 255)])
def test_two_calls_at_once(N, Kd):
    """Calls on two streams, each with a workspace of its own, while the other's run."""
    moe = moe_mod()
    rs = [tu.Routed(moe, 900, 6, 2, 8, seed=k) for k in (1, 2)]
    w = matrices(6, N, Kd, BF, 1, ints=2)
    xs, gs = [r.rows(Kd, BF, 2, ints=2) for r in rs], [r.rows(N, BF, 3, ints=2) for r in rs]
    wd, streams = w.cuda(), [torch.cuda.Stream() for _ in rs]
    d = [dict(x=x.cuda(), gy=g.cuda(), y=torch.full((r.cap, N), 7.0, dtype=BF, device="cuda"),
              gx=torch.full((r.cap, Kd), 7.0, dtype=BF, device="cuda"), gw=torch.empty(6, N, Kd, device="cuda"),
              ws=tu.workspace(moe, r, N, Kd)) for r, x, g in zip(rs, xs, gs)]
    torch.cuda.synchronize()
    for _ in range(20):
        for r, t, s in zip(rs, d, streams):
            at = r.handle, r.shape, r.layout
            moe.moe_grouped_gemm(*at, wd, t["x"], t["y"], t["ws"], stream=s)
            moe.moe_grouped_gemm_backward_data(*at, wd, t["gy"], t["gx"], t["ws"], stream=s)
            moe.moe_grouped_gemm_backward_weight(*at, t["x"], t["gy"], t["gw"], t["ws"], stream=s)
    torch.cuda.synchronize()
    for r, t, x, g in zip(rs, d, xs, gs):
        assert_rows(r, t["y"], tu.gemm_forward(r, w, x))
        assert_rows(r, t["gx"], tu.gemm_data(r, w, g))
        assert torch.equal(t["gw"].cpu(), tu.gemm_weight(r, g, x).float())


@pytest.mark.parametrize("N,Kd", [(264, 136), (65, 33)])
def test_short_calls_behind_one_another(N, Kd):
    """Calls of a tile or two, each pair of SMs leaving as soon as its last results are stored: the commits of its last
    stages have arrived in both CTAs by then."""
    moe = moe_mod()
    r = tu.Routed(moe, 40, 3, 2, 8, empty=(1,))
    w = matrices(3, N, Kd, BF, 1, ints=2)
    x, gy = r.rows(Kd, BF, 2, ints=2), r.rows(N, BF, 3, ints=2)
    wd, xd, gd, ws = w.cuda(), x.cuda(), gy.cuda(), tu.workspace(moe, r, N, Kd)
    y, gx = (torch.full((r.cap, c), 7.0, dtype=BF, device="cuda") for c in (N, Kd))
    gw = torch.empty(3, N, Kd, device="cuda")
    for _ in range(200):
        moe.moe_grouped_gemm(r.handle, r.shape, r.layout, wd, xd, y, ws)
        moe.moe_grouped_gemm_backward_data(r.handle, r.shape, r.layout, wd, gd, gx, ws)
        moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, xd, gd, gw, ws)
    torch.cuda.synchronize()
    assert int(r.handle.status.item()) == 0
    assert_rows(r, y, tu.gemm_forward(r, w, x))
    assert_rows(r, gx, tu.gemm_data(r, w, gy))
    assert torch.equal(gw.cpu(), tu.gemm_weight(r, gy, x).float())


def test_first_calls_of_a_process_in_a_capture():
    """Nothing of the calls' own setup needs a call outside a capture first."""
    import os
    import subprocess
    import sys

    code = '''
import torch, train_util as tu
from gpu_util import moe_mod
moe = moe_mod()
r = tu.Routed(moe, 40, 4, 2, 8)
outs = []
for N, Kd in ((64, 128), (33, 50)):
    x, gy = r.rows(Kd, tu.BF, 1, ints=2), r.rows(N, tu.BF, 2, ints=2)
    w = torch.randint(-2, 3, (4, N, Kd)).to(tu.BF)
    outs.append((w, x, gy, w.cuda(), x.cuda(), gy.cuda(), torch.zeros(r.cap, N, dtype=tu.BF, device="cuda"),
                 torch.zeros(4, N, Kd, device="cuda"), tu.workspace(moe, r, N, Kd)))
h = torch.randn(8, 256, device="cuda")
n, c, s = torch.empty_like(h), torch.empty(8, 256, dtype=torch.uint8, device="cuda"), torch.empty(8, 2, device="cuda")
pre, act = torch.zeros(r.cap, 64, device="cuda"), torch.zeros(r.cap, 32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for w, x, gy, wd, xd, gd, y, gw, ws in outs:
        moe.moe_grouped_gemm(r.handle, r.shape, r.layout, wd, xd, y, ws)
        moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, xd, gd, gw, ws)
    moe.moe_rms_norm(h, None, 1e-6, n, codes=c, scales=s)
    moe.moe_swiglu(r.handle, r.shape, r.layout, pre, act)
g.replay()
torch.cuda.synchronize()
for w, x, gy, wd, xd, gd, y, gw, ws in outs:
    assert torch.equal(y.cpu()[r.routed], tu.gemm_forward(r, w, x)[r.routed].to(tu.BF))
    assert torch.equal(gw.cpu(), tu.gemm_weight(r, gy, x).float())
assert bool((n - h * (h.square().mean(1, keepdim=True) + 1e-6) ** -0.5).abs().max() < 1e-5)
print("captured")
'''
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=300)
    assert p.returncode == 0 and "captured" in p.stdout, p.stdout + p.stderr


def test_tiles_that_take_longer_than_a_wait_may(tmp_path):
    """Built with a limit of 3 ms on a wait without progress, gradients whose tile of 2^21 rows takes 10 ms (aligned) to
    30 ms are whole: the roles that wait for the tile go on while its stages do. (With the limit of 2 s that is a tile of
    2^27 rows, which the call accepts.)"""
    import concurrent.futures as cf
    import os
    import subprocess
    import sys

    from permute_grouped_expert_gb300 import _build as b

    def compile_one(src):
        short = os.path.basename(src) == "grouped_gemm.cu"
        kept = os.path.join(b.BUILD, os.path.basename(src) + ".o")
        if not short and os.path.exists(kept) and os.path.getmtime(kept) >= max(map(os.path.getmtime, b._deps())):
            return kept
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        limit = ["-DMOE_WAIT_LIMIT_NS=3000000ull"] if short else []
        subprocess.run([b.nvcc(), *b.ARCH, *b.FLAGS, *limit, "-c", src, "-o", obj], check=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        objs = list(ex.map(compile_one, b._sources()))
    lib = str(tmp_path / "libmoe_short_waits.so")
    subprocess.run([b.nvcc(), *b.ARCH, "-shared", "-o", lib, *objs, "-lcudart"], check=True)
    code = """
import ctypes, sys
real = ctypes.CDLL
ctypes.CDLL = lambda path, *a, **k: real(sys.argv[1] if str(path).endswith("libmoe_gb300.so") else path, *a, **k)
import numpy as np, torch, train_util as tu
from gpu_util import moe_mod
moe = moe_mod()
rows, few, E = 1 << 21, 100, 5
r = tu.Routed(moe, 64, E, 1, 1)
counts = np.array([0, rows, 0, few, 0], np.int32)
off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
cap = int(off[-1])
shape, layout = moe.Shape(cap, 128, E, 1), moe.Layout(1, cap)
r.handle.padded_offsets.copy_(torch.from_numpy(off))
r.handle.tokens_per_expert.copy_(torch.from_numpy(counts))
r.handle.status.zero_()
g = torch.Generator(device="cuda").manual_seed(1)
for N, Kd in ((33, 17), (64, 40), (257, 24)):
    x, gy = (torch.randint(-1, 2, (cap, c), generator=g, device="cuda").to(tu.BF) for c in (Kd, N))
    ref = torch.zeros(E, N, Kd, dtype=torch.float64, device="cuda")
    for e in (1, 3):
        ref[e] = gy[off[e]:off[e + 1]].double().T @ x[off[e]:off[e + 1]].double()
    ws = torch.empty(moe.moe_grouped_gemm_workspace_size(shape, layout, N, Kd), dtype=torch.uint8, device="cuda")
    for dtype in (tu.BF, tu.F32):
        gw = torch.empty(E, N, Kd, dtype=dtype, device="cuda")
        moe.moe_grouped_gemm_backward_weight(r.handle, shape, layout, x, gy, gw, ws)
        torch.cuda.synchronize()
        a, z = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        moe.moe_grouped_gemm_backward_weight(r.handle, shape, layout, x, gy, gw, ws)
        z.record()
        torch.cuda.synchronize()
        assert int(r.handle.status.item()) == 0, (N, Kd, dtype)
        assert torch.equal(gw, ref.to(dtype)), (N, Kd, dtype)
        assert a.elapsed_time(z) > 3.0, "a tile shorter than the limit shows nothing"
print("whole")
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    p = subprocess.run([sys.executable, "-c", code, lib], capture_output=True, text=True, env=env, timeout=300)
    assert p.returncode == 0 and "whole" in p.stdout, p.stdout + p.stderr


@pytest.mark.parametrize("N,Kd", [(40, 24), (33, 17)])
def test_one_row_of_any_stride(N, Kd):
    """A buffer of one row has no stride that matters, zero and odd ones among them."""
    moe = moe_mod()
    r = tu.Routed(moe, 1, 1, 1, 1)
    w, x, gy = matrices(1, N, Kd, BF, 1, ints=2), r.rows(Kd, BF, 2, ints=2), r.rows(N, BF, 3, ints=2)
    for stride in (0, 1, N + Kd, 1000003):
        at = lambda t: t.cuda().as_strided(t.shape, (stride, 1))
        y, gx = at(torch.zeros(1, N, dtype=BF)), at(torch.zeros(1, Kd, dtype=BF))
        gw, ws = torch.empty(1, N, Kd, device="cuda"), tu.workspace(moe, r, N, Kd)
        moe.moe_grouped_gemm(r.handle, r.shape, r.layout, w.cuda(), at(x), y, ws)
        moe.moe_grouped_gemm_backward_data(r.handle, r.shape, r.layout, w.cuda(), at(gy), gx, ws)
        moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, at(x), at(gy), gw, ws)
        assert torch.equal(y.cpu(), tu.gemm_forward(r, w, x).to(BF))
        assert torch.equal(gx.cpu(), tu.gemm_data(r, w, gy).to(BF))
        assert torch.equal(gw.cpu(), tu.gemm_weight(r, gy, x).float())


def test_refusals():
    moe = moe_mod()
    r = tu.Routed(moe, 10, 2, 1, 8)
    w = matrices(2, 64, 32, BF, 1).cuda()
    x, y = torch.zeros(r.cap, 32, dtype=BF, device="cuda"), torch.zeros(r.cap, 64, dtype=BF, device="cuda")
    ws = tu.workspace(moe, r, 64, 32)
    call = lambda w=w, x=x, y=y, ws=ws: moe.moe_grouped_gemm(r.handle, r.shape, r.layout, w, x, y, ws)
    call()
    for bad in (dict(w=w[:1]), dict(w=w.float()), dict(x=x.half()), dict(x=y), dict(y=y[:3]), dict(w=w.transpose(1, 2)),
                dict(x=torch.zeros(r.cap, 64, dtype=BF, device="cuda")[:, ::2]), dict(ws=ws.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(moe.MoeError):
        call(ws=ws[:ws.numel() // 2])
    wide = torch.zeros(r.cap, 96, dtype=BF, device="cuda")
    with pytest.raises(moe.MoeError):  # y over x
        call(x=wide[:, :32], y=wide[:, 16:80])
    gw = torch.zeros(2, 64, 32, dtype=BF, device="cuda")
    with pytest.raises(moe.MoeError):  # an addend beside a 16-bit gradient
        moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, x, y, gw, ws, gw.float())
    with pytest.raises(moe.MoeError):  # a gradient of the other 16-bit type
        moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, x, y, gw.half(), ws)
    big = torch.zeros(2 * 64 * 32 + 4, device="cuda")
    with pytest.raises(moe.MoeError):  # an addend that overlaps the gradient
        moe.moe_grouped_gemm_backward_weight(r.handle, r.shape, r.layout, x, y, big[4:].view(2, 64, 32), ws,
                                             big[:-4].view(2, 64, 32))
