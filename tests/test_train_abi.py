"""Host-side checks (no GPU) of the root-mean-square norm, the products grouped by expert and SwiGLU: bad arguments are
refused by the C entry points before anything is enqueued.  The pointers below are never dereferenced."""
import ctypes

import pytest

byref = ctypes.byref
FAKE = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__.build_library()
    import permute_grouped_expert_gb300 as m

    return m


def rows(moe, data=0x10000, stride=64):
    return byref(moe._Rows(data, stride))


def routed(moe, shape=None, layout=None, handle=None):
    return (byref(moe._HandleDev(*([0x10000] * 8)) if handle is None else handle),
            byref(moe._Shape(4, 0, 2, 1, 0) if shape is None else shape),
            byref(moe._Layout(1, 4) if layout is None else layout))


def bad_routings(moe):
    S, L = moe._Shape, moe._Layout
    for s in (S(-1, 0, 2, 1, 0), S(4, 0, 0, 1, 0), S(4, 0, 1025, 1, 0), S(4, 0, 2, 0, 0), S(4, 0, 2, 3, 0),
              S(4, 0, 200, 129, 0), S(1 << 31, 0, 2, 1, 0)):
        yield routed(moe, shape=s)
    for cap in (-1, 1 << 31):
        yield routed(moe, layout=L(1, cap))
    yield routed(moe, handle=moe._HandleDev())
    yield (None,) + routed(moe)[1:]
    yield routed(moe)[:1] + (None,) + routed(moe)[2:]
    yield routed(moe)[:2] + (None,)


def test_rms_norm_refusals(moe):
    lib = moe.library()

    def call(n, x=None, res=None, y=0x20000, s=None, rstd=None, codes=None, scales=None, w=None):
        return lib.moe_rms_norm(byref(n) if n else None, x or rows(moe), res, w, rows(moe, y) if y else None, s, rstd,
                                codes, scales, None)

    N = moe._Norm
    for n in (N(-1, 64, 1, 1, 1e-5), N(4, 0, 1, 1, 1e-5), N(4, (1 << 20) + 1, 1, 1, 1e-5), N(4, 64, 3, 3, 1e-5),
              N(4, 64, 0, 1, 1e-5), N(4, 64, 1, 1, -1.0), N(4, 64, 1, 1, float("inf")), None):
        assert call(n) == moe.MOE_ERR_INVALID_ARG
    good, p = N(4, 64, 1, 1, 1e-5), ctypes.c_void_p
    bad = [dict(y=None), dict(codes=p(0x30000)), dict(scales=p(0x30000)), dict(y=0x10000), dict(s=rows(moe, 0x40000)),
           dict(x=rows(moe, stride=63)), dict(x=rows(moe, 0x10001)), dict(rstd=p(0x30002)), dict(w=p(0x30001)),
           dict(codes=p(0x30000), scales=p(0x40002)), dict(codes=p(0x30000), scales=p(0x30010)),
           dict(codes=p(0x10008), scales=p(0x40000)), dict(codes=p(0x40000), scales=p(0x20000)),
           dict(res=rows(moe, 0x50000), codes=p(0x50000), scales=p(0x40000)),
           dict(res=rows(moe, 0x50000), s=rows(moe, 0x50000 + 128))]
    for b in bad:
        assert call(good, **b) == moe.MOE_ERR_INVALID_ARG, b
    assert call(N(0, 64, 1, 1, 1e-5)) == moe.MOE_OK  # no rows: nothing to launch


def test_rms_norm_backward_refusals(moe):
    lib = moe.library()
    need = moe.moe_rms_norm_workspace_size(4, 64)
    assert need >= 64 * 4

    def call(gx=0x40000, ws=FAKE, nbytes=need, rstd=FAKE, gw=FAKE, gy=0x20000):
        return lib.moe_rms_norm_backward(byref(moe._Norm(4, 64, 1, 0, 0.0)), rows(moe, gy), rows(moe, 0x30000), None,
                                         rstd, None, rows(moe, gx), gw, ws, nbytes, None)

    assert call(nbytes=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    for b in (dict(ws=None), dict(ws=ctypes.c_void_p(0x10008)), dict(rstd=None), dict(gx=0x30000),
              dict(gx=0x20000 + 16), dict(gw=ctypes.c_void_p(0x10002))):
        assert call(**b) == moe.MOE_ERR_INVALID_ARG, b
    for bad in ((-1, 64), (4, 0), (4, (1 << 20) + 1)):
        with pytest.raises(moe.MoeError):
            moe.moe_rms_norm_workspace_size(*bad)


def workspace_bytes(moe, shape=(4, 0, 2, 1, 0), cap=4, N=64, Kd=32):
    return moe.moe_grouped_gemm_workspace_size(moe.Shape(*shape), moe.Layout(1, cap), N, Kd)


@pytest.mark.parametrize("data", [False, True])
def test_grouped_gemm_refusals(moe, data):
    lib = moe.library()
    need = workspace_bytes(moe)

    def call(r=None, g=None, w=FAKE, x=0x100000, y=0x200000, sx=64, sy=64, ws=FAKE, nbytes=need):
        fn = lib.moe_grouped_gemm_backward_data if data else lib.moe_grouped_gemm
        g = moe._Gemm(64, 32, 1) if g is None else g
        return fn(*(r or routed(moe)), byref(g), w, rows(moe, x, sx), rows(moe, y, sy), ws, nbytes, None)

    for r in bad_routings(moe):
        assert call(r=r) == moe.MOE_ERR_INVALID_ARG
    G = moe._Gemm
    for g in (G(0, 32, 1), G(64, 0, 1), G((1 << 20) + 1, 32, 1), G(64, (1 << 20) + 1, 1), G(64, 32, 0), G(64, 32, 3)):
        assert call(g=g) == moe.MOE_ERR_INVALID_ARG
    for b in (dict(w=None), dict(w=ctypes.c_void_p(0x10001)), dict(x=0), dict(y=0), dict(x=0x100001), dict(sx=31),
              dict(sy=31), dict(y=0x100000), dict(y=0x100000 + 64), dict(y=0x10000 + 100), dict(ws=None),
              dict(ws=ctypes.c_void_p(0x10008))):
        assert call(**b) == moe.MOE_ERR_INVALID_ARG, b
    assert call(nbytes=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    none = routed(moe, shape=moe._Shape(0, 0, 2, 1, 0))
    assert call(r=none) == moe.MOE_OK  # no tokens: nothing to launch
    assert call(r=routed(moe, layout=moe._Layout(1, 0))) == moe.MOE_OK


def test_grouped_gemm_backward_weight_refusals(moe):
    lib = moe.library()
    need = workspace_bytes(moe)

    def call(r=None, g=None, x=0x100000, gy=0x200000, out=0, add=None, gw=0x300000, ws=FAKE, nbytes=need):
        g = moe._Gemm(64, 32, 1) if g is None else g
        return lib.moe_grouped_gemm_backward_weight(*(r or routed(moe)), byref(g), rows(moe, x), rows(moe, gy), out, add,
                                                    gw, ws, nbytes, None)

    for r in bad_routings(moe):
        assert call(r=r) == moe.MOE_ERR_INVALID_ARG
    for b in (dict(g=moe._Gemm(64, 32, 0)), dict(out=2), dict(out=3), dict(out=1, add=0x400000), dict(add=0x400002),
              dict(add=0x300010), dict(gw=None), dict(gw=0x300002), dict(gw=0x100000), dict(gw=0x200000 - 8), dict(x=0),
              dict(gy=0), dict(ws=None)):
        assert call(**b) == moe.MOE_ERR_INVALID_ARG, b
    assert call(nbytes=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert call(r=routed(moe, layout=moe._Layout(1, (1 << 27) + 1)), x=0x1000, gy=1 << 50, gw=1 << 52) == \
        moe.MOE_ERR_UNSUPPORTED


def test_more_tiles_than_can_be_counted_are_refused(moe):
    layout, g = moe._Layout(1, (1 << 31) - 1), moe._Gemm(1 << 20, 1, 1)
    assert moe.library().moe_grouped_gemm(*routed(moe, layout=layout), byref(g), FAKE, rows(moe, 1 << 50, 1),
                                          rows(moe, 1 << 54, 1 << 20), FAKE, 1 << 20, None) == moe.MOE_ERR_INVALID_ARG


def test_grouped_gemm_workspace_size(moe):
    assert workspace_bytes(moe) % 16 == 0
    for bad in (dict(shape=(-1, 0, 2, 1, 0)), dict(shape=(4, 0, 0, 1, 0)), dict(cap=-1), dict(N=0), dict(Kd=(1 << 20) + 1)):
        with pytest.raises(moe.MoeError):
            workspace_bytes(moe, **bad)


def test_swiglu_refusals(moe):
    lib = moe.library()

    def call(r=None, I=32, dtype=1, pre=0x100000, probs=None, act=0x200000, stride=64):
        return lib.moe_swiglu(*(r or routed(moe)), I, dtype, rows(moe, pre, stride), probs, rows(moe, act), None)

    def back(r=None, I=32, dtype=1, ga=0x200000, gpre=0x300000, gp=None):
        return lib.moe_swiglu_backward(*(r or routed(moe)), I, dtype, rows(moe, 0x100000), None, rows(moe, ga),
                                       rows(moe, gpre), gp, None)

    for r in list(bad_routings(moe)) + [routed(moe, handle=moe._HandleDev(0x10000, 0x10000))]:  # no token_of
        assert call(r=r) == back(r=r) == moe.MOE_ERR_INVALID_ARG
    for b in (dict(I=0), dict(I=(1 << 20) + 1), dict(dtype=3), dict(pre=0), dict(act=0), dict(pre=0x100001),
              dict(stride=63), dict(act=0x100000), dict(probs=0x10001)):
        assert call(**b) == moe.MOE_ERR_INVALID_ARG, b
    for b in (dict(I=0), dict(dtype=9), dict(ga=0), dict(gpre=0), dict(gpre=0x100000 + 128), dict(gpre=0x200000),
              dict(gp=0x10002)):
        assert back(**b) == moe.MOE_ERR_INVALID_ARG, b
    none = routed(moe, shape=moe._Shape(0, 0, 2, 1, 0))
    assert call(r=none) == back(r=none) == moe.MOE_OK
