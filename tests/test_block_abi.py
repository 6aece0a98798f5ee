"""Host-side checks (no GPU) of the operators around the layer: bad arguments are
refused by the C entry points before anything is enqueued, and the workspace
query behaves as documented.  The pointers below are never dereferenced."""
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


def rows(moe, stride=64, data=0x10000):
    return byref(moe._Rows(data, stride))


def test_constants_match_the_header(moe):
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")).read()
    pairs = re.findall(r"\bMOE_((?:ELEM|SCORE|W4)_\w+)\s*=\s*(\d+)", text)
    assert len(pairs) == 7
    for name, value in pairs:
        assert getattr(moe, name) == int(value), name


def test_layer_norm_refusals(moe):
    lib = moe.library()

    def call(n, x=None, y=None, res=None, s=None, w=None, mean=None):
        return lib.moe_layer_norm(byref(n), x or rows(moe), res, w, None, y or rows(moe, data=0x90000), s, mean, None,
                                  None)

    bad = [moe._Norm(-1, 64, 1, 1, 1e-5), moe._Norm(4, 0, 1, 1, 1e-5), moe._Norm(4, (1 << 20) + 1, 1, 1, 1e-5),
           moe._Norm(4, 64, 3, 3, 1e-5), moe._Norm(4, 64, 0, 1, 1e-5), moe._Norm(4, 64, 1, 2, 1e-5),
           moe._Norm(4, 64, 1, 1, -1e-5), moe._Norm(4, 64, 1, 1, float("nan"))]
    for n in bad:
        assert call(n) == moe.MOE_ERR_INVALID_ARG, (n.rows, n.H, n.dtype, n.param_dtype, n.eps)
    good = moe._Norm(4, 64, 1, 1, 1e-5)
    far = lambda: rows(moe, data=0x20000)
    assert call(good, x=rows(moe, stride=63)) == moe.MOE_ERR_INVALID_ARG      # rows overlap
    assert call(good, x=rows(moe, data=0x10001)) == moe.MOE_ERR_INVALID_ARG   # half an element off
    assert call(good, y=rows(moe)) == moe.MOE_ERR_INVALID_ARG                 # y over x
    assert call(good, s=far()) == moe.MOE_ERR_INVALID_ARG                     # a sum without a residual
    assert call(good, res=far(), s=rows(moe, data=0x20000 + 128)) == moe.MOE_ERR_INVALID_ARG  # one row off
    assert call(good, w=ctypes.c_void_p(0x30001)) == moe.MOE_ERR_INVALID_ARG
    assert call(good, mean=ctypes.c_void_p(0x30002)) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_layer_norm(None, rows(moe), None, None, None, far(), None, None, None, None) == \
        moe.MOE_ERR_INVALID_ARG
    none = moe._Norm(0, 64, 1, 1, 1e-5)
    assert call(none) == moe.MOE_OK  # no rows: nothing to launch


def test_layer_norm_backward_refusals(moe):
    lib = moe.library()
    n = moe._Norm(4, 64, 1, 0, 0.0)
    need = moe.moe_layer_norm_workspace_size(4, 64)
    assert need >= 64 * 8

    def call(gx=0x40000, ws=FAKE, nbytes=need, mean=FAKE, gw=FAKE, gy=0x20000):
        return lib.moe_layer_norm_backward(byref(n), rows(moe, data=gy), rows(moe, data=0x30000), None, mean, FAKE,
                                           None, rows(moe, data=gx), gw, None, ws, nbytes, None)

    assert call(nbytes=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert call(ws=None) == moe.MOE_ERR_INVALID_ARG
    assert call(ws=ctypes.c_void_p(0x10008)) == moe.MOE_ERR_INVALID_ARG
    assert call(mean=None) == moe.MOE_ERR_INVALID_ARG
    assert call(gx=0x30000) == moe.MOE_ERR_INVALID_ARG       # over h
    assert call(gx=0x20000 + 16) == moe.MOE_ERR_INVALID_ARG  # over grad_y, shifted
    for bad in ((-1, 64), (4, 0), (4, (1 << 20) + 1)):
        with pytest.raises(moe.MoeError):
            moe.moe_layer_norm_workspace_size(*bad)


def test_router_refusals(moe):
    lib = moe.library()

    def call(r, fmt=0, map_=FAKE, probs=FAKE, logits=None):
        return lib.moe_router_topk(byref(r), logits or rows(moe), None, fmt, map_, probs, None, None)

    R = moe._Router
    for r in (R(-1, 16, 2, 0, 0, 1, 1.0), R(4, 0, 1, 0, 0, 1, 1.0), R(4, 1025, 2, 0, 0, 1, 1.0),
              R(4, 16, 0, 0, 0, 1, 1.0), R(4, 16, 17, 0, 0, 1, 1.0), R(4, 200, 129, 0, 0, 1, 1.0),
              R(4, 16, 2, 5, 0, 1, 1.0), R(4, 16, 2, 0, 2, 1, 1.0), R(4, 16, 2, 0, 0, 1, float("nan")),
              R(1 << 40, 16, 2, 0, 0, 1, 1.0)):
        assert call(r) == moe.MOE_ERR_INVALID_ARG, (r.T, r.E, r.K)
    good = R(4, 16, 2, 0, 0, 1, 1.0)
    assert call(good, fmt=2) == moe.MOE_ERR_INVALID_ARG
    assert call(good, map_=None) == moe.MOE_ERR_INVALID_ARG
    assert call(good, probs=None) == moe.MOE_ERR_INVALID_ARG
    assert call(good, map_=ctypes.c_void_p(0x10001)) == moe.MOE_ERR_INVALID_ARG
    assert call(good, logits=rows(moe, stride=15)) == moe.MOE_ERR_INVALID_ARG
    assert call(R(0, 16, 2, 0, 0, 1, 1.0), map_=None, probs=None) == moe.MOE_OK
    assert lib.moe_router_topk_backward(byref(good), rows(moe), 0, FAKE, None, rows(moe, data=0x90000), None) == \
        moe.MOE_ERR_INVALID_ARG


def test_w4_refusals(moe):
    lib = moe.library()

    def call(w, x=None, y=None, act=0, M=2, add=None):
        return lib.moe_w4_matvec(byref(w), M, x or rows(moe, stride=256), act, add, y or rows(moe, data=0x90000), None)

    def weight(N=16, Kd=256, group=64, dtype=1, codes=0x50000, scales=0x60000):
        return moe._W4(N, Kd, group, dtype, codes, scales, None)

    for w in (weight(N=0), weight(Kd=0), weight(Kd=40), weight(group=16), weight(group=256), weight(dtype=0),
              weight(codes=0), weight(codes=0x50008), weight(scales=0), weight(scales=0x60001), weight(N=1 << 25),
              weight(Kd=1 << 21)):
        assert call(w) == moe.MOE_ERR_INVALID_ARG
    good = weight()
    assert call(good, M=-1) == moe.MOE_ERR_INVALID_ARG
    assert call(good, act=2) == moe.MOE_ERR_INVALID_ARG
    assert call(weight(N=15), act=1) == moe.MOE_ERR_INVALID_ARG
    assert call(good, act=1, add=rows(moe, data=0xa0000)) == moe.MOE_ERR_INVALID_ARG
    assert call(good, x=rows(moe, stride=252)) == moe.MOE_ERR_INVALID_ARG
    assert call(good, x=rows(moe, stride=260)) == moe.MOE_ERR_INVALID_ARG   # rows off the 16-byte grid
    assert call(good, x=rows(moe, stride=256, data=0x10008)) == moe.MOE_ERR_INVALID_ARG
    assert call(good, y=rows(moe, data=0x10100)) == moe.MOE_ERR_INVALID_ARG  # y inside x
    assert call(good, add=rows(moe, data=0x90002)) == moe.MOE_ERR_INVALID_ARG  # over y, shifted
    assert call(good, M=0) == moe.MOE_OK
    handle = moe._HandleDev(*([FAKE] * 8))
    x, y = rows(moe, stride=256, data=0x100000), rows(moe, data=0x900000)
    grouped = lambda s, l: lib.moe_grouped_w4_matvec(byref(handle), byref(s), byref(l), byref(good), x, 0, y, None)
    assert grouped(moe._Shape(4, 0, 8, 9, 0), moe._Layout(32, 64)) == moe.MOE_ERR_INVALID_ARG
    assert grouped(moe._Shape(4, 0, 2000, 2, 0), moe._Layout(32, 64)) == moe.MOE_ERR_INVALID_ARG
    assert grouped(moe._Shape(4, 0, 8, 2, 0), moe._Layout(32, 1 << 31)) == moe.MOE_ERR_INVALID_ARG
    assert grouped(moe._Shape(0, 0, 8, 2, 0), moe._Layout(32, 64)) == moe.MOE_OK
    assert lib.moe_quantize_w4_rows(FAKE, 4, 100, 64, 1, FAKE, FAKE, None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_quantize_w4_rows(FAKE, 0, 128, 64, 1, FAKE, FAKE, None, None) == moe.MOE_OK


def test_matrices_beyond_the_address_space(moe):
    """Rows times stride that no memory holds (and no 64-bit sum of bytes) are refused, overlapping or not."""
    lib = moe.library()
    far, many = 1 << 40, 1 << 39
    at = lambda i: rows(moe, stride=far, data=0x10000 + 0x1000 * i)
    bad = moe.MOE_ERR_INVALID_ARG
    norm = moe._Norm(many, 64, 1, 1, 1e-5)
    assert lib.moe_layer_norm(byref(norm), at(0), None, None, None, at(1), None, None, None, None) == bad
    assert lib.moe_layer_norm_backward(byref(norm), at(0), at(1), None, FAKE, FAKE, None, at(2), None, None, None, 0,
                                       None) == bad
    router = moe._Router(many // 64, 32, 2, 0, 0, 1, 1.0)
    assert lib.moe_router_topk(byref(router), at(0), None, 0, FAKE, FAKE, None, None) == bad
    assert lib.moe_router_topk_backward(byref(router), at(0), 0, FAKE, FAKE, at(1), None) == bad
    w = moe._W4(16, 256, 64, 1, 0x50000, 0x60000, None)
    assert lib.moe_w4_matvec(byref(w), 1 << 31, at(0), 0, None, at(1), None) == bad
    handle = moe._HandleDev(*([FAKE] * 8))
    assert lib.moe_grouped_w4_matvec(byref(handle), byref(moe._Shape(4, 0, 8, 2, 0)),
                                     byref(moe._Layout(32, (1 << 31) - 1)), byref(w), at(0), 0, at(1), None) == bad
