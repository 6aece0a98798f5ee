"""Plain 64-bit forms of the experts' training products, SwiGLU and the
root-mean-square norm, the routing they run on, and the error bounds their fp32
kernels keep (U, chains of additions and roundings as in block_util)."""
import numpy as np
import torch

import block_util as bu
from block_util import U

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


class Routed:
    """A routing on the GPU and its segments: handle, shape, layout; host offsets, counts, routed (bool [cap])."""

    def __init__(self, moe, T, E, K, m, cap=None, seed=0, empty=(), skew=0.0):
        r = np.random.default_rng(seed)
        score = r.gumbel(size=(T, E)) - skew * np.log1p(np.arange(E))
        score[:, list(empty)] = -1e9
        ids = np.sort(np.argsort(-score, axis=1)[:, :K], axis=1).astype(np.int16)
        self.full = T * K + E * (m - 1)
        self.cap = self.full if cap is None else cap
        self.shape, self.layout = moe.Shape(T, 128, E, K), moe.Layout(m, self.cap)
        self.handle = moe.Handle.empty(self.shape, self.layout)
        ws = torch.empty(moe.moe_preprocess_workspace_size(self.shape), dtype=torch.uint8, device="cuda")
        moe.moe_preprocess(moe.Routing(0, torch.from_numpy(ids).cuda()), self.shape, self.layout, self.handle, ws)
        counts = np.bincount(ids.reshape(-1), minlength=E)
        off = np.concatenate([[0], np.cumsum((counts + m - 1) // m * m)])
        assert np.array_equal(self.handle.padded_offsets.cpu().numpy(), off)
        self.segments = [(e, int(min(off[e], self.cap)), int(min(off[e] + counts[e], self.cap))) for e in range(E)]
        self.routed = torch.zeros(self.cap, dtype=torch.bool)
        for _, b, n in self.segments:
            self.routed[b:n] = True

    def rows(self, cols, dtype, seed, scale=1.0, ints=None, rest=float("nan")):
        """Random rows (of small whole numbers where ints is given); `rest` in every row that is not routed."""
        g = torch.Generator().manual_seed(seed)
        if ints is None:
            x = (torch.randn(self.cap, cols, generator=g) * scale).to(dtype)
        else:
            x = torch.randint(-ints, ints + 1, (self.cap, cols), generator=g).to(dtype)
        x[~self.routed] = rest
        return x


def workspace(moe, r, N, Kd):
    n = moe.moe_grouped_gemm_workspace_size(r.shape, r.layout, N, Kd)
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


def gemm_forward(r, w, x):
    y = torch.zeros(r.cap, w.shape[1], dtype=torch.float64)
    for e, b, n in r.segments:
        y[b:n] = x[b:n].double() @ w[e].double().T
    return y


def gemm_data(r, w, gy):
    return gemm_forward(r, w.transpose(1, 2), gy)


def gemm_weight(r, gy, x):
    gw = torch.zeros(r.shape.E, gy.shape[1], x.shape[1], dtype=torch.float64)
    for e, b, n in r.segments:
        gw[e] = gy[b:n].double().T @ x[b:n].double()
    return gw


def gemm_tol(ref, absolute, chain, dtype):
    """Products of 16-bit numbers are exact in fp32.  Each of the `chain` additions loses at most 2 U of what is summed
    (cut off, not rounded), and the result is rounded once."""
    return 1.01 * 2 * U * (chain + 1) * absolute + bu.rounding(ref, dtype)


# ------------------------------------------------------------------- SwiGLU

def swiglu(pre, p):
    I = pre.shape[1] // 2
    u, g = pre.double()[:, :I], pre.double()[:, I:]
    a = g * torch.sigmoid(g) * u
    return a if p is None else a * p.double()[:, None]


def swiglu_tol(pre, p, dtype):
    # exp to 2 + 1.173 |g| ulp ((4 + 2.35 |g|) U, CUDA's bound of its fast one), 1 + z to U, the quotient to 2 ulp (4 U),
    # and four products: below (14 + 2.4 |g|) U of the result
    a = swiglu(pre, p)
    g = pre.double()[:, pre.shape[1] // 2:].abs()
    return (14 + 2.4 * g) * U * a.abs() + bu.rounding(a, dtype) + 2.0 ** -140


def swiglu_backward(pre, p, ga):
    """(grad_pre, grad_probs, their bounds before rounding)"""
    I = pre.shape[1] // 2
    u, g, d = pre.double()[:, :I], pre.double()[:, I:], ga.double()
    s = torch.sigmoid(g)
    act = g * s
    terms = d * act * u
    q = d if p is None else d * p.double()[:, None]
    gu, gg = q * act, q * u * s * (1 + g * (1 - s))
    # s and 1 - s to (10 + 2.4 |g|) U, as in swiglu_tol; 1 + g (1 - s) may cancel: its error is that of its two parts
    e = (10 + 2.4 * g.abs()) * U
    tg = (q * u * s).abs() * (4 * U + e) * ((1 + g * (1 - s)).abs() + 1 + (g * (1 - s)).abs())
    tp = ((4 * U + e) * terms.abs()).sum(1) + (I / 32 + 24) * U * terms.abs().sum(1)
    return torch.cat([gu, gg], 1), terms.sum(1), torch.cat([(6 * U + e) * gu.abs(), tg], 1) + 2.0 ** -140, tp


# ----------------------------------------------------------------- RMS norm

def rms_forward(h, w, eps):
    h = h.double()
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    v = h * rstd[:, None]
    return (v if w is None else v * w.double()), rstd


def rms_forward_tol(h, w, eps):
    """Bounds of v (before its rounding) and rstd: the mean of squares to a chain of H / 32 terms and a tree, half of
    which reaches its root."""
    v, rstd = rms_forward(h, w, eps)
    rel = 0.5 * (h.shape[1] / 32 + 24) * U + 4 * U
    return v.abs() * (rel + 4 * U) * 1.01 + 2.0 ** -148, rstd * (rel + U) * 1.01


def rms_backward(gy, h, w, rstd, gsum):
    gy, rstd = gy.double(), rstd.double()[:, None]
    xhat = h.double() * rstd
    u = gy * w.double() if w is not None else gy
    gx = rstd * (u - xhat * (u * xhat).mean(1, keepdim=True))
    if gsum is not None:
        gx = gx + gsum.double()
    return gx, (gy * xhat).sum(0)


def rms_backward_tol(gy, h, w, rstd, gsum, dtype):
    rows, H = h.shape
    gx, gw = rms_backward(gy, h, w, rstd, gsum)
    rstd = rstd.double()[:, None]
    g, xhat = gy.double().abs(), (h.double() * rstd).abs()
    u = g * w.double().abs() if w is not None else g
    c = H / 32 + 24
    tol = rstd * ((c + 8) * U * xhat * (u * xhat).mean(1, keepdim=True) + 8 * U * u)
    if gsum is not None:
        tol = tol + 2 * U * (gsum.double().abs() + gx.abs())
    cr = min(rows, rows / 8 + 340) + 8
    return tol * 1.01 + bu.rounding(gx, dtype), cr * U * (g * xhat).sum(0)
