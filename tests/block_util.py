"""Plain 64-bit forms of the operators around the layer (layer norm, router,
4-bit matrix-vector products) and the error bounds their fp32 kernels keep.

U is fp32's unit roundoff.  A sum of n fp32 terms whose longest chain of
additions is c differs from the exact sum by at most c * U * sum|terms| to first
order, whatever the order; every bound below is made of such terms and of one
rounding of the result to its type."""
import numpy as np
import torch

U = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half the spacing of the subnormals
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def f64(t):
    return t.detach().cpu().to(torch.float64)


def randn(*shape, seed=0, scale=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def rounding(v, dtype):
    return ROUND[dtype] * v.abs() + TINY[dtype]


def assert_within(got, want, tol, what=""):
    got = f64(got)
    want, tol = want.cpu(), tol.cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    bad &= ~(torch.isnan(got) & torch.isnan(want))
    bad &= ~(got == want)  # infinities
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: got {got[i]}, want "
                             f"{want[i]}, tolerance {tol.expand_as(want)[i]}")


# ---------------------------------------------------------------- layer norm

def norm_forward(h, w, b, eps):
    """64-bit layer norm of rows h and its statistics: (y, mean, rstd, xhat)."""
    h = h.double()
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    xhat = d * rstd[:, None]
    y = xhat
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean, rstd, xhat


def norm_forward_tol(h, w, b, eps, dtype):
    """Bounds of (y, mean, rstd).  Chains: at most H / 32 terms a lane and a few
    tree steps.  The mean's error shifts every deviation; the variance about a
    shifted mean grows by the shift squared."""
    H = h.shape[1]
    y, mean, rstd, xhat = norm_forward(h, w, b, eps)
    c = H / 32 + 24
    e_mean = c * U * h.double().abs().mean(1) + U * mean.abs()
    var = 1.0 / rstd ** 2 - eps
    d_abs = (h.double() - mean[:, None]).abs()
    # a deviation carries its own rounding and the mean's error
    e_var = c * U * var + 2 * (d_abs * (U * d_abs + e_mean[:, None])).mean(1) + e_mean ** 2
    e_rel = 0.5 * e_var * rstd ** 2 + 4 * U
    wa = w.double().abs() if w is not None else torch.ones(H, dtype=torch.float64)
    base = (xhat * wa).abs()
    tol = wa * (e_mean * rstd)[:, None] + base * (e_rel[:, None] + 6 * U)
    if b is not None:
        tol = tol + 2 * U * (base + b.double().abs())
    return tol * 1.01 + rounding(y, dtype), e_mean * 1.01 + U * mean.abs(), rstd * (e_rel + U) * 1.01


def norm_backward(gy, h, w, mean, rstd, gsum):
    gy, mean, rstd = gy.double(), mean.double()[:, None], rstd.double()[:, None]
    xhat = (h.double() - mean) * rstd
    u = gy * w.double() if w is not None else gy
    gx = rstd * (u - u.mean(1, keepdim=True) - xhat * (u * xhat).mean(1, keepdim=True))
    if gsum is not None:
        gx = gx + gsum.double()
    return gx, (gy * xhat).sum(0), gy.sum(0)


def norm_backward_tol(gy, h, w, mean, rstd, gsum, dtype):
    rows, H = h.shape
    gx, gw, gb = norm_backward(gy, h, w, mean, rstd, gsum)
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    g = gy.double().abs()
    xhat = ((h.double() - mean) * rstd).abs()
    u = g * w.double().abs() if w is not None else g
    c = H / 32 + 24
    m1, m2 = u.mean(1, keepdim=True), (u * xhat).mean(1, keepdim=True)
    # sums to c U, xhat to 2 U, u to U, and a handful of roundings of the terms
    tol = rstd * ((c + 8) * U * (m1 + xhat * m2) + 8 * U * u)
    if gsum is not None:
        tol = tol + 2 * U * (gsum.double().abs() + gx.abs())
    # columns: chains of at most rows / 8 terms a thread and some hundreds of partial sums
    cr = min(rows, rows / 8 + 340) + 8
    return tol * 1.01 + rounding(gx, dtype), cr * U * (g * xhat).sum(0), cr * U * g.sum(0)


# -------------------------------------------------------------------- router

def router_scores(logits, sigmoid, bias):
    """Selection scores in 64 bits; -inf where an expert is masked or NaN."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    if bias is None:
        return l
    with np.errstate(over="ignore"):
        s = (1.0 / (1.0 + np.exp(-l)) if sigmoid else l) + np.asarray(bias, np.float64)
    if not sigmoid:  # the sum is rounded to fp32 once
        s = s.astype(np.float32).astype(np.float64)
    s = np.where(np.isneginf(l) | np.isnan(s), -np.inf, s)
    return s


def router_select(scores, K):
    """bool [T][E]: the K largest scores of each row, ties to the lowest index, never -inf."""
    T, E = scores.shape
    on = np.zeros((T, E), bool)
    for t in range(T):
        for e in np.argsort(-scores[t], kind="stable")[:K]:
            on[t, e] = scores[t, e] > -np.inf
    return on


def router_weights(logits, live, on, sigmoid, renorm, scale):
    """64-bit weights [T][E], 0 off the map, by ratios that stay finite at any logit."""
    l = np.where(live, np.asarray(logits, np.float64), -np.inf)
    part = on if (renorm or sigmoid) else live
    w = np.zeros(l.shape)
    for t in range(l.shape[0]):
        idx = np.nonzero(part[t])[0]
        if not len(idx):
            continue
        v = l[t, idx]
        if sigmoid:
            logs = -np.logaddexp(0.0, -v)
            s = np.exp(logs - logs.max()) / np.exp(logs - logs.max()).sum() if renorm else np.exp(logs)
        else:
            with np.errstate(invalid="ignore"):
                d = np.where(v == v.max(), 0.0, v - v.max())
            s = np.exp(d) / np.exp(d).sum()
        w[t, idx] = s
    return np.where(on, w, 0.0) * scale


def router_tol(logits, live, w, E):
    """exp(l - top): its argument's rounding gives |l - top| U, the function a few
    U, the sum a chain of E / 32 + 5 terms; two divisions and the scale."""
    l = np.where(live & np.isfinite(logits), np.asarray(logits, np.float64), np.nan)
    spread = np.nan_to_num(np.nanmax(l, 1, initial=-np.inf, where=~np.isnan(l)) -
                           np.nanmin(l, 1, initial=np.inf, where=~np.isnan(l)), nan=0.0, posinf=0.0, neginf=0.0)
    return np.abs(w) * U * (2 * np.minimum(spread, 200.0)[:, None] + E / 32 + 48) + 2.0 ** -126


def router_backward(logits, on, gp, sigmoid, renorm, scale):
    """64-bit gradient of the logits; gp [T][E] with anything off the map."""
    l = np.asarray(logits, np.float64)
    live = l > -np.inf
    on = on & live
    g = np.where(on, gp, 0.0)
    n = router_weights(l, live, on if (sigmoid or renorm) else live, sigmoid, renorm, 1.0)
    if not sigmoid and not renorm:
        return scale * n * (g - (g * n).sum(1, keepdims=True))
    rest = 1.0 / (1.0 + np.exp(np.minimum(np.where(live, l, 0.0), 700.0))) if sigmoid else 1.0
    dot = (g * n).sum(1, keepdims=True) if renorm else 0.0
    return scale * n * rest * (g - dot)


def dense_to_full(ids, probs, E):
    """Dense ids / values [T][K] as (on, values) [T][E]."""
    T, K = ids.shape
    on = np.zeros((T, E), bool)
    v = np.zeros((T, E))
    for t in range(T):
        for k in range(K):
            if ids[t, k] >= 0:
                on[t, ids[t, k]] = True
                v[t, ids[t, k]] = probs[t, k]
    return on, v


# ------------------------------------------------------------ 4-bit products

def w4_random(N, Kd, group, dtype, zeros, seed, lead=()):
    g = torch.Generator().manual_seed(seed)
    G = -(-Kd // group)
    codes = torch.randint(0, 256, (*lead, N, Kd // 2), generator=g, dtype=torch.uint8)
    scales = (0.01 * (0.5 + torch.rand(*lead, N, G, generator=g))).to(dtype)
    z = torch.randint(0, 256, (*lead, N, (G + 1) // 2), generator=g, dtype=torch.uint8) if zeros else None
    return codes, scales, z


def w4_dequant(codes, scales, zeros, group):
    """64-bit weights [.., N][Kd]."""
    Kd, G = codes.shape[-1] * 2, scales.shape[-1]
    q = torch.empty(*codes.shape[:-1], Kd, dtype=torch.float64)
    q[..., 0::2], q[..., 1::2] = (codes & 15).double(), (codes >> 4).double()
    if zeros is None:
        z = torch.full(scales.shape, 8.0, dtype=torch.float64)
    else:
        z = torch.empty(*zeros.shape[:-1], zeros.shape[-1] * 2, dtype=torch.float64)
        z[..., 0::2], z[..., 1::2] = (zeros & 15).double(), (zeros >> 4).double()
        z = z[..., :G]
    at = torch.arange(Kd) // group
    return (q - z[..., at]) * scales.double()[..., at]


def w4_product(x, W, group, swiglu=False, addend=None, dtype=torch.bfloat16):
    """(64-bit y, tolerance).  Products are exact; a group is summed in steps of 8
    products whose partial sums may be cut instead of rounded (2 U), then the
    groups and a few warps in fp32."""
    x = x.double()
    y = x @ W.T
    c = group / 8 + W.shape[1] / group + 24
    tol = c * 2 * U * (x.abs() @ W.abs().T)
    if swiglu:
        n = y.shape[1] // 2
        up, gate, eu, eg = y[:, :n], y[:, n:], tol[:, :n], tol[:, n:]
        silu = gate * torch.sigmoid(gate)
        # |silu'| <= 1.1
        y = silu * up
        tol = silu.abs() * eu + 1.1 * eg * (up.abs() + eu) + 12 * U * y.abs()
    if addend is not None:
        y = y + addend.double()
        tol = tol + U * y.abs()
    return y, tol * 1.01 + rounding(y, dtype)
