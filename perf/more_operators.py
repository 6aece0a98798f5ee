"""The operators that the MoE layer's training and its 8-bit path need beside those of operators.py, as cases to measure.

* products grouped by expert over dispatched rows, of ragged sizes: the forward
  product, the gradient of the rows and the gradient of the weights;
* SwiGLU of the dispatched rows between FC1 and FC2, with the routes'
  probabilities, and its gradient;
* root-mean-square norm with the residual sum, in the rows' type and in E4M3 with
  a scale per 128 elements (what the dispatch takes), and its gradient.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, where ``own`` is true, with the calls a user
makes of this package.  ``exact`` computes it from its definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
BLOCK = 128  # elements that share a scale of the 8-bit output


def _moe():
    import permute_grouped_expert_gb300 as moe

    return moe


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through its 8 experts' FC2 in bf16 (256 experts, intermediate 2048 -> hidden 7168)
        dict(name="gemm_decode1", op="gemm", T=1, E=256, top=8, N=7168, K=2048, m=32, dtype="bf16", skew=False),
        # 64 decoded tokens through the same matrices in f16: two rows an expert
        dict(name="gemm_decode64", op="gemm", T=64, E=256, top=8, N=7168, K=2048, m=32, dtype="f16", skew=False),
        # FC1 of a training step or a prompt: 8192 tokens, popularity of the experts as in the dsv3 workload
        dict(name="gemm_train", op="gemm", T=8192, E=256, top=8, N=4096, K=7168, m=32, dtype="bf16", skew=True),
        # gradient of FC1's rows in the mid workload (64 experts, hidden 2048, intermediate 1024)
        dict(name="gemm_dgrad_mid", op="gemm_dgrad", T=4096, E=64, top=8, N=2048, K=2048, m=32, dtype="bf16",
             skew=False),
        # a research-size model with odd widths and unpadded segments, nothing aligned to 16 bytes
        dict(name="gemm_dgrad_odd", op="gemm_dgrad", T=777, E=16, top=3, N=1001, K=1537, m=1, dtype="f16",
             skew=False),
        # gradient of FC1's weights in the mid workload, kept in fp32 for the optimizer
        dict(name="gemm_wgrad_mid", op="gemm_wgrad", T=4096, E=64, top=8, N=2048, K=2048, m=32, dtype="bf16",
             gdtype="f32", skew=False),
        # a small ragged layer, gradient in the weights' type, popular and idle experts
        dict(name="gemm_wgrad_small", op="gemm_wgrad", T=1000, E=8, top=2, N=520, K=1000, m=8, dtype="bf16",
             gdtype="bf16", skew=True),
        # between FC1 and FC2 in training, dsv3 widths: probabilities inside the expert
        dict(name="swiglu_train", op="swiglu", T=8192, E=256, top=8, I=2048, m=32, dtype="bf16", probs=True,
             skew=True),
        # its gradient, and that of the probabilities
        dict(name="swiglu_bwd_train", op="swiglu_bwd", T=8192, E=256, top=8, I=2048, m=32, dtype="bf16", probs=True,
             skew=True),
        # one decoded token: residual sum, norm for the router and the 8-bit rows for the experts
        dict(name="rms_decode1", op="rms", rows=1, H=7168, dtype="bf16", pdtype="bf16", residual=True, rstd=False,
             y=True, codes=True),
        # the same for a prompt or a training step
        dict(name="rms_train", op="rms", rows=8192, H=7168, dtype="bf16", pdtype="bf16", residual=True, rstd=True,
             y=True, codes=True),
        # its backward pass, fp32 master weights, the residual stream's gradient joined
        dict(name="rms_bwd_train", op="rms_bwd", rows=8192, H=7168, dtype="bf16", pdtype="f32", grad_sum=True),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    return min(max(v, lo), hi)


def _width(rng, lo, hi):
    """A matrix's side: mostly a multiple of 128 or of 8, at times any number."""
    v, step = _log(rng, lo, hi), rng.choice([128, 128, 8, 8, 1])
    return max(v // step * step, lo)


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm_dgrad", "gemm_dgrad", "gemm_wgrad", "gemm_wgrad", "swiglu", "swiglu_bwd",
                     "rms", "rms_bwd"])
    if op in ("rms", "rms_bwd"):
        H = _width(rng, 64, 16384)
        dtype = rng.choice(["bf16", "f16", "f32"])
        rows = max(1, min(_log(rng, 1, 65536), 8192 * 7168 // H // (2 if dtype == "f32" else 1)))
        pdtype = rng.choice([dtype, "f32"])
        if op == "rms_bwd":
            return dict(op=op, rows=rows, H=H, dtype=dtype, pdtype=pdtype, grad_sum=rng.random() < 0.5)
        kind = rng.choice(["y", "codes", "both"])
        return dict(op=op, rows=rows, H=H, dtype=dtype, pdtype=pdtype, residual=rng.random() < 0.5,
                    rstd=rng.random() < 0.5, y=kind != "codes", codes=kind != "y")
    E = rng.choice([1, 4, 8, 16, 32, 64, 128, 256])
    top, T = min(E, rng.choice([1, 2, 4, 8])), _log(rng, 1, 8192)
    c = dict(op=op, T=T, E=E, top=top, m=rng.choice([1, 8, 32]), skew=T >= 512 and rng.random() < 0.5)
    if op in ("swiglu", "swiglu_bwd"):
        return dict(c, I=_width(rng, 64, 4096), dtype=rng.choice(["bf16", "f16", "f32"]), probs=rng.random() < 0.5)
    c.update(N=_width(rng, 64, 8192), K=_width(rng, 64, 8192), dtype=rng.choice(["bf16", "f16"]))
    while E * c["N"] * c["K"] > 2e9:  # weights of 4 GB at the most
        c["N"], c["K"] = max(c["N"] // 2, 64), max(c["K"] // 2, 64)
    while c["T"] * top * c["N"] * c["K"] > 1e12:
        c["T"] //= 2
    c["skew"] = c["skew"] and c["T"] >= 512
    if op == "gemm_wgrad":
        c["gdtype"] = rng.choice(["f32", c["dtype"]])
    return c


# -------------------------------------------------------------------- inputs

def _gen(seed, stream):
    return torch.Generator(device=DEV).manual_seed((seed * 1000003 + stream * 7919) & 0x7FFFFFFFFFFF)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _plan(c, seed):
    """Routing of the tokens and the padded segments it gives: (ids [T][top] ascending, rows, segments, row of each
    route in segment order, its token); rows is the buffer's capacity."""
    r = np.random.default_rng([seed, 11])
    T, E, top, m = c["T"], c["E"], c["top"], c["m"]
    score = r.gumbel(size=(T, E))
    if c["skew"]:  # popularity falls with the rank, ranks in random order
        score += -1.2 * np.log(1.0 + r.permutation(E))
    ids = np.sort(np.argpartition(-score, top - 1, axis=1)[:, :top], axis=1)
    counts = np.bincount(ids.reshape(-1), minlength=E)
    offsets = np.concatenate([[0], np.cumsum((counts + m - 1) // m * m)])
    order = np.argsort(ids.reshape(-1), kind="stable")
    expert = ids.reshape(-1)[order]
    first = np.concatenate([[0], np.cumsum(counts)])
    rows = offsets[expert] + np.arange(T * top) - first[expert]
    segments = [(e, int(offsets[e]), int(counts[e])) for e in range(E) if counts[e]]
    return ids.astype(np.int16), T * top + E * (m - 1), segments, rows, order // top


def _routed(s, c, seed):
    """The plan of the state; rows of it as an index of the device."""
    ids, s["cap"], s["segments"], rows, tokens = _plan(c, seed)
    s["rows"] = torch.from_numpy(rows).to(DEV)
    if own:
        moe = _moe()
        s["shape"] = moe.Shape(T=c["T"], H=128, E=c["E"], K=c["top"])
        s["layout"] = moe.Layout(c["m"], s["cap"])
        s["handle"] = moe.Handle.empty(s["shape"], s["layout"], DEV)
        ws = torch.empty(moe.moe_preprocess_workspace_size(s["shape"]), dtype=torch.uint8, device=DEV)
        moe.moe_preprocess(moe.Routing(moe.ROUTING_DENSE_I16, torch.from_numpy(ids).to(DEV)), s["shape"],
                           s["layout"], s["handle"], ws)
    return torch.from_numpy(tokens).to(DEV)


def _spread(s, values):
    """A buffer of the plan's rows that holds `values` [routes, ..] in its segments and zeros in its pad rows."""
    out = torch.zeros(s["cap"], *values.shape[1:], dtype=values.dtype, device=DEV)
    out[s["rows"]] = values
    return out


def _norm_rows(c, seed):
    """Hidden states with a few loud channels, as a residual stream has."""
    g = _gen(seed, 1)
    loud = torch.exp(0.5 * _randn(g, c["H"]))
    x = (_randn(g, c["rows"], c["H"]) * loud).to(TORCH[c["dtype"]])
    return g, x, (1.0 + 0.2 * _randn(g, c["H"])).to(TORCH[c["pdtype"]])


def prepare(case, seed):
    c = dict(case)
    s, op = dict(case=c), c["op"]
    if op.startswith("gemm"):
        tokens = _routed(s, c, seed)
        g, dt, N, K = _gen(seed, 2), TORCH[c["dtype"]], c["N"], c["K"]
        if op != "gemm_dgrad":
            s["x"] = _spread(s, _randn(g, c["T"], K, dtype=dt)[tokens])
        if op != "gemm":
            s["gy"] = _spread(s, _randn(g, c["T"], N, dtype=dt)[tokens])
        if op != "gemm_wgrad":
            s["w"] = _randn(g, c["E"], N, K, dtype=dt).mul_((K if op == "gemm" else N) ** -0.5)
        if own:
            moe = _moe()
            if op == "gemm_wgrad":
                s["out"] = torch.empty(c["E"], N, K, dtype=TORCH[c["gdtype"]], device=DEV)
            else:  # rows outside the routed ones belong to the caller and keep what they hold
                s["out"] = torch.zeros(s["cap"], N if op == "gemm" else K, dtype=dt, device=DEV)
            s["ws"] = torch.empty(moe.moe_grouped_gemm_workspace_size(s["shape"], s["layout"], N, K),
                                  dtype=torch.uint8, device=DEV)
    elif op.startswith("swiglu"):
        tokens = _routed(s, c, seed)
        g, dt, n = _gen(seed, 3), TORCH[c["dtype"]], tokens.shape[0]
        s["pre"] = _spread(s, (1.5 * _randn(g, n, 2 * c["I"])).to(dt))
        s["probs"] = _spread(s, torch.rand(n, generator=g, device=DEV)) if c["probs"] else None
        if op == "swiglu_bwd":
            s["ga"] = _spread(s, _randn(g, n, c["I"]).to(dt))
        if own:
            s["out"] = torch.zeros(s["cap"], c["I"] * (1 if op == "swiglu" else 2), dtype=dt, device=DEV)
            s["gp"] = torch.zeros(s["cap"], device=DEV) if c["probs"] and op == "swiglu_bwd" else None
    elif op == "rms":
        g, s["x"], s["w"] = _norm_rows(c, seed)
        s["residual"] = (2.0 * _randn(g, c["rows"], c["H"])).to(s["x"].dtype) if c["residual"] else None
        if own:
            s["y"] = torch.empty_like(s["x"]) if c["y"] else None
            s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
            s["rstd"] = torch.empty(c["rows"], device=DEV) if c["rstd"] else None
            s["codes"] = torch.empty(c["rows"], c["H"], dtype=torch.float8_e4m3fn, device=DEV) if c["codes"] else None
            s["scales"] = torch.empty(c["rows"], -(-c["H"] // BLOCK), device=DEV) if c["codes"] else None
    elif op == "rms_bwd":
        g, s["x"], s["w"] = _norm_rows(c, seed)
        s["gy"] = _randn(g, c["rows"], c["H"]).to(s["x"].dtype)
        s["gsum"] = _randn(g, c["rows"], c["H"]).to(s["x"].dtype) if c["grad_sum"] else None
        # the statistic that the forward pass kept
        s["rstd"] = torch.rsqrt(s["x"].double().square_().mean(1) + EPS).float()
        if own:
            moe = _moe()
            s["gx"], s["gw"] = torch.empty_like(s["x"]), torch.empty(c["H"], device=DEV)
            s["ws"] = torch.empty(moe.moe_rms_norm_workspace_size(c["rows"], c["H"]), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    return (_RUN_OWN if own else _RUN_PLAIN)[op](state, state["case"])


def _own_gemm(s, c):
    _moe().moe_grouped_gemm(s["handle"], s["shape"], s["layout"], s["w"], s["x"], s["out"], s["ws"])
    return [s["out"]]


def _own_gemm_dgrad(s, c):
    _moe().moe_grouped_gemm_backward_data(s["handle"], s["shape"], s["layout"], s["w"], s["gy"], s["out"], s["ws"])
    return [s["out"]]


def _own_gemm_wgrad(s, c):
    _moe().moe_grouped_gemm_backward_weight(s["handle"], s["shape"], s["layout"], s["x"], s["gy"], s["out"], s["ws"])
    return [s["out"]]


def _own_swiglu(s, c):
    _moe().moe_swiglu(s["handle"], s["shape"], s["layout"], s["pre"], s["out"], probs=s["probs"])
    return [s["out"]]


def _own_swiglu_bwd(s, c):
    _moe().moe_swiglu_backward(s["handle"], s["shape"], s["layout"], s["pre"], s["ga"], s["out"], probs=s["probs"],
                               grad_probs=s["gp"])
    return [s["out"], s["gp"]] if c["probs"] else [s["out"]]


def _own_rms(s, c):
    _moe().moe_rms_norm(s["x"], s["w"], EPS, s["y"], residual=s["residual"], sum_out=s["sum"], rstd=s["rstd"],
                        codes=s["codes"], scales=s["scales"])
    return [s[k] for k in ("y", "codes", "scales", "sum", "rstd") if s[k] is not None]


def _own_rms_bwd(s, c):
    _moe().moe_rms_norm_backward(s["gy"], s["x"], s["w"], s["rstd"], s["gx"], grad_weight=s["gw"], workspace=s["ws"],
                                 grad_sum=s["gsum"])
    return [s["gx"], s["gw"]]


_RUN_OWN = dict(gemm=_own_gemm, gemm_dgrad=_own_gemm_dgrad, gemm_wgrad=_own_gemm_wgrad, swiglu=_own_swiglu,
                swiglu_bwd=_own_swiglu_bwd, rms=_own_rms, rms_bwd=_own_rms_bwd)


def _plain_gemm(s, c):
    y = torch.zeros(s["cap"], c["N"], dtype=s["x"].dtype, device=DEV)
    for e, beg, n in s["segments"]:
        y[beg:beg + n] = s["x"][beg:beg + n].float() @ s["w"][e].float().T
    return [y]


def _plain_gemm_dgrad(s, c):
    gx = torch.zeros(s["cap"], c["K"], dtype=s["gy"].dtype, device=DEV)
    for e, beg, n in s["segments"]:
        gx[beg:beg + n] = s["gy"][beg:beg + n].float() @ s["w"][e].float()
    return [gx]


def _plain_gemm_wgrad(s, c):
    gw = torch.zeros(c["E"], c["N"], c["K"], dtype=TORCH[c["gdtype"]], device=DEV)
    for e, beg, n in s["segments"]:
        gw[e] = s["gy"][beg:beg + n].float().T @ s["x"][beg:beg + n].float()
    return [gw]


def _plain_swiglu(s, c):
    # columns 0..I-1 are up, I..2I-1 gate (the w3_w1 order of the grouped MLP)
    up, gate = s["pre"].float().chunk(2, dim=1)
    a = gate / (1.0 + torch.exp(-gate)) * up
    if c["probs"]:
        a = a * s["probs"][:, None]
    return [a.to(s["pre"].dtype)]


def _plain_swiglu_bwd(s, c):
    up, gate = s["pre"].float().chunk(2, dim=1)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    act, ga = gate * sig, s["ga"].float()
    gp = (ga * act * up).sum(1)
    if c["probs"]:
        ga = ga * s["probs"][:, None]
    out = torch.cat([ga * act, ga * up * sig * (1.0 + gate * (1.0 - sig))], 1).to(s["pre"].dtype)
    return [out, gp] if c["probs"] else [out]


def _plain_rms(s, c):
    x = s["x"]
    if c["residual"]:  # the norm reads the sum as it is stored
        x = (x.float() + s["residual"].float()).to(x.dtype)
    h = x.float()
    rstd = 1.0 / torch.sqrt((h * h).sum(1) / c["H"] + EPS)
    v = h * rstd[:, None] * s["w"].float()
    out = [v.to(x.dtype)] if c["y"] else []
    if c["codes"]:  # of the row before its rounding to the output's type
        full = -(-c["H"] // BLOCK) * BLOCK
        b = v if full == c["H"] else torch.cat([v, v.new_zeros(c["rows"], full - c["H"])], 1)
        b = b.view(c["rows"], -1, BLOCK)
        scale = b.abs().amax(2) / 448.0
        scale = torch.where(scale == 0, 1.0, scale)
        codes = (b / scale[:, :, None]).clamp(-448.0, 448.0).view(c["rows"], -1)[:, :c["H"]]
        out += [codes.to(torch.float8_e4m3fn), scale]
    out += [x] if c["residual"] else []
    return out + [rstd] if c["rstd"] else out


def _plain_rms_bwd(s, c):
    gy, rstd = s["gy"].float(), s["rstd"][:, None]
    xhat = s["x"].float() * rstd
    u = gy * s["w"].float()
    gx = rstd * (u - xhat * ((u * xhat).sum(1, keepdim=True) / c["H"]))
    if c["grad_sum"]:
        gx = gx + s["gsum"].float()
    return [gx.to(s["x"].dtype), (gy * xhat).sum(0)]


_RUN_PLAIN = dict(gemm=_plain_gemm, gemm_dgrad=_plain_gemm_dgrad, gemm_wgrad=_plain_gemm_wgrad, swiglu=_plain_swiglu,
                  swiglu_bwd=_plain_swiglu_bwd, rms=_plain_rms, rms_bwd=_plain_rms_bwd)


# ----------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    global own
    keep, own = own, False  # inputs only: no library objects
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    return _EXACT[case["op"]](s, case)


def _exact_gemm(s, c):
    """Every matrix product as one contraction an expert, in blocks of features."""
    f64 = dict(dtype=torch.float64, device=DEV)
    if c["op"] == "gemm_wgrad":
        out = torch.zeros(c["E"], c["N"], c["K"], **f64)
        for e, beg, n in s["segments"]:
            torch.mm(s["gy"].narrow(0, beg, n).t().double(), s["x"].narrow(0, beg, n).double(), out=out[e])
        return [out]
    forward = c["op"] == "gemm"
    a = s["x"] if forward else s["gy"]
    out = torch.zeros(s["cap"], c["N"] if forward else c["K"], **f64)
    for e, beg, n in s["segments"]:
        w = s["w"][e].double()
        torch.mm(a.narrow(0, beg, n).double(), w.t() if forward else w, out=out.narrow(0, beg, n))
    return [out]


def _exact_swiglu(s, c):
    I = c["I"]
    a = torch.nn.functional.silu(s["pre"][:, I:].double()).mul_(s["pre"][:, :I].double())
    return [a.mul_(s["probs"].double().unsqueeze(1)) if c["probs"] else a]


def _exact_swiglu_bwd(s, c):
    with torch.enable_grad():
        pre = s["pre"].double().requires_grad_(True)
        a = torch.nn.functional.silu(pre[:, c["I"]:]) * pre[:, :c["I"]]
        if not c["probs"]:
            return [torch.autograd.grad(a, pre, s["ga"].double())[0]]
        p = s["probs"].double().requires_grad_(True)
        return list(torch.autograd.grad(a * p[:, None], (pre, p), s["ga"].double()))


def _exact_rms(s, c):
    h, out = s["x"].double(), []
    if c["residual"]:
        h = h + s["residual"].double()
    total = h
    h = h.to(s["x"].dtype).double()  # the norm is defined on the sum as stored
    rstd = (torch.linalg.vector_norm(h, dim=1).square() / c["H"] + EPS) ** -0.5
    v = torch.einsum("rh,r,h->rh", h, rstd, s["w"].double())
    if c["y"]:
        out.append(v)
    if c["codes"]:
        scale = torch.stack([p.abs().amax(1) for p in v.split(BLOCK, dim=1)], 1) / 448.0
        scale = torch.where(scale == 0, 1.0, scale)
        out += [v / scale.repeat_interleave(BLOCK, dim=1)[:, :c["H"]], scale]
    if c["residual"]:
        out.append(total)
    return out + [rstd] if c["rstd"] else out


def _exact_rms_bwd(s, c):
    # the Jacobian of h -> h rstd(h) w, applied to gy
    g, h, r = s["gy"].double(), s["x"].double(), s["rstd"].double()
    u = g * s["w"].double()
    gx = torch.einsum("rh,r->rh", u, r) - torch.einsum("rh,r->rh", h, r ** 3 * torch.einsum("rh,rh->r", u, h) / c["H"])
    if c["grad_sum"]:
        gx = gx + s["gsum"].double()
    return [gx, torch.einsum("rh,rh,r->h", g, h, r)]


_EXACT = dict(gemm=_exact_gemm, gemm_dgrad=_exact_gemm, gemm_wgrad=_exact_gemm, swiglu=_exact_swiglu,
              swiglu_bwd=_exact_swiglu_bwd, rms=_exact_rms, rms_bwd=_exact_rms_bwd)


# ---------------------------------------------------------------------- work

def work(case):
    """Each input read once and each output written once; one operation per product and per sum."""
    c = case
    op = c["op"]
    if op in ("rms", "rms_bwd"):
        n, b, p = c["rows"] * c["H"], BYTES[c["dtype"]], BYTES[c["pdtype"]]
        if op == "rms_bwd":
            return {"bytes": n * b * (4 if c["grad_sum"] else 3) + c["H"] * (p + 4) + 4 * c["rows"], "flops": n * 11}
        nbytes = n * b * ((3 if c["residual"] else 1) + (1 if c["y"] else 0)) + c["H"] * p
        if c["codes"]:
            nbytes += n + 4 * c["rows"] * -(-c["H"] // BLOCK)
        return {"bytes": nbytes + (4 * c["rows"] if c["rstd"] else 0), "flops": n * (5 + (2 if c["codes"] else 0))}
    rows = c["T"] * c["top"]
    if op in ("swiglu", "swiglu_bwd"):
        n, b = rows * c["I"], BYTES[c["dtype"]]
        if op == "swiglu":
            return {"bytes": n * b * 3 + (4 * rows if c["probs"] else 0), "flops": n * 6}
        return {"bytes": n * b * 5 + (8 * rows if c["probs"] else 0), "flops": n * 14}
    flops = 2 * rows * c["N"] * c["K"]
    if op == "gemm_wgrad":
        return {"bytes": c["E"] * c["N"] * c["K"] * BYTES[c["gdtype"]] + rows * (c["N"] + c["K"]) * 2, "flops": flops}
    active = c["E"] * (1.0 - (1.0 - c["top"] / c["E"]) ** c["T"])  # experts some token is expected to reach
    return {"bytes": int(active * c["N"] * c["K"] * 2) + rows * (c["N"] + c["K"]) * 2, "flops": flops}
