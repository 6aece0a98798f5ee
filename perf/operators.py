"""The operators around the MoE layer's dispatch -> experts -> combine path, as cases to measure.

Three operators stand next to that path in a pre-norm MoE block:

* layer norm, forward (with the residual sum fused) and backward (with the
  reductions of the weight's and the bias's gradients);
* the router: top-k selection and route probabilities from the logits, written
  in the library's routing layouts, and the gradient of the logits;
* matrix-vector products with 4-bit weights and group scales: one weight matrix
  for a few tokens, or one matrix per expert over the dispatched rows, with the
  SwiGLU epilogue of the expert MLP.

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
EPS = 1e-5


def _moe():
    import permute_grouped_expert_gb300 as moe

    return moe


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step: the residual sum and the norm before the router
        dict(name="norm_decode1", op="norm", rows=1, H=7168, dtype="bf16", pdtype="bf16", residual=True, stats=False),
        # the norm before the MoE layer in training, DeepSeek-V3-like widths (dsv3 workload)
        dict(name="norm_train", op="norm", rows=8192, H=7168, dtype="bf16", pdtype="bf16", residual=True, stats=True),
        # its backward pass: fp32 master weights, the residual stream's gradient joined
        dict(name="norm_bwd_train", op="norm_bwd", rows=8192, H=7168, dtype="bf16", pdtype="f32", grad_sum=True),
        # an odd width and row count in full precision (a research-size model, no vector alignment)
        dict(name="norm_bwd_odd", op="norm_bwd", rows=1531, H=1537, dtype="f32", pdtype="f32", grad_sum=False),
        # decode batch of 64 tokens over 256 experts, top-8, weights renormalised over the chosen
        dict(name="router_decode64", op="router", T=64, E=256, K=8, dtype="f32", score="softmax", renorm=True,
             format="dense", masked=False),
        # the stress workload's routing (65536 tokens, 256 experts, top-36) with some experts masked off
        dict(name="router_stress", op="router", T=65536, E=256, K=36, dtype="f32", score="softmax", renorm=False,
             format="dense", masked=True),
        # gradient of the logits in training: sigmoid scores renormalised over 8 of 256, dense routing
        dict(name="router_bwd_dsv3", op="router_bwd", T=8192, E=256, K=8, dtype="f32", score="sigmoid", renorm=True,
             format="dense", masked=False),
        # gradient of the logits of the mid workload: sparse Boolean routing, softmax over all experts, bf16 logits
        dict(name="router_bwd_mid", op="router_bwd", T=4096, E=64, K=8, dtype="bf16", score="softmax", renorm=False,
             format="sparse", masked=False),
        # single-token decode of a shared expert's FC1 + SwiGLU (hidden 7168, intermediate 2048), group scales of 128
        dict(name="w4_decode1", op="w4", M=1, N=4096, K=7168, group=128, dtype="bf16", zeros=False, swiglu=True,
             addend=False),
        # a small batch on a ragged projection with zero points, groups of 64, added onto the residual stream
        dict(name="w4_batch13", op="w4", M=13, N=4099, K=8224, group=64, dtype="f16", zeros=True, swiglu=False,
             addend=True),
        # one decoded token through its 8 experts' FC2 (intermediate 2048 -> hidden 7168)
        dict(name="w4_experts_token1", op="w4_experts", T=1, E=256, top=8, N=7168, K=2048, group=128, dtype="bf16",
             zeros=False, swiglu=False, m=32),
        # 64 decoded tokens through their experts' FC1 + SwiGLU (decode64 workload), zero points
        dict(name="w4_experts_decode64", op="w4_experts", T=64, E=256, top=8, N=4096, K=7168, group=128,
             dtype="bf16", zeros=True, swiglu=True, m=32),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    v = min(max(v, lo), hi)
    return v + 1 if v == 3072 else v


def _odd_or_even(rng, v, step):
    """v as drawn (often odd), or rounded up to a multiple of step."""
    if rng.random() < 0.4:
        return v
    v = (v + step - 1) // step * step
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "router", "router_bwd", "w4", "w4_experts"])
    if op in ("norm", "norm_bwd"):
        H = min(_odd_or_even(rng, _log(rng, 64, 16384), 128), 16384)
        rows = max(1, min(_log(rng, 1, 65536), 8192 * 7168 // H))
        rows = rows - 1 if rows == 3072 else rows
        dtype = rng.choice(["bf16", "f16", "f32"])
        if dtype == "f32":
            rows = max(1, rows // 2)
        pdtype = rng.choice([dtype, "f32"])
        if op == "norm":
            return dict(op=op, rows=rows, H=H, dtype=dtype, pdtype=pdtype, residual=rng.random() < 0.5,
                        stats=rng.random() < 0.5)
        return dict(op=op, rows=rows, H=H, dtype=dtype, pdtype=pdtype, grad_sum=rng.random() < 0.5)
    if op in ("router", "router_bwd"):
        E = _odd_or_even(rng, _log(rng, 2, 1024), 8)
        E = min(E, 1024)
        T = max(1, min(_log(rng, 1, 131072), 65536 * 256 // E))
        T = T - 1 if T == 3072 else T
        K = min(E, _log(rng, 1, 40))
        return dict(op=op, T=T, E=E, K=K, dtype=rng.choice(["f32", "bf16", "f16"]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5,
                    format=rng.choice(["dense", "sparse"]), masked=op == "router" and rng.random() < 0.3)
    swiglu = rng.random() < 0.5
    group = rng.choice([32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    zeros = rng.random() < 0.5
    if op == "w4":
        N = _odd_or_even(rng, _log(rng, 256, 32768), 64)
        K = (_log(rng, 256, 16384) + 31) // 32 * 32
        K = K + 32 if K == 3072 else K
        N += N % 2 if swiglu else 0
        return dict(op=op, M=_log(rng, 1, 32), N=N, K=K, group=group, dtype=dtype, zeros=zeros, swiglu=swiglu,
                    addend=not swiglu and rng.random() < 0.5)
    E = rng.choice([8, 16, 32, 64, 128, 256])
    # hidden and intermediate sizes of the expert matrices: multiples of 128, as the path's shapes are
    K = (_log(rng, 256, 7168) + 127) // 128 * 128
    N = (_log(rng, 256, 7168) + 127) // 128 * 128
    K = K + 128 if K == 3072 else K
    N = N + 128 if N == 3072 else N
    return dict(op=op, T=_log(rng, 1, 64), E=E, top=rng.choice([1, 2, 4, 8]), N=N, K=K, group=group, dtype=dtype,
                zeros=zeros, swiglu=swiglu, m=rng.choice([1, 8, 32]))


# -------------------------------------------------------------------- inputs

def _gen(seed, stream):
    return torch.Generator(device=DEV).manual_seed((seed * 1000003 + stream * 7919) & 0x7FFFFFFFFFFF)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _norm_inputs(c, seed):
    """Hidden states with a few loud channels and a small mean, as a residual stream has."""
    g = _gen(seed, 1)
    dt, pt = TORCH[c["dtype"]], TORCH[c["pdtype"]]
    loud = torch.exp(0.5 * _randn(g, c["H"]))
    x = (_randn(g, c["rows"], c["H"]) * loud + 0.1).to(dt)
    w = (1.0 + 0.2 * _randn(g, c["H"])).to(pt)
    b = (0.1 * _randn(g, c["H"])).to(pt)
    return g, dt, x, w, b


def _router_logits(c, seed):
    g = _gen(seed, 2)
    logits = _randn(g, c["T"], c["E"])
    if c["masked"]:
        # experts switched off for some tokens, and a few padding tokens that go nowhere
        logits.masked_fill_(torch.rand(c["T"], c["E"], generator=g, device=DEV) < 0.2, float("-inf"))
        logits.masked_fill_(torch.rand(c["T"], 1, generator=g, device=DEV) < 0.01, float("-inf"))
    return g, logits.to(TORCH[c["dtype"]])


def _w4_weights(g, c, *lead):
    N, K, group = c["N"], c["K"], c["group"]
    G = (K + group - 1) // group
    codes = torch.randint(0, 256, (*lead, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = (0.004 * torch.exp(0.3 * _randn(g, *lead, N, G))).to(TORCH[c["dtype"]])
    zeros = torch.randint(0, 256, (*lead, N, (G + 1) // 2), generator=g, device=DEV,
                          dtype=torch.uint8) if c["zeros"] else None
    return codes, scales, zeros


def _expert_plan(c, seed):
    """Routing of the tokens and the padded segments it gives: ids [T][top] ascending, offsets, counts, row order."""
    r = np.random.default_rng([seed, 5])
    T, E, top, m = c["T"], c["E"], min(c["top"], c["E"]), c["m"]
    ids = np.sort(np.argsort(r.standard_normal((T, E)), axis=1)[:, :top], axis=1)
    counts = np.bincount(ids.reshape(-1), minlength=E)
    offsets = np.concatenate([[0], np.cumsum((counts + m - 1) // m * m)])
    cap = T * top + E * (m - 1)
    rows, tokens = [], []
    seen = np.zeros(E, np.int64)
    for t in range(T):
        for e in ids[t]:
            rows.append(int(offsets[e] + seen[e]))
            tokens.append(t)
            seen[e] += 1
    return ids.astype(np.int16), counts, offsets, cap, rows, tokens


def _expert_inputs(c, seed):
    g = _gen(seed, 4)
    ids, counts, offsets, cap, rows, tokens = _expert_plan(c, seed)
    x = _randn(g, c["T"], c["K"]).to(TORCH[c["dtype"]])
    xp = torch.zeros(cap, c["K"], dtype=x.dtype, device=DEV)
    xp[torch.tensor(rows, device=DEV)] = x[torch.tensor(tokens, device=DEV)]
    codes, scales, zeros = _w4_weights(g, c, c["E"])
    segments = [(e, int(offsets[e]), int(counts[e])) for e in range(c["E"]) if counts[e]]
    return ids, cap, xp, codes, scales, zeros, segments


def prepare(case, seed):
    c = dict(case)
    s = dict(case=c)
    op = c["op"]
    if op == "norm":
        g, dt, s["x"], s["w"], s["b"] = _norm_inputs(c, seed)
        s["residual"] = (2.0 * _randn(g, c["rows"], c["H"])).to(dt) if c["residual"] else None
        if own:
            s["y"] = torch.empty_like(s["x"])
            s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
            s["mean"] = torch.empty(c["rows"], device=DEV) if c["stats"] else None
            s["rstd"] = torch.empty(c["rows"], device=DEV) if c["stats"] else None
    elif op == "norm_bwd":
        g, dt, s["x"], s["w"], _ = _norm_inputs(c, seed)
        s["gy"] = _randn(g, c["rows"], c["H"]).to(dt)
        s["gsum"] = _randn(g, c["rows"], c["H"]).to(dt) if c["grad_sum"] else None
        x = s["x"].double()  # the statistics the forward pass kept
        mean = x.mean(1)
        s["mean"] = mean.float()
        s["rstd"] = torch.rsqrt(x.sub_(mean[:, None]).square_().mean(1) + EPS).float()
        del x
        if own:
            moe = _moe()
            s["gx"] = torch.empty_like(s["x"])
            s["gw"] = torch.empty(c["H"], device=DEV)
            s["gb"] = torch.empty(c["H"], device=DEV)
            s["ws"] = torch.empty(moe.moe_layer_norm_workspace_size(c["rows"], c["H"]), dtype=torch.uint8, device=DEV)
    elif op in ("router", "router_bwd"):
        g, s["logits"] = _router_logits(c, seed)
        T, E, K = c["T"], c["E"], c["K"]
        sparse = c["format"] == "sparse"
        if op == "router_bwd":
            ids = _top_ids(s["logits"].float(), K)
            if sparse:
                s["map"] = torch.zeros(T, E, dtype=torch.uint8, device=DEV).scatter_(1, ids, 1)
                # a sparse gradient carries zeros off the map, as the dispatch's backward writes it
                s["gp"] = _randn(g, T, E) * s["map"]
            else:
                s["map"] = ids.to(torch.int16)
                s["gp"] = _randn(g, T, K)
        if own:
            moe = _moe()
            s["cfg"] = moe.Router(E, K, score=moe.SCORE_SIGMOID if c["score"] == "sigmoid" else moe.SCORE_SOFTMAX,
                                  renormalize=c["renorm"], scale=1.0)
            fmt = moe.ROUTING_SPARSE_BOOL if sparse else moe.ROUTING_DENSE_I16
            if op == "router":
                s["map"] = torch.empty(T, E if sparse else K, dtype=torch.uint8 if sparse else torch.int16,
                                       device=DEV)
                s["routing"] = moe.Routing(fmt, s["map"], torch.empty(s["map"].shape, device=DEV))
            else:
                s["routing"] = moe.Routing(fmt, s["map"])
                s["gl"] = torch.empty_like(s["logits"])
    elif op == "w4":
        g = _gen(seed, 3)
        s["codes"], s["scales"], s["zeros"] = _w4_weights(g, c)
        s["x"] = _randn(g, c["M"], c["K"]).to(TORCH[c["dtype"]])
        n_out = c["N"] // 2 if c["swiglu"] else c["N"]
        s["addend"] = _randn(g, c["M"], n_out).to(TORCH[c["dtype"]]) if c["addend"] else None
        if own:
            moe = _moe()
            s["weight"] = moe.W4Weight(s["codes"], s["scales"], s["zeros"], c["group"])
            s["y"] = torch.empty(c["M"], n_out, dtype=s["x"].dtype, device=DEV)
    elif op == "w4_experts":
        ids, cap, s["x"], s["codes"], s["scales"], s["zeros"], s["segments"] = _expert_inputs(c, seed)
        n_out = c["N"] // 2 if c["swiglu"] else c["N"]
        if own:
            moe = _moe()
            s["weight"] = moe.W4Weight(s["codes"], s["scales"], s["zeros"], c["group"])
            s["shape"] = moe.Shape(T=c["T"], H=c["K"], E=c["E"], K=ids.shape[1])
            s["layout"] = moe.Layout(c["m"], cap)
            s["handle"] = moe.Handle.empty(s["shape"], s["layout"], DEV)
            ws = torch.empty(moe.moe_preprocess_workspace_size(s["shape"]), dtype=torch.uint8, device=DEV)
            moe.moe_preprocess(moe.Routing(moe.ROUTING_DENSE_I16, torch.from_numpy(ids).to(DEV)), s["shape"],
                               s["layout"], s["handle"], ws)
            # rows outside the routed ones belong to the caller and keep what they hold
            s["y"] = torch.zeros(cap, n_out, dtype=s["x"].dtype, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    return (_RUN_OWN if own else _RUN_PLAIN)[op](state, state["case"])


def _own_norm(s, c):
    _moe().moe_layer_norm(s["x"], s["w"], s["b"], EPS, s["y"], residual=s["residual"], sum_out=s["sum"],
                          mean=s["mean"], rstd=s["rstd"])
    out = [s["y"]]
    if c["residual"]:
        out.append(s["sum"])
    return out + [s["mean"], s["rstd"]] if c["stats"] else out


def _own_norm_bwd(s, c):
    _moe().moe_layer_norm_backward(s["gy"], s["x"], s["w"], s["mean"], s["rstd"], s["gx"], grad_weight=s["gw"],
                                   grad_bias=s["gb"], workspace=s["ws"], grad_sum=s["gsum"])
    return [s["gx"], s["gw"], s["gb"]]


def _own_router(s, c):
    _moe().moe_router_topk(s["cfg"], s["logits"], s["routing"])
    return [s["routing"].map, s["routing"].probs]


def _own_router_bwd(s, c):
    _moe().moe_router_topk_backward(s["cfg"], s["logits"], s["routing"], s["gp"], s["gl"])
    return [s["gl"]]


def _own_w4(s, c):
    moe = _moe()
    moe.moe_w4_matvec(s["weight"], s["x"], s["y"], activation=moe.W4_SWIGLU if c["swiglu"] else moe.W4_NONE,
                      addend=s["addend"])
    return [s["y"]]


def _own_w4_experts(s, c):
    moe = _moe()
    moe.moe_grouped_w4_matvec(s["handle"], s["shape"], s["layout"], s["weight"], s["x"], s["y"],
                              activation=moe.W4_SWIGLU if c["swiglu"] else moe.W4_NONE)
    return [s["y"]]


_RUN_OWN = dict(norm=_own_norm, norm_bwd=_own_norm_bwd, router=_own_router, router_bwd=_own_router_bwd, w4=_own_w4,
                w4_experts=_own_w4_experts)


def _plain_norm(s, c):
    # the norm reads the residual sum as it is stored
    x = s["x"]
    if c["residual"]:
        x = (x.float() + s["residual"].float()).to(x.dtype)
    h = x.float()
    mean = h.sum(1) / c["H"]
    d = h - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / c["H"] + EPS)
    y = (d * rstd[:, None] * s["w"].float() + s["b"].float()).to(x.dtype)
    out = [y, x] if c["residual"] else [y]
    return out + [mean, rstd] if c["stats"] else out


def _plain_norm_bwd(s, c):
    gy, w, rstd = s["gy"].float(), s["w"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    gw, gb = (gy * xhat).sum(0), gy.sum(0)
    gh = gy * w
    gx = rstd * (gh - gh.sum(1, keepdim=True) / c["H"] - xhat * ((gh * xhat).sum(1, keepdim=True) / c["H"]))
    if c["grad_sum"]:
        gx = gx + s["gsum"].float()
    return [gx.to(s["x"].dtype), gw, gb]


def _top_ids(l, K):
    """The K largest logits of each row, ties to the lowest index, as ascending expert ids; masked (-inf) experts
    are never chosen and leave -1 in the last slots."""
    E = l.shape[1]
    order = torch.sort(l, dim=1, descending=True, stable=True)
    ids = torch.where(torch.isinf(order.values[:, :K]), E, order.indices[:, :K])
    ids = torch.sort(ids, dim=1).values
    return torch.where(ids == E, -1, ids)


def _plain_router(s, c):
    l = s["logits"].float()
    ids = _top_ids(l, c["K"])
    kept = ids >= 0
    at = ids.clamp(min=0)
    chosen = l.gather(1, at).masked_fill(~kept, float("-inf"))
    if c["score"] == "softmax":
        base = chosen if c["renorm"] else l
        top = l.max(1, keepdim=True).values
        top = torch.where(torch.isinf(top), 0.0, top)
        z = torch.exp(base - top).sum(1, keepdim=True)
        p = torch.exp(chosen - top) / torch.where(z == 0, 1.0, z)
    else:
        p = 1.0 / (1.0 + torch.exp(-chosen))
        if c["renorm"]:
            z = p.sum(1, keepdim=True)
            p = p / torch.where(z == 0, 1.0, z)
    p = torch.where(kept, p, 0.0)
    if c["format"] == "dense":
        return [ids.to(torch.int16), p]
    T, E = l.shape
    m = torch.zeros(T, E + 1, dtype=torch.uint8, device=l.device).scatter_(1, torch.where(kept, ids, E), 1)
    ps = torch.zeros(T, E + 1, device=l.device).scatter_(1, torch.where(kept, ids, E), p)
    return [m[:, :E].contiguous(), ps[:, :E].contiguous()]


def _plain_router_bwd(s, c):
    l = s["logits"].float()
    if c["format"] == "dense":
        ids = s["map"].long()
        on = torch.zeros_like(l).scatter_(1, ids, 1.0)
        g = torch.zeros_like(l).scatter_(1, ids, s["gp"])
    else:
        on, g = s["map"].float(), s["gp"]
    if c["score"] == "softmax":
        e = torch.exp(l - l.max(1, keepdim=True).values)
        if c["renorm"]:
            e = e * on
        p = e / e.sum(1, keepdim=True)
        gl = p * (g * on - (g * on * p).sum(1, keepdim=True))
    else:
        sg = 1.0 / (1.0 + torch.exp(-l))
        if c["renorm"]:
            n = sg * on / (sg * on).sum(1, keepdim=True)
            gl = n * (1.0 - sg) * (g - (g * n).sum(1, keepdim=True))
        else:
            gl = sg * (1.0 - sg) * g * on
    return [gl.to(s["logits"].dtype)]


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)


def _plain_dequant(codes, scales, zeros, group):
    K, G = codes.shape[-1] * 2, scales.shape[-1]
    q = _nibbles(codes).float()
    z = _nibbles(zeros)[..., :G].float() if zeros is not None else torch.full_like(scales, 8.0, dtype=torch.float32)
    q = q - z.repeat_interleave(group, dim=-1)[..., :K]
    return q * scales.float().repeat_interleave(group, dim=-1)[..., :K]


def _plain_swiglu(v):
    # rows 0..I-1 of the weight are up, rows I..2I-1 gate (the w3_w1 order of the grouped MLP)
    up, gate = v.chunk(2, dim=-1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_w4(s, c):
    v = s["x"].float() @ _plain_dequant(s["codes"], s["scales"], s["zeros"], c["group"]).T
    if c["swiglu"]:
        v = _plain_swiglu(v)
    if c["addend"]:
        v = v + s["addend"].float()
    return [v.to(s["x"].dtype)]


def _plain_w4_experts(s, c):
    n_out = c["N"] // 2 if c["swiglu"] else c["N"]
    y = torch.zeros(s["x"].shape[0], n_out, dtype=s["x"].dtype, device=s["x"].device)
    for e, beg, n in s["segments"]:
        z = s["zeros"][e] if s["zeros"] is not None else None
        v = s["x"][beg:beg + n].float() @ _plain_dequant(s["codes"][e], s["scales"][e], z, c["group"]).T
        y[beg:beg + n] = _plain_swiglu(v) if c["swiglu"] else v
    return [y]


_RUN_PLAIN = dict(norm=_plain_norm, norm_bwd=_plain_norm_bwd, router=_plain_router, router_bwd=_plain_router_bwd,
                  w4=_plain_w4, w4_experts=_plain_w4_experts)


# ----------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    global own
    keep, own = own, False  # inputs only: no library objects
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    return _EXACT[case["op"]](s, case)


def _exact_norm(s, c):
    h = s["x"].double()
    out = []
    if c["residual"]:
        h = h + s["residual"].double()
        out = [h]
        h = h.to(s["x"].dtype).double()  # the norm is defined on the sum as stored
    var, mean = torch.var_mean(h, dim=1, unbiased=False)
    rstd = (var + EPS) ** -0.5
    y = torch.addcmul(s["b"].double(), (h - mean[:, None]) * rstd[:, None], s["w"].double())
    return [y] + out + ([mean, rstd] if c["stats"] else [])


def _exact_norm_bwd(s, c):
    # the Jacobian of (h - mean) * rstd applied to gy * w, one row at a time in matrix form
    g, x, rstd = s["gy"].double(), s["x"].double(), s["rstd"].double()
    xhat = torch.einsum("rh,r->rh", x - s["mean"].double().unsqueeze(1), rstd)
    gw, gb = torch.einsum("rh,rh->h", g, xhat), g.sum(0)
    u = g * s["w"].double()
    c1 = u.mean(1)
    c2 = torch.einsum("rh,rh->r", u, xhat) / c["H"]
    gx = torch.einsum("rh,r->rh", u - c1.unsqueeze(1) - xhat * c2.unsqueeze(1), rstd)
    if c["grad_sum"]:
        gx = gx + s["gsum"].double()
    return [gx, gw, gb]


def _exact_router(s, c):
    l = s["logits"].double()
    T, E = l.shape
    live = l > float("-inf")
    # rank of every expert: how many come before it (a larger logit, or an equal one at a lower index)
    order = torch.argsort(-l, dim=1, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, torch.arange(E, device=l.device).expand(T, E))
    on = (rank < c["K"]) & live
    if c["score"] == "softmax":
        p = torch.softmax(torch.where(on | ((not c["renorm"]) & live), l, float("-inf")), dim=1)
    else:
        p = torch.sigmoid(l)
        if c["renorm"]:
            p = p / (p * on).sum(1, keepdim=True)
    p = torch.where(on, p, 0.0)
    if c["format"] == "sparse":
        return [on.to(torch.uint8), p]
    slot = torch.where(on, torch.cumsum(on, 1) - 1, c["K"])
    eid = torch.arange(E, device=l.device).expand(T, E)
    ids = torch.full((T, c["K"] + 1), -1, dtype=torch.int64, device=l.device).scatter_(1, slot, eid)[:, :c["K"]]
    pd = torch.zeros(T, c["K"] + 1, dtype=torch.float64, device=l.device).scatter_(1, slot, p)[:, :c["K"]]
    ids[:, :] = torch.where(torch.arange(c["K"], device=l.device) < on.sum(1, keepdim=True), ids, -1)
    return [ids.to(torch.int16), pd]


def _exact_router_bwd(s, c):
    with torch.enable_grad():
        l = s["logits"].double().requires_grad_(True)
        on = s["map"] != 0 if c["format"] == "sparse" else None
        if on is None:
            on = torch.zeros(l.shape, dtype=torch.bool, device=l.device)
            on.scatter_(1, s["map"].long(), True)
        if c["score"] == "softmax":
            p = torch.softmax(l.masked_fill(~on, float("-inf")) if c["renorm"] else l, dim=1)
        else:
            p = torch.sigmoid(l)
            if c["renorm"]:
                p = p / (p * on).sum(1, keepdim=True)
        w = p.gather(1, s["map"].long()) if c["format"] == "dense" else torch.where(on, p, 0.0)
        return [torch.autograd.grad(w, l, s["gp"].double())[0]]


def _exact_product(x, codes, scales, zeros, group):
    """sum_k x[k] (q[k] - z) s, group by group."""
    K = x.shape[1]
    G = scales.shape[-1]
    v = 0.0
    x = x.double()
    for i in range(G):
        b = codes[:, i * group // 2:min((i + 1) * group, K) // 2]
        lo, hi = (b & 15).double(), (b >> 4).double()
        z = 8.0 if zeros is None else ((zeros[:, i // 2] >> (4 * (i % 2))) & 15).double()[:, None]
        part = x[:, i * group:min((i + 1) * group, K)]
        v = v + (part[:, 0::2] @ (lo - z).T + part[:, 1::2] @ (hi - z).T) * scales[:, i].double()
    return v


def _exact_swiglu(v):
    n = v.shape[-1] // 2
    return v[:, :n] * v[:, n:] * torch.sigmoid(v[:, n:])


def _exact_w4(s, c):
    v = _exact_product(s["x"], s["codes"], s["scales"], s["zeros"], c["group"])
    if c["swiglu"]:
        v = _exact_swiglu(v)
    return [v + s["addend"].double() if c["addend"] else v]


def _exact_w4_experts(s, c):
    n_out = c["N"] // 2 if c["swiglu"] else c["N"]
    y = torch.zeros(s["x"].shape[0], n_out, dtype=torch.float64, device=DEV)
    for e, beg, n in s["segments"]:
        v = _exact_product(s["x"][beg:beg + n], s["codes"][e], s["scales"][e],
                           None if s["zeros"] is None else s["zeros"][e], c["group"])
        y[beg:beg + n] = _exact_swiglu(v) if c["swiglu"] else v
    return [y]


_EXACT = dict(norm=_exact_norm, norm_bwd=_exact_norm_bwd, router=_exact_router, router_bwd=_exact_router_bwd,
              w4=_exact_w4, w4_experts=_exact_w4_experts)


# ---------------------------------------------------------------------- work

def work(case):
    """Each input read once and each output written once; one operation per product and per sum."""
    c = case
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        n, b, p = c["rows"] * c["H"], BYTES[c["dtype"]], BYTES[c["pdtype"]]
        if op == "norm":
            nbytes = n * b * (4 if c["residual"] else 2) + 2 * c["H"] * p + (8 * c["rows"] if c["stats"] else 0)
            return {"bytes": nbytes, "flops": n * (8 + (1 if c["residual"] else 0))}
        nbytes = n * b * (4 if c["grad_sum"] else 3) + c["H"] * (p + 8) + 8 * c["rows"]
        return {"bytes": nbytes, "flops": n * 15}
    if op in ("router", "router_bwd"):
        T, E, K = c["T"], c["E"], c["K"]
        routing = T * E * 5 if c["format"] == "sparse" else T * K * 6
        n = T * E * BYTES[c["dtype"]]
        if op == "router":
            return {"bytes": n + routing, "flops": 4 * T * E}
        # renormalised scores and sigmoids look at the chosen logits alone; the gradient is dense all the same
        dense_in = c["score"] == "softmax" and not c["renorm"]
        read = n if dense_in else T * K * BYTES[c["dtype"]]
        return {"bytes": read + n + routing, "flops": 6 * T * (E if dense_in else K)}
    G = (c["K"] + c["group"] - 1) // c["group"]
    matrix = c["N"] * (c["K"] // 2 + G * 2 + ((G + 1) // 2 if c["zeros"] else 0))
    n_out = c["N"] // 2 if c["swiglu"] else c["N"]
    if op == "w4":
        M = c["M"]
        return {"bytes": matrix + M * c["K"] * 2 + M * n_out * (4 if c["addend"] else 2),
                "flops": 2 * M * c["N"] * c["K"]}
    top = min(c["top"], c["E"])
    rows = c["T"] * top
    active = c["E"] * (1.0 - (1.0 - top / c["E"]) ** c["T"])  # experts some token is expected to reach
    return {"bytes": int(active * matrix) + rows * (c["K"] + n_out) * 2, "flops": 2 * rows * c["N"] * c["K"]}
