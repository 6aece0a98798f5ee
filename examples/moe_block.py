"""A pre-norm MoE block around the library's dispatch -> experts -> combine path.

    python examples/moe_block.py

* ``decode_step``: the block of one decode step, routed experts and a shared
  expert with 4-bit weights:
      s = x + residual,  h = layer_norm(s)
      s + sum over the routes of p_k expert_k(h) + shared(h)
* ``TrainBlock``: forward and backward of the block in training, with identity
  experts (the expert MLP's own backward is not part of the library):
      y = s + sum over the routes of p_k h,  gradients of x, norm and router

The router's linear layer is the model's own (a torch product); everything
else runs in the library's kernels, stream-ordered and without host
synchronisation, so that a step can be captured in one CUDA graph.
"""
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import permute_grouped_expert_gb300 as moe  # noqa: E402

EPS = 1e-5


def _bf16(*shape, device="cuda"):
    return torch.empty(*shape, dtype=torch.bfloat16, device=device)


def quantized(w: torch.Tensor, group: int, zero_points: bool = True) -> moe.W4Weight:
    """The 4-bit weights of bf16 matrices [.., N, Kd]."""
    *lead, N, Kd = w.shape
    G = -(-Kd // group)
    u8 = dict(dtype=torch.uint8, device=w.device)
    q = moe.W4Weight(torch.empty(*lead, N, Kd // 2, **u8), _bf16(*lead, N, G, device=w.device),
                     torch.empty(*lead, N, (G + 1) // 2, **u8) if zero_points else None, group)
    moe.moe_quantize_w4_rows(w.contiguous(), group, q.codes, q.scales, q.zeros)
    return q


@dataclasses.dataclass
class Weights:
    """Weights of a decode block: norm, router, routed experts and the shared expert."""
    norm_w: torch.Tensor       # [H]
    norm_b: torch.Tensor       # [H]
    router: torch.Tensor       # [E, H]
    w13: moe.W4Weight          # [E, 2I, H]
    w2: moe.W4Weight           # [E, H, I]
    shared_w13: moe.W4Weight   # [2I, H]
    shared_w2: moe.W4Weight    # [H, I]


class DecodeBlock:
    """The block at a fixed number of tokens, with the buffers a step needs."""

    def __init__(self, weights: Weights, T: int, K: int, pad_multiple: int = 8):
        self.w = weights
        E, H = weights.router.shape
        I = weights.shared_w2.codes.shape[-1] * 2
        cap = T * K + E * (pad_multiple - 1)
        dev = weights.router.device
        self.shape, self.layout = moe.Shape(T, H, E, K), moe.Layout(pad_multiple, cap)
        self.cfg = moe.Router(E, K)
        self.sum, self.h = _bf16(T, H), _bf16(T, H)
        self.logits = _bf16(T, E)
        self.routing = moe.Routing(moe.ROUTING_DENSE_I16, torch.empty(T, K, dtype=torch.int16, device=dev),
                                   torch.empty(T, K, device=dev))
        self.handle = moe.Handle.empty(self.shape, self.layout, dev)
        self.ws = torch.empty(moe.moe_preprocess_workspace_size(self.shape), dtype=torch.uint8, device=dev)
        self.rows, self.probs = _bf16(cap, H), torch.empty(cap, device=dev)
        self.act, self.out_rows = _bf16(cap, I), _bf16(cap, H)
        self.shared_act, self.y = _bf16(T, I), _bf16(T, H)

    def step(self, x: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
        w = self.w
        moe.moe_layer_norm(x, w.norm_w, w.norm_b, EPS, self.h, residual=residual, sum_out=self.sum)
        torch.matmul(self.h, w.router.T, out=self.logits)
        moe.moe_router_topk(self.cfg, self.logits, self.routing)
        moe.moe_preprocess(self.routing, self.shape, self.layout, self.handle, self.ws)
        moe.moe_dispatch_permute(self.handle, self.shape, self.layout, moe.DTYPE_BF16, self.h, None, self.routing,
                                 self.rows, self.probs)
        moe.moe_grouped_w4_matvec(self.handle, self.shape, self.layout, w.w13, self.rows, self.act, moe.W4_SWIGLU)
        moe.moe_grouped_w4_matvec(self.handle, self.shape, self.layout, w.w2, self.act, self.out_rows)
        moe.moe_combine_unpermute(self.handle, self.shape, self.layout, self.out_rows, self.probs, self.y)
        # the shared expert on top, then the residual stream
        moe.moe_w4_matvec(w.shared_w13, self.h, self.shared_act, moe.W4_SWIGLU)
        moe.moe_w4_matvec(w.shared_w2, self.shared_act, self.y, addend=self.y)
        return self.y.add_(self.sum)


class TrainBlock:
    """Forward and backward of the block with identity experts."""

    def __init__(self, norm_w, norm_b, router, T: int, K: int, pad_multiple: int = 32):
        self.norm_w, self.norm_b, self.router = norm_w, norm_b, router
        E, H = router.shape
        cap = T * K + E * (pad_multiple - 1)
        dev = router.device
        f32 = dict(dtype=torch.float32, device=dev)
        self.shape, self.layout = moe.Shape(T, H, E, K), moe.Layout(pad_multiple, cap)
        self.cfg = moe.Router(E, K, renormalize=False)
        self.routing = moe.Routing(moe.ROUTING_DENSE_I16, torch.empty(T, K, dtype=torch.int16, device=dev),
                                   torch.empty(T, K, **f32))
        self.handle = moe.Handle.empty(self.shape, self.layout, dev)
        self.ws = torch.empty(moe.moe_preprocess_workspace_size(self.shape), dtype=torch.uint8, device=dev)
        self.norm_ws = torch.empty(moe.moe_layer_norm_workspace_size(T, H), dtype=torch.uint8, device=dev)
        self.sum, self.h, self.y = _bf16(T, H), _bf16(T, H), _bf16(T, H)
        self.mean, self.rstd = torch.empty(T, **f32), torch.empty(T, **f32)
        self.rows, self.probs = _bf16(cap, H), torch.empty(cap, **f32)
        self.g_rows, self.g_probs_rows = _bf16(cap, H), torch.empty(cap, **f32)
        self.g_h, self.g_probs = _bf16(T, H), torch.empty(T, K, **f32)
        self.g_logits = torch.empty(T, E, **f32)
        self.g_x = _bf16(T, H)
        self.g_norm_w, self.g_norm_b = torch.empty(H, **f32), torch.empty(H, **f32)

    def forward(self, x: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
        moe.moe_layer_norm(x, self.norm_w, self.norm_b, EPS, self.h, residual=residual, sum_out=self.sum,
                           mean=self.mean, rstd=self.rstd)
        self.logits = self.h.float() @ self.router.T
        moe.moe_router_topk(self.cfg, self.logits, self.routing)
        moe.moe_preprocess(self.routing, self.shape, self.layout, self.handle, self.ws)
        moe.moe_dispatch_permute(self.handle, self.shape, self.layout, moe.DTYPE_BF16, self.h, None, self.routing,
                                 self.rows, self.probs)
        moe.moe_combine_unpermute(self.handle, self.shape, self.layout, self.rows, self.probs, self.y)
        return self.y + self.sum

    def backward(self, g_out: torch.Tensor):
        """(grad of x and of the residual, of the norm's weight and bias, of the router)"""
        moe.moe_combine_backward(self.handle, self.shape, self.layout, g_out, self.rows, self.probs, self.g_rows,
                                 self.g_probs_rows)
        moe.moe_dispatch_backward(self.handle, self.shape, self.layout, moe.ROUTING_DENSE_I16, self.g_rows,
                                  self.g_probs_rows, self.g_h, self.g_probs)
        moe.moe_router_topk_backward(self.cfg, self.logits, self.routing, self.g_probs, self.g_logits)
        g_router = self.g_logits.T @ self.h.float()
        self.g_h.add_((self.g_logits @ self.router).to(torch.bfloat16))
        moe.moe_layer_norm_backward(self.g_h, self.sum, self.norm_w, self.mean, self.rstd, self.g_x,
                                    grad_weight=self.g_norm_w, grad_bias=self.g_norm_b, workspace=self.norm_ws,
                                    grad_sum=g_out)
        return self.g_x, self.g_norm_w, self.g_norm_b, g_router


def random_weights(E: int, H: int, I: int, group: int, seed: int = 0) -> Weights:
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *shape, scale: (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)
    return Weights(1 + r(H, scale=0.1), r(H, scale=0.1), r(E, H, scale=H ** -0.5),
                   quantized(r(E, 2 * I, H, scale=H ** -0.5), group), quantized(r(E, H, I, scale=I ** -0.5), group),
                   quantized(r(2 * I, H, scale=H ** -0.5), group), quantized(r(H, I, scale=I ** -0.5), group))


def main():
    T, H, E, K, I = 64, 1024, 32, 4, 512
    block = DecodeBlock(random_weights(E, H, I, 128), T, K)
    x, residual = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, H, device="cuda").bfloat16()
    block.step(x, residual)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, residual)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(20):
        graph.replay()
    b.record()
    torch.cuda.synchronize()
    print(f"decode block: {T} tokens, {E} experts top-{K}: {a.elapsed_time(b) / 20 * 1e3:.1f} us a step, "
          f"output rms {y.float().square().mean().sqrt().item():.3f}")

    T = 2048
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    train = TrainBlock((1 + 0.1 * r(H)).bfloat16(), (0.1 * r(H)).bfloat16(), r(E, H) * H ** -0.5, T, K)
    out = train.forward(r(T, H).bfloat16(), r(T, H).bfloat16())
    grads = train.backward(r(T, H).bfloat16())
    print(f"train block: {T} tokens, output rms {out.float().square().mean().sqrt().item():.3f}, gradient norms " +
          ", ".join(f"{v.float().norm().item():.2f}" for v in grads))


if __name__ == "__main__":
    main()
