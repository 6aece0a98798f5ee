"""The experts' training operators and the RMS norm refuse every tensor that is not on the current device, before the
library is called: on the host, with stand-ins for tensors and the library."""
import pytest
import torch

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Tensor:
    """What the binding asks of a contiguous tensor, on a device of any number."""

    def __init__(self, dtype, *shape, device=1):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device

    is_cuda = property(lambda self: self.index >= 0)
    device = property(lambda self: torch.device("cuda", self.index) if self.is_cuda else torch.device("cpu"))

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def stride(self):
        return tuple(torch.empty(self.shape, device="meta").stride())

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 4096


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def moe(monkeypatch):
    import __graft_entry__

    __graft_entry__.build_library()
    import permute_grouped_expert_gb300 as m

    monkeypatch.setattr(m, "_lib", Library())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    return m


CAP, E, N, KD, T, H = 16, 3, 24, 40, 5, 256


def calls():
    """(call, its tensors); those of the handle under their own names."""
    handle = dict(tokens_per_expert=Tensor(I32, E), padded_offsets=Tensor(I32, E + 1), token_of=Tensor(I32, CAP),
                  status=Tensor(I32, 1))
    gemm = dict(workspace=Tensor(U8, 64))
    w, rows = Tensor(BF, E, N, KD), lambda c, t=BF: Tensor(t, CAP, c)
    yield "moe_grouped_gemm", handle, dict(gemm, weight=w, x=rows(KD), y=rows(N))
    yield "moe_grouped_gemm_backward_data", handle, dict(gemm, weight=w, grad_y=rows(N), grad_x=rows(KD))
    yield "moe_grouped_gemm_backward_weight", handle, dict(gemm, x=rows(KD), grad_y=rows(N), grad_weight=Tensor(F32, E, N, KD),
                                                           addend=Tensor(F32, E, N, KD))
    yield "moe_swiglu", handle, dict(pre=rows(2 * N), act=rows(N), probs=Tensor(F32, CAP))
    yield "moe_swiglu_backward", handle, dict(pre=rows(2 * N), grad_act=rows(N), grad_pre=rows(2 * N),
                                              probs=Tensor(F32, CAP), grad_probs=Tensor(F32, CAP))
    hidden = lambda: Tensor(BF, T, H)
    yield "moe_rms_norm", None, dict(x=hidden(), weight=Tensor(BF, H), y=hidden(), residual=hidden(), sum_out=hidden(),
                                     rstd=Tensor(F32, T), codes=Tensor(U8, T, H), scales=Tensor(F32, T, 2))
    yield "moe_rms_norm_backward", None, dict(grad_y=hidden(), h=hidden(), weight=Tensor(BF, H), rstd=Tensor(F32, T),
                                              grad_x=hidden(), grad_weight=Tensor(F32, H), workspace=Tensor(U8, 4096),
                                              grad_sum=hidden())


@pytest.mark.parametrize("name", [c[0] for c in calls()])
def test_tensors_of_another_device_are_refused(moe, name):
    _, handle, tensors = next(c for c in calls() if c[0] == name)

    def call(handle, tensors):
        at = {}
        if handle is not None:
            other = {k: Tensor(I32, 1) for k in ("row_of", "slot_of", "total_rows", "overflow")}
            at = dict(handle=moe.Handle(**handle, **other), shape=moe.Shape(T, 128, E, 1), layout=moe.Layout(1, CAP))
        if name == "moe_rms_norm":
            at["eps"] = 1e-6
        getattr(moe, name)(**at, **tensors, stream=0)

    call(handle, tensors)
    assert moe._lib.calls == [name]
    for group in filter(None, (handle, tensors)):
        for k, t in group.items():
            for index in (0, -1):
                moved = dict(group)
                moved[k] = Tensor(t.dtype, *t.shape, device=index)
                with pytest.raises(ValueError):
                    call(*((moved, tensors) if group is handle else (handle, moved)))
    assert moe._lib.calls == [name]
