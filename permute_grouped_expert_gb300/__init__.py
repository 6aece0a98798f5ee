"""GB300-native (sm_103a) single-GPU MoE dispatch -> grouped expert MLP -> combine.

A thin ctypes binding over ``libmoe_gb300.so``, whose C ABI is declared in
``include/moe.h``.  The binding only marshals arguments: torch tensors become
device pointers, shapes become the C structs, and the current torch CUDA stream
becomes the ``stream`` argument.  Every step of the path runs in the library's
CUDA kernels; there is no CPU fallback.  If the library has not been built the
import fails with an explicit error.

The four calls of one MoE layer forward keep their C names:
``moe_preprocess``, ``moe_dispatch_permute``, ``moe_grouped_mlp`` and
``moe_combine_unpermute``.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gb300.so")

# --------------------------------------------------------------- C mirrors

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_CUDA = 3
MOE_ERR_WORKSPACE_TOO_SMALL = 4
MOE_ERR_RING_EARLY_REUSE = 5
MOE_ERR_RING_DOUBLE_RELEASE = 6

ROUTING_DENSE_I16 = 0
ROUTING_SPARSE_BOOL = 1

DTYPE_BF16 = 0
DTYPE_FP8_E4M3_B128 = 1
DTYPE_BF16_TO_FP8 = 2
DTYPE_NVFP4 = 3
DTYPE_BF16_TO_NVFP4 = 4

COMBINE_BF16 = 0
COMBINE_MXFP8 = 1
COMBINE_MXFP4 = 2

DEV_ERR_BAD_EXPERT = 1
DEV_ERR_TOO_MANY_ROUTES = 2
DEV_ERR_TIMEOUT = 4
DEV_ERR_BOUNDS = 8  # bounds-checked builds only
DEV_ERR_NAN_LOGIT = 16

ELEM_F32 = 0
ELEM_BF16 = 1
ELEM_F16 = 2

SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1

W4_NONE = 0
W4_SWIGLU = 1


class _Shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("E", ctypes.c_int64), ("K", ctypes.c_int64),
                ("I", ctypes.c_int64)]


class _Layout(ctypes.Structure):
    _fields_ = [("pad_multiple", ctypes.c_int64), ("capacity", ctypes.c_int64)]


class _Routing(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("map", ctypes.c_void_p), ("probs", ctypes.c_void_p)]


class _HandleDev(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("tokens_per_expert", "padded_offsets", "row_of", "token_of",
                                               "slot_of", "total_rows", "overflow", "status")]


class _Nvfp4Globals(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("fc1_input_scale", "fc2_input_scale", "w13_scale_2",
                                               "w2_scale_2")]


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64)]


class _Norm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("H", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class _Router(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int64), ("K", ctypes.c_int64),
                ("logits_dtype", ctypes.c_int32), ("score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class _W4(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("Kd", ctypes.c_int64), ("group", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p)]


# Every symbol include/moe.h declares, with its ctypes signature.
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SIGNATURES = {
    "moe_capacity": [_I64, ctypes.c_double, _I64, ctypes.POINTER(_I64)],
    "moe_routing_map_bytes": [ctypes.c_int32, _I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "moe_decode_bucket": [_I64, ctypes.POINTER(_I64), ctypes.c_int32, ctypes.POINTER(_I64)],
    "moe_last_cuda_error": [],
    "moe_status_string": [ctypes.c_int],
    "moe_preprocess_workspace_size": [ctypes.POINTER(_Shape), ctypes.POINTER(ctypes.c_size_t)],
    "moe_preprocess": [ctypes.POINTER(_Routing), ctypes.POINTER(_Shape), ctypes.POINTER(_Layout),
                       ctypes.POINTER(_HandleDev), _P, ctypes.c_size_t, _P],
    "moe_preprocess_noalloc": [ctypes.POINTER(_Routing), ctypes.POINTER(_Shape), ctypes.POINTER(_Layout),
                               ctypes.POINTER(_HandleDev), _P],
    "moe_dispatch_permute": [ctypes.POINTER(_HandleDev), ctypes.POINTER(_Shape), ctypes.POINTER(_Layout),
                             ctypes.c_int32, _P, _P, ctypes.POINTER(_Routing), _P, _P, _P, _P],
    "moe_combine_unpermute": [ctypes.POINTER(_HandleDev), ctypes.POINTER(_Shape), ctypes.POINTER(_Layout),
                              _P, _P, _P, _P],
    "moe_combine_backward": [ctypes.POINTER(_HandleDev), ctypes.POINTER(_Shape), ctypes.POINTER(_Layout),
                             _P, _P, _P, _P, _P, _P],
    "moe_dispatch_backward": [ctypes.POINTER(_HandleDev), ctypes.POINTER(_Shape), ctypes.POINTER(_Layout),
                              ctypes.c_int32, _P, _P, _P, _P, _P],
    "moe_grouped_mlp_workspace_size": [ctypes.POINTER(_Shape), ctypes.POINTER(_Layout), ctypes.c_int32,
                                       ctypes.POINTER(ctypes.c_size_t)],
    "moe_grouped_mlp": [ctypes.POINTER(_HandleDev), ctypes.POINTER(_Shape), ctypes.POINTER(_Layout),
                        ctypes.c_int32, _P, _P, _P, _P, _P, _P, ctypes.POINTER(_Nvfp4Globals), _P,
                        ctypes.c_size_t, _P, _P],
    "moe_grouped_mlp_ex": [ctypes.POINTER(_HandleDev), ctypes.POINTER(_Shape), ctypes.POINTER(_Layout),
                           ctypes.c_int32, _P, _P, _P, _P, _P, _P, ctypes.POINTER(_Nvfp4Globals), _P,
                           ctypes.c_size_t, ctypes.c_int32, _P, _P, _P, _P],
    "moe_combine_unpermute_fmt": [ctypes.POINTER(_HandleDev), ctypes.POINTER(_Shape), ctypes.POINTER(_Layout),
                                  ctypes.c_int32, _P, _P, _P, _P, _P],
    "moe_quantize_mx_rows": [_P, _I64, _I64, ctypes.c_int32, _P, _P, _P],
    "moe_grouped_mlp_kernel_count": [ctypes.POINTER(_Shape), ctypes.POINTER(_Layout), ctypes.c_int32,
                                     ctypes.POINTER(ctypes.c_int32)],
    "moe_profile_next_grouped_mlp": [_P, _P, _P],
    "moe_debug_next_grouped_mlp_silent_token_tile": [_I64],
    "moe_debug_preprocess_silent_tile": [ctypes.POINTER(_Routing), ctypes.POINTER(_Shape), ctypes.POINTER(_Layout),
                                         ctypes.POINTER(_HandleDev), _P, ctypes.c_size_t, ctypes.c_int64, _P],
    "moe_quantize_fp8_blocks": [_P, _I64, _I64, _I64, _P, _P, _P],
    "moe_quantize_nvfp4_rows": [_P, _I64, _I64, _P, _P, _P, _P],
    # descriptors (moe_norm, moe_router, moe_w4, moe_rows) by address
    "moe_layer_norm": [_P] * 10,
    "moe_layer_norm_workspace_size": [_I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "moe_layer_norm_backward": [_P] * 11 + [ctypes.c_size_t, _P],
    "moe_router_topk": [_P, _P, _P, ctypes.c_int32, _P, _P, _P, _P],
    "moe_router_topk_backward": [_P, _P, ctypes.c_int32, _P, _P, _P, _P],
    "moe_w4_matvec": [_P, _I64, _P, ctypes.c_int32, _P, _P, _P],
    "moe_grouped_w4_matvec": [ctypes.POINTER(_HandleDev), ctypes.POINTER(_Shape), ctypes.POINTER(_Layout), _P, _P,
                              ctypes.c_int32, _P, _P],
    "moe_quantize_w4_rows": [_P, _I64, _I64, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P],
    "moe_ring_create": [ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(_P)],
    "moe_ring_acquire": [_P, _P, ctypes.POINTER(ctypes.c_int32)],
    "moe_ring_release": [_P, ctypes.c_int32, _P],
    "moe_ring_destroy": [_P],
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; g.build()'` "
            "(nvcc, sm_103a) before using permute_grouped_expert_gb300")
    lib = ctypes.CDLL(LIB_PATH)
    for name, args in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name in ("moe_last_cuda_error", "moe_status_string") else ctypes.c_int
    return lib


_lib = _load()


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = _lib.moe_status_string(status).decode()
        if status == MOE_ERR_CUDA:
            msg += " (" + _lib.moe_last_cuda_error().decode() + ")"
        super().__init__(f"{what}: {msg}")
        self.status = status


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        # the handle of torch.cuda.current_stream() without building the stream object (3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ------------------------------------------------------------ public types

@dataclasses.dataclass(frozen=True)
class Shape:
    T: int
    H: int
    E: int
    K: int
    I: int = 0

    def c(self):
        return _Shape(self.T, self.H, self.E, self.K, self.I)


@dataclasses.dataclass(frozen=True)
class Layout:
    pad_multiple: int
    capacity: int

    def c(self):
        return _Layout(self.pad_multiple, self.capacity)


@dataclasses.dataclass
class Routing:
    """format: ROUTING_DENSE_I16 (map int16 [T, K], probs float [T, K]) or
    ROUTING_SPARSE_BOOL (map uint8 [T, E], probs float [T, E]); probs optional."""
    format: int
    map: torch.Tensor
    probs: Optional[torch.Tensor] = None

    def c(self):
        return _Routing(self.format, _ptr(self.map), _ptr(self.probs))


@dataclasses.dataclass
class Handle:
    """The device arrays moe_preprocess fills (see moe_handle_dev in moe.h)."""
    tokens_per_expert: torch.Tensor
    padded_offsets: torch.Tensor
    row_of: torch.Tensor
    token_of: torch.Tensor
    slot_of: torch.Tensor
    total_rows: torch.Tensor
    overflow: torch.Tensor
    status: torch.Tensor

    @staticmethod
    def empty(shape: Shape, layout: Layout, device="cuda") -> "Handle":
        i32 = dict(dtype=torch.int32, device=device)
        return Handle(
            tokens_per_expert=torch.empty(shape.E, **i32), padded_offsets=torch.empty(shape.E + 1, **i32),
            row_of=torch.empty(max(shape.T * shape.K, 1), **i32), token_of=torch.empty(max(layout.capacity, 1), **i32),
            slot_of=torch.empty(max(layout.capacity, 1), **i32), total_rows=torch.empty(1, **i32),
            overflow=torch.empty(1, **i32), status=torch.empty(1, **i32))

    def c(self):
        return _HandleDev(*(_ptr(getattr(self, f.name)) for f in dataclasses.fields(self)))


@dataclasses.dataclass
class Nvfp4Globals:
    fc1_input_scale: torch.Tensor  # float [1]
    fc2_input_scale: torch.Tensor  # float [1]
    w13_scale_2: torch.Tensor      # float [E]
    w2_scale_2: torch.Tensor       # float [E]

    def c(self):
        return _Nvfp4Globals(_ptr(self.fc1_input_scale), _ptr(self.fc2_input_scale), _ptr(self.w13_scale_2),
                             _ptr(self.w2_scale_2))


# --------------------------------------------------------------- host calls

def moe_capacity(rows: int, factor: float, align: int = 4) -> int:
    out = _I64()
    _check(_lib.moe_capacity(rows, factor, align, ctypes.byref(out)), "moe_capacity")
    return out.value


def moe_decode_bucket(tokens: int, ladder) -> int:
    """Smallest bucket of ``ladder`` (ascending token counts) that holds ``tokens``."""
    arr = (_I64 * len(ladder))(*ladder)
    out = _I64()
    _check(_lib.moe_decode_bucket(tokens, arr, len(ladder), ctypes.byref(out)), "moe_decode_bucket")
    return out.value


def moe_routing_map_bytes(fmt: int, T: int, E: int, K: int) -> int:
    out = ctypes.c_size_t()
    _check(_lib.moe_routing_map_bytes(fmt, T, E, K, ctypes.byref(out)), "moe_routing_map_bytes")
    return out.value


def moe_preprocess_workspace_size(shape: Shape) -> int:
    out = ctypes.c_size_t()
    _check(_lib.moe_preprocess_workspace_size(ctypes.byref(shape.c()), ctypes.byref(out)),
           "moe_preprocess_workspace_size")
    return out.value


def moe_grouped_mlp_workspace_size(shape: Shape, layout: Layout, w_dtype: int) -> int:
    out = ctypes.c_size_t()
    _check(_lib.moe_grouped_mlp_workspace_size(ctypes.byref(shape.c()), ctypes.byref(layout.c()), w_dtype,
                                               ctypes.byref(out)), "moe_grouped_mlp_workspace_size")
    return out.value


def moe_grouped_mlp_kernel_count(shape: Shape, layout: Layout, w_dtype: int) -> int:
    out = ctypes.c_int32()
    _check(_lib.moe_grouped_mlp_kernel_count(ctypes.byref(shape.c()), ctypes.byref(layout.c()), w_dtype,
                                             ctypes.byref(out)), "moe_grouped_mlp_kernel_count")
    return out.value


# ------------------------------------------------------------- device calls

def moe_preprocess(routing: Routing, shape: Shape, layout: Layout, handle: Handle, workspace: torch.Tensor,
                   stream=None) -> None:
    _check(_lib.moe_preprocess(ctypes.byref(routing.c()), ctypes.byref(shape.c()), ctypes.byref(layout.c()),
                               ctypes.byref(handle.c()), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_preprocess")


def moe_preprocess_noalloc(routing: Routing, shape: Shape, layout: Layout, handle: Handle, stream=None) -> None:
    """moe_preprocess without a caller workspace: for callers that cannot
    allocate device memory (a plugin whose host application owns all device
    memory, a loop that must not call cudaMalloc).  Uses the library's fixed
    scratch array; see moe_preprocess_noalloc in moe.h for its limits."""
    _check(_lib.moe_preprocess_noalloc(ctypes.byref(routing.c()), ctypes.byref(shape.c()), ctypes.byref(layout.c()),
                                       ctypes.byref(handle.c()), _stream(stream)), "moe_preprocess_noalloc")


def moe_dispatch_permute(handle: Handle, shape: Shape, layout: Layout, in_dtype: int, x: torch.Tensor,
                         x_scales: Optional[torch.Tensor], routing: Routing, out_tokens: torch.Tensor,
                         out_probs: Optional[torch.Tensor] = None, out_scales: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    _check(_lib.moe_dispatch_permute(ctypes.byref(handle.c()), ctypes.byref(shape.c()),
                                     ctypes.byref(layout.c()), in_dtype, _ptr(x), _ptr(x_scales),
                                     ctypes.byref(routing.c()), _ptr(out_tokens), _ptr(out_probs),
                                     _ptr(out_scales), _stream(stream)), "moe_dispatch_permute")


def moe_grouped_mlp(handle: Handle, shape: Shape, layout: Layout, w_dtype: int, perm_tokens: torch.Tensor,
                    perm_scales: Optional[torch.Tensor], w13: torch.Tensor, w13_scales: Optional[torch.Tensor],
                    w2: torch.Tensor, w2_scales: Optional[torch.Tensor], globals_: Optional[Nvfp4Globals],
                    workspace: torch.Tensor, out_fc2: torch.Tensor, stream=None) -> None:
    g = ctypes.byref(globals_.c()) if globals_ is not None else None
    _check(_lib.moe_grouped_mlp(ctypes.byref(handle.c()), ctypes.byref(shape.c()), ctypes.byref(layout.c()),
                                w_dtype, _ptr(perm_tokens), _ptr(perm_scales), _ptr(w13), _ptr(w13_scales),
                                _ptr(w2), _ptr(w2_scales), g, _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _ptr(out_fc2), _stream(stream)),
           "moe_grouped_mlp")


def moe_grouped_mlp_ex(handle: Handle, shape: Shape, layout: Layout, w_dtype: int, perm_tokens: torch.Tensor,
                       perm_scales: Optional[torch.Tensor], w13: torch.Tensor, w13_scales: Optional[torch.Tensor],
                       w2: torch.Tensor, w2_scales: Optional[torch.Tensor], globals_: Optional[Nvfp4Globals],
                       workspace: torch.Tensor, out_format: int, out_fc2: torch.Tensor,
                       out_fc2_scales: Optional[torch.Tensor] = None, fc2_row_probs: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    g = ctypes.byref(globals_.c()) if globals_ is not None else None
    _check(_lib.moe_grouped_mlp_ex(ctypes.byref(handle.c()), ctypes.byref(shape.c()), ctypes.byref(layout.c()),
                                   w_dtype, _ptr(perm_tokens), _ptr(perm_scales), _ptr(w13), _ptr(w13_scales),
                                   _ptr(w2), _ptr(w2_scales), g, _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), out_format, _ptr(out_fc2),
                                   _ptr(out_fc2_scales), _ptr(fc2_row_probs), _stream(stream)),
           "moe_grouped_mlp_ex")


def moe_combine_unpermute_fmt(handle: Handle, shape: Shape, layout: Layout, in_format: int,
                              expert_out: torch.Tensor, expert_out_scales: Optional[torch.Tensor],
                              perm_probs: Optional[torch.Tensor], y: torch.Tensor, stream=None) -> None:
    _check(_lib.moe_combine_unpermute_fmt(ctypes.byref(handle.c()), ctypes.byref(shape.c()),
                                          ctypes.byref(layout.c()), in_format, _ptr(expert_out),
                                          _ptr(expert_out_scales), _ptr(perm_probs), _ptr(y), _stream(stream)),
           "moe_combine_unpermute_fmt")


def moe_quantize_mx_rows(x: torch.Tensor, fmt: int, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    H = x.shape[-1]
    R = x.numel() // H
    _check(_lib.moe_quantize_mx_rows(_ptr(x), R, H, fmt, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_quantize_mx_rows")


def moe_combine_unpermute(handle: Handle, shape: Shape, layout: Layout, expert_out: torch.Tensor,
                          perm_probs: Optional[torch.Tensor], y: torch.Tensor, stream=None) -> None:
    _check(_lib.moe_combine_unpermute(ctypes.byref(handle.c()), ctypes.byref(shape.c()), ctypes.byref(layout.c()),
                                      _ptr(expert_out), _ptr(perm_probs), _ptr(y), _stream(stream)),
           "moe_combine_unpermute")


def moe_combine_backward(handle: Handle, shape: Shape, layout: Layout, grad_y: torch.Tensor,
                         expert_out: Optional[torch.Tensor], perm_probs: Optional[torch.Tensor],
                         grad_expert_out: torch.Tensor, grad_perm_probs: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    _check(_lib.moe_combine_backward(ctypes.byref(handle.c()), ctypes.byref(shape.c()), ctypes.byref(layout.c()),
                                     _ptr(grad_y), _ptr(expert_out), _ptr(perm_probs), _ptr(grad_expert_out),
                                     _ptr(grad_perm_probs), _stream(stream)), "moe_combine_backward")


def moe_dispatch_backward(handle: Handle, shape: Shape, layout: Layout, routing_format: int,
                          grad_perm_tokens: torch.Tensor, grad_perm_probs: Optional[torch.Tensor],
                          grad_x: torch.Tensor, grad_probs: Optional[torch.Tensor] = None, stream=None) -> None:
    _check(_lib.moe_dispatch_backward(ctypes.byref(handle.c()), ctypes.byref(shape.c()), ctypes.byref(layout.c()),
                                      routing_format, _ptr(grad_perm_tokens), _ptr(grad_perm_probs), _ptr(grad_x),
                                      _ptr(grad_probs), _stream(stream)), "moe_dispatch_backward")


def moe_profile_next_grouped_mlp(ev_before_fc1, ev_after_fc1, ev_after_fc2) -> None:
    """Record three torch.cuda.Event objects around FC1 / FC2 of the next moe_grouped_mlp call."""
    handles = [ctypes.c_void_p(e.cuda_event) if e is not None else None
               for e in (ev_before_fc1, ev_after_fc1, ev_after_fc2)]
    _check(_lib.moe_profile_next_grouped_mlp(*handles), "moe_profile_next_grouped_mlp")


def moe_debug_next_grouped_mlp_silent_token_tile(token_tile: int) -> None:
    """Testing hook: the next fused bf16 grouped MLP call lets token tile
    `token_tile`'s FC1 tiles withhold their completion publication (-1 cancels)."""
    _check(_lib.moe_debug_next_grouped_mlp_silent_token_tile(token_tile),
           "moe_debug_next_grouped_mlp_silent_token_tile")


def moe_debug_preprocess_silent_tile(routing: Routing, shape: Shape, layout: Layout, handle: Handle,
                                     workspace: torch.Tensor, silent_tile: int, stream=None) -> None:
    """Testing hook: preprocess with one tile withholding its lookback publication (see moe.h)."""
    _check(_lib.moe_debug_preprocess_silent_tile(ctypes.byref(routing.c()), ctypes.byref(shape.c()),
                                                 ctypes.byref(layout.c()), ctypes.byref(handle.c()), _ptr(workspace),
                                                 workspace.numel() * workspace.element_size(), silent_tile,
                                                 _stream(stream)), "moe_debug_preprocess_silent_tile")


def moe_quantize_fp8_blocks(w: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    G, N, Kd = w.shape
    _check(_lib.moe_quantize_fp8_blocks(_ptr(w), G, N, Kd, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_quantize_fp8_blocks")


def moe_quantize_nvfp4_rows(x: torch.Tensor, global_scale: torch.Tensor, packed: torch.Tensor,
                            scales: torch.Tensor, stream=None) -> None:
    Kd = x.shape[-1]
    R = x.numel() // Kd
    _check(_lib.moe_quantize_nvfp4_rows(_ptr(x), R, Kd, _ptr(global_scale), _ptr(packed), _ptr(scales),
                                        _stream(stream)), "moe_quantize_nvfp4_rows")


# ------------------------------------------- operators around the layer

_ELEM = {torch.float32: ELEM_F32, torch.bfloat16: ELEM_BF16, torch.float16: ELEM_F16}


def _elem(t: torch.Tensor) -> int:
    if t.dtype not in _ELEM:
        raise ValueError(f"float32, bfloat16 or float16 tensor expected, got {t.dtype}")
    return _ELEM[t.dtype]


# The descriptors of a call are packed into one buffer (moe_norm, moe_router or
# moe_w4, then moe_rows after moe_rows) and passed by address: a few C structs
# built one by one cost more time than a small kernel takes.
_ROWS_BYTES = 16


def _address(buf: bytearray) -> int:
    return ctypes.addressof(ctypes.c_char.from_buffer(buf))


def _rows(t: torch.Tensor, name: str, shape, dtype: torch.dtype):
    """Address and row stride of a 2-D tensor with unit column stride; its rows may lie apart."""
    if not t.is_cuda:
        raise ValueError(f"{name}: device tensor expected")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {dtype} expected, got {t.dtype}")
    row, col = t.stride()
    if col != 1 and shape[1] > 1:
        raise ValueError(f"{name}: adjacent columns expected (stride(1) == 1)")
    return t.data_ptr(), row if shape[0] > 1 else shape[1]


_ABSENT = (0, 0)


def _dense(t: Optional[torch.Tensor], name: str, shape, dtype: torch.dtype):
    """Address of a contiguous tensor of this shape and type."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name}: {dtype} {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: device tensor expected")
    if not t.is_contiguous():
        raise ValueError(f"{name}: contiguous tensor expected")
    return t.data_ptr()


def _matrix(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name}: 2-D tensor expected")
    return t.shape


def _param_dtype(x: torch.Tensor, weight, bias) -> torch.dtype:
    dtype = weight.dtype if weight is not None else bias.dtype if bias is not None else x.dtype
    if dtype is not x.dtype and dtype is not torch.float32:
        raise ValueError(f"weight, bias: {x.dtype} or float32 expected, got {dtype}")
    return dtype


_NORM_CALL = struct.Struct("=qqiif4x" + "qq" * 4)  # moe_norm, then four moe_rows
_NORM_ROWS = 32


def moe_layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor], eps: float,
                   y: torch.Tensor, residual: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                   mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None, stream=None) -> None:
    """y = layer_norm(x + residual) * weight + bias per row of x [rows, H]; sum_out
    takes the residual sum, mean and rstd (float [rows]) what the backward reads."""
    shape, dtype = _matrix(x, "x"), x.dtype
    pdtype = _param_dtype(x, weight, bias)
    buf = bytearray(_NORM_CALL.size)
    _NORM_CALL.pack_into(buf, 0, *shape, _elem(x), _ELEM[pdtype], eps, *_rows(x, "x", shape, dtype),
                         *(_ABSENT if residual is None else _rows(residual, "residual", shape, dtype)),
                         *_rows(y, "y", shape, dtype),
                         *(_ABSENT if sum_out is None else _rows(sum_out, "sum_out", shape, dtype)))
    a = _address(buf)
    r = a + _NORM_ROWS
    _check(_lib.moe_layer_norm(a, r, r + _ROWS_BYTES, _dense(weight, "weight", shape[1:], pdtype),
                               _dense(bias, "bias", shape[1:], pdtype), r + 2 * _ROWS_BYTES, r + 3 * _ROWS_BYTES,
                               _dense(mean, "mean", shape[:1], torch.float32),
                               _dense(rstd, "rstd", shape[:1], torch.float32), _stream(stream)), "moe_layer_norm")


def moe_layer_norm_workspace_size(rows: int, H: int) -> int:
    out = ctypes.c_size_t()
    _check(_lib.moe_layer_norm_workspace_size(rows, H, ctypes.byref(out)), "moe_layer_norm_workspace_size")
    return out.value


def moe_layer_norm_backward(grad_y: torch.Tensor, h: torch.Tensor, weight: Optional[torch.Tensor],
                            mean: torch.Tensor, rstd: torch.Tensor, grad_x: torch.Tensor,
                            grad_weight: Optional[torch.Tensor] = None, grad_bias: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, grad_sum: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """Gradients of moe_layer_norm; h is the normalised row matrix (x, or sum_out
    where there was a residual) and grad_sum the gradient that reaches it past
    the norm.  workspace is needed for grad_weight / grad_bias (float [H])."""
    shape, dtype, f32 = _matrix(h, "h"), h.dtype, torch.float32
    pdtype = _param_dtype(h, weight, None)
    buf = bytearray(_NORM_CALL.size)
    _NORM_CALL.pack_into(buf, 0, *shape, _elem(h), _ELEM[pdtype], 0.0, *_rows(grad_y, "grad_y", shape, dtype),
                         *_rows(h, "h", shape, dtype),
                         *(_ABSENT if grad_sum is None else _rows(grad_sum, "grad_sum", shape, dtype)),
                         *_rows(grad_x, "grad_x", shape, dtype))
    a = _address(buf)
    r = a + _NORM_ROWS
    if workspace is not None and not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace: contiguous device tensor expected")
    _check(_lib.moe_layer_norm_backward(
        a, r, r + _ROWS_BYTES, _dense(weight, "weight", shape[1:], pdtype), _dense(mean, "mean", shape[:1], f32),
        _dense(rstd, "rstd", shape[:1], f32), r + 2 * _ROWS_BYTES, r + 3 * _ROWS_BYTES,
        _dense(grad_weight, "grad_weight", shape[1:], f32), _dense(grad_bias, "grad_bias", shape[1:], f32),
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)),
        "moe_layer_norm_backward")


@dataclasses.dataclass(frozen=True)
class Router:
    """Top-k router over E experts: score SCORE_SOFTMAX or SCORE_SIGMOID; with
    renormalize the chosen scores are divided by their sum; scale multiplies the
    weights last (see moe_router in moe.h)."""
    E: int
    K: int
    score: int = SCORE_SOFTMAX
    renormalize: bool = True
    scale: float = 1.0

    def map_shape(self, fmt: int, T: int):
        return (T, self.E) if fmt == ROUTING_SPARSE_BOOL else (T, self.K)


_MAP_DTYPE = {ROUTING_DENSE_I16: torch.int16, ROUTING_SPARSE_BOOL: torch.uint8}
_ROUTER_CALL = struct.Struct("=qqqiiif" + "qq" * 2)  # moe_router, then two moe_rows
_ROUTER_ROWS = 40


def _router_call(router: Router, logits: torch.Tensor, routing: Routing, grad_logits: Optional[torch.Tensor]):
    """(buffer, its address, address of the map, shape of the map)"""
    shape = _matrix(logits, "logits")
    if shape[1] != router.E:
        raise ValueError(f"logits: {router.E} columns expected, got {shape[1]}")
    if routing.format not in _MAP_DTYPE:
        raise ValueError("unknown routing format")
    buf = bytearray(_ROUTER_CALL.size)
    _ROUTER_CALL.pack_into(buf, 0, shape[0], router.E, router.K, _elem(logits), router.score,
                           1 if router.renormalize else 0, router.scale, *_rows(logits, "logits", shape, logits.dtype),
                           *(_ABSENT if grad_logits is None else
                             _rows(grad_logits, "grad_logits", shape, logits.dtype)))
    map_shape = router.map_shape(routing.format, shape[0])
    return buf, _address(buf), _dense(routing.map, "routing.map", map_shape, _MAP_DTYPE[routing.format]), map_shape


def moe_router_topk(router: Router, logits: torch.Tensor, routing: Routing,
                    select_bias: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """Writes routing.map and routing.probs (both required) from logits [T, E];
    status (int32 [1], optional) collects DEV_ERR_NAN_LOGIT."""
    buf, a, map_, map_shape = _router_call(router, logits, routing, None)
    _check(_lib.moe_router_topk(a, a + _ROUTER_ROWS, _dense(select_bias, "select_bias", (router.E,), torch.float32),
                                routing.format, map_, _dense(routing.probs, "routing.probs", map_shape, torch.float32),
                                _dense(status, "status", (1,), torch.int32), _stream(stream)), "moe_router_topk")


def moe_router_topk_backward(router: Router, logits: torch.Tensor, routing: Routing, grad_probs: torch.Tensor,
                             grad_logits: torch.Tensor, stream=None) -> None:
    """grad_logits [T, E] from grad_probs in the layout of routing.map."""
    buf, a, map_, map_shape = _router_call(router, logits, routing, grad_logits)
    _check(_lib.moe_router_topk_backward(a, a + _ROUTER_ROWS, routing.format, map_,
                                         _dense(grad_probs, "grad_probs", map_shape, torch.float32),
                                         a + _ROUTER_ROWS + _ROWS_BYTES, _stream(stream)), "moe_router_topk_backward")


@dataclasses.dataclass
class W4Weight:
    """4-bit weights with group scales: codes uint8 [N, Kd/2] (or [E, N, Kd/2], one
    matrix per expert), scales bfloat16 / float16 [.., N, ceil(Kd/group)], zeros
    uint8 [.., N, ceil(ceil(Kd/group)/2)] or None (z = 8); see moe_w4 in moe.h."""
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: Optional[torch.Tensor]
    group: int


_W4_CALL = struct.Struct("=qqiiQQQ" + "qq" * 3)  # moe_w4, then three moe_rows
_W4_ROWS = 48


def _w4_call(weight: W4Weight, lead: tuple, x: torch.Tensor, y: torch.Tensor, activation: int,
             addend: Optional[torch.Tensor], rows: int):
    """(buffer, its address): the weight, x, addend, y"""
    shape, dtype = weight.codes.shape, weight.scales.dtype
    if len(shape) != len(lead) + 2 or weight.group < 1:
        raise ValueError(f"codes: {len(lead) + 2}-D tensor expected, got {tuple(shape)}")
    N, Kd = shape[-2], shape[-1] * 2
    G = -(-Kd // weight.group)
    y_shape = (rows, N // 2 if activation == W4_SWIGLU else N)
    buf = bytearray(_W4_CALL.size)
    _W4_CALL.pack_into(buf, 0, N, Kd, weight.group, _elem(weight.scales),
                       _dense(weight.codes, "codes", (*lead, N, shape[-1]), torch.uint8),
                       _dense(weight.scales, "scales", (*lead, N, G), dtype),
                       _dense(weight.zeros, "zeros", (*lead, N, (G + 1) // 2), torch.uint8) or 0,
                       *_rows(x, "x", (rows, Kd), dtype),
                       *(_ABSENT if addend is None else _rows(addend, "addend", y_shape, dtype)),
                       *_rows(y, "y", y_shape, dtype))
    return buf, _address(buf)


def moe_w4_matvec(weight: W4Weight, x: torch.Tensor, y: torch.Tensor, activation: int = W4_NONE,
                  addend: Optional[torch.Tensor] = None, stream=None) -> None:
    """y [M, N or N/2] = act(x [M, Kd] . W^T) (+ addend)."""
    M = _matrix(x, "x")[0]
    buf, a = _w4_call(weight, (), x, y, activation, addend, M)
    r = a + _W4_ROWS
    _check(_lib.moe_w4_matvec(a, M, r, activation, r + _ROWS_BYTES, r + 2 * _ROWS_BYTES, _stream(stream)),
           "moe_w4_matvec")


def moe_grouped_w4_matvec(handle: Handle, shape: Shape, layout: Layout, weight: W4Weight, x: torch.Tensor,
                          y: torch.Tensor, activation: int = W4_NONE, stream=None) -> None:
    """moe_w4_matvec of every dispatched row x [cap, Kd] with its expert's matrix, into y [cap, N or N/2]."""
    buf, a = _w4_call(weight, (shape.E,), x, y, activation, None, layout.capacity)
    r = a + _W4_ROWS
    _check(_lib.moe_grouped_w4_matvec(ctypes.byref(handle.c()), ctypes.byref(shape.c()), ctypes.byref(layout.c()), a, r,
                                      activation, r + 2 * _ROWS_BYTES, _stream(stream)), "moe_grouped_w4_matvec")


def moe_quantize_w4_rows(w: torch.Tensor, group: int, codes: torch.Tensor, scales: torch.Tensor,
                         zeros: Optional[torch.Tensor] = None, stream=None) -> None:
    """w [.., Kd] (bfloat16 / float16) -> the tensors of a W4Weight."""
    lead, Kd = tuple(w.shape[:-1]), w.shape[-1]
    R = w.numel() // Kd if Kd else 0
    G = (Kd + group - 1) // group if group > 0 else 0
    _check(_lib.moe_quantize_w4_rows(_ptr(w), R, Kd, group, _elem(w),
                                     _dense(codes, "codes", (*lead, Kd // 2), torch.uint8),
                                     _dense(scales, "scales", (*lead, G), w.dtype),
                                     _dense(zeros, "zeros", (*lead, (G + 1) // 2), torch.uint8), _stream(stream)),
           "moe_quantize_w4_rows")


class Ring:
    """Host-side ring of caller-owned output slots (moe_ring_* in moe.h)."""

    def __init__(self, n_slots: int, use_events: bool = True):
        self._r = ctypes.c_void_p()
        _check(_lib.moe_ring_create(n_slots, 1 if use_events else 0, ctypes.byref(self._r)), "moe_ring_create")

    def acquire(self, stream=None) -> int:
        slot = ctypes.c_int32()
        s = _stream(stream) if torch.cuda.is_available() else None
        _check(_lib.moe_ring_acquire(self._r, s, ctypes.byref(slot)), "moe_ring_acquire")
        return slot.value

    def release(self, slot: int, stream=None) -> None:
        s = _stream(stream) if torch.cuda.is_available() else None
        _check(_lib.moe_ring_release(self._r, slot, s), "moe_ring_release")

    def close(self) -> None:
        if self._r:
            _check(_lib.moe_ring_destroy(self._r), "moe_ring_destroy")
            self._r = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def library():
    """The loaded ctypes library (for symbol checks)."""
    return _lib


def exported_symbols():
    return list(_SIGNATURES)
