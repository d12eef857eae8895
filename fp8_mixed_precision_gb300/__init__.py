"""Python binding of the GB300 FP8 linear-layer library (libfp8lin.so).

Argument marshalling only: every function below allocates its outputs with
torch on the current CUDA device and the call's stream (`stream`, by default
the current one), passes raw device pointers and that stream to the C ABI
declared in include/fp8lin.h, and raises FP8Error on a non-OK status.  Names follow the C ABI.  There is no fallback: if the
compiled library is missing, importing works but the first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass, field

import torch

__all__ = [
    "FP8Error", "lib", "RECIPE", "ROLE", "FORMAT", "SCALING",
    "fp8_quantize", "fp8_scale_shape", "fp8_gemm", "fp8_linear_fwd", "fp8_linear_bwd",
    "fp8_gelu_fwd", "fp8_gelu_bwd", "fp8_grad_accumulate", "fp8_get_device_status",
    "fp8_launch_count", "fp8_profile_begin", "fp8_profile_end", "WeightCache", "LinearContext",
    "fp8_quantize_delayed", "fp8_debug_wait_timeout", "HostPipeline", "amax_partials_buffer",
    "fp8_amax_partials", "fp8_linear_fwd_after_amax", "fp8_linear_bwd_after_amax",
    "ACTIVATION", "fp8_rmsnorm_fwd", "fp8_rmsnorm_bwd", "rmsnorm_buffers", "rmsnorm_workspace",
    "fp8_gated_fwd", "fp8_gated_fwd_quantized", "fp8_gated_bwd", "GatedContext", "gated_context",
    "gated_workspace", "gated_norm_columns", "fp8_gated_ctx_layout", "GradClip", "NormBuffers",
    "SCORE", "fp8_route_fwd", "fp8_route_bwd", "ExpertOrder", "expert_rows", "fp8_expert_order",
    "fp8_expert_gather", "fp8_expert_combine", "fp8_expert_combine_bwd", "W4Weight", "fp8_w4_quantize",
    "fp8_w4_linear", "fp8_w4_gated", "fp8_w4_experts", "w4_workspace", "w4_experts_workspace",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8lin.so")

RECIPE = {"tensorwise": 0, "block": 1, "delayed": 2}
ROLE = {"act": 0, "weight": 1, "grad": 2}
FORMAT = {"e4m3": 0, "e5m2": 1}
SCALING = {"tensor": 0, "1x128_128x128": 1, "1x128_1x128": 2}

ACTIVATION = {"silu": 0, "gelu": 1}
SCORE = {"softmax": 0, "sigmoid": 1}
_DTYPE = {torch.bfloat16: 0, torch.float32: 1}

_c_i64 = ctypes.c_int64
_c_p = ctypes.c_void_p
_c_sz = ctypes.c_size_t
_c_int = ctypes.c_int

_SIGS = {
    "fp8_status_string": (ctypes.c_char_p, [_c_int]),
    "fp8_launch_count": (ctypes.c_uint64, []),
    "fp8_quantize": (_c_int, [_c_p, _c_i64, _c_i64, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p,
                              _c_p, _c_p, _c_sz, _c_p]),
    "fp8_quantize_workspace_size": (_c_int, [_c_int, _c_i64, _c_i64, ctypes.POINTER(_c_sz)]),
    "fp8_scale_shape": (_c_int, [_c_int, _c_int, _c_i64, _c_i64, _c_int,
                                 ctypes.POINTER(_c_i64), ctypes.POINTER(_c_i64)]),
    "fp8_gemm": (_c_int, [_c_p, _c_int, _c_p, _c_p, _c_int, _c_p, _c_i64, _c_i64, _c_i64, _c_int,
                          _c_p, _c_p, _c_sz, _c_p]),
    "fp8_gemm_workspace_size": (_c_int, [_c_i64, _c_i64, _c_i64, _c_int, ctypes.POINTER(_c_sz)]),
    "fp8_weight_cache_create": (_c_int, [ctypes.POINTER(_c_p)]),
    "fp8_weight_cache_destroy": (None, [_c_p]),
    "fp8_weight_cache_register": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p,
                                           _c_p, _c_p, _c_p, _c_p, _c_sz,
                                           ctypes.POINTER(ctypes.c_int32)]),
    "fp8_weight_cache_begin_cycle": (_c_int, [_c_p]),
    "fp8_weight_cache_get": (_c_int, [_c_p, ctypes.c_int32, ctypes.c_uint64, _c_int, _c_p,
                                      ctypes.POINTER(_c_int)]),
    "fp8_linear_ctx_size": (_c_int, [_c_int, _c_i64, _c_i64, ctypes.POINTER(_c_sz)]),
    "fp8_linear_workspace_size": (_c_int, [_c_int, _c_i64, _c_i64, _c_i64, ctypes.POINTER(_c_sz)]),
    "fp8_linear_fwd": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, ctypes.c_int32, _c_int, _c_p, _c_p,
                                _c_p, _c_sz, _c_p]),
    "fp8_linear_bwd": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, ctypes.c_int32, _c_int, _c_p,
                                _c_p, _c_p, _c_sz, _c_p]),
    "fp8_gelu_fwd": (_c_int, [_c_p, _c_p, _c_i64, _c_p]),
    "fp8_gelu_bwd": (_c_int, [_c_p, _c_p, _c_p, _c_i64, _c_p]),
    "fp8_grad_accumulate": (_c_int, [_c_p, _c_p, _c_i64, _c_p]),
    "fp8_get_device_status": (_c_int, [_c_p]),
    "fp8_profile_begin": (_c_int, []),
    "fp8_debug_wait_timeout": (_c_int, [ctypes.c_uint64, _c_p]),
    "fp8_quantize_delayed": (_c_int, [_c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p,
                                      ctypes.c_int32, _c_i64, _c_p, _c_sz, _c_p]),
    "fp8_weight_cache_register_delayed": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p,
                                                   _c_p, _c_p, ctypes.c_int32, _c_p, _c_sz,
                                                   ctypes.POINTER(ctypes.c_int32)]),
    "fp8_gelu_quantize": (_c_int, [_c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p,
                                   _c_p, _c_p]),
    "fp8_gelu_bwd_quantize": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p, _c_p,
                                       _c_p, _c_p, _c_p]),
    "fp8_linear_ctx_layout": (_c_int, [_c_int, _c_i64, _c_i64, _c_p, ctypes.POINTER(_c_p),
                                       ctypes.POINTER(_c_p), ctypes.POINTER(_c_p)]),
    "fp8_linear_fwd_quantized": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, ctypes.c_int32, _c_int,
                                          _c_p, _c_p, _c_sz, _c_p]),
    "fp8_linear_bwd_quantized": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p,
                                          ctypes.c_int32, _c_int, _c_p, _c_p, _c_p, _c_sz, _c_p]),
}


class _HostIO(ctypes.Structure):
    _fields_ = [("X", _c_p), ("W", _c_p), ("dY", _c_p), ("Y", _c_p), ("dX", _c_p), ("dW", _c_p)]


class _DeviceIO(ctypes.Structure):
    _fields_ = [("X", _c_p), ("dY", _c_p), ("Y", _c_p), ("dX", _c_p), ("dW", _c_p),
                ("ctx", _c_p), ("ws", _c_p), ("ws_bytes", _c_sz)]


_SIGS.update({
    "fp8_amax_partials": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_sz, _c_p]),
    "fp8_linear_fwd_after_amax": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, ctypes.c_int32, _c_int,
                                           _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "fp8_linear_bwd_after_amax": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p, ctypes.c_int32,
                                           _c_int, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "fp8_host_pipeline_create": (_c_int, [_c_int, ctypes.POINTER(_c_p)]),
    "fp8_host_pipeline_destroy": (None, [_c_p]),
    "fp8_linear_step_host": (_c_int, [_c_p, _c_int, _c_i64, ctypes.POINTER(_HostIO),
                                      ctypes.POINTER(_DeviceIO), _c_p, ctypes.c_int32, _c_int,
                                      ctypes.c_uint64]),
    "fp8_host_pipeline_fork": (_c_int, [_c_p, _c_p]),
    "fp8_host_pipeline_join": (_c_int, [_c_p, _c_p]),
    "fp8_host_pipeline_sync": (_c_int, [_c_p]),
})


class _GradDesc(ctypes.Structure):
    _fields_ = [("src", _c_p), ("dst", _c_p), ("n", _c_i64), ("dtype", _c_int)]


_SIGS.update({
    "fp8_rmsnorm_fwd": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_i64, _c_i64, ctypes.c_float] +
                        [_c_p] * 11),
    "fp8_rmsnorm_workspace_size": (_c_int, [_c_i64, _c_i64, ctypes.POINTER(_c_sz)]),
    "fp8_rmsnorm_bwd": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_i64, _c_i64, _c_p, _c_p,
                                 _c_p, _c_sz, _c_p]),
    "fp8_gated_ctx_size": (_c_int, [_c_int, _c_i64, _c_i64, _c_i64, ctypes.POINTER(_c_sz)]),
    "fp8_gated_ctx_layout": (_c_int, [_c_int, _c_i64, _c_i64, _c_i64, _c_p] +
                             [ctypes.POINTER(_c_p)] * 5),
    "fp8_gated_workspace_size": (_c_int, [_c_int, _c_i64, _c_i64, _c_i64, _c_int,
                                          ctypes.POINTER(_c_sz)]),
    "fp8_gated_fwd": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, ctypes.c_int32, _c_int, _c_int, _c_p,
                               _c_p, _c_p, _c_sz, _c_p]),
    "fp8_gated_fwd_quantized": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, ctypes.c_int32, _c_int,
                                         _c_int, _c_p, _c_p, _c_p]),
    "fp8_gated_bwd": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, ctypes.c_int32, _c_int, _c_int,
                               _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "fp8_grad_clip_create": (_c_int, [ctypes.POINTER(_GradDesc), _c_i64, ctypes.POINTER(_c_p)]),
    "fp8_grad_clip_destroy": (None, [_c_p]),
    "fp8_grad_clip_table_size": (_c_int, [_c_p, ctypes.POINTER(_c_sz)]),
    "fp8_grad_clip_table_write": (_c_int, [_c_p, _c_p, _c_sz]),
    "fp8_grad_clip_workspace_size": (_c_int, [_c_p, ctypes.POINTER(_c_sz)]),
    "fp8_grad_clip_run": (_c_int, [_c_p, _c_p, ctypes.c_float, _c_p, _c_p, _c_sz, _c_p]),
    "fp8_grad_norm": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
})


class _W4(ctypes.Structure):
    _fields_ = [("codes", _c_p), ("scale", _c_p), ("zero", _c_p), ("E", _c_i64), ("rows", _c_i64),
                ("K", _c_i64), ("group", _c_int)]


_SIGS.update({
    "fp8_route_fwd": (_c_int, [_c_p, _c_int, _c_p, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int,
                               _c_int, _c_int, ctypes.c_float, _c_p, _c_p, _c_p]),
    "fp8_route_bwd": (_c_int, [_c_p, _c_p, _c_int, _c_p, _c_p, _c_i64, _c_i64, _c_int, _c_int,
                               _c_int, ctypes.c_float, _c_p, _c_p]),
    "fp8_expert_rows": (_c_i64, [_c_i64, _c_i64, _c_i64]),
    "fp8_expert_order_workspace_size": (_c_int, [_c_i64, _c_i64, ctypes.POINTER(_c_sz)]),
    "fp8_expert_order": (_c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz,
                                  _c_p]),
    "fp8_expert_gather": (_c_int, [_c_p, _c_i64, _c_i64, _c_int, _c_i64, _c_i64, _c_p, _c_p, _c_p,
                                   _c_p, _c_p]),
    "fp8_expert_combine": (_c_int, [_c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p, _c_p]),
    "fp8_expert_combine_bwd": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_int, _c_i64, _c_i64] +
                               [_c_p] * 7),
    "fp8_w4_quantize": (_c_int, [_c_p, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p, _c_p]),
    "fp8_w4_workspace_size": (_c_int, [ctypes.POINTER(_W4), _c_i64, _c_int, ctypes.POINTER(_c_sz)]),
    "fp8_w4_linear": (_c_int, [_c_p, _c_i64, ctypes.POINTER(_W4), _c_p, _c_p, _c_sz, _c_p]),
    "fp8_w4_gated": (_c_int, [_c_p, _c_i64, ctypes.POINTER(_W4), _c_int, _c_p, _c_p, _c_sz, _c_p]),
    "fp8_w4_experts_workspace_size": (_c_int, [_c_i64, _c_int, _c_i64, _c_i64, _c_i64, _c_i64,
                                               ctypes.POINTER(_c_sz)]),
    "fp8_w4_experts": (_c_int, [_c_p, _c_i64, _c_int, _c_p, _c_p, ctypes.POINTER(_W4),
                                ctypes.POINTER(_W4), _c_int, _c_p, _c_p, _c_sz, _c_p]),
})


class _KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 64), ("launches", ctypes.c_uint64),
                ("total_ms", ctypes.c_double), ("bytes", ctypes.c_double),
                ("flops", ctypes.c_double), ("m", ctypes.c_int64), ("n", ctypes.c_int64),
                ("k", ctypes.c_int64)]

_lib = None


class FP8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib().fp8_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: status {status} ({msg})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded C library (built in-tree by build.py)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m fp8_mixed_precision_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        L.fp8_profile_end.restype = _c_int
        L.fp8_profile_end.argtypes = [ctypes.POINTER(_KernelStat), _c_int, ctypes.POINTER(_c_int)]
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise FP8Error(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    """The cudaStream_t of `stream`, by default of the current stream (read
    without building a torch Stream object, which takes 3 us on this CPU)."""
    if stream is not None:
        return stream.cuda_stream
    if not torch.cuda.is_initialized():
        return torch.cuda.current_stream().cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


_CURRENT = contextlib.nullcontext()


def _on(stream):
    """Calls make their tensors under the stream that their kernels run on, as
    `with torch.cuda.stream(stream)` would: the memory is then free of earlier
    work in that stream's order and goes back to it in that order.
    What a call returns belongs to that stream; what it is given has to be
    ready there, and kept until the work is done."""
    return _CURRENT if stream is None else torch.cuda.stream(stream)


def _need_bf16_cuda(t, name):
    if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")


def fp8_launch_count() -> int:
    return int(lib().fp8_launch_count())


def fp8_scale_shape(recipe: str, role: str, rows: int, cols: int, colwise: bool):
    sr, sc = _c_i64(), _c_i64()
    _check(lib().fp8_scale_shape(RECIPE[recipe], ROLE[role], rows, cols, int(colwise),
                                 ctypes.byref(sr), ctypes.byref(sc)), "fp8_scale_shape")
    return (sr.value, sc.value)


def _quant_ws_bytes(recipe, rows, cols):
    b = _c_sz()
    _check(lib().fp8_quantize_workspace_size(RECIPE[recipe], rows, cols, ctypes.byref(b)),
           "fp8_quantize_workspace_size")
    return b.value


def _empty_bytes(n, device):
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device=device)


def fp8_quantize(x: torch.Tensor, recipe: str, role: str, rowwise: bool = True,
                 colwise: bool = True, stream=None) -> dict:
    """Quantize a bf16 [R, C] tensor; returns dict(row, col, row_scale,
    row_scale_inv, col_scale, col_scale_inv) (absent layouts are None)."""
    _need_bf16_cuda(x, "x")
    R, C = x.shape
    dev = x.device
    out = dict(row=None, col=None, row_scale=None, row_scale_inv=None, col_scale=None,
               col_scale_inv=None)
    rs = fp8_scale_shape(recipe, role, R, C, False)
    cs = fp8_scale_shape(recipe, role, R, C, True)
    with _on(stream):
        if rowwise or recipe == "tensorwise":
            out["row_scale"] = torch.empty(rs, dtype=torch.float32, device=dev)
            out["row_scale_inv"] = torch.empty(rs, dtype=torch.float32, device=dev)
        if colwise:
            out["col_scale"] = torch.empty(cs, dtype=torch.float32, device=dev)
            out["col_scale_inv"] = torch.empty(cs, dtype=torch.float32, device=dev)
        if rowwise:
            out["row"] = torch.empty((R, C), dtype=torch.uint8, device=dev)
        if colwise:
            out["col"] = torch.empty((C, R), dtype=torch.uint8, device=dev)
        ws = _empty_bytes(_quant_ws_bytes(recipe, R, C), dev)
    _check(lib().fp8_quantize(_ptr(x), R, C, RECIPE[recipe], ROLE[role], _ptr(out["row"]),
                              _ptr(out["col"]), _ptr(out["row_scale"]), _ptr(out["row_scale_inv"]),
                              _ptr(out["col_scale"]), _ptr(out["col_scale_inv"]), _ptr(ws),
                              ws.numel(), _stream(stream)), "fp8_quantize")
    return out


def fp8_quantize_delayed(x: torch.Tensor, role: str, history: torch.Tensor, step: int,
                         rowwise: bool = True, colwise: bool = True, stream=None) -> dict:
    """DelayedScaling quantize: scale from max(history), then history[step %
    len] = amax(x).  history: float32 CUDA tensor (updated in place)."""
    _need_bf16_cuda(x, "x")
    if history.dtype != torch.float32 or not history.is_cuda:
        raise ValueError("history must be a float32 CUDA tensor")
    R, C = x.shape
    dev = x.device
    with _on(stream):
        out = dict(row=torch.empty((R, C), dtype=torch.uint8, device=dev) if rowwise else None,
                   col=torch.empty((C, R), dtype=torch.uint8, device=dev) if colwise else None,
                   scale=torch.empty(1, dtype=torch.float32, device=dev),
                   scale_inv=torch.empty(1, dtype=torch.float32, device=dev))
        ws = _empty_bytes(_quant_ws_bytes("tensorwise", R, C), dev)
    _check(lib().fp8_quantize_delayed(_ptr(x), R, C, ROLE[role], _ptr(out["row"]), _ptr(out["col"]),
                                      _ptr(out["scale"]), _ptr(out["scale_inv"]), _ptr(history),
                                      history.numel(), int(step), _ptr(ws), ws.numel(),
                                      _stream(stream)), "fp8_quantize_delayed")
    return out


def fp8_gemm(a: torch.Tensor, a_fmt: str, a_scale_inv: torch.Tensor, b: torch.Tensor, b_fmt: str,
             b_scale_inv: torch.Tensor, scaling: str, out: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """C[M, N] bf16 = sum_k (a[m,k] sa)(b[n,k] sb); a [M, K], b [N, K] uint8."""
    M, K = a.shape
    N, K2 = b.shape
    if K2 != K:
        raise ValueError("inner dimensions differ")
    dev = a.device
    wsb = _c_sz()
    _check(lib().fp8_gemm_workspace_size(M, N, K, SCALING[scaling], ctypes.byref(wsb)),
           "fp8_gemm_workspace_size")
    with _on(stream):
        C = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        ws = _empty_bytes(wsb.value, dev)
    _check(lib().fp8_gemm(_ptr(a), FORMAT[a_fmt], _ptr(a_scale_inv), _ptr(b), FORMAT[b_fmt],
                          _ptr(b_scale_inv), M, N, K, SCALING[scaling], _ptr(C), _ptr(ws),
                          wsb.value, _stream(stream)), "fp8_gemm")
    return C


@dataclass
class _Entry:
    w: torch.Tensor
    recipe: str
    row: torch.Tensor
    col: torch.Tensor
    row_scale: torch.Tensor
    row_scale_inv: torch.Tensor
    col_scale: torch.Tensor
    col_scale_inv: torch.Tensor
    ws: torch.Tensor
    history: torch.Tensor | None = None


class WeightCache:
    """Owns an fp8_weight_cache and the device buffers of its FP8 weights."""

    def __init__(self):
        h = ctypes.c_void_p()
        _check(lib().fp8_weight_cache_create(ctypes.byref(h)), "fp8_weight_cache_create")
        self._h = h
        self.entries: list[_Entry] = []

    @property
    def handle(self):
        return self._h

    def register(self, w: torch.Tensor, recipe: str, history_len: int = 16) -> int:
        _need_bf16_cuda(w, "w")
        O, K = w.shape
        dev = w.device
        if recipe == "delayed":
            s = torch.empty(1, dtype=torch.float32, device=dev)
            si = torch.empty(1, dtype=torch.float32, device=dev)
            e = _Entry(w=w, recipe=recipe,
                       row=torch.empty((O, K), dtype=torch.uint8, device=dev),
                       col=torch.empty((K, O), dtype=torch.uint8, device=dev),
                       row_scale=s, row_scale_inv=si, col_scale=s, col_scale_inv=si,
                       ws=_empty_bytes(_quant_ws_bytes("tensorwise", O, K), dev),
                       history=torch.zeros(history_len, dtype=torch.float32, device=dev))
            out = ctypes.c_int32()
            _check(lib().fp8_weight_cache_register_delayed(
                self._h, _ptr(w), O, K, _ptr(e.row), _ptr(e.col), _ptr(s), _ptr(si),
                _ptr(e.history), history_len, _ptr(e.ws), e.ws.numel(), ctypes.byref(out)),
                "fp8_weight_cache_register_delayed")
            self.entries.append(e)
            return out.value
        rs = fp8_scale_shape(recipe, "weight", O, K, False)
        cs = fp8_scale_shape(recipe, "weight", O, K, True)
        e = _Entry(w=w, recipe=recipe,
                   row=torch.empty((O, K), dtype=torch.uint8, device=dev),
                   col=torch.empty((K, O), dtype=torch.uint8, device=dev),
                   row_scale=torch.empty(rs, dtype=torch.float32, device=dev),
                   row_scale_inv=torch.empty(rs, dtype=torch.float32, device=dev),
                   col_scale=torch.empty(cs, dtype=torch.float32, device=dev),
                   col_scale_inv=torch.empty(cs, dtype=torch.float32, device=dev),
                   ws=_empty_bytes(_quant_ws_bytes(recipe, O, K), dev))
        out = ctypes.c_int32()
        _check(lib().fp8_weight_cache_register(
            self._h, _ptr(w), O, K, RECIPE[recipe], _ptr(e.row), _ptr(e.col), _ptr(e.row_scale),
            _ptr(e.row_scale_inv), _ptr(e.col_scale), _ptr(e.col_scale_inv), _ptr(e.ws),
            e.ws.numel(), ctypes.byref(out)), "fp8_weight_cache_register")
        self.entries.append(e)
        return out.value

    def begin_cycle(self):
        _check(lib().fp8_weight_cache_begin_cycle(self._h), "fp8_weight_cache_begin_cycle")

    def get(self, h: int, version: int = 0, use_cache: bool = True, stream=None) -> bool:
        """Make weight h's FP8 copy current; True if it was re-quantized."""
        rq = ctypes.c_int()
        _check(lib().fp8_weight_cache_get(self._h, h, version, int(use_cache), _stream(stream),
                                          ctypes.byref(rq)), "fp8_weight_cache_get")
        return bool(rq.value)

    def __del__(self):
        if getattr(self, "_h", None) is not None and _lib is not None:
            _lib.fp8_weight_cache_destroy(self._h)
            self._h = None


@dataclass
class LinearContext:
    ctx: torch.Tensor
    N: int
    K: int
    extra: dict = field(default_factory=dict)


def _ctx_bytes(recipe, N, K):
    b = _c_sz()
    _check(lib().fp8_linear_ctx_size(RECIPE[recipe], N, K, ctypes.byref(b)), "fp8_linear_ctx_size")
    return b.value


def linear_workspace(recipe: str, N: int, K: int, O: int, device) -> torch.Tensor:
    b = _c_sz()
    _check(lib().fp8_linear_workspace_size(RECIPE[recipe], N, K, O, ctypes.byref(b)),
           "fp8_linear_workspace_size")
    return _empty_bytes(b.value, device)


def fp8_linear_fwd(x: torch.Tensor, cache: WeightCache, h: int, recipe: str,
                   ws: torch.Tensor | None = None, y: torch.Tensor | None = None,
                   ctx: LinearContext | None = None, stream=None):
    """Y = X W^T with FP8 operands; returns (Y, LinearContext)."""
    _need_bf16_cuda(x, "x")
    N, K = x.shape
    O = cache.entries[h].w.shape[0]
    dev = x.device
    with _on(stream):
        if y is None:
            y = torch.empty((N, O), dtype=torch.bfloat16, device=dev)
        if ctx is None:
            ctx = LinearContext(_empty_bytes(_ctx_bytes(recipe, N, K), dev), N, K)
        if ws is None:
            ws = linear_workspace(recipe, N, K, O, dev)
    _check(lib().fp8_linear_fwd(_ptr(x), N, K, cache.handle, h, RECIPE[recipe], _ptr(y),
                                _ptr(ctx.ctx), _ptr(ws), ws.numel(), _stream(stream)),
           "fp8_linear_fwd")
    return y, ctx


def fp8_linear_bwd(dy: torch.Tensor, ctx: LinearContext, cache: WeightCache, h: int, recipe: str,
                   need_dx: bool = True, ws: torch.Tensor | None = None,
                   dx: torch.Tensor | None = None, dw: torch.Tensor | None = None, stream=None):
    """Returns (dX or None, dW) for Y = X W^T."""
    _need_bf16_cuda(dy, "dy")
    N, O = dy.shape
    K = ctx.K
    dev = dy.device
    with _on(stream):
        if need_dx and dx is None:
            dx = torch.empty((N, K), dtype=torch.bfloat16, device=dev)
        if dw is None:
            dw = torch.empty((O, K), dtype=torch.bfloat16, device=dev)
        if ws is None:
            ws = linear_workspace(recipe, N, K, O, dev)
    _check(lib().fp8_linear_bwd(_ptr(dy), N, O, _ptr(ctx.ctx), cache.handle, h, RECIPE[recipe],
                                _ptr(dx) if need_dx else None, _ptr(dw), _ptr(ws), ws.numel(),
                                _stream(stream)), "fp8_linear_bwd")
    return (dx if need_dx else None), dw


def fp8_gelu_fwd(h: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _need_bf16_cuda(h, "h")
    with _on(stream):
        a = out if out is not None else torch.empty_like(h)
    _check(lib().fp8_gelu_fwd(_ptr(h), _ptr(a), h.numel(), _stream(stream)), "fp8_gelu_fwd")
    return a


def fp8_gelu_bwd(da: torch.Tensor, h: torch.Tensor, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    _need_bf16_cuda(da, "da")
    _need_bf16_cuda(h, "h")
    with _on(stream):
        dh = out if out is not None else torch.empty_like(h)
    _check(lib().fp8_gelu_bwd(_ptr(da), _ptr(h), _ptr(dh), h.numel(), _stream(stream)),
           "fp8_gelu_bwd")
    return dh


def fp8_grad_accumulate(acc: torch.Tensor, dw: torch.Tensor, stream=None) -> torch.Tensor:
    if acc.dtype != torch.float32 or not acc.is_cuda:
        raise ValueError("acc must be a float32 CUDA tensor")
    _need_bf16_cuda(dw, "dw")
    _check(lib().fp8_grad_accumulate(_ptr(acc), _ptr(dw), acc.numel(), _stream(stream)),
           "fp8_grad_accumulate")
    return acc


def fp8_get_device_status(stream=None) -> int:
    return int(lib().fp8_get_device_status(_stream(stream)))


def fp8_profile_begin():
    """Start per-kernel event timing of this library's launches."""
    _check(lib().fp8_profile_begin(), "fp8_profile_begin")


def fp8_profile_end(by_shape: bool = False) -> list:
    """Stop timing; one dict per kernel name (by_shape: per kernel name and
    launch shape) with launches, total_ms, bytes, flops (and m, n, k)."""
    cap = 512
    arr = (_KernelStat * cap)()
    n = _c_int()
    _check(lib().fp8_profile_end(arr, cap, ctypes.byref(n)), "fp8_profile_end")
    recs = [dict(name=arr[i].name.decode(), launches=int(arr[i].launches),
                 total_ms=float(arr[i].total_ms), bytes=float(arr[i].bytes),
                 flops=float(arr[i].flops), m=int(arr[i].m), n=int(arr[i].n), k=int(arr[i].k))
            for i in range(min(n.value, cap))]
    if by_shape:
        return recs
    agg = {}
    for r in recs:
        a = agg.setdefault(r["name"], dict(name=r["name"], launches=0, total_ms=0.0, bytes=0.0,
                                           flops=0.0))
        for key in ("launches", "total_ms", "bytes", "flops"):
            a[key] += r[key]
    return list(agg.values())


def fp8_debug_wait_timeout(limit_ns: int, stream=None):
    """Enqueue the bounded-wait probe (a wait that nothing satisfies)."""
    _check(lib().fp8_debug_wait_timeout(int(limit_ns), _stream(stream)), "fp8_debug_wait_timeout")


class QuantizedTensor:
    """Caller-owned FP8 buffers of one [R, C] tensor under the block recipe:
    row [R, C] + row scales, and the transposed layout, either owned here or
    placed inside a linear context (col_ptrs from fp8_linear_ctx_layout)."""

    def __init__(self, R: int, C: int, role: str, device, col_ptrs=None):
        self.R, self.C = R, C
        rs = fp8_scale_shape("block", role, R, C, False)
        cs = fp8_scale_shape("block", role, R, C, True)
        self.row = torch.empty((R, C), dtype=torch.uint8, device=device)
        self.row_scale = torch.empty(rs, dtype=torch.float32, device=device)
        self.row_scale_inv = torch.empty(rs, dtype=torch.float32, device=device)
        if col_ptrs is None:
            self.col = torch.empty((C, R), dtype=torch.uint8, device=device)
            self.col_scale = torch.empty(cs, dtype=torch.float32, device=device)
            self.col_scale_inv = torch.empty(cs, dtype=torch.float32, device=device)
            self.col_ptrs = (_ptr(self.col), _ptr(self.col_scale), _ptr(self.col_scale_inv))
        else:
            self.col = self.col_scale = self.col_scale_inv = None
            self.col_ptrs = col_ptrs


def fp8_linear_ctx_layout(recipe: str, ctx: LinearContext):
    """Device pointers of the transposed FP8 input and its scales inside ctx."""
    a, b_, c = _c_p(), _c_p(), _c_p()
    _check(lib().fp8_linear_ctx_layout(RECIPE[recipe], ctx.N, ctx.K, _ptr(ctx.ctx), ctypes.byref(a),
                                       ctypes.byref(b_), ctypes.byref(c)), "fp8_linear_ctx_layout")
    return (a, b_, c)


def fp8_gelu_quantize(h: torch.Tensor, q: QuantizedTensor, recipe: str = "block", stream=None):
    """q <- 1x128 E4M3 quantization of bf16(GELU(h)); the bf16 GELU output is not written."""
    _need_bf16_cuda(h, "h")
    R, C = h.shape
    _check(lib().fp8_gelu_quantize(_ptr(h), R, C, RECIPE[recipe], _ptr(q.row), q.col_ptrs[0],
                                   _ptr(q.row_scale), _ptr(q.row_scale_inv), q.col_ptrs[1],
                                   q.col_ptrs[2], _stream(stream)), "fp8_gelu_quantize")
    return q


def fp8_gelu_bwd_quantize(da: torch.Tensor, h: torch.Tensor, q: QuantizedTensor,
                          recipe: str = "block", stream=None):
    """q <- 1x128 E5M2 quantization of bf16(dA * GELU'(H)); dH is not written."""
    _need_bf16_cuda(da, "da")
    _need_bf16_cuda(h, "h")
    R, C = h.shape
    _check(lib().fp8_gelu_bwd_quantize(_ptr(da), _ptr(h), R, C, RECIPE[recipe], _ptr(q.row),
                                       q.col_ptrs[0], _ptr(q.row_scale), _ptr(q.row_scale_inv),
                                       q.col_ptrs[1], q.col_ptrs[2], _stream(stream)),
           "fp8_gelu_bwd_quantize")
    return q


def fp8_linear_fwd_quantized(xq: QuantizedTensor, cache: WeightCache, h: int, recipe: str,
                             ws: torch.Tensor, y: torch.Tensor, stream=None):
    _check(lib().fp8_linear_fwd_quantized(_ptr(xq.row), _ptr(xq.row_scale_inv), xq.R, xq.C,
                                          cache.handle, h, RECIPE[recipe], _ptr(y), _ptr(ws),
                                          ws.numel(), _stream(stream)), "fp8_linear_fwd_quantized")
    return y


def fp8_linear_bwd_quantized(gq: QuantizedTensor, ctx: LinearContext, cache: WeightCache, h: int,
                             recipe: str, ws: torch.Tensor, dx, dw: torch.Tensor, stream=None):
    _check(lib().fp8_linear_bwd_quantized(_ptr(gq.row), _ptr(gq.row_scale_inv), gq.col_ptrs[0],
                                          gq.col_ptrs[2], gq.R, gq.C, _ptr(ctx.ctx), cache.handle,
                                          h, RECIPE[recipe], _ptr(dx), _ptr(dw), _ptr(ws),
                                          ws.numel(), _stream(stream)), "fp8_linear_bwd_quantized")
    return dx, dw


class HostPipeline:
    """Owns an fp8_host_pipeline: one fwd+bwd of an isolated FP8 linear per
    step() call, with inputs and results in (pinned) host tensors and the
    host<->device copies done by the library on its own streams."""

    def __init__(self, slots: int):
        h = ctypes.c_void_p()
        _check(lib().fp8_host_pipeline_create(slots, ctypes.byref(h)), "fp8_host_pipeline_create")
        self._h = h

    def step(self, slot: int, host: dict, dev: dict, ctx: LinearContext, ws: torch.Tensor,
             cache: WeightCache, h: int, recipe: str, version: int):
        """host: X, W, dY, Y, dX (or None), dW as CPU bf16 tensors; dev: X, dY, Y,
        dX (or None), dW as CUDA bf16 tensors (W goes to the buffer registered
        for handle h)."""
        N = host["X"].shape[0]
        hio = _HostIO(*[_ptr(host[k]) for k in ("X", "W", "dY", "Y", "dX", "dW")])
        dio = _DeviceIO(*[_ptr(dev[k]) for k in ("X", "dY", "Y", "dX", "dW")], _ptr(ctx.ctx),
                        _ptr(ws), ws.numel())
        _check(lib().fp8_linear_step_host(self._h, slot, N, ctypes.byref(hio), ctypes.byref(dio),
                                          cache.handle, h, RECIPE[recipe], version),
               "fp8_linear_step_host")

    def fork(self, stream=None):
        _check(lib().fp8_host_pipeline_fork(self._h, _stream(stream)), "fp8_host_pipeline_fork")

    def join(self, stream=None):
        _check(lib().fp8_host_pipeline_join(self._h, _stream(stream)), "fp8_host_pipeline_join")

    def sync(self):
        _check(lib().fp8_host_pipeline_sync(self._h), "fp8_host_pipeline_sync")

    def __del__(self):
        if getattr(self, "_h", None) is not None and _lib is not None:
            _lib.fp8_host_pipeline_destroy(self._h)
            self._h = None


def amax_partials_buffer(rows: int, cols: int, device) -> torch.Tensor:
    """Device buffer for fp8_amax_partials of a [rows, cols] tensor."""
    return _empty_bytes(_quant_ws_bytes("tensorwise", rows, cols), device)


def fp8_amax_partials(x: torch.Tensor, partials: torch.Tensor, stream=None) -> torch.Tensor:
    """First tensorwise pass alone (per-CTA maxima of |x|) into `partials`."""
    _need_bf16_cuda(x, "x")
    R, C = x.shape
    _check(lib().fp8_amax_partials(_ptr(x), R, C, _ptr(partials), partials.numel(),
                                   _stream(stream)), "fp8_amax_partials")
    return partials


def fp8_linear_fwd_after_amax(x: torch.Tensor, x_partials: torch.Tensor, cache: WeightCache,
                              h: int, recipe: str, ws: torch.Tensor, y: torch.Tensor,
                              ctx: LinearContext, stream=None):
    """fp8_linear_fwd with X's amax pass already run by fp8_amax_partials."""
    _need_bf16_cuda(x, "x")
    N, K = x.shape
    _check(lib().fp8_linear_fwd_after_amax(_ptr(x), _ptr(x_partials), N, K, cache.handle, h,
                                           RECIPE[recipe], _ptr(y), _ptr(ctx.ctx), _ptr(ws),
                                           ws.numel(), _stream(stream)),
           "fp8_linear_fwd_after_amax")
    return y, ctx


def fp8_linear_bwd_after_amax(dy: torch.Tensor, dy_partials: torch.Tensor, ctx: LinearContext,
                              cache: WeightCache, h: int, recipe: str, ws: torch.Tensor,
                              dx: torch.Tensor | None, dw: torch.Tensor, stream=None):
    """fp8_linear_bwd with dY's amax pass already run by fp8_amax_partials."""
    _need_bf16_cuda(dy, "dy")
    N, O = dy.shape
    _check(lib().fp8_linear_bwd_after_amax(_ptr(dy), _ptr(dy_partials), N, O, _ptr(ctx.ctx),
                                           cache.handle, h, RECIPE[recipe], _ptr(dx), _ptr(dw),
                                           _ptr(ws), ws.numel(), _stream(stream)),
           "fp8_linear_bwd_after_amax")
    return dx, dw


# ---------------------------------------------------------------- RMS norm
def _need(t, name, shape, dtype, dev):
    """dev: index of the CUDA device of the call's input."""
    if not (t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")


def _bytes(t, name, dev):
    """The size of a workspace."""
    if not (t.get_device() == dev and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous tensor on cuda:{dev}")
    return t.nbytes


class NormBuffers(dict):
    """Output buffers of fp8_rmsnorm_fwd.  Their shapes are checked on the first
    call that writes them and again after any change of the entries."""

    checked = None
    r_is_input = False  # the result of a call without a residual: r is its x, no buffer

    def __setitem__(self, key, value):
        self.checked = None
        if key == "r":
            self.r_is_input = False
        super().__setitem__(key, value)

    def __delitem__(self, key):
        self.checked = None
        super().__delitem__(key)

    def update(self, *args, **kw):
        for key, value in dict(*args, **kw).items():
            self[key] = value

    def __ior__(self, other):
        self.update(other)
        return self

    def setdefault(self, key, default=None):
        self.checked = None
        return super().setdefault(key, default)

    def pop(self, *args):
        self.checked = None
        return super().pop(*args)

    def popitem(self):
        self.checked = None
        return super().popitem()

    def clear(self):
        self.checked = None
        super().clear()

    def check(self, R, C, wanted, dev):
        """wanted: (r, rowwise, colwise, y) to be written for an [R, C] input on cuda:dev."""
        nb, rb = -(-C // 128), -(-R // 128)
        r, row, col, y = wanted
        bf16, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
        for key, want, shape, dtype in (
                ("rstd", True, (R,), f32), ("rstd_lo", col, (R,), f32), ("r", r, (R, C), bf16), ("y", y, (R, C), bf16),
                ("row", row, (R, C), u8), ("row_scale", row, (R, nb), f32),
                ("row_scale_inv", row, (R, nb), f32), ("col", col, (C, -(-R // 16) * 16), u8),
                ("col_scale", col, (C, rb), f32), ("col_scale_inv", col, (C, rb), f32)):
            if want:
                if self.get(key) is None or (key == "r" and self.r_is_input):
                    raise ValueError(f"out has no buffer for {key}")
                _need(self[key], key, shape, dtype, dev)
        self.checked = (R, C, wanted, dev)


def rmsnorm_buffers(R: int, C: int, device, residual: bool = True, rowwise: bool = True,
                    colwise: bool = True, bf16: bool = False) -> NormBuffers:
    """Output buffers of fp8_rmsnorm_fwd for an [R, C] input, to be passed as
    `out` by callers that keep them between calls (absent outputs are None)."""
    Rp, nb, rb = -(-R // 16) * 16, -(-C // 128), -(-R // 128)

    def f32(*shape):
        return torch.empty(shape, dtype=torch.float32, device=device)

    return NormBuffers(
        r=torch.empty((R, C), dtype=torch.bfloat16, device=device) if residual else None,
        rstd=f32(R), rstd_lo=f32(R) if colwise else None,
        y=torch.empty((R, C), dtype=torch.bfloat16, device=device) if bf16 else None,
        row=torch.empty((R, C), dtype=torch.uint8, device=device) if rowwise else None,
        row_scale=f32(R, nb) if rowwise else None, row_scale_inv=f32(R, nb) if rowwise else None,
        col=torch.empty((C, Rp), dtype=torch.uint8, device=device) if colwise else None,
        col_scale=f32(C, rb) if colwise else None, col_scale_inv=f32(C, rb) if colwise else None)


def rmsnorm_workspace(R: int, C: int, device) -> torch.Tensor:
    b = _c_sz()
    _check(lib().fp8_rmsnorm_workspace_size(R, C, ctypes.byref(b)), "fp8_rmsnorm_workspace_size")
    return _empty_bytes(b.value, device)


def fp8_rmsnorm_fwd(x: torch.Tensor, w: torch.Tensor, residual: torch.Tensor | None = None,
                    eps: float = 1e-6, rowwise: bool = True, colwise: bool = True,
                    bf16: bool = False, out: dict | None = None, stream=None) -> dict:
    """Residual addition, RMS norm and FP8 output of a bf16 [R, C] x; w is a
    bf16 or float32 [C].  Returns dict(r, rstd, rstd_lo, y, row, row_scale,
    row_scale_inv, col, col_scale, col_scale_inv), absent ones None: r is the
    residual stream bf16(x + residual) (x itself without a residual), row
    [R, C] and col [C, R rounded up to 16] the E4M3 bytes of the norm in 1x128
    blocks, y the norm in bf16.  out: buffers of rmsnorm_buffers to write."""
    _need_bf16_cuda(x, "x")
    R, C = x.shape
    dev = x.get_device()
    if w.dtype not in _DTYPE:
        raise ValueError("w must be bf16 or float32")
    _need(w, "w", (C,), w.dtype, dev)
    if residual is not None:
        _need(residual, "residual", (R, C), torch.bfloat16, dev)
    if out is None:
        with _on(stream):
            out = rmsnorm_buffers(R, C, x.device, residual is not None, rowwise, colwise, bf16)
    if not isinstance(out, NormBuffers):
        out = NormBuffers(out)
    wanted = (residual is not None, rowwise, colwise, bf16)
    if out.checked != (R, C, wanted, dev):
        out.check(R, C, wanted, dev)
    _check(lib().fp8_rmsnorm_fwd(
        x.data_ptr(), _ptr(residual), w.data_ptr(), _DTYPE[w.dtype], R, C, eps,
        _ptr(out["r"]) if residual is not None else None, out["rstd"].data_ptr(),
        _ptr(out["rstd_lo"]) if colwise else None, _ptr(out["y"]) if bf16 else None,
        _ptr(out["row"]) if rowwise else None, _ptr(out["col"]) if colwise else None,
        _ptr(out.get("row_scale")), _ptr(out.get("row_scale_inv")), _ptr(out.get("col_scale")),
        _ptr(out.get("col_scale_inv")), _stream(stream)), "fp8_rmsnorm_fwd")
    if residual is not None:
        return out
    result = NormBuffers(out, r=x)
    result.r_is_input = True
    return result


def fp8_rmsnorm_bwd(dy: torch.Tensor, r: torch.Tensor, rstd: torch.Tensor, w: torch.Tensor,
                    dr: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                    dw: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """Returns (dx, dw): dx bf16, the gradient of x and of the residual, dw
    float32; dr is the gradient that the stream r has from elsewhere."""
    _need_bf16_cuda(dy, "dy")
    R, C = dy.shape
    dev = dy.get_device()
    _need(r, "r", (R, C), torch.bfloat16, dev)
    _need(rstd, "rstd", (R,), torch.float32, dev)
    if w.dtype not in _DTYPE:
        raise ValueError("w must be bf16 or float32")
    _need(w, "w", (C,), w.dtype, dev)
    if dr is not None:
        _need(dr, "dr", (R, C), torch.bfloat16, dev)
    with _on(stream):
        if dx is None:
            dx = torch.empty_like(dy)
        if dw is None:
            dw = torch.empty(C, dtype=torch.float32, device=dy.device)
        if ws is None:
            ws = rmsnorm_workspace(R, C, dy.device)
    _need(dx, "dx", (R, C), torch.bfloat16, dev)
    _need(dw, "dw", (C,), torch.float32, dev)
    _check(lib().fp8_rmsnorm_bwd(_ptr(dy), _ptr(dr), _ptr(r), _ptr(rstd), _ptr(w), _DTYPE[w.dtype],
                                 R, C, _ptr(dx), _ptr(dw), _ptr(ws), _bytes(ws, "ws", dev), _stream(stream)),
           "fp8_rmsnorm_bwd")
    return dx, dw


# ---------------------------------------------------------------- gated feed-forward
@dataclass
class GatedContext:
    """What a gated forward pass keeps for its backward pass: the device buffer,
    its shape, and the activation and recipe (set by the forward pass; the
    recipes place and size what the buffer holds differently)."""
    ctx: torch.Tensor
    N: int
    K: int
    F: int
    act: str = "silu"
    recipe: str | None = None

    def check(self, recipe: str, N: int, K: int, F: int, dev: int):
        """Refuses a buffer that a call of this recipe and shape cannot use."""
        if (self.N, self.K, self.F) != (N, K, F):
            raise ValueError("ctx was made for another shape")
        if self.recipe is not None and (self.recipe == "block") != (recipe == "block"):
            raise ValueError(f"ctx was made for the {self.recipe} recipe")
        if _bytes(self.ctx, "ctx", dev) < _gated_ctx_bytes(recipe, N, K, F):
            raise ValueError("ctx is smaller than the recipe's context")


@functools.lru_cache(maxsize=256)
def _gated_ctx_bytes(recipe, N, K, F):
    b = _c_sz()
    _check(lib().fp8_gated_ctx_size(RECIPE[recipe], N, K, F, ctypes.byref(b)), "fp8_gated_ctx_size")
    return b.value


def gated_context(recipe: str, N: int, K: int, F: int, device) -> GatedContext:
    return GatedContext(_empty_bytes(_gated_ctx_bytes(recipe, N, K, F), device), N, K, F, recipe=recipe)


def gated_workspace(recipe: str, N: int, K: int, F: int, device, train: bool = True) -> torch.Tensor:
    b = _c_sz()
    _check(lib().fp8_gated_workspace_size(RECIPE[recipe], N, K, F, int(train), ctypes.byref(b)),
           "fp8_gated_workspace_size")
    return _empty_bytes(b.value, device)


def fp8_gated_ctx_layout(recipe: str, ctx: GatedContext):
    """Device pointers inside ctx: (transposed FP8 input, its scale, its
    scale_inv, G, U)."""
    ctx.check(recipe, ctx.N, ctx.K, ctx.F, ctx.ctx.get_device())
    p = [_c_p() for _ in range(5)]
    _check(lib().fp8_gated_ctx_layout(RECIPE[recipe], ctx.N, ctx.K, ctx.F, _ptr(ctx.ctx),
                                      *[ctypes.byref(q) for q in p]), "fp8_gated_ctx_layout")
    return tuple(p)


def gated_norm_columns(recipe: str, ctx: GatedContext) -> dict:
    """The transposed part of ctx as output buffers of fp8_rmsnorm_fwd (col,
    col_scale, col_scale_inv; block recipe), so that a norm fills the context
    that fp8_gated_fwd_quantized then uses."""
    if recipe != "block":
        raise ValueError("the norm's FP8 output is the block recipe's")
    p = fp8_gated_ctx_layout(recipe, ctx)
    base = ctx.ctx.data_ptr()
    Np, rb = -(-ctx.N // 16) * 16, -(-ctx.N // 128)

    def at(q, rows, cols, dtype, size):
        off = q.value - base
        return ctx.ctx[off:off + rows * cols * size].view(dtype).view(rows, cols)

    return dict(col=at(p[0], ctx.K, Np, torch.uint8, 1),
                col_scale=at(p[1], ctx.K, rb, torch.float32, 4),
                col_scale_inv=at(p[2], ctx.K, rb, torch.float32, 4))


def _gated_out(x, cache, h, recipe, y, ctx, train, stream):
    """(N, K, F, y, ctx) of a forward call on x [N, K], in bf16 or FP8."""
    N, K = x.shape
    if not 0 <= h < len(cache.entries):
        raise ValueError("no such weight handle")
    w = cache.entries[h].w
    dev = w.get_device()
    if x.get_device() != dev:
        raise ValueError(f"the input must be on cuda:{dev}, as the weight")
    F = w.shape[0] // 2
    if y is None or (train and ctx is None):
        with _on(stream):
            if y is None:
                y = torch.empty((N, F), dtype=torch.bfloat16, device=x.device)
            if train and ctx is None:
                ctx = gated_context(recipe, N, K, F, x.device)
    _need(y, "y", (N, F), torch.bfloat16, dev)
    if train:
        ctx.check(recipe, N, K, F, dev)
    return N, K, F, y, ctx if train else None


def fp8_gated_fwd(x: torch.Tensor, cache: WeightCache, h: int, recipe: str, act: str = "silu",
                  train: bool = True, ws: torch.Tensor | None = None, y: torch.Tensor | None = None,
                  ctx: GatedContext | None = None, stream=None):
    """H = act(X Wg^T) * (X Wu^T) for the weight [Wg; Wu] of handle h; returns
    (H, GatedContext), the context None with train=False."""
    _need_bf16_cuda(x, "x")
    N, K, F, y, ctx = _gated_out(x, cache, h, recipe, y, ctx, train, stream)
    if ws is None:
        with _on(stream):
            ws = gated_workspace(recipe, N, K, F, x.device, train=False)
    _check(lib().fp8_gated_fwd(_ptr(x), N, K, cache.handle, h, RECIPE[recipe], ACTIVATION[act],
                               _ptr(y), _ptr(ctx.ctx) if train else None, _ptr(ws),
                               _bytes(ws, "ws", x.get_device()), _stream(stream)), "fp8_gated_fwd")
    if train:
        ctx.act, ctx.recipe = act, recipe
    return y, ctx


def fp8_gated_fwd_quantized(row: torch.Tensor, row_scale_inv: torch.Tensor, cache: WeightCache,
                            h: int, recipe: str, act: str = "silu", y: torch.Tensor | None = None,
                            ctx: GatedContext | None = None, stream=None):
    """fp8_gated_fwd on an input given as E4M3 bytes [N, K] and scale_inv
    ([N, ceil(K / 128)] under the block recipe, else one); with ctx its
    transposed part (fp8_gated_ctx_layout) is already filled."""
    if not (row.is_cuda and row.dtype == torch.uint8 and row.is_contiguous()):
        raise ValueError("row must be a contiguous uint8 CUDA tensor")
    N, K = row.shape
    nb = -(-K // 128)
    t = row_scale_inv
    if not (t.get_device() == row.get_device() and t.dtype == torch.float32 and t.is_contiguous()):
        raise ValueError("row_scale_inv must be a contiguous float32 tensor on the device of row")
    if not (t.shape in ((N, nb), (N * nb,)) if recipe == "block" else t.numel() == 1):
        raise ValueError(f"row_scale_inv must hold {f'{N} x {nb} values' if recipe == 'block' else 'one value'}")
    _, _, _, y, ctx = _gated_out(row, cache, h, recipe, y, ctx, ctx is not None, stream)
    _check(lib().fp8_gated_fwd_quantized(_ptr(row), _ptr(row_scale_inv), N, K, cache.handle, h,
                                         RECIPE[recipe], ACTIVATION[act], _ptr(y),
                                         None if ctx is None else _ptr(ctx.ctx), _stream(stream)),
           "fp8_gated_fwd_quantized")
    if ctx is not None:
        ctx.act, ctx.recipe = act, recipe
    return y, ctx


def fp8_gated_bwd(dh: torch.Tensor, ctx: GatedContext, cache: WeightCache, h: int, recipe: str,
                  need_dx: bool = True, ws: torch.Tensor | None = None,
                  dx: torch.Tensor | None = None, dw: torch.Tensor | None = None, stream=None):
    """Returns (dX or None, dW [2F, K]) of the forward pass that made ctx."""
    if not 0 <= h < len(cache.entries):
        raise ValueError("no such weight handle")
    w = cache.entries[h].w
    N, K, F, dev = ctx.N, ctx.K, ctx.F, w.get_device()
    _need(dh, "dh", (N, F), torch.bfloat16, dev)
    ctx.check(recipe, N, K, F, dev)
    if w.shape != (2 * F, K):
        raise ValueError("ctx was made with a weight of another shape")
    with _on(stream):
        if need_dx and dx is None:
            dx = torch.empty((N, K), dtype=torch.bfloat16, device=w.device)
        if dw is None:
            dw = torch.empty((2 * F, K), dtype=torch.bfloat16, device=w.device)
        if ws is None:
            ws = gated_workspace(recipe, N, K, F, w.device)
    if need_dx:
        _need(dx, "dx", (N, K), torch.bfloat16, dev)
    _need(dw, "dw", (2 * F, K), torch.bfloat16, dev)
    _check(lib().fp8_gated_bwd(_ptr(dh), N, F, _ptr(ctx.ctx), cache.handle, h, RECIPE[recipe],
                               ACTIVATION[ctx.act], _ptr(dx) if need_dx else None, _ptr(dw),
                               _ptr(ws), _bytes(ws, "ws", dev), _stream(stream)), "fp8_gated_bwd")
    return (dx if need_dx else None), dw


# ---------------------------------------------------------------- gradient clipping
def _disjoint(src, dst):
    """Each dst is its own src or apart from it, and apart from all others."""
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), i, w)
             for w, ts in enumerate((src, dst)) for i, t in enumerate(ts) if t.numel()]
    far = ([], [])  # the two furthest ends so far of sources and of outputs (one may be the tensor's own)
    for lo, hi, i, w in sorted(spans):
        for w2 in (0, 1):
            for hi2, lo2, i2 in far[w2]:
                if lo < hi2 and (w or w2) and not (w != w2 and i == i2 and (lo, hi) == (lo2, hi2)):
                    raise ValueError("clipped tensors must not overlap (out may be the gradients themselves)")
        far[w][:] = sorted(far[w] + [(hi, lo, i)])[-2:]


class GradClip:
    """Global norm and clipping of a fixed set of gradient tensors (bf16 or
    float32, contiguous, any sizes).  out: tensors of the same types and sizes
    that take the clipped gradients; by default the gradients themselves.

    The plan is for the memory that the tensors have when it is made, and keeps
    that memory: right for gradients that stay where they are (accumulators,
    flat buffers).  Gradients allocated anew, or moved by `g.data = ...`, need a
    new plan (a table of 24 bytes per 8192 to 32768 elements, made on the host
    and uploaded with a synchronisation).  Calls of one plan share its workspace,
    so they have to follow one another (on one stream, or with a wait between
    streams)."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError("out must have one tensor per gradient")
        for g, o in zip(self.grads, self.out):
            if g.dtype not in _DTYPE or not g.is_cuda:
                raise ValueError("gradients must be bf16 or float32 CUDA tensors")
            dev = self.grads[0].get_device()
            _need(g, "gradient", g.shape, g.dtype, dev)
            _need(o, "out", g.shape, g.dtype, dev)
        _disjoint(self.grads, self.out)
        self._memory = [t.detach() for t in self.grads + self.out]
        n = len(self.grads)
        descs = (_GradDesc * max(n, 1))(*[_GradDesc(g.data_ptr(), o.data_ptr(), g.numel(),
                                                    _DTYPE[g.dtype])
                                          for g, o in zip(self.grads, self.out)])
        h = _c_p()
        _check(lib().fp8_grad_clip_create(descs, n, ctypes.byref(h)), "fp8_grad_clip_create")
        self._h = h
        b = _c_sz()
        _check(lib().fp8_grad_clip_table_size(h, ctypes.byref(b)), "fp8_grad_clip_table_size")
        host = torch.empty(max(b.value, 16), dtype=torch.uint8)
        _check(lib().fp8_grad_clip_table_write(h, _ptr(host), host.numel()),
               "fp8_grad_clip_table_write")
        dev = self.grads[0].device if n else torch.device("cuda")
        _check(lib().fp8_grad_clip_workspace_size(h, ctypes.byref(b)),
               "fp8_grad_clip_workspace_size")
        self._ws = _empty_bytes(b.value, dev)
        # the upload returns once it is done, and all that this stream had queued
        # before it: from here on any stream may use the table and the workspace
        self._table = host.to(dev)
        self._streams = {_stream()}
        self._device = dev
        self._norms, self._norms_on = [], None  # norms not yet handed out

    def _begin(self, stream):
        """(cudaStream_t, norm) of a call.  The plan's memory outlives the work there.
        The norm is one of 64 allocated together on the current stream (nine
        vectors, a call with an allocation 9.4 us, here 6.9); that of a captured
        call comes from the graph's pool, which lives as long as its replays."""
        raw = _stream(stream)
        if raw not in self._streams:
            s = torch.cuda.current_stream() if stream is None else stream
            for t in (self._table, self._ws):
                t.record_stream(s)
            self._streams.add(raw)
        if stream is None and not torch._C._cuda_isCurrentStreamCapturing():
            if not self._norms or raw != self._norms_on:
                block = torch.empty(64, dtype=torch.float32, device=self._device)
                self._norms, self._norms_on = list(block.split(1)), raw
            return raw, self._norms.pop()
        with _on(stream):
            return raw, torch.empty(1, dtype=torch.float32, device=self._device)

    def clip(self, max_norm: float, stream=None):
        """Scales the gradients to a global norm of at most max_norm; returns
        (norm, out), the norm as a new float32 device tensor of the unclipped
        gradients.  A norm that is not finite leaves them as they are."""
        raw, norm = self._begin(stream)
        _check(lib().fp8_grad_clip_run(self._h, self._table.data_ptr(), max_norm, norm.data_ptr(),
                                       self._ws.data_ptr(), self._ws.numel(), raw), "fp8_grad_clip_run")
        return norm, self.out

    def norm(self, stream=None) -> torch.Tensor:
        """The global norm alone (a new float32 device tensor)."""
        raw, norm = self._begin(stream)
        _check(lib().fp8_grad_norm(self._h, self._table.data_ptr(), norm.data_ptr(), self._ws.data_ptr(),
                                   self._ws.numel(), raw), "fp8_grad_norm")
        return norm

    def __del__(self):
        if getattr(self, "_h", None) is not None and _lib is not None:
            _lib.fp8_grad_clip_destroy(self._h)
            self._h = None


# ---------------------------------------------------------------- routing to experts
def _here(t, name, stream):
    """Index of t's device, which has to be the one that the call's stream is on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if torch.cuda.is_initialized():
        on = torch._C._cuda_getDevice() if stream is None else stream.device_index
        if on != dev:
            raise ValueError(f"{name} is on cuda:{dev}, the call's stream on cuda:{on}")
    return dev


def _route_input(logits, k, stream):
    if logits.dtype not in _DTYPE or logits.dim() != 2 or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous bf16 or float32 tensor [T, E]")
    return (*logits.shape, _here(logits, "logits", stream))


def fp8_route_fwd(logits: torch.Tensor, k: int, score: str = "softmax", bias: torch.Tensor | None = None,
                  groups: int = 1, groups_kept: int | None = None, group_top: int = 1,
                  renormalize: bool = True, scale: float = 1.0,
                  out: tuple[torch.Tensor, torch.Tensor] | None = None, stream=None):
    """The k experts of each token and their weights, from logits [T, E] in bf16
    or float32; returns (weights float32 [T, k], experts int32 [T, k]).  bias:
    float32 [E], added to the scores for the choice alone; groups: only experts
    of the groups_kept best of that many groups (by the sum of a group's
    group_top best scores) are chosen.  Experts with a logit of -inf are never
    chosen: slots left over have expert -1 and weight 0.  out: tensors to write."""
    T, E, dev = _route_input(logits, k, stream)
    if bias is not None:
        _need(bias, "bias", (E,), torch.float32, dev)
    if out is None:
        with _on(stream):
            w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
            e = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    else:
        w, e = out
        _need(w, "weights", (T, k), torch.float32, dev)
        _need(e, "experts", (T, k), torch.int32, dev)
    _check(lib().fp8_route_fwd(logits.data_ptr(), _DTYPE[logits.dtype], _ptr(bias), T, E, k, SCORE[score], groups,
                               groups if groups_kept is None else groups_kept, group_top, renormalize, scale,
                               w.data_ptr(), e.data_ptr(), _stream(stream)), "fp8_route_fwd")
    return w, e


def fp8_route_bwd(dweights: torch.Tensor, logits: torch.Tensor, weights: torch.Tensor, experts: torch.Tensor,
                  score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of the logits [T, E], in their type, from that of the weights;
    logits, weights, experts, score, renormalize and scale of fp8_route_fwd."""
    k = experts.shape[-1]
    T, E, dev = _route_input(logits, k, stream)
    _need(experts, "experts", (T, k), torch.int32, dev)
    _need(weights, "weights", (T, k), torch.float32, dev)
    _need(dweights, "dweights", (T, k), torch.float32, dev)
    if out is None:
        with _on(stream):
            out = torch.empty_like(logits)
    else:
        _need(out, "out", (T, E), logits.dtype, dev)
    _check(lib().fp8_route_bwd(dweights.data_ptr(), logits.data_ptr(), _DTYPE[logits.dtype], weights.data_ptr(),
                               experts.data_ptr(), T, E, k, SCORE[score], renormalize, scale, out.data_ptr(),
                               _stream(stream)), "fp8_route_bwd")
    return out


# ---------------------------------------------------------------- rows in the experts' order
class ExpertOrder:
    """The T k slots (t k + j: choice j of token t) sorted by expert.  counts [E]
    and offsets [E + 1]: rows of each expert, where they begin (multiples of
    align), and the rows in use; position [T, k]: a slot's row, -1 without an
    expert; order [rows]: a row's slot, -1 in the gap behind an expert's rows,
    undefined past offsets[E].  rows: the rows that any choice can need.  The
    tensors are views of one int32 buffer, made when asked for."""

    __slots__ = ("T", "k", "E", "align", "rows", "buffer", "device", "_at", "_views")

    def __init__(self, T: int, k: int, E: int, align: int, device):
        self.T, self.k, self.E, self.align = T, k, E, align
        self.rows = expert_rows(T, k, E, align)
        self.buffer = torch.empty(2 * E + 1 + T * k + self.rows, dtype=torch.int32, device=device)
        self.device = self.buffer.get_device()
        at = self.buffer.data_ptr()
        # addresses of counts, offsets, position and order
        self._at = (at, at + 4 * E, at + 4 * (2 * E + 1), at + 4 * (2 * E + 1 + T * k))
        self._views = None

    def _view(self, i):
        if self._views is None:
            c, o, p, r = torch.unsafe_split_with_sizes(self.buffer, (self.E, self.E + 1, self.T * self.k, self.rows))
            self._views = (c, o, p.view(self.T, self.k), r)
        return self._views[i]

    counts = property(lambda self: self._view(0))
    offsets = property(lambda self: self._view(1))
    position = property(lambda self: self._view(2))
    order = property(lambda self: self._view(3))


@functools.lru_cache(maxsize=1024)
def expert_rows(T: int, k: int, n_experts: int, align: int = 1) -> int:
    """Rows of a buffer in the experts' order that any choice fits."""
    return int(lib().fp8_expert_rows(T * k, n_experts, align))


@functools.lru_cache(maxsize=1024)
def _order_bytes(slots, E):
    b = _c_sz()
    _check(lib().fp8_expert_order_workspace_size(slots, E, ctypes.byref(b)), "fp8_expert_order_workspace_size")
    return b.value


def fp8_expert_order(experts: torch.Tensor, n_experts: int, align: int = 1, out: ExpertOrder | None = None,
                     ws: torch.Tensor | None = None, stream=None) -> ExpertOrder:
    """The order of the choices experts int32 [T, k] (values outside 0 ..
    n_experts - 1: no expert).  align = 16 gives every expert a row count that
    the FP8 linear takes.  out: an order of the same shape to write again."""
    if experts.dtype != torch.int32 or experts.dim() != 2 or not experts.is_contiguous():
        raise ValueError("experts must be a contiguous int32 tensor [T, k]")
    dev = _here(experts, "experts", stream)
    T, k = experts.shape
    E, slots = n_experts, T * k
    need = _order_bytes(slots, E)
    if out is None:
        with _on(stream):
            out = ExpertOrder(T, k, E, align, experts.device)
    elif (out.T, out.k, out.E, out.align, out.device) != (T, k, E, align, dev):
        raise ValueError("out is an order of another shape or device")
    if ws is None and need:
        with _on(stream):
            ws = _empty_bytes(need, experts.device)
    _check(lib().fp8_expert_order(experts.data_ptr(), slots, E, align, *out._at, _ptr(ws),
                                  0 if ws is None else _bytes(ws, "ws", dev), _stream(stream)), "fp8_expert_order")
    return out


def _order_on(order: ExpertOrder, dev: int):
    if order.device != dev:
        raise ValueError(f"order must be on cuda:{dev}")


def fp8_expert_gather(x: torch.Tensor, order: ExpertOrder, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Token rows x [T, C] in the experts' order: [order.rows, C], zeros in the
    gaps between experts, rows past order.offsets[E] as they were."""
    _need_bf16_cuda(x, "x")
    dev = _here(x, "x", stream)
    _order_on(order, dev)
    T, C = x.shape
    if T != order.T:
        raise ValueError(f"x must have {order.T} rows")
    if out is None:
        with _on(stream):
            out = torch.empty((order.rows, C), dtype=torch.bfloat16, device=x.device)
    else:
        _need(out, "out", (order.rows, C), torch.bfloat16, dev)
    counts, offsets, position, _ = order._at
    _check(lib().fp8_expert_gather(x.data_ptr(), T, C, order.k, order.E, order.align, counts, offsets, position,
                                   out.data_ptr(), _stream(stream)), "fp8_expert_gather")
    return out


def fp8_expert_combine(z: torch.Tensor, order: ExpertOrder, weights: torch.Tensor | None = None,
                       out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] z[row of (t, j)], [T, C]; without weights the
    plain sum, which is the backward pass of fp8_expert_gather."""
    _need_bf16_cuda(z, "z")
    dev = _here(z, "z", stream)
    _order_on(order, dev)
    T, k = order.T, order.k
    rows, C = z.shape
    if rows != order.rows:
        raise ValueError(f"z must have {order.rows} rows")
    if weights is not None:
        _need(weights, "weights", (T, k), torch.float32, dev)
    if out is None:
        with _on(stream):
            out = torch.empty((T, C), dtype=torch.bfloat16, device=z.device)
    else:
        _need(out, "out", (T, C), torch.bfloat16, dev)
    _check(lib().fp8_expert_combine(z.data_ptr(), T, C, k, order._at[2], _ptr(weights), out.data_ptr(),
                                    _stream(stream)), "fp8_expert_combine")
    return out


def fp8_expert_combine_bwd(dy: torch.Tensor, z: torch.Tensor, order: ExpertOrder, weights: torch.Tensor,
                           dz: torch.Tensor | None = None, dweights: torch.Tensor | None = None, stream=None):
    """Returns (dz [order.rows, C], dweights float32 [T, k]); dz is zero in the
    gaps between experts and as it was past order.offsets[E]."""
    _need_bf16_cuda(dy, "dy")
    dev = _here(dy, "dy", stream)
    _order_on(order, dev)
    T, k, C = order.T, order.k, dy.shape[-1]
    _need(dy, "dy", (T, C), torch.bfloat16, dev)
    _need(z, "z", (order.rows, C), torch.bfloat16, dev)
    _need(weights, "weights", (T, k), torch.float32, dev)
    if dz is None or dweights is None:
        with _on(stream):
            if dz is None:
                dz = torch.empty_like(z)
            if dweights is None:
                dweights = torch.empty((T, k), dtype=torch.float32, device=dy.device)
    _need(dz, "dz", (order.rows, C), torch.bfloat16, dev)
    _need(dweights, "dweights", (T, k), torch.float32, dev)
    counts, offsets, position, _ = order._at
    _check(lib().fp8_expert_combine_bwd(dy.data_ptr(), z.data_ptr(), T, C, k, order.E, order.align, counts, offsets,
                                        position, weights.data_ptr(), dz.data_ptr(), dweights.data_ptr(),
                                        _stream(stream)), "fp8_expert_combine_bwd")
    return dz, dweights


# ---------------------------------------------------------------- 4-bit weights
class W4Weight:
    """A 4-bit weight [N, K], or a stack [E, N, K]: codes uint8 [..., K / 2] (the
    even k in the low four bits), scale bf16 and zero uint8 [..., ceil(K / group)]
    (zero None: 8), W = scale * (code - zero) in groups of 32, 64 or 128 along K."""

    __slots__ = ("codes", "scale", "zero", "group", "E", "N", "K", "stack", "device", "_c")

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor | None = None,
                 group: int = 128):
        if codes.dtype != torch.uint8 or codes.dim() not in (2, 3) or not codes.is_cuda or not codes.is_contiguous():
            raise ValueError("codes must be a contiguous uint8 CUDA tensor [N, K / 2] or [E, N, K / 2]")
        if group not in (32, 64, 128):
            raise ValueError("group must be 32, 64 or 128")
        dev = codes.get_device()
        self.stack = codes.dim() == 3
        self.E = codes.shape[0] if self.stack else 1
        self.N, self.K = codes.shape[-2], 2 * codes.shape[-1]
        if self.N % 16 or self.K % 32:
            raise ValueError("a 4-bit weight has rows in multiples of 16 and K in multiples of 32")
        shape = (*codes.shape[:-1], -(-self.K // group))
        _need(scale, "scale", shape, torch.bfloat16, dev)
        if zero is not None:
            _need(zero, "zero", shape, torch.uint8, dev)
        self.codes, self.scale, self.zero, self.group, self.device = codes, scale, zero, group, codes.device
        self._c = _W4(codes.data_ptr(), scale.data_ptr(), _ptr(zero), self.E, self.N, self.K, group)


def fp8_w4_quantize(w: torch.Tensor, group: int = 128, zero: bool = False, stream=None) -> W4Weight:
    """4-bit codes, scales (and zero points) of a bf16 weight [N, K] or stack
    [E, N, K], rounded to the nearest."""
    _need_bf16_cuda(w, "w")
    _here(w, "w", stream)
    if w.dim() not in (2, 3):
        raise ValueError("w must be [N, K] or [E, N, K]")
    K = w.shape[-1]
    if K % 32 or w.shape[-2] % 16 or group not in (32, 64, 128):
        raise ValueError("a 4-bit weight has rows in multiples of 16, K in multiples of 32 and groups of 32, 64 or 128")
    shape = (*w.shape[:-1], -(-K // group))
    with _on(stream):
        codes = torch.empty((*w.shape[:-1], K // 2), dtype=torch.uint8, device=w.device)
        scale = torch.empty(shape, dtype=torch.bfloat16, device=w.device)
        z = torch.empty(shape, dtype=torch.uint8, device=w.device) if zero else None
    _check(lib().fp8_w4_quantize(w.data_ptr(), w.shape[:-1].numel(), K, group, codes.data_ptr(), scale.data_ptr(),
                                 _ptr(z), _stream(stream)), "fp8_w4_quantize")
    return W4Weight(codes, scale, z, group)


def _w4_input(x, w, stream):
    _need_bf16_cuda(x, "x")
    dev = _here(x, "x", stream)
    if x.dim() != 2 or x.shape[1] != w.K:
        raise ValueError(f"x must be [T, {w.K}]")
    if w.device != x.device:
        raise ValueError("the weight must be on the device of x")
    return x.shape[0], dev


@functools.lru_cache(maxsize=1024)
def _w4_bytes(N, K, group, T, gated):
    b = _c_sz()
    any_address = 16  # the size depends on the shape alone
    _check(lib().fp8_w4_workspace_size(_W4(any_address, any_address, None, 1, N, K, group), T, gated, ctypes.byref(b)),
           "fp8_w4_workspace_size")
    return b.value


def w4_workspace(w: W4Weight, T: int, gated: bool = False) -> torch.Tensor:
    """Workspace of fp8_w4_linear or fp8_w4_gated for callers that keep it."""
    return _empty_bytes(_w4_bytes(w.N, w.K, w.group, T, gated), w.device)


def _w4_ws(w, T, gated, ws, dev, stream):
    """(tensor, pointer, bytes) of a call's workspace."""
    if ws is None:
        need = _w4_bytes(w.N, w.K, w.group, T, gated)
        if not need:
            return None, None, 0
        with _on(stream):
            ws = _empty_bytes(need, w.device)
    return ws, ws.data_ptr(), _bytes(ws, "ws", dev)


def fp8_w4_linear(x: torch.Tensor, w: W4Weight, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """y [T, N] = x W^T for bf16 x [T, K], written for few tokens."""
    T, dev = _w4_input(x, w, stream)
    if w.stack:
        raise ValueError("w is a stack of weights")
    if out is None:
        with _on(stream):
            out = torch.empty((T, w.N), dtype=torch.bfloat16, device=x.device)
    else:
        _need(out, "out", (T, w.N), torch.bfloat16, dev)
    ws, at, size = _w4_ws(w, T, False, ws, dev, stream)
    _check(lib().fp8_w4_linear(x.data_ptr(), T, w._c, out.data_ptr(), at, size, _stream(stream)), "fp8_w4_linear")
    return out


def fp8_w4_gated(x: torch.Tensor, w: W4Weight, act: str = "silu", out: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h [T, F] = act(x Wg^T) * (x Wu^T) for the weight [Wg; Wu] of 2F rows."""
    T, dev = _w4_input(x, w, stream)
    if w.stack or w.N % 32:
        raise ValueError("w must be one weight with an even number of 16-row blocks")
    if out is None:
        with _on(stream):
            out = torch.empty((T, w.N // 2), dtype=torch.bfloat16, device=x.device)
    else:
        _need(out, "out", (T, w.N // 2), torch.bfloat16, dev)
    ws, at, size = _w4_ws(w, T, True, ws, dev, stream)
    _check(lib().fp8_w4_gated(x.data_ptr(), T, w._c, ACTIVATION[act], out.data_ptr(), at, size, _stream(stream)),
           "fp8_w4_gated")
    return out


@functools.lru_cache(maxsize=256)
def _w4_experts_bytes(T, k, E, K, F, N):
    b = _c_sz()
    _check(lib().fp8_w4_experts_workspace_size(T, k, E, K, F, N, ctypes.byref(b)), "fp8_w4_experts_workspace_size")
    return b.value


def w4_experts_workspace(T: int, k: int, gate_up: W4Weight, down: W4Weight) -> torch.Tensor:
    return _empty_bytes(_w4_experts_bytes(T, k, gate_up.E, gate_up.K, down.K, down.N), gate_up.device)


def fp8_w4_experts(x: torch.Tensor, weights: torch.Tensor, experts: torch.Tensor, gate_up: W4Weight, down: W4Weight,
                   act: str = "silu", ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """y [T, N] = sum_j weights[t, j] (act(x Wg_e^T) * (x Wu_e^T)) Wd_e^T with e =
    experts[t, j]: the gated MLP of each token's experts, gate_up a stack [E, 2F,
    K], down one [E, N, F].  weights and experts [T, k] as of fp8_route_fwd.  ws:
    a w4_experts_workspace, of one call at a time."""
    T, dev = _w4_input(x, gate_up, stream)
    k = experts.shape[-1]
    _need(experts, "experts", (T, k), torch.int32, dev)
    _need(weights, "weights", (T, k), torch.float32, dev)
    if gate_up.N != 2 * down.K or gate_up.E != down.E or down.device != x.device:
        raise ValueError("gate_up [E, 2F, K] and down [E, N, F] do not belong together")
    if out is None or ws is None:
        with _on(stream):
            if out is None:
                out = torch.empty((T, down.N), dtype=torch.bfloat16, device=x.device)
            if ws is None:
                ws = w4_experts_workspace(T, k, gate_up, down)
    _need(out, "out", (T, down.N), torch.bfloat16, dev)
    _check(lib().fp8_w4_experts(x.data_ptr(), T, k, weights.data_ptr(), experts.data_ptr(), gate_up._c, down._c,
                                ACTIVATION[act], out.data_ptr(), ws.data_ptr(), _bytes(ws, "ws", dev),
                                _stream(stream)), "fp8_w4_experts")
    return out
