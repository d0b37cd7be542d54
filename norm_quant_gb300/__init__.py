"""MoE combine/finalize, few-token serving operators and the feed-forward
block for many tokens on one GB300 -- Python binding of ``libnqg.so``.

Argument marshalling only: every step of the path runs in the library's
CUDA kernels.  Tensors are torch CUDA tensors (torch provides device memory
and streams); bf16 tensors may be ``torch.bfloat16`` or raw 16-bit views.
The entry points have the names of the C ABI in ``include/moe_combine.h``,
``include/moe_layer.h`` and ``include/moe_block.h``.

There is no fallback: if the library is not built, every call raises.
Build it with ``norm_quant_gb300.build.build()`` (``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes as C
import os
import struct
import threading

from .build import LIB_PATH, build  # noqa: F401  (re-exported)

QUANT = {None: 0, "none": 0, "mxfp8": 1, "nvfp4": 2, "mxfp4": 3}
IO_DTYPE = {"bf16": 0, "fp16": 1}
WEIGHT_DTYPE = {"fp32": 0, "bf16": 1, "fp16": 2}
LAYOUT = {"linear": 0, "swizzled": 1, "128x4": 1}
W_FORMAT = {None: 0, "none": 0, "nvfp4": 1, "int4": 2}
SCORING = {"softmax": 0, "sigmoid": 1}
ACTIVATION = {"silu": 0, "gelu_tanh": 1}
GATE = {None: 0, "none": 0, "channel": 1, "token": 2}
FEW_TOKENS = 64  # MOE_FEW_TOKENS
EXPERT_LAYOUT = {"grouped": 0, "slot_major": 1}
MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_INVALID_EXPERT = 4
MOE_ERR_CUDA = 5
MOE_ERR_ROW_OUT_OF_RANGE = 6
MOE_ERR_DEVICE_TIMEOUT = 7
ABI_VERSION = 4


class MoeCombineArgs(C.Structure):
    """Mirror of ``moe_combine_args`` (include/moe_combine.h)."""
    _fields_ = [
        ("T", C.c_int64), ("H", C.c_int32), ("top_k", C.c_int32),
        ("expert_out", C.c_void_p), ("n_expert_rows", C.c_int64),
        ("row_map", C.c_void_p), ("router_weights", C.c_void_p),
        ("shared_out", C.c_void_p), ("residual", C.c_void_p), ("gamma", C.c_void_p),
        ("eps", C.c_float), ("weight_bias", C.c_float),
        ("quant", C.c_int32), ("sf_layout", C.c_int32), ("global_scale", C.c_float),
        ("expert_layout", C.c_int32),
        ("combined_out", C.c_void_p), ("residual_out", C.c_void_p), ("norm_out", C.c_void_p),
        ("quant_out", C.c_void_p), ("scales_out", C.c_void_p), ("status", C.c_void_p),
        ("io_dtype", C.c_int32), ("weight_dtype", C.c_int32),
    ]


class MoeLinearW4Args(C.Structure):
    """Mirror of ``moe_linear_w4_args`` (include/moe_layer.h)."""
    _fields_ = [
        ("M", C.c_int64), ("N", C.c_int32), ("K", C.c_int32),
        ("x", C.c_void_p), ("x_stride", C.c_int64),
        ("w", C.c_void_p), ("w_scales", C.c_void_p), ("w_zeros", C.c_void_p),
        ("global_scale", C.c_float), ("w_format", C.c_int32), ("group_size", C.c_int32), ("io_dtype", C.c_int32),
        ("out", C.c_void_p), ("out_stride", C.c_int64),
    ]


class MoeLayerArgs(C.Structure):
    """Mirror of ``moe_layer_args`` (include/moe_layer.h)."""
    _fields_ = [
        ("T", C.c_int64), ("H", C.c_int32), ("I", C.c_int32), ("E", C.c_int32), ("top_k", C.c_int32),
        ("x", C.c_void_p), ("x_stride", C.c_int64), ("topk_ids", C.c_void_p), ("router_weights", C.c_void_p),
        ("w13", C.c_void_p), ("w13_scales", C.c_void_p), ("w13_zeros", C.c_void_p), ("w13_global", C.c_void_p),
        ("w2", C.c_void_p), ("w2_scales", C.c_void_p), ("w2_zeros", C.c_void_p), ("w2_global", C.c_void_p),
        ("shared_out", C.c_void_p), ("residual", C.c_void_p), ("out", C.c_void_p),
        ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t), ("status", C.c_void_p),
        ("w_format", C.c_int32), ("group_size", C.c_int32), ("activation", C.c_int32),
        ("io_dtype", C.c_int32), ("weight_dtype", C.c_int32),
    ]


class MoeGatedLinearArgs(C.Structure):
    """Mirror of ``moe_gated_linear_args`` (include/moe_block.h)."""
    _fields_ = [
        ("rows", C.c_int64), ("H", C.c_int32), ("I", C.c_int32), ("E", C.c_int32), ("activation", C.c_int32),
        ("offsets", C.c_void_p), ("x", C.c_void_p), ("x_stride", C.c_int64), ("w13", C.c_void_p),
        ("gate_up", C.c_void_p), ("gate_up_stride", C.c_int64), ("out", C.c_void_p), ("out_stride", C.c_int64),
        ("status", C.c_void_p), ("io_dtype", C.c_int32),
    ]


class MoeGatedLinearBackwardArgs(C.Structure):
    """Mirror of ``moe_gated_linear_backward_args`` (include/moe_block.h)."""
    _fields_ = [
        ("rows", C.c_int64), ("H", C.c_int32), ("I", C.c_int32), ("E", C.c_int32), ("activation", C.c_int32),
        ("offsets", C.c_void_p), ("d_out", C.c_void_p), ("d_out_stride", C.c_int64), ("gate_up", C.c_void_p),
        ("gate_up_stride", C.c_int64), ("x", C.c_void_p), ("x_stride", C.c_int64), ("w13", C.c_void_p),
        ("d_x", C.c_void_p), ("d_x_stride", C.c_int64), ("d_w13", C.c_void_p), ("workspace", C.c_void_p),
        ("workspace_bytes", C.c_size_t), ("status", C.c_void_p), ("io_dtype", C.c_int32), ("grad_dtype", C.c_int32),
    ]


class MoeGroupedLinearArgs(C.Structure):
    """Mirror of ``moe_grouped_linear_args`` (include/moe_block.h)."""
    _fields_ = [
        ("rows", C.c_int64), ("K", C.c_int32), ("N", C.c_int32), ("E", C.c_int32), ("io_dtype", C.c_int32),
        ("offsets", C.c_void_p), ("x", C.c_void_p), ("x_stride", C.c_int64), ("w", C.c_void_p), ("out", C.c_void_p),
        ("out_stride", C.c_int64), ("status", C.c_void_p),
    ]


class MoeGroupedLinearBackwardArgs(C.Structure):
    """Mirror of ``moe_grouped_linear_backward_args`` (include/moe_block.h)."""
    _fields_ = [
        ("rows", C.c_int64), ("K", C.c_int32), ("N", C.c_int32), ("E", C.c_int32), ("io_dtype", C.c_int32),
        ("offsets", C.c_void_p), ("d_out", C.c_void_p), ("d_out_stride", C.c_int64), ("x", C.c_void_p),
        ("x_stride", C.c_int64), ("w", C.c_void_p), ("d_x", C.c_void_p), ("d_x_stride", C.c_int64),
        ("d_w", C.c_void_p), ("status", C.c_void_p), ("grad_dtype", C.c_int32),
    ]


class MoeBlockNormArgs(C.Structure):
    """Mirror of ``moe_block_norm_args`` (include/moe_block.h)."""
    _fields_ = [
        ("T", C.c_int64), ("H", C.c_int32), ("io_dtype", C.c_int32), ("y", C.c_void_p), ("residual", C.c_void_p),
        ("post_gamma", C.c_void_p), ("pre_gamma", C.c_void_p), ("gate", C.c_void_p), ("gate_kind", C.c_int32),
        ("block_scale", C.c_float), ("residual_scale", C.c_float), ("eps", C.c_float), ("weight_bias", C.c_float),
        ("residual_out", C.c_void_p), ("norm_out", C.c_void_p),
    ]


class MoeBlockNormBackwardArgs(C.Structure):
    """Mirror of ``moe_block_norm_backward_args`` (include/moe_block.h)."""
    _fields_ = [
        ("T", C.c_int64), ("H", C.c_int32), ("io_dtype", C.c_int32), ("y", C.c_void_p), ("residual", C.c_void_p),
        ("post_gamma", C.c_void_p), ("pre_gamma", C.c_void_p), ("gate", C.c_void_p), ("gate_kind", C.c_int32),
        ("block_scale", C.c_float), ("residual_scale", C.c_float), ("eps", C.c_float), ("weight_bias", C.c_float),
        ("d_residual_out", C.c_void_p), ("d_norm_out", C.c_void_p), ("d_y", C.c_void_p), ("d_residual", C.c_void_p),
        ("d_post_gamma", C.c_void_p), ("d_pre_gamma", C.c_void_p), ("d_gate", C.c_void_p), ("workspace", C.c_void_p),
        ("workspace_bytes", C.c_size_t),
    ]


_BLOCK_ARGS = {"moe_gated_linear": MoeGatedLinearArgs, "moe_gated_linear_backward": MoeGatedLinearBackwardArgs,
               "moe_grouped_linear": MoeGroupedLinearArgs, "moe_grouped_linear_backward": MoeGroupedLinearBackwardArgs,
               "moe_block_norm": MoeBlockNormArgs, "moe_block_norm_backward": MoeBlockNormBackwardArgs}


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {moe_status_string(status)} ({status})")
        self.status = status


_lock = threading.Lock()
_lib = None

# C symbols declared in include/*.h, with (restype, argtypes).
SYMBOLS = {
    "moe_abi_version": (C.c_int, []),
    "moe_status_string": (C.c_char_p, [C.c_int]),
    "moe_combine_args_size": (C.c_size_t, []),
    "moe_build_row_map_workspace_size": (C.c_int, [C.c_int64, C.c_int32, C.c_int32,
                                                   C.POINTER(C.c_size_t)]),
    "moe_build_row_map": (C.c_int, [C.c_void_p, C.c_int64, C.c_int32, C.c_int32, C.c_void_p,
                                    C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t,
                                    C.c_void_p]),
    "moe_build_row_map_check": (C.c_int, [C.c_void_p, C.c_void_p]),
    "moe_build_row_map_launches": (C.c_int, [C.c_int64, C.c_int32, C.c_int32, C.POINTER(C.c_int32)]),
    "moe_build_row_map_noalloc": (C.c_int, [C.c_void_p, C.c_int64, C.c_int32, C.c_int32, C.c_void_p,
                                            C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "moe_combine": (C.c_int, [C.POINTER(MoeCombineArgs), C.c_void_p]),
    "moe_scales_bytes": (C.c_int, [C.c_int64, C.c_int32, C.c_int32, C.c_int32,
                                   C.POINTER(C.c_size_t)]),
    "moe_tuning_set": (C.c_int, [C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32]),
    "moe_debug_stall": (C.c_int, [C.c_int64]),
    "moe_dispatch_permute": (C.c_int, [C.c_void_p, C.c_int64, C.c_int32, C.c_void_p, C.c_int32,
                                       C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p]),
    "moe_select_experts": (C.c_int, [C.c_void_p, C.c_int64, C.c_int32, C.c_int64, C.c_int32, C.c_int32,
                                     C.c_int32, C.c_int32, C.c_float, C.c_void_p, C.c_void_p, C.c_int32,
                                     C.c_void_p]),
    "moe_linear_w4": (C.c_int, [C.c_void_p, C.c_void_p]),
    "moe_linear_w4_args_size": (C.c_size_t, []),
    "moe_layer_workspace_size": (C.c_int, [C.c_int64, C.c_int32, C.c_int32, C.POINTER(C.c_size_t)]),
    "moe_layer": (C.c_int, [C.c_void_p, C.c_void_p]),
    "moe_layer_args_size": (C.c_size_t, []),
    "moe_gated_linear_backward_workspace_size": (C.c_int, [C.c_int64, C.c_int32, C.POINTER(C.c_size_t)]),
    "moe_block_norm_backward_workspace_size": (C.c_int, [C.c_int64, C.c_int32, C.POINTER(C.c_size_t)]),
}
for _name in _BLOCK_ARGS:
    SYMBOLS[_name] = (C.c_int, [C.c_void_p, C.c_void_p])
    SYMBOLS[_name + "_args_size"] = (C.c_size_t, [])


def lib() -> C.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "norm_quant_gb300.build.build() (no fallback path exists)")
            L = C.CDLL(LIB_PATH)
            for name, (res, args) in SYMBOLS.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            if L.moe_abi_version() != ABI_VERSION:
                raise RuntimeError("libnqg.so ABI version mismatch")
            if L.moe_combine_args_size() != C.sizeof(MoeCombineArgs):
                raise RuntimeError("moe_combine_args layout mismatch")
            if (not L.moe_linear_w4_args_size() == C.sizeof(MoeLinearW4Args) == _LINEAR_W4.size
                    or not L.moe_layer_args_size() == C.sizeof(MoeLayerArgs) == _LAYER.size):
                raise RuntimeError("moe_layer.h argument layout mismatch")
            if any(not getattr(L, name + "_args_size")() == C.sizeof(cls) == _PACK[name].size
                   for name, cls in _BLOCK_ARGS.items()):
                raise RuntimeError("moe_block.h argument layout mismatch")
            _lib = L
    return _lib


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def moe_abi_version() -> int:
    return int(lib().moe_abi_version())


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _need(t, nbytes: int, name: str):
    """Raises ValueError if tensor t (when given) holds fewer than nbytes
    bytes: the kernels take plain pointers and would read or write past a
    buffer that is too small."""
    if t is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes; this call needs {nbytes}")


def _scales_bytes(T: int, H: int, vec: int, sf_layout: str) -> int:
    """Bytes of a scale matrix: linear T x C, or 128x4 with rows padded to
    128 and columns to 4 (the library's moe_scales_bytes)."""
    cols = H // vec
    if sf_layout == "linear":
        return T * cols
    return -(-T // 128) * 128 * (-(-cols // 4) * 4)


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


_raw_stream = None  # torch's getter of a device's current stream as an integer


def _stream_of(stream, t):
    """_stream() for the few-token operators, whose kernels take a few
    microseconds: the current stream of t's device without a Stream object."""
    global _raw_stream
    if stream is not None:
        return getattr(stream, "cuda_stream", stream)
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _raw_stream(t.get_device())


def _check(st: int, what: str):
    if st != MOE_OK:
        raise MoeError(st, what)


def moe_build_row_map_workspace_size(T: int, top_k: int, E: int) -> int:
    n = C.c_size_t(0)
    _check(lib().moe_build_row_map_workspace_size(T, top_k, E, C.byref(n)),
           "moe_build_row_map_workspace_size")
    return n.value


def moe_build_row_map(topk_ids, E: int, counts, offsets, row_map, src_row=None,
                      workspace=None, stream=None) -> None:
    """topk_ids int32 [T, k] -> counts [E], offsets [E+1], row_map [T, k],
    src_row [>= N_valid] (optional).  workspace: uint8 CUDA tensor of at least
    moe_build_row_map_workspace_size(T, k, E) bytes."""
    T, k = topk_ids.shape
    _need(topk_ids, T * k * 4, "topk_ids")
    _need(counts, E * 4, "counts")
    _need(offsets, (E + 1) * 4, "offsets")
    _need(row_map, T * k * 4, "row_map")
    _check(lib().moe_build_row_map(_ptr(topk_ids), T, k, E, _ptr(counts), _ptr(offsets),
                                   _ptr(row_map), _ptr(src_row), _ptr(workspace),
                                   workspace.numel() * workspace.element_size() if workspace is not None else 0,
                                   _stream(stream)),
           "moe_build_row_map")


def moe_build_row_map_noalloc(topk_ids, E: int, counts, offsets, row_map, src_row=None,
                              error_flag=None, stream=None) -> None:
    """moe_build_row_map without a workspace, for callers that cannot
    allocate device memory: the library's own fixed scratch array is used
    (see include/moe_combine.h for its size limit and sharing rules)."""
    T, k = topk_ids.shape
    _need(topk_ids, T * k * 4, "topk_ids")
    _need(counts, E * 4, "counts")
    _need(offsets, (E + 1) * 4, "offsets")
    _need(row_map, T * k * 4, "row_map")
    _need(error_flag, 4, "error_flag")
    _check(lib().moe_build_row_map_noalloc(_ptr(topk_ids), T, k, E, _ptr(counts), _ptr(offsets),
                                           _ptr(row_map), _ptr(src_row), _ptr(error_flag), _stream(stream)),
           "moe_build_row_map_noalloc")


def moe_build_row_map_check(workspace, stream=None) -> int:
    """Synchronises the stream; MOE_OK or MOE_ERR_INVALID_EXPERT."""
    return int(lib().moe_build_row_map_check(_ptr(workspace), _stream(stream)))


def moe_build_row_map_launches(T: int, top_k: int, E: int) -> int:
    """Kernels moe_build_row_map launches for this shape on the current device (1, 3, or 0)."""
    n = C.c_int32(-1)
    _check(lib().moe_build_row_map_launches(T, top_k, E, C.byref(n)), "moe_build_row_map_launches")
    return n.value


def moe_scales_bytes(T: int, H: int, quant: str, sf_layout: str = "linear") -> int:
    n = C.c_size_t(0)
    _check(lib().moe_scales_bytes(T, H, QUANT[quant], LAYOUT[sf_layout], C.byref(n)), "moe_scales_bytes")
    return n.value


def moe_dispatch_permute(x, row_map, x_grouped, status=None, stream=None) -> None:
    """x [T, H] bf16 -> x_grouped [n_rows, H]: row row_map[t, j] >= 0 gets x[t]."""
    T, H = x.shape
    _need(x, T * H * 2, "x")
    _need(row_map, T * row_map.shape[1] * 4, "row_map")
    _need(status, 4, "status")
    _check(lib().moe_dispatch_permute(_ptr(x), T, H, _ptr(row_map), row_map.shape[1], _ptr(x_grouped),
                                      int(x_grouped.shape[0]), _ptr(status), _stream(stream)),
           "moe_dispatch_permute")


def moe_tuning_set(vpt: int = 0, rows_per_slot: int = 0, ring_kib: int = 0, ctas_per_sm: int = 0,
                   route_cluster: int = 0, combine_split: int = 0) -> None:
    """Overrides the launch plans (0 = automatic); results do not depend on it."""
    _check(lib().moe_tuning_set(vpt, rows_per_slot, ring_kib, ctas_per_sm, route_cluster, combine_split),
           "moe_tuning_set")


def moe_debug_stall(slots: int = -1) -> None:
    """Test hook: the combine's CTA 0 stops staging rows after `slots` ring
    slots, so its bounded waits run out and the status reports a timeout
    (-1 turns it off)."""
    _check(lib().moe_debug_stall(slots), "moe_debug_stall")


def combine_args(*, expert_out, row_map, router_weights, shared_out=None, residual=None,
                 gamma=None, eps=1e-6, weight_bias=0.0, quant=None, sf_layout="linear",
                 global_scale=1.0, combined_out=None, residual_out=None, norm_out=None,
                 quant_out=None, scales_out=None, status=None, H=None,
                 expert_layout="grouped", io_dtype="bf16", weight_dtype="fp32") -> MoeCombineArgs:
    """Fills a MoeCombineArgs from tensors (T and top_k from router_weights'
    shape).  expert_layout "slot_major": expert_out is [top_k, T, H] and
    row_map may be None."""
    T, k = router_weights.shape
    if H is None:
        H = int(expert_out.shape[-1])
    n_rows = int(expert_out.numel() // H) if H else 0
    _need(router_weights, T * k * (4 if weight_dtype == "fp32" else 2), "router_weights")
    if expert_layout == "slot_major":
        _need(expert_out, k * T * H * 2, "expert_out")
    else:
        _need(row_map, T * k * 4, "row_map")
    for name, t in (("shared_out", shared_out), ("residual", residual), ("combined_out", combined_out),
                    ("residual_out", residual_out), ("norm_out", norm_out)):
        _need(t, T * H * 2, name)
    _need(gamma, H * 2, "gamma")
    if quant:
        _need(quant_out, T * (H if quant == "mxfp8" else H // 2), "quant_out")
        vec = 16 if quant == "nvfp4" else 32
        if H % vec == 0:  # otherwise the library rejects the call itself
            _need(scales_out, _scales_bytes(T, H, vec, sf_layout), "scales_out")
    _need(status, 4, "status")
    return MoeCombineArgs(
        T=T, H=H, top_k=k, expert_out=_ptr(expert_out), n_expert_rows=n_rows,
        expert_layout=EXPERT_LAYOUT[expert_layout],
        row_map=_ptr(row_map), router_weights=_ptr(router_weights), shared_out=_ptr(shared_out),
        residual=_ptr(residual), gamma=_ptr(gamma), eps=eps, weight_bias=weight_bias,
        quant=QUANT[quant], sf_layout=LAYOUT[sf_layout], global_scale=global_scale,
        combined_out=_ptr(combined_out), residual_out=_ptr(residual_out), norm_out=_ptr(norm_out),
        quant_out=_ptr(quant_out), scales_out=_ptr(scales_out), status=_ptr(status),
        io_dtype=IO_DTYPE[io_dtype], weight_dtype=WEIGHT_DTYPE[weight_dtype])


def moe_combine(stream=None, **kw) -> None:
    """Enqueues the combine; keyword arguments as in combine_args()."""
    args = kw.pop("args", None) or combine_args(**kw)
    _check(lib().moe_combine(C.byref(args), _stream(stream)), "moe_combine")


def _rows(t, elem: int, name: str):
    """(rows, width, pointer, elements from row to row) of a 2-D CUDA tensor of
    elem-byte elements whose rows may be strided; ValueError otherwise.

    The few-token operators' kernels take a few microseconds, so their checks
    and arguments are put together in as few calls as they take."""
    if not t.is_cuda:
        raise ValueError(f"{name}: tensors must be CUDA tensors")
    if t.dim() != 2 or t.element_size() != elem:
        raise ValueError(f"{name} is {tuple(t.shape)} of {t.element_size()}-byte elements; this call needs a matrix "
                         f"of {elem}-byte elements")
    rows, width = t.shape
    stride, one = t.stride()
    if one != 1 and width > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return rows, width, t.data_ptr(), stride if rows > 1 else width


def _sized(t, nbytes: int, elem: int, name: str):
    """Pointer of a contiguous CUDA tensor of elem-byte elements that holds at
    least nbytes, or 0 for None.  Elements of another size (int64 ids, codes
    packed into wider words) hold something else than the call takes them for."""
    if t is None:
        return 0
    if t.itemsize != elem:
        raise ValueError(f"{name} has {t.itemsize}-byte elements; this call takes {elem}-byte ones")
    if t.nbytes < nbytes:
        _need(t, nbytes, name)
    if not t.is_cuda or not t.is_contiguous():
        _ptr(t)
    return t.data_ptr()


def _scale_bytes(w_format, group_size: int, elements: int):
    """(bytes of the scales, bytes of the zero points, bytes of a scale) of `elements` 4-bit weights."""
    if w_format == "nvfp4":
        return elements // 16, 0, 1
    if w_format == "int4" and group_size > 0:
        return elements // group_size * 2, elements // group_size, 2
    return 0, 0, 2 if w_format == "int4" else 1


def moe_select_experts(logits, topk_ids, router_weights, *, scoring="softmax", renormalize=True, scale=1.0,
                       logits_dtype="fp32", weight_dtype="fp32", stream=None) -> None:
    """logits [T, E] (rows may be strided) -> topk_ids int32 [T, k], the k
    experts with the largest logits in descending order (ties by the lower
    index; -1 where fewer are open), and router_weights [T, k]."""
    T, E, lp, stride = _rows(logits, 4 if logits_dtype == "fp32" else 2, "logits")
    k = topk_ids.shape[-1]
    we = 4 if weight_dtype == "fp32" else 2
    st = lib().moe_select_experts(lp, T, E, stride, WEIGHT_DTYPE[logits_dtype], k, SCORING[scoring],
                                  1 if renormalize else 0, scale, _sized(topk_ids, T * k * 4, 4, "topk_ids"),
                                  _sized(router_weights, T * k * we, we, "router_weights"),
                                  WEIGHT_DTYPE[weight_dtype], _stream_of(stream, logits))
    if st:
        raise MoeError(st, "moe_select_experts")


# MoeLinearW4Args and MoeLayerArgs as the bytes of their fields: a third of the time a ctypes structure takes
_LINEAR_W4 = struct.Struct("@qiiPqPPPfiiiPq")
_LAYER = struct.Struct("@qiiiiPqPPPPPPPPPPPPPPNPiiiii4x")


def _linear_w4_fields(x, w, w_scales, out, w_format="nvfp4", group_size=0, zeros=None, global_scale=1.0,
                      io_dtype="bf16"):
    M, K, xp, xs = _rows(x, 2, "x")
    rows, N, op, os_ = _rows(out, 2, "out")
    if rows != M:
        raise ValueError(f"out has {rows} rows; x has {M}")
    sb, zb, se = _scale_bytes(w_format, group_size, N * K)
    return (M, N, K, xp, xs, _sized(w, N * K // 2, 1, "w"), _sized(w_scales, sb, se, "w_scales"),
            _sized(zeros, zb, 1, "zeros"), global_scale, W_FORMAT[w_format], group_size, IO_DTYPE[io_dtype], op, os_)


def linear_w4_args(x, w, w_scales, out, *, w_format="nvfp4", group_size=0, zeros=None, global_scale=1.0,
                   io_dtype="bf16") -> MoeLinearW4Args:
    """Fills a MoeLinearW4Args from tensors: x [M, K], w uint8 [N, K / 2], out [M, N]."""
    return MoeLinearW4Args(*_linear_w4_fields(x, w, w_scales, out, w_format, group_size, zeros, global_scale, io_dtype))


def moe_linear_w4(x, w, w_scales, out, *, stream=None, **kw) -> None:
    """out [M, N] = x [M, K] W^T with W in 4 bits; M <= 64.  Keyword arguments
    as in linear_w4_args()."""
    st = lib().moe_linear_w4(_LINEAR_W4.pack(*_linear_w4_fields(x, w, w_scales, out, **kw)), _stream_of(stream, x))
    if st:
        raise MoeError(st, "moe_linear_w4")


def moe_layer_workspace_size(T: int, top_k: int, I: int) -> int:
    n = C.c_size_t(0)
    _check(lib().moe_layer_workspace_size(T, top_k, I, C.byref(n)), "moe_layer_workspace_size")
    return n.value


def _layer_fields(x, topk_ids, router_weights, w13, w2, out, workspace, w13_scales=None, w2_scales=None,
                  w13_zeros=None, w2_zeros=None, w13_global=None, w2_global=None, w_format="none", group_size=0,
                  activation="silu", shared_out=None, residual=None, status=None, io_dtype="bf16",
                  weight_dtype="fp32"):
    E, H, inner = w2.shape
    if x.shape[-1] != H:
        raise ValueError(f"w2 has rows for H = {H}; x has H = {x.shape[-1]}")
    T, H, xp, xs = _rows(x, 2, "x")
    k = topk_ids.shape[-1]
    fmt = W_FORMAT[w_format]
    if fmt:
        inner *= 2
    n2 = E * H * inner
    s2, z2, se = _scale_bytes(w_format, group_size, n2)
    rows = T * H * 2
    b2, ce = (n2 // 2, 1) if fmt else (n2 * 2, 2)  # bytes of w2 and of its elements
    we = 4 if weight_dtype == "fp32" else 2
    return (T, H, inner, E, k, xp, xs, _sized(topk_ids, T * k * 4, 4, "topk_ids"),
            _sized(router_weights, T * k * we, we, "router_weights"),
            _sized(w13, 2 * b2, ce, "w13"), _sized(w13_scales, 2 * s2, se, "w13_scales"),
            _sized(w13_zeros, 2 * z2, 1, "w13_zeros"), _sized(w13_global, 4 * E, 4, "w13_global"),
            _sized(w2, b2, ce, "w2"), _sized(w2_scales, s2, se, "w2_scales"),
            _sized(w2_zeros, z2, 1, "w2_zeros"), _sized(w2_global, 4 * E, 4, "w2_global"),
            _sized(shared_out, rows, 2, "shared_out"), _sized(residual, rows, 2, "residual"),
            _sized(out, rows, 2, "out"),
            _ptr(workspace), workspace.nbytes, _sized(status, 4, 4, "status"),
            fmt, group_size, ACTIVATION[activation], IO_DTYPE[io_dtype], WEIGHT_DTYPE[weight_dtype])


def layer_args(**kw) -> MoeLayerArgs:
    """Fills a MoeLayerArgs from tensors, all by name: x [T, H], topk_ids and
    router_weights [T, k], w13, w2, out, workspace, and optionally w13_scales,
    w2_scales, w13_zeros, w2_zeros, w13_global, w2_global, w_format ("none"),
    group_size, activation ("silu"), shared_out, residual, status, io_dtype
    ("bf16") and weight_dtype ("fp32").  E, H and I come from w2's shape
    [E, H, I] (16-bit weights) or [E, H, I / 2] (4-bit codes)."""
    return MoeLayerArgs(*_layer_fields(**kw))


def moe_layer(stream=None, **kw) -> None:
    """Enqueues a whole expert layer for up to 64 tokens; keyword arguments as
    in layer_args() (or args=, a MoeLayerArgs)."""
    args = kw.pop("args", None)
    if args is not None:
        st = lib().moe_layer(C.byref(args), _stream(stream))
    else:
        st = lib().moe_layer(_LAYER.pack(*_layer_fields(**kw)), _stream_of(stream, kw["x"]))
    if st:
        raise MoeError(st, "moe_layer")


# ------------------------------------------------------------------ the block for many tokens

# The structures of moe_block.h as the bytes of their fields, in the order and with the padding of the ctypes mirrors.
_CODES = {C.c_int64: "q", C.c_int32: "i", C.c_float: "f", C.c_void_p: "P", C.c_size_t: "N"}
_PACK = {name: struct.Struct("@" + "".join(_CODES[t] for _, t in cls._fields_) + "0q") for name, cls in _BLOCK_ARGS.items()}


_calls = {}  # name -> (the library's function, the packer of its argument)


def _call(name: str, fields, stream, t) -> None:
    fn = _calls.get(name)
    if fn is None:
        fn = _calls[name] = getattr(lib(), name), _PACK[name].pack
    st = fn[0](fn[1](*fields), _stream_of(stream, t))
    if st:
        raise MoeError(st, name)


def _matrix(t, rows: int, width: int, name: str):
    """Pointer and stride of a matrix [rows, width] of 16-bit elements whose rows may be strided, or (0, 0) for None."""
    if t is None:
        return 0, 0
    r, w, p, stride = _rows(t, 2, name)
    if r != rows or w != width:
        raise ValueError(f"{name} is [{r}, {w}]; this call needs [{rows}, {width}]")
    return p, stride


def _experts(w, name: str, width):
    """(experts, rows, columns) of weights [E, rows, columns]; ValueError unless there are `width` columns (None: any)."""
    if w.dim() != 3 or (width is not None and w.shape[2] != width):
        raise ValueError(f"{name} is {tuple(w.shape)}; this call needs three dimensions"
                         + ("" if width is None else f", the last of {width}"))
    return w.shape


def _gradient(t, shape, grad_dtype: str, name: str):
    """Pointer of a contiguous gradient of this shape, or 0 for None."""
    if t is None:
        return 0
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} is {tuple(t.shape)}; this call needs {tuple(shape)}")
    size = 4 if grad_dtype == "fp32" else 2
    return _sized(t, t.numel() * size, size, name)


def _offsets(offsets, E: int):
    return _sized(offsets, (E + 1) * 4, 4, "offsets")


def moe_gated_linear(x, w13, out, *, offsets=None, gate_up=None, activation="silu", status=None, io_dtype="bf16",
                     stream=None) -> None:
    """out [R, I] = act(x W1^T) * (x W3^T) for x [R, H] and w13 [E, 2 I, H]
    (W1's I rows, then W3's): row r goes through expert e where offsets[e] <= r <
    offsets[e + 1] (int32 [E + 1]; None with one expert: every row).  gate_up
    [R, 2 I], if given, receives both products for moe_gated_linear_backward."""
    R, H, xp, xs = _rows(x, 2, "x")
    E, two, _ = _experts(w13, "w13", H)
    if two % 2:
        raise ValueError(f"w13 has {two} rows an expert; this call needs W1's and as many of W3")
    inner = two // 2
    gp, gs = _matrix(gate_up, R, 2 * inner, "gate_up")
    op, os_ = _matrix(out, R, inner, "out")
    _call("moe_gated_linear", (
        R, H, inner, E, ACTIVATION[activation], _offsets(offsets, E), xp, xs, _sized(w13, E * 4 * inner * H, 2, "w13"),
        gp, gs, op, os_, _sized(status, 4, 4, "status"), IO_DTYPE[io_dtype]), stream, x)


def moe_gated_linear_backward_workspace_size(rows: int, I: int) -> int:
    n = C.c_size_t(0)
    _check(lib().moe_gated_linear_backward_workspace_size(rows, I, C.byref(n)), "moe_gated_linear_backward_workspace_size")
    return n.value


def moe_gated_linear_backward(d_out, gate_up, *, x=None, w13=None, d_x=None, d_w13=None, workspace=None, offsets=None,
                              activation="silu", status=None, io_dtype="bf16", grad_dtype=None, stream=None) -> None:
    """Gradients of moe_gated_linear: d_x [R, H] (needs w13) and d_w13
    [E, 2 I, H] (needs x) of grad_dtype ("fp32", or io_dtype, the default).
    gate_up is what the forward call left.  workspace: uint8 CUDA tensor of
    moe_gated_linear_backward_workspace_size(R, I) bytes."""
    R, inner, dp, ds = _rows(d_out, 2, "d_out")
    gp, gs = _matrix(gate_up, R, 2 * inner, "gate_up")
    grad = grad_dtype or io_dtype
    if (d_x is not None and w13 is None) or (d_w13 is not None and x is None):
        raise ValueError("d_x needs w13 and d_w13 needs x")
    if w13 is None and d_w13 is None:
        raise ValueError("d_x or d_w13 has to be given")
    E, two, H = _experts(w13 if w13 is not None else d_w13, "w13", None)
    if two != 2 * inner:
        raise ValueError(f"w13 has {two} rows an expert; d_out has {inner} columns, which need {2 * inner}")
    xp, xs = _matrix(x, R, H, "x")
    op, os_ = _matrix(d_x, R, H, "d_x")
    _call("moe_gated_linear_backward", (
        R, H, inner, E, ACTIVATION[activation], _offsets(offsets, E), dp, ds, gp, gs, xp, xs,
        _sized(w13, E * 4 * inner * H, 2, "w13"), op, os_, _gradient(d_w13, (E, two, H), grad, "d_w13"),
        _ptr(workspace) or 0, 0 if workspace is None else workspace.nbytes, _sized(status, 4, 4, "status"),
        IO_DTYPE[io_dtype], WEIGHT_DTYPE[grad]), stream, d_out)


def moe_grouped_linear(x, w, out, *, offsets=None, status=None, io_dtype="bf16", stream=None) -> None:
    """out [R, N] = x W[e]^T for x [R, K] and w [E, N, K]; rows and experts as
    in moe_gated_linear()."""
    R, K, xp, xs = _rows(x, 2, "x")
    E, N, _ = _experts(w, "w", K)
    op, os_ = _matrix(out, R, N, "out")
    _call("moe_grouped_linear", (R, K, N, E, IO_DTYPE[io_dtype], _offsets(offsets, E), xp, xs,
                                 _sized(w, E * 2 * N * K, 2, "w"), op, os_, _sized(status, 4, 4, "status")), stream, x)


def moe_grouped_linear_backward(d_out, *, x=None, w=None, d_x=None, d_w=None, offsets=None, status=None,
                                io_dtype="bf16", grad_dtype=None, stream=None) -> None:
    """Gradients of moe_grouped_linear: d_x [R, K] (needs w) and d_w [E, N, K]
    (needs x) of grad_dtype ("fp32", or io_dtype, the default)."""
    R, N, dp, ds = _rows(d_out, 2, "d_out")
    grad = grad_dtype or io_dtype
    if (d_x is not None and w is None) or (d_w is not None and x is None):
        raise ValueError("d_x needs w and d_w needs x")
    if w is None and d_w is None:
        raise ValueError("d_x or d_w has to be given")
    E, n, K = _experts(w if w is not None else d_w, "w", None)
    if n != N:
        raise ValueError(f"w has {n} rows an expert; d_out has {N} columns")
    xp, xs = _matrix(x, R, K, "x")
    op, os_ = _matrix(d_x, R, K, "d_x")
    _call("moe_grouped_linear_backward", (
        R, K, N, E, IO_DTYPE[io_dtype], _offsets(offsets, E), dp, ds, xp, xs, _sized(w, E * 2 * N * K, 2, "w"), op, os_,
        _gradient(d_w, (E, N, K), grad, "d_w"), _sized(status, 4, 4, "status"), WEIGHT_DTYPE[grad]), stream, d_out)


def _gate(gate, gate_kind, T: int, H: int):
    kind = GATE[gate_kind]
    if (gate is None) != (kind == 0):
        raise ValueError(f"gate_kind {gate_kind!r} and gate {'missing' if gate is None else 'given'}")
    if kind == 1:
        return _sized(gate, 2 * H, 2, "gate"), kind
    return _sized(gate, 4 * T, 4, "gate"), kind


def moe_block_norm(y, residual=None, *, post_gamma=None, pre_gamma=None, gate=None, gate_kind=None, block_scale=1.0,
                   residual_scale=1.0, eps=1e-6, weight_bias=0.0, residual_out=None, norm_out=None, io_dtype="bf16",
                   stream=None) -> None:
    """The norms after a block and before the next: residual_out [T, H] =
    residual_scale * residual + block_scale * gate * norm(y; post_gamma) and
    norm_out [T, H] = norm(that, unrounded; pre_gamma).  gate_kind "channel": gate
    [H] of io_dtype; "token": fp32 [T]."""
    T, H = y.shape
    size = 2 * T * H
    gp, kind = _gate(gate, gate_kind, T, H)
    _call("moe_block_norm", (
        T, H, IO_DTYPE[io_dtype], _sized(y, size, 2, "y"), _sized(residual, size, 2, "residual"),
        _sized(post_gamma, 2 * H, 2, "post_gamma"), _sized(pre_gamma, 2 * H, 2, "pre_gamma"), gp, kind, block_scale,
        residual_scale, eps, weight_bias, _sized(residual_out, size, 2, "residual_out"),
        _sized(norm_out, size, 2, "norm_out")), stream, y)


def moe_block_norm_backward_workspace_size(T: int, H: int) -> int:
    n = C.c_size_t(0)
    _check(lib().moe_block_norm_backward_workspace_size(T, H, C.byref(n)), "moe_block_norm_backward_workspace_size")
    return n.value


def moe_block_norm_backward(y, residual=None, *, post_gamma=None, pre_gamma=None, gate=None, gate_kind=None,
                            block_scale=1.0, residual_scale=1.0, eps=1e-6, weight_bias=0.0, d_residual_out=None,
                            d_norm_out=None, d_y=None, d_residual=None, d_post_gamma=None, d_pre_gamma=None, d_gate=None,
                            workspace=None, io_dtype="bf16", stream=None) -> None:
    """Gradients of moe_block_norm from those of its outputs (d_residual_out,
    d_norm_out): d_y and d_residual [T, H], and in fp32 d_post_gamma [H],
    d_pre_gamma [H] and d_gate ([H] or [T]).  workspace: uint8 CUDA tensor of
    moe_block_norm_backward_workspace_size(T, H) bytes, for the sums over tokens."""
    T, H = y.shape
    size = 2 * T * H
    gp, kind = _gate(gate, gate_kind, T, H)
    _call("moe_block_norm_backward", (
        T, H, IO_DTYPE[io_dtype], _sized(y, size, 2, "y"), _sized(residual, size, 2, "residual"),
        _sized(post_gamma, 2 * H, 2, "post_gamma"), _sized(pre_gamma, 2 * H, 2, "pre_gamma"), gp, kind, block_scale,
        residual_scale, eps, weight_bias, _sized(d_residual_out, size, 2, "d_residual_out"),
        _sized(d_norm_out, size, 2, "d_norm_out"), _sized(d_y, size, 2, "d_y"),
        _sized(d_residual, size, 2, "d_residual"), _sized(d_post_gamma, 4 * H, 4, "d_post_gamma"),
        _sized(d_pre_gamma, 4 * H, 4, "d_pre_gamma"), _sized(d_gate, 4 * (T if kind == 2 else H), 4, "d_gate"),
        _ptr(workspace) or 0, 0 if workspace is None else workspace.nbytes), stream, y)
