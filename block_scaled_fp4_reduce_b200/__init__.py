"""Python binding of the B200 block-scaled FP4 library (libfp4.so).

Argument marshalling only: every step of the quantise / dequantise / scale
search path runs in the library's CUDA kernels.  PyTorch supplies device
memory and streams.  There is no CPU fallback: if libfp4.so is missing the
import of the entry points fails with an error saying how to build it.

Low-level functions carry the C names of include/fp4.h and take torch
tensors for the pointers; the snake-case helpers below them allocate the
outputs and return them.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp4.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "fp4.h")

# fp4_status / fp4_dtype / fp4_format values (include/fp4.h).
OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_ALIGN, ERR_NONFINITE, ERR_RANGE, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_INDEX = range(10)
F32, BF16 = 0, 1
NVFP4, MXFP4 = 0, 1
MX_FLOOR, MX_CEIL = 0, 1
# fp4_gemm_kernel
GEMM_AUTO, GEMM_CTA, GEMM_CTA_PAIR = 0, 1, 2

_lib = None


class FP4Error(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = int(status)
        msg = lib().fp4_status_string(self.status).decode()
        super().__init__(f"{where}: {msg} (status {self.status})" if where else msg)


def lib() -> ctypes.CDLL:
    """The loaded libfp4.so (built by __graft_entry__.build() or
    `python -m block_scaled_fp4_reduce_b200.build`)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m block_scaled_fp4_reduce_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        sig = {
            "fp4_status_string": (ctypes.c_char_p, [I]),
            "fp4_version": (I, []),
            "fp4_workspace_bytes": (SZ, [I, I64, I64]),
            "fp4_tensor_amax": (I, [P, I, I64, P, P, SZ, P, P]),
            "fp4_nvfp4_quantize": (I, [P, I, I64, I64, P, P, P, P, SZ, P, P]),
            "fp4_nvfp4_quantize_with_amax": (I, [P, I, I64, I64, P, P, P, P, P, P]),
            "fp4_nvfp4_quantize_noalloc": (I, [P, I, I64, I64, P, P, P, P, P]),
            "fp4_mxfp4_quantize": (I, [P, I, I64, I64, P, P, P, P]),
            "fp4_mxfp4_quantize_ceil": (I, [P, I, I64, I64, P, P, P, P]),
            "fp4_nvfp4_quantize_four_over_six": (I, [P, I, I64, I64, P, P, P, P, P, SZ, P, P]),
            "fp4_dequantize": (I, [I, P, P, P, I64, I64, P, I, P]),
            "fp4_scale_search": (I, [P, I, I64, I64, P, P, P, P, P, SZ, P, P]),
            "fp4_scale_search_with_amax": (I, [P, I, I64, I64, P, P, P, P, P, P, P]),
            "fp4_scale_search_grid": (I, [P, I, I64, I64, I, I, I, P, P, P, P, P, SZ, P, P]),
            "fp4_e2m1_round": (I, [P, P, I64, P]),
            "fp4_e2m1_roundtrip": (I, [P, P, I64, P]),
            "fp4_nv_encode_quotient": (I, [P, P, P, I64, P]),
            "fp4_test_bounded_wait": (I, [ctypes.c_uint32, P, P, P]),
            "fp4_grouped_workspace_bytes": (SZ, [I]),
            "fp4_nvfp4_quantize_grouped": (I, [P, I, I, P, SZ, P, P]),
            "fp4_tensor_amax_grouped": (I, [P, I, I, P, SZ, P, P]),
            "fp4_nvfp4_quantize_grouped_with_amax": (I, [P, I, I, P, P, P]),
            "fp4_mxfp4_quantize_grouped": (I, [P, I, I, P, P]),
            "fp4_mxfp4_quantize_ceil_grouped": (I, [P, I, I, P, P]),
            "fp4_dequantize_grouped": (I, [I, P, I, I, P]),
            "fp4_grouped_plan": (I, [P, I, I64, I, P, P, P, P, I]),
            "fp4_set_launch_unit_limit": (I, [I64]),
            "fp4_mma_scales_bytes": (SZ, [I64, I64]),
            "fp4_scales_to_mma_layout": (I, [P, I64, I64, P, P]),
            "fp4_nvfp4_gemm": (I, [P, P, P, P, P, P, I64, I64, I64, P, P, P]),
            "fp4_nvfp4_gemm_ex": (I, [P, P, P, P, P, P, I64, I64, I64, P, I, P, P]),
            "fp4_nvfp4_quantize_padded": (I, [P, I, I64, I64, P, P, P, P, SZ, P, P]),
            "fp4_nvfp4_quantize_padded_with_amax": (I, [P, I, I64, I64, P, P, P, P, P, P]),
            "fp4_mxfp4_quantize_padded": (I, [P, I, I64, I64, I, P, P, P, P]),
            "fp4_dequantize_padded": (I, [I, P, P, P, I64, I64, P, I, P]),
            "fp4_nvfp4_quantize_columns": (I, [P, I, I64, I64, P, P, P, P, SZ, P, P]),
            "fp4_nvfp4_quantize_columns_with_amax": (I, [P, I, I64, I64, P, P, P, P, P, P]),
            "fp4_mxfp4_quantize_columns": (I, [P, I, I64, I64, I, P, P, P, P]),
            "fp4_kv_write": (I, [P, P, P, I, I64, I64, I64, P, I, P, P]),
            "fp4_kv_read": (I, [P, P, I64, P, P, I, I64, I64, P, P]),
            "fp4_kv_attention_workspace_bytes": (SZ, [P, I64, I64, I64, I64]),
            "fp4_kv_attention": (I, [P, P, I, I64, I64, I64, I64, P, I64, P, ctypes.c_float, I64, P, P, P, SZ, P, P]),
            "fp4_linear_workspace_bytes": (SZ, [I64, I64]),
            "fp4_linear": (I, [I, P, I, I64, I64, I64, P, P, P, I64, P, I, P, SZ, P, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def declared_entry_points() -> list[str]:
    """Names of the functions include/fp4.h declares."""
    with open(HEADER_PATH) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b(fp4_[a-z0-9_]+)\s*\(", text)))


# ---------------------------------------------------------------- helpers --

def _p(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"fp32 or bf16 tensor required, got {t.dtype}")


def _shape2(x: torch.Tensor):
    if not x.is_contiguous():
        raise ValueError("contiguous row-major tensor required")
    if x.dim() == 1:
        return 1, x.shape[0]
    return x.numel() // x.shape[-1] if x.shape[-1] else 0, x.shape[-1]


def _check(st: int, where: str):
    if st != OK:
        raise FP4Error(st, where)


# -------------------------------------------------------- C-ABI wrappers ---

def fp4_tensor_amax(x, amax, workspace, status, stream=None) -> int:
    return lib().fp4_tensor_amax(_p(x), _dtype_code(x), x.numel(), _p(amax), _p(workspace),
                                 workspace.numel() * workspace.element_size(), _p(status), _stream(stream))


def fp4_nvfp4_quantize(x, packed, scales, global_scale, workspace, status, stream=None) -> int:
    R, C = _shape2(x)
    return lib().fp4_nvfp4_quantize(_p(x), _dtype_code(x), R, C, _p(packed), _p(scales), _p(global_scale),
                                    _p(workspace), workspace.numel() * workspace.element_size(),
                                    _p(status), _stream(stream))


def fp4_nvfp4_quantize_with_amax(x, amax, packed, scales, global_scale, status, stream=None) -> int:
    R, C = _shape2(x)
    return lib().fp4_nvfp4_quantize_with_amax(_p(x), _dtype_code(x), R, C, _p(amax), _p(packed), _p(scales),
                                              _p(global_scale), _p(status), _stream(stream))


def fp4_nvfp4_quantize_noalloc(x, packed, scales, global_scale, status, stream=None) -> int:
    R, C = _shape2(x)
    return lib().fp4_nvfp4_quantize_noalloc(_p(x), _dtype_code(x), R, C, _p(packed), _p(scales),
                                            _p(global_scale), _p(status), _stream(stream))


def fp4_mxfp4_quantize(x, packed, scales, status, stream=None) -> int:
    R, C = _shape2(x)
    return lib().fp4_mxfp4_quantize(_p(x), _dtype_code(x), R, C, _p(packed), _p(scales), _p(status),
                                    _stream(stream))


def fp4_mxfp4_quantize_ceil(x, packed, scales, status, stream=None) -> int:
    R, C = _shape2(x)
    return lib().fp4_mxfp4_quantize_ceil(_p(x), _dtype_code(x), R, C, _p(packed), _p(scales), _p(status),
                                         _stream(stream))


def fp4_nvfp4_quantize_four_over_six(x, packed, scales, global_scale, block_loss, workspace, status,
                                     stream=None) -> int:
    R, C = _shape2(x)
    return lib().fp4_nvfp4_quantize_four_over_six(_p(x), _dtype_code(x), R, C, _p(packed), _p(scales),
                                                  _p(global_scale), _p(block_loss), _p(workspace),
                                                  workspace.numel() * workspace.element_size(),
                                                  _p(status), _stream(stream))


def fp4_dequantize(fmt, packed, scales, global_scale, rows, cols, y, stream=None) -> int:
    return lib().fp4_dequantize(fmt, _p(packed), _p(scales), _p(global_scale), rows, cols, _p(y),
                                _dtype_code(y), _stream(stream))


def fp4_scale_search(x, packed, scales, global_scale, block_loss, workspace, status, stream=None) -> int:
    R, C = _shape2(x)
    return lib().fp4_scale_search(_p(x), _dtype_code(x), R, C, _p(packed), _p(scales), _p(global_scale),
                                  _p(block_loss), _p(workspace), workspace.numel() * workspace.element_size(),
                                  _p(status), _stream(stream))


def fp4_scale_search_with_amax(x, amax, packed, scales, global_scale, block_loss, status, stream=None) -> int:
    R, C = _shape2(x)
    return lib().fp4_scale_search_with_amax(_p(x), _dtype_code(x), R, C, _p(amax), _p(packed), _p(scales),
                                            _p(global_scale), _p(block_loss), _p(status), _stream(stream))


class QuantItem(ctypes.Structure):
    """struct fp4_quant_item (include/fp4.h)."""
    _fields_ = [("x", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("global_scale", ctypes.c_void_p)]


class DequantItem(ctypes.Structure):
    """struct fp4_dequant_item (include/fp4.h)."""
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("global_scale", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


def quant_items(xs, packed, scales, global_scales=None):
    """A ctypes array of fp4_quant_item for matching lists of tensors."""
    arr = (QuantItem * len(xs))()
    for i, x in enumerate(xs):
        R, C = _shape2(x)
        arr[i] = QuantItem(_p(x), R, C, _p(packed[i]), _p(scales[i]),
                           _p(global_scales[i]) if global_scales is not None else None)
    return arr


def dequant_items(qs, ys):
    arr = (DequantItem * len(qs))()
    for i, (q, y) in enumerate(zip(qs, ys)):
        arr[i] = DequantItem(_p(q.packed), _p(q.scales), _p(q.global_scale), _p(y), q.rows, q.cols)
    return arr


def _group_dtype(xs) -> int:
    codes = {_dtype_code(x) for x in xs}
    if len(codes) > 1:
        raise TypeError("all matrices of a grouped call share one dtype")
    return codes.pop() if codes else BF16


def fp4_nvfp4_quantize_grouped(items, dtype, workspace, status, stream=None) -> int:
    return lib().fp4_nvfp4_quantize_grouped(ctypes.cast(items, ctypes.c_void_p), len(items), dtype,
                                            _p(workspace), workspace.numel() * workspace.element_size(),
                                            _p(status), _stream(stream))


def fp4_tensor_amax_grouped(items, dtype, workspace, status, stream=None) -> int:
    return lib().fp4_tensor_amax_grouped(ctypes.cast(items, ctypes.c_void_p), len(items), dtype,
                                         _p(workspace), workspace.numel() * workspace.element_size(),
                                         _p(status), _stream(stream))


def fp4_nvfp4_quantize_grouped_with_amax(items, dtype, amax_words, status, stream=None) -> int:
    return lib().fp4_nvfp4_quantize_grouped_with_amax(ctypes.cast(items, ctypes.c_void_p), len(items), dtype,
                                                      _p(amax_words), _p(status), _stream(stream))


def tensor_amax_grouped(xs, status=None, stream=None):
    """Per-matrix amax of every matrix in xs: (fp32 [len(xs)] on the device,
    status word)."""
    dev = xs[0].device if xs else torch.device("cuda")
    st = status if status is not None else new_status(dev)
    ws = torch.empty(lib().fp4_grouped_workspace_bytes(len(xs)) // 4, dtype=torch.float32, device=dev)
    items = quant_items(xs, [None] * len(xs), [None] * len(xs))
    _check(fp4_tensor_amax_grouped(items, _group_dtype(xs), ws, st, stream), "fp4_tensor_amax_grouped")
    return ws[:len(xs)], st


def fp4_mxfp4_quantize_grouped(items, dtype, status, ceil=False, stream=None) -> int:
    fn = lib().fp4_mxfp4_quantize_ceil_grouped if ceil else lib().fp4_mxfp4_quantize_grouped
    return fn(ctypes.cast(items, ctypes.c_void_p), len(items), dtype, _p(status), _stream(stream))


def fp4_dequantize_grouped(fmt, items, out_dtype, stream=None) -> int:
    return lib().fp4_dequantize_grouped(fmt, ctypes.cast(items, ctypes.c_void_p), len(items), out_dtype,
                                        _stream(stream))


def grouped_plan(units, max_units, max_entries):
    """The grouped calls' launch plan for items of `units` work units (host
    only): a list of (launch, item, first unit, units) pieces."""
    import numpy as np
    n = len(units)
    u = np.ascontiguousarray(units, dtype=np.int64)
    cap = 2 * n + 16
    while True:
        lo, it = np.zeros(cap, np.int32), np.zeros(cap, np.int32)
        fi, co = np.zeros(cap, np.int64), np.zeros(cap, np.int64)
        k = lib().fp4_grouped_plan(u.ctypes.data if n else None, n, max_units, max_entries, lo.ctypes.data,
                                   it.ctypes.data, fi.ctypes.data, co.ctypes.data, cap)
        if k < 0:
            raise ValueError("fp4_grouped_plan: invalid arguments")
        if k <= cap:
            return list(zip(lo[:k].tolist(), it[:k].tolist(), fi[:k].tolist(), co[:k].tolist()))
        cap = k


def fp4_e2m1_round(v, codes, stream=None) -> int:
    return lib().fp4_e2m1_round(_p(v), _p(codes), v.numel(), _stream(stream))


def fp4_e2m1_roundtrip(v, out, stream=None) -> int:
    return lib().fp4_e2m1_roundtrip(_p(v), _p(out), v.numel(), _stream(stream))


def fp4_nv_encode_quotient(x, d, codes, stream=None) -> int:
    return lib().fp4_nv_encode_quotient(_p(x), _p(d), _p(codes), x.numel(), _stream(stream))


def fp4_test_bounded_wait(tries: int, status, elapsed_ns, stream=None) -> int:
    return lib().fp4_test_bounded_wait(tries, _p(status), _p(elapsed_ns), _stream(stream))


# ------------------------------------------------- allocating helpers ------

@dataclasses.dataclass
class Quantized:
    """Packed codes [R, C/2], block scales [R, C/G] (uint8), the NVFP4 global
    scale g (fp32 [1], None for MXFP4) and the device status word."""
    fmt: int
    packed: torch.Tensor
    scales: torch.Tensor
    global_scale: torch.Tensor | None
    status: torch.Tensor
    rows: int
    cols: int
    block_loss: torch.Tensor | None = None

    def check(self, where: str = "fp4"):
        st = int(self.status.item())
        if st != OK:
            raise FP4Error(st, where)
        return self


def workspace_for(x: torch.Tensor) -> torch.Tensor:
    """A zero-filled workspace (the library keeps its counter word at zero)."""
    n = lib().fp4_workspace_bytes(NVFP4, *_shape2(x))
    return torch.zeros(n, dtype=torch.uint8, device=x.device)


def new_status(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def nvfp4_quantize(x: torch.Tensor, workspace=None, status=None, stream=None) -> Quantized:
    R, C = _shape2(x)
    dev = x.device
    packed = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((R, C // 16), dtype=torch.uint8, device=dev)
    g = torch.empty(1, dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else workspace_for(x)
    st = status if status is not None else new_status(dev)
    _check(fp4_nvfp4_quantize(x, packed, scales, g, ws, st, stream), "fp4_nvfp4_quantize")
    return Quantized(NVFP4, packed, scales, g, st, R, C)


def mxfp4_quantize(x: torch.Tensor, status=None, stream=None) -> Quantized:
    R, C = _shape2(x)
    dev = x.device
    packed = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((R, C // 32), dtype=torch.uint8, device=dev)
    st = status if status is not None else new_status(dev)
    _check(fp4_mxfp4_quantize(x, packed, scales, st, stream), "fp4_mxfp4_quantize")
    return Quantized(MXFP4, packed, scales, None, st, R, C)


def mxfp4_quantize_ceil(x: torch.Tensor, status=None, stream=None) -> Quantized:
    R, C = _shape2(x)
    dev = x.device
    packed = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((R, C // 32), dtype=torch.uint8, device=dev)
    st = status if status is not None else new_status(dev)
    _check(fp4_mxfp4_quantize_ceil(x, packed, scales, st, stream), "fp4_mxfp4_quantize_ceil")
    return Quantized(MXFP4, packed, scales, None, st, R, C)


def nvfp4_quantize_four_over_six(x: torch.Tensor, with_loss: bool = True, workspace=None, status=None,
                                 stream=None) -> Quantized:
    R, C = _shape2(x)
    dev = x.device
    packed = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((R, C // 16), dtype=torch.uint8, device=dev)
    g = torch.empty(1, dtype=torch.float32, device=dev)
    loss = torch.empty((R, C // 16), dtype=torch.float32, device=dev) if with_loss else None
    ws = workspace if workspace is not None else workspace_for(x)
    st = status if status is not None else new_status(dev)
    _check(fp4_nvfp4_quantize_four_over_six(x, packed, scales, g, loss, ws, st, stream),
           "fp4_nvfp4_quantize_four_over_six")
    return Quantized(NVFP4, packed, scales, g, st, R, C, block_loss=loss)


def dequantize(q: Quantized, out_dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    y = out if out is not None else torch.empty((q.rows, q.cols), dtype=out_dtype, device=q.packed.device)
    _check(fp4_dequantize(q.fmt, q.packed, q.scales, q.global_scale, q.rows, q.cols, y, stream),
           "fp4_dequantize")
    return y


def _padded(n: int, group: int) -> int:
    return -(-n // group) * group


def nvfp4_quantize_padded(x: torch.Tensor, workspace=None, status=None, stream=None, amax=None) -> Quantized:
    """NVFP4 of x [R, K] for any K: rows padded with +0 to whole 16-blocks
    (packed [R, ceil(K/16)*8], scales [R, ceil(K/16)]).  With `amax` (a
    device float32 holding the tensor amax) the call skips its own amax
    pass (fp4_nvfp4_quantize_padded_with_amax)."""
    R, K = _shape2(x)
    dev = x.device
    Kp = _padded(K, 16)
    packed = torch.empty((R, Kp // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((R, Kp // 16), dtype=torch.uint8, device=dev)
    g = torch.empty(1, dtype=torch.float32, device=dev)
    st = status if status is not None else new_status(dev)
    if amax is not None:
        _check(lib().fp4_nvfp4_quantize_padded_with_amax(_p(x), _dtype_code(x), R, K, _p(amax), _p(packed),
                                                         _p(scales), _p(g), _p(st), _stream(stream)),
               "fp4_nvfp4_quantize_padded_with_amax")
        return Quantized(NVFP4, packed, scales, g, st, R, K)
    ws = workspace if workspace is not None else workspace_for(x)
    _check(lib().fp4_nvfp4_quantize_padded(_p(x), _dtype_code(x), R, K, _p(packed), _p(scales), _p(g), _p(ws),
                                           ws.numel() * ws.element_size(), _p(st), _stream(stream)),
           "fp4_nvfp4_quantize_padded")
    return Quantized(NVFP4, packed, scales, g, st, R, K)


def mxfp4_quantize_padded(x: torch.Tensor, rule: int = MX_FLOOR, status=None, stream=None) -> Quantized:
    """MXFP4 of x [R, K] for any K: rows padded with +0 to whole 32-blocks."""
    R, K = _shape2(x)
    dev = x.device
    Kp = _padded(K, 32)
    packed = torch.empty((R, Kp // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((R, Kp // 32), dtype=torch.uint8, device=dev)
    st = status if status is not None else new_status(dev)
    _check(lib().fp4_mxfp4_quantize_padded(_p(x), _dtype_code(x), R, K, rule, _p(packed), _p(scales), _p(st),
                                           _stream(stream)), "fp4_mxfp4_quantize_padded")
    return Quantized(MXFP4, packed, scales, None, st, R, K)


def dequantize_padded(q: Quantized, out_dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """Dequantise a padded layout into the logical [q.rows, q.cols]."""
    y = out if out is not None else torch.empty((q.rows, q.cols), dtype=out_dtype, device=q.packed.device)
    _check(lib().fp4_dequantize_padded(q.fmt, _p(q.packed), _p(q.scales), _p(q.global_scale), q.rows, q.cols,
                                       _p(y), _dtype_code(y), _stream(stream)), "fp4_dequantize_padded")
    return y


def nvfp4_quantize_columns(x: torch.Tensor, workspace=None, status=None, stream=None, amax=None) -> Quantized:
    """NVFP4 of W^T for x = W [R, C]: blocks down the columns of W; the
    result describes the logical [C, R] transpose in the padded layout.
    With `amax` (device float32, the amax of W) the call skips its own amax
    pass (fp4_nvfp4_quantize_columns_with_amax)."""
    R, C = _shape2(x)
    dev = x.device
    Rp = _padded(R, 16)
    packed = torch.empty((C, Rp // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((C, Rp // 16), dtype=torch.uint8, device=dev)
    g = torch.empty(1, dtype=torch.float32, device=dev)
    st = status if status is not None else new_status(dev)
    if amax is not None:
        _check(lib().fp4_nvfp4_quantize_columns_with_amax(_p(x), _dtype_code(x), R, C, _p(amax), _p(packed),
                                                          _p(scales), _p(g), _p(st), _stream(stream)),
               "fp4_nvfp4_quantize_columns_with_amax")
        return Quantized(NVFP4, packed, scales, g, st, C, R)
    ws = workspace if workspace is not None else workspace_for(x)
    _check(lib().fp4_nvfp4_quantize_columns(_p(x), _dtype_code(x), R, C, _p(packed), _p(scales), _p(g), _p(ws),
                                            ws.numel() * ws.element_size(), _p(st), _stream(stream)),
           "fp4_nvfp4_quantize_columns")
    return Quantized(NVFP4, packed, scales, g, st, C, R)


def mxfp4_quantize_columns(x: torch.Tensor, rule: int = MX_FLOOR, status=None, stream=None) -> Quantized:
    """MXFP4 of W^T for x = W [R, C] (column-wise 32-blocks)."""
    R, C = _shape2(x)
    dev = x.device
    Rp = _padded(R, 32)
    packed = torch.empty((C, Rp // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((C, Rp // 32), dtype=torch.uint8, device=dev)
    st = status if status is not None else new_status(dev)
    _check(lib().fp4_mxfp4_quantize_columns(_p(x), _dtype_code(x), R, C, rule, _p(packed), _p(scales), _p(st),
                                            _stream(stream)), "fp4_mxfp4_quantize_columns")
    return Quantized(MXFP4, packed, scales, None, st, C, R)


def scales_to_mma(scales: torch.Tensor, stream=None) -> torch.Tensor:
    """Block scales [rows, blocks] -> the tiled layout of the tensor-core MMA
    (flat uint8, fp4_mma_scales_bytes long)."""
    rows, nb = scales.shape
    out = torch.empty(lib().fp4_mma_scales_bytes(rows, nb), dtype=torch.uint8, device=scales.device)
    _check(lib().fp4_scales_to_mma_layout(_p(scales), rows, nb, _p(out), _stream(stream)), "fp4_scales_to_mma_layout")
    return out


def nvfp4_gemm(qa: Quantized, qb: Quantized, out=None, status=None, stream=None,
               kernel: int = GEMM_AUTO) -> torch.Tensor:
    """D [M, N] fp32 = g_a g_b A B^T on the tensor cores for NVFP4 A [M, K]
    and B [N, K] (M, N multiples of 128, K of 256; GEMM_CTA_PAIR needs M, N
    multiples of 256)."""
    if qa.fmt != NVFP4 or qb.fmt != NVFP4 or qa.cols != qb.cols:
        raise ValueError("two NVFP4 operands with the same K required")
    M, N, K = qa.rows, qb.rows, qa.cols
    dev = qa.packed.device
    d = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=dev)
    st = status if status is not None else new_status(dev)
    sa, sb = scales_to_mma(qa.scales, stream), scales_to_mma(qb.scales, stream)
    _check(lib().fp4_nvfp4_gemm_ex(_p(qa.packed), _p(sa), _p(qa.global_scale), _p(qb.packed), _p(sb),
                                   _p(qb.global_scale), M, N, K, _p(d), kernel, _p(st), _stream(stream)),
           "fp4_nvfp4_gemm_ex")
    return d


def nvfp4_quantize_grouped(xs, status=None, stream=None) -> list[Quantized]:
    """NVFP4 quantisation of every matrix in xs, each with its own g, in a
    few launches (bit-identical to nvfp4_quantize per matrix)."""
    dev = xs[0].device if xs else torch.device("cuda")
    outs = [(torch.empty((R, C // 2), dtype=torch.uint8, device=dev),
             torch.empty((R, C // 16), dtype=torch.uint8, device=dev),
             torch.empty(1, dtype=torch.float32, device=dev)) for R, C in map(_shape2, xs)]
    st = status if status is not None else new_status(dev)
    ws = torch.empty(lib().fp4_grouped_workspace_bytes(len(xs)), dtype=torch.uint8, device=dev)
    items = quant_items(xs, [o[0] for o in outs], [o[1] for o in outs], [o[2] for o in outs])
    _check(fp4_nvfp4_quantize_grouped(items, _group_dtype(xs), ws, st, stream), "fp4_nvfp4_quantize_grouped")
    return [Quantized(NVFP4, p, s, g, st, *_shape2(x)) for x, (p, s, g) in zip(xs, outs)]


def mxfp4_quantize_grouped(xs, ceil: bool = False, status=None, stream=None) -> list[Quantized]:
    """MXFP4 quantisation of every matrix in xs in a few launches."""
    dev = xs[0].device if xs else torch.device("cuda")
    outs = [(torch.empty((R, C // 2), dtype=torch.uint8, device=dev),
             torch.empty((R, C // 32), dtype=torch.uint8, device=dev)) for R, C in map(_shape2, xs)]
    st = status if status is not None else new_status(dev)
    items = quant_items(xs, [o[0] for o in outs], [o[1] for o in outs])
    _check(fp4_mxfp4_quantize_grouped(items, _group_dtype(xs), st, ceil, stream), "fp4_mxfp4_quantize_grouped")
    return [Quantized(MXFP4, p, s, None, st, *_shape2(x)) for x, (p, s) in zip(xs, outs)]


def dequantize_grouped(qs, out_dtype=torch.bfloat16, outs=None, stream=None) -> list[torch.Tensor]:
    """Dequantise every Quantized in qs (all NVFP4 or all MXFP4)."""
    fmts = {q.fmt for q in qs}
    if len(fmts) > 1:
        raise ValueError("all items of a grouped dequantisation share one format")
    ys = outs if outs is not None else [
        torch.empty((q.rows, q.cols), dtype=out_dtype, device=q.packed.device) for q in qs]
    code = _dtype_code(ys[0]) if ys else (F32 if out_dtype == torch.float32 else BF16)
    _check(fp4_dequantize_grouped(fmts.pop() if fmts else NVFP4, dequant_items(qs, ys), code, stream),
           "fp4_dequantize_grouped")
    return ys


# ------------------------------------------- single-token serving -----------

def _cuda(t: torch.Tensor, what: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{what}: a CUDA tensor required")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: {dtype} required, got {t.dtype}")
    return t


# The current stream's handle without building a Stream object (3 us of the 5 us that a call of the library
# takes); torch.cuda.current_stream where torch does not offer it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name: str, index: int, stream, *args) -> None:
    """The entry point `name` on device `index` (the library launches on the
    current device), on `stream` or that device's current stream."""
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _call(name, index, stream, *args)
    s = _raw_stream(index) if stream is None else _stream(stream)
    st = getattr(_lib, name)(*args, s)
    if st != OK:
        raise FP4Error(st, name)


def _on(stream, index: int):
    """A context with `stream` (a stream or its handle) current on device `index`: what a call allocates for
    itself, its zero-fill and its later reuse are then ordered with its kernels."""
    if hasattr(stream, "cuda_stream"):
        if stream.device.index != index:
            raise ValueError(f"stream: one of cuda:{index} required, got {stream.device}'s")
        return torch.cuda.stream(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=index) if stream
                             else torch.cuda.default_stream(index))


def _same_device(index: int, *tensors) -> None:
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors of a call live on one device: cuda:{index} and {t.device}")


def _status(given, own: torch.Tensor) -> torch.Tensor:
    """The status word of a call: the given one, or its handle's."""
    if given is None:
        return own
    if given.dtype != torch.int32 or given.numel() < 1:
        raise TypeError("status: an int32 word required")
    return given


def _workspace(ws: torch.Tensor) -> int:
    """Its bytes."""
    if not ws.is_contiguous():
        raise ValueError("workspace: a contiguous tensor required")
    return ws.numel() * ws.element_size()


class KVCacheStruct(ctypes.Structure):
    """struct fp4_kv_cache (include/fp4.h)."""
    _fields_ = [("format", ctypes.c_int), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int64),
                ("k_packed", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_packed", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("k_global_scale", ctypes.c_void_p),
                ("v_global_scale", ctypes.c_void_p)]


class KVCache:
    """A paged FP4 cache of keys and values over the caller's tensors:
    packed codes [pages, heads, page_size, head_dim/2] and scale bytes
    [pages, heads, page_size, head_dim/G] (uint8, contiguous) of each, and
    for NVFP4 one fp32 global scale per head.  `status` is the device word
    that its calls report data errors in (`check()` reads it)."""

    def __init__(self, fmt, k_packed, k_scales, v_packed, v_scales, k_global_scale=None, v_global_scale=None,
                 status=None):
        if fmt not in (NVFP4, MXFP4):
            raise ValueError("fmt: NVFP4 or MXFP4")
        group = 16 if fmt == NVFP4 else 32
        dev, self.index = _cuda(k_packed, "k_packed").device, k_packed.get_device()
        _same_device(self.index, k_scales, v_packed, v_scales, status)
        for name, t in (("k_packed", k_packed), ("k_scales", k_scales), ("v_packed", v_packed), ("v_scales", v_scales)):
            if t.dtype != torch.uint8 or t.dim() != 4 or not t.is_contiguous():
                raise ValueError(f"{name}: contiguous uint8 [pages, heads, page_size, bytes] required")
        self.num_pages, self.heads, self.page_size, half = k_packed.shape
        self.head_dim = half * 2
        scales = (self.num_pages, self.heads, self.page_size, self.head_dim // group)
        if v_packed.shape != k_packed.shape or k_scales.shape != scales or v_scales.shape != scales:
            raise ValueError("keys and values share one shape, with one scale byte for each block of head_dim")
        if fmt == NVFP4:
            for name, g in (("k_global_scale", k_global_scale), ("v_global_scale", v_global_scale)):
                if g is None or g.dtype != torch.float32 or g.shape != (self.heads,) or not g.is_contiguous():
                    raise ValueError(f"{name}: contiguous float32 [heads] required for NVFP4")
            _same_device(self.index, k_global_scale, v_global_scale)
        self.fmt, self.device = fmt, dev
        self.k_packed, self.k_scales, self.v_packed, self.v_scales = k_packed, k_scales, v_packed, v_scales
        self.k_global_scale, self.v_global_scale = k_global_scale, v_global_scale
        self.status = new_status(dev) if status is None else _status(status, status)
        nv = fmt == NVFP4
        self._struct = KVCacheStruct(fmt, self.heads, self.head_dim, self.page_size, self.num_pages, _p(k_packed),
                                     _p(k_scales), _p(v_packed), _p(v_scales), _p(k_global_scale) if nv else None,
                                     _p(v_global_scale) if nv else None)
        self._ref = ctypes.addressof(self._struct)
        lib()

    def check(self, where: str = "KVCache"):
        st = int(self.status.item())
        if st != OK:
            raise FP4Error(st, where)
        return self


def kv_cache(num_pages: int, heads: int, head_dim: int, page_size: int = 64, fmt: int = NVFP4, k_global_scale=None,
             v_global_scale=None, device="cuda") -> KVCache:
    """An empty (zero-filled) cache.  NVFP4 global scales: one number or a
    [heads] tensor each, amax / 2688 of a calibration run (default 1 / 64:
    values up to 42 before they saturate)."""
    group = 16 if fmt == NVFP4 else 32

    def zeros(last):
        return torch.zeros((num_pages, heads, page_size, last), dtype=torch.uint8, device=device)

    def scale(g):
        if fmt != NVFP4:
            return None
        g = torch.as_tensor(1 / 64 if g is None else g, dtype=torch.float32, device=device)
        return g.expand(heads).contiguous()
    return KVCache(fmt, zeros(head_dim // 2), zeros(head_dim // group), zeros(head_dim // 2),
                   zeros(head_dim // group), scale(k_global_scale), scale(v_global_scale))


def _token_rows(t: torch.Tensor, what: str, tokens: int, heads: int, dim: int) -> int:
    """Token stride of a [tokens, heads, dim] tensor whose heads and elements are contiguous."""
    if t.shape != (tokens, heads, dim):
        raise ValueError(f"{what}: [{tokens}, {heads}, {dim}] required, got {list(t.shape)}")
    one, head, el = t.stride()
    if tokens and (el != 1 or (heads > 1 and head != dim)):
        raise ValueError(f"{what}: contiguous heads and elements required")
    return one if tokens > 1 else heads * dim


def _slot_list(slots: torch.Tensor) -> int:
    if slots.dtype != torch.int64 or not slots.is_cuda or not slots.is_contiguous():
        raise ValueError("slots: a contiguous int64 CUDA tensor required")
    return slots.numel()


def kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, rule: int = MX_FLOOR, status=None,
             stream=None) -> None:
    """Quantise k, v [tokens, heads, head_dim] (bf16 or fp32; views of a fused
    projection may keep their token stride) into the cache's `slots` (int64
    [tokens], negative = padding).  Data errors go to `status` (default: the
    cache's)."""
    T, H, D = _slot_list(slots), cache.heads, cache.head_dim
    if k.dtype != v.dtype:
        raise TypeError("k and v share one dtype")
    ks, vs = _token_rows(k, "k", T, H, D), _token_rows(v, "v", T, H, D)
    st = _status(status, cache.status)
    _same_device(cache.index, k, v, slots, status)
    _call("fp4_kv_write", cache.index, stream, cache._ref, k.data_ptr(), v.data_ptr(), _dtype_code(k), T, ks, vs,
          slots.data_ptr(), rule, st.data_ptr())


def kv_read(cache: KVCache, slots: torch.Tensor, out_dtype=torch.bfloat16, k=None, v=None, status=None, stream=None):
    """The keys and values in `slots` (int64 [tokens]; negative gives zeros)
    as [tokens, heads, head_dim] tensors of out_dtype, or into k and v."""
    if stream is not None and (k is None or v is None):
        with _on(stream, cache.index):
            return kv_read(cache, slots, out_dtype, k, v, status)
    T, H, D = _slot_list(slots), cache.heads, cache.head_dim
    if k is None:
        k = slots.new_empty((T, H, D), dtype=out_dtype)
    if v is None:
        v = torch.empty_like(k) if k.is_contiguous() else slots.new_empty((T, H, D), dtype=k.dtype)
    if k.dtype != v.dtype:
        raise TypeError("k and v share one dtype")
    ks, vs = _token_rows(k, "k", T, H, D), _token_rows(v, "v", T, H, D)
    st = _status(status, cache.status)
    _same_device(cache.index, k, v, slots, status)
    _call("fp4_kv_read", cache.index, stream, cache._ref, slots.data_ptr(), T, k.data_ptr(), v.data_ptr(),
          _dtype_code(k), ks, vs, st.data_ptr())
    return k, v


def kv_attention_workspace(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor) -> torch.Tensor:
    """A (zero-filled) workspace for kv_attention calls of this shape, or of
    smaller batches, on caches of this head_dim, on one stream at a time."""
    B, L, HQ, _ = q.shape
    n = lib().fp4_kv_attention_workspace_bytes(cache._ref, B, L, HQ, page_table.shape[1])
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=cache.device)


def kv_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, scale=None,
                 window: int = 0, out=None, lse=None, workspace=None, status=None, stream=None):
    """Attention of the last q_tokens tokens of every sequence over the
    cache: q [batch, q_tokens, q_heads, head_dim] (bf16 or fp32; a token
    stride is kept), page_table int32 [batch, width], seq_lens int32 [batch]
    (new tokens counted, already written), scale 1/sqrt(head_dim) by default,
    window 0 = all earlier tokens.  head_dim 64, 128 or 256.  Returns (out, lse [batch, q_tokens,
    q_heads] fp32)."""
    if stream is not None and (out is None or lse is None or workspace is None):
        with _on(stream, cache.index):
            return kv_attention(q, cache, page_table, seq_lens, scale, window, out, lse, workspace, status)
    if q.dim() != 4 or q.shape[3] != cache.head_dim:
        raise ValueError(f"q: [batch, q_tokens, q_heads, {cache.head_dim}] required, got {list(q.shape)}")
    B, L, HQ, D = q.shape
    for what, t, dims in (("page_table", page_table, 2), ("seq_lens", seq_lens, 1)):
        if t.dtype != torch.int32 or t.dim() != dims or t.size(0) != B or not t.is_contiguous():
            raise ValueError(f"{what}: contiguous int32 [{B}{', width' if dims == 2 else ''}] required")
    if q.is_contiguous():
        one = HQ * D
    else:
        sb, sl, sh, el = q.stride()
        one = sl if L > 1 else sb if B > 1 else HQ * D
        if el != 1 or (HQ > 1 and sh != D) or (B > 1 and sb != one * L):
            raise ValueError("q: contiguous heads and elements and one stride from token to token required")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out: contiguous, with q's shape and dtype")
    if lse is None:
        lse = seq_lens.new_empty((B, L, HQ), dtype=torch.float32)
    elif lse.shape != (B, L, HQ) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse: contiguous float32 [batch, q_tokens, q_heads]")
    ws = kv_attention_workspace(q, cache, page_table) if workspace is None else workspace
    ws_bytes = _workspace(ws)
    st = _status(status, cache.status)
    _same_device(cache.index, q, page_table, seq_lens, out, lse, ws, status)
    _call("fp4_kv_attention", cache.index, stream, cache._ref, q.data_ptr(), _dtype_code(q), B, L, HQ, one,
          page_table.data_ptr(), page_table.size(1), seq_lens.data_ptr(), D ** -0.5 if scale is None else scale, window,
          out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws_bytes, st.data_ptr())
    return out, lse


class LinearWeight:
    """An FP4 weight [n, k] laid out for `linear`: packed codes [n, Kp/2]
    (padded layout), the scale bytes in the MMA layout, the NVFP4 global
    scale (None for MXFP4).  Kp, k rounded up to whole blocks, is a multiple
    of 32: an NVFP4 weight of an odd number of blocks a row is refused.
    `status` as for KVCache."""

    def __init__(self, fmt, packed, scales_mma, global_scale, n: int, k: int, status=None):
        group = 16 if fmt == NVFP4 else 32
        kp = _padded(k, group)
        if fmt not in (NVFP4, MXFP4):
            raise ValueError("fmt: NVFP4 or MXFP4")
        if kp % 32:
            raise ValueError(f"k: rounded up to whole blocks of {group} a multiple of 32 required, got {k}")
        dev, self.index = _cuda(packed, "packed", torch.uint8).device, packed.get_device()
        _cuda(scales_mma, "scales_mma", torch.uint8)
        if packed.numel() != n * kp // 2 or not packed.is_contiguous():
            raise ValueError(f"packed: contiguous [{n}, {kp // 2}] required")
        if scales_mma.numel() != lib().fp4_mma_scales_bytes(n, kp // group) or not scales_mma.is_contiguous():
            raise ValueError("scales_mma: the MMA layout of the [n, Kp/G] scales required (scales_to_mma)")
        if fmt == NVFP4 and (global_scale is None or global_scale.dtype != torch.float32 or global_scale.numel() != 1):
            raise ValueError("global_scale: one float32 required for NVFP4")
        _same_device(self.index, scales_mma, global_scale if fmt == NVFP4 else None, status)
        self.fmt, self.n, self.k, self.device = fmt, n, k, dev
        self.packed, self.scales_mma, self.global_scale = packed, scales_mma, global_scale
        self._packed, self._scales, self._g = _p(packed), _p(scales_mma), _p(global_scale) if fmt == NVFP4 else None
        self.status = new_status(dev) if status is None else _status(status, status)

    def check(self, where: str = "LinearWeight"):
        st = int(self.status.item())
        if st != OK:
            raise FP4Error(st, where)
        return self


def linear_weight(q: Quantized, stream=None) -> LinearWeight:
    """The quantised weight [n, k] (nvfp4_quantize, mxfp4_quantize, the
    padded and column-wise layouts, ...) laid out for `linear`, once."""
    index = _cuda(q.packed, "packed").get_device()
    _same_device(index, q.scales)
    if stream is not None:
        with _on(stream, index):
            return linear_weight(q)
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return linear_weight(q)
    return LinearWeight(q.fmt, q.packed, scales_to_mma(q.scales), q.global_scale, q.rows, q.cols)


def linear_workspace(rows: int, w: LinearWeight) -> torch.Tensor:
    """A workspace for `linear` calls of up to `rows` rows with w, on one
    stream at a time."""
    return torch.empty(max(lib().fp4_linear_workspace_bytes(rows, w.k), 16), dtype=torch.uint8, device=w.device)


def linear(x: torch.Tensor, w: LinearWeight, out_dtype=None, out=None, workspace=None, status=None,
           stream=None) -> torch.Tensor:
    """y [..., n] = x [..., k] W^T for a few rows of unquantised activations
    (bf16 or fp32; rows of a 2-D x may be strided) and an FP4 weight.
    out_dtype: x's by default."""
    if stream is not None and (out is None or workspace is None):
        with _on(stream, w.index):
            return linear(x, w, out_dtype, out, workspace, status)
    shape = x.shape
    if not shape or shape[-1] != w.k:
        raise ValueError(f"x: [..., {w.k}] required, got {list(shape)}")
    rows = shape[:-1].numel()
    if x.is_contiguous():
        stride = w.k
    elif x.dim() == 2 and (x.stride(1) == 1 or w.k == 1):
        stride = x.stride(0) if rows > 1 else w.k
    else:
        raise ValueError("x: contiguous elements required, and contiguous rows beyond two dimensions")
    if out is None:
        y = x.new_empty((*shape[:-1], w.n), dtype=out_dtype or x.dtype)
    else:
        y = out
        if y.shape != (*shape[:-1], w.n) or not y.is_contiguous() or (out_dtype is not None and y.dtype != out_dtype):
            raise ValueError(f"out: contiguous {[*shape[:-1], w.n]} of the output dtype required")
    ws = linear_workspace(rows, w) if workspace is None else workspace
    ws_bytes = _workspace(ws)
    st = _status(status, w.status)
    _same_device(w.index, x, y, ws, status)
    _call("fp4_linear", w.index, stream, w.fmt, x.data_ptr(), _dtype_code(x), rows, w.k, stride, w._packed,
          w._scales, w._g, w.n, y.data_ptr(), _dtype_code(y), ws.data_ptr(), ws_bytes,
          st.data_ptr())
    return y


def scale_search(x: torch.Tensor, with_loss: bool = True, workspace=None, status=None, stream=None,
                 grid=None) -> Quantized:
    """MSE scale search; `grid` = (n_cand, p, q) searches the candidates
    (p + k) / q x A_b / (6g), k < n_cand (default: the fixed 64, 147, 210)."""
    R, C = _shape2(x)
    dev = x.device
    packed = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((R, C // 16), dtype=torch.uint8, device=dev)
    g = torch.empty(1, dtype=torch.float32, device=dev)
    loss = torch.empty((R, C // 16), dtype=torch.float32, device=dev) if with_loss else None
    ws = workspace if workspace is not None else workspace_for(x)
    st = status if status is not None else new_status(dev)
    if grid is None:
        _check(fp4_scale_search(x, packed, scales, g, loss, ws, st, stream), "fp4_scale_search")
    else:
        n_cand, p, q = grid
        _check(lib().fp4_scale_search_grid(_p(x), _dtype_code(x), R, C, int(n_cand), int(p), int(q), _p(packed),
                                           _p(scales), _p(g), _p(loss), _p(ws), ws.numel() * ws.element_size(),
                                           _p(st), _stream(stream)), "fp4_scale_search_grid")
    return Quantized(NVFP4, packed, scales, g, st, R, C, block_loss=loss)


def tensor_amax(x: torch.Tensor, workspace=None, status=None, stream=None):
    dev = x.device
    a = torch.empty(1, dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else workspace_for(x)
    st = status if status is not None else new_status(dev)
    _check(fp4_tensor_amax(x, a, ws, st, stream), "fp4_tensor_amax")
    return a, st


def e2m1_round(v: torch.Tensor, stream=None) -> torch.Tensor:
    codes = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    _check(fp4_e2m1_round(v, codes, stream), "fp4_e2m1_round")
    return codes


def e2m1_roundtrip(v: torch.Tensor, stream=None) -> torch.Tensor:
    out = torch.empty((v.numel(), 2), dtype=torch.float32, device=v.device)
    _check(fp4_e2m1_roundtrip(v, out, stream), "fp4_e2m1_roundtrip")
    return out


def nv_encode_quotient(x: torch.Tensor, d: torch.Tensor, stream=None) -> torch.Tensor:
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(fp4_nv_encode_quotient(x, d, codes, stream), "fp4_nv_encode_quotient")
    return codes
