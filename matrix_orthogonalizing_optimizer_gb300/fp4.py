"""Python API of the operators on matrices in microscaled 4-bit floating point: quantisation along
rows, columns or both, the values back, and the products A B^T and X X^T on the 4-bit tensor cores.

Dense tensors follow the rules of the matrix calls (bfloat16, float16 or float32, 2-D or 3-D, rows on
16-byte boundaries); a Fp4Matrix holds a matrix, or a batch of them, in 4 bits. Everything that a
call is given lies on one device, whichever is the current one.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import GnsFp4, load
from ._lib import check as check_rc
from .api import (_CallStatus, _dtype_code, _elsewhere, _launch, _on_stream, _one_device, _stream_ptr, batch_of,
                  empty_padded)

_FORMATS = {"nvfp4": _lib.GNS_NVFP4, "mxfp4": _lib.GNS_MXFP4}
_BLOCK = {"nvfp4": 16, "mxfp4": 32}


def _format_code(fmt: str) -> int:
    if fmt not in _FORMATS:
        raise ValueError(f"fmt must be one of {sorted(_FORMATS)}")
    return _FORMATS[fmt]


def _tiles(rows: int, cols: int, fmt: str):
    blocks = -(-cols // _BLOCK[fmt])
    return -(-rows // 128), -(-blocks // 4), 512


class Fp4Matrix:
    """A matrix (or a batch of them) in 4-bit floating point, as include/gns.h lays it out (gns_fp4). It keeps its
    tensors alive, and describes the memory that they have when it is made: its attributes cannot be assigned,
    and a tensor that got new memory needs a new Fp4Matrix.

    codes: uint8, (rows, bytes) or (count, rows, bytes), two codes a byte (the first in the low
        half), at least ceil(cols / 32) * 16 bytes a row; rows on 16-byte boundaries.
    scales: uint8, (row tiles, block tiles, 512) or (count, ...), without gaps inside a matrix.
    tensor_scale: float32, one for each matrix ("nvfp4"; a power of two from quantize_fp4, else any finite number that is
        not negative), or None ("mxfp4").
    cols: values in a row."""

    # addresses and sizes are noted once: the kernels would go on reading the memory of a tensor that was put elsewhere
    _FIXED = frozenset(("codes", "scales", "tensor_scale", "fmt", "shape", "device", "index", "_struct", "_ref"))

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, tensor_scale: Optional[torch.Tensor], cols: int,
                 fmt: str = "nvfp4"):
        code = _format_code(fmt)
        if not codes.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if codes.dim() not in (2, 3):
            raise ValueError("codes must be 2-D or 3-D")
        cols = int(cols)
        *lead, rows, width = codes.shape
        if cols < 1 or width < -(-cols // 32) * 16 or (width > 1 and codes.stride(-1) != 1):
            raise ValueError(f"codes must hold {-(-cols // 32) * 16} bytes a row, one behind the other, for {cols} columns")
        want = (*lead, *_tiles(rows, cols, fmt))
        if tuple(scales.shape) != want:
            raise ValueError(f"scales must have the shape {want}, not {tuple(scales.shape)}")
        inner = scales if not lead or lead[0] == 0 else scales[0]
        if not inner.is_contiguous():
            raise ValueError("the scales of a matrix must be contiguous")
        count = lead[0] if lead else 1
        if fmt == "nvfp4":
            if (tensor_scale is None or tensor_scale.dtype != torch.float32 or tensor_scale.numel() != count
                    or not tensor_scale.is_contiguous()):
                raise ValueError(f"tensor_scale must be a contiguous float32 tensor of {count} entries")
        elif tensor_scale is not None:
            raise ValueError("mxfp4 has no tensor_scale")
        index = codes.get_device()
        _one_device(index, scales=scales, tensor_scale=tensor_scale)
        q = GnsFp4()
        b = q.codes
        b.ptr, b.count, b.rows, b.cols = codes.data_ptr(), count, rows, cols
        b.ld = 2 * (codes.stride(-2) if rows > 1 else -(-cols // 32) * 16)
        b.stride = 2 * codes.stride(0) if count > 1 else rows * b.ld
        q.scales = scales.data_ptr()
        q.scale_stride = scales.stride(0) if lead else scales.numel()
        q.tensor_scale = tensor_scale.data_ptr() if tensor_scale is not None else None
        q.format = code
        self.__dict__.update(codes=codes, scales=scales, tensor_scale=tensor_scale, fmt=fmt, device=codes.device, index=index,
                             shape=torch.Size((*lead, rows, cols)), _struct=q, _ref=ctypes.byref(q))

    def __setattr__(self, name, value):
        if name in self._FIXED:
            raise AttributeError(f"{name} of an Fp4Matrix cannot be assigned: make a new one")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        if name in self._FIXED:
            raise AttributeError(f"{name} of an Fp4Matrix cannot be deleted")
        super().__delattr__(name)

    def __repr__(self):
        return f"Fp4Matrix(shape={tuple(self.shape)}, fmt={self.fmt!r}, device='{self.device}')"


def empty_fp4(shape, fmt: str = "nvfp4", device=None) -> Fp4Matrix:
    """An uninitialised Fp4Matrix of `shape`, (rows, cols) or (count, rows, cols)."""
    _format_code(fmt)
    if len(shape) not in (2, 3) or any(int(n) < 1 for n in shape):
        raise ValueError("shape must be (rows, cols) or (count, rows, cols), every size at least 1")
    *lead, rows, cols = (int(n) for n in shape)
    device = torch.device("cuda") if device is None else device
    codes = torch.empty((*lead, rows, -(-cols // 32) * 16), dtype=torch.uint8, device=device)
    scales = torch.empty((*lead, *_tiles(rows, cols, fmt)), dtype=torch.uint8, device=device)
    g = torch.empty(lead[0] if lead else 1, dtype=torch.float32, device=device) if fmt == "nvfp4" else None
    return Fp4Matrix(codes, scales, g, cols, fmt)


def _parts(q: Fp4Matrix):
    return (q.codes, q.scales) if q.tensor_scale is None else (q.codes, q.scales, q.tensor_scale)


def _new(shape, fmt, device, stream) -> Fp4Matrix:
    q = _on_stream(stream, lambda: empty_fp4(shape, fmt, device))
    if stream is not None:  # the caller, who is on the current stream, gets it
        for t in _parts(q):
            t.record_stream(torch.cuda.current_stream(device))
    return q


def _fp4(name: str, q, index: Optional[int] = None) -> Fp4Matrix:
    if not isinstance(q, Fp4Matrix):
        raise TypeError(f"{name} must be a Fp4Matrix")
    if index is not None and q.index != index:
        raise _elsewhere(name, index)
    return q


_AXES = {"rows": (True, False), "cols": (False, True), "both": (True, True)}


def quantize_fp4(x: torch.Tensor, fmt: str = "nvfp4", axes: str = "rows", out: Optional[Fp4Matrix] = None,
                 out_t: Optional[Fp4Matrix] = None, amax: Optional[torch.Tensor] = None, status=None, stream=None,
                 check: bool = True):
    """Brings x into 4 bits (gns_fp4_quantize; fmt "nvfp4" or "mxfp4"): along its rows (axes "rows"), along its
    columns ("cols": the Fp4Matrix of the transpose), or both with one reading ("both": returns
    the pair). out and out_t, where one is given, are written and say which axes are wanted.

    amax: a CUDA float32 tensor with the largest magnitude of each matrix ("nvfp4"), e.g. an
        earlier step's; without it x is read once more for its own.
    Inf or NaN in x make the scale of their block NaN, and are a device condition (see
    gram_ns_batched)."""
    _format_code(fmt)
    if axes not in _AXES:
        raise ValueError(f"axes must be one of {sorted(_AXES)}")
    xb = batch_of(x)
    code = _dtype_code(x)
    index = x.device.index
    if out is None and out_t is None:
        rows, cols = _AXES[axes]
        *lead, r, c = x.shape
        out = _new((*lead, r, c), fmt, x.device, stream) if rows else None
        out_t = _new((*lead, c, r), fmt, x.device, stream) if cols else None
    for name, q in (("out", out), ("out_t", out_t)):
        if q is not None and _fp4(name, q, index).fmt != fmt:
            raise ValueError(f"{name} must be of the format {fmt}")
    if amax is not None:
        _one_device(index, amax=amax)
        if amax.dtype != torch.float32 or amax.numel() != xb.count or not amax.is_contiguous():
            raise ValueError(f"amax must be a contiguous float32 tensor of {xb.count} entries")
    cs = _CallStatus(status, x.device, check, stream)
    rc = _launch(index, load().gns_fp4_quantize, ctypes.byref(xb), code, out._ref if out is not None else None,
                 out_t._ref if out_t is not None else None, amax.data_ptr() if amax is not None else None, cs.ptr(),
                 _stream_ptr(stream, x.device))
    check_rc(rc, "gns_fp4_quantize")
    cs.done("gns_fp4_quantize")
    return out if out_t is None else out_t if out is None else (out, out_t)


def dequantize_fp4(q: Fp4Matrix, out: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                   stream=None) -> torch.Tensor:
    """The values of q in `out`, or in a new tensor of type `dtype`."""
    _fp4("q", q)
    if out is None:
        out = _on_stream(stream, lambda: empty_padded(q.shape, dtype, q.device), returned=True)
    ob = batch_of(out)
    code = _dtype_code(out)
    _one_device(q.index, out=out)
    rc = _launch(q.index, load().gns_fp4_dequantize, q._ref, ctypes.byref(ob), code, _stream_ptr(stream, q.device))
    check_rc(rc, "gns_fp4_dequantize")
    return out


def _product(entry: str, operands, shape, c, d, alpha, beta, dtype, status, stream, check):
    first = operands[0]
    if d is None:
        dtype = dtype if dtype is not None else c.dtype if c is not None else torch.bfloat16
        d = _on_stream(stream, lambda: empty_padded(shape, dtype, first.device), returned=True)
    elif dtype is not None and d.dtype != dtype:
        raise TypeError(f"d must be of type {dtype}")
    if beta != 0.0:
        if c is None:
            raise ValueError("c is required when beta != 0")
        if c.dtype != d.dtype:
            raise TypeError("c must be of d's type")
    db = batch_of(d)
    cb = batch_of(c) if c is not None else None
    code = _dtype_code(d)
    _one_device(first.index, c=c, d=d)
    cs = _CallStatus(status, first.device, check, stream)
    rc = _launch(first.index, getattr(load(), entry), *[q._ref for q in operands],
                 ctypes.byref(cb) if cb is not None else None, ctypes.byref(db), float(alpha), float(beta), code,
                 cs.ptr(), _stream_ptr(stream, first.device))
    check_rc(rc, entry)
    cs.done(entry)
    return d


def fp4_gemm(a: Fp4Matrix, b: Fp4Matrix, c: Optional[torch.Tensor] = None, d: Optional[torch.Tensor] = None,
             alpha: float = 1.0, beta: float = 0.0, dtype: Optional[torch.dtype] = None, status=None, stream=None,
             check: bool = True) -> torch.Tensor:
    """d <- alpha a b^T + beta c (gns_fp4_gemm) of a (m x k) and b (n x k), or batches of them; a new tensor of
    type `dtype` (c's, else bfloat16) where no d is given. d may be c.

    The forward product of a layer y = x w^T is fp4_gemm(xq, wq); with (xq, xt), (wq, wt) and
    (gq, gt) from quantize_fp4(..., axes="both") of x, w and dy, its gradients are
    dx = fp4_gemm(gq, wt) and dw = fp4_gemm(gt, xt)."""
    _fp4("a", a)
    _fp4("b", b, a.index)
    return _product("gns_fp4_gemm", (a, b), (*a.shape[:-1], b.shape[-2]), c, d, alpha, beta, dtype, status, stream,
                    check)


def fp4_sym_gemm_xxt(x: Fp4Matrix, c: Optional[torch.Tensor] = None, d: Optional[torch.Tensor] = None,
                     alpha: float = 1.0, beta: float = 0.0, dtype: Optional[torch.dtype] = None, status=None,
                     stream=None, check: bool = True) -> torch.Tensor:
    """d <- alpha x x^T + beta c (gns_fp4_sym_gemm_xxt); c must be symmetric, d may be c."""
    _fp4("x", x)
    return _product("gns_fp4_sym_gemm_xxt", (x,), (*x.shape[:-1], x.shape[-2]), c, d, alpha, beta, dtype, status,
                    stream, check)
