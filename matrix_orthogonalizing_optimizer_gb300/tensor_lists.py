"""Python API of the operators over lists of tensors: the global gradient norm, clipping by it,
and the AdamW step of the parameters beside Muon's matrices (embeddings, heads, gains, biases).

A list may mix shapes and dtypes (bfloat16, float16, float32). Its tensors are CUDA tensors
without gaps in memory (contiguous, or a permutation of a contiguous tensor such as a
transpose), or batches of rows with a pitch: leading dimensions that collapse to one, then
rows, then a contiguous last dimension. They may start at any element. Everything that a call is
given lies on one device, whichever is the current one. Every call takes a
plain sequence of tensors or a TensorList, which describes the tensors to the library once; a
program that keeps its parameters, states and gradients in the same buffers keeps their
TensorLists too.
"""
from __future__ import annotations

import ctypes
import math
import struct
from dataclasses import dataclass
from functools import cached_property
from typing import Optional, Sequence, Union

import torch

from . import _lib
from ._lib import GnsAdamwParams, GnsTensor, load
from ._lib import check as check_rc
from .api import _CallStatus, _device_scalar, _dtype_code, _elsewhere, _on_stream, _status_ptr, alloc_workspace


# Field by field a descriptor costs ten times what one packed write does.
_PACK = struct.Struct("PqqqqqiI").pack_into
assert struct.calcsize("PqqqqqiI") == ctypes.sizeof(GnsTensor)
_CODES = {torch.bfloat16: _lib.GNS_BF16, torch.float16: _lib.GNS_F16, torch.float32: _lib.GNS_F32}


def _describe(array, at: int, t: torch.Tensor):
    """Writes the descriptor of one tensor at byte `at`; returns what has to agree between the
    roles of an operator: its shape, and the order of its dimensions in memory unless that is the
    usual."""
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    code = _CODES.get(t.dtype)
    if code is None:
        code = _dtype_code(t)  # says what is supported
    shape = tuple(t.shape)
    n = len(shape)
    if t.is_contiguous():
        if n == 1:
            _PACK(array, at, t.data_ptr(), 1, 1, shape[0], shape[0], shape[0], code, 0)
        elif n == 2:
            rows, cols = shape
            _PACK(array, at, t.data_ptr(), 1, rows, cols, cols, rows * cols, code, 0)
        elif n == 0:
            _PACK(array, at, t.data_ptr(), 1, 1, 1, 1, 1, code, 0)
        else:
            rows, cols = shape[-2:]
            _PACK(array, at, t.data_ptr(), math.prod(shape[:-2]), rows, cols, cols, rows * cols, code, 0)
        return shape
    steps = t.stride()
    if n == 2 and steps[1] == 1 and steps[0] >= shape[1]:
        _PACK(array, at, t.data_ptr(), 1, shape[0], shape[1], steps[0], shape[0] * steps[0], code, 0)
        return shape
    if n == 3 and steps[2] == 1 and steps[1] >= shape[2] and steps[0] >= (shape[1] - 1) * steps[1] + shape[2]:
        _PACK(array, at, t.data_ptr(), *shape, steps[1], steps[0], code, 0)
        return shape
    # a dimension of size 1 has a stride of no meaning
    dims = [d for d in range(n) if shape[d] != 1]
    order = tuple(sorted(dims, key=lambda d: (-steps[d], -shape[d], d)))
    whole = 1
    for d in reversed(order):
        if steps[d] != whole:
            break
        whole *= shape[d]
    else:  # a permutation of a contiguous tensor: the one that it permutes
        count, rows, cols = math.prod([shape[d] for d in order[:-2]]), shape[order[-2]], shape[order[-1]]
        _PACK(array, at, t.data_ptr(), count, rows, cols, cols, rows * cols, code, 0)
        return shape, order
    # leading dimensions that lie evenly behind one another are one
    rows, ld = (shape[-2], steps[-2]) if n > 1 else (1, 0)
    cols, one = shape[-1], steps[-1]
    lead = [d for d in dims if d < n - 2]
    count, stride = math.prod([shape[d] for d in lead]), steps[lead[-1]] if lead else 0
    if any(steps[a] != steps[b] * shape[b] for a, b in zip(lead, lead[1:])) or (one != 1 and cols > 1) or (
            rows > 1 and ld < cols) or (count > 1 and stride < (rows - 1) * ld * (rows > 1) + cols):
        raise ValueError(f"a tensor of shape {shape} with strides {tuple(t.stride())} is neither without gaps nor a "
                         "batch of rows with a contiguous last dimension: make it contiguous")
    _PACK(array, at, t.data_ptr(), count, rows, cols, max(ld, cols), stride, code, 0)
    return shape


class TensorList:
    """The library's descriptors of a list of tensors, which it keeps alive. Made once for
    buffers that stay where they are; a tensor that got new memory needs a new TensorList. An
    entry may be None (an AdamW master that a tensor has not)."""

    def __init__(self, tensors: Sequence[Optional[torch.Tensor]]):
        self.tensors = list(tensors)
        if not self.tensors:
            raise ValueError("need at least one tensor")
        self.array = (GnsTensor * len(self.tensors))()
        self.address = ctypes.addressof(self.array)
        self.device = None
        layout = []
        array, size, at = self.array, ctypes.sizeof(GnsTensor), 0
        for t in self.tensors:
            if t is None:
                layout.append(None)
            else:
                layout.append(_describe(array, at, t))
                if self.device is None:
                    self.device = t.device
                elif self.device != t.device:
                    raise ValueError("the tensors of a list must live on one device")
            at += size
        self.index = None if self.device is None else self.device.index
        # where there is one device it is the current one: asking takes 0.2 us of a call's 6
        self.one_device = torch.cuda.device_count() == 1
        self.has_none = None in layout
        self.layout = layout
        # two lists of hundreds of tensors, and their devices, compare at once
        self.layout_key = hash((self.index, *layout))
        self.reordered = any(x is not None and x and type(x[0]) is tuple for x in layout)

    @cached_property
    def has_empty(self) -> bool:
        return any(x and 0 in x for x in self.layout)

    def __len__(self):
        return len(self.tensors)


def tensor_list(tensors: Union[TensorList, torch.Tensor, Sequence[Optional[torch.Tensor]]]) -> TensorList:
    """The TensorList of a sequence of tensors (or of one tensor); a TensorList is itself."""
    if isinstance(tensors, TensorList):
        return tensors
    return TensorList([tensors] if isinstance(tensors, torch.Tensor) else tensors)


def _stream(stream: Optional[torch.cuda.Stream], index: int) -> int:
    """The stream's handle; for the device's current one without building a Stream object, which
    takes as long as a launch."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device.index != index:
        raise _elsewhere("stream", index)
    return stream.cuda_stream


def _device_of(x: TensorList):
    """The context in which the tensors' device is the current one, where a launch belongs: a
    stream's handle of 0 is the current device's default stream."""
    if x.index is None:
        raise ValueError("every gradient and every weight must be a tensor")
    return torch.cuda.device(x.index)


def _same_layout(name: str, a: TensorList, b: TensorList, optional: bool = False) -> None:
    if a.layout_key == b.layout_key:
        return
    if a.index != b.index and b.index is not None:
        raise _elsewhere(name, a.index)
    if optional and not a.reordered and not b.reordered and not b.has_empty and len(a) == len(b):
        # the library compares the shapes itself: what it cannot see is the order in memory, and an empty
        # tensor where it takes one for none
        return
    if len(a) != len(b):
        raise ValueError(f"{name}: {len(b)} tensors, expected {len(a)}")
    for i, (x, y) in enumerate(zip(a.layout, b.layout)):
        if x != y and not (optional and y is None):
            raise ValueError(f"{name}[{i}]: shape (and order in memory) {y}, expected {x}")


def list_workspace_size(n: int) -> int:
    """Bytes of workspace grad_norm and clip_grads need for a list of n tensors."""
    need = load().gns_list_workspace_size(int(n))
    if need == 0:
        raise _lib.GnsError(f"list_workspace_size: {_lib.last_error()}")
    return int(need)


_NORMS = {2: _lib.GNS_NORM_L2, math.inf: _lib.GNS_NORM_INF}


def _norm_code(norm_type) -> int:
    code = _NORMS.get(norm_type)
    if code is None:
        raise ValueError("norm_type must be 2 or math.inf")
    return code


def _norm_buffers(grads: TensorList, result, workspace, stream):
    if grads.has_none:
        raise ValueError("every gradient must be a tensor")
    if result is None:
        result = _on_stream(stream, lambda: torch.empty(2, dtype=torch.float32, device=grads.device), returned=True)
    elif (result.dtype != torch.float32 or result.get_device() != grads.index or result.numel() != 2
          or not result.is_contiguous()):
        raise ValueError(f"result must be a contiguous float32 tensor of 2 entries on cuda:{grads.index}")
    if workspace is None:
        workspace = _on_stream(stream, lambda: alloc_workspace(list_workspace_size(len(grads)), grads.device))
    elif workspace.get_device() != grads.index:
        raise _elsewhere("workspace", grads.index)
    return result, workspace


def grad_norm(grads, max_norm: Optional[float] = None, norm_type: float = 2.0, eps: float = 1e-6, result=None,
              workspace=None, status=None, stream=None, check: bool = True) -> torch.Tensor:
    """Global norm of a list of gradients: the square root of the sum of squares over all of
    them (norm_type 2), or their largest magnitude (math.inf). Returns `result`, a float32
    tensor: result[0] the norm, result[1] the scale min(1, max_norm / (norm + eps)) that clips
    the gradients to max_norm (1 without max_norm, also where the norm is not finite), which
    adamw_step and muon_step take as grad_scale without a pass over the gradients. A norm that is not finite is a device
    condition (see gram_ns_batched): it raises GnsDeviceError unless `status` is given or
    `check` is off. With `stream` the call runs there: whoever reads the result on another
    stream waits for that one first."""
    g = tensor_list(grads)
    if not g.one_device and torch._C._cuda_getDevice() != g.index:
        with _device_of(g):
            return grad_norm(g, max_norm, norm_type, eps, result, workspace, status, stream, check)
    code = _norm_code(norm_type)
    result, ws = _norm_buffers(g, result, workspace, stream)
    cs = _CallStatus(None, g.device, check, stream) if status is None else None
    rc = load().gns_grad_norm(g.address, len(g), code, math.inf if max_norm is None else float(max_norm), float(eps),
                              result.data_ptr(), ws.data_ptr(), ws.numel(),
                              cs.ptr() if cs else _status_ptr(status, g.index), _stream(stream, g.index))
    if rc:
        check_rc(rc, "gns_grad_norm")
    if cs:
        cs.done("gns_grad_norm")
    return result


def clip_grads(grads, max_norm: float, norm_type: float = 2.0, eps: float = 1e-6, outs=None, result=None,
               workspace=None, status=None, stream=None, check: bool = True) -> torch.Tensor:
    """Clips a list of gradients to the global norm max_norm: each is multiplied by grad_norm's
    scale, in place or, with `outs` (a list of the same shapes and dtypes), into other buffers.
    Returns `result` as grad_norm does (the norm before clipping, the scale)."""
    g = tensor_list(grads)
    if not g.one_device and torch._C._cuda_getDevice() != g.index:
        with _device_of(g):
            return clip_grads(g, max_norm, norm_type, eps, outs, result, workspace, status, stream, check)
    code = _norm_code(norm_type)
    out_address = None
    if outs is not None:
        o = tensor_list(outs)
        _same_layout("outs", g, o)
        out_address = o.address
    result, ws = _norm_buffers(g, result, workspace, stream)
    cs = _CallStatus(None, g.device, check, stream) if status is None else None
    rc = load().gns_clip_grads(g.address, out_address, len(g), code, float(max_norm), float(eps), result.data_ptr(),
                               ws.data_ptr(), ws.numel(), cs.ptr() if cs else _status_ptr(status, g.index),
                               _stream(stream, g.index))
    if rc:
        check_rc(rc, "gns_clip_grads")
    if cs:
        cs.done("gns_clip_grads")
    return result


@dataclass
class AdamWParams:
    """Hyper-parameters of one AdamW step (gns_adamw_params); step is the number of the step, 1
    for the first."""
    lr: float
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.01
    step: int = 1

    def c_struct(self) -> GnsAdamwParams:
        return GnsAdamwParams(self.lr, self.beta1, self.beta2, self.eps, self.weight_decay, self.step)


def adamw_step(W, G, M, V, lr: Optional[float] = None, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.01, step: int = 1, masters=None, params: Optional[AdamWParams] = None,
               grad_scale: Optional[torch.Tensor] = None, step_count: Optional[torch.Tensor] = None, status=None,
               stream=None, check: bool = True):
    """One AdamW step in place on the lists W (weights), M and V (float32 first and second
    moments) with the gradients G; `params` supplies every hyper-parameter when given.

    masters: float32 copies of 16-bit weights (None for a weight that has none): the master is
        updated and W receives it rounded.
    grad_scale: a CUDA float32 tensor of one element that multiplies the gradients, e.g.
        result[1:] of grad_norm.
    step_count: a CUDA int32 tensor of one element that holds the step's number in place of
        `step`; a step captured into a CUDA graph needs it, as the graph replays `step` as it was."""
    w, g, m, v = tensor_list(W), tensor_list(G), tensor_list(M), tensor_list(V)
    if not w.one_device and torch._C._cuda_getDevice() != w.index:
        with _device_of(w):
            return adamw_step(w, g, m, v, lr, beta1, beta2, eps, weight_decay, step, masters, params, grad_scale,
                              step_count, status, stream, check)
    if params is None:
        if lr is None:
            raise ValueError("adamw_step needs lr (or params)")
        params = AdamWParams(lr, beta1, beta2, eps, weight_decay, step)
    if w.has_none:
        raise ValueError("every weight must be a tensor")
    if not w.layout_key == g.layout_key == m.layout_key == v.layout_key:
        _same_layout("G", w, g)
        _same_layout("M", w, m)
        _same_layout("V", w, v)
    master_address = None
    if masters is not None:
        p = tensor_list(masters)
        _same_layout("masters", w, p, optional=True)
        master_address = p.address
    cs = _CallStatus(None, w.device, check, stream) if status is None else None
    rc = load().gns_adamw_step(w.address, g.address, m.address, v.address, master_address, len(w),
                               ctypes.byref(params.c_struct()),
                               _device_scalar("grad_scale", grad_scale, torch.float32, w.index),
                               _device_scalar("step_count", step_count, torch.int32, w.index),
                               cs.ptr() if cs else _status_ptr(status, w.index), _stream(stream, w.index))
    if rc:
        check_rc(rc, "gns_adamw_step")
    if cs:
        cs.done("gns_adamw_step")
