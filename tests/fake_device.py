"""Stand-ins for device memory, streams, devices and the library: what the Python API does around a call, tested
where there is no GPU (or only one)."""
import contextlib
import math

import pytest
import torch

from matrix_orthogonalizing_optimizer_gb300 import api, tensor_lists


class Memory:
    """A device tensor as far as the calls look at one."""
    is_cuda = True

    def __init__(self, shape, dtype, device, stream=None):
        self.shape = torch.Size((shape,) if isinstance(shape, int) else shape)
        self.dtype, self.device, self.stream, self.recorded = dtype, device, stream, []

    def data_ptr(self):
        return 1 << 20

    def get_device(self):
        return self.device.index

    def numel(self):
        return math.prod(self.shape)

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def element_size(self):
        return 4

    def stride(self, d=None):
        s = [math.prod(self.shape[i + 1:]) for i in range(len(self.shape))]
        return tuple(s) if d is None else s[d]

    def record_stream(self, stream):
        self.recorded.append(stream)

    def __getitem__(self, _):
        return self


class Stream:
    def __init__(self, name, index=0):
        self.waits = 0
        self.name, self.cuda_stream, self.device = name, 77, torch.device("cuda", index)

    def synchronize(self):
        self.waits += 1


class Library:
    """Every entry point: notes its name and the current device, and succeeds; sizes are some bytes."""

    def __init__(self, devices):
        self.devices, self.calls = devices, []

    def __getattr__(self, name):
        if "size" in name:
            return lambda *a: 4096
        return lambda *a: self.calls.append((name, self.devices[-1])) or 0


@pytest.fixture
def world(monkeypatch):
    here = Stream("current")
    now, made, devices = [here], [], [0]
    library = Library(devices)
    device = torch.device("cuda", 0)

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    @contextlib.contextmanager
    def on_device(d):
        devices.append(d if isinstance(d, int) else torch.device(d).index)
        yield
        devices.pop()

    def empty(*shape, dtype=torch.float32, device=device, **_):
        shape = shape[0] if len(shape) == 1 else shape
        made.append(Memory(shape, dtype, device, now[-1]))
        return made[-1]

    def current_stream(d=None):
        index = 0 if d is None else torch.device(d).index
        return now[-1] if now[-1].device.index == index else Stream("another device's", index)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    # a tensor is one tensor, not a list of its rows
    monkeypatch.setattr(api, "_as_list", lambda x: [x] if isinstance(x, Memory) else list(x))
    monkeypatch.setattr(torch.cuda, "device", on_device)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: devices[-1])
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: now[-1].cuda_stream, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: devices[-1], raising=False)
    for m in (api, tensor_lists):
        monkeypatch.setattr(m, "load", lambda: library)
    return {"here": here, "made": made, "device": device, "library": library, "status": Memory(1, torch.int32, device)}


def tensor(w, *shape, dtype=torch.bfloat16, index=0):
    return Memory(shape, dtype, torch.device("cuda", index))


class OnDevice:
    """A CPU tensor that says it lives on a GPU: describing it launches nothing."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    dtype = property(lambda s: s.t.dtype)
    shape = property(lambda s: s.t.shape)
    device = property(lambda s: s.t.device)

    def data_ptr(self):
        return self.t.data_ptr()

    def numel(self):
        return self.t.numel()

    def stride(self, d=None):
        return self.t.stride() if d is None else self.t.stride(d)

    def is_contiguous(self):
        return self.t.is_contiguous()

    def permute(self, order):
        return OnDevice(self.t.permute(order))
