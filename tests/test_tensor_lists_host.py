"""Lists of tensors on the host: what gns_grad_norm, gns_clip_grads and gns_adamw_step refuse before
anything is launched (the pointers here are fake), and how tensors are described to them."""
import ctypes
import math

import pytest

from matrix_orthogonalizing_optimizer_gb300 import _lib, build

torch = pytest.importorskip("torch")
from matrix_orthogonalizing_optimizer_gb300 import tensor_lists  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


WS = ctypes.c_void_p(1 << 30)
RESULT = ctypes.c_void_p(1 << 29)


def _list(*entries):
    """entries: dicts over count, rows, cols, ld, stride, dtype, ptr."""
    arr = (_lib.GnsTensor * len(entries))()
    for i, e in enumerate(entries):
        t = arr[i]
        t.x.count, t.x.rows, t.x.cols = e.get("count", 1), e.get("rows", 1), e.get("cols", 64)
        t.x.ld = e.get("ld", t.x.cols)
        t.x.stride = e.get("stride", t.x.rows * t.x.ld)
        t.x.ptr = e.get("ptr", (i + 1) << 20)
        t.dtype = e.get("dtype", _lib.GNS_F32)
    return arr


def _norm(lib, arr, n=None, norm_type=0, max_norm=1.0, eps=1e-6, result=RESULT, ws=WS, ws_bytes=1 << 28):
    return lib.gns_grad_norm(arr, len(arr) if n is None else n, norm_type, max_norm, eps, result, ws, ws_bytes, None, None)


def test_workspace_size(lib):
    one = lib.gns_list_workspace_size(1)
    assert 0 < one <= 1 << 16
    assert lib.gns_list_workspace_size(100000) > one
    assert lib.gns_list_workspace_size(0) == 0 and b"at least one" in _lib.last_error().encode()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(n=0), _lib.GNS_ERR_INVALID, "at least one"),
    (dict(norm_type=2), _lib.GNS_ERR_INVALID, "norm type"),
    (dict(max_norm=-1.0), _lib.GNS_ERR_INVALID, "max_norm"),
    (dict(max_norm=math.nan), _lib.GNS_ERR_INVALID, "max_norm"),
    (dict(eps=-1.0), _lib.GNS_ERR_INVALID, "eps"),
    (dict(eps=math.inf), _lib.GNS_ERR_INVALID, "eps"),
    (dict(result=None), _lib.GNS_ERR_INVALID, "null"),
    (dict(result=ctypes.c_void_p(2)), _lib.GNS_ERR_INVALID, "unaligned"),
    (dict(ws=None), _lib.GNS_ERR_WORKSPACE, "null workspace"),
    (dict(ws=ctypes.c_void_p(128)), _lib.GNS_ERR_WORKSPACE, "256"),
    (dict(ws_bytes=64), _lib.GNS_ERR_WORKSPACE, "too small"),
])
def test_norm_refuses_arguments(lib, kw, code, msg):
    assert _norm(lib, _list({}), **kw) == code
    assert msg in _lib.last_error()


@pytest.mark.parametrize("entry,msg", [
    (dict(dtype=3), "dtype"),
    (dict(ptr=None), "null data pointer"),
    (dict(ptr=(1 << 20) + 2), "aligned to an element"),
    (dict(cols=-1), ">= 0"),
    (dict(rows=4, cols=8, ld=7), "ld must"),
    (dict(count=2, rows=4, cols=8, ld=10, stride=37), "overlap"),
    (dict(count=2, rows=1, cols=8, stride=7), "overlap"),
    (dict(count=1 << 20, rows=1 << 20, cols=2, ld=2), "2^40"),
])
def test_lists_refuse_tensors(lib, entry, msg):
    """Every operator says which tensor of which list it refuses."""
    arr = _list({}, entry)
    assert _norm(lib, arr) == _lib.GNS_ERR_INVALID
    assert msg in _lib.last_error() and "grads[1]" in _lib.last_error()


def test_pitched_rows_beyond_32_bits_are_refused(lib):
    assert _norm(lib, _list(dict(rows=1 << 31, cols=2, ld=3))) == _lib.GNS_ERR_UNSUPPORTED


def test_clip_refuses_outs(lib):
    def clip(g, o):
        return lib.gns_clip_grads(g, o, len(g), 0, 1.0, 1e-6, RESULT, WS, 1 << 28, None, None)

    g = _list(dict(rows=4, cols=8))
    assert clip(g, _list(dict(rows=8, cols=4))) == _lib.GNS_ERR_INVALID and "shape" in _lib.last_error()
    assert clip(g, _list(dict(rows=4, cols=8, dtype=_lib.GNS_BF16))) == _lib.GNS_ERR_INVALID and "dtype" in _lib.last_error()
    assert clip(g, _list(dict(rows=4, cols=8, ld=9))) == _lib.GNS_ERR_INVALID and "layout" in _lib.last_error()


def _adamw(lib, w=None, g=None, m=None, v=None, master=None, step_count=None, scale=None, **kw):
    base = dict(rows=4, cols=8)
    lists = [_list(dict(base, ptr=(k + 1) << 20, **(e or {}))) for k, e in enumerate((w, g, m, v))]
    p = _lib.GnsAdamwParams(kw.pop("lr", 1e-3), kw.pop("beta1", 0.9), kw.pop("beta2", 0.99), kw.pop("eps", 1e-8),
                            kw.pop("weight_decay", 0.0), kw.pop("step", 1))
    ms = None if master is None else _list(dict(base, ptr=9 << 20, **master))
    return lib.gns_adamw_step(*lists, ms, 1, ctypes.byref(p), scale, step_count, None, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(lr=math.nan), "finite"),
    (dict(weight_decay=math.inf), "finite"),
    (dict(beta1=1.0), "beta1"),
    (dict(beta2=-0.1), "beta1 and beta2"),
    (dict(eps=0.0), "eps"),
    (dict(step=0), "step"),
    (dict(scale=ctypes.c_void_p(2)), "unaligned"),
    (dict(step_count=ctypes.c_void_p(2)), "unaligned"),
    (dict(g=dict(cols=9)), "G[0]"),
    (dict(m=dict(dtype=_lib.GNS_BF16)), "M[0]: must be f32"),
    (dict(v=dict(dtype=_lib.GNS_F16)), "V[0]: must be f32"),
    (dict(master={}), "f32 weight takes no master"),
    (dict(w=dict(dtype=_lib.GNS_BF16), master=dict(dtype=_lib.GNS_BF16)), "master[0]: must be f32"),
    (dict(w=dict(dtype=_lib.GNS_BF16), master=dict(cols=16)), "master[0]"),
])
def test_adamw_refuses(lib, kw, msg):
    assert _adamw(lib, **kw) == _lib.GNS_ERR_INVALID
    assert msg in _lib.last_error()


def test_adamw_refuses_aliases(lib):
    w, o = _list(dict(ptr=1 << 20)), _list(dict(ptr=2 << 20))
    p = _lib.GnsAdamwParams(1e-3, 0.9, 0.99, 1e-8, 0.0, 1)
    assert lib.gns_adamw_step(w, o, o, _list(dict(ptr=3 << 20)), None, 1, ctypes.byref(p), None, None, None, None) == _lib.GNS_ERR_INVALID
    assert "alias" in _lib.last_error()


class _Fake:
    """A CPU tensor that says it lives on a GPU: describing it launches nothing."""

    def __init__(self, t):
        self.t = t

    is_cuda = True
    dtype = property(lambda s: s.t.dtype)
    shape = property(lambda s: s.t.shape)
    device = property(lambda s: s.t.device)
    data_ptr = lambda s: s.t.data_ptr()  # noqa: E731
    numel = lambda s: s.t.numel()  # noqa: E731
    stride = lambda s, d=None: s.t.stride() if d is None else s.t.stride(d)  # noqa: E731
    is_contiguous = lambda s: s.t.is_contiguous()  # noqa: E731
    permute = lambda s, o: _Fake(s.t.permute(o))  # noqa: E731


def _described(t):
    x = tensor_lists.TensorList([_Fake(t)]).array[0].x
    return x.count, x.rows, x.cols, x.ld, x.stride


@pytest.mark.parametrize("t,want", [
    (torch.empty(()), (1, 1, 1, 1, 1)),
    (torch.empty(5), (1, 1, 5, 5, 5)),
    (torch.empty(2, 3, 4, 5), (6, 4, 5, 5, 20)),
    (torch.empty(4, 6).t(), (1, 4, 6, 6, 24)),
    (torch.empty(2, 3, 4, 5).permute(0, 2, 3, 1), (6, 4, 5, 5, 20)),
    (torch.empty(4, 8)[:, :5], (1, 4, 5, 8, 0)),
    (torch.empty(3, 4, 8)[:, :, :5], (3, 4, 5, 8, 32)),
    (torch.empty(3, 4, 8)[:, 1:3], (3, 2, 8, 8, 32)),
    (torch.empty(2, 3, 4, 8)[..., :5], (6, 4, 5, 8, 32)),
    (torch.empty(0, 7), (1, 0, 7, 7, 0)),
])
def test_descriptions(t, want):
    got = _described(t)
    assert got[:3] == want[:3]
    if want[1] > 1:
        assert got[3] == want[3]
    if want[0] > 1:
        assert got[4] == want[4]


@pytest.mark.parametrize("t", [torch.empty(8)[::2], torch.empty(1, 6).expand(4, 6), torch.empty(6, 8)[:, :4].t(),
                               torch.empty(1).expand(9), torch.empty(2, 3, 4, 8)[:, :2, :3, :5]])
def test_descriptions_refused(t):
    with pytest.raises(ValueError, match="contiguous"):
        _described(t)


def test_python_refusals():
    with pytest.raises(ValueError, match="CUDA"):
        tensor_lists.tensor_list([torch.zeros(3)])
    with pytest.raises(ValueError, match="at least one"):
        tensor_lists.tensor_list([])
    with pytest.raises(TypeError, match="dtype"):
        tensor_lists.tensor_list([_Fake(torch.zeros(3, dtype=torch.float64))])
    a, b = (tensor_lists.TensorList([_Fake(torch.empty(*s))]) for s in ((4, 6), (6, 4)))
    with pytest.raises(ValueError, match="outs.0."):
        tensor_lists._same_layout("outs", a, b)
    # the same elements in another order in memory are not the same tensor
    c = tensor_lists.TensorList([_Fake(torch.empty(6, 4).t())])
    with pytest.raises(ValueError, match="order"):
        tensor_lists._same_layout("G", a, c)
    with pytest.raises(ValueError, match="norm_type"):
        tensor_lists._norm_code(1.0)
