"""adamw_step's hyper-parameters are doubles, its arithmetic fp32: what fp32 does not hold is refused, and
at the edge of what it holds an element without gradient and state stays what it is."""
import ctypes

import pytest

from matrix_orthogonalizing_optimizer_gb300 import _lib, build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _refused(lib, **kw):
    """The call's code; nothing is launched where it is refused (a scale that is not aligned is refused in
    any case, after the parameters, so that no call gets further)."""
    lists = []
    for k in range(4):
        t = (_lib.GnsTensor * 1)()
        t[0].x.ptr, t[0].x.count, t[0].x.rows, t[0].x.cols, t[0].x.ld, t[0].x.stride = (k + 1) << 20, 1, 1, 64, 64, 64
        t[0].dtype = _lib.GNS_F32
        lists.append(t)
    p = _lib.GnsAdamwParams(kw.get("lr", 1e-3), kw.get("beta1", 0.9), 0.99, kw.get("eps", 1e-8), kw.get("weight_decay", 0.0), 1)
    return lib.gns_adamw_step(*lists, None, 1, ctypes.byref(p), ctypes.c_void_p(2), None, None, None), _lib.last_error()


@pytest.mark.parametrize("kw,msg", [
    (dict(eps=1e-40), "eps"),    # its reciprocal is not finite in fp32
    (dict(eps=2.0 ** -128), "eps"),
    (dict(eps=1e-46), "eps"),    # zero in fp32
    (dict(eps=1e300), "eps"),    # infinite in fp32
    (dict(lr=1e39), "lr"),
    (dict(lr=-1e39), "lr"),
    (dict(lr=5e37), "lr"),       # lr / (1 - beta1), the first step's size
    (dict(lr=1e30, weight_decay=1e10), "weight_decay"),
])
def test_refused(lib, kw, msg):
    code, error = _refused(lib, **kw)
    assert code == _lib.GNS_ERR_INVALID
    assert msg in error and "fp32" in error


@pytest.mark.parametrize("kw", [dict(eps=2.0 ** -128 + 2.0 ** -149), dict(eps=1e-30), dict(eps=1e30), dict(lr=3e37),
                                dict(lr=5e37, beta1=0.0), dict(lr=-1e-3), dict(lr=1e30, weight_decay=1e8)])
def test_not_refused(lib, kw):
    """The parameters pass: what is refused is the scale behind them."""
    code, error = _refused(lib, **kw)
    assert code == _lib.GNS_ERR_INVALID and "grad_scale" in error


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("kw", [dict(eps=2.0 ** -128 + 2.0 ** -149), dict(eps=1e-38), dict(eps=1e-30), dict(lr=3e37)])
def test_elements_without_gradient_and_state_stay(dtype, kw):
    import matrix_orthogonalizing_optimizer_gb300 as gns

    w = torch.linspace(-2.0, 2.0, 4101, device="cuda").to(dtype)
    before = w.clone()
    g, m, v = (torch.zeros(4101, device="cuda") for _ in range(3))
    for count in (None, torch.ones(1, dtype=torch.int32, device="cuda")):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        gns.adamw_step([w], [g], [m], [v], **{"lr": 1e-2, "weight_decay": 0.0, **kw}, step_count=count, status=st)
        assert int(st) == 0
        assert torch.equal(w, before) and not m.any() and not v.any()
