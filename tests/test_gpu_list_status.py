"""The status word of adamw_step at the edge of each weight type: what counts as a non-finite weight is
what is stored."""
import pytest

torch = pytest.importorskip("torch")
gns = pytest.importorskip("matrix_orthogonalizing_optimizer_gb300")

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
# factors that take a type's largest value past, and not past, half a step above it
OVER = {F16: 1.003, BF: 1.003, F32: 1.5}
UNDER = {F16: 1.0002, BF: 1.001, F32: 0.999}


def _layouts(dtype):
    """One tensor of each way in which a kernel may take an element: in a whole vector, in the edge behind
    the last one, in single elements (no alignment), in the last vector of a row with a pitch."""
    yield "vector", torch.zeros(4096, dtype=dtype, device="cuda"), 1234
    yield "edge", torch.zeros(4101, dtype=dtype, device="cuda"), 4100
    yield "single", torch.zeros(1030, dtype=dtype, device="cuda")[1:1027], 700
    yield "row", torch.zeros(7, 24, dtype=dtype, device="cuda")[:, :21], 3 * 21 + 20
    yield "last row", torch.zeros(7, 24, dtype=dtype, device="cuda")[:, :21], 6 * 21 + 20


def _decay(w, at, value, factor, master):
    """A step without gradients, which only multiplies the weights; the status."""
    w[tuple(int(i) for i in torch.unravel_index(torch.tensor(at), w.shape))] = value
    g = torch.zeros(w.shape, dtype=w.dtype, device="cuda")
    m, v = (torch.zeros(w.shape, dtype=F32, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    masters = [w.float()] if master else None
    gns.adamw_step([w], [g], [m], [v], lr=1.0, weight_decay=1.0 - factor, masters=masters, status=st)
    return int(st), masters


@pytest.mark.parametrize("dtype,master", [(F16, False), (F16, True), (BF, False), (BF, True), (F32, False)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_weight_that_is_stored_as_infinity_is_reported(dtype, master, sign):
    value = sign * torch.finfo(dtype).max
    for name, w, at in _layouts(dtype):
        st, masters = _decay(w, at, value, OVER[dtype], master)
        assert int(torch.isinf(w).sum()) == 1, name
        assert st == 1, name
        if master:  # the master holds the value still, so that no later step would see it
            assert bool(torch.isfinite(masters[0]).all()), name


@pytest.mark.parametrize("dtype,master", [(F16, False), (F16, True), (BF, False), (BF, True), (F32, False)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_largest_weight_is_not_reported(dtype, master, sign):
    value = sign * torch.finfo(dtype).max
    for name, w, at in _layouts(dtype):
        st, _ = _decay(w, at, value, UNDER[dtype], master)
        assert bool(torch.isfinite(w).all()) and st == 0, name
        assert float(w.double().abs().max()) >= 0.99 * abs(value), name


@pytest.mark.parametrize("dtype,master", [(F16, False), (F16, True), (BF, False), (BF, True), (F32, False)])
def test_weight_that_becomes_nan_is_reported(dtype, master):
    for name, w, at in _layouts(dtype):
        g = torch.zeros(w.shape, dtype=F32, device="cuda")
        g.view(-1)[at] = float("nan")
        m, v = (torch.zeros(w.shape, dtype=F32, device="cuda") for _ in range(2))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        gns.adamw_step([w], [g], [m], [v], lr=1e-2, masters=[w.float()] if master else None, status=st)
        assert int(st) == 1 and int(torch.isnan(w).sum()) == 1, name
