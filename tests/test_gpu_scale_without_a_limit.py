"""Without a maximum (max_norm infinite) nothing is clipped: the scale is 1 whatever the norm is, a NaN or an
infinity among the gradients included, and the gradients stay as they are. The status word and the norm tell."""
import math

import pytest

torch = pytest.importorskip("torch")
gns = pytest.importorskip("matrix_orthogonalizing_optimizer_gb300")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [100, 400003])  # a short list, and one that takes two launches
@pytest.mark.parametrize("norm_type", [2.0, math.inf])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_scale_is_one(n, norm_type, value):
    t = torch.linspace(-1.0, 1.0, n, device="cuda")
    t[n // 2] = value
    before = t.clone()
    out = torch.zeros_like(t)

    def check(r, status):
        assert int(status) == 1
        assert float(r[1]) == 1.0
        assert math.isnan(float(r[0])) if math.isnan(value) else float(r[0]) == math.inf

    for call in (lambda st: gns.grad_norm([t], norm_type=norm_type, status=st),
                 lambda st: gns.grad_norm([t], max_norm=math.inf, norm_type=norm_type, status=st),
                 lambda st: gns.clip_grads([t], math.inf, norm_type=norm_type, status=st),
                 lambda st: gns.clip_grads([t], math.inf, norm_type=norm_type, outs=[out], status=st)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        check(call(status), status)
        assert torch.equal(t.view(torch.int32), before.view(torch.int32))
    assert torch.equal(torch.nan_to_num(out, 7.0, 8.0, 9.0), torch.nan_to_num(before, 7.0, 8.0, 9.0))
