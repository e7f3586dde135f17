"""Batches of single rows: a row has no stride of its own, and is described with the smallest pitch that keeps rows aligned, so
that rows which lie next to one another on 16-byte boundaries make a batch."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from fake_device import OnDevice  # noqa: E402
from matrix_orthogonalizing_optimizer_gb300 import NsParams, _lib, api, build  # noqa: E402


class Batch(OnDevice):
    def dim(self):
        return self.t.dim()

    def unsqueeze(self, d):
        return Batch(self.t.unsqueeze(d))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("dtype,code,unit", [(torch.float32, _lib.GNS_F32, 4), (torch.bfloat16, _lib.GNS_BF16, 8), (torch.float16, _lib.GNS_F16, 8)])
@pytest.mark.parametrize("cols", [1, 3, 4, 5, 8, 12, 20, 24, 100])
@pytest.mark.parametrize("count", [1, 2, 7])
def test_rows_next_to_one_another(lib, count, cols, dtype, code, unit):
    pitch = -(-cols // unit) * unit
    t = torch.empty(count, 1, pitch, dtype=dtype)[..., :cols]
    b = api.batch_of(Batch(t))
    assert (b.count, b.rows, b.cols, b.ld, b.stride) == (count, 1, cols, pitch, pitch)
    ns = NsParams().c_struct()
    assert lib.gns_workspace_size(_lib.GNS_OP_GRAM_NS, ctypes.byref(b), 1, code, ctypes.byref(ns), None) > 0, _lib.last_error()
    # further apart, and one matrix of one row
    wide = torch.empty(count, 3, pitch, dtype=dtype)[:, :1, :cols]
    b = api.batch_of(Batch(wide))
    assert (b.ld, b.stride) == (pitch, 3 * pitch if count > 1 else pitch)
    b = api.batch_of(Batch(t[0]))
    assert (b.count, b.rows, b.cols, b.ld, b.stride) == (1, 1, cols, pitch, pitch)
    # rows that overlap are refused
    if count > 1 and pitch > unit:
        close = torch.empty(count * pitch, dtype=dtype).as_strided((count, 1, cols), (pitch - unit, pitch, 1))
        b = api.batch_of(Batch(close))
        assert lib.gns_workspace_size(_lib.GNS_OP_GRAM_NS, ctypes.byref(b), 1, code, ctypes.byref(ns), None) == 0
        assert "stride" in _lib.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [4, 12, 20, 100])
def test_batches_of_single_fp32_rows(cols):
    import matrix_orthogonalizing_optimizer_gb300 as gns
    x = torch.randn(5, 1, cols, generator=torch.Generator().manual_seed(cols)).cuda()
    got = gns.gram_ns_batched(x)[0]
    for i in range(5):
        assert torch.equal(got[i], gns.gram_ns_batched(x[i])[0])
    # NorMuon's second moments are such rows
    w, g, m = (torch.randn(5, cols, 128, device="cuda").bfloat16() for _ in range(3))
    v = torch.zeros(5, 1, cols, device="cuda")
    ones = [(w[i].clone(), g[i].clone(), m[i].clone(), v[i].clone()) for i in range(5)]
    p = gns.MuonParams(lr=0.1, flavor="normuon")
    gns.muon_step(w, g, m, V=v, params=p)
    for i, (wi, gi, mi, vi) in enumerate(ones):
        gns.muon_step(wi, gi, mi, V=vi, params=p)
        torch.testing.assert_close(v[i], vi, rtol=1e-5, atol=0)
        torch.testing.assert_close(w[i], wi, rtol=2.0**-7, atol=0)
