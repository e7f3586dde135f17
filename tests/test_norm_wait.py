"""The wait in grad_norm's last block, by the library's self-test of it: no share comes, the limit is short, and
nothing faults or hangs (each wait of the self-test ends at its limit)."""
import ctypes
import math

import pytest

from matrix_orthogonalizing_optimizer_gb300 import _lib, build

torch = pytest.importorskip("torch")

LIMIT_US = 20000


def _run(nslots, early, late, norm_type=0):
    lib = _lib.load()
    ws = torch.full((max(nslots * 16, 256),), 255, dtype=torch.uint8, device="cuda")  # whatever was there before
    result = torch.zeros(6, device="cuda")
    out = torch.zeros(3, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rc = lib.gns_selftest_norm_wait(ws.data_ptr(), ws.numel(), nslots, early, late, norm_type, LIMIT_US, result.data_ptr(),
                                    out.data_ptr(), status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0, _lib.last_error()
    torch.cuda.synchronize()
    return result.tolist(), [t / 1000 for t in out.tolist()], int(status), ws


@pytest.mark.gpu
@pytest.mark.parametrize("norm_type", [0, 1])
@pytest.mark.parametrize("nslots,early,late", [(1, 0, 0), (1, 0, 1), (608, 0, 608), (608, 607, 1), (608, 300, 200), (1300, 0, 1300),
                                               (4000, 3999, 1), (4000, 1, 3000)])
def test_wait_runs_out(nslots, early, late, norm_type):
    result, us, status, ws = _run(nslots, early, late, norm_type)
    assert math.isnan(result[0]) and math.isnan(result[2])  # the late shares are not the second gathering's
    assert status & _lib.GNS_DEVST_TIMEOUT
    # one limit for all slots of a thread: 4000 slots are 16 for each of them
    assert all(LIMIT_US <= t < 1.5 * LIMIT_US for t in us[:2])
    assert result[4] == pytest.approx(1.0 if norm_type else math.sqrt(nslots), rel=1e-6)
    assert us[2] < LIMIT_US / 4
    assert not ws[: nslots * 16].any()  # ready for the next replay


@pytest.mark.gpu
@pytest.mark.parametrize("nslots", [1, 257, 608, 4000])
def test_no_wait_where_every_share_is_there(nslots):
    result, us, _, _ = _run(nslots, nslots, 0)
    assert result[0] == pytest.approx(math.sqrt(nslots), rel=1e-6) and us[0] < LIMIT_US / 4
    assert math.isnan(result[2])  # the shares were taken: the same number finds none
    assert result[4] == pytest.approx(math.sqrt(nslots), rel=1e-6)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("kw,code", [
    (dict(ws=None), _lib.GNS_ERR_INVALID), (dict(result=None), _lib.GNS_ERR_INVALID), (dict(nslots=0), _lib.GNS_ERR_INVALID),
    (dict(nslots=1 << 17), _lib.GNS_ERR_INVALID), (dict(early=5, late=6), _lib.GNS_ERR_INVALID), (dict(late=-1), _lib.GNS_ERR_INVALID),
    (dict(norm_type=2), _lib.GNS_ERR_INVALID), (dict(limit_us=0), _lib.GNS_ERR_INVALID), (dict(limit_us=1000001), _lib.GNS_ERR_INVALID),
    (dict(result=ctypes.c_void_p(2)), _lib.GNS_ERR_INVALID), (dict(out=ctypes.c_void_p(4)), _lib.GNS_ERR_INVALID),
    (dict(ws=ctypes.c_void_p(128)), _lib.GNS_ERR_WORKSPACE), (dict(ws_bytes=159), _lib.GNS_ERR_WORKSPACE)])
def test_refusals(lib, kw, code):
    a = dict(ws=ctypes.c_void_p(1 << 20), ws_bytes=160, nslots=10, early=0, late=0, norm_type=0, limit_us=10,
             result=ctypes.c_void_p(1 << 21), out=None)
    a.update(kw)
    assert lib.gns_selftest_norm_wait(a["ws"], a["ws_bytes"], a["nslots"], a["early"], a["late"], a["norm_type"], a["limit_us"],
                                      a["result"], a["out"], None, None) == code
