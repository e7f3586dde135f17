"""The launch grid bounds a batch that is brought into 4 bits; nothing is launched here."""
import pytest

torch = pytest.importorskip("torch")
from matrix_orthogonalizing_optimizer_gb300 import _lib  # noqa: E402
from test_fp4_host import R, batch, held, lib, refused  # noqa: E402, F401


@pytest.mark.parametrize("fmt", [_lib.GNS_NVFP4, _lib.GNS_MXFP4])
@pytest.mark.parametrize("rows", [True, False])
def test_more_tiles_than_a_grid_has_are_refused(lib, fmt, rows):  # noqa: F811
    shape = (65535, 4194240) if rows else (4194240, 65535)
    x = batch(65535, 65535, 4194240, ptr=1 << 26)
    q = held(65535, *shape, fmt=fmt, scale_stride=1 << 60)
    refused(lib.gns_fp4_quantize(R(x), _lib.GNS_BF16, R(q) if rows else None, None if rows else R(q), None, None, None), "2^31 - 1")
