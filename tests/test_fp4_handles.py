"""An Fp4Matrix describes the memory that it was made of, and holds on to it."""
import gc
import weakref

import pytest

torch = pytest.importorskip("torch")
from fake_device import Memory, world  # noqa: E402, F401
from matrix_orthogonalizing_optimizer_gb300 import fp4  # noqa: E402


@pytest.fixture
def q(world):  # noqa: F811
    def mem(shape, dtype=torch.uint8):
        return Memory(shape, dtype, torch.device("cuda", 0))

    return fp4.Fp4Matrix(mem((2, 100, 80)), mem((2, 1, 3, 512)), mem((2,), torch.float32), 160)


@pytest.mark.parametrize("name", ["codes", "scales", "tensor_scale", "fmt", "shape", "device", "index", "_struct", "_ref"])
def test_nothing_of_it_can_be_put_in_another_place(q, name):
    before = getattr(q, name)
    with pytest.raises(AttributeError, match="Fp4Matrix"):
        setattr(q, name, before)
    with pytest.raises(AttributeError, match="Fp4Matrix"):
        delattr(q, name)
    assert getattr(q, name) is before
    q.layer = 3  # what a user notes on it stays the user's
    assert q.layer == 3


def test_it_keeps_its_memory(q):
    alive = [weakref.ref(t) for t in (q.codes, q.scales, q.tensor_scale)]
    gc.collect()
    assert all(r() is not None for r in alive)
    assert q._struct.codes.ptr == q.codes.data_ptr() and q._struct.scales == q.scales.data_ptr()
