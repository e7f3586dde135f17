"""masters of adamw_step: None is the one way to say that a weight has none."""
import pytest

torch = pytest.importorskip("torch")
from fake_device import Memory, world  # noqa: E402, F401
from matrix_orthogonalizing_optimizer_gb300 import tensor_lists  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def _step(masters, shapes=((8, 8), (3, 5))):
    cuda = torch.device("cuda", 0)
    roles = [[Memory(s, dt, cuda) for s in shapes] for dt in (BF, BF, F32, F32)]
    ms = [None if s is None else Memory(s, F32, cuda) for s in masters]
    tensor_lists.adamw_step(*roles, lr=0.1, masters=ms, status=Memory(1, torch.int32, cuda))


@pytest.mark.parametrize("masters", [[(0,), (3, 5)], [(0, 8), None], [(8, 8), (0,)], [None, (3, 0)]])
def test_an_empty_tensor_is_not_a_missing_master(world, masters):
    with pytest.raises(ValueError, match="masters"):
        _step(masters)
    assert not world["library"].calls


@pytest.mark.parametrize("masters", [[(8, 8), (3, 5)], [None, (3, 5)], [(8, 8), None], [None, None]])
def test_none_is_a_missing_master(world, masters):
    _step(masters)
    assert world["library"].calls == [("gns_adamw_step", 0)]


def test_empty_weights_have_empty_masters(world):
    _step([(0,), (3, 5), None], shapes=((0,), (3, 5), (2, 0)))
    assert world["library"].calls == [("gns_adamw_step", 0)]
