"""Layouts of the tensors of a list: a dimension of size 1 has a stride of no meaning, so it changes neither
the order in memory nor whether the rows lie evenly."""
import pytest

torch = pytest.importorskip("torch")
from fake_device import OnDevice  # noqa: E402
from matrix_orthogonalizing_optimizer_gb300 import tensor_lists  # noqa: E402


def _list(t):
    return tensor_lists.TensorList([OnDevice(t)])


def _described(t):
    x = _list(t).array[0].x
    return x.count, x.rows, x.cols, x.ld, x.stride


def _strided(shape, steps):
    size = 1 + sum((n - 1) * s for n, s in zip(shape, steps))
    return torch.as_strided(torch.empty(size), shape, steps)


def _elements(t):
    """Offsets of a description's elements, in its order."""
    count, rows, cols, ld, stride = _described(t)
    return [b * stride + i * ld + j for b in range(count) for i in range(rows) for j in range(cols)]


SAME_ORDER = [
    ((6, 1, 4), [(1, 6, 6), (1, 1, 6), (1, 99, 6), (1, 0, 6)]),
    ((1, 6, 4), [(24, 1, 6), (1, 1, 6), (6, 1, 6)]),
    ((6, 4, 1), [(1, 6, 24), (1, 6, 1), (1, 6, 6)]),
    ((3, 1, 5, 1, 2), [(1, 1, 6, 1, 3), (1, 30, 6, 3, 3), (1, 3, 6, 6, 3)]),
]


@pytest.mark.parametrize("shape,strides", SAME_ORDER)
def test_size_one_does_not_change_the_order_in_memory(shape, strides):
    lists = [_list(_strided(shape, s)) for s in strides]
    for l in lists[1:]:
        tensor_lists._same_layout("G", lists[0], l)
    assert len({_described(_strided(shape, s)) for s in strides}) == 1
    n = torch.Size(shape).numel()
    for s in strides:
        assert _elements(_strided(shape, s)) == list(range(n))


@pytest.mark.parametrize("shape,a,b", [((6, 1, 4), (1, 6, 6), (4, 4, 1)), ((3, 1, 5, 2), (1, 1, 6, 3), (1, 1, 3, 15)),
                                       ((4, 1, 4), (1, 4, 4), (4, 4, 1))])
def test_other_orders_in_memory_are_still_told_apart(shape, a, b):
    with pytest.raises(ValueError, match="order"):
        tensor_lists._same_layout("G", _list(_strided(shape, a)), _list(_strided(shape, b)))


@pytest.mark.parametrize("t,want", [
    (torch.empty(2, 9, 4, 8)[:, :1, :, :5], (2, 4, 5, 8, 288)),
    (torch.empty(2, 3, 9, 4, 8)[:, :, :1, :, :5], (6, 4, 5, 8, 288)),
    (torch.empty(9, 2, 3, 4, 8)[:1, :, :, :, :5], (6, 4, 5, 8, 32)),
    (torch.empty(7, 9, 8)[:, :1, :5], (7, 1, 5, 5, 72)),
    (torch.empty(5, 9, 9, 8)[:, :1, :1, :5], (5, 1, 5, 8, 648)),
    (torch.empty(4, 8)[:, :5].unsqueeze(2), (4, 5, 1, 1, 8)),
    (torch.empty(2, 1, 4, 8)[..., :5], (2, 4, 5, 8, 32)),
])
def test_size_one_does_not_keep_rows_from_lying_evenly(t, want):
    got = _described(t)
    assert got[:3] == want[:3] and (got[4] == want[4] or want[0] == 1) and (got[3] == want[3] or want[1] == 1)
    offsets = [int(x) - t.storage_offset() for x in
               torch.as_strided(torch.arange(t.untyped_storage().nbytes() // 4), t.shape, t.stride(), t.storage_offset()).reshape(-1)]
    assert _elements(t) == offsets
    # whole, with the same shape: the same matrices and rows, as the library compares them
    assert _described(torch.empty(t.shape))[:3] == got[:3]


@pytest.mark.parametrize("t", [torch.empty(2, 3, 4, 8)[:, :2, :3, :5], torch.empty(1, 6).expand(4, 6), torch.empty(8)[::2],
                               torch.empty(3, 1, 8)[..., ::2], torch.empty(1, 5, 1).expand(3, 5, 4), torch.empty(6, 1, 8)[..., :4].transpose(0, 2)])
def test_refused_as_before(t):
    with pytest.raises(ValueError, match="contiguous"):
        _list(t)


@pytest.mark.gpu
def test_calls_on_such_layouts():
    """Against the same calls on whole copies, bit by bit (every element's arithmetic is its own)."""
    import matrix_orthogonalizing_optimizer_gb300 as gns

    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def filled(shape, steps):
        size = 1 + sum((n - 1) * s for n, s in zip(shape, steps))
        return torch.as_strided(torch.randn(size, generator=g, device="cuda"), shape, steps)

    layouts = [((60, 1, 44), [(1, 60, 60), (1, 1, 60), (1, 99, 60), (1, 0, 60)]),
               ((2, 1, 40, 50), [(28800, 3200, 64, 1), (28800, 1, 64, 1), (3000, 7, 56, 1), (2000, 2000, 50, 1)])]
    roles = [[filled(shape, strides[r]) for shape, strides in layouts] for r in range(4)]
    for v in roles[3]:
        v.abs_()
    whole = [[t.contiguous().clone() for t in l] for l in roles]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gns.adamw_step(*roles, lr=1e-2, step=3, status=st)
    gns.adamw_step(*whole, lr=1e-2, step=3, status=st)
    for a, b in zip(roles, whole):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    r = gns.clip_grads(roles[1], 1.0, status=st)
    want = torch.sqrt(sum((t.double() ** 2).sum() for t in whole[1]))
    assert abs(float(r[0]) - float(want)) <= 2.0 ** -18 * float(want)
    for x, y in zip(roles[1], whole[1]):
        assert torch.equal(x, y * r[1])
    assert int(st) == 0
