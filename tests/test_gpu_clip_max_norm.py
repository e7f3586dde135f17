"""Clipping by the largest magnitude, in each of the kernels that clip, and the norm's precision over
runs long enough to need it.

The largest magnitude is one of the values, so the norm is compared exactly. The scale max_norm / (N +
eps) is one f32 sum and one quotient, the clipped values one product rounded once: those are compared
bit by bit with the same f32 operations done by torch on the device's own scale."""
import math

import pytest

torch = pytest.importorskip("torch")
gns = pytest.importorskip("matrix_orthogonalizing_optimizer_gb300")

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def _bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == F32 else torch.int16)


def _lists(kind, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(17)

    def one(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    if kind == "short":  # one launch of one cluster
        return [one(n) for n in (1, 7, 64, 1001, 40000)]
    if kind == "short_rows":
        return [one(5, 24)[:, :21], one(3, 9, 16)[:, :8, :11], one(33, 72)[:, :65]]
    if kind == "long":
        return [one(700001), one(1111, 1003), one(5)]
    if kind == "long_rows":
        return [one(301, 2056)[:, :2051], one(3, 200, 1016)[:, :199, :1011]]
    if kind == "mixed":
        return [one(300001), one(64, 2056)[:, :2051], one(1000).float(), one(400, 512).to(BF), one(99).to(F16)]
    if kind == "many":  # several launches of each layout
        return [one(37) for _ in range(1700)] + [one(3, 8)[:, :5] for _ in range(700)]
    raise ValueError(kind)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("kind", ["short", "short_rows", "long", "long_rows", "mixed", "many"])
@pytest.mark.parametrize("mode", ["in_place", "outs"])
def test_clip_by_the_largest_magnitude(kind, dtype, mode):
    ts = _lists(kind, dtype)
    ts[-1][..., -1] = 50.0  # the largest is the last element of the list (and of a row)
    before = [t.clone() for t in ts]
    largest = max(float(t.double().abs().max()) for t in ts)
    assert largest == 50.0
    outs = [torch.zeros_like(t) for t in ts] if mode == "outs" else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = gns.clip_grads(ts, 5.0, norm_type=math.inf, outs=outs, status=st)
    assert int(st) == 0
    assert float(r[0]) == largest
    assert abs(float(r[1]) - 5.0 / (largest + 1e-6)) <= 3 * U * float(r[1])  # eps, the sum, the quotient
    for t, b, o in zip(ts, before, outs or ts):
        assert torch.equal(_bits(o), _bits((b.float() * r[1]).to(b.dtype)))
        if outs:
            assert torch.equal(_bits(t), _bits(b))


@pytest.mark.parametrize("kind", ["short", "short_rows", "long", "long_rows"])
@pytest.mark.parametrize("value,norm,scale", [(math.inf, math.inf, 0.0), (-math.inf, math.inf, 0.0), (math.nan, math.nan, math.nan)])
def test_clip_non_finite_by_the_largest_magnitude(kind, value, norm, scale):
    ts = _lists(kind, BF)
    ts[1][..., -1] = value
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = gns.clip_grads(ts, 1.0, norm_type=math.inf, status=st).tolist()
    assert int(st) == 1
    for got, want in zip(r, (norm, scale)):
        assert got == want or (math.isnan(got) and math.isnan(want))
    assert bool(torch.isnan(ts[1][..., -1]).all())
    if scale == 0.0:
        assert not ts[0].any()
    else:
        assert bool(torch.isnan(ts[0]).all())


@pytest.mark.parametrize("kind", ["short", "long", "long_rows"])
def test_clip_below_the_largest_magnitude_leaves_gradients_alone(kind):
    ts = _lists(kind, F16)
    before = [t.clone() for t in ts]
    r = gns.clip_grads(ts, 100.0, norm_type=math.inf)
    assert float(r[1]) == 1.0
    for t, b in zip(ts, before):
        assert torch.equal(_bits(t), _bits(b))


def test_norm_keeps_what_long_runs_of_small_squares_add():
    """Each block of the norm takes a run of 128 chunks here. The first chunk of every run holds ones and the
    others a value whose squares, 64 of a thread's chunk, come to just under half a step of the first
    chunk's 64 in f32: a plain f32 sum of the runs loses every one of them, 127 times 2^-24 of the sum, that
    is 3.8e-6 of the norm.

    Bound: the squares (16 bits) and a thread's sums of 64 equal ones are exact, the two-sum holds what its
    sum loses; then come the sum of both parts (1 unit of U = 2^-24), a warp's 5 and a block's 8 sums, a
    thread's 3 slots, 13 sums again, the root and the product behind it (1 each): 30 of the sum at most,
    so 15 of the norm, and 2: 17 U = 1.0e-6."""
    blocks = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    run, chunk = 128, 256 * 8 * 8  # chunks of a block, elements of a chunk
    small = 255.0 * 2.0 ** -20  # its square: 0.992 * 2^-24
    t = torch.full((blocks, run, chunk), small, dtype=BF, device="cuda")
    assert float(t[0, 0, 0]) == small
    t[:, 0] = 1.0
    want = math.sqrt(blocks * chunk * (1.0 + (run - 1) * small * small))
    got = float(gns.grad_norm([t])[0])
    assert abs(got - want) <= 17 * U * want
