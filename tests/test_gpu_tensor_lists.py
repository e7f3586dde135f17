"""grad_norm, clip_grads and adamw_step on the GPU against plain implementations in 64 bits, at the
layouts, sizes and values where such kernels go wrong.

Tolerances. A norm adds at most 64 squares in f32 before it goes on in f64, so its sum is within
64 * 2^-24 of the exact one, its root within half of that, and one more rounding to f32 follows:
2^-18 holds with room. A clipped gradient is one f32 product rounded once, so it is compared bit by
bit. AdamW's bounds are counted from its formula in `adamw_bounds`.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
gns = pytest.importorskip("matrix_orthogonalizing_optimizer_gb300")

pytestmark = pytest.mark.gpu

NORM_TOL = 2.0 ** -18
U = 2.0 ** -24  # half a unit in the last place of f32
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed), device="cuda") * scale).to(dtype)


def _make(kind, dtype, seed, scale=1.0):
    """A list of tensors of one layout."""
    def flat(n, offset=0):
        buf = _randn((n + offset + 8,), dtype, seed + n, scale)
        return buf[offset:offset + n]

    if kind == "sizes":
        return [flat(n) for n in (1, 2, 7, 8, 9, 15, 255, 2047, 2048, 2049, 8191, 8192, 8193, 70001)]
    if kind == "offsets":  # every alignment of the first element
        return [flat(4099, o) for o in range(9)] + [flat(n, 5) for n in (1, 2, 3, 4, 11)]
    if kind == "many":  # more tensors than one launch holds
        r = np.random.RandomState(12)  # the same sizes for every role
        sizes = r.randint(1, 40, 1100)
        buf = _randn((int(sizes.sum()),), dtype, seed, scale)
        return list(torch.split(buf, sizes.tolist()))
    if kind == "pitched":  # rows with a pitch: 16-byte, 32-byte and no alignment; whole tiles and ragged ones
        return [_randn((3, 17, 64), dtype, seed, scale)[:, :, :53], _randn((2, 5, 48), dtype, seed + 1, scale)[:, :, :41],
                _randn((4, 9, 13), dtype, seed + 2, scale)[:, 1:7, 2:11], _randn((301, 9), dtype, seed + 3, scale)[:, :1],
                _randn((5, 20011), dtype, seed + 4, scale)[:, 1:20009], _randn((6, 1, 24), dtype, seed + 5, scale)[:, :, :20],
                _randn((7, 24), dtype, seed + 6, scale)[:1, 1:9]]
    if kind == "pitched_stacks":  # rows on 16 bytes, matrices that do not follow at the rows' pitch
        return [_randn((3, 20, 64), dtype, seed, scale)[:, :17, :53], _randn((5, 9, 32), dtype, seed + 1, scale)[:, :8, :],
                _randn((2, 3, 4112), dtype, seed + 2, scale)[:, :2, :4100], _randn((4, 2, 2064), dtype, seed + 3, scale)[:, :1, :2057]]
    if kind == "many_pitched":
        return [_randn((3, 5), dtype, seed + i, scale)[:, :4] for i in range(520)]
    if kind == "shapes":  # scalars, empty tensors, more dimensions, other orders in memory
        return [_randn((), dtype, seed, scale), _randn((0,), dtype, seed, scale), _randn((3, 0, 5), dtype, seed, scale),
                _randn((2, 3, 4, 5), dtype, seed + 1, scale), _randn((33, 65), dtype, seed + 2, scale).t(),
                _randn((2, 8, 9, 10), dtype, seed + 3, scale).permute(0, 2, 3, 1), _randn((1, 1, 77), dtype, seed + 4, scale)]
    if kind == "large":
        return [_randn((3, 1111, 1003), dtype, seed, scale), _randn((5000000,), dtype, seed + 1, scale), _randn((999,), dtype, seed + 2, scale)]
    raise ValueError(kind)


KINDS = ["sizes", "offsets", "many", "pitched", "pitched_stacks", "many_pitched", "shapes", "large"]


def _norm64(ts):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in ts))


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------ norm

@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("kind", KINDS)
def test_norm(kind, dtype):
    ts = _make(kind, dtype, 1)
    r = gns.grad_norm(ts)
    want = _norm64(ts)
    assert abs(float(r[0]) - want) <= NORM_TOL * want
    assert float(r[1]) == 1.0
    assert torch.equal(r, gns.grad_norm(ts))  # a fixed order: the same bits again
    inf = gns.grad_norm(ts, norm_type=math.inf)
    assert float(inf[0]) == max(float(t.double().abs().max()) for t in ts if t.numel())


def test_norm_of_mixed_types_and_layouts():
    ts = _make("sizes", BF, 3) + _make("pitched", F16, 4) + _make("offsets", F32, 5) + _make("shapes", BF, 6)
    r = gns.grad_norm(gns.tensor_list(ts), max_norm=2.0)
    want = _norm64(ts)
    assert abs(float(r[0]) - want) <= NORM_TOL * want
    scale = 2.0 / (want + 1e-6)
    assert abs(float(r[1]) - scale) <= NORM_TOL * scale


@pytest.mark.parametrize("dtype,value", [(F32, 1e30), (F32, 3e38), (BF, 1e38), (F32, 1e-30), (F32, 1e-44), (BF, 1e-35),
                                         (F16, 65504.0), (F16, 6e-8), (F32, 1e-19), (F32, 1.9e19)])
@pytest.mark.parametrize("n", [1, 9, 100003])
def test_norm_of_extreme_values(dtype, value, n):
    """Squares that leave f32's range do not spoil the norm."""
    t = torch.full((n,), value, dtype=dtype, device="cuda")
    want = float(t[0].double()) * math.sqrt(n)
    st = _status()
    r = gns.grad_norm([t], status=st)
    if want > 3.4e38:  # the norm itself does not fit
        assert float(r[0]) == math.inf and int(st) == 1
    else:
        assert int(st) == 0
        # subnormal results have fewer bits: half of the smallest subnormal beside the relative part
        assert abs(float(r[0]) - want) <= NORM_TOL * want + 2.0 ** -150


def test_norm_of_values_far_apart():
    ts = [torch.full((50,), 1e-30, device="cuda"), torch.full((70000,), 1e25, device="cuda"), torch.zeros(5, device="cuda"),
          torch.full((3,), 1.0, dtype=BF, device="cuda")]
    want = _norm64(ts)
    assert abs(float(gns.grad_norm(ts)[0]) - want) <= NORM_TOL * want
    small = [torch.full((50,), 1e-30, device="cuda"), torch.full((7,), 1e-12, device="cuda"), torch.zeros(50000, device="cuda")]
    want = _norm64(small)
    assert abs(float(gns.grad_norm(small)[0]) - want) <= NORM_TOL * want


def test_norm_of_zeros():
    r = gns.grad_norm([torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")], max_norm=1.0)
    assert r.tolist() == [0.0, 1.0]
    r = gns.grad_norm([torch.zeros(0, device="cuda")], max_norm=1.0)
    assert r.tolist() == [0.0, 1.0]
    r = gns.grad_norm([torch.full((5,), -0.0, device="cuda")])
    assert r.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("norm_type", [2.0, math.inf])
def test_norm_of_non_finite_values(dtype, norm_type):
    for values, norm, scale in (([math.inf], math.inf, 0.0), ([-math.inf, 1.0], math.inf, 0.0),
                                ([math.nan], math.nan, math.nan), ([math.inf, math.nan], math.nan, math.nan)):
        ts = _make("sizes", dtype, 2)
        for i, v in enumerate(values):
            ts[-1 - i][3 + 4000 * i if i == 0 else 0] = v
        st = _status()
        r = gns.grad_norm(ts, max_norm=1.0, norm_type=norm_type, status=st)
        got = r.tolist()
        assert int(st) == 1
        assert got[0] == norm or (math.isnan(norm) and math.isnan(got[0]))
        assert got[1] == scale or (math.isnan(scale) and math.isnan(got[1]))
        with pytest.raises(gns.GnsDeviceError, match="non-finite"):
            gns.grad_norm(ts, norm_type=norm_type)


@pytest.mark.parametrize("max_norm,eps", [(0.0, 1e-6), (1.0, 0.0), (1e-20, 1e-6), (5.0, 1e-6), (1e9, 1e-6), (math.inf, 1e-6)])
def test_scale(max_norm, eps):
    t = torch.full((400,), 0.25, device="cuda")  # norm 5
    got = float(gns.grad_norm([t], max_norm=max_norm, eps=eps)[1])
    want = min(1.0, max_norm / (5.0 + eps))
    assert abs(got - want) <= NORM_TOL * want


def test_norm_of_a_tensor_beyond_32_bits():
    n = 2 ** 31 + 4099
    t = torch.zeros(n, dtype=BF, device="cuda")
    t[2 ** 31 - 3:2 ** 31 + 5] = 2.0
    t[-1] = 3.0
    want = math.sqrt(8 * 4 + 9)
    assert abs(float(gns.grad_norm([t])[0]) - want) <= NORM_TOL * want
    r = gns.clip_grads([t], want / 2, eps=0.0)
    assert t[-1].item() == pytest.approx(1.5, rel=2.0 ** -8) and t[2 ** 31 + 4].item() == pytest.approx(1.0, rel=2.0 ** -8)
    assert float(r[1]) == pytest.approx(0.5, rel=2.0 ** -17)


def test_pitched_rows_beyond_32_bits():
    t = torch.zeros(70001, 40008, dtype=BF, device="cuda")[:, :40003]
    t[-1, -3:] = 2.0
    t[53700, 5] = 3.0  # near element 2^31
    t[0, 0] = 1.0
    want = math.sqrt(3 * 4 + 9 + 1)
    assert abs(float(gns.grad_norm([t])[0]) - want) <= NORM_TOL * want
    whole = torch.as_strided(t, (70001, 40008), (40008, 1))
    whole[:, 40003:] = 7.0  # beside the rows
    r = gns.clip_grads([t], want / 2, eps=0.0)
    assert abs(float(r[0]) - want) <= NORM_TOL * want
    half = torch.tensor(2.0, device="cuda").mul(r[1]).to(BF)
    assert t[-1, -3:].tolist() == [half.item()] * 3 and float(t[53700, 5]) == float((3.0 * r[1]).to(BF))
    assert bool((whole[:, 40003:] == 7.0).all())


# ------------------------------------------------------------------------------------ clipping

def _copies(ts):
    """Tensors of the same layout, in memory of their own."""
    out = []
    for t in ts:
        buf = torch.empty(t.untyped_storage().nbytes() // t.element_size(), dtype=t.dtype, device="cuda")
        buf.copy_(torch.as_strided(t, (buf.numel(),), (1,), 0))
        out.append(torch.as_strided(buf, t.shape, t.stride(), t.storage_offset()))
    return out


def _whole(t):
    return torch.as_strided(t, (t.untyped_storage().nbytes() // t.element_size(),), (1,), 0)


def _bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == F32 else torch.int16)


def _scaled(t, scale):
    return (t.float() * scale).to(t.dtype)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("mode", ["in_place", "outs", "packed_outs"])
def test_clip(kind, dtype, mode):
    ts = _copies(_make(kind, dtype, 7))
    before = [t.clone() for t in ts]
    around = [_whole(t).clone() for t in ts]
    max_norm = 0.3 * _norm64(ts)
    if mode == "in_place":
        outs = None
        r = gns.clip_grads(ts, max_norm)
        got = ts
    else:
        if mode == "packed_outs":  # alignments that no shift of the first unit makes the same
            outs = []
            for t in ts:
                buf = torch.zeros(t.numel() + 3, dtype=t.dtype, device="cuda")
                outs.append(torch.as_strided(buf, t.shape, t.contiguous().stride(), 3) if t.is_contiguous() or kind != "shapes"
                            else torch.as_strided(buf, t.shape, t.stride(), 3))
        else:
            outs = _copies(ts)
            for o in outs:
                o.zero_()
        r = gns.clip_grads(ts, max_norm, outs=outs)
        got = outs
    assert float(r[1]) < 1.0
    for t, b, o in zip(ts, before, got):
        assert torch.equal(_bits(o), _bits(_scaled(b, r[1])))
        if outs is not None:
            assert torch.equal(_bits(t), _bits(b))
    if mode != "packed_outs":  # nothing beside the tensors is written (tensors of "many" share memory)
        if kind != "many":
            for t, b, a in zip(got, before, around):
                torch.as_strided(a, t.shape, t.stride(), t.storage_offset()).copy_(_scaled(b, r[1]))
                assert torch.equal(_bits(_whole(t)), _bits(a))
    else:
        for o in outs:
            assert not torch.as_strided(o, (3,), (1,), 0).any()


def test_clip_leaves_gradients_below_the_norm_alone():
    ts = _make("sizes", BF, 8) + _make("pitched", F32, 9)
    before = [t.clone() for t in ts]
    r = gns.clip_grads(ts, 1.01 * _norm64(ts))
    assert float(r[1]) == 1.0
    outs = [torch.zeros_like(t) for t in ts]
    gns.clip_grads(ts, math.inf, outs=outs)
    for t, b, o in zip(ts, before, outs):
        assert torch.equal(_bits(t), _bits(b)) and torch.equal(_bits(o), _bits(b))


def test_clip_with_outs_that_are_partly_the_gradients():
    ts = [_randn((100,), F32, 1), _randn((50,), F32, 2)]
    before = [t.clone() for t in ts]
    other = torch.zeros(50, device="cuda")
    r = gns.clip_grads(ts, math.inf, outs=[ts[0], other])
    assert float(r[1]) == 1.0 and torch.equal(ts[0], before[0]) and torch.equal(other, before[1])
    r = gns.clip_grads(ts, 1.0, outs=[ts[0], other])
    assert torch.equal(ts[0], before[0] * r[1]) and torch.equal(other, before[1] * r[1])


def test_clip_non_finite():
    t = torch.tensor([1.0, math.inf, -2.0], device="cuda")
    st = _status()
    gns.clip_grads([t], 1.0, status=st)
    assert int(st) == 1
    assert t[0] == 0.0 and torch.isnan(t[1]) and t[2] == 0.0
    t = torch.tensor([1.0, math.nan], device="cuda")
    gns.clip_grads([t], 1.0, status=st)
    assert torch.isnan(t).all()


@pytest.mark.parametrize("values", [(1e30,), (1e-30,), (1e25, 1e-30, 1.0), (3e-12, 1e-30), (1e-44,), (0.0,)])
@pytest.mark.parametrize("n", [5, 3000, 200003])
def test_clip_of_extreme_values(values, n):
    """Short lists and long ones take different kernels: both keep squares out of f32's range right."""
    ts = [torch.full((n,), v, device="cuda") for v in values] + [torch.zeros(7, device="cuda")]
    before = [t.clone() for t in ts]
    want = _norm64(ts)
    r = gns.clip_grads(ts, 0.25 * want, eps=0.0)
    assert abs(float(r[0]) - want) <= NORM_TOL * want + 2.0 ** -150
    for t, b in zip(ts, before):
        assert torch.equal(_bits(t), _bits(_scaled(b, r[1])))


# ------------------------------------------------------------------------------------ AdamW

P = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def _adamw64(w, g, m, v, scale, step):
    """The step in 64 bits (a b-c sum of each new moment beside it for the bounds)."""
    g = g.double() * scale
    m = P["beta1"] * m.double() + (1 - P["beta1"]) * g
    v = P["beta2"] * v.double() + (1 - P["beta2"]) * g * g
    update = P["lr"] / (1 - P["beta1"] ** step) * m / ((v / (1 - P["beta2"] ** step)).sqrt() + P["eps"])
    w = (1 - P["lr"] * P["weight_decay"]) * w.double()
    return w - update, m, v, w, update


def adamw_bounds(w, g, m, v, scale, step):
    """Absolute bounds of the f32 results, counted in units of U = 2^-24, each constant and each
    operation giving at most one:
    m: the scaled gradient 1 (and 1 for the scale itself), 1 - beta1 and its product 2, beta1 1, the sum 1: 6 of |beta1 m| + |(1-beta1) g|;
    v: twice the gradient's 2, 1 - beta2 and two products 3, beta2 1, the sum 1: 9 of v, which is a sum of positive terms;
    update: m's, then half of v's 9, the root 1, 1/sqrt(1 - beta2^t) 1, the sum 1, the quotient 1, the step size 1, their product
    1: 11 of |update|, and m's error in the same proportion; the step's number on the device costs expm1's and log's few units
    more: 16 in all;
    w: the decay 1 and its product's share of the last sum, 2 of |w|, 1 of |update|."""
    gs = g.double().abs() * scale
    mag = P["beta1"] * m.double().abs() + (1 - P["beta1"]) * gs
    w64, m64, v64, decayed, update = _adamw64(w, g, m, v, scale, step)
    gain = P["lr"] / (1 - P["beta1"] ** step) / ((v64 / (1 - P["beta2"] ** step)).sqrt() + P["eps"])
    tiny = 2.0 ** -148
    bm = 6 * U * mag + tiny
    bv = 9 * U * v64 + tiny
    bw = 6 * U * mag * gain + 17 * U * update.abs() + 3 * U * decayed.abs() + tiny
    return bw, bm, bv


def _half_ulp(x, dtype):
    if dtype == F32:
        return torch.zeros_like(x)
    bits, least = (7, -126) if dtype == BF else (10, -14)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** least)))
    return 0.5001 * 2.0 ** (e - bits)


def _adamw_check(ws, gs, ms, vs, masters, scale=None, step=1, step_count=None):
    c = 1.0 if scale is None else float(scale)
    src = [w.clone() if p is None else p.clone() for w, p in zip(ws, masters or [None] * len(ws))]
    old = [(a.clone(), b.clone(), d.clone()) for a, b, d in zip(gs, ms, vs)]
    st = _status()
    gns.adamw_step(ws, gs, ms, vs, masters=masters, params=gns.AdamWParams(step=7 if step_count is not None else step, **P),
                   grad_scale=scale, step_count=step_count, status=st)
    assert int(st) == 0
    for i, (w, g, m, v) in enumerate(zip(ws, gs, ms, vs)):
        if not w.numel():
            continue
        g0, m0, v0 = old[i]
        assert torch.equal(_bits(g), _bits(g0))
        w64, m64, v64, _, _ = _adamw64(src[i], g0, m0, v0, c, step)
        bw, bm, bv = adamw_bounds(src[i], g0, m0, v0, c, step)
        assert bool(((m.double() - m64).abs() <= bm).all()), i
        assert bool(((v.double() - v64).abs() <= bv).all()), i
        p = masters[i] if masters else None
        if p is not None:
            assert bool(((p.double() - w64).abs() <= bw).all()), i
            assert torch.equal(_bits(w), _bits(p.to(w.dtype)))
        else:
            assert bool(((w.double() - w64).abs() <= bw + _half_ulp(w64, w.dtype)).all()), i


def _adamw_lists(kind, wdt, gdt, master, seed=0):
    ws = _copies(_make(kind, wdt, 20 + seed, 0.05))
    gs = _copies(_make(kind, gdt, 40 + seed, 0.01))
    ms = _copies(_make(kind, F32, 60 + seed, 0.003))
    vs = _copies(_make(kind, F32, 80 + seed, 0.01))
    for v in vs:
        v.square_()
    masters = None
    if master:
        masters = _copies(_make(kind, F32, 20 + seed, 0.05))
    return ws, gs, ms, vs, masters


TYPES = [(F32, F32, False), (BF, BF, False), (BF, BF, True), (BF, F32, False), (BF, F32, True), (F16, F16, False),
         (F16, F32, True), (F16, BF, False), (F32, BF, False), (F32, F16, False), (BF, F16, True)]


@pytest.mark.parametrize("wdt,gdt,master", TYPES)
@pytest.mark.parametrize("kind", ["sizes", "offsets", "pitched", "pitched_stacks", "shapes"])
def test_adamw(kind, wdt, gdt, master):
    _adamw_check(*_adamw_lists(kind, wdt, gdt, master), step=3)


@pytest.mark.parametrize("wdt,gdt,master", [(F32, F32, False), (BF, BF, True), (BF, F32, False)])
@pytest.mark.parametrize("kind", ["many", "many_pitched", "large"])
def test_adamw_long_lists(kind, wdt, gdt, master):
    _adamw_check(*_adamw_lists(kind, wdt, gdt, master), scale=torch.full((1,), 0.3, device="cuda"), step=100)


@pytest.mark.parametrize("wdt,gdt,master", [(F32, F32, False), (BF, BF, True), (F16, F32, False)])
def test_adamw_alignments_that_differ_between_roles(wdt, gdt, master):
    ws, gs, ms, vs, masters = [], [], [], [], [] if master else None
    for o in [(0, 1, 2, 3, 4), (5, 5, 5, 5, 5), (4, 4, 4, 0, 4), (1, 9, 17, 25, 33), (0, 0, 4, 4, 4), (8, 0, 0, 4, 0)]:
        for n in (1, 6, 1000, 4097):
            ws.append(_randn((n + 40,), wdt, n, 0.05)[o[0]:o[0] + n])
            gs.append(_randn((n + 40,), gdt, n + 1, 0.01)[o[1]:o[1] + n])
            ms.append(_randn((n + 40,), F32, n + 2, 0.003)[o[2]:o[2] + n])
            vs.append((_randn((n + 40,), F32, n + 3, 0.01)[o[3]:o[3] + n]).square_())
            if master:
                masters.append(_randn((n + 40,), F32, n + 4, 0.05)[o[4]:o[4] + n])
    whole = [[_whole(t).clone() for t in l] for l in (ws, ms, vs)]
    _adamw_check(ws, gs, ms, vs, masters, step=2)
    for l, b in zip((ws, ms, vs), whole):
        for t, a in zip(l, b):
            torch.as_strided(a, t.shape, t.stride(), t.storage_offset()).copy_(t)
            assert torch.equal(_bits(_whole(t)), _bits(a))


def test_adamw_mixed_list():
    """One list of every type, with masters where they are wanted, pitches and empty tensors."""
    lists = [[], [], [], [], []]
    for i, (wdt, gdt, master) in enumerate(TYPES):
        for kind in ("sizes", "pitched", "shapes"):
            ws, gs, ms, vs, ps = _adamw_lists(kind, wdt, gdt, master, seed=i)
            for l, x in zip(lists, (ws, gs, ms, vs, ps or [None] * len(ws))):
                l += x
    # a pitch in one role only
    lists[0].append(_randn((7, 16), BF, 1)[:, :11])
    for l, dt in zip(lists[1:4], (BF, F32, F32)):
        l.append(_randn((7, 11), dt, 2).abs())
    lists[4].append(None)
    _adamw_check(*lists, scale=torch.full((1,), 2.5, device="cuda"), step=11)


def test_adamw_step_count_on_the_device():
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in (1, 2, 50, 100000):
        count.fill_(step)
        _adamw_check(*_adamw_lists("sizes", F32, F32, False, seed=step % 50), step=step, step_count=count)


@pytest.mark.parametrize("beta1,beta2", [(0.0, 0.0), (0.9, 0.0), (0.0, 0.999)])
def test_adamw_without_memory(beta1, beta2, monkeypatch):
    monkeypatch.setitem(P, "beta1", beta1)
    monkeypatch.setitem(P, "beta2", beta2)
    for count in (None, torch.full((1,), 4, dtype=torch.int32, device="cuda")):
        _adamw_check(*_adamw_lists("sizes", F32, BF, False), step=4, step_count=count)


def test_adamw_rows_without_gradient_or_state():
    """Rows of an embedding that no token has touched only decay."""
    w = _randn((64, 33), BF, 1, 0.05)
    g, m, v = (torch.zeros(64, 33, dtype=dt, device="cuda") for dt in (BF, F32, F32))
    before = w.clone()
    gns.adamw_step([w], [g], [m], [v], lr=1e-2, weight_decay=0.0)
    assert torch.equal(_bits(w), _bits(before)) and not m.any() and not v.any()


def test_adamw_non_finite():
    st = _status()
    w, m, v = (torch.ones(5000, device="cuda") for _ in range(3))
    g = torch.zeros(5000, device="cuda")
    g[4321] = math.nan
    gns.adamw_step([w], [g], [m], [v], lr=1e-2, status=st)
    assert int(st) == 1
    assert int(torch.isnan(w).sum()) == 1 and bool(torch.isnan(w[4321]))
    with pytest.raises(gns.GnsDeviceError, match="non-finite"):
        gns.adamw_step([w], [g], [m], [v], lr=1e-2)


def test_adamw_beyond_32_bits():
    n = 2 ** 31 + 1003
    w, g = (torch.zeros(n, dtype=BF, device="cuda") for _ in range(2))
    m, v = (torch.zeros(n, dtype=F32, device="cuda") for _ in range(2))
    at = slice(n - 3000, n)
    w[at], g[at] = _randn((3000,), BF, 1, 0.05), _randn((3000,), BF, 2, 0.01)
    w0, g0 = w[at].clone(), g[at].clone()
    gns.adamw_step([w], [g], [m], [v], params=gns.AdamWParams(step=2, **P))
    z = torch.zeros(3000, device="cuda")
    w64, m64, v64, _, _ = _adamw64(w0, g0, z, z, 1.0, 2)
    bw, bm, bv = adamw_bounds(w0, g0, z, z, 1.0, 2)
    assert bool(((w[at].double() - w64).abs() <= bw + _half_ulp(w64, BF)).all())
    assert bool(((m[at].double() - m64).abs() <= bm).all()) and bool(((v[at].double() - v64).abs() <= bv).all())
    assert not w[:1000].any() and not m[2 ** 31 - 2000 - 1003:2 ** 31 - 2000].any()


def test_adamw_descends():
    """Against differences: along the step that a gradient gives, the loss falls as its slope says."""
    w = _randn((257,), F32, 1)
    target = _randn((257,), F32, 2)
    loss = lambda x: float(((x.double() - target.double()) ** 2).sum() / 2)  # noqa: E731
    m, v = torch.zeros_like(w), torch.zeros_like(w)
    before = loss(w)
    g = (w - target).clone()
    w0 = w.clone()
    gns.adamw_step([w], [g], [m], [v], lr=1e-4, weight_decay=0.0)
    slope = float((g.double() * (w.double() - w0.double())).sum())
    assert loss(w) < before
    # the second-order part is half the step's square
    assert abs(loss(w) - before - slope) <= 0.51 * float(((w.double() - w0.double()) ** 2).sum())


# ------------------------------------------------------------------------------------ streams, graphs, plans

def test_captured_clip_and_step_match_eager():
    """grad_norm and adamw_step captured once and replayed, the step's number counted on the device."""
    ws, gs, ms, vs, ps = _adamw_lists("sizes", BF, BF, True)
    lists = [_copies(x) for x in (ws, gs, ms, vs, ps)]
    status = _status()
    result = torch.empty(2, device="cuda")
    work = gns.alloc_workspace(gns.list_workspace_size(len(ws)), "cuda")

    def step(ws, gs, ms, vs, ps, **kw):
        gns.grad_norm(gs, max_norm=0.5, result=result, workspace=work, status=status)
        gns.adamw_step(ws, gs, ms, vs, masters=ps, grad_scale=result[1:], status=status, lr=1e-2, **kw)

    for t in (1, 2, 3):
        step(ws, gs, ms, vs, ps, step=t)
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            count.add_(1)
            step(*lists, step_count=count)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert int(status) == 0 and int(count) == 3
    for a, b in zip((ws, ms, vs, ps), (lists[0], lists[2], lists[3], lists[4])):
        for x, y in zip(a, b):
            # the corrections 1 - beta^t are formed on the device: a few units in the last place apart
            assert float((x.double() - y.double()).abs().max()) <= 2.0 ** (-7 if x.dtype == BF else -18) * max(1e-3, float(x.double().abs().max()))


def test_replayed_norm_reads_the_gradients_anew():
    """A captured norm gives the gradients' norm at each replay, not an earlier one's."""
    ts = _make("large", BF, 3) + _make("pitched", F32, 4)
    result = torch.empty(2, device="cuda")
    work = gns.alloc_workspace(gns.list_workspace_size(len(ts)), "cuda")
    status = _status()
    gns.grad_norm(ts, result=result, workspace=work, status=status)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gns.grad_norm(ts, result=result, workspace=work, status=status)
    first = _norm64(ts)
    for k in range(1, 30):
        torch._foreach_mul_(ts, 2.0 if k % 3 else 0.25)
        graph.replay()
        want = first * 2.0 ** (k - 3 * (k // 3))
        assert abs(float(result[0]) - want) <= NORM_TOL * want, k
    assert int(status) == 0


@pytest.mark.parametrize("kind", ["sizes", "large", "pitched"])
def test_replayed_clipping(kind):
    """Clipping captured once: each replay clips the gradients that are there then."""
    ts = _make(kind, BF, 9)
    base = [t.clone() for t in ts]
    outs = [torch.empty_like(t) for t in ts]
    result = torch.empty(2, device="cuda")
    work = gns.alloc_workspace(gns.list_workspace_size(len(ts)), "cuda")
    status = _status()
    lists = gns.tensor_list(ts), gns.tensor_list(outs)
    max_norm = 0.5 * _norm64(ts)
    call = lambda: gns.clip_grads(lists[0], max_norm, outs=lists[1], result=result, workspace=work, status=status)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for factor in (1.0, 4.0, 0.25, 2.0):
        for t, b in zip(ts, base):
            t.copy_(b * factor)
        graph.replay()
        want = 2.0 * max_norm * factor
        assert abs(float(result[0]) - want) <= NORM_TOL * want
        for t, o in zip(ts, outs):
            assert torch.equal(_bits(o), _bits(_scaled(t, result[1])))
    assert int(status) == 0


@pytest.mark.parametrize("kind", ["sizes", "large", "many", "many_pitched"])
def test_calls_in_a_row_share_a_workspace(kind):
    """Nothing waits between the calls, and the workspace holds whatever was there before."""
    ts = _make(kind, BF, 6)
    work = gns.alloc_workspace(gns.list_workspace_size(len(ts)), "cuda")
    work.fill_(255)
    results = torch.empty(60, 2, device="cuda")
    outs = _copies(ts)
    status = _status()
    lists, out_lists = gns.tensor_list(ts), gns.tensor_list(outs)
    for k in range(60):
        if k % 2:
            gns.grad_norm(lists, result=results[k], workspace=work, status=status)
        else:
            gns.clip_grads(lists, math.inf, outs=out_lists, result=results[k], workspace=work, status=status)
        torch._foreach_mul_(ts, 2.0 if k % 4 < 2 else 0.5)
    got = results[:, 0].tolist()
    assert int(status) == 0
    want = got[1]  # after one doubling
    for k, x in enumerate(got):
        expected = want * (0.5, 1.0, 2.0, 1.0)[k % 4]
        if kind == "sizes" and k % 2 == 0:  # the short list's clipping adds in another order
            assert abs(x - expected) <= NORM_TOL * expected
        else:
            assert x == expected, k  # the same order, values times a power of two: the same bits


def test_another_stream():
    ts = _make("large", BF, 5)
    want = _norm64(ts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        # result and workspace come from the current stream's memory, which goes on being used there
        r = gns.grad_norm(ts, stream=side, check=False)
        torch.full((4096,), -1.0, device="cuda")
        side.synchronize()
        assert abs(float(r[0]) - want) <= NORM_TOL * want


def test_argument_checks():
    t = torch.ones(8, device="cuda")
    for bad in (torch.empty(2), torch.empty(3, device="cuda"), torch.empty(2, device="cuda", dtype=BF), torch.empty(4, device="cuda")[::2]):
        with pytest.raises(ValueError, match="result"):
            gns.grad_norm([t], result=bad)
    with pytest.raises(ValueError, match="every gradient"):
        gns.grad_norm([t, None])
    with pytest.raises(gns.GnsError, match="max_norm"):
        gns.clip_grads([t], -1.0)
    with pytest.raises(ValueError, match="G.0."):
        gns.adamw_step([t], [t[:4]], [t], [t], lr=1.0)
    with pytest.raises(ValueError, match="lr"):
        gns.adamw_step([t], [t], [t], [t])
    for bad in (torch.ones(1), torch.ones(2, device="cuda"), torch.ones(1, device="cuda", dtype=BF)):
        with pytest.raises(ValueError, match="grad_scale"):
            gns.adamw_step([t], [t.clone()], [t.clone()], [t.clone()], lr=1.0, grad_scale=bad)
    with pytest.raises(gns.GnsError, match="alias"):
        gns.adamw_step([t], [t], [t.clone()], [t.clone()], lr=1.0)
    with pytest.raises(gns.GnsError, match="workspace too small"):
        gns.grad_norm([t], workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
