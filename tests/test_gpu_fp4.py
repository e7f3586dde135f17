"""Matrices in microscaled 4-bit floating point on the GPU against the 64-bit oracle: codes and scales to the bit, products
within a bound from arithmetic, and the operators' behaviour as calls (streams, graphs, padding, refusals)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_gb300 as gns  # noqa: E402
from oracle import fp4  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FORMATS = ["nvfp4", "mxfp4"]


def padded(t, extra=0):
    """A copy on the GPU whose rows start on 16-byte boundaries, `extra` 16-byte units apart; NaN lies between them."""
    step = 16 // t.element_size()
    cols = t.shape[-1]
    buf = torch.full((*t.shape[:-1], (-(-cols // step) + extra) * step), float("nan"), dtype=t.dtype, device="cuda")
    buf[..., :cols].copy_(t)
    return buf[..., :cols]


def matrices(seed, shape, dtype, spread=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal((*shape[:-1], 1)))
    return torch.from_numpy(x).to(DTYPES[dtype])


def as_batch(q):
    """codes, scales, tensor scale in numpy, with the count in front."""
    c = q.codes.cpu().numpy()
    s = q.scales.cpu().numpy()
    return (c, s) if c.ndim == 3 else (c[None], s[None])


def held_exactly(q, x64, amax=None):
    """q holds the oracle's codes and scales of the matrices x64 (count, rows, cols), zeros in all padding."""
    codes, scales = as_batch(q)
    for i, x in enumerate(x64):
        code, byte, g = fp4.quantize(x, q.fmt, None if amax is None else amax[i])
        want_c, want_s = fp4.pack_codes(code, codes.shape[-1]), fp4.pack_scales(byte)
        # the sign of a zero code is free
        assert ((codes[i] == want_c) | same_values(codes[i], want_c)).all(), (i, np.argwhere(codes[i] != want_c)[:4])
        assert (scales[i] == want_s).all(), (i, np.argwhere(scales[i] != want_s)[:4])
        if g is not None:
            assert float(q.tensor_scale[i]) == g


def same_values(a, b):
    half = lambda x: np.where((x & 7) == 0, 0, x)  # noqa: E731
    return (half(a & 15) == half(b & 15)) & (half(a >> 4) == half(b >> 4))


def oracle_values(x64, fmt):
    return np.stack([fp4.values(*fp4.quantize(x, fmt), fmt) for x in x64])


SHAPES = [(1, 1, 1), (1, 1, 17), (1, 128, 512), (2, 129, 65), (3, 5, 1000), (1, 300, 31), (2, 257, 48), (1, 2, 4100), (1, 700, 129)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize_and_back(shape, dtype, fmt):
    x = matrices(1, shape, dtype)
    x64 = x.double().numpy()
    d = padded(x, extra=1)
    q, qt = gns.quantize_fp4(d, fmt, axes="both")
    assert q.shape == x.shape and qt.shape == x.mT.shape
    held_exactly(q, x64)
    held_exactly(qt, x64.transpose(0, 2, 1))
    q1, qt1 = gns.quantize_fp4(d, fmt), gns.quantize_fp4(d, fmt, axes="cols")
    for a, b in ((q, q1), (qt, qt1)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    for name, t in DTYPES.items():  # values are exact in fp32, rounded once below
        want = torch.from_numpy(oracle_values(x64, fmt))
        got = gns.dequantize_fp4(q, dtype=t)
        assert got.shape == x.shape and torch.equal(got.cpu().double(), want.float().to(t).double()), name
    got = gns.dequantize_fp4(qt, out=padded(torch.zeros(*qt.shape), extra=1))
    assert torch.equal(got.cpu().double(), torch.from_numpy(oracle_values(x64.transpose(0, 2, 1), fmt)))


@pytest.mark.parametrize("fmt", FORMATS)
def test_values_on_the_borders(fmt):
    """Quotients that lie on a border between two codes, one fp32 step beside it, and every fp16 number as a value."""
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    rows = []
    for s in fp4.E4M3[1:][::3] if fmt == "nvfp4" else 2.0 ** np.arange(-30, 30, 7):
        v = np.float32(border * s)
        rows.append(np.concatenate([[6 * s], v, np.nextafter(v, np.float32(0)), -np.nextafter(v, np.float32(9e9)), [0.0] * 7]))
    x = torch.from_numpy(np.array(rows, dtype=np.float32))[None]
    x[0, 0, -1] = 2688.0
    q, qt = gns.quantize_fp4(padded(x), fmt, axes="both")
    held_exactly(q, x.double().numpy())
    held_exactly(qt, x.double().numpy().transpose(0, 2, 1))
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.float16)
    every = every[torch.isfinite(every)][: 2048 * 31].reshape(1, -1, 64)
    held_exactly(gns.quantize_fp4(padded(every), fmt), every.double().numpy())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", [1e-45, 3e-39, 1e-37, 1e-30, 1e30, 3.4e38])
def test_sizes_at_the_ends_of_fp32(fmt, size):
    rng = np.random.default_rng(3)
    x = torch.from_numpy((np.float32(size) * rng.uniform(-1, 1, (1, 40, 70)).astype(np.float32)))
    x[0, 0, 0] = size
    q, qt = gns.quantize_fp4(padded(x), fmt, axes="both")
    held_exactly(q, x.double().numpy())
    held_exactly(qt, x.double().numpy().transpose(0, 2, 1))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_matrices_of_zeros_and_mixed_sizes(dtype):
    x = matrices(4, (4, 130, 50), dtype)
    x[1] = 0
    x[2] *= 1e-3
    x[3, :, ::2] = -0.0
    for fmt in FORMATS:
        q, qt = gns.quantize_fp4(padded(x), fmt, axes="both")
        held_exactly(q, x.double().numpy())
        held_exactly(qt, x.double().numpy().transpose(0, 2, 1))
        assert not gns.dequantize_fp4(q)[1].any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_nonfinite_values_stay_in_their_blocks(fmt, bad):
    x = matrices(5, (2, 200, 100), "bf16")
    x[0, 3, 7] = x[1, 199, 99] = bad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, qt = gns.quantize_fp4(padded(x), fmt, axes="both", status=status)
    assert int(status) == 1
    held_exactly(q, x.double().numpy())
    held_exactly(qt, x.double().numpy().transpose(0, 2, 1))
    with pytest.raises(gns.GnsDeviceError):
        gns.quantize_fp4(padded(x), fmt)
    # the row's products are NaN, the others are not
    status.zero_()
    d = gns.fp4_gemm(q, q, status=status, dtype=torch.float32).cpu()
    assert int(status) == 1
    rows = torch.isnan(d).all(2)
    assert rows[0, 3] and rows[1, 199] and rows.sum() == 2 and torch.isfinite(d[0, 4]).sum() == 199


def test_given_amax():
    x = matrices(6, (6, 64, 96), "f32", spread=0.0)
    x64 = x.double().numpy()
    given = np.float32([np.abs(x64[0]).max(), 0.01, 1e-30, 1e30, 0.0, np.inf])  # right, too small by much, ..., no size at all
    q, qt = gns.quantize_fp4(padded(x), axes="both", amax=torch.from_numpy(given).cuda())
    held_exactly(q, x64, given.astype(np.float64))
    held_exactly(qt, x64.transpose(0, 2, 1), given.astype(np.float64))
    x[2] *= 1e30  # the quotient passes fp32's range
    held_exactly(gns.quantize_fp4(padded(x), amax=torch.from_numpy(given).cuda()), x.double().numpy(), given.astype(np.float64))


# ---- products ----


def random_held(seed, shape, fmt, extra=0):
    """An Fp4Matrix of normal values, with rows `extra` 16-byte units further apart, and its values in 64 bits."""
    count, rows, cols = shape
    x = np.random.default_rng(seed).standard_normal(shape)
    got = [fp4.quantize(m, fmt) for m in x]
    width = -(-cols // 32) * 16 + 16 * extra
    codes = torch.full((count, rows, width), 0xFF, dtype=torch.uint8)
    want = -(-cols // 32) * 16
    codes[..., :want] = torch.from_numpy(np.stack([fp4.pack_codes(c) for c, _, _ in got]))
    tiles = np.stack([fp4.pack_scales(b) for _, b, _ in got])
    if rows % 128:  # scales behind the last row are not read
        r = np.arange(rows % 128, 128)
        at = ((r % 32) * 16 + r // 32 * 4)[:, None] + np.arange(4)
        tiles[:, -1, :, :][:, :, at] = 0x7F if fmt == "nvfp4" else 0xFF
    g = torch.tensor([g for _, _, g in got], dtype=torch.float32).cuda() if fmt == "nvfp4" else None
    q = gns.Fp4Matrix(codes.cuda(), torch.from_numpy(tiles).cuda(), g, cols, fmt)
    return q, np.stack([fp4.values(*t, fmt) for t in got])


def check_product(got, a, b, dtype, alpha=1.0, beta=0.0, c=None):
    """|error| <= half a step of the type of the result, plus what the sum may lose: each of the K / 64 matrix instructions
    adds 64 products (each exact) to the accumulator; products and accumulator are cut or rounded at 2^-23 of the largest, twice
    at most, and the largest is at most sum |a b|. The epilogue's multiplications and addition round at 2^-24 each."""
    want = alpha * (a @ b.transpose(0, 2, 1))
    size = abs(alpha) * (np.abs(a) @ np.abs(b).transpose(0, 2, 1))
    if beta:
        want = want + beta * c
        size = size + abs(beta) * np.abs(c)
    k = a.shape[2]
    t = DTYPES[dtype]
    bound = (torch.finfo(t).eps / 2) * np.abs(want) * (1 + 2.0**-7) + ((k / 64 + 1) * 2.0**-22 + 4 * 2.0**-24) * size
    bound = bound + torch.finfo(t).smallest_normal * torch.finfo(t).eps
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= bound).all(), (np.argwhere(off > bound)[:4], off.max(), bound[off > bound][:4])


PRODUCTS = [(1, 1, 1, 1), (1, 1, 64, 64), (1, 3, 5, 17), (2, 1, 300, 1000), (1, 16, 129, 256), (1, 33, 70, 4100), (3, 129, 127, 65),
            (1, 128, 128, 512), (2, 257, 130, 300), (1, 300, 520, 1025), (1, 515, 700, 96), (1, 64, 1000, 2048), (1, 1025, 1, 40), (1, 300, 11000, 300), (2, 2050, 2100, 130)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", PRODUCTS, ids=str)
def test_gemm(shape, dtype, fmt):
    count, m, n, k = shape
    a, va = random_held(11, (count, m, k), fmt)
    b, vb = random_held(12, (count, n, k), fmt, extra=1)
    check_product(gns.fp4_gemm(a, b, dtype=DTYPES[dtype]), va, vb, dtype)
    # with an addend, into rows of another pitch; what lies between them stays
    c = torch.from_numpy(np.random.default_rng(13).standard_normal((count, m, n))).to(DTYPES[dtype])
    d = padded(torch.zeros(count, m, n, dtype=DTYPES[dtype]), extra=1)
    gns.fp4_gemm(a, b, c=padded(c), d=d, alpha=-0.75, beta=1.5)
    check_product(d, va, vb, dtype, -0.75, 1.5, c.double().numpy())
    between = d.as_strided((count, m, d.stride(1)), d.stride())[..., n:]
    assert torch.isnan(between).all()
    # in place
    e = padded(c)
    gns.fp4_gemm(a, b, c=e, d=e, alpha=-0.75, beta=1.5)
    assert torch.equal(e, d)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 5, 100), (1, 128, 512), (3, 130, 300), (2, 333, 2001), (1, 600, 257), (1, 5000, 300)], ids=str)
def test_gram(shape, dtype, fmt):
    x, vx = random_held(21, shape, fmt)
    d = gns.fp4_sym_gemm_xxt(x, alpha=1 / 64, dtype=DTYPES[dtype])
    check_product(d, vx, vx, dtype, 1 / 64)
    assert torch.equal(d, d.mT)
    c = np.random.default_rng(22).standard_normal((shape[0], shape[1], shape[1]))
    c = torch.from_numpy(c + c.transpose(0, 2, 1)).to(DTYPES[dtype])
    e = padded(c, extra=1)
    gns.fp4_sym_gemm_xxt(x, c=e, d=e, alpha=1 / 64, beta=0.5)
    check_product(e, vx, vx, dtype, 1 / 64, 0.5, c.double().numpy())
    assert torch.equal(e, e.mT)


def test_products_of_every_code_and_scale():
    """One value a block, so that each sum has few terms: every pair of codes and a wide range of scales."""
    for fmt in FORMATS:
        n = fp4.BLOCK[fmt]
        byte = np.arange(1, 127, dtype=np.uint8) if fmt == "nvfp4" else np.arange(97, 157, dtype=np.uint8)
        rows = 16 * len(byte)
        code = np.zeros((rows, n), dtype=np.uint8)
        code[:, 0] = np.tile(np.arange(16), len(byte))
        byte = np.repeat(byte, 16)[:, None]
        g = 0.25 if fmt == "nvfp4" else None
        q = gns.Fp4Matrix(torch.from_numpy(fp4.pack_codes(code)).cuda(), torch.from_numpy(fp4.pack_scales(byte)).cuda(),
                          None if g is None else torch.tensor([g]).cuda(), n, fmt)
        v = fp4.values(code, byte, g, fmt)[:, :1]
        got = gns.fp4_gemm(q, q, dtype=torch.float32).double().cpu().numpy()
        np.testing.assert_array_equal(got, v @ v.T)  # products of at most 12 bits are exact


def test_overflow_of_the_result_is_reported():
    a, va = random_held(31, (1, 40, 64), "mxfp4")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = gns.fp4_gemm(a, a, alpha=60000.0, dtype=torch.float16, status=status)
    assert int(status) == 1 and torch.isinf(d).any()
    status.zero_()
    gns.fp4_gemm(a, a, alpha=60000.0, dtype=torch.bfloat16, status=status)
    assert int(status) == 0


# ---- as they are used ----


def test_training_products():
    """y = x w^T, dx = dy w and dw = dy^T x with all operands through 4 bits, dw added to what earlier passes left; the
    gradients are those of L = sum(y * dy) in the held values (checked against differences of L)."""
    m, n, k = 200, 144, 96
    x, w, dy = matrices(41, (m, k), "bf16", 0.3), matrices(42, (n, k), "bf16", 0.3), matrices(43, (m, n), "bf16", 0.3)
    for fmt in FORMATS:
        (xq, xt), (wq, wt), (gq, gt) = (gns.quantize_fp4(padded(t), fmt, axes="both") for t in (x, w, dy))
        y = gns.fp4_gemm(xq, wq)
        dx = gns.fp4_gemm(gq, wt, dtype=torch.float32)
        before = torch.ones(n, k, device="cuda")
        dw = gns.fp4_gemm(gt, xt, c=before, d=before, beta=1.0)
        v = {s: gns.dequantize_fp4(q, dtype=torch.float32).double().cpu().numpy()[None]
             for s, q in (("x", xq), ("xt", xt), ("w", wq), ("wt", wt), ("g", gq), ("gt", gt))}
        check_product(y[None], v["x"], v["w"], "bf16")
        check_product(dx[None], v["g"], v["wt"], "f32")
        check_product(dw[None], v["gt"], v["xt"], "f32", 1.0, 1.0, np.ones((1, n, k)))
        # L is linear in x: its difference along e is sum(dx * e), dx formed from the values that wt holds
        e = np.random.default_rng(44).standard_normal((m, k))
        loss = lambda z: float((z @ v["wt"][0] * v["g"][0]).sum())  # noqa: E731
        diff = (loss(v["x"][0] + 0.5 * e) - loss(v["x"][0] - 0.5 * e))
        assert abs(diff - float((dx.double().cpu().numpy() * e).sum())) <= 1e-5 * np.abs(dx.cpu().numpy() * e).sum()


def test_streams_and_graphs():
    x, w = padded(matrices(51, (33, 4096), "bf16")), padded(matrices(52, (1000, 4096), "bf16"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    wq = gns.quantize_fp4(w, status=status)
    want = gns.fp4_gemm(gns.quantize_fp4(x), wq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gns.fp4_gemm(gns.quantize_fp4(x, stream=side), wq, stream=side)
    assert torch.equal(got, want)
    # captured and replayed on other inputs
    xs, q, d = x.clone(), gns.empty_fp4((33, 4096)), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gns.quantize_fp4(xs, out=q, status=status)
        gns.fp4_gemm(q, wq, d=d, status=status)
    for scale in (1.0, -0.5, 3.0):
        xs.copy_(x * scale)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, gns.fp4_gemm(gns.quantize_fp4(x * scale), wq))
    assert int(status) == 0


def test_two_calls_at_once():
    """Calls on two streams share nothing."""
    xs = [padded(matrices(60 + i, (4, 512, 2048), "bf16")) for i in range(2)]
    want = [gns.fp4_sym_gemm_xxt(gns.quantize_fp4(x)) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    status = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [[], []]
        for i in range(2):
            for _ in range(4):
                q = gns.quantize_fp4(xs[i], stream=streams[i], status=status[i])
                got[i].append(gns.fp4_sym_gemm_xxt(q, stream=streams[i], status=status[i]))
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(g, want[i]) for g in got[i])


def test_the_same_call_gives_the_same_bits():
    a, _ = random_held(71, (1, 16, 11008), "nvfp4")
    b, _ = random_held(72, (1, 512, 11008), "nvfp4")
    first = gns.fp4_gemm(a, b, dtype=torch.float32)
    assert all(torch.equal(first, gns.fp4_gemm(a, b, dtype=torch.float32)) for _ in range(5))


def test_guards_around_outputs():
    """Nothing is written outside the held matrix and the result."""
    for fmt in FORMATS:
        for rows, cols in ((1, 1), (130, 70), (257, 33)):
            x = padded(matrices(81, (rows, cols), "f32"))
            q = gns.empty_fp4((rows, cols), fmt)
            pools = []
            for t in (q.codes, q.scales):
                pool = torch.full((t.numel() + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
                pools.append((pool, pool[4096:4096 + t.numel()].view(t.shape)))
            g = torch.full((3,), 7.0, device="cuda")
            q = gns.Fp4Matrix(pools[0][1], pools[1][1], g[1:2] if fmt == "nvfp4" else None, cols, fmt)
            gns.quantize_fp4(x, fmt, out=q)
            held_exactly(q, x.double().cpu().numpy()[None])
            for pool, t in pools:
                assert (pool[:4096] == 0xA5).all() and (pool[4096 + t.numel():] == 0xA5).all()
            assert float(g[0]) == float(g[2]) == 7.0
