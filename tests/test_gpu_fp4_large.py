"""Matrices in 4 bits at the sizes where the large paths run: rings of operands that wrap, groups of CTAs with several tiles,
the largest magnitudes of large matrices, and what lies around and between the outputs."""
import functools

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_gb300 as gns  # noqa: E402
from fp4_tilings import GEMMS, GRAMS  # noqa: E402
from oracle import fp4  # noqa: E402
from test_gpu_fp4 import DTYPES, FORMATS, check_product, held_exactly, matrices, oracle_values, padded, random_held  # noqa: E402

pytestmark = pytest.mark.gpu

held_once = functools.lru_cache(maxsize=2)(random_held)


@pytest.mark.parametrize("shape", GEMMS, ids=str)
@pytest.mark.parametrize("fmt", FORMATS)
def test_gemm_of_many_slices(fmt, shape):
    count, m, n, k = shape
    a, va = held_once(91, (count, m, k), fmt)
    b, vb = held_once(92, (count, n, k), fmt, extra=1)
    for name, dtype in DTYPES.items():
        check_product(gns.fp4_gemm(a, b, dtype=dtype), va, vb, name)
    c = torch.from_numpy(np.random.default_rng(93).standard_normal((count, m, n), dtype=np.float32))
    d = padded(c)
    gns.fp4_gemm(a, b, c=d, d=d, alpha=-0.75, beta=1.5)
    check_product(d, va, vb, "f32", -0.75, 1.5, c.double().numpy())


@pytest.mark.parametrize("shape", GRAMS, ids=str)
@pytest.mark.parametrize("fmt", FORMATS)
def test_gram_of_many_slices(fmt, shape):
    x, vx = random_held(94, shape, fmt)
    for name, dtype in DTYPES.items():
        d = gns.fp4_sym_gemm_xxt(x, alpha=1 / 64, dtype=dtype)
        check_product(d, vx, vx, name, 1 / 64)
        assert torch.equal(d, d.mT)


def test_largest_magnitudes_of_many_large_matrices():
    """11 matrices of 99 tiles each: one launch finds all their largest magnitudes, the next one takes each matrix's own."""
    x = matrices(95, (11, 1100, 1300), "f32") * (10.0 ** torch.arange(-5, 6))[:, None, None].float()
    d = padded(x)
    q, qt = gns.quantize_fp4(d, axes="both")
    x64 = x.double().numpy()
    held_exactly(q, x64)
    held_exactly(qt, x64.transpose(0, 2, 1))
    for axes, want in (("rows", q), ("cols", qt)):
        got = gns.quantize_fp4(d, axes=axes)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
        assert torch.equal(got.tensor_scale, want.tensor_scale)


def pool_of(shape):
    """A uint8 tensor of `shape` (rows 32 bytes further apart than they need to be) amid a larger one, and that one."""
    n = int(np.prod(shape))
    pool = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    return pool, pool[4096:4096 + n].view(shape)


@pytest.mark.parametrize("axes", ["rows", "cols", "both"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 130, 70), (3, 257, 33), (2, 31, 300), (2, 513, 520)], ids=str)
def test_nothing_is_written_around_or_between_what_is_held(shape, fmt, axes):
    x = matrices(96, shape, "bf16")
    made = []
    for s, wanted in ((shape, axes != "cols"), ((shape[0], shape[2], shape[1]), axes != "rows")):
        if not wanted:
            made.append(None)
            continue
        count, rows, cols = s
        width = -(-cols // 32) * 16
        blocks = -(-cols // fp4.BLOCK[fmt])
        codes, wide = pool_of((count, rows, width + 32))
        scales, tiles = pool_of((count, -(-rows // 128), -(-blocks // 4), 512))
        g = torch.full((count + 2,), 7.0, device="cuda")
        q = gns.Fp4Matrix(wide[..., :width], tiles, g[1:-1] if fmt == "nvfp4" else None, cols, fmt)
        made.append((q, codes, wide, scales, tiles, g, width))
    gns.quantize_fp4(padded(x, extra=1), fmt, out=made[0] and made[0][0], out_t=made[1] and made[1][0])
    x64 = x.double().numpy()
    for entry, want in zip(made, (x64, x64.transpose(0, 2, 1))):
        if entry is None:
            continue
        q, codes, wide, scales, tiles, g, width = entry
        assert (wide[..., width:] == 0xA5).all()
        for pool, t in ((codes, wide), (scales, tiles)):
            assert (pool[:4096] == 0xA5).all() and (pool[4096 + t.numel():] == 0xA5).all()
        assert float(g[0]) == float(g[-1]) == 7.0
        tight = gns.Fp4Matrix(wide[..., :width].contiguous(), tiles, q.tensor_scale, q.shape[-1], fmt)
        held_exactly(tight, want)
        for dtype in DTYPES.values():  # and back, into rows of another pitch: what lies between them stays
            out = padded(torch.zeros(*q.shape, dtype=dtype), extra=1)
            gns.dequantize_fp4(q, out=out)
            between = out.as_strided((*q.shape[:2], out.stride(1)), out.stride())[..., q.shape[-1]:]
            assert torch.isnan(between).all()
            assert torch.equal(out.cpu().double(), torch.from_numpy(oracle_values(want, fmt)).float().to(dtype).double())
