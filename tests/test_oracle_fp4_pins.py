"""The 4-bit oracle against the formats' definitions: every code and scale decodes to itself, the borders between codes,
the extremes, and the layout in memory."""
import numpy as np
import pytest

from oracle import fp4


def test_grids():
    assert len(fp4.E4M3) == 127 and fp4.E4M3[-1] == 448.0 and fp4.E4M3[1] == 2.0**-9 and fp4.E4M3[8] == 2.0**-6
    assert (np.diff(fp4.E4M3) > 0).all() and fp4.E4M3[0x38] == 1.0


@pytest.mark.parametrize("a,code", [(0.25, 0), (0.2500001, 1), (0.75, 2), (0.7499, 1), (1.25, 2), (1.26, 3), (1.75, 4), (2.5, 4),
                                    (2.51, 5), (3.5, 6), (3.49, 5), (5.0, 6), (5.01, 7), (6.0, 7), (1e9, 7), (0.0, 0)])
def test_borders(a, code):
    assert fp4.nearest(np.array([a]), fp4.E2M1)[0] == code


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_held_values_are_held_exactly(fmt):
    rng = np.random.default_rng(1)
    code = rng.integers(0, 16, (40, 96)).astype(np.uint8)
    code[code == 8] = 0  # -0 is held as 0 where the scale is 0 only
    code[:, ::16] = 7  # each block reaches 6 d, so that its scale is found again
    byte = rng.integers(1, 0x7E, (40, 6)) if fmt == "nvfp4" else rng.integers(1, 250, (40, 3))
    byte = byte.astype(np.uint8)
    byte[0, 0] = 0x7E if fmt == "nvfp4" else byte[0, 0]  # the matrix reaches 6 * 448 g
    g = 2.0**-20 if fmt == "nvfp4" else None
    x = fp4.values(code, byte, g, fmt)
    c2, b2, g2 = fp4.quantize(x, fmt)
    assert (c2 == code).all() and (b2 == byte).all() and g2 == g
    np.testing.assert_array_equal(fp4.values(c2, b2, g2, fmt), x)


@pytest.mark.parametrize("most,g", [(2688.0, 1.0), (2688.0001, 2.0), (1344.0, 0.5), (0.0, 0.0), (1e-45, 2.0**-126), (3.4e38, 2.0**117)])
def test_tensor_scale(most, g):
    assert fp4.tensor_scale(most) == g


def test_relative_error_of_a_block():
    """Within a block nothing is off by more than a sixth of the block's largest value (half the widest step, 1, plus what
    the scale's own rounding, 1 / 16, cuts off at the top); MXFP4 cuts off at 6 of up to 8."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((64, 256))
    for fmt, most in (("nvfp4", 1.0 / 6.0 * (1 + 1 / 16)), ("mxfp4", 0.25)):
        n = fp4.BLOCK[fmt]
        off = np.abs(fp4.values(*fp4.quantize(x, fmt), fmt) - x).reshape(64, -1, n).max(2)
        assert (off <= most * np.abs(x).reshape(64, -1, n).max(2) + 1e-15).all()


def test_nonfinite_blocks():
    x = np.ones((2, 40))
    x[0, 3], x[1, 33] = np.inf, np.nan
    for fmt, nan in (("nvfp4", 0x7F), ("mxfp4", 0xFF)):
        code, byte, g = fp4.quantize(x, fmt)
        n = fp4.BLOCK[fmt]
        assert byte[0, 0] == nan and byte[1, 33 // n] == nan and (byte == nan).sum() == 2
        v = fp4.values(code, byte, g, fmt)
        assert np.isnan(v[0, :n]).all() and np.isfinite(v[0, n:]).all()


def test_layout():
    code = np.arange(70, dtype=np.uint8).reshape(2, 35) % 16
    p = fp4.pack_codes(code)
    assert p.shape == (2, 32) and p[0, 0] == (1 << 4) and p[1, 17] == code[1, 34] and (p[:, 18:] == 0).all()
    byte = np.arange(130 * 5).reshape(130, 5).astype(np.uint8)
    t = fp4.pack_scales(byte)
    assert t.shape == (2, 2, 512)
    assert t[0, 0, 0] == byte[0, 0] and t[0, 0, 1] == byte[0, 1] and t[0, 0, 4] == byte[32, 0] and t[0, 0, 16] == byte[1, 0]
    assert t[1, 1, 16] == byte[129, 4] and t[1, 1, 17] == 0
