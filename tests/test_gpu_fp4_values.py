"""The values of matrices in 4 bits whose own scale is any fp32 number."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_gb300 as gns  # noqa: E402
from oracle import fp4  # noqa: E402

pytestmark = pytest.mark.gpu

# significant bits, exponent of the smallest normal number, largest number
TYPES = {torch.bfloat16: (8, -126, float(torch.finfo(torch.bfloat16).max)), torch.float16: (11, -14, 65504.0),
         torch.float32: (24, -126, float(torch.finfo(torch.float32).max))}


def rounded(v, dtype):
    """v (64 bits) rounded once to dtype, to nearest, ties to even."""
    bits, low, most = TYPES[dtype]
    step = np.exp2(np.maximum(np.frexp(v)[1] - 1, low) - (bits - 1.0))
    r = np.rint(v / step) * step
    return np.where(np.abs(r) > most, np.copysign(np.inf, v), r)


def every_value():
    """Codes and scales of a matrix that holds every code times every finite e4m3 scale: row = scale, block of 16 = the codes."""
    return np.tile(np.arange(16, dtype=np.uint8), (127, 1)), np.arange(127, dtype=np.uint8)[:, None]


def held(g):
    code, byte = every_value()
    n = len(g)
    codes = torch.from_numpy(np.repeat(fp4.pack_codes(code)[None], n, 0)).cuda()
    scales = torch.from_numpy(np.repeat(fp4.pack_scales(byte)[None], n, 0)).cuda()
    return gns.Fp4Matrix(codes, scales, torch.from_numpy(np.float32(g)).cuda(), 16)


def twice_rounded_differs(dtype, n):
    """n scales g for which some code s g rounded to fp32 first and then to dtype is not that number rounded once."""
    rng = np.random.default_rng(5)
    v = np.unique(fp4.values(*every_value(), 1.0, "nvfp4"))
    v = v[v > 0]
    got = []
    while len(got) < n:
        g = np.float32(rng.uniform(1.0, 2.0, 4096))
        p = v[None, :] * g[:, None].astype(np.float64)
        hit = (rounded(rounded(p, torch.float32), dtype) != rounded(p, dtype)).any(1)
        got.extend(g[hit])
    return np.float32(got[:n])


ENDS = np.float32([0.0, 2.0**-126, 2.0**-149, 2.0**-140, 3 * 2.0**-130, 1e-39, 1e-30, 2.0**117, 2.0**120, 2.0**126, 1.9 * 2.0**118, 2.0**127, 3.4e38])
USUAL = np.float32([0.3, 1.0, 4.25 / 2688.0, 123.0 / 2688.0, 1e-4, 7e8, 2.0**-20])


@pytest.mark.parametrize("dtype", list(TYPES), ids=str)
def test_values_are_rounded_once_whatever_the_matrix_scale(dtype):
    g = np.concatenate([ENDS, USUAL] + [twice_rounded_differs(t, 24) for t in (torch.bfloat16, torch.float16)])
    code, byte = every_value()
    got = gns.dequantize_fp4(held(g), dtype=dtype).double().cpu().numpy()
    for i, x in enumerate(g):
        want = rounded(fp4.values(code, byte, 1.0, "nvfp4") * float(x), dtype)  # (code s g has 30 bits: exact in 64)
        assert (got[i] == want).all(), (x, np.argwhere(got[i] != want)[:4])
