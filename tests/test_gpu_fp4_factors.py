"""Products in 4 bits with alpha and the matrices' scales anywhere in fp32, against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_gb300 as gns  # noqa: E402
from oracle import fp4  # noqa: E402

pytestmark = pytest.mark.gpu

# significant bits, exponent of the smallest normal number, largest number
TYPES = {torch.bfloat16: (8, -126, float(torch.finfo(torch.bfloat16).max)), torch.float16: (11, -14, 65504.0),
         torch.float32: (24, -126, float(torch.finfo(torch.float32).max))}


# alpha and the scales of a and b; the sums are from 2^-20 to about 10^7
FACTORS = [
    (1e-30, 2.0**-60, 2.0**60), (1e-30, 2.0**60, 2.0**-60), (1e30, 2.0**40, 2.0**-60), (1e30, 2.0**-60, 2.0**40),
    (1e-10, 2.0**-100, 2.0**100), (1e-10, 2.0**100, 2.0**-100), (1e10, 2.0**100, 2.0**-100), (-1e10, 2.0**-100, 2.0**100),
    (1.0, 0.3, 1e-3), (-3.7, 1e27, 1e-27), (1e-10, 1e-27, 1e27), (1.0, 2.0**-80, 2.0**-50), (1e38, 2.0**-126, 2.0**-3),
    (1e-38, 2.0**-20, 2.0**30), (1e-3, 3e-30, 4e-9), (3e38, 2.0**100, 2.0**-126), (2.0**-130, 1.0, 1.0), (2.0**-149, 2.0**120, 2.0**20),
    (1e-38, 1e-30, 1e-30), (1e38, 1e30, 1e30), (0.0, 1e30, 1e30), (0.0, 1e38, 1e38),
]


@pytest.mark.parametrize("dtype", list(TYPES), ids=str)
@pytest.mark.parametrize("alpha,ga,gb", FACTORS, ids=str)
def test_products_over_the_whole_range_of_alpha_and_scales(alpha, ga, gb, dtype):
    """alpha ga gb rounds at 2^-24, its product with the sum at 2^-24 (twice where the factor is taken in two parts), the
    sum itself as everywhere: K / 64 + 1 = 2 instructions, 2^-22 of the sum of magnitudes each. Results below the
    normal numbers of fp32 are off by half of 2^-149 twice, and then by half a step of the type."""
    rng = np.random.default_rng(9)
    m, n, k = 40, 50, 64
    parts = []
    for rows, g in ((m, ga), (n, gb)):
        code = rng.integers(0, 16, (rows, k)).astype(np.uint8)
        byte = rng.integers(1, 127, (rows, k // 16)).astype(np.uint8)
        code[1], byte[1] = 1, 1  # the smallest value there is, 2^-10
        code[2] = 0
        q = gns.Fp4Matrix(torch.from_numpy(fp4.pack_codes(code)).cuda(), torch.from_numpy(fp4.pack_scales(byte)).cuda(),
                          torch.tensor([g], dtype=torch.float32).cuda(), k)
        parts.append((q, fp4.values(code, byte, 1.0, "nvfp4")))
    (a, va), (b, vb) = parts
    f = float(np.float32(alpha)) * float(np.float32(ga)) * float(np.float32(gb))
    want, size = f * (va @ vb.T), abs(f) * (np.abs(va) @ np.abs(vb).T)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gns.fp4_gemm(a, b, alpha=alpha, dtype=dtype, status=status).double().cpu().numpy()
    eps = torch.finfo(dtype).eps / 2
    off_sum = (2 * 2.0**-22 + 4 * 2.0**-24) * size + 2.0**-149
    least = 2.0**(TYPES[dtype][1] - TYPES[dtype][0])  # half the smallest step of the type
    bound = eps * np.abs(want) * (1 + 2.0**-7) + off_sum * (1 + 2 * eps) + least
    most = TYPES[dtype][2]
    large = np.abs(want) - off_sum > most * (1 + eps)   # Inf, whichever way the sum was rounded
    small = np.abs(want) + bound < most
    assert (np.abs(got - want) <= bound)[small].all(), np.argwhere((np.abs(got - want) > bound) & small)[:4]
    assert (got[large] == np.copysign(np.inf, want[large])).all()
    assert not np.isnan(got).any() and (got[2] == 0).all() and (got[:, 2] == 0).all()
    assert int(status) == int(np.isinf(got).any())
