"""Matrices in 4 bits at the ends of what the calls take: more than 2^31 values, the longest rows and columns, the most matrices,
MXFP4's whole range of scales, and parts of what is held."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_gb300 as gns  # noqa: E402
from oracle import fp4  # noqa: E402
from test_gpu_fp4 import FORMATS, check_product, held_exactly, matrices, oracle_values, padded, random_held  # noqa: E402

pytestmark = pytest.mark.gpu


def same(a, b):
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    assert a.tensor_scale is None or torch.equal(a.tensor_scale, b.tensor_scale)


def test_more_than_two_to_the_31_values():
    """The last rows and columns, against a call on them alone."""
    rows, cols = 547 * 128, 33024
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    assert x.numel() > 2**31
    amax = x.abs().max().float().view(1)
    q, qt = gns.quantize_fp4(x, axes="both")
    same(q, gns.quantize_fp4(x, amax=amax))
    last = gns.quantize_fp4(x[-256:], amax=amax)
    assert torch.equal(q.codes[-256:], last.codes) and torch.equal(q.scales[-2:], last.scales)
    right = gns.quantize_fp4(x[:, -256:].contiguous(), axes="cols", amax=amax)
    assert torch.equal(qt.codes[-256:], right.codes) and torch.equal(qt.scales[-2:], right.scales)
    del qt
    v = gns.dequantize_fp4(q)
    assert torch.equal(v[-256:], gns.dequantize_fp4(last)) and torch.equal(v[:256], gns.dequantize_fp4(gns.quantize_fp4(x[:256], amax=amax)))
    del v, q
    # a result of that size, with an addend (K = 64: one matrix instruction, the same sum in every tiling)
    a, b = gns.quantize_fp4(x[:, :64].contiguous()), gns.quantize_fp4(x[:cols, 64:128].contiguous())
    d = gns.fp4_gemm(a, b, c=x, beta=0.5)
    end = gns.Fp4Matrix(a.codes[-256:], a.scales[-2:], a.tensor_scale, 64)
    assert torch.equal(d[-256:], gns.fp4_gemm(end, b, c=x[-256:], beta=0.5))


@pytest.mark.parametrize("fmt", FORMATS)
def test_the_longest_columns_and_rows(fmt):
    x = matrices(101, (1, 4194240, 3), "bf16", spread=0.5)
    x64 = x.double().numpy()
    q, qt = gns.quantize_fp4(padded(x), fmt, axes="both")
    held_exactly(q, x64)
    held_exactly(qt, x64.transpose(0, 2, 1))
    v, vt = (gns.dequantize_fp4(t, dtype=torch.float32) for t in (q, qt))
    assert torch.equal(v.cpu().double(), torch.from_numpy(oracle_values(x64, fmt)))
    want = oracle_values(x64.transpose(0, 2, 1), fmt)
    assert torch.equal(vt.cpu().double(), torch.from_numpy(want))
    check_product(gns.fp4_gemm(qt, qt, dtype=torch.float32), want, want, "f32")
    w, vw = random_held(102, (1, 5, 3), fmt)
    check_product(gns.fp4_gemm(q, w, dtype=torch.bfloat16), v.cpu().double().numpy(), vw, "bf16")


@pytest.mark.parametrize("fmt", FORMATS)
def test_the_most_matrices(fmt):
    x = padded(matrices(103, (65535, 2, 17), "bf16"))
    q, qt = gns.quantize_fp4(x, fmt, axes="both")
    d, r = gns.fp4_gemm(q, q), gns.fp4_sym_gemm_xxt(qt)
    v, vt = gns.dequantize_fp4(q), gns.dequantize_fp4(qt)
    for part in (slice(0, 3), slice(32766, 32770), slice(65530, 65535)):
        p, pt = gns.quantize_fp4(x[part], fmt, axes="both")
        for whole, some in ((q, p), (qt, pt)):
            assert torch.equal(whole.codes[part], some.codes) and torch.equal(whole.scales[part], some.scales)
        held_exactly(p, x[part].double().cpu().numpy())
        for whole, some in ((d, gns.fp4_gemm(p, p)), (r, gns.fp4_sym_gemm_xxt(pt)), (v, gns.dequantize_fp4(p)), (vt, gns.dequantize_fp4(pt))):
            assert torch.equal(whole[part], some)


def test_mxfp4_scales_from_end_to_end():
    """Blocks of the scale 2^(a - 127) times blocks of the scale 2^(b - 127), for all a and b with products that fp32 holds: each
    sum is one product, of 4 bits times a power of two."""
    code = np.zeros((255 * 2, 32), dtype=np.uint8)
    code[0::2, 5], code[1::2, 5] = 7, 9  # 6 and -0.5
    byte = np.repeat(np.arange(255, dtype=np.uint8), 2)[:, None]
    q = gns.Fp4Matrix(torch.from_numpy(fp4.pack_codes(code)).cuda(), torch.from_numpy(fp4.pack_scales(byte)).cuda(), None, 32, "mxfp4")
    v = fp4.values(code, byte, None, "mxfp4")[:, 5]
    assert torch.equal(gns.dequantize_fp4(q, dtype=torch.float32).cpu().double()[:, 5], torch.from_numpy(v).float().double())
    want = v[:, None] * v[None, :]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gns.fp4_gemm(q, q, dtype=torch.float32, status=status).double().cpu().numpy()
    assert int(status) == 1  # those beyond fp32
    normal = (np.abs(want) >= 2.0**-126) & (np.abs(want) < 2.0**128)
    np.testing.assert_array_equal(got[normal], want[normal])
    assert (np.abs(got[np.abs(want) < 2.0**-126]) <= 2.0**-126).all()  # below the normal numbers: that or nothing
    assert np.isinf(got[np.abs(want) >= 2.0**128]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_parts_of_what_is_held(fmt):
    """Matrices of a batch, and rows from a multiple of 128 on, are matrices again."""
    x = padded(matrices(104, (5, 300, 200), "bf16"))
    q = gns.quantize_fp4(x, fmt)
    g = q.tensor_scale
    some = gns.Fp4Matrix(q.codes[1:4], q.scales[1:4], None if g is None else g[1:4], 200, fmt)
    rows = gns.Fp4Matrix(q.codes[:, 128:], q.scales[:, 1:], g, 200, fmt)
    d = gns.fp4_gemm(q, q, dtype=torch.float32)
    assert torch.equal(gns.fp4_gemm(some, some, dtype=torch.float32), d[1:4])
    assert torch.equal(gns.fp4_gemm(rows, q, dtype=torch.float32), d[:, 128:])
    assert torch.equal(gns.fp4_sym_gemm_xxt(rows, dtype=torch.float32), d[:, 128:, 128:])
    assert torch.equal(gns.dequantize_fp4(rows), gns.dequantize_fp4(q)[:, 128:])
    one = gns.Fp4Matrix(q.codes[3], q.scales[3], None if g is None else g[3:4], 200, fmt)
    assert torch.equal(gns.fp4_gemm(one, one, dtype=torch.float32), d[3])


@pytest.mark.parametrize("fmt", FORMATS)
def test_scales_that_are_not_read(fmt):
    """A batch of few rows whose tiles hold NaN in all scales behind the last row, in every tiling of B's rows."""
    for m, n, k in ((1, 1, 32), (5, 65, 300), (33, 129, 700), (127, 193, 513)):
        a, va = random_held(105, (2, m, k), fmt)
        b, vb = random_held(106, (2, n, k), fmt)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        check_product(gns.fp4_gemm(a, b, dtype=torch.float32, status=status), va, vb, "f32")
        assert int(status) == 0
