"""What the calls on matrices in 4 bits refuse, and where they allocate and launch: no GPU needed, nothing is launched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from fake_device import Memory, Stream, world  # noqa: E402, F401
from matrix_orthogonalizing_optimizer_gb300 import _lib, build, fp4  # noqa: E402

F32, BF16, U8, I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32


# ---- the C ABI ----


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def batch(count=2, rows=100, cols=160, ld=None, stride=None, ptr=1 << 20):
    b = _lib.GnsBatch()
    b.ptr, b.count, b.rows, b.cols = ptr, count, rows, cols
    b.ld = (cols + 31) // 32 * 32 if ld is None else ld
    b.stride = rows * b.ld if stride is None else stride
    return b


def held(count=2, rows=100, cols=160, fmt=_lib.GNS_NVFP4, scales=1 << 24, scale_stride=None, g=1 << 25, **kw):
    q = _lib.GnsFp4()
    q.codes = batch(count, rows, cols, **kw)
    q.scales, q.format = scales, fmt
    q.scale_stride = 1 << 20 if scale_stride is None else scale_stride
    q.tensor_scale = g if fmt == _lib.GNS_NVFP4 else None
    return q


R = ctypes.byref


def refused(rc, *words):
    text = _lib.last_error()
    assert rc in (_lib.GNS_ERR_INVALID, _lib.GNS_ERR_UNSUPPORTED) and all(w in text for w in words), (rc, text)


def test_scale_bytes(lib):
    assert lib.gns_fp4_scale_bytes(1, 1, _lib.GNS_NVFP4) == 512
    assert lib.gns_fp4_scale_bytes(129, 65, _lib.GNS_NVFP4) == 2 * 2 * 512
    assert lib.gns_fp4_scale_bytes(128, 65, _lib.GNS_MXFP4) == 512
    assert lib.gns_fp4_scale_bytes(128, 129, _lib.GNS_MXFP4) == 1024
    for args in ((0, 5, 0), (5, 0, 0), (5, 5, 2), (1 << 40, 1 << 40, 0)):
        assert lib.gns_fp4_scale_bytes(*args) == 0


BAD_HELD = [
    (dict(fmt=7), "format"), (dict(ld=168), "32"), (dict(stride=100 * 160 + 8), "32"), (dict(ptr=(1 << 20) + 8), "aligned"),
    (dict(ptr=0), "null"), (dict(scales=0), "scales"), (dict(scales=(1 << 24) + 4), "scales"), (dict(scale_stride=520), "multiple of 16"),
    (dict(scale_stride=512 * 2), "scale_stride"), (dict(g=0), "tensor_scale"), (dict(g=(1 << 25) + 2), "tensor_scale"), (dict(rows=0), ">= 1"),
    (dict(ld=128), "ld < cols"), (dict(count=65536), "too large"),
]


@pytest.mark.parametrize("kw,word", BAD_HELD, ids=str)
def test_every_call_checks_what_is_held(lib, kw, word):
    q = held(**kw)
    x, d = batch(rows=q.codes.rows or 1, count=2), batch(2, 100, 100, ptr=1 << 22)
    refused(lib.gns_fp4_quantize(R(x), _lib.GNS_BF16, R(q), None, None, None, None), word)
    refused(lib.gns_fp4_quantize(R(x), _lib.GNS_BF16, None, R(q), None, None, None), word)
    refused(lib.gns_fp4_dequantize(R(q), R(x), _lib.GNS_F16, None), word)
    refused(lib.gns_fp4_gemm(R(q), R(held()), None, R(d), 1.0, 0.0, _lib.GNS_F32, None, None), "a", word)
    refused(lib.gns_fp4_gemm(R(held()), R(q), None, R(d), 1.0, 0.0, _lib.GNS_F32, None, None), "b", word)
    refused(lib.gns_fp4_sym_gemm_xxt(R(q), None, R(d), 1.0, 0.0, _lib.GNS_F32, None, None), "x", word)


def test_quantize_refuses(lib):
    x, q, qt = batch(ptr=1 << 26), held(), held(rows=160, cols=100, ptr=1 << 21, scales=1 << 23, g=1 << 19)
    call = lambda x=x, q=q, qt=qt, amax=None, dt=_lib.GNS_BF16: lib.gns_fp4_quantize(  # noqa: E731
        R(x), dt, R(q) if q else None, R(qt) if qt else None, amax, None, None)
    refused(call(dt=9), "dtype")
    refused(call(q=None, qt=None), "one of them")
    refused(call(q=held(rows=99)), "shape of x")
    refused(call(qt=held()), "transpose")
    refused(call(qt=held(rows=160, cols=100, fmt=_lib.GNS_MXFP4, ptr=1 << 21, scales=1 << 23)), "one format")
    refused(call(qt=held(rows=160, cols=100, ptr=1 << 20, scales=1 << 23, g=1 << 19)), "share")
    refused(call(qt=held(rows=160, cols=100, ptr=1 << 21, g=1 << 19)), "share")
    refused(call(qt=held(rows=160, cols=100, ptr=1 << 21, scales=1 << 23)), "share")
    refused(call(x=batch(ptr=1 << 20)), "alias")
    refused(call(x=batch(ld=164, ptr=1 << 26)), "16 bytes")
    refused(call(q=held(fmt=_lib.GNS_MXFP4), qt=None, amax=1 << 18), "amax")
    mx = held(fmt=_lib.GNS_MXFP4)
    mx.tensor_scale = 1 << 25
    refused(call(q=mx, qt=None), "tensor_scale")


def test_dequantize_refuses(lib):
    refused(lib.gns_fp4_dequantize(R(held()), R(batch(ptr=1 << 26)), 5, None), "dtype")
    refused(lib.gns_fp4_dequantize(R(held()), R(batch(cols=128, ptr=1 << 26)), _lib.GNS_BF16, None), "shape of q")
    refused(lib.gns_fp4_dequantize(R(held()), R(batch()), _lib.GNS_BF16, None), "alias")


def test_products_refuse(lib):
    a, b = held(), held(rows=64, ptr=1 << 21)
    c, d = batch(2, 100, 64, ptr=1 << 22), batch(2, 100, 64, ptr=1 << 23)

    def call(a=a, b=b, c=c, d=d, alpha=1.0, beta=0.0, dt=_lib.GNS_BF16):
        return lib.gns_fp4_gemm(R(a), R(b), R(c) if c is not None else None, R(d), alpha, beta, dt, None, None)

    refused(call(dt=4), "dtype")
    refused(call(b=held(rows=64, ptr=1 << 21, fmt=_lib.GNS_MXFP4)), "one format")
    refused(call(b=held(count=1, rows=64, ptr=1 << 21)), "counts")
    refused(call(b=held(rows=64, cols=128, ptr=1 << 21)), "long rows")
    refused(call(d=batch(2, 64, 100, ptr=1 << 23)), "rows of a")
    refused(call(alpha=float("nan")), "finite")
    refused(call(beta=float("inf")), "finite")
    refused(call(beta=1.0, c=None), "c is required")
    refused(call(beta=1.0, c=batch(2, 100, 96, ptr=1 << 22)), "shape of d")
    refused(call(beta=1.0, c=batch(2, 100, 64, ld=96, ptr=1 << 23)), "same ld")
    refused(call(d=batch(2, 100, 64, ptr=1 << 20)), "alias")
    refused(call(d=batch(2, 100, 64, ptr=1 << 24)), "alias")
    refused(lib.gns_fp4_sym_gemm_xxt(R(a), None, R(batch(2, 100, 64, ptr=1 << 23)), 1.0, 0.0, _lib.GNS_BF16, None, None), "rows of x")


# ---- Python ----


@pytest.fixture
def gpu(world, monkeypatch):  # noqa: F811
    monkeypatch.setattr(fp4, "load", lambda: world["library"])
    return world


def mem(shape, dtype, index=0):
    return Memory(shape, dtype, torch.device("cuda", index))


def matrix(rows=100, cols=160, count=2, fmt="nvfp4", index=0):
    g = mem((count,), F32, index) if fmt == "nvfp4" else None
    tiles = fp4._tiles(rows, cols, fmt)
    return fp4.Fp4Matrix(mem((count, rows, -(-cols // 32) * 16), U8, index), mem((count, *tiles), U8, index), g, cols, fmt)


def status(index=0):
    return mem(1, I32, index)


def test_fp4_matrix_refuses(gpu):
    codes, scales, g = mem((2, 100, 80), U8), mem((2, 1, 3, 512), U8), mem((2,), F32)
    assert fp4.Fp4Matrix(codes, scales, g, 160).shape == (2, 100, 160)
    assert fp4.Fp4Matrix(codes, scales, g, 129).shape == (2, 100, 129)
    for args, error in [((codes, scales, g, 161), "bytes a row"), ((codes, scales, g, 0), "bytes a row"),
                        ((codes, mem((2, 1, 2, 512), U8), g, 160), "shape"), ((codes, scales, None, 160), "tensor_scale"),
                        ((codes, scales, mem((1,), F32), 160), "tensor_scale"), ((codes, scales, mem((2,), BF16), 160), "tensor_scale"),
                        ((codes, scales, g, 160, "fp4"), "fmt"), ((codes, mem((2, 1, 2, 512), U8), g, 160, "mxfp4"), "tensor_scale"),
                        ((codes, mem((2, 1, 3, 512), U8, 1), g, 160), "scales must be on"),
                        ((codes, scales, mem((2,), F32, 1), 160), "tensor_scale must be on"), ((mem((100,), U8), scales, g, 160), "2-D")]:
        with pytest.raises(ValueError, match=error):
            fp4.Fp4Matrix(*args)
    with pytest.raises(TypeError):
        fp4.Fp4Matrix(mem((2, 100, 80), I32), scales, g, 160)
    for shape in ((3,), (0, 5), (2, 0, 5)):
        with pytest.raises(ValueError, match="shape"):
            fp4.empty_fp4(shape)


def quantize(gpu, index=0, **kw):
    return fp4.quantize_fp4(**{"x": mem((2, 100, 160), BF16, index), "status": status(index), **kw})


def dequantize(gpu, index=0, **kw):
    return fp4.dequantize_fp4(**{"q": matrix(index=index), **kw})


def gemm(gpu, index=0, **kw):
    return fp4.fp4_gemm(**{"a": matrix(index=index), "b": matrix(64, index=index), "status": status(index), **kw})


def gram(gpu, index=0, **kw):
    return fp4.fp4_sym_gemm_xxt(**{"x": matrix(index=index), "status": status(index), **kw})


STREAM = lambda i: Stream("side", i)  # noqa: E731
ELSEWHERE = [
    (quantize, "out", lambda i: matrix(index=i)), (quantize, "out_t", lambda i: matrix(160, 100, index=i)),
    (quantize, "amax", lambda i: mem((2,), F32, i)), (quantize, "status", status), (quantize, "stream", STREAM),
    (dequantize, "out", lambda i: mem((2, 100, 160), F32, i)), (dequantize, "stream", STREAM),
    (gemm, "b", lambda i: matrix(64, index=i)), (gemm, "c", lambda i: mem((2, 100, 64), BF16, i)),
    (gemm, "d", lambda i: mem((2, 100, 64), BF16, i)), (gemm, "status", status), (gemm, "stream", STREAM),
    (gram, "c", lambda i: mem((2, 100, 100), BF16, i)), (gram, "d", lambda i: mem((2, 100, 100), BF16, i)),
    (gram, "status", status), (gram, "stream", STREAM),
]


@pytest.mark.parametrize("call,name,make", ELSEWHERE, ids=[f"{c.__name__}-{n}" for c, n, _ in ELSEWHERE])
def test_what_lies_on_another_device_is_refused(gpu, call, name, make):
    call(gpu, **{name: make(0)})
    assert len(gpu["library"].calls) == 1
    with pytest.raises(ValueError, match=name):
        call(gpu, **{name: make(1)})
    assert len(gpu["library"].calls) == 1


@pytest.mark.parametrize("call,name", [(quantize, "gns_fp4_quantize"), (dequantize, "gns_fp4_dequantize"), (gemm, "gns_fp4_gemm"),
                                       (gram, "gns_fp4_sym_gemm_xxt")])
@pytest.mark.parametrize("index", [0, 1])
def test_calls_launch_on_the_device_of_their_tensors(gpu, call, name, index):
    call(gpu, index)
    assert gpu["library"].calls == [(name, index)]


@pytest.mark.parametrize("call", [quantize, dequantize, gemm, gram])
def test_outputs_come_from_the_pool_of_the_calls_stream(gpu, call):
    side = Stream("side")
    call(gpu, stream=side)
    made = [t for t in gpu["made"] if t.shape]  # (a scalar on the host tells the size of a type)
    assert made and all(t.stream is side and t.recorded == [gpu["here"]] for t in made)


def test_python_refuses(gpu):
    with pytest.raises(ValueError, match="fmt"):
        quantize(gpu, fmt="e2m1")
    with pytest.raises(ValueError, match="axes"):
        quantize(gpu, axes="k")
    with pytest.raises(ValueError, match="format"):
        quantize(gpu, fmt="mxfp4", out=matrix())
    with pytest.raises(ValueError, match="amax"):
        quantize(gpu, amax=mem((1,), F32))
    with pytest.raises(TypeError, match="out must be"):
        quantize(gpu, out=mem((2, 100, 160), U8))
    for call, name in ((dequantize, "q"), (gemm, "a"), (gemm, "b"), (gram, "x")):
        with pytest.raises(TypeError, match=name):
            call(gpu, **{name: mem((2, 100, 160), BF16)})
    with pytest.raises(ValueError, match="c is required"):
        gemm(gpu, beta=1.0)
    with pytest.raises(TypeError, match="type"):
        gemm(gpu, beta=1.0, c=mem((2, 100, 64), F32), d=mem((2, 100, 64), BF16))
    with pytest.raises(TypeError, match="type"):
        gemm(gpu, dtype=F32, d=mem((2, 100, 64), BF16))
    assert gpu["library"].calls == []


def test_types_of_new_results(gpu):
    assert gemm(gpu).dtype == BF16
    assert gemm(gpu, dtype=F32).dtype == F32
    assert gemm(gpu, c=mem((2, 100, 64), torch.float16), beta=1.0).dtype == torch.float16
    assert dequantize(gpu, dtype=F32).dtype == F32
    q, qt = quantize(gpu, axes="both")
    assert q.shape == (2, 100, 160) and qt.shape == (2, 160, 100)
    assert quantize(gpu, fmt="mxfp4", axes="cols").tensor_scale is None
