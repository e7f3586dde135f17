"""The operators on matrices in microscaled 4-bit floating point that are measured, and on what.

  quantize    a batch of matrices into 4 bits, along its rows, its columns or both, and back into values
  dequantize  the values of a batch that is held in 4 bits
  gemm        D = alpha A B^T + beta C of two batches held in 4 bits
  gram        D = alpha X X^T + beta C of one
  linear      a layer's product: the activations into 4 bits, then times weights held in 4 bits
  step        the three products of a layer's training step, all operands brought into 4 bits on the way

A value is held as one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} times the scale of its block:
  nvfp4  blocks of 16 along a row; scales in e4m3 (4 bits of exponent, 3 of mantissa), times one power of two of the matrix
  mxfp4  blocks of 32 along a row; scales are powers of two in 8 bits
Two codes share a byte (the first in the low half); a row takes a multiple of 16 bytes. Scales lie in tiles
of 128 rows x 4 blocks, 512 bytes each: row r, block k at (r % 32) * 16 + (r / 32) * 4 + k.
Everything behind a row's last value and behind the last block is zero.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def listed():
    return [
        # one matrix of 128 x 512, the smallest that the framework orthogonalizes: a call that is all latency
        {"name": "quantize-matrix-f32", "op": "quantize", "fmt": "nvfp4", "count": 1, "rows": 128, "cols": 512, "dtype": "f32", "axes": "rows"},
        # a ragged batch, along both axes, rows padded to 16 bytes
        {"name": "quantize-ragged-f16", "op": "quantize", "fmt": "mxfp4", "count": 7, "rows": 1001, "cols": 1333, "dtype": "f16", "axes": "both"},
        # sixteen experts' projections after their optimizer step, for the forward and the backward product: the largest
        {"name": "quantize-experts-bf16", "op": "quantize", "fmt": "nvfp4", "count": 16, "rows": 2048, "cols": 8192, "dtype": "bf16", "axes": "both"},
        # an MLP projection read back for a path without 4-bit products
        {"name": "dequantize-layer-bf16", "op": "dequantize", "fmt": "nvfp4", "count": 1, "rows": 11008, "cols": 4096, "dtype": "bf16"},
        # odd sizes into f32
        {"name": "dequantize-ragged-f32", "op": "dequantize", "fmt": "mxfp4", "count": 5, "rows": 777, "cols": 1291, "dtype": "f32"},
        # one token through an MLP projection: the weights are read once and nothing else counts
        {"name": "gemm-token-bf16", "op": "gemm", "fmt": "nvfp4", "count": 1, "m": 1, "n": 4096, "k": 11008, "dtype": "bf16", "beta": 0.0},
        # a decoding batch of odd size, added to what is there
        {"name": "gemm-decode-f16", "op": "gemm", "fmt": "mxfp4", "count": 1, "m": 41, "n": 11008, "k": 4096, "dtype": "f16", "beta": 1.0},
        # 16384 tokens through an MLP projection: the largest
        {"name": "gemm-layer-bf16", "op": "gemm", "fmt": "nvfp4", "count": 1, "m": 16384, "n": 11008, "k": 4096, "dtype": "bf16", "beta": 0.0},
        # the Gram matrices of the benchmark's batch
        {"name": "gram-batch-bf16", "op": "gram", "fmt": "nvfp4", "count": 24, "rows": 1024, "cols": 4096, "dtype": "bf16", "beta": 0.0},
        # Gram matrices of odd sizes, added to f32 ones
        {"name": "gram-ragged-f32", "op": "gram", "fmt": "mxfp4", "count": 5, "rows": 333, "cols": 2001, "dtype": "f32", "beta": 0.5},
        # four tokens' activations into 4 bits and through a projection: latency again, two calls
        {"name": "linear-tokens-bf16", "op": "linear", "fmt": "nvfp4", "m": 4, "n": 11008, "k": 4096, "dtype": "bf16"},
        # a training step's products for 4096 tokens: y = x w^T, dx = dy w, dw = dy^T x
        {"name": "step-layer-bf16", "op": "step", "fmt": "nvfp4", "m": 4096, "n": 11008, "k": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "dequantize", "gemm", "gemm", "gemm", "gram", "linear", "step"])
    c = {"op": op, "fmt": rng.choice(["nvfp4", "mxfp4"]), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op in ("quantize", "dequantize"):
        rows = _log(rng, 1, 16384)
        cols = _log(rng, 1, min(16384, 1.5e8 / rows))
        c.update(count=_log(rng, 1, max(1, min(256, 1.5e8 / (rows * cols)))), rows=rows, cols=cols)
        if op == "quantize":
            c["axes"] = rng.choice(["rows", "cols", "both"])
    elif op == "gram":
        rows, cols = _log(rng, 2, 2048), _log(rng, 16, 16384)
        c.update(count=_log(rng, 1, max(1, min(64, 2e11 / (rows * rows * cols), 1e8 / (rows * cols)))), rows=rows, cols=cols, beta=rng.choice([0.0, 0.0, 0.5]))
    else:
        n, k = _log(rng, 16, 11008), _log(rng, 16, 11008)
        most = 1.7e11 if op == "step" else 7e11
        m = _log(rng, 1, 64) if rng.random() < 0.5 else _log(rng, 64, min(16384, most / (n * k)))
        if op == "gemm":
            c.update(count=_log(rng, 1, max(1, min(64, 5e11 / (m * n * k), 5e7 / (n * k), 5e7 / (m * n)))), beta=rng.choice([0.0, 0.0, 1.0]))
        c.update(m=m, n=n, k=k)
    return c


# ---- what is held in 4 bits, in plain form ----


def _pow2(e):
    """2^e in f32 for whole e from -149 up to 127."""
    e = e.to(torch.int32)
    return torch.where(e >= -126, ((e + 127).clamp(min=1) << 23).view(torch.float32), ((1 << 22) >> (-127 - e).clamp(0, 22)).to(torch.int32).view(torch.float32))


def _exponent(a):
    """floor(log2(a)) of a > 0."""
    return torch.frexp(a)[1] - 1


def quantize_plain(x, fmt):
    """(magnitudes' indices 0 .. 7 plus 8 for the negative, scales' bytes, the matrices' own scales) of x (count, rows, cols)."""
    x = x.float()
    count, rows, cols = x.shape
    block = BLOCK[fmt]
    blocks = -(-cols // block)
    x = torch.nn.functional.pad(x, (0, blocks * block - cols))
    own_scale = None
    if fmt == "nvfp4":
        # the smallest power of two that keeps the largest block's scale within e4m3: 6 * 448 = 1.3125 * 2^11
        most = x.abs().amax((1, 2))
        e = _exponent(most)
        over = (most * _pow2((-e).clamp(max=126)) > 1.3125).to(torch.int32)
        own_scale = torch.where(most > 0, _pow2((e - 11 + over).clamp(min=-126)), 0.0)
        x = torch.where(most[:, None, None] > 0, x / own_scale[:, None, None], 0.0)
    x = x.view(count, rows, blocks, block)
    most = x.abs().amax(3)
    if fmt == "nvfp4":
        scale8 = (most / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        scale = scale8.float()
        a = torch.where(scale[..., None] > 0, x.abs() / scale[..., None], 0.0)
        scales = scale8.view(torch.uint8)
    else:
        e = torch.where(most > 0, (_exponent(most) - 2).clamp(min=-127), -127)
        a = x.abs() * _pow2(-e)[..., None]
        scales = (e + 127).to(torch.uint8)
    index = (a > 0.25).to(torch.uint8)  # the nearest; between two, the one whose last bit is 0
    for border, reached in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        index += (a >= border) if reached else (a > border)
    index = torch.where((x < 0), index + 8, index)
    return index.view(count, rows, blocks * block), scales, own_scale


def pack(index, scales, cols):
    """The codes' bytes and the scales' tiles."""
    count, rows, have = index.shape
    index = torch.nn.functional.pad(index, (0, -(-cols // 32) * 32 - have))
    codes = index[..., 0::2] | (index[..., 1::2] << 4)
    blocks = scales.shape[2]
    tr, tk = -(-rows // 128), -(-blocks // 4)
    scales = torch.nn.functional.pad(scales, (0, tk * 4 - blocks, 0, tr * 128 - rows))
    tiles = scales.view(count, tr, 4, 32, tk, 4).permute(0, 1, 4, 3, 2, 5).reshape(count, tr, tk, 512)
    return codes.contiguous(), tiles.contiguous()


def values_of(index, scales, own_scale, fmt, cols):
    """The values in f32 that indices and scales stand for."""
    count, rows, blocks = scales.shape
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=index.device)
    v = table[index.long()].view(count, rows, blocks, BLOCK[fmt])
    s = scales.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else _pow2(scales.to(torch.int32) - 127)
    v = (v * s[..., None]).view(count, rows, blocks * BLOCK[fmt])[..., :cols]
    return v if own_scale is None else v * own_scale[:, None, None]


def unpack(codes, tiles, rows, cols, fmt):
    """Indices and scales' bytes out of what pack() laid out."""
    count = codes.shape[0]
    blocks = -(-cols // BLOCK[fmt])
    index = torch.stack([codes & 15, codes >> 4], 3).view(count, rows, -1)[..., : blocks * BLOCK[fmt]]
    tr, tk = tiles.shape[1:3]
    scales = tiles.view(count, tr, tk, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(count, tr * 128, tk * 4)
    return index, scales[:, :rows, :blocks].contiguous()


def read_plain(h):
    """The values in f32 of a batch held in 4 bits."""
    index, scales = unpack(h["codes"], h["scales"], h["rows"], h["cols"], h["fmt"])
    return values_of(index, scales, h["own_scale"], h["fmt"], h["cols"])


def through_plain(x, fmt):
    """The values in f32 of x (count, rows, cols) after it went through 4 bits."""
    index, scales, own_scale = quantize_plain(x, fmt)
    return values_of(index, scales, own_scale, fmt, x.shape[2])


# ---- inputs ----


def _matrices(gen, count, rows, cols, dtype, std):
    """(count, rows, cols), rows on 16-byte boundaries; columns differ in size, as activations' and weights' do."""
    step = 16 // dtype.itemsize
    t = torch.empty((count, rows, -(-cols // step) * step), dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)[..., :cols]
    return t.mul_(torch.empty(cols, device="cuda").normal_(0.0, 0.7, generator=gen).exp_().to(dtype))


def _held(gen, count, rows, cols, fmt, std):
    """A batch held in 4 bits, as an earlier call has left it."""
    x = _matrices(gen, count, rows, cols, torch.bfloat16, std)
    index, scales, own_scale = quantize_plain(x, fmt)
    codes, tiles = pack(index, scales, cols)
    h = {"codes": codes, "scales": tiles, "own_scale": own_scale, "rows": rows, "cols": cols, "fmt": fmt}
    if own:
        import matrix_orthogonalizing_optimizer_gb300 as gns

        h["matrix"] = gns.Fp4Matrix(codes, tiles, own_scale, cols, fmt)
    return h


def _symmetric(gen, count, n, dtype, std):
    step = 16 // dtype.itemsize
    c = torch.empty((count, n, -(-n // step) * step), dtype=dtype, device="cuda")[..., :n]
    v = torch.empty((count, n, n), device="cuda").normal_(0.0, std, generator=gen)
    return c.copy_(torch.triu(v) + torch.triu(v, 1).mT)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, fmt, dtype = case["op"], case["fmt"], DTYPES[case["dtype"]]
    s = {"case": case, "dtype": dtype}
    if op == "quantize":
        s["x"] = _matrices(gen, case["count"], case["rows"], case["cols"], dtype, 0.02)
    elif op == "dequantize":
        s["q"] = _held(gen, case["count"], case["rows"], case["cols"], fmt, 0.02)
    elif op == "gemm":
        s["a"] = _held(gen, case["count"], case["m"], case["k"], fmt, 1.0)
        s["b"] = _held(gen, case["count"], case["n"], case["k"], fmt, 1.0 / math.sqrt(case["k"]))
        s["alpha"] = 1.0
        s["c"] = _matrices(gen, case["count"], case["m"], case["n"], dtype, 1.0) if case["beta"] else None
    elif op == "gram":
        s["x"] = _held(gen, case["count"], case["rows"], case["cols"], fmt, 1.0)
        s["alpha"] = 1.0 / case["cols"]
        s["c"] = _symmetric(gen, case["count"], case["rows"], dtype, 1.0) if case["beta"] else None
    elif op == "linear":
        s["x"] = _matrices(gen, 1, case["m"], case["k"], dtype, 1.0)
        s["w"] = _held(gen, 1, case["n"], case["k"], fmt, 1.0 / math.sqrt(case["k"]))
    else:
        s["x"] = _matrices(gen, 1, case["m"], case["k"], dtype, 1.0)
        s["w"] = _matrices(gen, 1, case["n"], case["k"], dtype, 1.0 / math.sqrt(case["k"]))
        s["dy"] = _matrices(gen, 1, case["m"], case["n"], dtype, 0.01)
    if own:  # the buffers that a program keeps from step to step
        import matrix_orthogonalizing_optimizer_gb300 as gns

        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        held = lambda count, rows, cols: gns.empty_fp4((count, rows, cols), fmt, "cuda")  # noqa: E731
        plane = lambda count, rows, cols: gns.empty_padded((count, rows, cols), dtype, "cuda")  # noqa: E731
        if op == "quantize":
            count, rows, cols = case["count"], case["rows"], case["cols"]
            s["q"] = held(count, rows, cols) if case["axes"] != "cols" else None
            s["qt"] = held(count, cols, rows) if case["axes"] != "rows" else None
            s["v"] = plane(count, rows, cols) if s["q"] else None
            s["vt"] = plane(count, cols, rows) if s["qt"] else None
        elif op == "dequantize":
            s["v"] = plane(case["count"], case["rows"], case["cols"])
        elif op in ("gemm", "gram"):
            m, n = (case["m"], case["n"]) if op == "gemm" else (case["rows"], case["rows"])
            s["d"] = plane(case["count"], m, n)
        else:
            m, n, k = case["m"], case["n"], case["k"]
            s["d"], s["xq"] = plane(1, m, n), held(1, m, k)
            if op == "step":
                s["dx"], s["dw"] = plane(1, m, k), plane(1, n, k)
                s["xt"], s["wq"], s["wt"], s["gq"], s["gt"] = held(1, k, m), held(1, n, k), held(1, k, n), held(1, m, n), held(1, n, m)
    return s


# ---- a pass ----


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import matrix_orthogonalizing_optimizer_gb300 as gns

    case, status = s["case"], s["status"]
    op, fmt = case["op"], case["fmt"]
    if op == "quantize":
        gns.quantize_fp4(s["x"], fmt, out=s["q"], out_t=s["qt"], status=status)
        return {n: gns.dequantize_fp4(s[q], out=s[n]) for q, n in (("q", "v"), ("qt", "vt")) if s[q] is not None}
    if op == "dequantize":
        return {"v": gns.dequantize_fp4(s["q"]["matrix"], out=s["v"])}
    if op == "gemm":
        return {"d": gns.fp4_gemm(s["a"]["matrix"], s["b"]["matrix"], c=s["c"], d=s["d"], alpha=s["alpha"], beta=case["beta"], status=status)}
    if op == "gram":
        return {"d": gns.fp4_sym_gemm_xxt(s["x"]["matrix"], c=s["c"], d=s["d"], alpha=s["alpha"], beta=case["beta"], status=status)}
    if op == "linear":
        gns.quantize_fp4(s["x"], fmt, out=s["xq"], status=status)
        return {"y": gns.fp4_gemm(s["xq"], s["w"]["matrix"], d=s["d"], status=status)}
    gns.quantize_fp4(s["x"], fmt, out=s["xq"], out_t=s["xt"], status=status)
    gns.quantize_fp4(s["w"], fmt, out=s["wq"], out_t=s["wt"], status=status)
    y = gns.fp4_gemm(s["xq"], s["wq"], d=s["d"], status=status)
    gns.quantize_fp4(s["dy"], fmt, out=s["gq"], out_t=s["gt"], status=status)
    dx = gns.fp4_gemm(s["gq"], s["wt"], d=s["dx"], status=status)
    return {"y": y, "dx": dx, "dw": gns.fp4_gemm(s["gt"], s["xt"], d=s["dw"], status=status)}


def run_plain(s):
    case, dtype = s["case"], s["dtype"]
    op, fmt = case["op"], case["fmt"]
    if op == "quantize":
        got = {}
        if case["axes"] != "cols":
            got["v"] = through_plain(s["x"], fmt).to(dtype)
        if case["axes"] != "rows":
            got["vt"] = through_plain(s["x"].mT, fmt).to(dtype)
        return got
    if op == "dequantize":
        return {"v": read_plain(s["q"]).to(dtype)}
    if op in ("gemm", "gram"):
        a = read_plain(s["a"] if op == "gemm" else s["x"])
        d = s["alpha"] * (a @ (read_plain(s["b"]) if op == "gemm" else a).mT)
        if case["beta"]:
            d = d + case["beta"] * s["c"].float()
        return {"d": d.to(dtype)}
    if op == "linear":
        return {"y": (through_plain(s["x"], fmt) @ read_plain(s["w"]).mT).to(dtype)}
    x, w, dy = s["x"], s["w"], s["dy"]
    return {
        "y": (through_plain(x, fmt) @ through_plain(w, fmt).mT).to(dtype),
        "dx": (through_plain(dy, fmt) @ through_plain(w.mT, fmt).mT).to(dtype),
        "dw": (through_plain(dy.mT, fmt) @ through_plain(x.mT, fmt).mT).to(dtype),
    }


def work(case):
    op, size, block = case["op"], DTYPES[case["dtype"]].itemsize, BLOCK[case["fmt"]]
    held = lambda rows, cols: rows * (-(-cols // 2) + -(-cols // block))  # noqa: E731
    if op in ("quantize", "dequantize"):
        r, c = case["rows"], case["cols"]
        if op == "dequantize":
            return {"bytes": case["count"] * (held(r, c) + r * c * size), "flops": 2 * case["count"] * r * c}
        # what is read, what is held, and the values that are read back from it
        sides = {"rows": [(r, c)], "cols": [(c, r)], "both": [(r, c), (c, r)]}[case["axes"]]
        return {"bytes": case["count"] * (r * c * size + sum(held(*x) + r * c * size for x in sides)), "flops": case["count"] * r * c * 5 * len(sides)}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": case["count"] * (held(m, k) + held(n, k) + m * n * size * (2 if case["beta"] else 1)), "flops": 2 * case["count"] * m * n * k}
    if op == "gram":  # a symmetric result has half of its products to be formed
        n, k = case["rows"], case["cols"]
        return {"bytes": case["count"] * (held(n, k) + n * n * size * (2 if case["beta"] else 1)), "flops": case["count"] * n * (n + 1) * k}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "linear":
        return {"bytes": m * k * size + held(n, k) + m * n * size, "flops": 2 * m * n * k + 5 * m * k}
    # x, w and dy in, y, dx and dw out
    return {"bytes": 2 * size * (m * k + n * k + m * n), "flops": 6 * m * n * k + 10 * (m * k + n * k + m * n)}


# ---- the definition in 64 bits ----

GRID4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
GRID8 = [m * 2.0**-9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def nearest(a, grid):
    """Index of the grid's value nearest to a >= 0; halfway between two, the even index; above the last, the last."""
    g = torch.tensor(grid, dtype=torch.float64, device=a.device)
    middle = (g[1:] + g[:-1]) / 2
    low = torch.bucketize(a, middle, right=False)
    high = torch.bucketize(a, middle, right=True)
    return torch.where(low % 2 == 0, low, high), g


def exact_through(x, fmt):
    got = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    block = BLOCK[fmt]
    for i in range(x.shape[0]):
        whole = float(x[i].abs().max())
        unit = 2.0 ** max(-126, math.ceil(math.log2(whole / 2688.0) - 1e-12)) if whole else 1.0
        for r in range(0, x.shape[1], 4096):
            v = x[i, r : r + 4096].double()
            n = v.shape[1]
            v = torch.cat([v, v.new_zeros(v.shape[0], -n % block)], 1).view(v.shape[0], -1, block)
            most = v.abs().amax(2, keepdim=True)
            if fmt == "nvfp4":
                k, g = nearest(most / unit / 6.0, GRID8)
                scale = g[k] * unit
            else:
                scale = torch.exp2((torch.log2(most).floor() - 2).clamp(min=-127.0))
            k, g = nearest(torch.where(scale > 0, v.abs() / scale, 0.0), GRID4)
            got[i, r : r + 4096] = (torch.sign(v) * g[k] * scale).view(v.shape[0], -1)[:, :n]
    return got


def exact_read(h):
    """The values in 64 bits, from the bits of each code and scale."""
    rows, cols, block = h["rows"], h["cols"], BLOCK[h["fmt"]]
    got = []
    for i in range(h["codes"].shape[0]):
        at = torch.arange(cols, device="cuda")
        code = (h["codes"][i][:, at // 2] >> (4 * (at % 2)).to(torch.uint8)) & 15
        e, m = (code >> 1) & 3, code & 1
        v = torch.where(e > 0, (2.0 + m.double()) * torch.exp2(e.double() - 2.0), m.double() * 0.5)
        v = torch.where(code >= 8, -v, v)
        r, k = torch.arange(rows, device="cuda")[:, None], (at // block)[None, :]
        byte = h["scales"][i][r // 128, k // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4].long()
        if h["fmt"] == "nvfp4":
            e, m = byte >> 3, (byte & 7).double()
            v = v * torch.where(e > 0, (8.0 + m) * torch.exp2(e.double() - 10.0), m * 2.0**-9) * h["own_scale"][i].double()
        else:
            v = v * torch.exp2(byte.double() - 127.0)
        got.append(v)
    return torch.stack(got)


def exact(case, seed):
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    op, fmt = case["op"], case["fmt"]
    if op == "quantize":
        got = {}
        if case["axes"] != "cols":
            got["v"] = exact_through(s["x"], fmt)
        if case["axes"] != "rows":
            got["vt"] = exact_through(s["x"].mT, fmt)
        return got
    if op == "dequantize":
        return {"v": exact_read(s["q"])}
    if op in ("gemm", "gram"):
        a = exact_read(s["a"] if op == "gemm" else s["x"])
        b = exact_read(s["b"]) if op == "gemm" else a
        d = s["alpha"] * torch.stack([p @ q.mT for p, q in zip(a, b)])
        return {"d": d + case["beta"] * s["c"].double() if case["beta"] else d}
    if op == "linear":
        return {"y": exact_through(s["x"], fmt) @ exact_read(s["w"]).mT}
    x, w, dy = s["x"], s["w"], s["dy"]
    return {
        "y": exact_through(x, fmt) @ exact_through(w, fmt).mT,
        "dx": exact_through(dy, fmt) @ exact_through(w.mT, fmt).mT,
        "dw": exact_through(dy.mT, fmt) @ exact_through(x.mT, fmt).mT,
    }
