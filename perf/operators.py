"""The operators of a training step's gradients that are measured, and on what.

  grad_norm   the global norm of a list of gradients, and the scale that clips them to a maximum norm
  clip_grads  the same, with the gradients scaled (in place, or into other buffers)
  adamw_step  one AdamW step of a list of tensors (the parameters beside Muon's matrices: embeddings, heads, gains)

A case is one list of tensors. As a training program keeps them, the tensors of one type are views of
one buffer, either each on a 256-byte boundary ("align": 1) or packed without a gap ("align": 0, so that
a tensor starts at any element), and the buffers are what a pass returns. "padded" matrices stand for
themselves: rows of odd length on 16-byte boundaries, as the framework's own matrices of odd width.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS_CLIP = 1e-6
ADAMW = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.1, "step": 100}


def listed():
    return [
        # the gains of 24 layers and the last norm's: 196 KB in 49 tensors, a call that is all latency
        {"name": "norm-gains-f32", "op": "grad_norm", "kind": "gains", "layers": 24, "width": 1024, "dtype": "f32", "align": 1},
        # the benchmark's 24 matrices of 1024 x 4096 in one batch: an ordinary layer stack of one shape
        {"name": "norm-batch-bf16", "op": "grad_norm", "kind": "batches", "tensors": 1, "count": 24, "rows": 1024, "cols": 4096, "dtype": "bf16", "padded": 0},
        # 300 tensors of odd sizes packed into one gradient buffer
        {"name": "norm-ragged-f16", "op": "grad_norm", "kind": "ragged", "tensors": 300, "elements": 30000001, "shape_seed": 1, "dtype": "f16", "align": 0},
        # the gradients of 256 experts' 2048 x 8192 projections: the largest, 8.6 GB
        {"name": "norm-experts-bf16", "op": "grad_norm", "kind": "batches", "tensors": 4, "count": 64, "rows": 2048, "cols": 8192, "dtype": "bf16", "padded": 0},
        # gains again, clipped: latency
        {"name": "clip-gains-f32", "op": "clip_grads", "kind": "gains", "layers": 24, "width": 1024, "dtype": "f32", "align": 1, "clipped": 1},
        # four layers of the dense-transformer set (4096 x 4096, 4096 x 11008, 11008 x 4096) with f32 gains
        {"name": "clip-layers-bf16", "op": "clip_grads", "kind": "layers", "layers": 4, "width": 4096, "ffn": 11008, "dtype": "bf16", "align": 1, "clipped": 1},
        # batches of odd width whose rows are padded to 16 bytes
        {"name": "clip-padded-f32", "op": "clip_grads", "kind": "batches", "tensors": 3, "count": 7, "rows": 1001, "cols": 1333, "dtype": "f32", "padded": 1, "clipped": 1},
        # an ordinary step whose norm lies below the maximum: the gradients stay as they are
        {"name": "clip-unclipped-bf16", "op": "clip_grads", "kind": "batches", "tensors": 1, "count": 24, "rows": 1024, "cols": 4096, "dtype": "bf16", "padded": 0, "clipped": 0},
        # the gains' step: latency
        {"name": "adamw-gains-f32", "op": "adamw_step", "kind": "gains", "layers": 24, "width": 1024, "dtype": "f32", "grad_dtype": "f32", "master": 0, "align": 1, "scaled": 0},
        # embedding and head of a small model with f32 masters, f32 gains beside them, gradients clipped on the way
        {"name": "adamw-embed-bf16", "op": "adamw_step", "kind": "embedding", "vocab": 32000, "width": 1024, "dtype": "bf16", "grad_dtype": "bf16", "master": 1, "align": 1, "scaled": 1},
        # odd sizes packed without a gap, bf16 weights updated from f32 accumulated gradients
        {"name": "adamw-ragged-bf16", "op": "adamw_step", "kind": "ragged", "tensors": 120, "elements": 10000019, "shape_seed": 2, "dtype": "bf16", "grad_dtype": "f32", "master": 0, "align": 0, "scaled": 1},
        # embedding and head of a large model with f32 masters: the largest
        {"name": "adamw-embed-large-bf16", "op": "adamw_step", "kind": "embedding", "vocab": 64000, "width": 4096, "dtype": "bf16", "grad_dtype": "bf16", "master": 1, "align": 1, "scaled": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grad_norm", "clip_grads", "adamw_step"])
    most = {"grad_norm": 2e9, "clip_grads": 5e8, "adamw_step": 4e8}[op]
    c = {"op": op, "kind": rng.choice(["gains", "layers", "ragged", "batches", "embedding"]), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if c["kind"] == "gains":
        c.update(layers=_log(rng, 1, 120), width=_log(rng, 1, 20000))
    elif c["kind"] == "layers":
        width = _log(rng, 64, 4096)
        ffn = int(width * rng.uniform(1.5, 4.5))
        c.update(width=width, ffn=ffn, layers=_log(rng, 1, max(1, min(48, most / (width * width + 3 * width * ffn)))))
    elif c["kind"] == "ragged":
        elements = _log(rng, 2000, most / 4)
        c.update(tensors=_log(rng, 1, min(700, elements // 4)), elements=elements, shape_seed=rng.randrange(1 << 20))
    elif c["kind"] == "batches":
        rows, cols = _log(rng, 1, 4096), _log(rng, 8, 8192)
        tensors = rng.randint(1, 6)
        c.update(tensors=tensors, count=_log(rng, 1, max(1, min(256, most / 8 / (tensors * rows * cols)))), rows=rows, cols=cols, padded=1)
    else:
        width = _log(rng, 64, 4096)
        c.update(vocab=_log(rng, 256, max(257, min(128000, most / 2 / width))), width=width)
    if c["kind"] != "batches":
        c["align"] = rng.randint(0, 1)
    if op == "clip_grads":
        c["clipped"] = int(rng.random() < 0.75)
    if op == "adamw_step":
        c.update(grad_dtype=rng.choice([c["dtype"], "f32"]), master=int(c["dtype"] != "f32" and rng.random() < 0.6), scaled=rng.randint(0, 1))
    return c


def shapes(case):
    """[(shape, whether it is a gain, which stays in f32 beside 16-bit matrices)]"""
    k = case["kind"]
    if k == "gains":
        return [((case["width"],), True)] * (2 * case["layers"] + 1)
    if k == "layers":
        d, f = case["width"], case["ffn"]
        return [((d,), True), ((d, d), False), ((d,), True), ((d, f), False), ((d, f), False), ((f, d), False)] * case["layers"]
    if k == "embedding":
        return [((case["vocab"], case["width"]), False), ((case["width"],), True), ((case["vocab"], case["width"]), False)]
    if k == "batches":
        return [((case["count"], case["rows"], case["cols"]), False)] * case["tensors"]
    r = random.Random(case["shape_seed"])
    part = [math.exp(r.uniform(0.0, 7.0)) for _ in range(case["tensors"])]
    whole = sum(part)
    return [((max(1, int(case["elements"] * p / whole)) | 1,), False) for p in part]


def elements(case):
    """{whether it is a gain: number of elements}"""
    n = {True: 0, False: 0}
    for shape, gain in shapes(case):
        n[gain] += math.prod(shape)
    return n


def buffers(case, dtype, fill):
    """(what a pass returns, the list of tensors): the tensors as views of one buffer for each type, or as themselves
    where they are padded. A gain has f32. fill(buffer): puts values into a new buffer."""
    todo = [(shape, torch.float32 if gain else dtype) for shape, gain in shapes(case)]
    if case["kind"] == "batches":
        made = []
        for shape, dt in todo:
            step = 16 // dt.itemsize if case["padded"] else 1
            made.append(fill(torch.empty((*shape[:-1], -(-shape[-1] // step) * step), dtype=dt, device="cuda"))[..., : shape[-1]])
        return made, made
    at, size = [], {}
    for shape, dt in todo:
        begin = size.get(dt, 0)
        if case["align"]:
            begin = -(-begin // 128) * 128
        at.append(begin)
        size[dt] = begin + math.prod(shape)
    whole = {dt: fill(torch.empty(n, dtype=dt, device="cuda")) for dt, n in size.items()}
    return list(whole.values()), [whole[dt][b : b + math.prod(shape)].view(shape) for (shape, dt), b in zip(todo, at)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    scale = random.Random(seed)
    op = case["op"]
    grad_dtype = DTYPES[case.get("grad_dtype", case["dtype"])]
    normal = lambda std: lambda t: t.normal_(0.0, std, generator=gen)  # noqa: E731
    zeros = lambda t: t.zero_()  # noqa: E731
    g_all, g = buffers(case, grad_dtype, normal(1e-3))
    for x in g:  # layers' gradients differ in size
        x.mul_(10.0 ** scale.uniform(-1.0, 0.5))
    seen = None
    if case["kind"] == "embedding":  # the tokens of a batch touch a part of the embedding's rows
        seen = torch.rand(case["vocab"], generator=gen, device="cuda") < 0.3
        g[0].mul_(seen.unsqueeze(1))
    s = {"case": case, "g": g, "g_all": g_all}
    s["max_norm"] = 1e-3 * math.sqrt(sum(elements(case).values())) * (0.05 if case.get("clipped", 1) else 100.0)
    if op == "clip_grads" and case["clipped"]:  # the clipped gradients go into buffers of their own
        s["o_all"], s["o"] = buffers(case, grad_dtype, zeros)
    if op == "adamw_step":
        dtype = DTYPES[case["dtype"]]
        s["m_all"], s["m"] = buffers(case, torch.float32, normal(3e-4))
        s["v_all"], s["v"] = buffers(case, torch.float32, normal(1e-3))
        for x in s["v_all"]:
            x.square_()
        if seen is not None:  # rows that no token has touched yet have no state
            old = torch.rand(case["vocab"], generator=gen, device="cuda") < 0.5
            s["m"][0].mul_(old.unsqueeze(1))
            s["v"][0].mul_(old.unsqueeze(1))
        s["w_all"], s["w"] = buffers(case, dtype, normal(0.02))
        s["p"] = None
        if case["master"]:  # f32 masters of the 16-bit weights, which are their rounded copies
            s["p_all"], s["p"] = buffers(case, torch.float32, normal(0.02))
            for w, p in zip(s["w"], s["p"]):
                w.copy_(p)
        s["scale"] = torch.full((1,), 0.37, dtype=torch.float32, device="cuda") if case["scaled"] else None
    if own:
        import matrix_orthogonalizing_optimizer_gb300 as gns

        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["lists"] = {k: gns.tensor_list(s[k]) for k in ("w", "g", "m", "v", "o") if k in s}
        if op == "adamw_step":
            s["params"] = gns.AdamWParams(**ADAMW)
            # a tensor that is f32 itself needs no master
            s["lists"]["p"] = gns.tensor_list([None if w.dtype == torch.float32 else p for w, p in zip(s["w"], s["p"])]) if s["p"] else None
        else:
            s["result"] = torch.empty(2, dtype=torch.float32, device="cuda")
            s["ws"] = gns.alloc_workspace(gns.list_workspace_size(len(g)), "cuda")
    return s


def returned(s):
    """Whole buffers, the gradients' untouched ones left out."""
    case = s["case"]
    if case["op"] == "grad_norm":
        return {"result": s["result"]}
    if case["op"] == "clip_grads":
        return {"result": s["result"], "grads": s["o_all"] if case["clipped"] else s["g_all"]}
    got = {"w": s["w_all"], "m": s["m_all"], "v": s["v_all"]}
    if s["p"]:
        got["p"] = s["p_all"]
    return got


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import matrix_orthogonalizing_optimizer_gb300 as gns

    l = s["lists"]
    op = s["case"]["op"]
    if op == "grad_norm":
        gns.grad_norm(l["g"], max_norm=s["max_norm"], result=s["result"], workspace=s["ws"], status=s["status"])
    elif op == "clip_grads":
        gns.clip_grads(l["g"], s["max_norm"], outs=l.get("o"), result=s["result"], workspace=s["ws"], status=s["status"])
    else:
        gns.adamw_step(l["w"], l["g"], l["m"], l["v"], masters=l["p"], params=s["params"], grad_scale=s["scale"], status=s["status"])
    return returned(s)


def run_plain(s):
    case = s["case"]
    if case["op"] == "adamw_step":
        p = s["p"] or s["w"]
        for w, q, g, m, v in zip(s["w"], p, s["g"], s["m"], s["v"]):
            adamw_plain(w, q, g, m, v, s["scale"])
        return returned(s)
    norm = torch.stack([g.float().square().sum() for g in s["g"]]).sum().sqrt()
    scale = torch.clamp(s["max_norm"] / (norm + EPS_CLIP), max=1.0)
    s["result"] = torch.stack([norm, scale])
    if case["op"] == "clip_grads":
        for o, g in zip(s["o"] if case["clipped"] else s["g"], s["g"]):
            o.copy_(g.float() * scale)
    return returned(s)


def adamw_plain(w, p, g, m, v, scale):
    """One tensor: p is the master, or w itself."""
    a = ADAMW
    g = g.float()
    if scale is not None:
        g = g * scale
    m.mul_(a["beta1"]).add_(g, alpha=1.0 - a["beta1"])
    v.mul_(a["beta2"]).add_(g * g, alpha=1.0 - a["beta2"])
    denom = (v / (1.0 - a["beta2"] ** a["step"])).sqrt().add_(a["eps"])
    if w.dtype == torch.float32:
        p = w
    new = p.float() * (1.0 - a["lr"] * a["weight_decay"]) - a["lr"] / (1.0 - a["beta1"] ** a["step"]) * (m / denom)
    if p is not w:
        p.copy_(new)
    w.copy_(new)


def work(case):
    n = elements(case)
    size = {True: 4, False: DTYPES[case["dtype"]].itemsize}
    total = n[True] + n[False]
    if case["op"] == "grad_norm":
        return {"bytes": n[True] * 4 + n[False] * size[False], "flops": 2 * total}
    if case["op"] == "clip_grads":  # gradients that are not clipped stay where they are
        once = n[True] * 4 + n[False] * size[False]
        return {"bytes": once * (2 if case["clipped"] else 1), "flops": 3 * total}
    per = 16 + DTYPES[case["grad_dtype"]].itemsize + (size[False] + 8 if case["master"] else 2 * size[False])  # m, v, g, then w alone or with its master
    return {"bytes": n[True] * 28 + n[False] * per, "flops": 14 * total}


def exact(case, seed):
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    if case["op"] == "adamw_step":
        return exact_adamw(s)
    total = math.fsum(float(torch.linalg.vecdot(x, x)) for g in s["g"] for y in g.reshape(-1).split(1 << 26) for x in (y.double(),))
    norm = math.sqrt(total)
    scale = min(1.0, s["max_norm"] / (norm + EPS_CLIP))
    got = {"result": torch.tensor([norm, scale], dtype=torch.float64)}
    if case["op"] == "clip_grads":
        if not case["clipped"]:
            scale = 1.0
        # what lies between the tensors of a buffer is zero where the clipped ones have buffers of their own
        got["grads"] = widened(case, s["o_all"] if case["clipped"] else s["g_all"], s["o"] if case["clipped"] else s["g"], [g.double() * scale for g in s["g"]])
    return got


def widened(case, whole, views, values):
    """The buffers in 64 bits, with `values` at the places of `views`."""
    if case["kind"] == "batches":
        return values
    got = [x.double() for x in whole]
    for view, value in zip(views, values):
        k = next(i for i, x in enumerate(whole) if x.dtype == view.dtype)
        b = view.storage_offset()
        got[k][b : b + view.numel()] = value.reshape(-1)
    return got


def exact_adamw(s):
    case, a = s["case"], ADAMW
    c = 1.0 if s["scale"] is None else float(s["scale"])
    new = {"w": [], "m": [], "v": []}
    for i, g in enumerate(s["g"]):
        g = g.double() * c
        m = s["m"][i].double() + (1.0 - a["beta1"]) * (g - s["m"][i].double())
        v = s["v"][i].double() + (1.0 - a["beta2"]) * (g.square() - s["v"][i].double())
        m_hat, v_hat = m / (1.0 - a["beta1"] ** a["step"]), v / (1.0 - a["beta2"] ** a["step"])
        w = s["p"][i] if s["p"] and s["w"][i].dtype != torch.float32 else s["w"][i]
        w = w.double()
        new["w"].append(w - a["lr"] * (m_hat / (v_hat.sqrt() + a["eps"]) + a["weight_decay"] * w))
        new["m"].append(m)
        new["v"].append(v)
    got = {k: widened(case, s[k + "_all"], s[k], new[k]) for k in ("w", "m", "v")}
    if s["p"]:  # beside a weight that is f32 itself lies no master
        got["p"] = widened(case, s["p_all"], s["p"], [p.double() if w.dtype == torch.float32 else x for w, p, x in zip(s["w"], s["p"], new["w"])])
    return got
