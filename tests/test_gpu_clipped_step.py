"""muon_step with grad_scale, for every flavour and layout that reads the gradient: the momentum bit by
bit against its formula, the rest of the step bit by bit against the same step from that momentum; and
the example of a whole clipped training step."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")
gns = pytest.importorskip("matrix_orthogonalizing_optimizer_gb300")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _tensors(count, rows, cols):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows * 1000 + cols)

    def one():
        t = gns.empty_padded((count, rows, cols), torch.bfloat16, "cuda")
        t.copy_(torch.randn((count, rows, cols), generator=g, device="cuda") / cols ** 0.5)
        return t

    return one(), one(), one()


def _like(t):
    c = gns.empty_padded(t.shape, t.dtype, t.device)
    c.copy_(t)
    return c


def _equal(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


SHAPES = [(3, 128, 384), (2, 384, 128), (2, 96, 203), (2, 203, 96), (1, 512, 1024), (2, 640, 640)]


def _kinds(rows, cols):
    kinds = [dict(), dict(flavor="normuon"), dict(flavor="rownorm"), dict(ns_dtype=torch.float16)]
    return kinds + [dict(frac=0.25)] if min(rows, cols) >= 96 else kinds


@pytest.mark.parametrize("count,rows,cols", SHAPES)
def test_scaled_muon_step(count, rows, cols):
    for c in (0.3, 1.0, 2.0 ** -5, 0.0):
        scale = torch.full((1,), c, device="cuda")
        for kind in _kinds(rows, cols):
            W, G, M = _tensors(count, rows, cols)
            p = gns.MuonParams(lr=0.02, momentum=0.95, weight_decay=0.1, **kind)
            V = torch.full((count, 1, min(rows, cols)), 0.5, device="cuda") if p.flavor == "normuon" else None
            W1, G1, M1 = _like(W), _like(G), _like(M)
            V1 = V.clone() if V is not None else None
            gns.muon_step(W1, G1, M1, V=V1, params=p, grad_scale=scale)
            assert _equal(G1, G)
            # the momentum: fp32 products, fp32 sum, one rounding
            frac = p.frac < 1.0
            m = M.float() if frac else M.float() * torch.tensor(0.95, device="cuda")
            new = (m + G.float() * scale).to(torch.bfloat16)
            # the same step from there with nothing to add
            W2, M2 = _like(W), _like(new)
            V2 = V.clone() if V is not None else None
            gns.muon_step(W2, _like(G).zero_(), M2, V=V2,
                          params=gns.MuonParams(lr=0.02, momentum=0.95 if frac else 1.0, weight_decay=0.1, **kind))
            assert _equal(M1, M2), (c, kind)
            assert _equal(W1, W2), (c, kind)
            if V is not None:
                assert torch.equal(V1, V2)


@pytest.mark.parametrize("kind", [dict(), dict(flavor="rownorm"), dict(frac=0.5)])
def test_scale_one_is_no_scale(kind):
    W, G, M = _tensors(2, 256, 512)
    p = gns.MuonParams(lr=0.02, **kind)
    W1, M1 = _like(W), _like(M)
    gns.muon_step(W, G, M, params=p)
    gns.muon_step(W1, G, M1, params=p, grad_scale=torch.ones(1, device="cuda"))
    assert _equal(W, W1) and _equal(M, M1)


def test_scale_of_a_norm_matches_clipping_first():
    """A power of two as the scale: clipping into bf16 first rounds nothing, so both ways agree."""
    W, G, M = _tensors(2, 256, 512)
    G.copy_(torch.sign(G))
    r = gns.grad_norm([G], max_norm=0.25 * math.sqrt(G.numel()), eps=0.0)
    assert float(r[1]) == 0.25
    W1, G1, M1 = _like(W), _like(G), _like(M)
    gns.clip_grads([G1], 0.25 * math.sqrt(G.numel()), eps=0.0)
    gns.muon_step(W1, G1, M1, lr=0.02)
    gns.muon_step(W, G, M, lr=0.02, grad_scale=r[1:])
    assert _equal(W, W1) and _equal(M, M1)


def test_scale_refusals():
    W, G, M = _tensors(1, 128, 256)
    for bad in (torch.ones(1), torch.ones(2, device="cuda"), torch.ones(1, device="cuda", dtype=torch.float16)):
        with pytest.raises(ValueError, match="grad_scale"):
            gns.muon_step(W, G, M, lr=0.02, grad_scale=bad)


def test_example_trains():
    spec = importlib.util.spec_from_file_location("clipped_training_step", os.path.join(ROOT, "examples", "clipped_training_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, norms = example.train(steps=40, log=lambda *_: None)
    assert all(math.isfinite(x) for x in losses + norms)
    assert losses[0] > 0.9 * math.log(512)  # an untrained model knows nothing
    assert losses[-1] < 0.5 * losses[0]
