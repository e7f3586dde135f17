"""A call with more than one GPU: everything that it is given lies on the device of its tensors, and that
is where it launches, whichever device is the current one. A pointer to another device's memory would
fault, and a stream's handle of 0 is the default stream of whatever device is current."""
import pytest

torch = pytest.importorskip("torch")
from fake_device import Memory, Stream, tensor, world  # noqa: E402, F401
from matrix_orthogonalizing_optimizer_gb300 import api, tensor_lists  # noqa: E402

F32, I32, U8 = torch.float32, torch.int32, torch.uint8


def _memory(shape, dtype, index):
    return Memory(shape, dtype, torch.device("cuda", index))


def _norm(w, index, **kw):
    tensor_lists.grad_norm([tensor(w, 8, 8, index=index)], **{"status": _memory(1, I32, index), **kw})


def _clip(w, index, **kw):
    tensor_lists.clip_grads([tensor(w, 8, 8, index=index)], 1.0, **{"status": _memory(1, I32, index), **kw})


def _adamw(w, index, **kw):
    roles = {k: [tensor(w, 8, 8, dtype=F32, index=index)] for k in "WGMV"}
    status = {"status": _memory(1, I32, index)}
    tensor_lists.adamw_step(**{**roles, **status, **kw}, lr=0.1)


def _lists(index, dtype=F32):
    return [_memory((8, 8), dtype, index)]


ELSEWHERE = [  # what may lie on another device, of each call
    (_norm, "result", lambda i: _memory(2, F32, i)),
    (_norm, "workspace", lambda i: _memory(1 << 20, U8, i)),
    (_norm, "status", lambda i: _memory(1, I32, i)),
    (_norm, "stream", lambda i: Stream("side", i)),
    (_clip, "outs", lambda i: _lists(i, torch.bfloat16)),
    (_clip, "result", lambda i: _memory(2, F32, i)),
    (_clip, "workspace", lambda i: _memory(1 << 20, U8, i)),
    (_clip, "status", lambda i: _memory(1, I32, i)),
    (_adamw, "G", _lists),
    (_adamw, "M", _lists),
    (_adamw, "V", _lists),
    (_adamw, "masters", _lists),
    (_adamw, "grad_scale", lambda i: _memory(1, F32, i)),
    (_adamw, "step_count", lambda i: _memory(1, I32, i)),
    (_adamw, "status", lambda i: _memory(1, I32, i)),
    (_adamw, "stream", lambda i: Stream("side", i)),
]


@pytest.mark.parametrize("call,name,make", ELSEWHERE, ids=[f"{c.__name__[1:]}-{n}" for c, n, _ in ELSEWHERE])
def test_lists_refuse_what_lies_on_another_device(world, call, name, make):
    call(world, 0, **{name: make(0)})
    assert len(world["library"].calls) == 1
    with pytest.raises(ValueError, match=name):
        call(world, 0, **{name: make(1)})
    assert len(world["library"].calls) == 1


def test_lists_refuse_a_workspace_on_the_host(world):
    host = Memory(1 << 20, U8, torch.device("cpu"))
    host.get_device = lambda: -1
    with pytest.raises(ValueError, match="workspace"):
        _norm(world, 0, workspace=host)


@pytest.mark.parametrize("call,name", [(_norm, "gns_grad_norm"), (_clip, "gns_clip_grads"), (_adamw, "gns_adamw_step")])
@pytest.mark.parametrize("index", [0, 1])
def test_lists_launch_on_the_device_of_their_tensors(world, call, name, index):
    call(world, index)
    assert world["library"].calls == [(name, index)]


def test_lists_of_no_tensor_are_refused(world):
    for call in (lambda: tensor_lists.grad_norm([None]), lambda: tensor_lists.clip_grads([None], 1.0),
                 lambda: tensor_lists.adamw_step([None], [None], [None], [None], lr=0.1)):
        with pytest.raises(ValueError, match="must be a tensor"):
            call()


def _matrix(index, *shape):
    return [_memory(shape or (2, 8, 16), torch.bfloat16, index)]


def _gram(w, index, **kw):
    api.gram_ns_batched(**{"xs": _matrix(index), "status": _memory(1, I32, index), **kw})


def _standard(w, index, **kw):
    api.ns_standard_batched(**{"xs": _matrix(index), "status": _memory(1, I32, index), **kw})


def _muon(w, index, **kw):
    roles = {k: _matrix(index) for k in "WGM"}
    api.muon_step(**{**roles, "lr": 0.1, "status": _memory(1, I32, index), **kw})


def _select(w, index, **kw):
    api.frac_row_select(**{"m": _matrix(index)[0], "k": 3, **kw})


def _gemm(w, index, **kw):
    roles = {k: _matrix(index)[0] for k in "abcd"}
    api.sym_gemm(**{**roles, "status": _memory(1, I32, index), **kw})


def _xxt(w, index, **kw):
    api.sym_gemm_xxt(**{"x": _matrix(index)[0], "c": _matrix(index)[0], "status": _memory(1, I32, index), **kw})


def _poly(w, index, **kw):
    roles = {k: _matrix(index)[0] for k in ("R", "Q", "Z", "RZ", "q_scratch")}
    api.sym_poly_update(**{**roles, "a": 1.0, "b": 1.0, "c": 1.0, "q_is_identity": False, "skip_r": False,
                           "status": _memory(1, I32, index), **kw})


def _one(index):
    return _matrix(index)[0]


STATUS, STREAM = lambda i: _memory(1, I32, i), lambda i: Stream("side", i)  # noqa: E731
WORKSPACE = lambda i: _memory(1 << 20, U8, i)  # noqa: E731
MATRICES = {
    _gram: dict(outs=_matrix, workspace=WORKSPACE, status=STATUS, stream=STREAM),
    _standard: dict(outs=_matrix, workspace=WORKSPACE, status=STATUS, stream=STREAM),
    _muon: dict(W=_matrix, G=_matrix, V=lambda i: [_memory((2, 1, 8), F32, i)], workspace=WORKSPACE, status=STATUS,
                stream=STREAM, grad_scale=lambda i: _memory(1, F32, i)),
    _select: dict(idx=lambda i: _memory((2, 3), I32, i), gathered=_one, workspace=WORKSPACE, stream=STREAM),
    _gemm: dict(b=_one, c=_one, d=_one, status=STATUS, stream=STREAM),
    _xxt: dict(c=_one, status=STATUS, stream=STREAM),
    _poly: dict(Q=_one, Z=_one, RZ=_one, q_scratch=_one, status=STATUS, stream=STREAM),
}


@pytest.mark.parametrize("call,name", [(c, n) for c, names in MATRICES.items() for n in names])
def test_matrices_refuse_what_lies_on_another_device(world, call, name):
    make = MATRICES[call][name]
    call(world, 0, **{name: make(0)})
    assert len(world["library"].calls) == 1
    with pytest.raises(ValueError, match=name):
        call(world, 0, **{name: make(1)})
    assert len(world["library"].calls) == 1


def test_groups_of_one_call_lie_on_one_device(world):
    with pytest.raises(ValueError, match="xs"):
        _gram(world, 0, xs=_matrix(0) + _matrix(1))


@pytest.mark.parametrize("call", list(MATRICES))
@pytest.mark.parametrize("index", [0, 1])
def test_matrices_launch_on_the_device_of_their_tensors(world, call, index):
    call(world, index)
    assert [i for _, i in world["library"].calls] == [index]
