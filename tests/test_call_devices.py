"""A call with more than one GPU: everything that it is given lies on the device of its tensors, and that
is where it launches, whichever device is the current one. A pointer to another device's memory would
fault, and a stream's handle of 0 is the default stream of whatever device is current."""
import pytest

torch = pytest.importorskip("torch")
from fake_device import Memory, Stream, tensor, world  # noqa: E402, F401
from matrix_orthogonalizing_optimizer_gb300 import tensor_lists  # noqa: E402

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
