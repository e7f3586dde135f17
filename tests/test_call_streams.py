"""What a call allocates by itself while it is given a stream: the memory has to come from that stream's
pool. Memory of the current stream's pool may be a block whose last use is still queued there, which
nothing orders before the work on the other stream.

On the CPU the allocator, the streams and the library are stand-ins that note what happens; on the GPU the
current stream is kept busy with writes to memory that it has just freed."""
import math

import pytest

torch = pytest.importorskip("torch")
from fake_device import Memory, Stream, tensor as _tensor, world  # noqa: E402, F401
from matrix_orthogonalizing_optimizer_gb300 import api, tensor_lists  # noqa: E402


LIST_CALLS = {
    "grad_norm": lambda w, **kw: tensor_lists.grad_norm([_tensor(w, 8, 8)], status=w["status"], **kw),
    "clip_grads": lambda w, **kw: tensor_lists.clip_grads([_tensor(w, 8, 8)], 1.0, status=w["status"], **kw),
}

MATRIX_CALLS = {
    "gram_ns_batched": lambda w, **kw: api.gram_ns_batched([_tensor(w, 2, 8, 16)], status=w["status"], **kw),
    "ns_standard_batched": lambda w, **kw: api.ns_standard_batched([_tensor(w, 2, 8, 16)], status=w["status"], **kw),
    "muon_step": lambda w, **kw: api.muon_step(*[[_tensor(w, 2, 8, 16)] for _ in range(3)], lr=0.1, status=w["status"], **kw),
    "frac_row_select": lambda w, **kw: api.frac_row_select(_tensor(w, 2, 8, 16), 3, **kw),
}


def _check(world, call):
    side = Stream("side")
    call(world, stream=side)
    made = [m for m in world["made"] if m.numel()]  # an empty tensor has no memory
    assert made and all(m.stream is side for m in made)
    world["made"].clear()
    call(world)
    assert all(m.stream is world["here"] for m in world["made"])


@pytest.mark.parametrize("name", sorted(LIST_CALLS))
def test_lists_allocate_on_the_call_s_stream(world, name):
    _check(world, LIST_CALLS[name])


@pytest.mark.parametrize("name", sorted(MATRIX_CALLS))
def test_matrices_allocate_on_the_call_s_stream(world, name):
    _check(world, MATRIX_CALLS[name])


def test_result_is_kept_for_the_stream_that_reads_it(world):
    """The caller reads the result on the current stream: freed, its memory waits for what is queued there."""
    r = tensor_lists.grad_norm([_tensor(world, 8, 8)], status=world["status"], stream=Stream("side"))
    assert r.recorded == [world["here"]]


class _Word(Memory):
    """A status word: what is queued on it, and on which stream."""
    value = 0

    def __getitem__(self, _):
        return self.value

    def cpu(self):
        return [self.value]

    def zero_(self):
        self.value = 0


def test_status_word_is_zeroed_before_other_streams_may_set_it(world, monkeypatch):
    """The module's own status word is zeroed on the current stream; a call on another stream may set its
    bits as soon as the host goes on."""
    here, side = world["here"], Stream("side")
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: _Word(1, torch.int32, world["device"]))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(api, "_OWNED_STATUS", {})
    tensor_lists.grad_norm([_tensor(world, 8, 8)], stream=side)
    assert here.waits == 1  # when the word was made
    tensor_lists.grad_norm([_tensor(world, 8, 8)], stream=side)
    assert here.waits == 1
    api._OWNED_STATUS[0].value = 1
    with pytest.raises(api._lib.GnsDeviceError):
        tensor_lists.grad_norm([_tensor(world, 8, 8)], stream=side)
    assert here.waits == 2 and api._OWNED_STATUS[0].value == 0  # when it was cleared


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["grad_norm", "clip_grads"])
def test_writes_queued_on_the_current_stream_do_not_reach_the_call(call):
    import matrix_orthogonalizing_optimizer_gb300 as gns

    ts = [torch.full((5000, 100), 0.5, device="cuda") for _ in range(9)]
    outs = [torch.empty_like(t) for t in ts]
    want = 0.5 * math.sqrt(9 * 500000)
    big = torch.empty(1 << 28, dtype=torch.float32, device="cuda")
    side = torch.cuda.Stream()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    size = gns.list_workspace_size(len(ts))
    torch.cuda.synchronize()
    for _ in range(5):
        freed = [torch.empty(2, device="cuda") for _ in range(64)] + [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(16)]
        for _ in range(20):
            big.fill_(1.0)
        for t in freed:
            t.fill_(255)
        freed = t = None
        if call == "grad_norm":
            r = gns.grad_norm(ts, max_norm=1.0, stream=side, status=status)
        else:
            r = gns.clip_grads(ts, 1.0, outs=outs, stream=side, status=status)
        torch.cuda.synchronize()
        assert abs(float(r[0]) - want) <= 2.0 ** -18 * want
        assert int(status) == 0
