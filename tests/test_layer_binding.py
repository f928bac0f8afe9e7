"""The layer operators' binding: streams and lifetimes of a call's tensors, with
host tensors, a stand-in for the library and for the streams (no GPU)."""
import numpy as np
import pytest
import torch

csf = pytest.importorskip("moe_weight_decode_amd")
layer = csf.layer


class Seen(torch.Tensor):
    """A host tensor that notes the stream it is recorded on."""

    def record_stream(self, stream):
        self.on = stream


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.waits = handle, 0

    def wait_stream(self, other):
        assert other.cuda_stream != self.cuda_stream
        self.waits += 1


def new(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Seen)


@pytest.fixture
def machine(monkeypatch):
    """Streams 1 .. 3, 1 the current one; `calls` lists the streams that calls went to."""
    class Machine:
        streams = {i: Stream(i) for i in (1, 2, 3)}
        now, calls = 1, []

    m = Machine()
    csf.library()
    monkeypatch.setattr(layer, "_device", lambda where, t, name: t.device)
    monkeypatch.setattr(layer, "_current", lambda index: m.now)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: m.streams[m.now])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: m.streams[handle])
    monkeypatch.setattr(torch, "empty", lambda *shape, dtype=torch.float32, device=None: new(*shape, dtype=dtype))
    monkeypatch.setattr(torch, "empty_like", lambda t: new(*t.shape, dtype=t.dtype))
    for name in layer._functions:
        monkeypatch.setitem(layer._functions, name, lambda *args: m.calls.append(args[-1]) or 0)
    m.calls.clear()
    return m


def operators():
    """A call of every operator that takes plain tensors, with its tensors."""
    i = torch.int32
    x, w, r = new(4, 64), new(64), new(4)
    sum, dsum, slots, gates = new(4, 64), new(4, 64), new(4, 2, dtype=i), new(4, 2)
    y, logits, many, dg = new(8, 64), new(4, 16), new(200, 16), new(4, 2)
    yield csf.rms_norm, (x, w, sum), dict(mxfp8=True), (x, w, sum)
    yield csf.rms_norm, (y, w, sum), dict(slots=slots, gates=gates), (y, w, sum, slots, gates)
    yield csf.rms_norm_backward, (x, sum, w, r, dsum), {}, (x, sum, w, r, dsum)
    yield csf.route, (many, 4), {}, (many,)
    yield csf.combine_backward, (x, y, slots, gates), {}, (x, y, slots, gates)
    yield csf.route_backward, (dg, logits, slots, gates), {}, (dg, logits, slots, gates)


def tensors(value):
    return [value] if isinstance(value, torch.Tensor) else [t for t in value if t is not None]


def test_a_call_on_another_stream_records_every_tensor(machine):
    """The inputs too: a caller may drop them once the call returns."""
    for function, args, kwargs, inputs in operators():
        out = tensors(function(*args, **kwargs, stream=machine.streams[2]))
        assert out and all(t.on is machine.streams[2] for t in (*inputs, *out)), function
    n = len(machine.calls)
    assert machine.calls == [2] * n and machine.streams[2].waits == n
    st = csf.prepare(np.full((2, 32, 8), 0x38, np.uint8), csf.NVFP4)._map(lambda t: t.as_subclass(Seen))
    call = layer._call("csf_moe_gated", (), None, torch.device("cpu"), (st, csf.csf_stack(), None), (), machine.streams[3])
    call()
    assert all(t.on is machine.streams[3] for t in (st.bases, st.offsets, st.exceptions, st.prefix, st.tile_index))


def test_a_bound_call_goes_to_the_stream_then_current(machine):
    """As into a graph that is captured after the call was bound."""
    for function, args, kwargs, inputs in operators():
        call = csf.bound(function, *args, **kwargs)
        assert machine.calls == []
        out = tensors(call())
        assert not any(hasattr(t, "on") for t in out)
        machine.now = 3
        call(), call()
        assert machine.calls == [1, 3, 3]
        assert all(t.on is machine.streams[3] for t in (*inputs, *out))
        machine.now = 1
        machine.calls.clear()


def test_a_bound_call_on_a_stream_waits_every_time(machine):
    """Inputs written between two calls come from the current stream."""
    for function, args, kwargs, inputs in operators():
        side = machine.streams[2]
        side.waits = 0
        call = csf.bound(function, *args, **kwargs, stream=side)
        for n in (1, 2, 3):
            call()
            assert side.waits == n
        machine.now = 2  # on it already
        call()
        assert side.waits == 3 and machine.calls == [2, 2, 2, 2]
        machine.now = 1
        machine.calls.clear()


def test_transposed_tensors_are_refused(machine):
    """As many elements in another order are no match: rows would be taken for columns."""
    i = torch.int32
    x, w, r, slots, gates = new(4, 64), new(64), new(4), new(4, 2, dtype=i), new(4, 2)
    turned, turned2 = new(64, 4), new(2, 4)
    for call in (lambda: csf.rms_norm(x, w, turned),
                 lambda: csf.rms_norm(new(8, 64), w, x, slots=slots, gates=turned2),
                 lambda: csf.rms_norm_backward(x, turned, w, r),
                 lambda: csf.rms_norm_backward(x, x, w, r, turned),
                 lambda: csf.combine_backward(x, new(8, 64), slots, turned2),
                 lambda: csf.route_backward(turned2, new(4, 16), slots, gates),
                 lambda: csf.route_backward(gates, new(4, 16), slots, turned2)):
        with pytest.raises(ValueError, match="shape"):
            call()
    assert machine.calls == []
