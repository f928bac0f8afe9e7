"""The layer operators' binding: streams and lifetimes of a call's tensors (no GPU)."""
import numpy as np
import pytest
import torch

csf = pytest.importorskip("moe_weight_decode_amd")


class Seen(torch.Tensor):
    """A host tensor that notes the stream it is recorded on."""

    def record_stream(self, stream):
        self.on = stream


def test_binding_records_every_tensor_on_another_stream(monkeypatch):
    """The inputs too: a caller may drop them once the call returns."""
    layer, side = csf.layer, object()
    monkeypatch.setattr(layer, "_device", lambda where, t, name: t.device)
    monkeypatch.setattr(layer, "_enter", lambda stream, dev: (0, side))

    def new(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(Seen)

    x, w, r, i = new(4, 64), new(64), new(4), torch.int32
    monkeypatch.setattr(torch, "empty", lambda *shape, dtype=torch.float32, device=None: new(*shape, dtype=dtype))
    monkeypatch.setattr(torch, "empty_like", lambda t: new(*t.shape, dtype=t.dtype))
    for make in (lambda: layer._rms_norm(x, w, x.clone(), new(4, 2, dtype=i), new(4, 2), mxfp8=True),
                 lambda: layer._rms_norm_backward(x, x.clone(), w, r, x.clone()),
                 lambda: layer._route(new(200, 16), 4),
                 lambda: layer._combine_backward(x, new(8, 64), new(4, 2, dtype=i), new(4, 2)),
                 lambda: layer._route_backward(new(4, 2), new(4, 16), new(4, 2, dtype=i), new(4, 2))):
        inputs, fresh = make()._keep
        tensors = [t for t in (*inputs, *fresh) if t is not None]
        assert len(tensors) > 2 and all(t.on is side for t in tensors)
    st = csf.prepare(np.full((2, 32, 8), 0x38, np.uint8), csf.NVFP4)
    st = st._map(lambda t: t.as_subclass(Seen))
    layer._call("csf_moe_gated", (), None, None, (st, csf.csf_stack(), None), (), side)
    assert all(t.on is side for t in (st.bases, st.offsets, st.exceptions, st.prefix, st.tile_index))
