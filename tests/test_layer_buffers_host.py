"""Whose memory a layer call's own buffers are, without a GPU: a call on an
explicit stream drops its workspace when it returns, so that memory has to
belong to that stream (memory of the current stream would be given away while
the call's kernels still run)."""
import contextlib
import types

import pytest
import torch

from fp8_block_scaled_pow2_b200 import layer as L


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream

    __hash__ = None


class FakeY:
    def __init__(self):
        self.recorded = []

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


@pytest.fixture
def fake(monkeypatch):
    """A layer whose allocations note the current (fake) stream; calls do nothing."""
    at = types.SimpleNamespace(stream=FakeStream(1), allocated=[], ran=[])

    @contextlib.contextmanager
    def on(stream):
        before, at.stream = at.stream, stream
        yield
        at.stream = before

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: at.stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
    monkeypatch.setattr(L.moe, "moe_layer_few_mxfp4", lambda *a, stream=None, **kw: at.ran.append(stream))
    layer = L.MoeLayer.__new__(L.MoeLayer)
    layer.device, layer.tid2eid, layer.w13_p, layer.w2_p, layer.I = torch.device("cpu"), None, None, None, 128
    layer.route_scale, layer.swiglu_limit, layer.has_shared, layer.route_norm = 1.5, 10.0, 1, 1

    def alloc(T, block_n=0):
        at.allocated.append(at.stream.cuda_stream)
        return types.SimpleNamespace(T=T, y=FakeY(), idx=None, w=None, workspace=None)

    layer.alloc = layer.alloc_few = alloc
    layer.segments = lambda x, logits, buf, stream=None, token_ids=None: [lambda: at.ran.append(stream)]
    return layer, at


@pytest.mark.parametrize("call", ["forward", "forward_few"])
@pytest.mark.parametrize("stream,owner,recorded", [
    (None, 1, []),                      # the current stream's memory, as ever
    (FakeStream(1), 1, []),             # the current stream by name
    (FakeStream(7), 7, [1]),            # another one: its memory; y may be read on the current stream
    (9, 9, [1]),                        # a raw handle
])
def test_own_buffers_belong_to_the_calls_stream(fake, call, stream, owner, recorded):
    layer, at = fake
    y = getattr(layer, call)(torch.zeros(3, 8), torch.zeros(3, 4), stream=stream)
    assert at.allocated == [owner] and y.recorded == recorded
    assert at.ran == [stream] and at.stream.cuda_stream == 1


@pytest.mark.parametrize("call", ["forward", "forward_few"])
def test_given_buffers_are_used(fake, call):
    layer, at = fake
    buf = layer.alloc(3)
    assert getattr(layer, call)(torch.zeros(3, 8), torch.zeros(3, 4), buf, stream=FakeStream(7)) is buf.y
    assert at.allocated == [1] and buf.y.recorded == []
