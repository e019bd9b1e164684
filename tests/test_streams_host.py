"""On which stream buffers are made, and what waits for their making (CPU only: the library's calls and
torch's streams are stood in for)."""
import contextlib

import pytest
import torch

from mixture_experts_layer_sort_amd import _lib as L
from mixture_experts_layer_sort_amd import layer, mx4


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.waited = handle, []

    def wait_stream(self, other):
        self.waited.append(other)


@pytest.fixture
def made_on(monkeypatch):
    """Streams on which torch.empty was called, and (entry point, stream) of the library's calls."""
    here, made, calls = [None], [], []

    @contextlib.contextmanager
    def stream_of(dev, stream):
        here.append(stream)
        yield
        here.pop()

    empty = torch.empty

    def fake_empty(*a, **kw):
        made.append(here[-1])
        return empty(*a, **kw)

    monkeypatch.setattr(mx4, "_stream_of", stream_of, raising=False)
    monkeypatch.setattr(torch, "empty", fake_empty)
    monkeypatch.setattr(L, "mx4", lambda codes, scales: None)
    monkeypatch.setattr(L, "_stream", lambda stream: stream)
    for name in ("moe_mx4_quantize", "moe_mx4_dequantize"):
        monkeypatch.setattr(L, name, lambda *a, name=name: calls.append((name, a[-1])))
    return made, calls


def test_4_bit_tensors_are_made_on_the_stream_that_fills_them(made_on):
    made, calls = made_on
    q = mx4.MoEMx4Tensor.weights(torch.zeros(2, 128, 128), stream="side")
    mx4.MoEMx4Tensor.rows(torch.zeros(3, 256), stream="side")
    assert made == ["side"] * 4 and calls == [("moe_mx4_quantize", "side")] * 2
    q.dequantize(stream="third")
    assert made[4:] == ["third"] and calls[2:] == [("moe_mx4_dequantize", "third")]
    mx4.MoEMx4Tensor.weights(torch.zeros(128, 128))
    assert made[5:] == [None] * 2


def test_a_first_call_on_another_stream_waits_for_the_making(monkeypatch):
    own, side = Stream(7), Stream(9)
    capturing = [False]
    monkeypatch.setattr(layer, "_stream_of", lambda dev, stream: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: side)
    dev = torch.device("cpu")

    def made():
        m = layer._Made(dev)
        m.stream, m.raw = own, own.cuda_stream
        return m

    m = made()
    assert m.before(dev, 9) == 9 and side.waited == [own]
    assert m.before(dev, 9) == 9 and m.before(dev, side) == 9 and m.before(dev, own) == 7 and side.waited == [own]
    m = made()  # calls on the stream of the making, refused ones perhaps, do not stand for the wait
    assert m.before(dev, own) == 7 and side.waited == [own]
    assert m.before(dev, side) == 9 and side.waited == [own, own]
    m = made()
    capturing[0] = True
    assert m.before(dev, side) == 9 and side.waited == [own, own]
    capturing[0] = False
    assert m.before(dev, side) == 9 and side.waited == [own] * 3
