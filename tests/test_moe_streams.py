"""Calls on a stream that is given: whatever a call reads or writes there stays
allocated until the stream is past it, also if the caller drops it at once."""

import contextlib
from types import SimpleNamespace

import pytest
import torch

DEVICE = torch.device("cuda", 0)


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU and notes the streams it is used on."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: DEVICE)

    def record_stream(self, stream):
        self.on = getattr(self, "on", []) + [stream]


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def M(monkeypatch):
    from experiment_network_simulation_amd import moe
    ok = lambda *a: 0
    lib = SimpleNamespace(msim_route=ok, msim_route_backward=ok, msim_dropout=ok, msim_traffic=ok)
    monkeypatch.setattr(moe, "load_library", lambda: lib)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: SimpleNamespace(device=device, cuda_stream=h))
    return moe


def calls(M):
    i32 = lambda *s: gpu(*s, dtype=torch.int32)
    x, bias, ids, w, load, g, dx = gpu(4, 8), gpu(8), i32(4, 2), gpu(4, 2), i32(8), gpu(4, 2), gpu(4, 8)
    yield [x, bias], lambda s: M.route(x, 2, bias=bias, stream=s)
    x, bias = gpu(4, 8), gpu(8)
    yield [x, bias, ids, w, load], lambda s: M.route(x, 2, bias=bias, out=M.Routing(ids, w, load), stream=s)
    x, ids, w = gpu(4, 8), i32(4, 2), gpu(4, 2)
    yield [x, ids, w], lambda s: M.route(x, 2, out=M.Routing(ids, w, None), stream=s)
    x, ids = gpu(4, 8), i32(4, 2)
    yield [x, ids, g, dx], lambda s: M.route_backward(x, ids, g, out=dx, stream=s)
    x, y = gpu(4, 8), gpu(4, 8)
    yield [x, y], lambda s: M.dropout(x, 0.5, 1, out=y, stream=s)
    gy = gpu(4, 8)
    yield [gy], lambda s: M.dropout_backward(gy, 0.5, 1, stream=s)
    ids, off, home, place, out = i32(4, 2), gpu(3, dtype=torch.int64), i32(2), i32(8), i32(2, 5)
    yield [ids, off, home, place, out], lambda s: M.traffic(ids, off, home, place, 5, out=out, stream=s)


def test_every_tensor_of_a_call_is_noted_on_its_stream(M):
    for n, (tensors, call) in enumerate(calls(M)):
        s = SimpleNamespace(device=DEVICE, cuda_stream=0x5150)
        call(s)
        assert all(s in getattr(t, "on", []) for t in tensors), n
    for n, (tensors, call) in enumerate(calls(M)):
        call(0x5150)                       # a raw handle
        assert all([s.cuda_stream for s in getattr(t, "on", [])] == [0x5150] for t in tensors), n


def test_a_stream_of_another_device_is_refused(M):
    for tensors, call in calls(M):
        with pytest.raises(ValueError, match="stream is on"):
            call(SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0x5150))


@pytest.mark.gpu
def test_inputs_that_are_dropped_after_the_call():
    """The stream is busy when the call is made, its input is freed, and other work asks for memory of that size."""
    from experiment_network_simulation_amd import moe
    torch.cuda.set_device(0)
    rows = 1 << 20                          # 32 MiB: a size that nothing else holds
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        x = torch.ones(rows, 8, device="cuda:0")
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)   # clock ticks: about 10 ms
        y = moe.dropout(x, 0.0, 1, stream=handle)
        was = x.data_ptr()
        del x
        z = torch.full((rows, 8), 7.0, device="cuda:0")
        assert z.data_ptr() != was
        s.synchronize()
        assert bool((y == 1.0).all()) and bool((z == 7.0).all())
