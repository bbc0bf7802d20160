"""Arguments that the binding has to refuse by itself or hand to the library, without a GPU."""

import pytest
import torch

from test_moe_streams import gpu


@pytest.fixture
def M(monkeypatch):
    from experiment_network_simulation_amd import moe
    monkeypatch.setattr(moe, "_run", lambda device, stream, call, *tensors: call(None))
    return moe


@pytest.mark.parametrize("segs", [0, 2])
@pytest.mark.parametrize("hosts", [16385, 1 << 31, (1 << 32) - 1])
def test_traffic_refuses_hosts_before_it_asks_for_their_memory(M, monkeypatch, segs, hosts):
    from experiment_network_simulation_amd.sim import MsimError
    asked = []
    monkeypatch.setattr(torch.Tensor, "new_empty", lambda self, *a, **k: asked.append(a) or torch.empty(0))
    i32 = lambda *s: gpu(*s, dtype=torch.int32)
    with pytest.raises(MsimError, match="HOSTS"):
        M.traffic(i32(4, 2), gpu(segs + 1, dtype=torch.int64), i32(segs), i32(8), hosts)
    assert not asked


def test_numbers_that_are_not_whole_are_refused(M):
    x = gpu(4, 8)
    for bad in (float("inf"), -float("inf"), float("nan"), 2.5, "2", 1 << 70):
        for call in (lambda: M.route(x, bad), lambda: M.route(x, 2, groups=bad), lambda: M.dropout(x, 0.5, bad),
                     lambda: M.dropout(x, 0.5, 1, offset=bad)):
            with pytest.raises(ValueError):
                call()


def test_results_in_given_tensors_count_as_changes(M, monkeypatch):
    """Autograd sees that a tensor it kept for a backward pass was written to."""
    from types import SimpleNamespace
    ok = lambda *a: 0
    monkeypatch.setattr(M, "load_library", lambda: SimpleNamespace(msim_route=ok, msim_route_backward=ok, msim_dropout=ok,
                                                                   msim_traffic=ok))
    i32 = lambda *s: gpu(*s, dtype=torch.int32)
    x, ids, w, load, dx, y, table = gpu(4, 8), i32(4, 2), gpu(4, 2), i32(8), gpu(4, 8), gpu(4, 8), i32(2, 5)
    M.route(x, 2, out=M.Routing(ids, w, load))
    M.route_backward(x, ids, w, out=dx)
    M.dropout(x, 0.5, 1, out=y)
    M.traffic(ids, gpu(3, dtype=torch.int64), i32(2), i32(8), 5, out=table)
    assert [t._version for t in (x, ids, w, load, dx, y, table)] == [0, 1, 1, 1, 1, 1, 1]
    M.route(x, 2, out=M.Routing(ids, w, None))
    M.dropout(y, 0.5, 1, out=y)
    assert [t._version for t in (ids, w, load, y)] == [2, 2, 1, 2]

    a = torch.ones(4, 8, requires_grad=True)
    kept = a.exp()                          # exp keeps its result for the backward pass
    M.dropout(kept.detach().as_subclass(type(y)), 0.5, 1, out=kept.detach().as_subclass(type(y)))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.sum().backward()

    with torch.inference_mode():            # tensors made there have no version
        z = gpu(4, 8)
        assert M.dropout(z, 0.5, 1, out=z) is z
