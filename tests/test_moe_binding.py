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
