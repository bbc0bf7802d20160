"""Expert-parallel routing without a GPU: the argument checks of the C calls (all
made before any HIP call) and of the binding, the host's reading of the random
stream, and the flows of a traffic matrix."""

import ctypes as C

import numpy as np
import pytest

from experiment_network_simulation_amd import inputs as I

E_ARG, E_LIMIT = -5, -7


@pytest.fixture(scope="module")
def S():
    from experiment_network_simulation_amd import sim
    sim.load_library()
    return sim


def route_spec(S, **kw):
    d = dict(version=S.ABI_VERSION, dtype=0, score=0, experts=8, top_k=2, groups=1, top_groups=1, group_top=1, renorm=1,
             scale=1.0, rows=4, row_stride=8)
    d.update(kw)
    return S.RouteSpec(*[d[n] for n, _ in S.RouteSpec._fields_])


BAD_ROUTE = [
    (dict(version=4), E_ARG, "version"), (dict(dtype=3), E_ARG, "dtype"), (dict(score=2), E_ARG, "score"),
    (dict(experts=0, top_k=0), E_ARG, "at least 1"), (dict(top_k=0), E_ARG, "at least 1"),
    (dict(renorm=2), E_ARG, "renorm"), (dict(scale=float("nan")), E_ARG, "scale"),
    (dict(scale=float("inf")), E_ARG, "scale"), (dict(row_stride=7), E_ARG, "row_stride"),
    (dict(experts=1025, row_stride=1025), E_LIMIT, "experts"),
    (dict(experts=64, row_stride=64, top_k=33), E_LIMIT, "top_k"), (dict(rows=1 << 40), E_LIMIT, "2^40"),
    (dict(row_stride=1 << 40), E_LIMIT, "2^40"),
]
BAD_FORWARD = [
    (dict(groups=3), E_ARG, "divide"), (dict(groups=0), E_ARG, "divide"),
    (dict(groups=4, top_groups=5), E_ARG, "top_groups"), (dict(groups=4, top_groups=0), E_ARG, "top_groups"),
    (dict(group_top=3), E_ARG, "group_top"), (dict(group_top=0), E_ARG, "group_top"),
    (dict(groups=4, top_groups=1, top_k=3), E_ARG, "top_k above"), (dict(top_k=9), E_ARG, "top_k above"),
    (dict(experts=128, row_stride=128, groups=128, top_groups=2), E_LIMIT, "groups"),
]


@pytest.mark.parametrize("bad,code,word", BAD_ROUTE + BAD_FORWARD)
def test_route_refuses(S, bad, code, word):
    lib = S.load_library()
    spec = route_spec(S, **bad)
    assert lib.msim_route(C.byref(spec), 16, None, 16, 16, None, None) == code
    assert word in lib.msim_last_error(None).decode()


@pytest.mark.parametrize("bad,code,word", BAD_ROUTE + [(dict(top_k=9), E_ARG, "top_k above")])
def test_route_backward_refuses(S, bad, code, word):
    lib = S.load_library()
    spec = route_spec(S, **bad)
    assert lib.msim_route_backward(C.byref(spec), 16, 16, 16, 16, 8, None) == code
    assert word in lib.msim_last_error(None).decode()


def test_route_refuses_missing_arrays(S):
    lib = S.load_library()
    spec = route_spec(S)
    assert lib.msim_route(None, 16, None, 16, 16, None, None) == E_ARG
    for a in ([None, 16, 16], [16, None, 16], [16, 16, None]):
        assert lib.msim_route(C.byref(spec), a[0], None, a[1], a[2], None, None) == E_ARG
        assert b"null" in lib.msim_last_error(None)
    assert lib.msim_route_backward(None, 16, 16, 16, 16, 8, None) == E_ARG
    for k in range(4):
        a = [16] * 4
        a[k] = None
        assert lib.msim_route_backward(C.byref(spec), *a, 8, None) == E_ARG
    assert lib.msim_route_backward(C.byref(spec), 16, 16, 16, 16, 7, None) == E_ARG
    assert lib.msim_route_backward(C.byref(spec), 16, 16, 16, 16, 1 << 40, None) == E_LIMIT
    assert lib.msim_route_backward(C.byref(route_spec(S, rows=0)), None, None, None, None, 8, None) == 0


def test_dropout_refuses(S):
    lib = S.load_library()

    def call(dtype=0, x=16, y=32, rows=4, cols=8, xs=8, ys=8, p=0.5, seed=1, offset=0, per_row=0):
        return lib.msim_dropout(dtype, x, y, rows, cols, xs, ys, p, seed, offset, per_row, None)

    for bad in (dict(dtype=3), dict(x=None), dict(y=None), dict(xs=7), dict(ys=7), dict(p=-0.1), dict(p=1.5),
                dict(p=float("nan")), dict(per_row=2), dict(y=16, ys=9)):
        assert call(**bad) == E_ARG, bad
    for bad in (dict(rows=1 << 40), dict(xs=1 << 40), dict(rows=1 << 39, cols=1 << 6, xs=1 << 6, ys=1 << 6)):
        assert call(**bad) == E_LIMIT, bad
    assert call(rows=0, x=None, y=None) == 0 and call(cols=0, x=None, y=None) == 0


def test_traffic_refuses(S):
    lib = S.load_library()

    def call(arrays=(16, 16, 16, 16, 16), **kw):
        d = dict(version=S.ABI_VERSION, experts=8, top_k=2, hosts=4, rows=4, n_seg=2, token_bytes=1, pkt_bytes=1,
                 drop=0.0, seed=0, offset=0, per_row=0, reserved=0)
        d.update(kw)
        spec = S.TrafficSpec(*[d[n] for n, _ in S.TrafficSpec._fields_])
        return lib.msim_traffic(C.byref(spec), *arrays, None)

    for bad in (dict(version=4), dict(experts=0), dict(top_k=0), dict(hosts=0), dict(token_bytes=0), dict(pkt_bytes=0),
                dict(drop=-1.0), dict(drop=1.01), dict(drop=float("nan")), dict(per_row=2), dict(reserved=1)):
        assert call(**bad) == E_ARG, bad
    for bad in (dict(top_k=33), dict(hosts=16385), dict(rows=1 << 32), dict(n_seg=1 << 32), dict(experts=(1 << 24) + 1)):
        assert call(**bad) == E_LIMIT, bad
    for k in range(5):
        a = [16] * 5
        a[k] = None
        assert call(a) == E_ARG, k
    assert lib.msim_traffic(None, 16, 16, 16, 16, 16, None) == E_ARG
    assert call([None] * 5, n_seg=0) == 0


def test_binding_refuses_before_any_call():
    import torch
    from experiment_network_simulation_amd import moe
    x = torch.zeros(4, 8)
    for call in (lambda: moe.route(x, 2), lambda: moe.dropout(x, 0.1, 1),
                 lambda: moe.route_backward(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)),
                 lambda: moe.traffic(torch.zeros(4, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64),
                                     torch.zeros(1, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), 4)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        moe.route([[1.0]], 1)


@pytest.mark.parametrize("seed,offset", [(0, 0), (7, 3), ((1 << 64) - 1, 5), (0xC5, (1 << 33) + 1)])
def test_draws_are_the_generators_outputs(seed, offset):
    """splitmix_draws reads the stream SplitMix64 walks: its first outputs from
    offset 0, and from any offset those of a generator moved on by it."""
    g = I.SplitMix64(seed + offset * 0x9E3779B97F4A7C15)
    assert I.splitmix_draws(seed, 9, offset).tolist() == [g.next() for _ in range(9)]


def test_flows_of_a_traffic_matrix():
    w = I.traffic_flows([[0, 3, 0], [1, 0, 2], [0, 0, 9]])
    assert list(zip(w.xsrc.tolist(), w.xdst.tolist(), w.xpkts.tolist())) == [(0, 1, 3), (1, 0, 1), (1, 2, 2)]
    w = I.traffic_flows([[0, 3, 0], [1, 0, 2], [0, 4, 0]], home=[0, 1, 0])      # two segments on host 0
    assert list(zip(w.xsrc.tolist(), w.xdst.tolist(), w.xpkts.tolist())) == [(0, 1, 7), (1, 0, 1), (1, 2, 2)]
    assert I.traffic_flows(np.zeros((4, 4), np.int32)).xsrc.size == 0
    for home in ([0, 1], [0, 1, 3], [0, 1, -1]):
        with pytest.raises(ValueError):
            I.traffic_flows(np.ones((3, 3)), home)
    most = 0x7FFFFFFF
    assert I.traffic_flows([[0, most], [0, 0], [0, most]], [0, 1, 0]).xpkts.tolist() == [2 * most]
    with pytest.raises(ValueError):
        I.traffic_flows([[0, most]] * 3 + [[1, 0]], [0, 0, 0, 1])


def test_router_designs_are_seeded_and_valid():
    a, b = I.route_design_space(40, 16, 64), I.route_design_space(40, 16, 64)
    for x, y in zip(a, b):
        assert all(np.array_equal(x[k], y[k]) for k in x)
        assert np.array_equal(np.bincount(x["place"], minlength=16), np.full(16, 4))
        assert x["top_k"] <= 64 // x["groups"] * x["top_groups"]
    assert len({d["top_k"] for d in a}) == 3 and len({d["drop"] for d in a}) == 3


def test_gate_logits_are_seeded_and_spread():
    a, b = I.gate_logits(5, 4096, 16), I.gate_logits(5, 4096, 16)
    assert a.dtype == np.float32 and a.shape == (4096, 16) and np.array_equal(a, b)
    assert not np.array_equal(a, I.gate_logits(6, 4096, 16))
    # 4,096 draws of deviation 1.5: the deviation of a column is within 5 of its standard errors
    assert np.all(np.abs(a.std(0) - 1.5) < 5 * 1.5 / np.sqrt(2 * 4096))
