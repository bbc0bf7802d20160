"""The products without a GPU: what the C calls and the binding refuse, what the
calls make of the runtime's answers, and which tensors a call notes on a stream
that is given."""

import contextlib
import ctypes as C
import json
import subprocess
import sys
from types import SimpleNamespace

import pytest
import torch

from test_moe_launch import E_HIP, ROOT, STAND_IN
from test_moe_streams import DEVICE, gpu

E_WORKSPACE, E_ARG, E_LIMIT = -3, -5, -7
AT = 4096                                   # an address that is never followed: on 256 bytes


@pytest.fixture(scope="module")
def S():
    from experiment_network_simulation_amd import sim
    sim.load_library()
    return sim


def linear_spec(S, **kw):
    d = dict(version=S.ABI_VERSION, dtype=2, out_dtype=2, act=0, cols=64, outs=32, rows=8, x_stride=64, weight_stride=64,
             out_stride=32, residual_stride=32, pre_stride=32, dx_stride=64, dweight_stride=64)
    d.update(kw)
    return S.LinearSpec(*[d[n] for n, _ in S.LinearSpec._fields_])


BAD_LINEAR = [
    (dict(version=4), E_ARG, "version"), (dict(dtype=3), E_ARG, "dtype"), (dict(out_dtype=1), E_ARG, "out_dtype"),
    (dict(act=5), E_ARG, "activation"), (dict(cols=0), E_ARG, "at least 1"), (dict(outs=0), E_ARG, "at least 1"),
    (dict(x_stride=63), E_ARG, "x_stride"), (dict(weight_stride=63), E_ARG, "weight_stride"),
    (dict(out_stride=31), E_ARG, "out_stride"), (dict(rows=1 << 31), E_LIMIT, "2^31"),
    (dict(cols=(1 << 20) + 1, x_stride=1 << 21, weight_stride=1 << 21), E_LIMIT, "MAX_LINEAR"),
    (dict(outs=(1 << 20) + 1, out_stride=1 << 21), E_LIMIT, "MAX_LINEAR"),
    (dict(rows=(1 << 31) - 1, cols=1 << 20, x_stride=1 << 20, weight_stride=1 << 20), E_LIMIT, "2^40"),
    (dict(x_stride=1 << 40), E_LIMIT, "stride"), (dict(residual_stride=1 << 40), E_LIMIT, "stride"),
]


@pytest.mark.parametrize("bad,code,word", BAD_LINEAR)
def test_linear_refuses(S, bad, code, word):
    lib, s, n = S.load_library(), linear_spec(S, **bad), C.c_uint64()
    for rc in (lambda: lib.msim_linear(C.byref(s), AT, AT, None, None, AT, None, AT, 1 << 40, None),
               lambda: lib.msim_linear_backward(C.byref(s), AT, AT, AT, AT, AT, AT, AT, AT, 1 << 40, None),
               lambda: lib.msim_linear_workspace(C.byref(s), AT, AT, C.byref(n)),
               lambda: lib.msim_linear_backward_workspace(C.byref(s), AT, AT, AT, 1, 1, 1, C.byref(n))):
        assert rc() == code and word in lib.msim_last_error(None).decode()


def test_linear_refuses_missing_arrays_and_workspaces(S):
    lib, n = S.load_library(), C.c_uint64()
    s = linear_spec(S)
    for k in range(3):
        a = [AT] * 3
        a[k] = None
        assert lib.msim_linear(C.byref(s), a[0], a[1], None, None, a[2], None, None, 0, None) == E_ARG
    assert lib.msim_linear(None, AT, AT, None, None, AT, None, None, 0, None) == E_ARG
    assert lib.msim_linear(C.byref(linear_spec(S, residual_stride=31)), AT, AT, None, AT, 2 * AT, None, None, 0, None) == E_ARG
    assert lib.msim_linear(C.byref(linear_spec(S, residual_stride=40)), AT, AT, None, AT, AT, None, None, 0, None) == E_ARG
    assert b"two strides" in lib.msim_last_error(None)
    assert lib.msim_linear(C.byref(linear_spec(S, pre_stride=31)), AT, AT, None, None, AT, AT, None, 0, None) == E_ARG
    assert lib.msim_linear(C.byref(linear_spec(S, rows=0)), None, None, None, None, None, None, None, 0, None) == 0
    # 333 rows of 65 columns lie on no 16 bytes: both operands are packed
    big = linear_spec(S, rows=333, cols=65, x_stride=65, weight_stride=65)
    assert lib.msim_linear_workspace(C.byref(big), AT, AT, C.byref(n)) == 0 and n.value > 0
    for ws, size in ((None, n.value), (AT, n.value - 1), (AT + 16, n.value)):
        assert lib.msim_linear(C.byref(big), AT, AT, None, None, AT, None, ws, size, None) == E_WORKSPACE
    assert lib.msim_linear_workspace(C.byref(big), AT, AT, None) == E_ARG
    # the backward pass
    assert lib.msim_linear_backward(C.byref(s), None, AT, None, AT, AT, AT, None, AT, 1 << 30, None) == E_ARG
    assert lib.msim_linear_backward(C.byref(s), AT, None, None, AT, AT, None, None, AT, 1 << 30, None) == E_ARG
    assert lib.msim_linear_backward(C.byref(s), AT, AT, None, None, AT, None, None, AT, 1 << 30, None) == E_ARG
    act = linear_spec(S, act=4)
    assert lib.msim_linear_backward(C.byref(act), AT, AT, None, AT, AT, AT, None, AT, 1 << 30, None) == E_ARG
    assert b"needs pre" in lib.msim_last_error(None)
    assert lib.msim_linear_backward(C.byref(linear_spec(S, dx_stride=63)), AT, AT, None, AT, AT, None, None, AT, 1 << 30, None) == E_ARG
    assert lib.msim_linear_backward(C.byref(linear_spec(S, dweight_stride=63)), AT, AT, None, AT, None, AT, None, AT, 1 << 30, None) == E_ARG
    assert lib.msim_linear_backward_workspace(C.byref(act), AT, AT, AT, 1, 1, 1, C.byref(n)) == 0 and n.value > 0
    assert lib.msim_linear_backward(C.byref(act), AT, AT, AT, AT, AT, AT, AT, AT, n.value - 1, None) == E_WORKSPACE


def layer_spec(S, route=(), **kw):
    r = dict(version=S.ABI_VERSION, dtype=0, score=0, experts=8, top_k=2, groups=1, top_groups=1, group_top=1, renorm=1,
             scale=1.0, rows=4, row_stride=8)
    r.update(route)
    d = dict(version=S.ABI_VERSION, dtype=2, act=4, gated=1, cols=64, hidden=32, x_stride=64, out_stride=64, residual_stride=64)
    d.update(kw)
    return S.LayerSpec(*[d[n] for n, _ in S.LayerSpec._fields_[:-1]], S.RouteSpec(*[r[n] for n, _ in S.RouteSpec._fields_]))


BAD_LAYER = [
    (dict(version=4), {}, E_ARG, "version"), (dict(dtype=3), {}, E_ARG, "dtype"), (dict(act=5), {}, E_ARG, "activation"),
    (dict(gated=2), {}, E_ARG, "gated"), (dict(cols=0), {}, E_ARG, "at least 1"), (dict(hidden=0), {}, E_ARG, "at least 1"),
    (dict(x_stride=63), {}, E_ARG, "x_stride"), (dict(out_stride=63), {}, E_ARG, "out_stride"),
    ({}, dict(dtype=2), E_ARG, "32-bit"), ({}, dict(row_stride=9), E_ARG, "32-bit"), ({}, dict(top_k=9), E_ARG, "top_k above"),
    ({}, dict(experts=1025, row_stride=1025), E_LIMIT, "experts"), ({}, dict(score=2), E_ARG, "score"),
    ({}, dict(scale=float("nan")), E_ARG, "scale"), ({}, dict(rows=513), E_LIMIT, "MAX_LAYER_ROWS"),
    (dict(hidden=(1 << 20) + 1), {}, E_LIMIT, "MAX_LINEAR"), (dict(hidden=1 << 20), dict(experts=16, row_stride=16), E_LIMIT, "2^24"),
    (dict(x_stride=1 << 40), {}, E_LIMIT, "stride"),
]


@pytest.mark.parametrize("bad,route,code,word", BAD_LAYER)
def test_layer_refuses(S, bad, route, code, word):
    lib, s, n = S.load_library(), layer_spec(S, route, **bad), C.c_uint64()
    assert lib.msim_layer(C.byref(s), AT, AT, None, AT, AT, None, None, AT, AT, AT, None, AT, 1 << 40, None) == code
    assert word in lib.msim_last_error(None).decode()
    assert lib.msim_layer_workspace(C.byref(s), C.byref(n)) == code


def test_layer_refuses_missing_arrays_and_workspaces(S):
    lib, n, s = S.load_library(), C.c_uint64(), layer_spec(S)
    for k in range(7):
        a = [AT] * 7
        a[k] = None
        assert lib.msim_layer(C.byref(s), a[0], a[1], None, a[2], a[3], None, None, a[4], a[5], a[6], None, AT, 1 << 30, None) == E_ARG
    assert lib.msim_layer(C.byref(layer_spec(S, residual_stride=63)), AT, AT, None, AT, AT, None, AT, AT, AT, AT, None, AT, 1 << 30, None) == E_ARG
    assert lib.msim_layer_workspace(C.byref(s), C.byref(n)) == 0 and n.value > 0
    for ws, size in ((None, n.value), (AT, n.value - 1), (AT + 16, n.value)):
        assert lib.msim_layer(C.byref(s), AT, AT, None, AT, AT, None, None, AT, AT, AT, None, ws, size, None) == E_WORKSPACE
    assert lib.msim_layer(None, AT, AT, None, AT, AT, None, None, AT, AT, AT, None, AT, 1, None) == E_ARG
    assert lib.msim_layer_workspace(C.byref(s), None) == E_ARG


def orth_spec(S, **kw):
    d = dict(version=S.ABI_VERSION, dtype=2, count=1, steps=5, rows=8, cols=16, eps=1e-7, a=3.4445, b=-4.775, c=2.0315, reserved=0)
    d.update(kw)
    return S.OrthogonalizeSpec(*[d[n] for n, _ in S.OrthogonalizeSpec._fields_])


BAD_ORTH = [
    (dict(version=4), E_ARG, "version"), (dict(dtype=3), E_ARG, "dtype"), (dict(rows=0), E_ARG, "at least 1"),
    (dict(cols=0), E_ARG, "at least 1"), (dict(reserved=1), E_ARG, "reserved"), (dict(eps=-1.0), E_ARG, "eps"),
    (dict(eps=float("nan")), E_ARG, "eps"), (dict(eps=float("inf")), E_ARG, "eps"), (dict(steps=65), E_LIMIT, "steps"),
    (dict(rows=(1 << 20) + 1), E_LIMIT, "MAX_LINEAR"), (dict(count=65537), E_LIMIT, "65,536"),
    (dict(rows=1 << 20, cols=1 << 20), E_LIMIT, "2^36"),
    # 30 grows past 24 in one step, 3 in three; NaN is no bound
    (dict(a=30.0, b=0.0, c=0.0), E_ARG, "range"), (dict(a=3.0, b=0.0, c=0.0), E_ARG, "range"),
    (dict(a=float("nan")), E_ARG, "range"), (dict(c=float("inf")), E_ARG, "range"), (dict(b=-40.0, c=40.0), E_ARG, "range"),
]


@pytest.mark.parametrize("bad,code,word", BAD_ORTH)
def test_orthogonalize_refuses(S, bad, code, word):
    lib, s, n = S.load_library(), orth_spec(S, **bad), C.c_uint64()
    assert lib.msim_orthogonalize(C.byref(s), AT, AT, AT, 1 << 40, None) == code
    assert word in lib.msim_last_error(None).decode()
    assert lib.msim_orthogonalize_workspace(C.byref(s), C.byref(n)) == code


def test_orthogonalize_takes_what_stays_in_range(S):
    lib, n = S.load_library(), C.c_uint64()
    for kw in (dict(), dict(steps=0), dict(steps=64), dict(a=1.5, b=-0.5, c=0.0, steps=30), dict(a=3.0, b=0.0, c=0.0, steps=2),
               dict(a=2.0, b=-1.5, c=0.5)):
        assert lib.msim_orthogonalize_workspace(C.byref(orth_spec(S, **kw)), C.byref(n)) == 0 and n.value > 0
    s = orth_spec(S)
    assert lib.msim_orthogonalize(C.byref(s), None, AT, AT, n.value, None) == E_ARG
    assert lib.msim_orthogonalize(C.byref(s), AT, None, AT, n.value, None) == E_ARG
    assert lib.msim_orthogonalize(C.byref(s), AT, AT, None, 1 << 30, None) == E_WORKSPACE
    assert lib.msim_orthogonalize(C.byref(s), AT, AT, AT, 1, None) == E_WORKSPACE
    assert lib.msim_orthogonalize(C.byref(orth_spec(S, count=0)), None, None, None, 0, None) == 0
    assert lib.msim_orthogonalize_workspace(C.byref(s), None) == E_ARG


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------


class Calls:
    """Stands in for the library: asks for no workspace and takes every call."""

    def __getattr__(self, name):
        def call(*a):
            if name.endswith("_workspace"):
                a[-1]._obj.value = 0
            return 0
        return call


@pytest.fixture
def M(monkeypatch):
    from experiment_network_simulation_amd import moe
    monkeypatch.setattr(moe, "load_library", lambda: Calls())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: SimpleNamespace(device=device, cuda_stream=h))
    return moe


def on():
    return SimpleNamespace(device=DEVICE, cuda_stream=0x5150)


def bf(*shape):
    return gpu(*shape, dtype=torch.bfloat16)


BAD_CALLS = [
    lambda M: M.linear(bf(4, 8), bf(5, 9), stream=on()),                                    # columns
    lambda M: M.linear(bf(4, 8), gpu(5, 8), stream=on()),                                   # types
    lambda M: M.linear(bf(4, 8, 1), bf(5, 8), stream=on()),
    lambda M: M.linear(bf(4, 8), bf(5, 8), bf(5), stream=on()),                             # a bias is float32
    lambda M: M.linear(bf(4, 8), bf(5, 8), gpu(4), stream=on()),
    lambda M: M.linear(bf(4, 8), bf(5, 8), act="tanh", stream=on()),
    lambda M: M.linear(bf(4, 8), bf(5, 8), residual=gpu(4, 5), stream=on()),                # of the result's type
    lambda M: M.linear(bf(4, 8), bf(5, 8), residual=bf(4, 6), stream=on()),
    lambda M: M.linear(bf(4, 8), bf(5, 8), out_dtype=torch.float16, stream=on()),
    lambda M: M.linear(bf(4, 8), bf(5, 8), pre=gpu(4, 5), stream=on()),
    lambda M: M.linear(bf(4, 8), bf(5, 8), out=gpu(4, 5), stream=on()),
    lambda M: M.linear(bf(4, 0), bf(5, 0), stream=on()),
    lambda M: M.linear(bf(4, 8), bf(0, 8), stream=on()),
    lambda M: M.linear(bf(8, 4).t(), bf(5, 8), stream=on()),
    lambda M: M.linear(torch.zeros(4, 8), torch.zeros(5, 8)),                               # not on a GPU
    lambda M: M.linear_backward(bf(4, 8), bf(5, 8), gpu(4, 5, dtype=torch.float16), stream=on()),
    lambda M: M.linear_backward(bf(4, 8), bf(5, 8), bf(4, 6), stream=on()),
    lambda M: M.linear_backward(bf(4, 8), bf(5, 8), bf(4, 5), act="silu", stream=on()),     # without pre
    lambda M: M.linear_backward(bf(4, 8), bf(5, 8), bf(4, 5), act="silu", pre=gpu(4, 5), stream=on()),
    lambda M: M.linear_backward(bf(4, 8), bf(5, 8), bf(4, 5), out=M.LinearGrads(bf(4, 8), bf(5, 9), None), stream=on()),
    lambda M: M.layer(bf(4, 8), bf(6, 9), bf(6, 10, 8), bf(6, 8, 5), 2, stream=on()),
    lambda M: M.layer(bf(4, 8), bf(6, 8), bf(6, 5, 8), bf(6, 8, 5), 2, stream=on()),        # gated: twice as many rows
    lambda M: M.layer(bf(4, 8), bf(6, 8), bf(6, 10, 8), bf(6, 8, 5), 7, stream=on()),
    lambda M: M.layer(bf(4, 8), bf(6, 8), bf(6, 10, 8), bf(6, 8, 5), 2, mask=gpu(4), stream=on()),
    lambda M: M.layer(bf(4, 8), bf(6, 8), bf(6, 10, 8), bf(6, 8, 5), 2, bias=gpu(5), stream=on()),
    lambda M: M.layer(bf(4, 8), bf(6, 8), bf(6, 10, 8), bf(6, 8, 5), 2, residual=bf(4, 9), stream=on()),
    lambda M: M.layer(bf(4, 8), bf(6, 8), bf(6, 10, 8), bf(6, 8, 5), 2, score="tanh", stream=on()),
    lambda M: M.layer(bf(4, 8), bf(6, 8), bf(6, 10, 8)[:, ::2], bf(6, 8, 5), 2, gated=False, stream=on()),
    lambda M: M.orthogonalize(bf(4), stream=on()),
    lambda M: M.orthogonalize(bf(4, 8).t(), stream=on()),
    lambda M: M.orthogonalize(gpu(4, 8, dtype=torch.float64), stream=on()),
    lambda M: M.orthogonalize(bf(0, 8), stream=on()),
    lambda M: M.orthogonalize(bf(4, 8), steps=65, stream=on()),
    lambda M: M.orthogonalize(bf(4, 8), steps=float("inf"), stream=on()),
    lambda M: M.orthogonalize(bf(4, 8), coefficients=(1.0, 2.0), stream=on()),
    lambda M: M.orthogonalize(bf(4, 8), out=gpu(4, 8), stream=on()),
    lambda M: M.orthogonalize([[1.0]], stream=on()),
]


@pytest.mark.parametrize("n", range(len(BAD_CALLS)))
def test_the_binding_refuses(M, n):
    with pytest.raises((ValueError, TypeError)):
        BAD_CALLS[n](M)


def good_calls(M):
    """(tensors of a call, those it writes, the call on a stream)"""
    i32 = lambda *s: gpu(*s, dtype=torch.int32)
    x, w, b, r, pre, y = bf(4, 8), bf(5, 8), gpu(5), bf(4, 5), bf(4, 5), bf(4, 5)
    yield [x, w, b, r, pre, y], [pre, y], lambda s: M.linear(x, w, b, act="gelu", residual=r, pre=pre, out=y, stream=s)
    x2, w2, g2, p2, dx, dw, db = bf(4, 8), bf(5, 8), gpu(4, 5), bf(4, 5), bf(4, 8), bf(5, 8), gpu(5)
    yield [x2, w2, g2, p2, dx, dw, db], [dx, dw, db], \
        lambda s: M.linear_backward(x2, w2, g2, act="silu", pre=p2, out=M.LinearGrads(dx, dw, db), stream=s)
    x3, g3, wi, wo, b3, m3, r3 = bf(4, 8), bf(6, 8), bf(6, 10, 8), bf(6, 8, 5), gpu(6), gpu(4, dtype=torch.bool), bf(4, 8)
    y3, ids, ww, load = bf(4, 8), i32(4, 2), gpu(4, 2), i32(6)
    yield [x3, g3, wi, wo, b3, m3, r3, y3, ids, ww, load], [y3, ids, ww, load], \
        lambda s: M.layer(x3, g3, wi, wo, 2, bias=b3, mask=m3, residual=r3, out=M.Layer(y3, M.Routing(ids, ww, load)), stream=s)
    u, o = bf(3, 4, 8), bf(3, 4, 8)
    yield [u, o], [o], lambda s: M.orthogonalize(u, out=o, stream=s)


def test_every_tensor_of_a_call_is_noted_and_what_it_writes_is_changed(M):
    for n, (tensors, written, call) in enumerate(good_calls(M)):
        s = on()
        call(s)
        assert all(s in getattr(t, "on", []) for t in tensors), n
        assert [t._version for t in written] == [1] * len(written), n
        assert all(t._version == 0 for t in tensors if not any(t is v for v in written)), n
        with pytest.raises(ValueError, match="stream is on"):
            call(SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0x5150))


# ---------------------------------------------------------------------------
# the runtime's answers
# ---------------------------------------------------------------------------

CALLS = r"""
import ctypes as C, json, sys
sys.path.insert(0, sys.argv[2])
S = C.CDLL(sys.argv[1], mode=C.RTLD_GLOBAL)            # before the library that is to use it
from experiment_network_simulation_amd import sim
lib = sim.load_library()
launches, refuse_at, pending = (C.c_int.in_dll(S, n) for n in ("launches", "refuse_at", "pending"))
AT, ALL = 4096, 1 << 40

def linear(rows, cols, outs, dtype=2, xs=None):
    s = sim.LinearSpec(sim.ABI_VERSION, dtype, dtype, 0, cols, outs, rows, xs or cols, cols, outs, outs, outs, cols, cols)
    return lambda: lib.msim_linear(C.byref(s), AT, AT, None, None, AT, None, AT, ALL, None)

def backward(rows, cols, outs, act=0, dx=AT, dw=AT, db=AT):
    s = sim.LinearSpec(sim.ABI_VERSION, 2, 2, act, cols, outs, rows, cols, cols, outs, outs, outs, cols, cols)
    return lambda: lib.msim_linear_backward(C.byref(s), AT, AT, AT, AT, dx, dw, db, AT, ALL, None)

def layer(rows, bias=None):
    r = sim.RouteSpec(sim.ABI_VERSION, 0, 1, 64, 4, 1, 1, 1, 1, 1.0, rows, 64)
    s = sim.LayerSpec(sim.ABI_VERSION, 2, 4, 1, 64, 32, 64, 64, 64, r)
    return lambda: lib.msim_layer(C.byref(s), AT, AT, bias, AT, AT, None, None, AT, AT, AT, AT, AT, ALL, None)

def orth(steps, rows, cols, count=1):
    s = sim.OrthogonalizeSpec(sim.ABI_VERSION, 0, count, steps, rows, cols, 1e-7, 3.4445, -4.775, 2.0315, 0)
    return lambda: lib.msim_orthogonalize(C.byref(s), AT, AT, AT, ALL, None)

calls = {"no rows": linear(0, 8, 8), "few rows": linear(8, 64, 64), "whole": linear(4096, 256, 4096),
         "packed": linear(500, 65, 70), "in parts": linear(100, 8192, 64), "backward": backward(100, 64, 64),
         "backward of nothing": backward(0, 64, 64), "through an activation": backward(3000, 64, 64, 4),
         "one gradient": backward(3000, 64, 64, 0, None, AT, None), "bias alone": backward(3000, 64, 64, 0, None, None, AT),
         "one token": layer(1), "tokens": layer(40), "tokens with bias": layer(40, AT), "no tokens": layer(0),
         "updates": orth(2, 64, 128), "no step": orth(0, 8, 8), "many rows": orth(2, 65, 128), "long update": orth(2, 64, 20000), "no update": orth(5, 8, 8, 0)}
out = {}
for name, call in calls.items():
    got, n, at = [], 0, 0
    while at <= n:                                     # 0: none is refused, another's error is pending
        launches.value, refuse_at.value, pending.value = 0, at, 0 if at else 999
        rc = call()
        if not at:
            n = launches.value
        got.append([rc, launches.value, pending.value, lib.msim_last_error(None).decode() if rc else ""])
        at += 1
    out[name] = [n, got]
print(json.dumps(out))
"""


def test_each_launch_answers_for_itself(tmp_path):
    (tmp_path / "s.c").write_text(STAND_IN)
    subprocess.check_call(["gcc", "-shared", "-fPIC", "-O1", "-o", str(tmp_path / "s.so"), str(tmp_path / "s.c")])
    r = subprocess.run([sys.executable, "-c", CALLS, str(tmp_path / "s.so"), ROOT], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    answers = json.loads(r.stdout.splitlines()[-1])
    for name, (n, got) in answers.items():
        assert got[0][:3] == [0, n, 999], (name, got[0])           # another's error stays its owner's
        for at in range(1, n + 1):                                  # and nothing follows a refused launch
            rc, launches, pending, why = got[at]
            assert (rc, launches, pending) == (E_HIP, at, 0) and "refused" in why, (name, at, got[at])
    few = {name: n for name, (n, _) in answers.items()}
    assert few["no rows"] == few["no update"] == 0 and few["no tokens"] == 1
    assert few["few rows"] == few["whole"] == 1 and few["packed"] == 2 and few["one token"] == 3
    assert few["backward"] == 2 and few["bias alone"] == 2
    # up to 64 rows: a norm, a launch that reads the update, one a step; otherwise a norm, a move, three products a step, a move
    assert few["no step"] == 2 and few["updates"] == 4
    assert few["many rows"] >= 9
    # a pass of two steps over X: P, a + B, (a + B) P, that times a + B, the next a + B, their product, and the update; P is joined
    assert few["long update"] == 11
