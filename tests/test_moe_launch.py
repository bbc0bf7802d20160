"""What the routing calls make of the runtime's answers, without a GPU: a
stand-in for the launches counts them, refuses one of them, or has an error of
somebody else's pending.  Nothing is executed, so the arrays may be anything."""

import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E_HIP = -4

STAND_IN = r"""
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3;
int launches, refuse_at, pending;
int hipLaunchKernel(const void *f, dim3 grid, dim3 block, void **args, size_t lds, void *stream)
{
    if (++launches != refuse_at) return 0;
    pending = 2;                     /* hipErrorOutOfMemory */
    return 2;
}
int hipGetLastError(void) { int e = pending; pending = 0; return e; }
int hipPeekAtLastError(void) { return pending; }
const char *hipGetErrorString(int e) { return e == 2 ? "refused" : "somebody else's"; }
"""

CALLS = r"""
import ctypes as C, json, sys
sys.path.insert(0, sys.argv[2])
S = C.CDLL(sys.argv[1], mode=C.RTLD_GLOBAL)            # before the library that is to use it
from experiment_network_simulation_amd import sim
lib = sim.load_library()
launches, refuse_at, pending = (C.c_int.in_dll(S, n) for n in ("launches", "refuse_at", "pending"))

def route(rows, experts, k, groups=1, top_groups=1, bias=None, load=16):
    s = sim.RouteSpec(sim.ABI_VERSION, 0, 1, experts, k, groups, top_groups, 1, 1, 1.0, rows, experts)
    return lambda: lib.msim_route(C.byref(s), 16, bias, 16, 16, load, None)

def backward(rows):
    s = sim.RouteSpec(sim.ABI_VERSION, 0, 1, 64, 4, 1, 1, 1, 1, 1.0, rows, 64)
    return lambda: lib.msim_route_backward(C.byref(s), 16, 16, 16, 16, 64, None)

def traffic(rows, segs):
    s = sim.TrafficSpec(sim.ABI_VERSION, 8, 2, 4, rows, segs, 1, 1, 0.0, 0, 0, 0, 0)
    return lambda: lib.msim_traffic(C.byref(s), 16, 16, 16, 16, 16, None)

def dropout(rows, per_row):
    return lambda: lib.msim_dropout(0, 16, 16, rows, 8, 8, 8, 0.5, 1, 0, per_row, None)

calls = {"no rows": (route(0, 8, 2), 1), "one workgroup": (route(8, 64, 2), 1),
         "counted behind": (route(5000, 64, 2), 2), "no load": (route(5000, 64, 2, load=None), 1),
         "undecided rows": (route(8, 64, 2, bias=16), 2), "undecided rows, no load": (route(8, 64, 2, bias=16, load=None), 2),
         "few experts": (route(20000, 8, 2), 2), "few experts, no load": (route(20000, 8, 2, load=None), 1),
         "a wavefront a row": (route(50, 64, 20), 2), "many groups": (route(50, 128, 4, 64, 8), 2),
         "backward": (backward(50), 1), "dropout": (dropout(9, 0), 1), "dropout of rows": (dropout(9, 1), 1),
         "traffic": (traffic(50, 3), 1), "traffic of long segments": (traffic(50000, 3), 3)}
out = {}
for name, (call, n) in calls.items():
    got = []
    for at in range(n + 1):                             # 0: none is refused, another's error is pending
        launches.value, refuse_at.value, pending.value = 0, at, 0 if at else 999
        rc = call()
        got.append([rc, launches.value, pending.value, lib.msim_last_error(None).decode() if rc else ""])
    out[name] = [n, got]
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    d = tmp_path_factory.mktemp("stand_in")
    (d / "s.c").write_text(STAND_IN)
    subprocess.check_call(["gcc", "-shared", "-fPIC", "-O1", "-o", str(d / "s.so"), str(d / "s.c")])
    r = subprocess.run([sys.executable, "-c", CALLS, str(d / "s.so"), ROOT], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.splitlines()[-1])


def test_an_error_that_was_pending_is_its_owners(answers):
    """All launches were accepted: the call succeeded, and whoever left an error finds it where it was."""
    for name, (n, got) in answers.items():
        assert got[0][:3] == [0, n, 999], (name, got[0])


def test_nothing_follows_a_refused_launch(answers):
    for name, (n, got) in answers.items():
        for at in range(1, n + 1):
            rc, launches, pending, why = got[at]
            assert (rc, launches, pending) == (E_HIP, at, 0) and "refused" in why, (name, at, got[at])
