"""The products at the ends of their ranges, without a GPU: what the calls launch
for no rows, and that no launch is larger than the runtime takes.  A stand-in for
the runtime counts work-items and executes nothing."""

import ctypes as C
import json
import subprocess
import sys

import pytest

from test_moe_launch import ROOT
from test_products import AT, E_ARG, S, layer_spec, linear_spec  # noqa: F401

# grids of 2^32 work-items or more are refused, as the runtime refuses them
RUNTIME = r"""
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3;
int launches;
unsigned grids[256], blocks[256];
int hipLaunchKernel(const void *f, dim3 grid, dim3 block, void **args, size_t lds, void *stream)
{
    if ((unsigned long long)grid.x * block.x >> 32 || !grid.x) return 9;     /* hipErrorInvalidConfiguration */
    if (launches < 256) {
        grids[launches] = grid.x;
        blocks[launches] = block.x;
    }
    launches++;
    return 0;
}
int hipGetLastError(void) { return 0; }
int hipPeekAtLastError(void) { return 0; }
const char *hipGetErrorString(int e) { return "refused"; }
"""

START = r"""
import ctypes as C, json, sys
sys.path.insert(0, sys.argv[2])
S = C.CDLL(sys.argv[1], mode=C.RTLD_GLOBAL)            # before the library that is to use it
from experiment_network_simulation_amd import sim
lib = sim.load_library()
launches = C.c_int.in_dll(S, "launches")
grids, blocks = (C.c_uint * 256).in_dll(S, "grids"), (C.c_uint * 256).in_dll(S, "blocks")
AT, ALL = 4096, 1 << 62

def run(call):
    launches.value = 0
    rc = call()
    return [rc, [[grids[k], blocks[k]] for k in range(min(launches.value, 256))], lib.msim_last_error(None).decode() if rc else ""]

def spec(rows, cols, outs, dtype=2, out_dtype=None, act=0):
    return sim.LinearSpec(sim.ABI_VERSION, dtype, dtype if out_dtype is None else out_dtype, act, cols, outs, rows, cols, cols, outs,
                          outs, outs, cols, cols)

def linear(*a, **k):
    s = spec(*a, **k)
    return run(lambda: lib.msim_linear(C.byref(s), AT, AT, None, None, AT, None, AT, ALL, None))

def backward(rows, cols, outs, dx=AT, dw=AT, db=AT, x=AT, weight=AT, grad=AT, pre=AT, **k):
    s = spec(rows, cols, outs, **k)
    return run(lambda: lib.msim_linear_backward(C.byref(s), x, weight, pre, grad, dx, dw, db, AT, ALL, None))

def orth(count, rows, cols, steps=1, dtype=2):
    s = sim.OrthogonalizeSpec(sim.ABI_VERSION, dtype, count, steps, rows, cols, 1e-7, 3.4445, -4.775, 2.0315, 0)
    return run(lambda: lib.msim_orthogonalize(C.byref(s), AT, AT, AT, ALL, None))
"""


@pytest.fixture(scope="module")
def launched(tmp_path_factory):
    """The answers to a list of calls, texts in terms of START: [code, [[workgroups, threads], ...], why] each."""
    d = tmp_path_factory.mktemp("runtime")
    (d / "s.c").write_text(RUNTIME)
    subprocess.check_call(["gcc", "-shared", "-fPIC", "-O1", "-o", str(d / "s.so"), str(d / "s.c")])

    def ask(calls):
        code = START + "print(json.dumps([" + ", ".join(calls) + "]))"
        r = subprocess.run([sys.executable, "-c", code, str(d / "s.so"), ROOT], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        return json.loads(r.stdout.splitlines()[-1])

    return ask


def test_a_gradient_of_no_rows_reads_no_array(S, launched):  # noqa: F811
    """There is no row of dx then, and x, weight and grad may be NULL: the weight is neither copied nor counted in the workspace,
    whether its rows end on 16 bytes or not."""
    for cols in (64, 65, 1, 7):
        none = "x=None, weight=None, grad=None, pre=None"
        alone, both, aligned = launched([f"backward(0, {cols}, 33, dw=None, db=None, {none})", f"backward(0, {cols}, 33, {none})",
                                         f"backward(0, 64, 33, dx=None, {none})"])
        assert alone[:2] == [0, []], (cols, alone)
        assert both[0] == 0 and len(both[1]) == len(aligned[1]), (cols, both, aligned)
        n, lib = C.c_uint64(9), S.load_library()
        s = linear_spec(S, rows=0, cols=cols, outs=4000, x_stride=cols, weight_stride=cols, out_stride=4000, dx_stride=cols, dweight_stride=cols)
        assert lib.msim_linear_backward_workspace(C.byref(s), None, None, None, 1, 0, 0, C.byref(n)) == 0 and n.value == 0, cols


MOST = (1 << 31) - 1
WIDE = ["linear(1 << 30, 8, 8)", "linear(1 << 30, 8, 8, dtype=0)", f"linear({MOST}, 8, 256)", f"linear({MOST}, 8, 1, dtype=1)",
        f"linear({MOST}, 1, 1, dtype=0)", f"linear({MOST}, 9, 300, act=2)", "linear(1 << 20, 8, 1 << 19)",
        f"backward({MOST}, 8, 8)", f"backward({MOST}, 300, 9, dtype=0, act=1)", f"backward({MOST}, 8, 8, out_dtype=0, dtype=1)",
        "backward(1 << 30, 8, 8, db=None, dw=None)", "backward(100, 1 << 20, 1 << 20)",
        "orth(65536, 8, 8)", "orth(65536, 1, 1)", "orth(65536, 1023, 1024, dtype=0)", "orth(65536, 1, 16384)", "orth(65536, 16384, 1)",
        "orth(65536, 64, 8192, steps=2)", "orth(65536, 65, 66)", "orth(1, 1 << 17, 1 << 18)"]


def test_no_launch_is_larger_than_the_runtime_takes(launched):
    """The largest counts and rows that the calls accept, where what is launched has 2^32 work-items and more in all: every part of
    it is below that, and the parts follow each other in steps of 8 workgroups."""
    large = 0
    large = 0
    for name, (rc, launches, why) in zip(WIDE, launched(WIDE)):
        assert rc == 0, (name, why)
        assert launches and all(0 < g * b < 1 << 32 for g, b in launches), (name, launches)
        for (g, b), (_, after) in zip(launches, launches[1:]):
            if g * b > (1 << 32) - 8 * b - 1:
                large += 1
                assert g % 8 == 0 and after == b, (name, launches)
    assert large >= 8


def test_norms_have_workgroups_for_elements_alone(launched):
    """Of 2,048 elements of 16 bits (1,024 of 32) each, up to 256 a matrix."""
    sizes = [(64, 8, 8, 2, 64), (64, 8, 8, 0, 64), (3, 64, 32, 2, 3), (3, 64, 33, 2, 6), (3, 64, 32, 0, 6), (2, 2048, 7168, 2, 512),
             (1, 100, 8191, 0, 256)]
    for (count, rows, cols, dtype, norm), (rc, launches, why) in zip(sizes, launched([f"orth({c}, {r}, {k}, dtype={d})" for c, r, k, d, _ in sizes])):
        assert rc == 0 and launches[0] == [norm, 256], (count, rows, cols, launches[0])


def test_a_layer_refuses_a_residual_that_is_out_with_another_stride(S):  # noqa: F811
    """As msim_linear: a row of one would be written before it is read as another of the other.  Of one row strides do not count."""
    lib, ws = S.load_library(), 1 << 40
    for rows, want in ((4, E_ARG), (2, E_ARG)):
        s = layer_spec(S, dict(rows=rows), out_stride=64, residual_stride=72)
        assert lib.msim_layer(C.byref(s), AT, AT, None, AT, AT, None, 2 * AT, 2 * AT, AT, AT, None, AT, ws, None) == want
        assert b"two strides" in lib.msim_last_error(None)
