"""Linear layers, their gradient, layers of experts and orthogonal updates on the
GPU against plain implementations in 64 bits.

Tolerances.  A sum of n products is made in 32 bits by matrix instructions that
add at least two products at a time, each addition off by at most 2^-23 (a
truncation) of a partial sum, which is at most S, the sum of the products'
magnitudes; joining parts adds fewer than 8 more: SUM(n) S with SUM(n) = (n / 2 +
8) 2^-23.  Where all products and partial sums are whole numbers below 2^24 the
sum is exact, in any order, and the result is the exact one rounded once.  A
rounding to type t is off by eps / 2 = U[t] relative.  Activations are off by 2^-20
relative to |z| + |value| (an exponential, a reciprocal and a polynomial with
an error of 2^-23 in the share of a normal distribution), and no slope of theirs
exceeds 1.13.
"""

import math

import pytest

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def T():
    import torch
    torch.cuda.set_device(0)
    return torch


@pytest.fixture(scope="module")
def M(T):
    from experiment_network_simulation_amd import moe
    return moe


@pytest.fixture(scope="module")
def types(T):
    return {"f32": T.float32, "f16": T.float16, "bf16": T.bfloat16}


U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def SUM(n):
    return (n / 2 + 8) * 2.0 ** -23


def act64(T, z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z * T.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * T.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + T.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope64(T, z, act):
    z = z.detach().clone().requires_grad_(True)
    return T.autograd.grad(act64(T, z, act).sum(), z)[0]


def wide(T, rows, cols, pad, make):
    """rows x cols, or a slice of a wider tensor that begins at an odd element"""
    t = make(rows, cols + pad)
    return t[:, pad - pad // 2:pad - pad // 2 + cols] if pad else t


def whole(T, g, dt, lo=-3, hi=3):
    return lambda *s: T.randint(lo, hi + 1, s, generator=g, device=DEV).to(dt)


def real(T, g, dt, scale=1.0):
    return lambda *s: (scale * T.randn(*s, generator=g, device=DEV)).to(dt)


def gen(T, seed):
    g = T.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# rows x cols -> outs: single elements, edges of every tile, few rows, parts of k, large tiles
SHAPES = [(1, 1, 1), (1, 8, 1), (3, 7, 5), (16, 64, 16), (17, 129, 33), (32, 1000, 100), (33, 2048, 64), (64, 31, 257),
          (65, 64, 64), (65, 8, 9), (100, 8192, 40), (128, 128, 128), (129, 127, 63), (200, 72, 520), (257, 260, 258),
          (1000, 96, 1000), (70, 5000, 70), (2049, 64, 1030), (4100, 128, 2050)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_linear_of_whole_numbers_is_exact(T, M, types, dt, pad):
    for n, (rows, cols, outs) in enumerate(SHAPES):
        g, t = gen(T, n), types[dt]
        x, w = wide(T, rows, cols, pad, whole(T, g, t)), wide(T, outs, cols, pad, whole(T, g, t))
        b = whole(T, g, T.float32)(outs)
        out_dtype = T.float32 if n % 2 else t
        r = wide(T, rows, outs, pad, whole(T, g, out_dtype))
        z = x.double() @ w.double().T
        print("linear", dt, pad, rows, cols, outs, flush=True)
        for act, bias, res in (("none", None, None), ("relu", b, r), ("none", b, None), ("none", None, r)):
            pre = T.full((rows, outs), 9.0, device=DEV, dtype=t) if act == "relu" else None
            out = wide(T, rows, outs, pad, lambda *s: T.full(s, 77.0, device=DEV, dtype=out_dtype)) if res is not None else None
            y = M.linear(x, w, bias, act=act, residual=res, out_dtype=out_dtype, pre=pre, out=out)
            want = z + bias.double() if bias is not None else z
            if pre is not None:
                assert T.equal(pre, want.to(t)), "pre"
            want = act64(T, want, act)
            want = want + res.double() if res is not None else want
            assert y.dtype == out_dtype and T.equal(y, want.to(out_dtype)), (rows, cols, outs, act)
            if out is not None and pad:           # nothing is written beside the rows
                base = out._base
                assert int((base != 77.0).sum()) == int((out != 77.0).sum())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
def test_linear_against_64_bits(T, M, types, dt, act):
    for n, (rows, cols, outs, pad) in enumerate([(5, 300, 40, 0), (40, 333, 65, 3), (300, 520, 200, 0), (130, 777, 131, 5),
                                                 (2100, 256, 1024, 0)]):
        g, t = gen(T, 100 + n), types[dt]
        x, w = wide(T, rows, cols, pad, real(T, g, t)), wide(T, outs, cols, pad, real(T, g, t, 2 / math.sqrt(cols)))
        b, r = real(T, g, T.float32, 0.5)(outs), wide(T, rows, outs, pad, real(T, g, t))
        y = M.linear(x, w, b, act=act, residual=r)
        z, S = x.double() @ w.double().T + b.double(), x.double().abs() @ w.double().abs().T + b.double().abs()
        a = act64(T, z, act)
        want = a + r.double()
        tol = 1.13 * SUM(cols) * S + (2 ** -20) * (z.abs() + a.abs()) + 2 ** -23 * (a.abs() + r.double().abs()) + U[dt] * want.abs() \
            + (2.0 ** -25 if dt == "f16" else 0)
        bad = (y.double() - want).abs() > tol
        print(dt, act, rows, cols, outs, float(((y.double() - want).abs() / tol).max()), flush=True)
        assert not bool(bad.any())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_gradients_of_whole_numbers_are_exact(T, M, types, dt, pad):
    for n, (rows, cols, outs) in enumerate(SHAPES + [(20000, 16, 24), (0, 16, 24)]):
        g, t = gen(T, 1000 + n), types[dt]
        x, w = wide(T, rows, cols, pad, whole(T, g, t)), wide(T, outs, cols, pad, whole(T, g, t))
        grad = wide(T, rows, outs, pad, whole(T, g, T.float32 if n % 2 else t, -2, 2))
        print("gradient", dt, pad, rows, cols, outs, flush=True)
        # relu's slope at whole numbers is 0 or 1
        for act in ("none", "relu"):
            pre = wide(T, rows, outs, pad, whole(T, g, t)) if act == "relu" else None
            d = grad.double() * (pre.double() > 0) if act == "relu" else grad.double()
            dx, dw, db = M.linear_backward(x, w, grad, act=act, pre=pre)
            assert T.equal(dx, (d @ w.double()).to(t)) and T.equal(dw, (d.T @ x.double()).to(t)), (rows, cols, outs, act)
            assert T.equal(db, d.sum(0).float())
        # one of them at a time, and into rows of a wider tensor
        out = M.LinearGrads(wide(T, rows, cols, pad, whole(T, g, t, 7, 7)), None, None)
        got = M.linear_backward(x, w, grad, out=out)
        assert got is out and T.equal(out.x, (grad.double() @ w.double()).to(t))
        out = M.LinearGrads(None, wide(T, outs, cols, pad, whole(T, g, t, 7, 7)), None)
        M.linear_backward(x, w, grad, out=out)
        assert T.equal(out.weight, (grad.double().T @ x.double()).to(t))
        got = M.linear_backward(x, w, grad, need_x=False, need_weight=False)
        assert got.x is None and got.weight is None and T.equal(got.bias, grad.double().sum(0).float())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_64_bits(T, M, types, dt, act):
    for n, (rows, cols, outs, pad) in enumerate([(5, 300, 40, 0), (260, 333, 65, 3), (1300, 100, 200, 0), (2050, 256, 264, 0)]):
        g, t = gen(T, 200 + n), types[dt]
        x, w = wide(T, rows, cols, pad, real(T, g, t)), wide(T, outs, cols, pad, real(T, g, t, 1 / math.sqrt(cols)))
        gr = wide(T, rows, outs, pad, real(T, g, T.float32 if n % 2 else t))
        pre = None if act == "none" else wide(T, rows, outs, pad, real(T, g, t, 2.0))
        dx, dw, db = M.linear_backward(x, w, gr, act=act, pre=pre)
        slope = T.ones_like(gr, dtype=T.float64) if pre is None else slope64(T, pre.double(), act)
        d = gr.double() * slope
        # the gradient in front of the activation: the slope's error, then a rounding
        ed = gr.double().abs() * 2 ** -20 * (2 + (pre.double().abs() if pre is not None else 0)) + d.abs() * (U[dt] + 2 ** -23) \
            + (2.0 ** -25 if dt == "f16" else 0)
        for what, got, want, tol in (
                ("x", dx, d @ w.double(), ed @ w.double().abs() + SUM(outs) * (d.abs() @ w.double().abs())),
                ("weight", dw, d.T @ x.double(), ed.T @ x.double().abs() + SUM(rows) * (d.abs().T @ x.double().abs())),
                ("bias", db, d.sum(0), ed.sum(0) + rows * 2 ** -24 * d.abs().sum(0))):
            tol = tol + U[dt if what != "bias" else "f32"] * want.abs() + 2.0 ** -25
            worst = float(((got.double() - want).abs() / tol).max())
            print(dt, act, rows, cols, outs, what, worst, flush=True)
            assert worst <= 1


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_gradients_against_differences(T, M, act):
    """Along a direction: (f(+h) - f(-h)) / 2h is off by h^2 / 6 times the third derivative (at most 1.7 for these) and by
    the values' error over h."""
    g = gen(T, 7)
    rows, cols, outs, h = 33, 40, 50, 2.0 ** -7
    x, w, b = real(T, g, T.float32)(rows, cols), real(T, g, T.float32, 0.2)(outs, cols), real(T, g, T.float32)(outs)
    gr = real(T, g, T.float32)(rows, outs)
    pre = T.empty(rows, outs, device=DEV)
    y = M.linear(x, w, b, act=act, pre=pre)
    grads = M.linear_backward(x, w, gr, act=act, pre=pre)
    ux, uw, ub = real(T, g, T.float32)(rows, cols), real(T, g, T.float32, 0.2)(outs, cols), real(T, g, T.float32)(outs)
    for dx, dw, db in ((ux, 0 * uw, 0 * ub), (0 * ux, uw, 0 * ub), (0 * ux, 0 * uw, ub)):
        f = [float((M.linear(x + s * dx, w + s * dw, b + s * db, act=act).double() * gr.double()).sum()) for s in (h, -h)]
        got = float((grads.x.double() * dx.double()).sum() + (grads.weight.double() * dw.double()).sum() + (grads.bias.double() * db.double()).sum())
        dz = (dx.double() @ w.double().T + x.double() @ dw.double().T + db.double()).abs()
        z = pre.double().abs() + h * dz
        tol = float((gr.double().abs() * (1.7 * dz ** 3 * h * h / 6 + (2 * 2 ** -20 * z + 1.2 * SUM(cols) * (x.double().abs() @ w.double().abs().T + 2)) / h)).sum())
        assert abs((f[0] - f[1]) / (2 * h) - got) <= tol, (act, f, got, tol)
        assert tol < 0.2 * float((gr.double().abs() * dz).sum())       # and that says something


def test_linear_carries_what_is_not_finite(T, M):
    """An infinity or NaN reaches the results of its row, or of its output, and no other."""
    for rows, cols, outs in ((5, 40, 33), (300, 136, 150)):
        g = gen(T, rows)
        x, w = real(T, g, T.bfloat16)(rows, cols), real(T, g, T.bfloat16)(outs, cols)
        clean = M.linear(x, w, act="silu")
        x[3, 7], x[4, 1], w[20, 2] = math.nan, math.inf, math.nan
        y = M.linear(x, w, act="silu")
        hit = T.zeros(rows, outs, dtype=T.bool, device=DEV)
        hit[3], hit[4], hit[:, 20] = True, True, True
        assert T.equal(y[~hit], clean[~hit])
        assert bool(y[3].isnan().all()) and bool(y[:, 20].isnan().all())
        inf = x[4].double() @ w.double().T
        assert T.equal(y[4].isnan(), (inf.isnan() | (inf == -math.inf))) and bool((y[4][inf == math.inf] == math.inf).all())


def test_linear_in_place_and_again(T, M):
    """The residual may be the output, and the same call gives the same bits."""
    for rows, cols, outs in ((40, 512, 65), (100, 8192, 40), (600, 640, 520)):
        g = gen(T, outs)
        x, w, r = real(T, g, T.float16)(rows, cols), real(T, g, T.float16)(outs, cols), real(T, g, T.float16)(rows, outs)
        y = M.linear(x, w, act="gelu", residual=r)
        assert T.equal(y, M.linear(x, w, act="gelu", residual=r))
        assert M.linear(x, w, act="gelu", residual=r, out=r) is r and T.equal(r, y)
        gr = real(T, g, T.float16)(rows, outs)
        for a, b in zip(M.linear_backward(x, w, gr), M.linear_backward(x, w, gr)):
            assert T.equal(a, b)


# ---------------------------------------------------------------------------
# a layer of experts
# ---------------------------------------------------------------------------


def layer_of(T, seed, dt, rows, cols, hidden, experts, gated=True, pad=0):
    g = gen(T, seed)
    n = 2 * hidden if gated else hidden
    return (wide(T, rows, cols, pad, real(T, g, dt)), real(T, g, dt, 1.5 / math.sqrt(cols))(experts, cols),
            real(T, g, dt, 1 / math.sqrt(cols))(experts, n, cols), real(T, g, dt, 1 / math.sqrt(hidden))(experts, cols, hidden), g)


def check_layer(T, M, dt, args, top_k, how, act, gated, mask, res, out=None):
    """The routing is route()'s own on the exact logits, y is within its bound."""
    x, gate, w_in, w_out, _ = args
    rows, hidden = x.shape[0], w_out.shape[2]
    r = M.layer(x, gate, w_in, w_out, top_k, act=act, gated=gated, mask=mask, residual=res, out=out, **how)
    logits = (x.double() @ gate.double().T).float()
    if mask is not None:
        logits = T.where(mask[:, None], logits, T.full_like(logits, -math.inf))
    want = M.route(logits, top_k, **how)
    assert T.equal(r.routing.ids, want.ids) and T.equal(r.routing.load, want.load)
    assert T.allclose(r.routing.weights, want.weights, rtol=2.0 ** -16, atol=0, equal_nan=True)
    y, tol = T.zeros_like(x, dtype=T.float64), T.zeros_like(x, dtype=T.float64)
    u = U[dt]
    for e in want.ids[want.ids >= 0].unique().tolist():
        t, k = (want.ids == e).nonzero(as_tuple=True)
        xe, wi, wo = x[t].double(), w_in[e].double(), w_out[e].double()
        a, S = xe @ wi.T, SUM(x.shape[1]) * (xe.abs() @ wi.abs().T)
        p = act64(T, a[:, :hidden], act)
        ep = 1.13 * S[:, :hidden] + 2 ** -20 * (a[:, :hidden].abs() + p.abs())
        if gated:
            b, eb = a[:, hidden:], S[:, hidden:]
            h, eh = p * b, ep * b.abs() + (p.abs() + ep) * eb
        else:
            h, eh = p, ep
        eh = eh + (u + 2 ** -23) * h.abs() + (2.0 ** -25 if dt == "f16" else 0)
        s = want.weights[t, k].double()[:, None].abs()
        o, S = h @ wo.T, (h.abs() + eh) @ wo.abs().T
        y[t] += want.weights[t, k].double()[:, None] * o
        tol[t] += s * (eh @ wo.abs().T + (SUM(hidden) + 2.0 ** -16) * S)
    tol += top_k * 2 ** -23 * (y.abs() + tol)
    if res is not None:
        y += res.double()
    tol += (u + 2 ** -23) * y.abs() + (2.0 ** -25 if dt == "f16" else 0)
    void = want.weights.isnan().any(1)
    assert bool(r.y[void].isnan().all())
    worst = ((r.y[~void].double() - y[~void]).abs() / tol[~void].clamp_min(1e-300)).max() if bool((~void).any()) else 0.0
    assert float(worst) <= 1, float(worst)
    return r


LAYERS = [
    # rows, cols, hidden, experts, top_k
    (1, 64, 32, 8, 2), (1, 2048, 256, 64, 8), (2, 7, 3, 300, 8), (3, 1000, 520, 40, 6), (4, 129, 33, 9, 1), (4, 256, 64, 4, 4),
    (5, 64, 32, 8, 2), (16, 320, 100, 16, 4), (17, 257, 129, 9, 2), (33, 72, 40, 3, 3), (40, 512, 64, 5, 1), (65, 100, 48, 2, 1),
    (100, 264, 136, 24, 3), (200, 128, 64, 1, 1), (512, 64, 16, 12, 2), (512, 33, 17, 1, 1),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gated", [True, False])
def test_layer_against_64_bits(T, M, types, dt, gated):
    for n, (rows, cols, hidden, experts, top_k) in enumerate(LAYERS):
        args = layer_of(T, n, types[dt], rows, cols, hidden, experts, gated, pad=n % 3)
        res = wide(T, rows, cols, n % 4, real(T, args[4], types[dt])) if n % 2 else None
        print("layer", dt, gated, rows, cols, hidden, experts, top_k, flush=True)
        how = dict(score="sigmoid" if n % 2 else "softmax", renorm=n % 3 != 0, scale=2.5 if n % 5 == 0 else 1.0)
        if n % 2:
            how["bias"] = 0.05 * T.randn(experts, device=DEV, generator=args[4])
        check_layer(T, M, dt, args, top_k, how, ACTS[n % 5], gated, None, res)


@pytest.mark.parametrize("rows", [1, 2, 4, 5, 33, 100])
def test_layer_masks(T, M, rows):
    """Padding rows that hold NaN, experts that are out, rows that find no expert, rows that the router voids, groups."""
    experts, top_k = 24, 6
    args = layer_of(T, rows, T.bfloat16, rows, 96, 40, experts)
    x, g = args[0], args[4]
    res = real(T, g, T.bfloat16)(rows, 96)
    mask = T.rand(rows, device=DEV, generator=g) < 0.6
    x[~mask] = math.nan
    bias = 0.05 * T.randn(experts, device=DEV, generator=g)
    groups = dict(groups=8, top_groups=3, group_top=2)
    for how in (dict(score="sigmoid", bias=bias, **groups), dict(score="softmax"), dict(score="softmax", bias=bias)):
        r = check_layer(T, M, "bf16", args, top_k, how, "silu", True, mask, res)
        assert T.equal(r.y[~mask], res[~mask]) and bool((r.routing.ids[~mask] == -1).all())
        assert bool((r.routing.weights[~mask] == 0).all())
    r = check_layer(T, M, "bf16", args, top_k, dict(score="softmax"), "silu", True, mask, None)
    assert bool((r.y[~mask] == 0).all())
    # all experts but two are out: four slots find none
    out = T.full((experts,), -math.inf, device=DEV)
    out[3], out[17] = 0.0, 0.0
    r = check_layer(T, M, "bf16", args, top_k, dict(score="sigmoid", bias=out), "silu", True, mask, res)
    assert bool((r.routing.ids[mask][:, 2:] == -1).all()) and bool((r.routing.ids[mask][:, :2] >= 0).all())
    # a NaN that is not masked voids its row alone
    x[~mask] = 1.0
    clean = M.layer(*args[:4], top_k, residual=res).y
    x[rows - 1, 5] = math.nan
    r = check_layer(T, M, "bf16", args, top_k, dict(), "silu", True, None, res)
    assert bool(r.y[rows - 1].isnan().all()) and T.equal(r.y[:rows - 1], clean[:rows - 1])


@pytest.mark.parametrize("rows", [3, 16, 17, 40])
@pytest.mark.parametrize("experts,groups,top_groups", [(256, 8, 4), (512, 16, 3), (1024, 1, 1), (1024, 64, 40)])
def test_layer_of_many_experts(T, M, rows, experts, groups, top_groups):
    args = layer_of(T, rows, T.float16, rows, 32, 8, experts)
    for how in (dict(score="sigmoid", bias=0.05 * T.randn(experts, device=DEV, generator=args[4]), group_top=2),
                dict(score="softmax", renorm=False)):
        check_layer(T, M, "f16", args, 8, dict(how, groups=groups, top_groups=top_groups), "silu", True, None, args[0])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [65, 193, 512])
def test_layer_of_crowded_experts(T, M, types, rows, dt):
    """A bias sends every token to one expert and most to another, so that experts have many runs of tokens, others none; with
    padding in between; the counts in the caller's array or in none."""
    args = layer_of(T, rows, types[dt], rows, 72, 40, 12)
    g = args[4]
    mask = T.rand(rows, device=DEV, generator=g) < 0.9
    args[0][~mask] = math.nan
    bias = T.zeros(12, device=DEV)
    bias[7], bias[2], bias[:2] = 9.0, 0.6, -math.inf
    how = dict(score="sigmoid", bias=bias)
    r = check_layer(T, M, dt, args, 3, how, "silu", True, mask, None)
    assert int(r.routing.load[7]) == int(mask.sum()) and int(r.routing.load[:2].sum()) == 0
    y = T.empty_like(r.y)
    M.layer(*args[:4], 3, mask=mask, out=M.Layer(y, r.routing._replace(load=None)), **how)
    assert T.equal(y, r.y)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_layer_rows_of_any_length(T, M, types, dt):
    """Weights whose rows end anywhere in 16 and in 256 bytes, and are shorter than that, the last in memory at its end."""
    for rows, n in ((3, 1), (3, 3), (3, 7), (20, 4), (20, 8), (5, 9), (40, 33), (3, 63), (20, 64), (40, 65), (3, 127), (5, 129), (20, 200), (40, 257)):
        for cols, hidden in ((n, 24), (24, n)):
            check_layer(T, M, dt, layer_of(T, n, types[dt], rows, cols, hidden, 6), 2, {}, "silu", True, None, None)
            check_layer(T, M, dt, layer_of(T, n, types[dt], rows, cols, hidden, 6, False), 2, {}, "relu", False, None, None)


def test_layer_reads_no_expert_that_is_not_chosen(T, M):
    for rows in (1, 3, 40):
        args = layer_of(T, 5, T.float16, rows, 64, 48, 16)
        ids = M.layer(*args[:4], 2).routing.ids
        for e in range(16):
            if not bool((ids == e).any()):
                args[2][e], args[3][e] = math.nan, math.nan
        check_layer(T, M, "f16", args, 2, {}, "gelu", True, None, None)


def test_layer_in_place_and_again(T, M):
    """The residual may be the output; rows behind a strided output's stay; the same call gives the same bits."""
    for rows in (0, 1, 4, 30):
        args = layer_of(T, 9, T.bfloat16, rows, 64, 48, 16)
        x, _, _, _, g = args
        res = real(T, g, T.bfloat16)(rows, 64)
        a = M.layer(*args[:4], 3, residual=res)
        b = M.layer(*args[:4], 3, residual=res)
        assert T.equal(a.y, b.y) and all(T.equal(p, q) for p, q in zip(a.routing, b.routing))
        base = T.full((rows + 2, 80), 7.0, device=DEV, dtype=T.bfloat16)
        base[1:rows + 1, 3:67] = res
        view = base[1:rows + 1, 3:67]
        c = M.layer(*args[:4], 3, residual=view, out=M.Layer(view, a.routing._replace(load=None)))
        assert c.y is view and T.equal(view, a.y)
        view.fill_(7.0)
        assert bool((base == 7.0).all())
        if not rows:
            assert not int(a.routing.load.sum())


# ---------------------------------------------------------------------------
# orthogonal updates
# ---------------------------------------------------------------------------


def orth64(T, u, steps, abc, eps=1e-7):
    x = u.double()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        p = x @ x.mT
        x = abc[0] * x + (abc[1] * p + abc[2] * (p @ p)) @ x
    return x.mT if tall else x


ABC = (3.4445, -4.7750, 2.0315)
MATRICES = [(1, 1), (1, 7), (8, 8), (33, 31), (64, 64), (65, 200), (200, 65), (130, 257), (256, 1000), (300, 300), (520, 264), (3, 8192), (64, 5000),
            (7000, 40), (50, 8193)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_orthogonalize_pairs_of_rows(T, M, types, dt):
    """Rows in pairs far apart that share two columns, and nothing else: every sum has at most two terms, so that the only
    errors are those of numbers of 22 bits (2^-22 relative) and what is left out of a product (2^-22), and zeros stay
    zeros.  Of the largest magnitude in its pair an element of P = X X^T is off by at most 2 (2 2^-22 + 2^-22) and its own
    rounding, 7 2^-22; of b P + c P^2 by |b| 8 + |c| (4 * 8), of X' by a 2 + 2 (73 + |b| 2 + |c| 4): under 260 2^-22."""
    for rows, cols in MATRICES:
        if rows < 2 or cols < 2:
            continue
        g = gen(T, rows)
        u = T.zeros(rows, cols, device=DEV)
        m = min(rows, cols) // 2
        at = T.randperm(cols, generator=g, device=DEV)
        for i, j in ((T.arange(m, device=DEV), rows - 1 - T.arange(m, device=DEV)),):
            for r in (i, j):
                for c in (at[:m], at[m:2 * m]):
                    u[r, c] = 0.2 + T.rand(m, generator=g, device=DEV)
        u = u.to(types[dt])
        y = M.orthogonalize(u, steps=1).double()
        want = orth64(T, u, 1, ABC)
        assert T.equal(y == 0, want == 0), (rows, cols)
        top = u.double().abs().max() / u.double().norm()
        worst = float((y - want).abs().max() / top)
        tol = 260 * 2.0 ** -22 + U[dt] * float(want.abs().max() / top)
        print(dt, rows, cols, worst, tol, flush=True)
        assert worst <= tol


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_orthogonalize_against_64_bits(T, M, types, dt):
    """The norm of the error after a step: of P at most (3 2^-22 + SUM(n)) |X|^2, twice that for P^2 at |P| <= 1.5, which the
    coefficients weigh: e = (3.5 + 2 * 4.8 + 4 * 2.1) 1.5 (3 2^-22 + SUM(n)) of the norm.  A later step multiplies what is
    there by at most its largest slope over singular values up to 1.21, 4.3."""
    for n, (rows, cols) in enumerate(MATRICES):
        g = gen(T, n)
        u = real(T, g, types[dt], 0.03)(2, rows, cols)
        u[1] *= 1e-3 if dt != "f16" else 0.5
        for steps in (0, 1, 2):
            y, want = M.orthogonalize(u, steps=steps).double(), orth64(T, u, steps, ABC)
            e = 32 * (3 * 2.0 ** -22 + SUM(max(rows, cols)))
            tol = (2.0 ** -22 + sum(e * 4.3 ** k for k in range(steps)) + U[dt]) * 1.5
            err = (y - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
            print(dt, rows, cols, steps, err.tolist(), tol, flush=True)
            assert bool((err <= tol).all())


@pytest.mark.parametrize("shape", [(70, 4481), (300, 8003), (8003, 300), (9, 200, 2000), (1024, 2600), (50, 8193)])
def test_orthogonalize_steps_without_the_update(T, M, types, shape):
    """Wide updates, of which several steps are taken at a time, with singular values over three orders.  Of P, a + B, (a + B) P,
    (a + B) P (a + B) and Q up to nine are rounded for three steps, each by at most 2^-23 of its norm; an error of P comes
    into a + B at most |b| + 2 |c| = 8.8 times, and what a + B are off by meets the other two factors, 3.5^2 at most:
    9 * 8.8 * 12 * 2^-23 = 1.2e-4 a group of steps, of which there are up to three."""
    *count, rows, cols = shape
    g = gen(T, rows)
    u = T.randn(*count, rows, cols, device=DEV, generator=g)
    u = (u * T.logspace(0, -3, rows, device=DEV)[:, None] if rows <= cols else u * T.logspace(0, -3, cols, device=DEV))
    for dt, steps in (("f32", 2), ("bf16", 3), ("f16", 4), ("f32", 5), ("f16", 5), ("f32", 6)):
        v = u.to(types[dt])
        y = M.orthogonalize(v, steps=steps).double()
        want = orth64(T, v, steps, ABC)
        err = float(((y - want).flatten(-2).norm(dim=-1) / want.flatten(-2).norm(dim=-1)).max())
        print(shape, dt, steps, err, flush=True)
        assert err <= U[dt] + 3 * 1.2e-4
        assert T.equal(y, M.orthogonalize(v, steps=steps).double())


def test_orthogonalize_moves_singular_values_to_one(T, M):
    """Five steps take singular values from 0.01 of the norm on to 0.65 .. 1.25 (the polynomial's own range, 0.68 .. 1.13
    there, and the errors above)."""
    for rows, cols in ((64, 64), (200, 77), (96, 700)):
        g = gen(T, rows)
        m = min(rows, cols)
        q = T.linalg.qr(T.randn(rows, m, device=DEV, dtype=T.float64, generator=g))[0]
        r = T.linalg.qr(T.randn(cols, m, device=DEV, dtype=T.float64, generator=g))[0]
        s = T.logspace(-1.6, 0, m, device=DEV, dtype=T.float64)
        s = s / s.norm()
        keep = s > 0.01
        u = ((q * s) @ r.T * 5.0).float()
        y = M.orthogonalize(u).double()
        got = (q.T @ y @ r).diagonal()
        assert bool((got[keep] > 0.65).all()) and bool((got < 1.25).all())
        want = orth64(T, u, 5, ABC)
        assert float((y - want).norm() / want.norm()) < 1e-3


def test_orthogonalize_edges(T, M):
    for dt in (T.float32, T.bfloat16):
        z = T.zeros(3, 20, 30, device=DEV, dtype=dt)
        assert bool((M.orthogonalize(z) == 0).all())
        z[1, 4, 5] = math.inf
        z[2, 0, 0] = math.nan
        y = M.orthogonalize(z)
        assert bool((y[0] == 0).all()) and bool(y[1].isnan().all()) and bool(y[2].isnan().all())
    big = T.full((8, 8), 1e38, device=DEV)
    big += T.eye(8, device=DEV) * 1e38                       # squares past 32 bits
    a, b = M.orthogonalize(big, steps=3), M.orthogonalize(big / 1e38 * 1e-30, steps=3, eps=0.0)
    assert bool(a.isfinite().all()) and T.allclose(a, b, rtol=1e-4, atol=1e-4)
    u = T.randn(5, 40, 24, device=DEV)
    y = M.orthogonalize(u)
    for k in range(5):                                       # each by itself
        assert T.allclose(y[k], M.orthogonalize(u[k].contiguous()), atol=1e-4)
    assert T.equal(y, M.orthogonalize(u))
    v = u.clone()
    assert M.orthogonalize(v, out=v) is v and T.equal(v, y)  # in place
    assert M.orthogonalize(u[:0]).shape == (0, 40, 24)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------


def test_a_gates_training_step(T, M):
    """Logits, routing, the router's gradient, that of the gate's weights and tokens, and the update: against the same in 64
    bits, differentiated by autograd."""
    g = gen(T, 11)
    rows, cols, experts, k = 700, 264, 40, 4
    x, w = real(T, g, T.bfloat16)(rows, cols), real(T, g, T.bfloat16, 1.5 / math.sqrt(cols))(experts, cols)
    gw = real(T, g, T.float32)(rows, k)
    logits = M.linear(x, w, out_dtype=T.float32)
    r = M.route(logits, k, score="sigmoid")
    dl = M.route_backward(logits, r.ids, gw, score="sigmoid")
    grads = M.linear_backward(x, w, dl)
    update = M.orthogonalize(grads.weight)
    x6, w6 = x.double().requires_grad_(True), w.double().requires_grad_(True)
    s = T.sigmoid(x6 @ w6.T).gather(1, r.ids.long())
    ((s / s.sum(1, keepdim=True)) * gw.double()).sum().backward()
    # a gradient is a sum of terms off by 2^-8 (rounded to bf16 for the product) and 2^-16 (the router's); then rounded
    d = dl.double().abs()
    for got, want, S in ((grads.x, x6.grad, d @ w.double().abs()), (grads.weight, w6.grad, d.T @ x.double().abs())):
        assert bool(((got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -14) * S + 2.0 ** -8 * want.abs()).all())
    want = orth64(T, grads.weight, 5, ABC)
    assert float((update.double() - want).norm() / want.norm()) < 2.0 ** -8 + 1e-3


def test_graph_of_many_runs_and_wide_updates(T, M):
    """A captured layer of experts with several runs of tokens, a gradient with a bias's and an update of several steps a pass:
    as the eager results at every replay, with new inputs and eager work between."""
    def inputs(seed):
        a = layer_of(T, seed, T.float16, 300, 72, 40, 5)
        w = real(T, a[4], T.float16)
        return [a[0], a[1], a[2], a[3], w(300, 5), w(70, 4490)]

    def run(x, gate, w_in, w_out, grad, wide):
        y, r = M.layer(x, gate, w_in, w_out, 2, residual=x)
        d = M.linear_backward(x, gate, grad, need_x=False)
        return [y, r.ids, r.weights, r.load, d.weight, d.bias, M.orthogonalize(wide)]

    args = inputs(0)
    run(*args)
    T.cuda.synchronize()
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        out = run(*args)
    for k in range(4):
        fresh = inputs(1 + k)
        for a, b in zip(args, fresh):
            a.copy_(b)
        want = run(*fresh)
        if k % 2:
            T.cuda.synchronize()
        g.replay()
        again = run(*fresh)
        T.cuda.synchronize()
        assert all(T.equal(a, b) for a, b in zip(out, want)) and all(T.equal(a, b) for a, b in zip(again, want))


def test_graphs_streams_and_workspaces(T, M):
    """Two graphs of all the operators, replayed in turn on new inputs with eager work and synchronisations between, and
    the same on a stream that is given: as the eager results, every time."""
    cols, experts = 264, 24

    def inputs(seed):
        a = layer_of(T, seed, T.bfloat16, 40, cols, 72, experts)
        big = real(T, a[4], T.bfloat16)(300, cols)
        return [a[0], a[1], a[2], a[3], big, real(T, a[4], T.bfloat16)(300, experts)]

    def run(x, gate, w_in, w_out, big, grad, stream=None):
        y, r = M.layer(x, gate, w_in, w_out, 3, residual=x, stream=stream)
        one = M.layer(x[:1], gate, w_in, w_out, 3, stream=stream)
        z = M.linear(big, gate, act="gelu", out_dtype=T.float32, stream=stream)
        few = M.linear(x, gate, stream=stream)
        d = M.linear_backward(big, gate, grad, stream=stream)
        return [y, r.ids, r.weights, r.load, one.y, z, few, d.x, d.weight, d.bias, M.orthogonalize(d.weight, stream=stream)]

    graphs = []
    run(*inputs(0))
    T.cuda.synchronize()
    for n in range(2):
        args = inputs(n)
        g = T.cuda.CUDAGraph()
        with T.cuda.graph(g):
            out = run(*args)
        graphs.append((g, args, out))
    for k in range(4):
        for n, (g, args, out) in enumerate(graphs):
            fresh = inputs(10 + 2 * k + n)
            for a, b in zip(args, fresh):
                a.copy_(b)
            want = run(*fresh)
            if k % 2:
                T.cuda.synchronize()
            g.replay()
            want2 = run(*fresh)
            T.cuda.synchronize()
            assert all(T.equal(a, b) for a, b in zip(out, want)) and all(T.equal(a, b) for a, b in zip(want, want2))
    s = [T.cuda.Stream() for _ in range(2)]
    a = [inputs(50), inputs(51)]
    want = [run(*v) for v in a]
    T.cuda.synchronize()
    for _ in range(3):
        got = [run(*v, stream=q) for v, q in zip(a, s)]
        T.cuda.synchronize()
        assert all(T.equal(p, q) for v, w in zip(got, want) for p, q in zip(v, w))


def test_weights_past_32_bits_of_bytes(T, M):
    """The last experts of a layer lie past 4 GiB."""
    experts, cols, hidden = 280, 2048, 4096
    w_in = T.zeros(experts, hidden, cols, device=DEV, dtype=T.float16)
    w_out = T.zeros(experts, cols, hidden, device=DEV, dtype=T.float16)
    g = gen(T, 3)
    gate = real(T, g, T.float16, 0.03)(experts, cols)
    for e in (277, 279):
        w_in[e], w_out[e] = real(T, g, T.float16, 0.02)(hidden, cols), real(T, g, T.float16, 0.02)(cols, hidden)
    bias = T.full((experts,), -math.inf, device=DEV)
    bias[277], bias[279] = 0.0, 0.0
    for rows in (1, 20):
        x = real(T, g, T.float16)(rows, cols)
        check_layer(T, M, "f16", (x, gate, w_in, w_out, g), 2, dict(score="sigmoid", bias=bias), "silu", False, None, None)


def test_a_product_past_32_bits_of_bytes(T, M):
    """Rows past 4 GiB of x, of the result and of the gradient: the last rows are those of a call of their own."""
    rows, cols, outs = 300_000, 8192, 8
    x = T.zeros(rows, cols, device=DEV, dtype=T.bfloat16)
    g = gen(T, 4)
    w = real(T, g, T.bfloat16)(outs, cols)
    x[-300:] = real(T, g, T.bfloat16)(300, cols)
    y = M.linear(x, w, out_dtype=T.float32)
    tail = x[-300:].double() @ w.double().T
    S = x[-300:].double().abs() @ w.double().abs().T
    assert bool(((y[-300:].double() - tail).abs() <= SUM(cols) * S).all()) and not bool(y[:-300].any())
    gr = T.zeros(rows, outs, device=DEV, dtype=T.bfloat16)
    gr[-300:] = whole(T, g, T.bfloat16)(300, outs)
    x[-300:] = whole(T, g, T.bfloat16)(300, cols)
    w = whole(T, g, T.bfloat16)(outs, cols)
    d = M.linear_backward(x, w, gr)
    assert T.equal(d.x[-300:], (gr[-300:].double() @ w.double()).bfloat16()) and not bool(d.x[:-300].any())
    assert T.equal(d.weight, (gr[-300:].double().T @ x[-300:].double()).bfloat16())
    assert T.equal(d.bias, gr[-300:].double().sum(0).float())
