"""The products at the ends of their ranges, on the GPU: what is far from 0, limits of
sizes, small differences of precision.  Bounds are derived beside each test; a
rounding to type t is off by at most U[t] relative.
"""

import math

import pytest

from test_gpu_products import ACTS, ABC, DEV, M, SUM, T, U, act64, gen, orth64, real, slope64, types, whole, wide  # noqa: F401

pytestmark = pytest.mark.gpu

FAR = [8.0, 11.9, 12.1, 19.9, 20.1, 40.0, 89.0, 104.0, 199.0, 201.0, 1e3, 6e4, 1e6, 1e10, 1.2e13, 3e13, 1e16, 1.8e19, 3e19, 1e25, 1e30, 3e38, math.inf]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("copies", [1, 40])
def test_slopes_far_from_zero(T, M, types, dt, act, copies):  # noqa: F811
    """A product with the identity shows the slopes.  From 104 on they are 0 and 1 (a sigmoid is below 2^-149 there, the others
    from 20 on), infinities included; before that a slope is off by 2^-20 (2 + |z|) as near 0.  A NaN stays one, and no other
    row or sum has it."""
    t = types[dt]
    z = T.tensor([s * v for v in FAR for s in (1, -1)] * copies, device=DEV).to(t)
    rows, n = z.numel(), 16
    pre, w = z[:, None].expand(rows, n).contiguous(), T.eye(n, device=DEV).to(t)
    x = T.ones(rows, 8, device=DEV).to(t)
    for grad_type in {t, T.float32}:
        one = T.ones(rows, n, device=DEV, dtype=grad_type)
        dx, _, db = M.linear_backward(w[:1].expand(rows, n).contiguous(), w, one, act=act, pre=pre, need_weight=False)
        finite = z.double().clamp(-1e30, 1e30)
        want = slope64(T, finite, act)
        far = z.abs() >= 104
        want = T.where(far, (z > 0).double(), want)
        tol = T.where(far, 0.0, 2.0 ** -20 * (2 + finite.abs()) + U[dt] * want.abs() + (2.0 ** -24 if dt == "f16" else 0))
        assert bool(((dx.double() - want[:, None]).abs() <= tol[:, None]).all()), (dt, act, (dx[:, 0].double() - want).tolist())
        assert bool(((db.double() - want.sum()).abs() <= 2.0 ** -20 * (2 + finite.abs()[~far]).sum() + rows * 2.0 ** -24 * want.abs().sum()).all())
        dw = M.linear_backward(x, w[:, :8].contiguous(), one, act=act, pre=pre, need_x=False).weight
        assert bool(dw.isfinite().all())
        torn = pre.clone()
        torn[5, 3] = math.nan
        got = M.linear_backward(x, w[:, :8].contiguous(), one, act=act, pre=torn)
        assert bool(got.x[5].isnan().all()) and bool(got.weight[3].isnan().all()) and bool(got.bias[3].isnan())
        got.x[5], got.weight[3], got.bias[3] = 0, 0, 0
        assert all(bool(v.isfinite().all()) for v in got)


def test_linear_of_two_launches(T, M):  # noqa: F811
    """2^30 rows: the products are 2^32 work-items and more, in several launches.  Rows at both ends and around the places where the
    launches part are those of a call of their own, all others are zeros."""
    rows, n = (1 << 30) + 70, 8
    g = gen(T, 12)
    x, w = T.zeros(rows, n, device=DEV, dtype=T.float16), whole(T, g, T.float16)(n, n)
    some = T.cat([T.arange(k, k + 300, device=DEV) for k in (0, rows // 4, (1 << 29) - 600, (1 << 30) - 600, rows - 300)])
    x[some] = whole(T, g, T.float16)(some.numel(), n)
    want = x[some].double() @ w.double().T
    y = M.linear(x, w)
    assert T.equal(y[some], want.to(T.float16))
    assert int(y.count_nonzero()) == int(want.count_nonzero())
    y.zero_()
    y[some] = whole(T, g, T.float16)(some.numel(), n)
    dx, dw, db = M.linear_backward(x, w, y)
    want = y[some].double() @ w.double()
    assert T.equal(dx[some], want.to(T.float16)) and int(dx.count_nonzero()) == int(want.count_nonzero())
    assert T.equal(dw, (y[some].double().T @ x[some].double()).to(T.float16)) and T.equal(db, y[some].double().sum(0).float())


@pytest.mark.parametrize("rows,cols", [(8, 8), (1, 16384)])
def test_orthogonalize_as_many_as_there_may_be(T, M, rows, cols):  # noqa: F811
    """65,536 updates, of which few are not zero: each by itself, the last ones too."""
    g = gen(T, rows)
    u = T.zeros(65536, rows, cols, device=DEV, dtype=T.bfloat16)
    at = T.tensor([0, 1, 32767, 32768, 65000, 65535], device=DEV)
    u[at] = real(T, g, T.bfloat16)(6, rows, cols)
    y = M.orthogonalize(u, steps=1)
    for k in at.tolist():
        assert T.equal(y[k], M.orthogonalize(u[k].contiguous(), steps=1)) if cols > 8192 else \
            T.allclose(y[k].float(), M.orthogonalize(u[k].contiguous(), steps=1).float(), atol=2.0 ** -7)
    y[at] = 0
    assert not bool(y.any())


def grid(T):  # noqa: F811
    """-13 .. 13 in steps of 2^-13, and small numbers of both signs"""
    z = T.arange(-13 * 8192, 13 * 8192 + 1, device=DEV, dtype=T.float64) / 8192
    small = T.logspace(-30, -4, 500, device=DEV, dtype=T.float64)
    return T.cat([z, small, -small])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("long", [True, False])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_activations_on_a_grid(T, M, types, dt, long, act):  # noqa: F811
    """A product of one column with 1 shows the activation, relative to its value, however small that is.  Of 32-bit results
    an exponential is off by 2^-23 and its argument's roundings, a sum, a quotient and a product by 2^-24 each: 2^-24 (8 + 5 |u|)
    where e^-u is taken; erfc by at most 16 units of 2^-23, its argument by 1.5 2^-24, which counts 2 x^2 = z^2 times.  16-bit
    results are off by 2^-17 before they are rounded.  What is multiplied by z is 0 below 2^-126."""
    t = types[dt]
    z = grid(T).to(t)
    to = T.float32 if long else t
    want = 0.5 * z.double() * T.special.erfc(-z.double() / math.sqrt(2)) if act == "gelu" else \
        z.double() * T.sigmoid(z.double()) if act == "silu" else \
        z.double() * T.sigmoid(math.sqrt(8 / math.pi) * (z.double() + 0.044715 * z.double() ** 3))
    u = z.double().abs() if act == "silu" else math.sqrt(8 / math.pi) * (z.double().abs() + 0.044715 * z.double().abs() ** 3)
    near = 2.0 ** -24 * (34 + 4 * z.double() ** 2) if act == "gelu" else 2.0 ** -24 * (8 + 5 * u)
    tol = want.abs() * (near if to == T.float32 else 2.0 ** -17 + U[dt]) + (2.0 ** -25 if to == T.float16 else 2.0 ** -126 * (1 + z.double().abs()))
    w = T.ones(1, 1, device=DEV, dtype=t)
    for x in (z[:, None].contiguous(), z[-1050:-1000, None].contiguous(), z[::5000][:16, None].contiguous()):
        y = M.linear(x, w, act=act, out_dtype=to)[:, 0].double()
        k = (z[None, :] == x[:50]).double().argmax(1) if x.shape[0] <= 64 else T.arange(z.numel(), device=DEV)
        worst = float(((y - want[k]).abs() / tol[k]).nan_to_num(math.inf).max())
        print(dt, long, act, x.shape[0], worst, flush=True)
        assert worst <= 1


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
def test_linear_has_no_other_result(T, M, types, dt, act):  # noqa: F811
    """Real values in every size of tile, each within its bound, which no NaN is."""
    for n, (rows, cols, outs, pad) in enumerate([(5, 300, 40, 0), (40, 333, 65, 3), (60, 96, 500, 0), (300, 520, 200, 0), (130, 777, 131, 5),
                                                 (2100, 256, 1024, 0), (100, 8192, 40, 0)]):
        g, t = gen(T, 300 + n), types[dt]
        x, w = wide(T, rows, cols, pad, real(T, g, t)), wide(T, outs, cols, pad, real(T, g, t, 2 / math.sqrt(cols)))
        b, r = real(T, g, T.float32, 0.5)(outs), wide(T, rows, outs, pad, real(T, g, t))
        y = M.linear(x, w, b, act=act, residual=r)
        z, S = x.double() @ w.double().T + b.double(), x.double().abs() @ w.double().abs().T + b.double().abs()
        a = act64(T, z, act)
        want = a + r.double()
        tol = 1.13 * SUM(cols) * S + (2 ** -20) * (z.abs() + a.abs()) + 2 ** -23 * (a.abs() + r.double().abs()) + U[dt] * want.abs() \
            + (2.0 ** -25 if dt == "f16" else 0)
        assert bool(((y.double() - want).abs() <= tol).all()), (rows, cols, outs)


def plain_steps(T, u, steps, dt):  # noqa: F811
    """The definition in products of type dt."""
    x = u.to(dt) if u.shape[-2] <= u.shape[-1] else u.to(dt).mT.contiguous()
    x = (x / (x.double().square().sum((-1, -2), keepdim=True).sqrt() + 1e-7)).to(dt)
    for _ in range(steps):
        p = x @ x.mT.contiguous()
        x = ABC[0] * x + (ABC[1] * p + ABC[2] * (p @ p)) @ x
    return (x if u.shape[-2] <= u.shape[-1] else x.mT).double()


@pytest.mark.parametrize("rows,cols", [(1024, 4096), (512, 2048), (256, 7168), (8003, 300), (70, 4481), (777, 3001), (1024, 2600), (64, 5000)])
def test_updates_of_32_bits_are_as_near_as_products_of_32_bits(T, M, rows, cols):  # noqa: F811
    """Numbers of 22 bits are rounded by 2^-23 where those of 32 bits are by 2^-24, at the same places of a step, and sums are of
    32 bits in both: twice the error of plain products at most, by the norm, against 64 bits."""
    g = gen(T, rows)
    m = min(rows, cols)
    rank = max(1, m // 8)
    noise = T.randn(rows, cols, device=DEV, generator=g)
    fall = noise * (T.logspace(0, -3, rows, device=DEV)[:, None] if rows <= cols else T.logspace(0, -3, cols, device=DEV))
    strong = T.randn(rows, rank, device=DEV, generator=g) * T.logspace(0, -1, rank, device=DEV)
    momentum = strong @ T.randn(rank, cols, device=DEV, generator=g) / math.sqrt(rank) + 0.3 * noise
    for name, u in (("noise", noise), ("three orders", fall), ("momentum", momentum)):
        for steps in (2, 3, 5):
            want = orth64(T, u, steps, ABC)
            plain, own = (float((y - want).norm() / want.norm()) for y in (plain_steps(T, u, steps, T.float32), M.orthogonalize(u, steps=steps).double()))
            print(rows, cols, name, steps, plain, own, flush=True)
            assert own <= 2 * plain + 2.0 ** -24, (name, steps, own, plain)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1024, 4096), (256, 7168), (8003, 300), (70, 4481), (300, 301), (40, 900), (64, 5000), (3, 8192)])
def test_updates_of_16_bits_are_off_by_their_rounding(T, M, types, dt, rows, cols):  # noqa: F811
    """Five steps end within 1e-5 of the norm before the result is rounded, which is at most U[dt] of each element and half the
    smallest f16 (2^-25) where that is more.  An element is then its exact value's rounding, but where that lies nearer to a
    border than the error: of borders every s = 2 U[dt] 2^floor(log2 |x|), for at most 2 e / s of those elements, e = 1e-5
    of the mean magnitude (a product of single f16, off by 1e-3, would miss most)."""
    g = gen(T, cols)
    u = (T.randn(rows, cols, device=DEV, generator=g) * T.logspace(0, -2, cols, device=DEV)).to(types[dt])
    for steps in (1, 2, 5):
        want = orth64(T, u, steps, ABC)
        y = M.orthogonalize(u, steps=steps).double()
        err = float((y - want).norm() / want.norm())
        print(dt, rows, cols, steps, err, flush=True)
        assert err <= 1e-5 + U[dt] + (2.0 ** -25 * math.sqrt(rows * cols) / float(want.norm()) if dt == "f16" else 0)
        e = 1e-5 * float(want.square().mean().sqrt())
        space = 2 * U[dt] * 2.0 ** want.abs().clamp_min(2.0 ** (-14 if dt == "f16" else -126)).log2().floor()
        other, most = int((y != want.to(types[dt]).double()).sum()), float((2 * e / space).clamp_max(1).sum())
        print(other, most, rows * cols, flush=True)
        assert other <= most + 3 * math.sqrt(most) + 1 and most < 0.5 * rows * cols       # and that says something


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("low,high,size", [(-9, -9, 1000.0), (6, 6, 1e-4), (-8, 1, 300.0), (-30, -29, 60000.0), (0, 0, 1.0)])
def test_f16_takes_gradients_in_the_range_of_32_bits(T, M, act, low, high, size):  # noqa: F811
    """Rows of a 32-bit grad of 10^low .. 10^high, far outside f16.  Its parts hold 2^-18 of an element, and the product of two
    low parts, 2^-18 of a term, is left out; three products a term make sums of three times as many."""
    for n, (rows, cols, outs, pad) in enumerate([(5, 300, 40, 0), (260, 333, 65, 3), (1300, 104, 200, 0), (2050, 256, 264, 0), (70, 31, 1, 1)]):
        g = gen(T, 400 + n)
        x, w = wide(T, rows, cols, pad, real(T, g, T.float16, size)), wide(T, outs, cols, pad, real(T, g, T.float16, size))
        x, w = x.clamp(-60000, 60000), w.clamp(-60000, 60000)
        scale = 10.0 ** (low + (high - low) * T.rand(rows, 1, device=DEV, generator=g))
        gr = wide(T, rows, outs, pad, lambda *s: scale * T.randn(*s, device=DEV, generator=g))
        pre = None if act == "none" else wide(T, rows, outs, pad, real(T, g, T.float16, 2.0))
        dx, dw, db = M.linear_backward(x, w, gr, act=act, pre=pre)
        one_x = M.linear_backward(x, w, gr, act=act, pre=pre, need_weight=False, need_bias=False).x
        one_w = M.linear_backward(x, w, gr, act=act, pre=pre, need_x=False, need_bias=False).weight
        slope = T.ones_like(gr, dtype=T.float64) if pre is None else slope64(T, pre.double(), act)
        d = gr.double() * slope
        ed = gr.double().abs() * 2 ** -20 * (2 + (pre.double().abs() if pre is not None else 0)) + d.abs() * 2.0 ** -17
        for what, both, alone, want, tol in (
                ("x", dx, one_x, d @ w.double(), ed @ w.double().abs() + SUM(3 * outs + 96) * (d.abs() @ w.double().abs())),
                ("weight", dw, one_w, d.T @ x.double(), ed.T @ x.double().abs() + SUM(3 * rows + 96) * (d.abs().T @ x.double().abs())),
                ("bias", db, db, d.sum(0), ed.sum(0) + rows * 2 ** -24 * d.abs().sum(0))):
            tol = tol + (U["f16"] * want.abs() + 2.0 ** -25 if what != "bias" else 2.0 ** -24 * want.abs())
            fits = (want.abs() + tol < 65504) | (what == "bias")         # an f16 result; 65,520 and more is an infinity
            over = (want.abs() - tol >= 65520) & ~fits
            assert float(fits.double().mean()) > 0.9
            for got in (both, alone):
                off = float(((got.double() - want).abs() / tol).nan_to_num(math.inf)[fits].max())
                assert T.equal(got[over], (want.sign() * math.inf)[over].half())
                print(act, low, rows, cols, outs, what, off, float(want.abs().max()), flush=True)
                assert off <= 1


@pytest.mark.parametrize("rows,cols,outs", [(9, 40, 24), (300, 136, 150)])
def test_f16_gradients_carry_what_is_not_finite(T, M, rows, cols, outs):  # noqa: F811
    """From a grad of 32 bits: an infinity or NaN reaches its row of dx, its row (of grad) or column (of x) of the weight's and its
    element of the bias's gradient, and nothing else; the largest numbers are no infinity before they are in f16."""
    g = gen(T, rows)
    x, w, gr = real(T, g, T.float16)(rows, cols), real(T, g, T.float16)(outs, cols), real(T, g, T.float32)(rows, outs)
    clean = M.linear_backward(x, w, gr)
    for bad in (math.inf, -math.inf, math.nan):
        x2, gr2 = x.clone(), gr.clone()
        gr2[3, 2], gr2[4, 7], x2[5, 1] = bad, math.nan, bad
        dx, dw, db = M.linear_backward(x2, w, gr2)
        hit = T.zeros(rows, cols, dtype=T.bool, device=DEV)
        hit[3], hit[4] = True, True
        assert T.equal(dx[~hit], clean.x[~hit]) and not bool(dx[hit].isfinite().any())
        hit = T.zeros(outs, cols, dtype=T.bool, device=DEV)
        hit[2], hit[7], hit[:, 1] = True, True, True
        assert T.equal(dw[~hit], clean.weight[~hit]) and not bool(dw[hit].isfinite().any())
        hit = T.zeros(outs, dtype=T.bool, device=DEV)
        hit[2], hit[7] = True, True
        assert T.equal(db[~hit], clean.bias[~hit]) and not bool(db[hit].isfinite().any())
    big, one = T.zeros(rows, outs, device=DEV), T.ones(outs, cols, device=DEV, dtype=T.float16)
    big[0, 0], big[1, 1] = T.finfo(T.float32).max, -T.finfo(T.float32).max
    dx = M.linear_backward(x, one, big, need_weight=False, need_bias=False).x
    assert bool((dx[0] == math.inf).all()) and bool((dx[1] == -math.inf).all()) and not bool(dx[2:].any())
    dx = M.linear_backward(x, one * 2.0 ** -24, big * 2.0 ** -100, need_weight=False, need_bias=False).x
    assert bool((dx[0] == 16.0).all()) and bool((dx[1] == -16.0).all())


def test_graph_of_f16_gradients(T, M):  # noqa: F811
    """Captured from grads of 32 bits, with and without an activation, replayed on new inputs with eager work between."""
    def inputs(seed):
        g = gen(T, seed)
        h, s = real(T, g, T.float16), real(T, g, T.float32, 1e-9)
        return [h(700, 96), h(200, 96), s(700, 200), h(700, 200), h(5000, 40), h(24, 40), s(5000, 24)]

    def run(x, w, gr, pre, x2, w2, gr2):
        return [*M.linear_backward(x, w, gr, act="gelu", pre=pre), *M.linear_backward(x2, w2, gr2), M.linear_backward(x, w, gr, need_x=False).weight]

    args = inputs(0)
    run(*args)
    T.cuda.synchronize()
    graph = T.cuda.CUDAGraph()
    with T.cuda.graph(graph):
        out = run(*args)
    for k in range(4):
        fresh = inputs(1 + k)
        for a, b in zip(args, fresh):
            a.copy_(b)
        want = run(*fresh)
        if k % 2:
            T.cuda.synchronize()
        graph.replay()
        again = run(*fresh)
        T.cuda.synchronize()
        assert all(T.equal(a, b) for a, b in zip(out, want)) and all(T.equal(a, b) for a, b in zip(again, want))
    s = T.cuda.Stream()
    s.wait_stream(T.cuda.current_stream())
    got = M.linear_backward(*fresh[:3], act="gelu", pre=fresh[3], stream=s)
    T.cuda.synchronize()
    assert all(T.equal(a, b) for a, b in zip(got, want[:3]))


@pytest.mark.parametrize("gated,act", [(True, "silu"), (False, "relu"), (True, "gelu")])
@pytest.mark.parametrize("size", [1.0, 600.0, 6000.0])
def test_f16_layers_hold_hidden_units_beyond_f16(T, M, gated, act, size):  # noqa: F811
    """Halves of `size`, whose products are far above 65,504, and an answer that f16 holds.  A hidden unit is in two parts: off by
    2^-22 relative, or 2^-25 where that is more (the second part's lowest place); what else is off as in a layer of small ones."""
    for n, (rows, cols, hidden, experts, top_k) in enumerate([(1, 64, 32, 8, 2), (1, 300, 1000, 4, 4), (3, 72, 257, 6, 2), (12, 64, 48, 40, 6),
                                                              (16, 320, 100, 16, 4), (40, 129, 33, 9, 1), (60, 256, 520, 3, 2), (100, 264, 136, 24, 3),
                                                              (200, 128, 64, 1, 1), (512, 64, 40, 12, 2), (150, 64, 1300, 2, 1)]):
        g = gen(T, 500 + n)
        top = size if gated else size * size / 10
        x, gate = real(T, g, T.float16)(rows, cols), real(T, g, T.float16, 1.5 / math.sqrt(cols))(experts, cols)
        w_in = real(T, g, T.float16, min(top, 60000.0) / math.sqrt(cols) / 8)(experts, 2 * hidden if gated else hidden, cols)
        w_out = real(T, g, T.float16, 8 / (top * top if gated else top) / math.sqrt(hidden))(experts, cols, hidden)
        r = M.layer(x, gate, w_in, w_out, top_k, act=act, gated=gated)
        y, tol, big = T.zeros(rows, cols, device=DEV, dtype=T.float64), T.zeros(rows, cols, device=DEV, dtype=T.float64), 0.0
        for e in r.routing.ids.unique().tolist():
            t, k = (r.routing.ids == e).nonzero(as_tuple=True)
            xe, wi, wo = x[t].double(), w_in[e].double(), w_out[e].double()
            a, S = xe @ wi.T, SUM(cols) * (xe.abs() @ wi.abs().T)
            p = act64(T, a[:, :hidden], act)
            ep = 1.13 * S[:, :hidden] + 2 ** -17 * (a[:, :hidden].abs() + p.abs())
            h, eh = (p * a[:, hidden:], ep * a[:, hidden:].abs() + (p.abs() + ep) * S[:, hidden:]) if gated else (p, ep)
            eh = eh + 2.0 ** -22 * h.abs() + 2.0 ** -25
            big = max(big, float(h.abs().max()))
            s = r.routing.weights[t, k].double()[:, None]
            y[t] += s * (h @ wo.T)
            tol[t] += s * (eh @ wo.abs().T + (SUM(2 * hidden + 32) + 2.0 ** -16) * ((h.abs() + eh) @ wo.abs().T))
        tol += top_k * 2 ** -23 * (y.abs() + tol) + U["f16"] * y.abs() + 2.0 ** -25
        off = float(((r.y.double() - y).abs() / tol).nan_to_num(math.inf).max())
        print(gated, act, size, rows, cols, hidden, experts, top_k, off, big, flush=True)
        assert off <= 1 and big < 2.6e8 and float(y.abs().max()) < 65000
        again = M.layer(x, gate, w_in, w_out, top_k, act=act, gated=gated)
        assert T.equal(r.y, again.y)
