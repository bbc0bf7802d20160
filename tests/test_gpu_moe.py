"""Expert-parallel routing on the GPU against plain 64-bit implementations:
the router (choice exact, weights to rounding), its gradient, dropout (bit
for bit), the traffic table (exact), and the run of them that ends in the
simulator.

Tolerances.  u = 2^-24 is half a step of float32 relative to the value.  A
weight is a quotient of sums of at most n positive exponentials: each
exponential is off by 2 u for the function and u |argument| for the rounding of
its argument, a sum of n positive terms by at most n u however it is ordered,
the quotient and the scale by u each.  So a weight is off by at most
(2 |largest argument| + 2 n + 16) u relative (rtol_weights), n the experts
without renorm and top_k with it.  A gradient is a few products of such
quotients: grad_bound adds the bounds of its terms, times the rounding to the
output's type.
"""

import numpy as np
import pytest

from experiment_network_simulation_amd import inputs as I

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def T():
    import torch
    torch.cuda.set_device(0)
    return torch


@pytest.fixture(scope="module")
def M(T):
    from experiment_network_simulation_amd import moe
    return moe


# ---------------------------------------------------------------------------
# the plain implementation, row by row in 64 bits
# ---------------------------------------------------------------------------


def scores(x, score):
    if score == "sigmoid":
        e = np.exp(-np.abs(x))
        return np.where(x >= 0, 1.0, e) / (1.0 + e)
    top = x.max()
    e = np.where(x > -np.inf, np.exp(x - top), 0.0)
    return e / e.sum()


def plain_row(x, k, score, bias, groups, top_groups, group_top, renorm, scale):
    """ids, weights of one row of 64-bit logits."""
    ids, w = np.full(k, -1), np.zeros(k)
    if np.isnan(x).any() or (score == "softmax" and np.isposinf(x).any()):
        return ids, np.full(k, np.nan)
    if not (x > -np.inf).any():
        return ids, w
    s = scores(x, score)
    key = x.copy()
    if bias is not None:
        key = np.where((x > -np.inf) & (bias > -np.inf), s + bias, -np.inf)
    if groups > 1:
        size = x.size // groups
        value = np.full(groups, -np.inf)
        for g in range(groups):
            m = key[g * size:(g + 1) * size]
            if bias is None and group_top == 2:
                m = np.where(m > -np.inf, s[g * size:(g + 1) * size], -np.inf)
            best = np.sort(m[m > -np.inf])[::-1][:group_top]
            if best.size:
                value[g] = best.sum()
        order = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        for g in range(groups):
            if g not in order:
                key[g * size:(g + 1) * size] = -np.inf
    order = [e for e in np.argsort(-key, kind="stable")[:k] if key[e] > -np.inf]
    ids[:len(order)] = order
    if not order:
        return ids, w
    if renorm:
        xs = x[order]
        if score == "softmax":
            q = np.exp(xs - xs.max())
        else:                                # by the logarithm of the scores: sums of tiny ones do not vanish
            ls = np.minimum(xs, 0) - np.log1p(np.exp(-np.abs(xs)))
            q = np.exp(ls - ls.max())
        w[:len(order)] = scale * (q / q.sum())
    else:
        w[:len(order)] = scale * s[order]
    return ids, w


def plain_route(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    x = logits.detach().cpu().double().numpy()
    b = None if bias is None else bias.detach().cpu().double().numpy()
    if b is not None:
        b = np.where(np.isnan(b), -np.inf, b)
    with np.errstate(invalid="ignore", over="ignore"):
        rows = [plain_row(r, k, score, b, groups, top_groups, group_top, renorm, scale) for r in x]
    ids = np.array([r[0] for r in rows]).reshape(len(rows), k)
    w = np.array([r[1] for r in rows]).reshape(len(rows), k)
    return ids, w, np.bincount(ids[ids >= 0], minlength=x.shape[1])


def rtol_weights(x, n):
    fin = x[np.isfinite(x)]
    span = float(fin.max() - fin.min()) if fin.size else 0.0
    return (2 * min(span, 104.0) + 2 * n + 16) * U          # exponentials below e^-104 are 0 in float32


def check_route(M, logits, k, **how):
    r = M.route(logits, k, **how)
    ids, w, load = plain_route(logits, k, **how)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.load.cpu().numpy(), load)
    n = k if how.get("renorm", True) else logits.shape[1]
    # below 2^-126 float32 has no full precision: an absolute bound there
    np.testing.assert_allclose(r.weights.cpu().numpy().astype(np.float64), w, equal_nan=True,
                               rtol=rtol_weights(logits.cpu().double().numpy(), n), atol=2.0 ** -125)
    return r


def logits_of(T, rows, experts, dtype, seed=0, pad=0, spread=1.5):
    x = T.from_numpy(I.gate_logits(seed + 17 * rows + experts, rows, experts + pad, spread)).to(DEV).to(dtype)
    return x[:, pad - pad // 2:pad - pad // 2 + experts] if pad else x


def bias_of(T, experts, seed=3, size=0.05):
    return T.from_numpy(I.gate_logits(seed, 1, experts, size, 0.0)[0]).to(DEV)


SHAPES = [  # rows, experts, top_k, groups, top_groups, group_top
    (1, 1, 1, 1, 1, 1), (1, 4, 2, 1, 1, 1), (3, 8, 8, 1, 1, 1), (65, 64, 6, 8, 3, 1), (5, 63, 5, 9, 4, 2),
    (130, 128, 8, 1, 1, 1), (257, 160, 6, 8, 3, 1), (33, 161, 7, 7, 3, 2), (300, 256, 8, 8, 4, 2), (9, 256, 32, 4, 4, 2),
    (17, 257, 3, 1, 1, 1), (12, 384, 8, 1, 1, 1), (40, 512, 10, 16, 4, 2), (7, 1000, 16, 20, 2, 1), (21, 1024, 32, 64, 9, 2),
    (18, 192, 16, 64, 6, 2), (50, 256, 1, 8, 1, 1), (70, 96, 4, 2, 1, 2), (31, 256, 9, 8, 5, 2), (29, 32, 4, 4, 2, 2),
    (19, 16, 4, 1, 1, 1), (27, 512, 8, 8, 4, 2), (23, 256, 16, 1, 1, 1), (26, 1024, 8, 1, 1, 1), (11, 510, 12, 5, 2, 1),
    (13, 400, 16, 16, 4, 2), (45, 6, 3, 2, 2, 1), (20, 3, 2, 1, 1, 1), (36, 5, 5, 1, 1, 1), (34, 224, 16, 7, 2, 2),
]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_route(T, M, shape, score, dtype):
    rows, experts, k, groups, top_groups, group_top = shape
    dt = getattr(T, dtype)
    how = dict(score=score, groups=groups, top_groups=top_groups, group_top=group_top)
    b = bias_of(T, experts, size=0.05 if score == "sigmoid" else 0.01)
    # sums of two sigmoids without bias may be equal in 64 bits by chance of the 16-bit grid (x and -x): with bias there
    plain = dict(how, group_top=1) if score == "sigmoid" and dtype != "float32" else how
    check_route(M, logits_of(T, rows, experts, dt, 1), k, renorm=True, scale=2.5, **plain)
    check_route(M, logits_of(T, rows, experts, dt, 2, pad=3), k, renorm=False, **plain)
    check_route(M, logits_of(T, rows, experts, dt, 3), k, bias=b, renorm=True, **how)
    check_route(M, logits_of(T, rows, experts, dt, 4, pad=8), k, bias=b, renorm=False, scale=0.5, **how)


@pytest.mark.parametrize("rows", [2, 63, 64, 1000, 5000])
def test_route_lengths(T, M, rows):
    b = bias_of(T, 64)
    check_route(M, logits_of(T, rows, 64, T.bfloat16, 5), 4, score="sigmoid", bias=b, groups=4, top_groups=2, group_top=2)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lower_expert(T, M, score, bias):
    b = T.zeros(256, device=DEV) if bias else None
    x = T.zeros(5, 256, device=DEV)
    x[1] = -0.0
    x[2, 100:] = 1.0
    x[3] = T.arange(256, device=DEV).remainder(3).float()
    x[4] = T.where(T.arange(256, device=DEV) % 2 == 0, 0.0, -0.0)
    for groups, top_groups in ((1, 1), (8, 3)):
        check_route(M, x, 8, score=score, bias=b, groups=groups, top_groups=top_groups)
    # a coarse grid of logits: ties in most rows
    y = (logits_of(T, 300, 256, T.float32, 6) * 4).round().to(T.bfloat16)
    check_route(M, y, 8, score=score, bias=b)
    check_route(M, y, 8, score=score, bias=b, groups=8, top_groups=4, group_top=1)


def test_route_tells_keys_apart_that_32_bits_do_not(T, M):
    """Keys are compared as the inputs define them.  Sigmoids of 18 .. 24 are 1
    in float32 and differ by 1e-8 and less; a bias that nearly undoes the order
    of two scores leaves a difference of 1e-9."""
    g = np.random.default_rng(8)
    x = T.from_numpy(g.uniform(18.0, 24.0, (200, 256)).astype(np.float32)).to(DEV)
    check_route(M, x, 8, score="sigmoid", bias=T.zeros(256, device=DEV))
    check_route(M, x, 8, score="sigmoid", bias=T.full((256,), 0.25, device=DEV), groups=8, top_groups=4, group_top=2)
    x = T.from_numpy(g.normal(0, 1, (200, 64)).astype(np.float32)).to(DEV)
    s = T.sigmoid(x[0].double())
    b = (0.9 - s).float()                     # row 0: all keys within 2^-25 of 0.9
    check_route(M, x, 8, score="sigmoid", bias=b)
    s = T.softmax(x[0].double(), 0)
    b = (0.5 - s).float()
    check_route(M, x, 8, score="softmax", bias=b, groups=8, top_groups=2, group_top=2)
    check_route(M, x, 8, score="softmax", bias=b)


@pytest.mark.parametrize("k", [8, 16])
@pytest.mark.parametrize("experts", [256, 512])
def test_route_tells_the_first_left_out_from_the_last_chosen(T, M, experts, k):
    """All choices are neighbours, and the first that is left out differs from
    the last chosen by less than 32 bits tell, in either order."""
    x = T.full((64, experts), -3.0, device=DEV)
    x[:, :k] = 3.0 - 0.25 * T.arange(k, device=DEV)
    x[:, k] = x[:, k - 1] + T.linspace(-1e-6, 1e-6, 64, device=DEV)
    x[1::2, k - 1], x[1::2, k] = x[1::2, k].clone(), x[1::2, k - 1].clone()
    for groups, top_groups in ((1, 1), (8, 2)):
        check_route(M, x, k, score="sigmoid", bias=T.zeros(experts, device=DEV), groups=groups, top_groups=top_groups)
        check_route(M, x, k, score="softmax", bias=T.full((experts,), 0.125, device=DEV), groups=groups,
                    top_groups=top_groups, group_top=2)


def test_route_of_large_biases(T, M):
    """Keys whose biases are far larger than the scores: sums of two that nearly cancel among them."""
    g = np.random.default_rng(4)
    x = logits_of(T, 200, 64, T.float32, 12)
    b = T.from_numpy(np.where(np.arange(64) % 8 == 0, 100.0, -100.0).astype(np.float32) + g.choice([0.0, 1e-5, 0.5], 64).astype(np.float32)).to(DEV)
    check_route(M, x, 4, score="sigmoid", bias=b, groups=8, top_groups=3, group_top=2)
    check_route(M, x, 8, score="softmax", bias=b * 1000, groups=4, top_groups=2, group_top=2)
    # the lowest value as a mask: such an expert comes last, but before none
    for low in (T.finfo(T.float32).min, -1e9, -3.5, -2.9):
        b = bias_of(T, 64)
        b[::3] = low
        for score in ("softmax", "sigmoid"):
            check_route(M, x, 8, score=score, bias=b)
            check_route(M, x, 4, score=score, bias=b, groups=8, top_groups=3, group_top=2)
            b[:60] = low
            check_route(M, x, 8, score=score, bias=b)
            check_route(M, x, 4, score=score, bias=b, groups=8, top_groups=3, group_top=1)
    b = bias_of(T, 64)
    b[5], b[9], b[40], b[41] = np.inf, np.inf, T.finfo(T.float32).max, 1e31
    check_route(M, x, 8, score="sigmoid", bias=b)
    check_route(M, x, 8, score="sigmoid", bias=b, groups=8, top_groups=2)


@pytest.mark.parametrize("experts,k", [(256, 8), (64, 4), (512, 16)])
def test_route_of_many_equal_keys(T, M, experts, k):
    """A coarse grid of logits with a bias that is the same for all, or for runs of experts."""
    x = (logits_of(T, 400, experts, T.float32, 13) * 2).round()
    for b in (T.zeros(experts, device=DEV), T.full((experts,), -0.5, device=DEV),
              (T.arange(experts, device=DEV) // 7 % 2).float() * 0.25):
        for score in ("softmax", "sigmoid"):
            check_route(M, x, k, score=score, bias=b)
            check_route(M, x.bfloat16(), k, score=score, bias=b, groups=8, top_groups=4)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top_groups", [(64, 1, 1), (256, 8, 4), (161, 7, 2)])
def test_route_masks(T, M, experts, groups, top_groups, score, dtype):
    """Masked experts, rows and groups that are empty or nearly, the lowest
    finite value as a mask, infinities and NaN."""
    dt = getattr(T, dtype)
    low = T.finfo(dt).min
    x = logits_of(T, 40, experts, T.float32, 9).to(dt)
    size = experts // groups
    x[0] = -np.inf
    x[1, 3:] = -np.inf                        # fewer experts than slots
    x[2, :-1] = -np.inf
    x[3] = low
    x[4, 2:] = low
    x[5, ::2] = -np.inf
    x[6, 5] = np.nan
    x[7, 5] = np.inf
    x[8, 5:7] = np.inf
    x[9] = np.nan
    x[10, :size] = -np.inf                    # a group without experts
    x[11, size - 1:] = -np.inf
    x[12, 1:] = -np.inf                       # one expert in all
    x[13, 5], x[13, 6] = np.nan, np.inf
    x[14] = T.finfo(dt).max
    x[15, 0], x[15, 1:] = T.finfo(dt).max, low
    x[16] = -50.0                             # sigmoids whose sum is tiny
    x[17] = -200.0
    x[18, ::3] = low
    b = bias_of(T, experts)
    b[4], b[9] = -np.inf, np.nan              # experts out of service
    for renorm in (True, False):
        for bias in (None, b):
            for top in (1, 2):
                if top == 2 and bias is None and score == "sigmoid":
                    continue
                check_route(M, x, 6, score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=top,
                            renorm=renorm)
    b[6] = np.inf                             # an expert that is always chosen
    check_route(M, x, 6, score=score, bias=b, groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_route_of_tiny_logits(T, M, dtype):
    """Logits below the smallest normal number, of both signs, keep their order."""
    x = (T.arange(64, device=DEV) * 37 % 64 - 31).float().repeat(6, 1)
    x = (x * T.tensor([1e-38, 1e-39, 2.0 ** -133, 2.0 ** -126, 1e-30, 1.0], device=DEV)[:, None]).to(getattr(T, dtype))
    for score in ("softmax", "sigmoid"):
        check_route(M, x, 8, score=score)
        check_route(M, x, 16, score=score, groups=4, top_groups=2)
        check_route(M, x, 20, score=score)


def test_route_of_no_rows_and_given_outputs(T, M):
    x = logits_of(T, 50, 64, T.float32, 10)
    r = M.route(x[:0], 4)
    assert r.ids.shape == (0, 4) and r.weights.shape == (0, 4) and r.load.tolist() == [0] * 64
    want = M.route(x, 4)
    out = M.Routing(T.full((50, 4), 7, dtype=T.int32, device=DEV), T.full((50, 4), 7.0, device=DEV),
                    T.full((64,), 7, dtype=T.int32, device=DEV))
    got = M.route(x, 4, out=out)
    assert got is out and all(T.equal(a, b) for a, b in zip(got, want))
    got = M.route(x, 4, out=out._replace(load=None))
    assert got.load is None and T.equal(got.ids, want.ids)


def many_rows(T, experts, dtype, seed, pad=0):
    """More than 2,048 rows an expert, among them masked, tied, void and empty ones."""
    rows = 2048 * experts + 77
    x = logits_of(T, rows, experts, T.float32, seed, pad=pad).to(dtype) if not pad else logits_of(T, rows, experts, dtype, seed, pad=pad)
    k = T.arange(rows, device=DEV) % 300
    x[k == 3] = -np.inf
    x[k == 5, ::2] = -np.inf
    x[k == 7, experts // 2] = np.nan
    x[k == 9, experts // 3] = np.inf
    x[k == 11] = 0.25
    x[k == 13] = T.finfo(dtype).min
    x[k == 15] = -0.0
    x[k == 17, 1:] = -np.inf
    x[(k >= 20) & (k < 120)] = (x[(k >= 20) & (k < 120)] * 2).round()
    return x


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,k", [(1, 1), (3, 2), (5, 5), (8, 2), (8, 8), (13, 4), (16, 7), (31, 8), (32, 6)])
def test_route_of_many_rows_of_few_experts(T, M, experts, k, score, dtype):
    """Sampled rows against the plain implementation, and all against calls of fewer rows, which go another way."""
    for pad, renorm, bias in ((0, True, False), (3, False, True), (0, True, True), (1, False, False)):
        x = many_rows(T, experts, getattr(T, dtype), 14, pad)
        b = None
        if bias:
            b = bias_of(T, experts, size=0.05)
            b[0] = b[experts - 1]                  # equal keys where the logits are
        how = dict(score=score, bias=b, renorm=renorm, scale=1.5)
        r = M.route(x, k, **how)
        few = [M.route(x[lo:lo + 2000], k, **how) for lo in range(0, x.shape[0], 2000)]
        assert T.equal(r.ids, T.cat([f.ids for f in few]))
        assert T.equal(r.load, T.stack([f.load for f in few]).sum(0).to(T.int32))
        np.testing.assert_allclose(r.weights.cpu(), T.cat([f.weights for f in few]).cpu(), equal_nan=True,
                                   rtol=2 * rtol_weights(x.cpu().double().numpy(), experts), atol=2.0 ** -125)
        ids, w, _ = plain_route(x[:300], k, **how)
        assert np.array_equal(r.ids[:300].cpu().numpy(), ids)
        n = k if renorm else experts
        np.testing.assert_allclose(r.weights[:300].cpu().numpy().astype(np.float64), w, equal_nan=True,
                                   rtol=rtol_weights(x[:300].cpu().double().numpy(), n), atol=2.0 ** -125)


def test_many_rows_tell_keys_apart_that_32_bits_do_not(T, M):
    g = np.random.default_rng(21)
    x = T.from_numpy(g.uniform(18.0, 24.0, (2048 * 8 + 5, 8)).astype(np.float32)).to(DEV)
    r = M.route(x, 4, score="sigmoid", bias=T.zeros(8, device=DEV))
    order = x.cpu().double().numpy()
    assert np.array_equal(r.ids.cpu().numpy(), np.argsort(-order, axis=1, kind="stable")[:, :4])


def test_route_is_deterministic(T, M):
    x = logits_of(T, 20000, 128, T.bfloat16, 11)
    a, b = M.route(x, 8, score="sigmoid"), M.route(x, 8, score="sigmoid")
    assert all(T.equal(p, q) for p, q in zip(a, b))
    assert int(a.load.sum()) == 20000 * 8


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------


def weights_of(x, ids, score, renorm, scale):
    """The weights as a function of 64-bit logits, the choice held fixed (torch, for its gradient and differences)."""
    import torch
    ok = ids >= 0
    at = ids.clamp_min(0)
    xs = torch.where(ok, x.gather(1, at), torch.zeros((), dtype=x.dtype))
    ls = torch.nn.functional.logsigmoid(xs) if score == "sigmoid" else xs
    if renorm:
        top = torch.where(ok, ls, torch.full((), -torch.inf, dtype=x.dtype)).amax(1, keepdim=True)
        q = torch.where(ok, torch.exp(ls - torch.where(top > -torch.inf, top, torch.zeros_like(top))),
                        torch.zeros((), dtype=x.dtype))
        return scale * q / q.sum(1, keepdim=True).clamp_min(1e-300)
    if score == "sigmoid":
        return torch.where(ok, scale * torch.sigmoid(xs), torch.zeros((), dtype=x.dtype))
    p = torch.softmax(x, 1)
    return torch.where(ok, scale * p.gather(1, at), torch.zeros((), dtype=x.dtype))


def plain_backward(T, x, ids, g, score, renorm, scale):
    """Gradient by the formula's own differentiation in 64 bits, on the CPU."""
    xd = x.detach().cpu().double()
    keep = xd > -np.inf
    xd = T.where(keep, xd, T.full((), -1e9, dtype=T.float64)).requires_grad_(True)   # exp(-1e9) is 0: the same scores
    i = ids.cpu().long()
    i = T.where((i >= 0) & keep.gather(1, i.clamp_min(0)), i, T.full_like(i, -1))
    w = weights_of(xd, i, score, renorm, scale)
    w.backward(T.where(i >= 0, g.cpu().double(), T.zeros((), dtype=T.float64)))
    return xd.grad.numpy(), w.detach().numpy()


def grad_bound(T, x, ids, g, want, w, score, renorm, scale, k):
    """Element bound: the terms of the sum q_j (g_j - mean) are at most
    2 scale max|g|, each factor off as a weight is; then the output's rounding."""
    xs = x.cpu().double().numpy()
    n = k if renorm else x.shape[1]
    rel = rtol_weights(xs, n) + 8 * U + 2 * k * U
    size = 2 * abs(scale) * k * np.abs(g.cpu().double().numpy()).max(1, keepdims=True)
    half = T.finfo(x.dtype).eps / 2
    tiny = float(T.finfo(x.dtype).smallest_normal) * T.finfo(x.dtype).eps
    return half * np.abs(want) * (1 + rel) + rel * size + tiny


def check_backward(T, M, x, ids, g, score, renorm, scale):
    dx = M.route_backward(x, ids, g, score=score, renorm=renorm, scale=scale)
    want, w = plain_backward(T, x, ids, g, score, renorm, scale)
    got = dx.detach().cpu().double().numpy()
    off = np.abs(got - want)
    bound = grad_bound(T, x, ids, g, want, w, score, renorm, scale, ids.shape[1])
    assert dx.dtype == x.dtype and dx.shape == x.shape
    assert (off <= bound).all(), (off - bound).max()
    return want


BACK_SHAPES = [(1, 1, 1), (1, 4, 2), (7, 8, 8), (65, 64, 6), (33, 161, 7), (130, 256, 8), (5, 257, 3), (12, 1000, 16),
               (9, 1024, 32), (40, 100, 5), (300, 128, 4)]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("shape", BACK_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_route_backward(T, M, shape, renorm, score, dtype):
    rows, experts, k = shape
    for pad in (0, 3, 8):
        x = logits_of(T, rows, experts, getattr(T, dtype), 20, pad=pad)
        ids = M.route(x, k, score=score, renorm=renorm).ids
        g = T.from_numpy(I.gate_logits(21, rows, k, 1.0, 0.0)).to(DEV)
        check_backward(T, M, x, ids, g, score, renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(T, M, renorm, score):
    """Along a random direction d: <gradient, d> against (f(x + h d) - f(x - h d)) / 2h
    in 64 bits, h = 1e-4: the rest is below h^2 |f'''| / 6 < 1e-7 for these sizes (third derivatives of
    the scores are below 1, |d| below 4, 40 x 6 weights of |g| below 5), besides the float32 rounding of the gradient."""
    x = logits_of(T, 40, 96, T.float32, 22)
    ids = M.route(x, 6, score=score).ids
    g = T.from_numpy(I.gate_logits(23, 40, 6, 1.0, 0.0)).to(DEV)
    d = T.from_numpy(I.gate_logits(24, 40, 96, 1.0, 0.0)).double()
    dx = M.route_backward(x, ids, g, score=score, renorm=renorm).cpu().double()
    f = lambda t: (weights_of(t, ids.cpu().long(), score, renorm, 1.0) * g.cpu().double()).sum(1)
    h = 1e-4
    diff = (f(x.cpu().double() + h * d) - f(x.cpu().double() - h * d)) / (2 * h)
    got = (dx * d).sum(1)
    rel = rtol_weights(x.cpu().double().numpy(), 96) + 20 * U
    assert ((diff - got).abs() <= 1e-6 + rel * 2 * 6 * 5 * 4 * 6).all()
    assert (diff.abs() > 1e-3).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("experts", [61, 256])
def test_route_backward_of_odd_rows(T, M, experts, renorm, score):
    """Rows that chose nothing, masked experts, an expert named twice, indices out of range."""
    x = logits_of(T, 12, experts, T.float32, 25)
    ids = M.route(x, 5, score=score).ids
    g = T.from_numpy(I.gate_logits(26, 12, 5, 1.0, 0.0)).to(DEV)
    ids[0] = -1
    ids[1, 2:] = -1
    ids[2, 3] = ids[2, 1]                      # the same expert twice: its gradients add up
    ids[3] = ids[3, 0]
    x[4, ::2] = -np.inf
    ids[4] = M.route(x[4:5], 5, score=score).ids[0]
    x[5, ids[5, 1]] = -np.inf                  # chosen, and out since
    x[6] = -np.inf
    x[7] = -80.0
    bad = ids.clone()
    bad[8, 1], bad[9, 2], bad[10, 0] = experts, -7, 2 ** 31 - 1
    ids[8, 1], ids[9, 2], ids[10, 0] = -1, -1, -1
    want = check_backward(T, M, x, ids, g, score, renorm, 1.0)
    assert not want[0].any() and not want[6].any()
    a = M.route_backward(x, ids, g, score=score, renorm=renorm)
    b = M.route_backward(x, bad, g, score=score, renorm=renorm)
    assert T.equal(a, b)
    # a row with a NaN that chose nothing has gradient zero
    x[0, 3] = np.nan
    assert not M.route_backward(x, ids, g, score=score, renorm=renorm)[0].any()


def test_route_backward_into_a_slice(T, M):
    x = logits_of(T, 30, 100, T.bfloat16, 27)
    r = M.route(x, 4)
    g = T.ones(30, 4, device=DEV) * T.arange(4, device=DEV)
    want = M.route_backward(x, r.ids, g)
    wide = T.full((30, 117), 9.0, dtype=T.bfloat16, device=DEV)
    out = M.route_backward(x, r.ids, g, out=wide[:, 5:105])
    assert T.equal(out, want) and (wide[:, :5] == 9).all() and (wide[:, 105:] == 9).all()


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------


def kept(n, p, seed, offset):
    d = I.splitmix_draws(seed, (n + 1) // 2, offset)
    half = np.stack([d & np.uint64(0xFFFFFFFF), d >> np.uint64(32)], 1).reshape(-1)[:n]
    return half >= np.uint64(int(p * 2.0 ** 32 + 0.5))


def plain_dropout(T, x, p, seed, offset=0, per_row=False):
    """One product in float32, rounded once to the type: bit for bit what the kernel has to give."""
    rows, cols = x.shape
    k = kept(rows, p, seed, offset).reshape(rows, 1) if per_row else kept(rows * cols, p, seed, offset).reshape(rows, cols)
    y = x.cpu().float() * (np.float32(1.0 / (1.0 - p)) if p < 1 else np.float32(0))
    return T.where(T.from_numpy(k), y, T.zeros(())).to(x.dtype)


def same_bits(T, a, b):
    it = T.int32 if a.dtype == T.float32 else T.int16
    return T.equal(a.cpu().contiguous().view(it), b.cpu().contiguous().view(it))


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 2, 0), (1, 7, 0), (3, 1, 0), (5, 16, 0), (17, 33, 0), (17, 33, 5),
                                           (64, 64, 8), (64, 64, 1), (1, 4099, 0), (130, 8, 0), (2049, 24, 0), (31, 1000, 16),
                                           (300, 7, 3)])
def test_dropout(T, M, rows, cols, pad, per_row, dtype):
    x = logits_of(T, rows, cols, getattr(T, dtype), 30, pad=pad)
    for p, seed, offset in ((0.1, 7, 0), (0.5, (1 << 64) - 1, (1 << 33) + 1), (0.3, 0xABCDEF0123456789, (1 << 64) - 3)):
        y = M.dropout(x, p, seed, offset=offset, per_row=per_row)
        assert same_bits(T, y, plain_dropout(T, x, p, seed, offset, per_row)), (p, seed, offset)
        assert same_bits(T, y, M.dropout_backward(x, p, seed, offset=offset, per_row=per_row))


def test_dropout_ends_of_p(T, M):
    x = logits_of(T, 9, 40, T.float32, 31)
    assert T.equal(M.dropout(x, 0.0, 1), x)
    x[3] = np.inf
    assert not M.dropout(x, 1.0, 1).any()
    # a share so small that no 32-bit draw is below it drops nothing
    assert same_bits(T, M.dropout(x, 1e-12, 5), plain_dropout(T, x, 1e-12, 5))


def test_dropout_of_values_that_are_not_finite(T, M):
    x = logits_of(T, 64, 64, T.bfloat16, 32)
    x[::2, ::3], x[1::2, ::5], x[:, 7] = np.inf, np.nan, -np.inf
    y = M.dropout(x, 0.5, 77)
    assert T.equal(y.isnan().cpu(), x.isnan().cpu() & T.from_numpy(kept(64 * 64, 0.5, 77, 0).reshape(64, 64)))
    assert (y.cpu()[~T.from_numpy(kept(64 * 64, 0.5, 77, 0).reshape(64, 64))] == 0).all()


@pytest.mark.parametrize("shift", [0, 1, 3])
def test_dropout_in_place_slices_and_alignment(T, M, shift):
    flat = T.from_numpy(I.gate_logits(33, 1, 64 * 40 + 8)[0]).to(DEV).half()
    x = flat[shift:shift + 64 * 40].view(64, 40)
    want = plain_dropout(T, x, 0.2, 3, 9)
    rest = flat[shift + 64 * 40:].clone()
    y = M.dropout(x, 0.2, 3, offset=9, out=x)
    assert y is x and same_bits(T, x, want) and T.equal(flat[shift + 64 * 40:], rest)
    wide = T.full((64, 51), 4.0, dtype=T.float16, device=DEV)
    src = logits_of(T, 64, 40, T.float16, 34)
    M.dropout(src, 0.2, 3, offset=9, out=wide[:, 6:46])
    assert same_bits(T, wide[:, 6:46], plain_dropout(T, src, 0.2, 3, 9))
    assert (wide[:, :6] == 4).all() and (wide[:, 46:] == 4).all()


def test_dropout_past_32_bits_of_elements(T, M):
    """5 x 2^30 two-byte elements (10 GiB): the draws and the addresses behind element 2^32 are those of 64-bit positions."""
    rows, cols = 5 * (1 << 10), 1 << 20
    x = T.ones(rows, cols, dtype=T.bfloat16, device=DEV)
    M.dropout(x, 0.25, 99, offset=12, out=x)
    for row in (0, 4095, 4096, 4097, rows - 1):
        at = row * cols
        d = I.splitmix_draws(99, cols // 2, 12 + at // 2)
        half = np.stack([d & np.uint64(0xFFFFFFFF), d >> np.uint64(32)], 1).reshape(-1)
        keep = T.from_numpy(half >= np.uint64(1 << 30))
        assert T.equal(x[row].cpu() != 0, keep), row
    del x
    T.cuda.empty_cache()


# ---------------------------------------------------------------------------
# traffic
# ---------------------------------------------------------------------------


def plain_traffic(ids, off, home, place, hosts, token_bytes=1, pkt_bytes=1, drop=0.0, seed=0, offset=0, per_row=False):
    rows, k = ids.shape
    keep = kept(rows, drop, seed, offset).repeat(k).reshape(rows, k) if per_row else \
        kept(rows * k, drop, seed, offset).reshape(rows, k)
    out = np.zeros((len(home), hosts), object)
    for s in range(len(home)):
        for t in range(max(0, min(int(off[s]), rows)), max(0, min(int(off[s + 1]), rows))):
            to = {int(place[e]) for e, ok in zip(ids[t], keep[t]) if ok and 0 <= e < len(place)}
            for h in to:
                if 0 <= h < hosts and h != home[s]:
                    out[s, h] += 1
    return np.array([[min(-(-int(n) * token_bytes // pkt_bytes), 0x7FFFFFFF) for n in r] for r in out],
                    np.int64).reshape(len(home), hosts)


def check_traffic(T, M, ids, off, home, place, hosts, **how):
    dev = lambda a, dt: T.from_numpy(np.asarray(a, dt)).to(DEV)
    got = M.traffic(dev(ids, np.int32), dev(off, np.int64), dev(home, np.int32), dev(place, np.int32), hosts, **how)
    want = plain_traffic(np.asarray(ids), off, home, place, hosts, **how)
    assert np.array_equal(got.cpu().numpy(), want)
    return got


@pytest.mark.parametrize("segs,hosts,tokens,experts,k", [(1, 1, 5, 4, 2), (8, 8, 16, 64, 2), (5, 3, 33, 7, 7), (128, 128, 20, 256, 8),
                                                         (3, 1024, 300, 1024, 8), (2, 16384, 64, 1000, 32), (40, 17, 1, 9, 1),
                                                         (1, 64, 5000, 128, 6), (2, 100, 2500, 256, 16), (300, 33, 9, 40, 3)])
def test_traffic(T, M, segs, hosts, tokens, experts, k):
    g = np.random.default_rng(segs * 1000 + hosts)
    n = g.integers(0, tokens + 1, segs)
    n[0] = tokens
    off = np.concatenate([[0], np.cumsum(n)])
    rows = int(off[-1]) + 3                      # rows behind the last segment belong to nobody
    ids = np.stack([g.permutation(experts)[:k] for _ in range(rows)])
    ids[g.random((rows, k)) < 0.1] = -1
    home, place = np.arange(segs) % hosts, g.integers(0, hosts, experts)
    check_traffic(T, M, ids, off, home, place, hosts)
    check_traffic(T, M, ids, off, home, place, hosts, token_bytes=14336, pkt_bytes=4096)
    check_traffic(T, M, ids, off, home, place, hosts, drop=0.3, seed=5, offset=(1 << 32) + 7)
    check_traffic(T, M, ids, off, home, place, hosts, drop=0.4, seed=6, per_row=True, token_bytes=100, pkt_bytes=64)


@pytest.mark.parametrize("segs,tokens,hosts,k", [(1, 20000, 40, 4), (3, 9000, 7, 8), (2, 30000, 300, 3)])
def test_traffic_of_few_long_segments(T, M, segs, tokens, hosts, k):
    """Segments that several workgroups share, of very different lengths."""
    g = np.random.default_rng(hosts)
    rows = segs * tokens
    off = np.sort(np.concatenate([[0, rows - 11], g.integers(0, rows // 4, segs - 1)]))
    ids = g.integers(-1, 50, (rows, k))
    place = g.integers(0, hosts, 50)
    out = T.full((segs, hosts), 77, dtype=T.int32, device=DEV)
    check_traffic(T, M, ids, off, np.arange(segs), place, hosts, token_bytes=1000, pkt_bytes=4096)
    got = check_traffic(T, M, ids, off, np.arange(segs), place, hosts, drop=0.5, seed=4)
    dev = lambda a, dt: T.from_numpy(np.asarray(a, dt)).to(DEV)
    assert T.equal(M.traffic(dev(ids, np.int32), dev(off, np.int64), dev(np.arange(segs), np.int32), dev(place, np.int32),
                             hosts, drop=0.5, seed=4, out=out), got)
    check_traffic(T, M, ids, [0] * segs + [rows], [-1] * segs, place, hosts, token_bytes=(1 << 32) - 1, pkt_bytes=3)


def test_traffic_counts_a_host_once_and_never_itself(T, M):
    place = [0, 0, 1, 1, 2, 2]
    ids = [[0, 1, 2], [2, 3, 3], [4, 5, 0], [-1, -1, -1], [5, 5, 5]]
    got = check_traffic(T, M, ids, [0, 5], [1], place, 3)
    assert got.tolist() == [[2, 0, 2]]
    assert check_traffic(T, M, ids, [0, 5], [-1], place, 3).tolist() == [[2, 2, 2]]     # tokens that lie on none of the hosts
    check_traffic(T, M, ids, [0, 2, 2, 5], [0, 1, 2], place, 3)                         # an empty segment


def test_traffic_of_bad_entries_and_bounds(T, M):
    """Experts, hosts and offsets out of range go nowhere; nothing outside the arrays is touched."""
    ids = [[0, 9, 1], [2 ** 31 - 1, -5, 3], [2, 2, -2 ** 31]]
    place = [0, 7, -3, 2]
    check_traffic(T, M, ids, [0, 3], [5], place, 3)
    check_traffic(T, M, ids, [0, 99], [5], place, 3)
    check_traffic(T, M, ids, [-4, 2], [5], place, 3)
    check_traffic(T, M, ids, [2, 1], [5], place, 3)
    check_traffic(T, M, ids, [1 << 40, (1 << 40) + 2], [5], place, 3)
    # more packets than the table holds
    got = check_traffic(T, M, ids, [0, 3], [5], place, 3, token_bytes=(1 << 32) - 1)
    assert got.max() == 0x7FFFFFFF


def test_traffic_drops_what_dropout_drops(T, M):
    w = T.ones(500, 6, device=DEV)
    ids = np.random.default_rng(3).integers(0, 40, (500, 6))
    off, home, place = [0, 200, 500], [0, 1], np.arange(40) % 12
    for per_row in (False, True):
        gone = M.dropout(w, 0.35, 17, offset=4, per_row=per_row).cpu().numpy() == 0
        a = check_traffic(T, M, ids, off, home, place, 12, drop=0.35, seed=17, offset=4, per_row=per_row)
        b = check_traffic(T, M, np.where(gone, -1, ids), off, home, place, 12)
        assert T.equal(a, b)
    assert not check_traffic(T, M, ids, off, home, place, 12, drop=1.0).any()


def test_traffic_of_nothing(T, M):
    i = lambda *s: T.zeros(*s, dtype=T.int32, device=DEV)
    off = T.zeros(1, dtype=T.int64, device=DEV)
    assert M.traffic(i(0, 2), off, i(0), i(4), 5).shape == (0, 5)
    out = T.full((3, 5), 8, dtype=T.int32, device=DEV)
    assert not M.traffic(i(0, 2), T.zeros(4, dtype=T.int64, device=DEV), i(3), i(4), 5, out=out).any()


# ---------------------------------------------------------------------------
# as they are used together
# ---------------------------------------------------------------------------


def test_binding_refuses(T, M):
    x = T.zeros(4, 8, device=DEV)
    ids, g = T.zeros(4, 2, dtype=T.int32, device=DEV), T.zeros(4, 2, device=DEV)
    off, home, place = T.zeros(2, dtype=T.int64, device=DEV), T.zeros(1, dtype=T.int32, device=DEV), T.zeros(8, dtype=T.int32, device=DEV)
    from experiment_network_simulation_amd.sim import MsimError
    bad = [(ValueError, lambda: M.route(x, 0)), (ValueError, lambda: M.route(x, 9)), (ValueError, lambda: M.route(x[0], 2)),
           (ValueError, lambda: M.route(x, 2.5)),
           (ValueError, lambda: M.route(x.t(), 2)), (TypeError, lambda: M.route(x.double(), 2)),
           (ValueError, lambda: M.route(x[:1].expand(4, 8), 2)), (ValueError, lambda: M.route(x, 2, score="cosine")),
           (TypeError, lambda: M.route(x, 2, bias=T.zeros(8, device=DEV, dtype=T.float16))),
           (ValueError, lambda: M.route(x, 2, bias=T.zeros(7, device=DEV))), (ValueError, lambda: M.route(x, 2, bias=T.zeros(8))),
           (MsimError, lambda: M.route(x, 2, groups=3)), (MsimError, lambda: M.route(x, 2, groups=2, top_groups=3)),
           (ValueError, lambda: M.route(x, 2, group_top=3)), (MsimError, lambda: M.route(x, 2, scale=float("nan"))),
           (MsimError, lambda: M.route(T.zeros(2, 1025, device=DEV), 2)),
           (ValueError, lambda: M.route(x, 2, out=M.Routing(ids, g, ids))),
           (TypeError, lambda: M.route(x, 2, out=M.Routing(ids.long(), g, None))),
           (TypeError, lambda: M.route_backward(x, ids.long(), g)), (ValueError, lambda: M.route_backward(x, ids, g[:3])),
           (TypeError, lambda: M.route_backward(x, ids, g.half())), (ValueError, lambda: M.route_backward(x, ids, g, out=x[:, :4])),
           (ValueError, lambda: M.dropout(x, -0.5, 1)), (ValueError, lambda: M.dropout(x, float("nan"), 1)),
           (ValueError, lambda: M.dropout(x, 0.5, -1)), (ValueError, lambda: M.dropout(x, 0.5, 1 << 64)),
           (ValueError, lambda: M.dropout(x, 0.5, 1, out=x.half())),
           (MsimError, lambda: M.traffic(ids, off, home, place, 16385)),
           (TypeError, lambda: M.traffic(ids, off.int(), home, place, 4)), (ValueError, lambda: M.traffic(ids, off, home[:0], place, 4)),
           (ValueError, lambda: M.traffic(ids, off, home, place, 0)), (ValueError, lambda: M.traffic(ids, off, home, place, 4, drop=2.0)),
           (ValueError, lambda: M.traffic(ids, off, home, place, 4, token_bytes=0)), (ValueError, lambda: M.traffic(ids[:, ::2], off, home, place, 4)),
           (ValueError, lambda: M.traffic(ids, off, home, place[:0], 4))]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    T.cuda.synchronize()


def pipeline(T, M, x, off, home, place, hosts, bias, grad):
    r = M.route(x, 4, score="sigmoid", bias=bias, groups=4, top_groups=2, group_top=2, scale=2.5)
    w = M.dropout(r.weights, 0.2, 41, offset=3)
    gw = M.dropout_backward(grad, 0.2, 41, offset=3)
    dx = M.route_backward(x, r.ids, gw, score="sigmoid", scale=2.5)
    p = M.traffic(r.ids, off, home, place, hosts, token_bytes=4096, pkt_bytes=4096, drop=0.2, seed=41, offset=3)
    return [r.ids, r.weights, r.load, w, dx, p]


def pipeline_inputs(T, seed, rows=16 * 40, experts=64, hosts=16):
    x = logits_of(T, rows, experts, T.bfloat16, seed)
    off = T.arange(0, rows + 1, rows // hosts, device=DEV)
    home = T.arange(hosts, dtype=T.int32, device=DEV)
    place = (T.arange(experts, device=DEV) * hosts // experts).to(T.int32)
    return x, off, home, place, hosts, bias_of(T, experts, seed), T.from_numpy(I.gate_logits(seed + 1, rows, 4)).to(DEV)


def test_routed_tokens_through_the_simulator(T, M, oracle):
    """Logits to completion ticks: the flows are those of the plain
    implementation and the simulation of them is the oracle's, bit for bit."""
    from experiment_network_simulation_amd.sim import Sim
    args = pipeline_inputs(T, 50)
    ids, w, load, wd, dx, pk = pipeline(T, M, *args)
    x, off, home, place, hosts, bias, grad = args
    wi, _, wl = plain_route(x, 4, "sigmoid", bias, 4, 2, 2, True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), wi) and np.array_equal(load.cpu().numpy(), wl)
    want = plain_traffic(wi, off.cpu().numpy(), home.cpu().numpy(), place.cpu().numpy(), hosts, 4096, 4096, 0.2, 41, 3)
    assert np.array_equal(pk.cpu().numpy(), want)
    assert same_bits(T, wd, plain_dropout(T, w, 0.2, 41, 3))
    batch = I.single_batch(I.fat_tree(4), I.traffic_flows(pk.cpu().numpy()), 8, 3)
    sim = Sim(batch, record=[0]).bind(DEV)
    sim.run()
    got, ref = sim.results(), oracle.run(oracle.OracleBatch(batch.pack()), 0)
    assert (int(got["status"][0]), int(got["tick"][0]), int(got["digest"][0])) == (ref["status"], ref["t_end"], ref["digest"])
    assert int(got["delivered"][0]) == int(want.sum())


def test_route_designs(T, M, oracle):
    """The exploration driver: the balance bias evens the load, a group limit
    bounds the hosts a token reaches, dropping assignments removes packets, and
    each design's ticks are the oracle's for its flows."""
    from experiment_network_simulation_amd import dse
    topo, hosts, experts = I.fat_tree(4), 16, 64
    x = T.from_numpy(I.gate_logits(60, 16 * 64, experts)).to(DEV)
    off, home = np.arange(17) * 64, np.arange(16)
    place = np.arange(experts) * hosts // experts
    base = dict(top_k=4, place=place, token_bytes=4096)
    designs = [dse.RouteDesign(**base), dse.RouteDesign(**base, balance_steps=40, balance_rate=0.01),
               dse.RouteDesign(**base, groups=16, top_groups=2, group_top=2), dse.RouteDesign(**base, drop=0.5),
               dse.RouteDesign(top_k=4, place=np.full(experts, -1), score="softmax")]
    got = dse.route_designs(x, off, home, designs, topo, dse.GpuEvaluator(), queue_pkts=8, ecmp_seed=1, seed=9)
    for r in got:
        if r.work.xsrc.size:
            ref = oracle.run(oracle.OracleBatch(I.single_batch(topo, r.work, 8, 1).pack()), 0)
            assert ref["status"] == 0 and ref["t_end"] == r.ticks
    assert got[1].busiest < got[0].busiest and got[1].bias.any() and not got[0].bias.any()
    assert got[2].packets <= 2 * 1024 < got[0].packets          # two groups, one host each
    assert got[3].packets < got[0].packets
    assert got[4].packets == 0 and got[4].ticks == 0


def test_on_another_stream(T, M):
    args = pipeline_inputs(T, 70)
    want = pipeline(T, M, *args)
    s = T.cuda.Stream()
    s.wait_stream(T.cuda.current_stream())
    with T.cuda.stream(s):
        got = pipeline(T, M, *args)
    s.synchronize()
    assert all(T.equal(a, b) for a, b in zip(got, want))
    r = M.route(args[0], 4, score="sigmoid", bias=args[5], groups=4, top_groups=2, group_top=2, scale=2.5, stream=s)
    s.synchronize()
    assert T.equal(r.ids, want[0]) and T.equal(r.load, want[2])
    r = M.route(args[0], 4, score="sigmoid", bias=args[5], groups=4, top_groups=2, group_top=2, scale=2.5, stream=s.cuda_stream)
    s.synchronize()
    assert T.equal(r.ids, want[0])


def test_past_32_bits_of_logits(T, M):
    """4.7 x 10^9 logits, and a gradient of as many: rows behind element 2^32 are routed as they are by themselves."""
    rows, experts = 9 << 20, 500
    x = T.empty(rows, experts, dtype=T.bfloat16, device=DEV).normal_(0, 1.5, generator=T.Generator(DEV).manual_seed(3))
    b = bias_of(T, experts)
    how = dict(score="sigmoid", bias=b, groups=10, top_groups=4, group_top=2)
    r = M.route(x, 6, **how)
    g = T.ones(rows, 6, device=DEV) * T.arange(6, device=DEV)
    dx = M.route_backward(x, r.ids, g, score="sigmoid")
    assert int(r.load.sum(dtype=T.int64)) == 6 * rows
    for lo in (0, (1 << 32) // experts - 20, rows - 40):
        part = M.route(x[lo:lo + 40], 6, **how)
        assert T.equal(part.ids, r.ids[lo:lo + 40])
        np.testing.assert_allclose(part.weights.cpu(), r.weights[lo:lo + 40].cpu(), rtol=64 * U)
        own = M.route_backward(x[lo:lo + 40], part.ids, g[:40], score="sigmoid")
        # another number of rows adds the same terms in another order: 2^-8 is a step of bfloat16
        np.testing.assert_allclose(own.float().cpu(), dx[lo:lo + 40].float().cpu(), rtol=2.0 ** -8, atol=1e-5)
    del x, dx, r, g
    T.cuda.empty_cache()


def test_past_32_bits_of_ids(T, M):
    """4.3 x 10^9 assignments: the last segment of tokens counts as it does by itself, with the same draws."""
    rows, k = (1 << 27) + 5, 32
    ids = T.arange(64, dtype=T.int32, device=DEV).repeat(rows * k // 64 + 1)[:rows * k].view(rows, k)
    off = T.tensor([0, 7, rows - 300, rows], device=DEV)
    home = T.tensor([1, 2, 3], dtype=T.int32, device=DEV)
    place = T.arange(64, dtype=T.int32, device=DEV) % 20
    got = M.traffic(ids, off, home, place, 20, drop=0.6, seed=8)
    lo = rows - 300
    keep = kept(300 * k, 0.6, 8, lo * k // 2).reshape(300, k)
    part = np.where(keep, ids[lo:].cpu().numpy(), -1)
    want = plain_traffic(part, [0, 300], [3], place.cpu().numpy(), 20)
    assert np.array_equal(got[2].cpu().numpy(), want[0])
    del ids
    T.cuda.empty_cache()


def test_on_two_streams_at_once(T, M):
    """Calls that overlap on two streams, each with outputs of its own."""
    a, b = pipeline_inputs(T, 100, rows=16 * 500), pipeline_inputs(T, 101, rows=16 * 700)
    want = [[t.clone() for t in pipeline(T, M, *args)] for args in (a, b)]
    T.cuda.synchronize()
    streams = [T.cuda.Stream(), T.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, args in zip(streams, (a, b)):
            with T.cuda.stream(s):
                got.append(pipeline(T, M, *args))
        T.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(T.equal(p, q) for p, q in zip(w, g))


def test_captured_and_replayed(T, M):
    """Two graphs of the run, replayed in turn on new inputs with eager work
    between: every replay equals the eager result."""
    a, b = pipeline_inputs(T, 80), pipeline_inputs(T, 81, rows=16 * 8)
    s = T.cuda.Stream()
    s.wait_stream(T.cuda.current_stream())
    with T.cuda.stream(s):
        pipeline(T, M, *a), pipeline(T, M, *b)
    T.cuda.current_stream().wait_stream(s)
    graphs = []
    for args in (a, b):
        g = T.cuda.CUDAGraph()
        with T.cuda.graph(g):
            out = pipeline(T, M, *args)
        graphs.append((g, args, out))
    for turn in range(4):
        for n, (g, args, out) in enumerate(graphs):
            args[0].copy_(logits_of(T, args[0].shape[0], 64, T.bfloat16, 90 + 2 * turn + n))
            want = [t.clone() for t in pipeline(T, M, *args)]
            T.cuda.synchronize()
            g.replay()
            graphs[1 - n][0].replay()
            T.cuda.synchronize()
            for p, q in zip(out, want):
                assert T.equal(p, q), (turn, n)
