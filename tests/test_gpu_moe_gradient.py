"""The router's gradient against its formula in 64 bits, element by element, in
every variant: 8, 16 and 32 lanes a row (more than 16,384 rows, more than 4,096,
and fewer), chosen logits only and all of them.

Bound of an element, u = 2^-24, K choices, E experts, A the largest argument of
an exponential (at most 104: below e^-104 float32 has nothing):
 - an exponential is off by 2 u and by its argument's error: A u where float32
   holds the difference, 3 A u where that is scaled by log2(e) as well; a
   quotient or product adds u, a sum of n positive terms n u.  So a chosen
   weight q is off by (2 A + K + 18) u renormalised, (4 A + E + 8) u as a
   softmax over all, (A + 9) u as a sigmoid; a score s of any expert by
   (6 A + E + 8) u;
 - M = sum |g| q: the mean g q is off by M times (q's error + (K + 2) u).
   q (g - mean) f, f = 1 - s of a sigmoid (8 u), is then off by
   q f (|g| + M) (2 q's error + (K + 16) u), s mean by s M (s's and q's errors +
   (K + 6) u); the sum of slots that name one expert and of both terms adds
   (K + 1) u of their sizes.
Everything is within rel = (11 A + 2 n + 5 K + 64) u of the size of its own
terms, n = E for the softmax over all, K otherwise; then the output's rounding.
"""

import pytest
import torch

from experiment_network_simulation_amd import inputs as I

U = 2.0 ** -24


def formula(x, ids, g, score, renorm, scale):
    """Gradient of the weights' product with g, and the size of the terms each element is the sum of."""
    x, g = x.double(), g.double()
    rows, E = x.shape
    ok = (ids >= 0) & (ids < E)
    at = torch.where(ok, ids, torch.zeros_like(ids)).long()
    xs = x.gather(1, at)
    ok &= xs > -torch.inf
    none, some = torch.zeros((), dtype=x.dtype, device=x.device), ok.any(1, keepdim=True)
    low = torch.full_like(none, -torch.inf)
    g = torch.where(ok, g, none)
    if score == "sigmoid":
        ls = xs.clamp_max(0) - torch.log1p(torch.exp(-xs.abs()))
    else:
        top = torch.where(some, x, none).amax(1, keepdim=True)
        e = torch.exp(x - top)
        s = e / e.sum(1, keepdim=True)
        ls = xs
    if renorm:
        ls = torch.where(ok, ls, low)
        most = ls.amax(1, keepdim=True)
        q = torch.exp(ls - torch.where(most > -torch.inf, most, none))
        q = torch.where(ok, q, none)
        q = q / q.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        q = torch.where(ok, torch.exp(ls) if score == "sigmoid" else s.gather(1, at), none)
    mean, size = (g * q).sum(1, keepdim=True), (g.abs() * q).sum(1, keepdim=True)
    f = torch.where(ok, torch.sigmoid(-xs), none) if score == "sigmoid" else torch.ones_like(q)
    d = scale * q * f * (g - mean if renorm else g)
    out = torch.zeros_like(x).scatter_add_(1, at, d)
    terms = torch.zeros_like(x).scatter_add_(1, at, abs(scale) * q * f * (g.abs() + size))
    if score == "softmax" and not renorm:
        out = torch.where(some, out - scale * mean * s, none)
        terms = torch.where(some, terms + abs(scale) * size * s, none)
    return out, terms


def bound(x, g, want, terms, score, renorm, scale, dtype):
    K, E = g.shape[1], x.shape[1]
    fin = torch.where(x.isfinite(), x, torch.zeros_like(x)).double()
    A = fin.abs().amax(1) if score == "sigmoid" else fin.amax(1) - fin.amin(1)
    A = A.clamp_max(104).unsqueeze(1)
    rel = (11 * A + 2 * (E if score == "softmax" and not renorm else K) + 5 * K + 64) * U
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    least = 2.0 ** -120 * abs(scale) * g.double().abs().sum(1, keepdim=True)     # float32's exponentials end at 2^-126
    return torch.finfo(dtype).eps / 2 * want.abs() * (1 + rel) + rel * terms + tiny + least


def off(got, x, ids, g, score, renorm, scale):
    """How far the worst element lies outside its bound: not above 1 where all are within."""
    want, terms = formula(x, ids, g, score, renorm, scale)
    b = bound(x, g, want, terms, score, renorm, scale, got.dtype)
    return float(((got.double() - want).abs() / b).nan_to_num(nan=torch.inf).max())


def inputs(rows, experts, k, dtype, seed, pad=0, device="cpu"):
    x = torch.from_numpy(I.gate_logits(seed, rows, experts + pad)).to(device).to(dtype)
    if pad:
        x = x[:, pad - pad // 2:pad - pad // 2 + experts]
    ids = torch.rand(rows, experts, generator=torch.Generator().manual_seed(seed)).topk(k, 1).indices.to(torch.int32).to(device)
    g = torch.from_numpy(I.gate_logits(seed + 1, rows, k, 1.0, 0.0)).to(device)
    return x, ids, g


def odd_rows(x, ids, score, at):
    """Ten rows from `at`: nothing or little chosen, an expert named more than once, masks, indices out of range."""
    E, k = x.shape[1], ids.shape[1]
    ids[at] = -1
    ids[at + 1, k // 2:] = -1
    ids[at + 2, k - 1] = ids[at + 2, 0]
    ids[at + 3] = ids[at + 3, 0].item()
    x[at + 4, ::2] = -torch.inf               # some of the chosen are out since
    x[at + 5] = -torch.inf
    x[at + 6] = -80.0
    ids[at + 7, 0], ids[at + 7, k // 2], ids[at + 7, k - 1] = E, -7, 2 ** 31 - 1
    x[at + 8, E // 2] = torch.inf if score == "sigmoid" else 60.0
    ids[at + 8, 0] = E // 2
    x[at + 9, E // 3], ids[at + 9] = torch.nan, -1


# ---------------------------------------------------------------------------
# the formula and the bound themselves, on the CPU
# ---------------------------------------------------------------------------


def weights(x, ids, score, renorm):
    xs = x.gather(1, ids.long())
    if renorm:
        ls = torch.nn.functional.logsigmoid(xs) if score == "sigmoid" else xs
        return torch.softmax(ls, 1)
    return torch.sigmoid(xs) if score == "sigmoid" else torch.softmax(x, 1).gather(1, ids.long())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("experts,k", [(9, 2), (96, 6), (1000, 16)])
def test_the_formula_against_differences(experts, k, renorm, score):
    """(f(x + h d) - f(x - h d)) / 2 h is off by h^2 / 6 of the third derivative along d, at most h^2 (2 max|d|)^3
    of each weight's size (cumulants of d under the weights), and by the rounding of f, 2^-50 of its size over h."""
    x, ids, g = inputs(40, experts, k, torch.float64, 3)
    g = g.double()
    d = torch.from_numpy(I.gate_logits(5, 40, experts, 1.0, 0.0)).double()
    h = 1e-5
    f = lambda t: (weights(t, ids, score, renorm) * g).sum(1)
    want, _ = formula(x, ids, g, score, renorm, 1.0)
    diff = (f(x + h * d) - f(x - h * d)) / (2 * h)
    size = (weights(x, ids, score, renorm) * g.abs()).sum(1)
    assert ((diff - (want * d).sum(1)).abs() <= size * (h ** 2 * (2 * d.abs().amax(1)) ** 3 + 2.0 ** -50 / h)).all()
    assert (diff.abs() > 1e-3 * size).any()


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("experts,k", [(61, 8), (257, 3), (1000, 16), (1024, 32)])
def test_the_bound_refuses_a_gradient_without_the_mean(experts, k, dtype):
    """Softmax over all: a float32 evaluation is within the bound; without the term that every expert gets, with it
    in the first 256 columns only, without it for the chosen ones, or with one slot missing from the mean, it is not."""
    dt = getattr(torch, dtype)
    for seed in (7, 8, 9):
        x, ids, g = inputs(12, experts, k, dt, seed)
        p = torch.softmax(x.float(), 1)
        at = ids.long()
        q = p.gather(1, at)
        mean = (g * q).sum(1, keepdim=True)
        own = torch.zeros_like(p).scatter_add_(1, at, g * q)
        chosen = torch.zeros_like(p).scatter_(1, at, 1.0)
        how = (x, ids, g, "softmax", False, 2.5)
        assert off((2.5 * (own - p * mean)).to(dt), *how) <= 1
        assert off((2.5 * own).to(dt), *how) > 1
        assert off((2.5 * (own - p * mean * chosen)).to(dt), *how) > 1
        assert off((2.5 * (own - p * mean * (1 - chosen))).to(dt), *how) > 1
        assert off((2.5 * (own - p * (mean - g[:, :1] * q[:, :1]))).to(dt), *how) > 1
        if experts > 256:
            first = (torch.arange(experts) < 256).float()
            assert off((2.5 * (own - p * mean * first)).to(dt), *how) > 1


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_the_bound_refuses_a_renormalised_gradient_without_the_mean(score, dtype):
    dt = getattr(torch, dtype)
    x, ids, g = inputs(12, 128, 8, dt, 11)
    at, q = ids.long(), weights(x.float(), ids, score, True)
    f = torch.sigmoid(-x.float().gather(1, at)) if score == "sigmoid" else 1.0
    put = lambda d: torch.zeros(12, 128).scatter_add_(1, at, d).to(dt)
    how = (x, ids, g, score, True, 1.0)
    assert off(put(q * f * (g - (g * q).sum(1, keepdim=True))), *how) <= 1
    assert off(put(q * f * g), *how) > 1


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_the_formula_of_odd_rows(renorm, score):
    x, ids, g = inputs(12, 40, 5, torch.float32, 13)
    odd_rows(x, ids, score, 1)
    want, terms = formula(x, ids, g, score, renorm, 1.0)
    assert want.isfinite().all() and (want.abs() <= terms * (1 + 1e-12)).all()
    assert not want[[1, 6, 10]].any() and want[[0, 2, 3, 5, 7, 8, 9, 11]].any(1).all()
    # the same expert twice is the sum of both
    a, b, c = (formula(x[:1], ids[:1], g[:1] * m, score, False, 1.0)[0] for m in
               (torch.tensor([1.0, 0, 0, 0, 0]), torch.tensor([0, 1.0, 0, 0, 0]), torch.tensor([1.0, 1.0, 0, 0, 0])))
    torch.testing.assert_close(a + b, c, rtol=1e-12, atol=1e-15)


# ---------------------------------------------------------------------------
# the kernels
# ---------------------------------------------------------------------------


@pytest.fixture(scope="module")
def M():
    torch.cuda.set_device(0)
    from experiment_network_simulation_amd import moe
    return moe


SMALL = [(1, 1, 1), (1, 4, 2), (12, 61, 8), (65, 64, 6), (33, 161, 7), (130, 256, 8), (25, 257, 3), (40, 100, 5), (12, 1000, 16),
         (19, 1024, 32), (300, 128, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("shape", SMALL, ids=lambda s: "x".join(map(str, s)))
def test_gradient(M, shape, renorm, score, dtype):
    rows, experts, k = shape
    for pad in (0, 3, 8):
        x, ids, g = inputs(rows, experts, k, getattr(torch, dtype), 20 + pad, pad, "cuda:0")
        if rows > 10:
            odd_rows(x, ids, score, rows - 10)
        dx = M.route_backward(x, ids, g, score=score, renorm=renorm, scale=2.5)
        assert dx.dtype == x.dtype and off(dx, x, ids, g, score, renorm, 2.5) <= 1, pad


LARGE = [(61, 1), (61, 8), (61, 9), (161, 8), (161, 16), (256, 8), (257, 5), (257, 9), (1000, 8), (1000, 16), (1000, 20), (9, 9)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("rows", [4097, 16385])
def test_gradient_of_many_rows(M, rows, renorm, score, dtype):
    """The variants of 16 and of 8 lanes a row; odd rows at both ends, the last of a workgroup that is not full."""
    for n, (experts, k) in enumerate(LARGE):
        x, ids, g = inputs(rows, experts, k, getattr(torch, dtype), 40 + n, (0, 3, 8, 1)[n % 4], "cuda:0")
        odd_rows(x, ids, score, 0)
        odd_rows(x, ids, score, rows // 2)
        odd_rows(x, ids, score, rows - 10)
        dx = M.route_backward(x, ids, g, score=score, renorm=renorm, scale=0.5)
        assert off(dx, x, ids, g, score, renorm, 0.5) <= 1, (experts, k)
        wide = torch.full((rows, experts + 7), 9.0, dtype=x.dtype, device=x.device)
        out = M.route_backward(x, ids, g, score=score, renorm=renorm, scale=0.5, out=wide[:, 3:3 + experts])
        assert torch.equal(out, dx) and bool((wide[:, :3] == 9).all()) and bool((wide[:, 3 + experts:] == 9).all()), (experts, k)
