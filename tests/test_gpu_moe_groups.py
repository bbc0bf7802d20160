"""Groups of experts whose worths are equal as real numbers: the lower group
stays, whatever their 64-bit sums round to.

The reference computes scores with 120 decimal digits and compares them with 40,
so that s(x) + s(-x) and 1, or the same scores and biases in another order, are
equal there.  Worths and keys that differ do so by more than 2^-46 of their size
(the reference asserts it), which 64-bit arithmetic tells apart: a worth is a sum
of four terms, a key of two, each term off by at most 4 x 2^-53 of its size.
"""

import decimal
import functools

import numpy as np
import pytest

from experiment_network_simulation_amd import inputs as I

DEV = "cuda:0"
WIDE, NARROW = decimal.Context(prec=120), decimal.Context(prec=40)
NONE = decimal.Decimal("-Infinity")


@functools.lru_cache(None)
def exp(x):
    return WIDE.exp(decimal.Decimal(x))


@functools.lru_cache(None)
def sigmoid(x):
    if x == np.inf:
        return decimal.Decimal(1)
    return WIDE.divide(1, WIDE.add(1, exp(-x)))


def told_apart(values):
    v = sorted(x for x in values if x > NONE)
    for a, b in zip(v, v[1:]):
        assert a == b or b - a > decimal.Decimal(2.0 ** -46) * max(abs(a), abs(b)), (a, b)


def real_row(x, k, score, bias, groups, top_groups):
    """ids of one row of finite logits (and -inf; sigmoid: and +inf), group_top 2."""
    x = [float(v) for v in x]
    live = [v > -np.inf and (bias is None or bias[e] > -np.inf) for e, v in enumerate(x)]
    if score == "sigmoid":
        s = [sigmoid(v) if ok else NONE for v, ok in zip(x, live)]
    else:
        # every logit that is in the row counts in the denominator
        total = functools.reduce(WIDE.add, [exp(v) for v in x if v > -np.inf], decimal.Decimal(0))
        s = [WIDE.divide(exp(v), total) if ok else NONE for v, ok in zip(x, live)]
    key = [WIDE.add(a, decimal.Decimal(float(bias[e]))) if bias is not None and a > NONE else a for e, a in enumerate(s)]
    size = len(x) // groups
    worth = []
    for g in range(groups):
        best = sorted((v for v in key[g * size:(g + 1) * size] if v > NONE), reverse=True)[:2]
        worth.append(NARROW.plus(functools.reduce(WIDE.add, best)) if best else NONE)
    told_apart(worth)
    stay = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
    if bias is None:
        key = [decimal.Decimal(v) for v in x]          # compared as they are
    key = [NARROW.plus(v) if e // size in stay else NONE for e, v in enumerate(key)]
    if bias is not None:
        told_apart(key)
    order = [e for e in sorted(range(len(x)), key=lambda e: (-key[e], e))[:k] if key[e] > NONE]
    return order + [-1] * (k - len(order))


def real_ids(x, k, score, bias, groups, top_groups):
    b = None if bias is None else bias.double().cpu().numpy()
    return np.array([real_row(r, k, score, b, groups, top_groups) for r in x.double().cpu().numpy()])


def tied_logits(rows, experts, groups, seed, inf):
    """Rows whose groups are worth the same in many ways, in values that all types hold: pairs x and -x, two
    zeros, one expert of score 1 (inf: sigmoid), the members of another group in another order; and some others."""
    g = np.random.default_rng(seed)
    size = experts // groups
    grid = lambda *n: np.round(np.abs(g.normal(0, 1.5, n)) * 16 + 1) / 16           # 8 bits from 1/16 to 16
    x = np.zeros((rows, groups, size))
    for r in range(rows):
        for a in range(groups):
            kind = g.integers(0, 5) if a else g.integers(0, 2)
            top = grid()
            m = np.concatenate([[top, -top], -top - grid(max(size - 2, 0))])[:size]
            if kind == 1 and size > 1:
                m[:2] = 0.0
                m[2:] = -grid(size - 2)
            elif kind == 2 and inf:
                m = np.where(np.arange(size) == 0, np.inf, -np.inf)
            elif kind == 3:
                m = x[r, g.integers(0, a)]
            elif kind == 4:
                m = np.round(g.normal(0, 1.5, size) * 16) / 16
            x[r, a] = g.permutation(m)
    return x.reshape(rows, experts)


SHAPES = [  # experts, groups, top_groups, top_k
    (4, 2, 1, 2), (32, 16, 5, 4), (64, 8, 3, 8), (64, 32, 7, 8), (63, 9, 4, 5), (128, 64, 20, 8), (64, 8, 4, 20), (512, 8, 3, 6),
]


def biases(kind, experts, groups, seed):
    """none; zero; one value for all; two values in an order of their own in each group; steps of 0.002 in
    float32, as a balance bias moves; with experts out of service."""
    if kind == "none":
        return None
    g = np.random.default_rng(seed)
    if kind == "zero":
        return np.zeros(experts, np.float32)
    if kind == "one":
        return np.full(experts, 0.1, np.float32)
    if kind == "orders":
        two = np.where(np.arange(experts // groups) % 2 == 0, 0.1, 0.2)
        return np.concatenate([g.permutation(two) for _ in range(groups)]).astype(np.float32)
    b = np.zeros(experts, np.float32)
    for _ in range(5):
        b += g.choice([-1, 1], experts).astype(np.float32) * np.float32(0.002)
    if kind == "out":
        b[::5] = -np.inf
    return b


KINDS = ["none", "zero", "one", "orders", "steps", "out"]


def test_the_sums_tie_only_as_real_numbers():
    """The inputs below hold rows whose worths are equal while their 64-bit sums, formed score by score, are not."""
    x = tied_logits(60, 64, 8, 64, False).reshape(60, 8, 8)
    top = np.sort(x, 2)[:, :, -2:]
    e = np.exp(-np.abs(top))
    s = np.where(top >= 0, 1.0, e) / (1.0 + e)
    pair = top.sum(2) == 0
    assert pair.any() and (s.sum(2)[pair] != 1.0).any()
    with decimal.localcontext(NARROW):
        assert {NARROW.plus(WIDE.add(sigmoid(float(a)), sigmoid(float(b)))) for a, b in top[pair]} == {decimal.Decimal(1)}


@pytest.fixture(scope="module")
def T():
    import torch
    torch.cuda.set_device(0)
    return torch


@pytest.fixture(scope="module")
def M(T):
    from experiment_network_simulation_amd import moe
    return moe


def same(T, M, x, k, score, bias, groups, top_groups):
    want = real_ids(x, k, score, bias, groups, top_groups)
    for renorm in (True, False):
        r = M.route(x, k, score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=2, renorm=renorm)
        got = r.ids.cpu().numpy()
        assert np.array_equal(got, want), [(i, got[i].tolist(), want[i].tolist()) for i in np.nonzero((got != want).any(1))[0][:5]]
        assert np.array_equal(r.load.cpu().numpy(), np.bincount(want[want >= 0], minlength=x.shape[1]))


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_four_experts(T, M, score):
    """s(2.65625) + s(-2.65625) and s(1.7265625) + s(-1.7265625) are both 1: the first group stays."""
    x = T.tensor([[2.65625, -2.65625, 1.7265625, -1.7265625], [1.7265625, -1.7265625, 2.65625, -2.65625],
                  [-2.65625, 2.65625, 0.0, -0.0], [-40.0, -41.0, -42.0, -40.0], [30.0, -30.0, 0.5, -0.5]], device=DEV)
    for dt in (T.float32, T.float16, T.bfloat16):
        for b in (None, T.zeros(4, device=DEV), T.full((4,), 0.1, device=DEV)):
            same(T, M, x[:3].to(dt), 2, score, b, 2, 1)
        same(T, M, x[3:].to(dt), 2, score, None, 2, 1)
    if score == "sigmoid":
        r = M.route(x[:3], 2, score=score, groups=2, top_groups=1, group_top=2)
        assert r.ids.tolist() == [[0, 1], [0, 1], [1, 0]]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_groups_of_equal_worth(T, M, shape, kind, score, dtype):
    experts, groups, top_groups, k = shape
    x = tied_logits(8 if experts > 128 else 60, experts, groups, experts, score == "sigmoid")
    x = T.from_numpy(x).to(DEV).to(getattr(T, dtype))
    b = biases(kind, experts, groups, 7)
    same(T, M, x, k, score, None if b is None else T.from_numpy(b).to(DEV), groups, top_groups)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("shape", [(300, 256, 8, 8, 4), (200, 63, 9, 4, 5), (100, 128, 64, 9, 8), (60, 96, 2, 1, 20)],
                         ids=lambda s: "x".join(map(str, s)))
def test_sums_of_two_sigmoids_without_bias(T, M, shape, dtype):
    """Ordinary logits of 16 bits: opposite ones are common."""
    rows, experts, groups, top_groups, k = shape
    x = T.from_numpy(I.gate_logits(rows, rows, experts, 1.5)).to(DEV).to(getattr(T, dtype))
    same(T, M, x, k, "sigmoid", None, groups, top_groups)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_masks_and_sums_of_two_sigmoids_without_bias(T, M, dtype):
    """Sums of very small scores keep their order; masked experts and groups, one expert left, +inf."""
    x = T.from_numpy(I.gate_logits(3, 20, 64, 1.5)).to(DEV).bfloat16().to(getattr(T, dtype))
    x[0] = -np.inf
    x[1, 3:] = -np.inf
    x[2] = -50.0
    x[3] = -50.0 - T.arange(64, device=DEV) % 11
    x[4] = -50.0 - (T.arange(64, device=DEV) * 29 % 64) / 4
    x[5, ::2] = -np.inf
    x[6, 7::8] = np.inf
    x[7, :8] = -np.inf
    x[8, 9:16] = -np.inf
    x[9] = 0.0
    x[10] = T.where(T.arange(64, device=DEV) % 2 == 0, 3.0, -3.0)
    for top_groups in (1, 3, 7):
        same(T, M, x, 6, "sigmoid", None, 8, top_groups)
