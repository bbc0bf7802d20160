"""Measured cases of the gate's and the experts' products: a matrix product with bias, activation and
residual and its gradient, a whole mixture-of-experts layer for a few tokens, and the orthogonal update of
the weights that are trained.

Each case is one pass through one operator as a program makes it that routes tokens to experts or trains
the gate.  With `own` false, `run` computes it from elementary torch operations; with `own` true it calls the
package.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _linear(name, rows, cols, outs, dtype, bias=False, act="none", residual=False, wide=False, pad=0):
    """wide: results in 32 bits, as a router takes its logits."""
    c = dict(op="linear", rows=rows, cols=cols, outs=outs, dtype=dtype, bias=bias, act=act, residual=residual, wide=wide,
             pad=pad)
    return dict(c, name=name) if name else c


def _linear_back(name, rows, cols, outs, dtype, act="none", wide=False, pad=0):
    c = dict(op="linear_backward", rows=rows, cols=cols, outs=outs, dtype=dtype, act=act, wide=wide, pad=pad)
    return dict(c, name=name) if name else c


def _layer(name, rows, cols, hidden, experts, top_k, dtype, score, bias, groups, top_groups, act="silu", gated=True,
           padding=False, residual=True):
    c = dict(op="layer", rows=rows, cols=cols, hidden=hidden, experts=experts, top_k=top_k, dtype=dtype, score=score,
             bias=bias, groups=groups, top_groups=top_groups, act=act, gated=gated, padding=padding, residual=residual)
    return dict(c, name=name) if name else c


def _orthogonalize(name, count, rows, cols, dtype):
    c = dict(op="orthogonalize", count=count, rows=rows, cols=cols, dtype=dtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # gate logits of a decoding step: eight tokens, 64 experts
        _linear("linear 8x2048->64 bf16", 8, 2048, 64, "bf16", wide=True),
        # gate logits of all tokens of the 1,024 hosts of the largest fat-tree, 14,336 bytes a token
        _linear("linear 131072x7168->256 bf16", 131072, 7168, 256, "bf16", wide=True),
        # a dense block of a training step
        _linear("linear 8192x4096->8192 bf16", 8192, 4096, 8192, "bf16", True, "gelu", True),
        # odd sizes: inputs that are slices of wider tensors
        _linear("linear 1003x1531->777 f16", 1003, 1531, 777, "f16", True, "silu", True, pad=5),
        # the gate's gradient in a training step of the largest fat-tree: tokens and weights
        _linear_back("linear back 131072x7168->256", 131072, 7168, 256, "bf16", wide=True),
        # all in 32 bits, through an activation, odd sizes
        _linear_back("linear back 2047x1000->513 f32", 2047, 1000, 513, "f32", "silu", pad=3),
        # one token: a decoding step of one sequence
        _layer("layer 1x2048, 2 of 64 bf16", 1, 2048, 1024, 64, 2, "bf16", "softmax", False, 1, 1),
        # a decoding batch of wide tokens: most experts are chosen by some token
        _layer("layer 32x7168, 8 of 128 bf16", 32, 7168, 2048, 128, 8, "bf16", "sigmoid", True, 8, 4),
        # odd sizes, several tokens an expert, padding rows behind the last token, no gate inside the experts
        _layer("layer 100x1000, 3 of 24 f16", 100, 1000, 520, 24, 3, "f16", "softmax", False, 1, 1, "gelu", False, True,
               False),
        # the update of a gate of 256 experts
        _orthogonalize("orthogonalize 256x7168 bf16", 1, 256, 7168, "bf16"),
        # the updates of four experts' matrices in one call
        _orthogonalize("orthogonalize 4x2048x7168 bf16", 4, 2048, 7168, "bf16"),
        # odd tall matrices in 32 bits
        _orthogonalize("orthogonalize 3x777x333 f32", 3, 777, 333, "f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear_backward", "layer", "layer", "orthogonalize"])
    dtype = rng.choice(list(DTYPES))
    if op in ("linear", "linear_backward"):
        # a multiple of eight, or whatever comes
        step = rng.choice([8, 8, 1])
        cols = max(1, _log(rng, 16, 8192) // step) * step
        outs = max(1, _log(rng, 8, 8192) // step) * step
        most = 2.4e11 if dtype != "f32" else 2.4e10
        rows = _log(rng, 1, max(1, min(131072, int(most / cols / outs))))
        act = rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"])
        wide, pad = rng.random() < 0.4, rng.choice([0, 0, 3, 8])
        if op == "linear":
            return _linear(None, rows, cols, outs, dtype, rng.random() < 0.5, act, rng.random() < 0.5, wide, pad)
        return _linear_back(None, rows, cols, outs, dtype, act, wide, pad)
    if op == "layer":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * max(2, _log(rng, 8, 256) // groups)
        top_groups = rng.randint(1, groups)
        top_k = min(rng.choice([1, 2, 4, 6, 8]), experts // groups * top_groups)
        step = rng.choice([64, 8, 1])
        cols = max(1, _log(rng, 64, 7168) // step) * step
        gated = rng.random() < 0.7
        parts = 3 if gated else 2
        hidden = max(1, _log(rng, 32, max(33, min(4096, int(5.0e9 / experts / cols / parts)))) // step) * step
        rows = _log(rng, 1, max(1, min(256, int(8.0e9 / top_k / parts / cols / hidden))))
        score = rng.choice(["softmax", "sigmoid"])
        return _layer(None, rows, cols, hidden, experts, top_k, dtype, score, rng.random() < 0.5, groups, top_groups,
                      rng.choice(["silu", "gelu", "gelu_tanh", "relu"]), gated, rng.random() < 0.3, rng.random() < 0.5)
    rows, cols = _log(rng, 8, 2048), _log(rng, 8, 7168)
    if rng.random() < 0.5:
        rows, cols = max(8, rows // 8 * 8), max(8, cols // 8 * 8)
    least, most = min(rows, cols), max(rows, cols)
    flops = 5 * (4 * least * least * most + 2 * least ** 3)
    return _orthogonalize(None, _log(rng, 1, max(1, min(64, int(6.0e11 / flops)))), rows, cols, dtype)


def _some(g, rows, cols, pad, dtype, scale=1.0):
    """A random [rows, cols] tensor, or with `pad` a slice of a wider one."""
    t = (scale * torch.randn(rows, cols + pad, generator=g, device="cuda")).to(dtype)
    return t[:, pad - pad // 2:pad - pad // 2 + cols] if pad else t


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    st = dict(case)
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("linear", "linear_backward"):
        R, Cc, N, pad = case["rows"], case["cols"], case["outs"], case["pad"]
        to = torch.float32 if case["wide"] else dt
        st["x"] = _some(g, R, Cc, pad, dt)
        st["weight"] = _some(g, N, Cc, pad, dt, 1.5 / math.sqrt(Cc))
        if case["op"] == "linear":
            st["b"] = 0.3 * torch.randn(N, generator=g, device=dev) if case["bias"] else None
            st["r"] = _some(g, R, N, pad, to) if case["residual"] else None
        else:
            # what the forward pass kept, and the gradient of its result
            st["pre"] = _some(g, R, N, pad, dt, 1.5) if case["act"] != "none" else None
            st["grad"] = _some(g, R, N, pad, to, 0.01)
        return st
    if case["op"] == "layer":
        T, Cc, F, E = case["rows"], case["cols"], case["hidden"], case["experts"]
        st["x"] = _some(g, T, Cc, 0, dt)
        popular = 1.0 + 0.3 * torch.randn(E, 1, generator=g, device=dev)
        st["gate"] = (popular * torch.randn(E, Cc, generator=g, device=dev) * (1.5 / math.sqrt(Cc))).to(dt)
        st["w_in"] = torch.randn(E, F * (2 if case["gated"] else 1), Cc, generator=g, device=dev, dtype=dt).mul_(1 / math.sqrt(Cc))
        st["w_out"] = torch.randn(E, Cc, F, generator=g, device=dev, dtype=dt).mul_(1 / math.sqrt(F))
        st["balance"] = (0.05 if case["score"] == "sigmoid" else 0.01) * torch.randn(E, generator=g, device=dev) \
            if case["bias"] else None
        # a batch that is not full: the rows behind the last token hold what was there before
        live = max(1, T - T // 5)
        st["mask"] = torch.arange(T, device=dev) < live if case["padding"] else None
        if case["padding"]:
            st["x"][live:] = math.nan
        st["r"] = st["x"] if case["residual"] and not case["padding"] else \
            _some(g, T, Cc, 0, dt) if case["residual"] else None
        return st
    B, m, n = case["count"], case["rows"], case["cols"]
    # a momentum: some directions that all steps share, over noise
    rank = max(1, min(m, n) // 8)
    strong = torch.randn(B, m, rank, generator=g, device=dev) * torch.logspace(0, -1, rank, device=dev)
    u = torch.matmul(strong, torch.randn(B, rank, n, generator=g, device=dev)) / math.sqrt(rank)
    st["update"] = (0.02 * (u + 0.3 * torch.randn(B, m, n, generator=g, device=dev))).to(dt)
    return st


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(st):
    z = torch.matmul(st["x"].float(), st["weight"].float().t())
    if st["b"] is not None:
        z = z + st["b"]
    y = _act(z, st["act"])
    if st["r"] is not None:
        y = y + st["r"].float()
    return y.to(torch.float32 if st["wide"] else st["x"].dtype)


def _plain_linear_backward(st):
    d = st["grad"].float()
    if st["pre"] is not None:
        d = d * _act_slope(st["pre"].float(), st["act"])
    dx = torch.matmul(d, st["weight"].float()).to(st["x"].dtype)
    dw = torch.matmul(d.t(), st["x"].float()).to(st["weight"].dtype)
    return dx, dw, d.sum(0, dtype=torch.float64).float()


def _scores(x, score):
    if score == "sigmoid":
        return torch.sigmoid(x)
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_layer(st):
    x, T, E, K, F = st["x"], st["rows"], st["experts"], st["top_k"], st["hidden"]
    live = torch.ones(T, 1, device=x.device, dtype=torch.bool) if st["mask"] is None else st["mask"][:, None]
    x = torch.where(live, x, torch.zeros_like(x))
    # logits and keys lie nearer to each other than 32 bits tell apart
    logits = torch.matmul(x.double(), st["gate"].double().t()).float()
    s = _scores(logits.double(), st["score"])
    key = logits.double() if st["balance"] is None else s + st["balance"].double()
    G = st["groups"]
    if G > 1:
        worth = key.view(T, G, E // G).amax(2)
        first = worth.sort(dim=1, descending=True, stable=True).indices[:, :st["top_groups"]]
        kept = torch.zeros_like(worth, dtype=torch.bool).scatter_(1, first, True)
        key = key.masked_fill(~kept.repeat_interleave(E // G, dim=1), -math.inf)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :K]
    w = s.gather(1, ids)
    w = torch.where(live, w / w.sum(1, keepdim=True), torch.zeros_like(w)).float()
    x = x.float()
    if T * K < E:                          # the experts that are named, one after another
        h = torch.matmul(st["w_in"][ids.view(-1)].float(), x.repeat_interleave(K, dim=0)[:, :, None])[:, :, 0]
    else:                                  # every expert for every token
        h = torch.matmul(x, st["w_in"].float().mT.contiguous())
    h = _act(h[..., :F], st["act"]) * h[..., F:] if st["gated"] else _act(h, st["act"])
    if T * K < E:
        o = torch.matmul(st["w_out"][ids.view(-1)].float(), h[:, :, None])[:, :, 0].view(T, K, -1)
        y = (o * w[:, :, None]).sum(1)
    else:
        share = torch.zeros(T, E, device=x.device).scatter_(1, ids, w)
        o = torch.matmul(h, st["w_out"].float().mT.contiguous())
        y = (o * share.t()[:, :, None]).sum(0)
    if st["r"] is not None:
        y = y + st["r"].float()
    return y.to(st["x"].dtype), torch.where(live, ids, torch.full_like(ids, -1)).to(torch.int32), w


def _plain_orthogonalize(st):
    u = st["update"].float()
    x = u if st["rows"] <= st["cols"] else u.mT.contiguous()
    x = x / (x.double().square().sum((1, 2), keepdim=True).sqrt() + 1e-7).float()
    a, b, c = COEFFICIENTS
    for _ in range(5):
        p = torch.matmul(x, x.mT.contiguous())
        x = a * x + torch.matmul(b * p + c * torch.matmul(p, p), x)
    return (x if st["rows"] <= st["cols"] else x.mT.contiguous()).to(st["update"].dtype)


def run(state):
    op = state["op"]
    if own:
        from experiment_network_simulation_amd import moe
        if op == "linear":
            return moe.linear(state["x"], state["weight"], state["b"], act=state["act"], residual=state["r"],
                              out_dtype=torch.float32 if state["wide"] else None)
        if op == "linear_backward":
            g = moe.linear_backward(state["x"], state["weight"], state["grad"], act=state["act"], pre=state["pre"])
            return g.x, g.weight, g.bias
        if op == "layer":
            y, r = moe.layer(state["x"], state["gate"], state["w_in"], state["w_out"], state["top_k"], act=state["act"],
                             gated=state["gated"], score=state["score"], bias=state["balance"], groups=state["groups"],
                             top_groups=state["top_groups"], mask=state["mask"], residual=state["r"])
            return y, r.ids, r.weights
        return moe.orthogonalize(state["update"])
    if op == "linear":
        return _plain_linear(state)
    if op == "linear_backward":
        return _plain_linear_backward(state)
    if op == "layer":
        return _plain_layer(state)
    return _plain_orthogonalize(state)


def work(case):
    size = DTYPES[case["dtype"]].itemsize
    if case["op"] in ("linear", "linear_backward"):
        R, Cc, N = case["rows"], case["cols"], case["outs"]
        to = 4 if case["wide"] else size
        if case["op"] == "linear":
            return {"bytes": (R * Cc + N * Cc) * size + R * N * to * (2 if case["residual"] else 1) + 4 * N * case["bias"],
                    "flops": 2 * R * Cc * N}
        return {"bytes": 2 * (R * Cc + N * Cc) * size + R * N * (to + (size if case["act"] != "none" else 0)) + 4 * N,
                "flops": 4 * R * Cc * N}
    if case["op"] == "layer":
        T, Cc, F, E, K = case["rows"], case["cols"], case["hidden"], case["experts"], case["top_k"]
        if case["padding"]:
            T = max(1, T - T // 5)
        parts = 3 if case["gated"] else 2
        touched = E * (1 - (1 - K / E) ** T)          # experts that some token chose, were all chosen alike
        return {"bytes": touched * parts * Cc * F * size + E * Cc * size + T * Cc * size * (3 if case["residual"] else 2)
                + 8 * T * K, "flops": 2 * T * Cc * (E + parts * F * K)}
    m, n = sorted((case["rows"], case["cols"]))
    return {"bytes": 2 * case["count"] * m * n * size, "flops": case["count"] * 5 * (4 * m * m * n + 2 * m ** 3)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_normal(z):
    """The share of a normal distribution below z."""
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _exact_act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return z * _exact_normal(z)
    if act == "gelu_tanh":                 # (1 + tanh(v)) / 2 = 1 / (1 + e^-2v)
        return z / (1.0 + torch.exp(-math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _exact_slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0).double()
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s + z * s * (1.0 - s)
    if act == "gelu":
        return _exact_normal(z) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        q = math.sqrt(8.0 / math.pi)
        s = 1.0 / (1.0 + torch.exp(-q * (z + 0.044715 * z ** 3)))
        return s + z * s * (1.0 - s) * q * (1.0 + 0.134145 * z * z)
    return torch.ones_like(z)


def exact(case, seed):
    st = prepare(case, seed)
    act = case.get("act")
    if case["op"] == "linear":
        y = st["x"].double() @ st["weight"].double().T
        if st["b"] is not None:
            y += st["b"].double()
        y = _exact_act(y, act)
        return y if st["r"] is None else y + st["r"].double()
    if case["op"] == "linear_backward":
        d = st["grad"].double()
        if act != "none":
            d *= _exact_slope(st["pre"].double(), act)
        return d @ st["weight"].double(), d.T.contiguous() @ st["x"].double(), d.sum(0)
    if case["op"] == "layer":
        T, E, K, F = case["rows"], case["experts"], case["top_k"], case["hidden"]
        live = T if st["mask"] is None else int(st["mask"].sum())
        x = st["x"][:live].double()
        z = (x @ st["gate"].double().T).float().double()
        s = 1.0 / (1.0 + torch.exp(-z)) if case["score"] == "sigmoid" else torch.softmax(z, 1)
        key = z if st["balance"] is None else s + st["balance"].double()
        if case["groups"] > 1:
            member = torch.arange(E, device=z.device) // (E // case["groups"])
            worth = torch.stack([key[:, member == k].max(1).values for k in range(case["groups"])], 1)
            place = torch.argsort(torch.argsort(worth, dim=1, descending=True, stable=True), dim=1)
            key = torch.where((place < case["top_groups"])[:, member], key, torch.full_like(key, -math.inf))
        ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :K]
        w = torch.take_along_dim(s, ids, 1)
        w = w / w.sum(1, keepdim=True)
        y = torch.zeros(T, case["cols"], device=z.device, dtype=torch.float64)
        if st["r"] is not None:
            y += st["r"].double()
        for e in ids.unique().tolist():
            t, k = (ids == e).nonzero(as_tuple=True)
            h = x[t] @ st["w_in"][e].double().T
            h = _exact_act(h[:, :F], act) * (h[:, F:] if case["gated"] else 1.0)
            y[t] += w[t, k, None] * (h @ st["w_out"][e].double().T)
        weights = torch.zeros(T, K, device=z.device, dtype=torch.float64)
        weights[:live] = w
        return y, None, weights
    x = st["update"].double()
    if case["rows"] > case["cols"]:
        x = x.transpose(1, 2)
    x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + 1e-7)
    a, b, c = COEFFICIENTS
    for _ in range(5):
        p = x @ x.transpose(1, 2)
        q = p @ x
        x = a * x + b * q + c * (p @ q)
    return (x.transpose(1, 2) if case["rows"] > case["cols"] else x).contiguous()
