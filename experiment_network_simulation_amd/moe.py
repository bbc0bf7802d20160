"""Expert-parallel routing on the GPU: from gate logits to all-to-all traffic, and
the products around the router: the gate's, its gradient and update, and a whole
layer for a few tokens.

Thin binding of msim_route, msim_route_backward, msim_dropout, msim_traffic,
msim_linear, msim_linear_backward, msim_layer and msim_orthogonalize
(include/msim.h has the definitions): argument checks and marshalling only,
every value is computed by the HIP library.

    r = route(logits, 8, score="sigmoid", bias=bias, groups=8, top_groups=4, group_top=2)
    w = dropout(r.weights, 0.1, seed)                  # assignments that do not travel
    pkts = traffic(r.ids, token_off, home, place, hosts, token_bytes=14336, pkt_bytes=4096,
                   drop=0.1, seed=seed)                # the same assignments, drawn again
    work = inputs.traffic_flows(pkts.cpu().numpy())    # explicit flows of an experiment

    logits = linear(x, gate, out_dtype=torch.float32)  # a training step of the gate
    r = route(logits, 8, score="sigmoid")
    d = route_backward(logits, r.ids, grad_weights, score="sigmoid")
    step = orthogonalize(linear_backward(x, gate, d).weight)

    y = layer(x, gate, w_in, w_out, 8, residual=x).y   # gate, router and experts of a decoding batch

All tensors are on one GPU, whichever is current.  A call enqueues on `stream`
(a torch stream or a raw handle; default: the current stream of the tensors'
device) and returns; results are allocated on that stream unless given as
`out`.  The caller orders the streams: a given `stream` has to wait for what made
the inputs, and what reads the results for `stream`; inputs and `out` may be
dropped at once, their memory stays until `stream` is past the call.  `out` must
not overlap an input (dropout's may be the input itself).  Bad arguments raise
ValueError or TypeError here, MsimError from the library; nothing is launched
then.  Results carry no autograd history: gradients are calls of their own; what
is written to `out` counts as a change in place.
"""

from __future__ import annotations

import ctypes as C
from typing import NamedTuple, Optional

import torch

from .sim import (ABI_VERSION, LINEAR_FEW, LINEAR_FEW_COLS, LINEAR_FEW_OUTS, MAX_TRAFFIC_HOSTS, LayerSpec, LinearSpec,
                  MsimError, OrthogonalizeSpec, RouteSpec, TrafficSpec, load_library)

__all__ = ["Routing", "route", "route_backward", "dropout", "dropout_backward", "traffic", "LinearGrads", "linear",
           "linear_backward", "Layer", "layer", "orthogonalize"]

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_SCORES = {"softmax": 0, "sigmoid": 1}
_ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


class Routing(NamedTuple):
    """What route() returns: ids int32 and weights float32 [rows, top_k], the
    chosen experts in descending order of key (-1 and 0 in slots that found
    none); load int32 [experts], the rows that chose each expert."""
    ids: torch.Tensor
    weights: torch.Tensor
    load: torch.Tensor


def _need(t, name: str, dtype, device, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device if device.type == 'cuda' else 'a GPU'}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_rows(t, name: str):
    """Checks for a [rows, columns] tensor whose columns lie next to each other;
    its device, rows, columns and row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, not on a GPU")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, not {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, not {t.dim()}")
    rows, cols = t.shape
    stride, inner = t.stride()
    if cols > 1 and inner != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if rows <= 1:
        stride = max(cols, 1)
    elif stride < cols:
        raise ValueError(f"{name}: rows overlap (stride {stride} for {cols} columns)")
    return t.device, rows, cols, stride


def _range(value, name: str, lo: int, hi: int) -> int:
    if type(value) is int and lo <= value <= hi:
        return value
    try:
        v = int(value)
    except OverflowError:                  # an infinity
        v = None
    if v is None or v != value or not lo <= v <= hi:
        raise ValueError(f"{name} must be a whole number in {lo} .. {hi}, not {value!r}")
    return v


class _There:
    """Makes the tensors' device and the given stream current, so that results
    are allocated there; its value is the stream's handle.  On a stream that is
    given the tensors are recorded: the allocator does not hand their memory out
    again before the stream is past this point."""

    def __init__(self, device, stream, tensors):
        given = stream is not None
        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        if given:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        self.ptr = stream.cuda_stream
        self._ctx = torch.cuda.stream(stream)

    def __enter__(self):
        self._ctx.__enter__()
        return self.ptr

    def __exit__(self, *exc):
        return self._ctx.__exit__(*exc)


def _run(device, stream, call, *tensors):
    """call(handle of the stream), with device and stream current; tensors: those
    the call is given, or None.  Where device and stream are current already,
    nothing is switched: torch's context managers cost as much as the call."""
    if stream is None and device.index == torch._C._cuda_getDevice():
        return call(torch._C._cuda_getCurrentRawStream(device.index))
    with _There(device, stream, tensors) as handle:
        return call(handle)


def _changed(*tensors):
    """Tells autograd that the library wrote to them: where one was kept for a
    backward pass, that raises instead of using the new values."""
    torch.autograd.graph.increment_version([t for t in tensors if t is not None])


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _call(rc: int):
    if rc != 0:
        raise MsimError(rc, load_library().msim_last_error(None).decode())


def _score(score: str) -> int:
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    return _SCORES[score]


def route(logits: torch.Tensor, top_k: int, *, score: str = "softmax", bias: Optional[torch.Tensor] = None,
          groups: int = 1, top_groups: int = 1, group_top: int = 1, renorm: bool = True, scale: float = 1.0,
          out: Optional[Routing] = None, stream=None) -> Routing:
    """Chooses top_k of the experts for every row of logits [rows, experts].

    score: "softmax" over the row or "sigmoid" of each logit.  bias (float32
    [experts]) is added to the scores for the choice, not to the weights.  With
    groups, only experts of the top_groups best groups are chosen, a group being
    worth the sum of its group_top (1 or 2) largest keys.  renorm divides a
    row's weights by their sum; scale multiplies them.  A logit of -inf takes
    an expert out; ties go to the lower expert."""
    dev, rows, experts, stride = _need_rows(logits, "logits")
    k = _range(top_k, "top_k", 1, max(experts, 1))
    if bias is not None:
        _need(bias, "bias", torch.float32, dev, (experts,))
    spec = RouteSpec(ABI_VERSION, _DTYPES[logits.dtype], _score(score), experts, k,
                     _range(groups, "groups", 1, 1 << 20), _range(top_groups, "top_groups", 1, 1 << 20),
                     _range(group_top, "group_top", 1, 2), 1 if renorm else 0, float(scale), rows, stride)
    if out is not None:
        _need(out.ids, "out.ids", torch.int32, dev, (rows, k))
        _need(out.weights, "out.weights", torch.float32, dev, (rows, k))
        if out.load is not None:
            _need(out.load, "out.load", torch.int32, dev, (experts,))

    def call(on):
        r = out
        if r is None:
            new = logits.new_empty
            r = Routing(new((rows, k), dtype=torch.int32), new((rows, k), dtype=torch.float32),
                        new(experts, dtype=torch.int32))
        _call(load_library().msim_route(C.byref(spec), logits.data_ptr(), _p(bias), r.ids.data_ptr(),
                                        r.weights.data_ptr(), _p(r.load), on))
        if out is not None:
            _changed(out.ids, out.weights, out.load)
        return r

    return _run(dev, stream, call, logits, bias, *(() if out is None else (out.ids, out.weights, out.load)))


def route_backward(logits: torch.Tensor, ids: torch.Tensor, grad: torch.Tensor, *, score: str = "softmax",
                   renorm: bool = True, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The gradient of route()'s weights with respect to the logits: grad
    (float32 [rows, top_k]) is that of the weights, ids are the forward pass's,
    score, renorm and scale the forward pass's arguments.  The choice itself,
    and so bias and groups, has no gradient."""
    dev, rows, experts, stride = _need_rows(logits, "logits")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a tensor of two dimensions")
    k = _range(ids.shape[1], "the number of ids in a row", 1, max(experts, 1))
    _need(ids, "ids", torch.int32, dev, (rows, k))
    _need(grad, "grad", torch.float32, dev, (rows, k))
    spec = RouteSpec(ABI_VERSION, _DTYPES[logits.dtype], _score(score), experts, k, 1, 1, 1, 1 if renorm else 0,
                     float(scale), rows, stride)
    out_stride = experts if out is None else _out_rows(out, "out", logits)

    def call(on):
        dx = logits.new_empty((rows, experts)) if out is None else out
        _call(load_library().msim_route_backward(C.byref(spec), logits.data_ptr(), ids.data_ptr(), grad.data_ptr(),
                                                 dx.data_ptr(), out_stride, on))
        if out is not None:
            _changed(out)
        return dx

    return _run(dev, stream, call, logits, ids, grad, out)


def _out_rows(out, name: str, like) -> int:
    stride = _need_rows(out, name)[3]
    if out.shape != like.shape or out.dtype != like.dtype or out.device != like.device:
        raise ValueError(f"{name} must be {like.dtype} {tuple(like.shape)} on {like.device}")
    return stride


def dropout(x: torch.Tensor, p: float, seed: int, *, offset: int = 0, per_row: bool = False,
            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [rows, columns] with each element (per_row: each row) dropped with
    probability p and the others divided by 1 - p.  The mask is a function of
    (seed, offset, element): it is never stored, and the same call on a
    gradient is the backward pass.  out may be x."""
    dev, rows, cols, xs = _need_rows(x, "x")
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be in [0, 1], not {p!r}")
    seed, offset = _range(seed, "seed", 0, (1 << 64) - 1), _range(offset, "offset", 0, (1 << 64) - 1)
    ys = max(cols, 1) if out is None else _out_rows(out, "out", x)

    def call(on):
        y = x.new_empty((rows, cols)) if out is None else out
        _call(load_library().msim_dropout(_DTYPES[x.dtype], x.data_ptr(), y.data_ptr(), rows, cols, xs, ys, float(p),
                                          seed, offset, 1 if per_row else 0, on))
        if out is not None:
            _changed(out)
        return y

    return _run(dev, stream, call, x, out)


def dropout_backward(grad: torch.Tensor, p: float, seed: int, *, offset: int = 0, per_row: bool = False,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of dropout()'s input, given that of its output and the
    arguments of the forward call."""
    return dropout(grad, p, seed, offset=offset, per_row=per_row, out=out, stream=stream)


def traffic(ids: torch.Tensor, token_off: torch.Tensor, home: torch.Tensor, place: torch.Tensor, hosts: int, *,
            token_bytes: int = 1, pkt_bytes: int = 1, drop: float = 0.0, seed: int = 0, offset: int = 0,
            per_row: bool = False, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Packets from every segment of tokens to every host, int32 [segments, hosts].

    ids: int32 [tokens, top_k] of route(); token_off: int64 [segments + 1], the
    tokens of segment s are token_off[s] .. token_off[s + 1] - 1; home: int32
    [segments], the host that holds them; place: int32 [experts], the host of
    each expert.  A token goes once to every host that holds an expert it chose,
    except its own; segments of several experiments go in one call.  With the
    defaults the result counts tokens.  drop, seed, offset and per_row leave out
    the assignments that dropout() of the weights with them drops."""
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a tensor of two dimensions")
    dev, (rows, k) = ids.device, ids.shape
    if k < 1:
        raise ValueError("ids must have at least one column")
    _need(ids, "ids", torch.int32, dev)
    _need(token_off, "token_off", torch.int64, dev)
    if token_off.dim() != 1 or token_off.numel() < 1:
        raise ValueError("token_off must have one dimension and an entry more than there are segments")
    n_seg = token_off.numel() - 1
    _need(home, "home", torch.int32, dev, (n_seg,))
    _need(place, "place", torch.int32, dev)
    if place.dim() != 1 or place.numel() < 1:
        raise ValueError("place must have one dimension and an entry for each expert")
    if not 0.0 <= drop <= 1.0:
        raise ValueError(f"drop must be in [0, 1], not {drop!r}")
    h = _range(hosts, "hosts", 1, (1 << 32) - 1)
    spec = TrafficSpec(ABI_VERSION, place.numel(), k, h, rows, n_seg,
                       _range(token_bytes, "token_bytes", 1, (1 << 32) - 1),
                       _range(pkt_bytes, "pkt_bytes", 1, (1 << 32) - 1), float(drop),
                       _range(seed, "seed", 0, (1 << 64) - 1), _range(offset, "offset", 0, (1 << 64) - 1),
                       1 if per_row else 0, 0)
    if out is not None:
        _need(out, "out", torch.int32, dev, (n_seg, h))

    def call(on):
        if h > MAX_TRAFFIC_HOSTS:          # refused before memory for such a table is asked for
            _call(load_library().msim_traffic(C.byref(spec), None, None, None, None, None, on))
        packets = ids.new_empty((n_seg, h)) if out is None else out
        _call(load_library().msim_traffic(C.byref(spec), ids.data_ptr(), token_off.data_ptr(), home.data_ptr(),
                                          place.data_ptr(), packets.data_ptr(), on))
        if out is not None:
            _changed(out)
        return packets

    return _run(dev, stream, call, ids, token_off, home, place, out)


class LinearGrads(NamedTuple):
    """What linear_backward() returns: the gradients of x [rows, cols] and weight
    [outs, cols] in their type, of bias float32 [outs]; None where not asked for."""
    x: Optional[torch.Tensor]
    weight: Optional[torch.Tensor]
    bias: Optional[torch.Tensor]


def _act(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, not {act!r}")
    return _ACTS[act]


def _like(t, name: str, dtype, device, shape) -> int:
    """Checks for a tensor of that type, device and shape with contiguous rows; its row stride."""
    stride = _need_rows(t, name)[3]
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on {device}, not {t.dtype} {tuple(t.shape)} on {t.device}")
    return stride


def _weights(x, weight):
    """Checks of x and weight; device, rows, columns, outs and the two row strides."""
    dev, rows, cols, xs = _need_rows(x, "x")
    _, outs, wide, ws = _need_rows(weight, "weight")
    if weight.device != dev or weight.dtype != x.dtype:
        raise ValueError(f"weight must be {x.dtype} on {dev}, not {weight.dtype} on {weight.device}")
    if wide != cols:
        raise ValueError(f"weight has {wide} columns, x has {cols}")
    if not 1 <= cols <= 1 << 20 or not 1 <= outs <= 1 << 20:
        raise ValueError(f"weight must have 1 .. {1 << 20} rows and columns, not {tuple(weight.shape)}")
    return dev, rows, cols, outs, xs, ws


def _workspace(like, query, *args):
    """Device memory of the size that the library asks for, and its size."""
    n = C.c_uint64()
    _call(query(*args, C.byref(n)))
    return (like.new_empty(n.value, dtype=torch.uint8) if n.value else None), n.value


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *, act: str = "none",
           residual: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
           pre: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """act(x weight^T + bias) + residual, rounded once: x [rows, cols], weight
    [outs, cols], bias float32 [outs], residual [rows, outs] of the result's type.

    act: "none", "relu", "gelu", "gelu_tanh" or "silu".  out_dtype: x's type or
    float32 (a router's logits).  pre, a [rows, outs] tensor of x's type, gets
    what goes into the activation, for linear_backward.  out may be residual."""
    dev, rows, cols, outs, xs, ws = _weights(x, weight)
    to = x.dtype if out_dtype is None else out_dtype
    if to != x.dtype and to != torch.float32:
        raise TypeError(f"out_dtype must be {x.dtype} or torch.float32, not {to}")
    if bias is not None:
        _need(bias, "bias", torch.float32, dev, (outs,))
    shape = (rows, outs)
    rs = outs if residual is None else _like(residual, "residual", to, dev, shape)
    ps = outs if pre is None else _like(pre, "pre", x.dtype, dev, shape)
    os = outs if out is None else _like(out, "out", to, dev, shape)
    spec = LinearSpec(ABI_VERSION, _DTYPES[x.dtype], _DTYPES[to], _act(act), cols, outs, rows, xs, ws, os, rs, ps, 0, 0)

    def call(on):
        lib = load_library()
        y = x.new_empty(shape, dtype=to) if out is None else out
        none = rows <= LINEAR_FEW and outs <= LINEAR_FEW_OUTS and cols <= LINEAR_FEW_COLS
        mem, size = (None, 0) if none else \
            _workspace(x, lib.msim_linear_workspace, C.byref(spec), x.data_ptr(), weight.data_ptr())
        _call(lib.msim_linear(C.byref(spec), x.data_ptr(), weight.data_ptr(), _p(bias), _p(residual), y.data_ptr(), _p(pre),
                              _p(mem), size, on))
        if out is not None or pre is not None:
            _changed(out, pre)
        return y

    return _run(dev, stream, call, x, weight, bias, residual, pre, out)


def linear_backward(x: torch.Tensor, weight: torch.Tensor, grad: torch.Tensor, *, act: str = "none",
                    pre: Optional[torch.Tensor] = None, need_x: bool = True, need_weight: bool = True,
                    need_bias: bool = True, out: Optional[LinearGrads] = None, stream=None) -> LinearGrads:
    """The gradients of linear()'s x, weight and bias, given that of its result
    (float32 or x's type [rows, outs]; the residual's gradient is grad itself) and
    for an activation what the forward pass kept in pre.  Through an activation,
    and from a float32 grad of bfloat16 arrays, the gradient in front of the
    products is rounded to x's type (half a step; the bias's is not); from a float32
    grad of float16 ones it has 16 bits and float32's range.  With out, those of its
    tensors that are not None are written, whatever the need flags say."""
    dev, rows, cols, outs, xs, ws = _weights(x, weight)
    if not isinstance(grad, torch.Tensor) or grad.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"grad must be a tensor of {x.dtype} or torch.float32")
    shape = (rows, outs)
    gs = _like(grad, "grad", grad.dtype, dev, shape)
    a = _act(act)
    if a and pre is None:
        raise ValueError(f"the gradient through {act} needs pre")
    ps = outs if pre is None else _like(pre, "pre", x.dtype, dev, shape)
    dxs = dws = cols
    if out is not None:
        dxs = cols if out.x is None else _like(out.x, "out.x", x.dtype, dev, (rows, cols))
        dws = cols if out.weight is None else _like(out.weight, "out.weight", x.dtype, dev, (outs, cols))
        if out.bias is not None:
            _need(out.bias, "out.bias", torch.float32, dev, (outs,))
    spec = LinearSpec(ABI_VERSION, _DTYPES[x.dtype], _DTYPES[grad.dtype], a, cols, outs, rows, xs, ws, gs, 0, ps, dxs, dws)

    def call(on):
        lib = load_library()
        new = x.new_empty
        g = out if out is not None else LinearGrads(new((rows, cols)) if need_x else None, new((outs, cols)) if need_weight else None,
                                                    new(outs, dtype=torch.float32) if need_bias else None)
        mem, size = _workspace(x, lib.msim_linear_backward_workspace, C.byref(spec), x.data_ptr(), weight.data_ptr(),
                               grad.data_ptr(), g.x is not None, g.weight is not None, g.bias is not None)
        _call(lib.msim_linear_backward(C.byref(spec), x.data_ptr(), weight.data_ptr(), _p(pre), grad.data_ptr(), _p(g.x),
                                       _p(g.weight), _p(g.bias), _p(mem), size, on))
        if out is not None:
            _changed(*out)
        return g

    return _run(dev, stream, call, x, weight, grad, pre, *(() if out is None else out))


class Layer(NamedTuple):
    """What layer() returns: y [rows, cols] in x's type, and the Routing it used."""
    y: torch.Tensor
    routing: Routing


def layer(x: torch.Tensor, gate: torch.Tensor, w_in: torch.Tensor, w_out: torch.Tensor, top_k: int, *, act: str = "silu",
          gated: bool = True, score: str = "softmax", bias: Optional[torch.Tensor] = None, groups: int = 1,
          top_groups: int = 1, group_top: int = 1, renorm: bool = True, scale: float = 1.0,
          mask: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None, out: Optional[Layer] = None,
          stream=None) -> Layer:
    """A whole mixture-of-experts layer for a few tokens (at most 512): routes
    every row of x [rows, cols] by its logits x gate^T as route() does, and sums
    what the chosen experts answer, by their weights, onto residual.

    gate [experts, cols]; an expert answers w_out[e] h with h = act(a) * b, a and
    b the two halves of w_in[e] x; without gated, h = act(w_in[e] x).  w_in
    [experts, 2 hidden (or hidden), cols], w_out [experts, cols, hidden]; all of
    x's type, to which h is rounded (float16: to 22 bits, and above 2.7e8 to an
    infinity).  act as in linear().  mask (bool [rows]): False for rows of padding,
    which route nowhere and get the residual alone, whatever x holds there.
    out.y may be residual."""
    dev, rows, cols, xs = _need_rows(x, "x")
    if not isinstance(gate, torch.Tensor) or gate.dim() != 2:
        raise ValueError("gate must be a tensor of two dimensions")
    if not isinstance(w_out, torch.Tensor) or w_out.dim() != 3:
        raise ValueError("w_out must be a tensor of three dimensions")
    experts, hidden = gate.shape[0], w_out.shape[2]
    if cols < 1 or hidden < 1 or experts < 1:
        raise ValueError("cols, hidden and experts must be at least 1")
    _need(gate, "gate", x.dtype, dev, (experts, cols))
    _need(w_in, "w_in", x.dtype, dev, (experts, 2 * hidden if gated else hidden, cols))
    _need(w_out, "w_out", x.dtype, dev, (experts, cols, hidden))
    k = _range(top_k, "top_k", 1, experts)
    if bias is not None:
        _need(bias, "bias", torch.float32, dev, (experts,))
    if mask is not None:
        _need(mask, "mask", torch.bool, dev, (rows,))
    rs = cols if residual is None else _like(residual, "residual", x.dtype, dev, (rows, cols))
    ys, load = cols, None
    if out is not None:
        ys = _like(out.y, "out.y", x.dtype, dev, (rows, cols))
        load = out.routing.load
        _need(out.routing.ids, "out.routing.ids", torch.int32, dev, (rows, k))
        _need(out.routing.weights, "out.routing.weights", torch.float32, dev, (rows, k))
        if load is not None:
            _need(load, "out.routing.load", torch.int32, dev, (experts,))
    limit = 1 << 20
    spec = LayerSpec(ABI_VERSION, _DTYPES[x.dtype], _act(act), 1 if gated else 0, _range(cols, "cols", 1, limit),
                     _range(hidden, "hidden", 1, limit), xs, ys, rs,
                     RouteSpec(ABI_VERSION, 0, _score(score), _range(experts, "experts", 1, limit), k, _range(groups, "groups", 1, limit),
                               _range(top_groups, "top_groups", 1, limit), _range(group_top, "group_top", 1, 2),
                               1 if renorm else 0, float(scale), rows, experts))

    def call(on):
        lib = load_library()
        mem, size = _workspace(x, lib.msim_layer_workspace, C.byref(spec))
        r = out
        if r is None:
            new = x.new_empty
            r = Layer(new((rows, cols)), Routing(new((rows, k), dtype=torch.int32), new((rows, k), dtype=torch.float32),
                                                 new(experts, dtype=torch.int32)))
        _call(lib.msim_layer(C.byref(spec), x.data_ptr(), gate.data_ptr(), _p(bias), w_in.data_ptr(), w_out.data_ptr(),
                             _p(mask), _p(residual), r.y.data_ptr(), r.routing.ids.data_ptr(), r.routing.weights.data_ptr(),
                             _p(r.routing.load), _p(mem), size, on))
        if out is not None:
            _changed(out.y, *out.routing)
        return r

    return _run(dev, stream, call, x, gate, w_in, w_out, bias, mask, residual,
                *(() if out is None else (out.y, *out.routing)))


def orthogonalize(update: torch.Tensor, *, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """update, a matrix [rows, cols] or a stack of them [count, rows, cols]
    (contiguous), each with its singular values moved towards 1: X = update /
    (norm + eps), then `steps` times X = a X + (b X X^T + c (X X^T)^2) X.  With
    the default coefficients singular values from about 0.01 of the norm on end
    within 0.7 .. 1.2.  Products are of 22 bits, errors of float32 updates those of
    float32 products; an update whose norm is far below eps has fewer bits.  out may
    be update."""
    if not isinstance(update, torch.Tensor):
        raise TypeError("update must be a tensor")
    if update.dtype not in _DTYPES:
        raise TypeError(f"update must be float32, float16 or bfloat16, not {update.dtype}")
    if update.dim() not in (2, 3):
        raise ValueError(f"update must have two or three dimensions, not {update.dim()}")
    dev = update.device
    _need(update, "update", update.dtype, dev)
    rows, cols = update.shape[-2:]
    count = update.shape[0] if update.dim() == 3 else 1
    if not 1 <= rows <= 1 << 20 or not 1 <= cols <= 1 << 20 or count > 65536:
        raise ValueError(f"update must hold at most 65536 matrices of 1 .. {1 << 20} rows and columns, not {tuple(update.shape)}")
    a, b, c = (float(v) for v in coefficients)
    spec = OrthogonalizeSpec(ABI_VERSION, _DTYPES[update.dtype], count, _range(steps, "steps", 0, 64), rows, cols, float(eps),
                             a, b, c, 0)
    if out is not None:
        _need(out, "out", update.dtype, dev, update.shape)

    def call(on):
        lib = load_library()
        mem, size = _workspace(update, lib.msim_orthogonalize_workspace, C.byref(spec))
        y = torch.empty_like(update) if out is None else out
        _call(lib.msim_orthogonalize(C.byref(spec), update.data_ptr(), y.data_ptr(), _p(mem), size, on))
        if out is not None:
            _changed(out)
        return y

    return _run(dev, stream, call, update, out)
