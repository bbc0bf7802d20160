"""Expert-parallel routing on the GPU: from gate logits to all-to-all traffic.

Thin binding of msim_route, msim_route_backward, msim_dropout and msim_traffic
(include/msim.h has the definitions): argument checks and marshalling only,
every value is computed by the HIP library.

    r = route(logits, 8, score="sigmoid", bias=bias, groups=8, top_groups=4, group_top=2)
    w = dropout(r.weights, 0.1, seed)                  # assignments that do not travel
    pkts = traffic(r.ids, token_off, home, place, hosts, token_bytes=14336, pkt_bytes=4096,
                   drop=0.1, seed=seed)                # the same assignments, drawn again
    work = inputs.traffic_flows(pkts.cpu().numpy())    # explicit flows of an experiment

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

from .sim import ABI_VERSION, MAX_TRAFFIC_HOSTS, MsimError, RouteSpec, TrafficSpec, load_library

__all__ = ["Routing", "route", "route_backward", "dropout", "dropout_backward", "traffic"]

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_SCORES = {"softmax": 0, "sigmoid": 1}


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
