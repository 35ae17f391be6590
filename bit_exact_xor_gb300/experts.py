"""Routing to experts (include/dcr_ops.h): which experts a token goes to, the
rows' order by expert that nvfp4_linear and nvfp4_matmul take as offsets, rows
into that order and back, and the gradients.  Argument marshalling only, by
the same rules as ops.py."""
import ctypes
from typing import NamedTuple

import torch

from . import OK, check
from .ops import DTYPES, MAX_EXPERTS, SIGMOID, SOFTMAX, _elsewhere, _fast, _flat, _lib, _matrix, _raw_stream, _refuse, _result_of

MAX_CHOSEN, MAX_GROUPS, ROUTE_PARTS = 32, 32, 152
SCORINGS = {"softmax": SOFTMAX, "sigmoid": SIGMOID}
_f32, _i32 = torch.float32, torch.int32


class Route(NamedTuple):
    """Where tokens go.  experts, weights, positions [tokens, k]: the chosen
    experts (int32, the best first), their weights (float32) and the rows of
    these slots in the experts' order (int32); -1, 0 and -1 in a slot without
    an expert.  offsets (int32, experts + 1 entries): the rows of expert e are
    offsets[e] to offsets[e + 1].  order (int32 [tokens * k]): the slot, token *
    k + place, of a row; -1 behind the last."""
    experts: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor
    order: torch.Tensor
    positions: torch.Tensor


class _RouteOpts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in ("scoring", "k", "groups", "group_top", "group_by", "renormalise")] + [("scale", ctypes.c_float)]


_ops = None


def _library():
    global _ops
    if _ops is None:
        L = _lib()
        VP, U32, U64 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64
        L.dcr_route.argtypes = [VP, U32, U64, U32, U64, VP, VP, VP, VP, VP, VP, VP, VP, VP, VP]
        L.dcr_route_grad.argtypes = [VP, U32, U64, U32, U64, VP, VP, VP, VP, U64, VP]
        L.dcr_experts_gather.argtypes = [VP, U32, U64, U64, U64, VP, U32, VP, VP, U32, U64, U64, VP]
        L.dcr_experts_combine.argtypes = [VP, U32, U64, U64, U64, VP, VP, U64, U32, VP, U32, U64, VP]
        L.dcr_experts_combine_grad.argtypes = [VP, U32, U64, U64, U64, VP, VP, U64, U32, VP, U32, U64, VP, U64, VP, VP]
        _ops = L
    return _ops


def _opts(scoring, k, groups, group_top, group_by, renormalise, scale):
    if scoring not in SCORINGS:
        _refuse("scoring must be softmax or sigmoid")
    for n in (k, groups, group_top, group_by):
        if not 0 <= n < 2**32:
            _refuse("k, groups, group_top and group_by must not be negative")
    return _RouteOpts(SCORINGS[scoring], k, groups, group_top, group_by, bool(renormalise), scale)


def route_experts(logits, k, scoring="softmax", bias=None, groups=1, group_top=None, group_by=2, renormalise=True, scale=1.0, mask=None,
                  stream=None):
    """dcr_route: a Route from a router's logits [tokens, experts] (float32,
    bfloat16 or float16).

    scoring: "softmax" or "sigmoid"; bias: float32 [experts], added to the
    scores where experts are chosen but not in their weights; with groups > 1
    only the group_top groups (default: all of them) count whose group_by best
    experts sum highest; renormalise: the chosen scores are divided by their
    sum; scale multiplies the weights; mask: bool or uint8 [tokens], False for
    tokens that go nowhere."""
    if stream is None:
        r = _fast.route(logits, k, SCORINGS.get(scoring), bias, groups, groups if group_top is None else group_top, group_by, renormalise,
                        scale, mask)
        if r is not None:
            return Route(*_result_of(r))
    tokens, experts, stride, t = _matrix(logits, "logits")
    dev = logits.device
    if stream is not None or dev.index != torch.cuda.current_device():
        return _elsewhere(route_experts, dev, stream, logits, k, scoring, bias, groups, group_top, group_by, renormalise, scale, mask)
    if not 1 <= experts <= MAX_EXPERTS:
        _refuse("experts must be 1 to %d" % MAX_EXPERTS)
    if not 1 <= k <= min(MAX_CHOSEN, experts):
        _refuse("k must be 1 to %d and at most the number of experts" % MAX_CHOSEN)
    o = _opts(scoring, k, groups, groups if group_top is None else group_top, group_by, renormalise, scale)
    pb = None if bias is None else _flat(bias, experts, _f32, "bias", dev)
    pm = None
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8):
            _refuse("mask must be bool or uint8")
        pm = _flat(mask, tokens, mask.dtype, "mask", dev)
    r = Route(torch.empty((tokens, k), dtype=_i32, device=dev), torch.empty((tokens, k), dtype=_f32, device=dev),
              torch.empty(experts + 1, dtype=_i32, device=dev), torch.empty(tokens * k, dtype=_i32, device=dev),
              torch.empty((tokens, k), dtype=_i32, device=dev))
    work = torch.empty(ROUTE_PARTS * ((experts + 3) // 4 * 4), dtype=_i32, device=dev)
    rc = _library().dcr_route(logits.data_ptr(), t, tokens, experts, stride, pb, pm, ctypes.byref(o), r.experts.data_ptr(),
                              r.weights.data_ptr(), r.offsets.data_ptr(), r.order.data_ptr(), r.positions.data_ptr(), work.data_ptr(),
                              _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return r


def _slots(x, tokens, k, dtype, what, dev):
    if tuple(x.shape) != (tokens, k):
        _refuse("%s must be [%d, %d]" % (what, tokens, k))
    return _flat(x, tokens * k, dtype, what, dev)


def route_experts_grad(logits, route, grad_weights, scoring="softmax", renormalise=True, scale=1.0, out=None, stream=None):
    """dcr_route_grad: the gradient by the logits, in their type, of a loss
    whose derivative by route.weights is grad_weights (float32 [tokens, k]).
    scoring, renormalise and scale are those of route_experts; out: a matrix to
    write to (logits itself, to save the memory)."""
    if stream is None and out is None:
        r = _fast.route_grad(logits, route.experts, grad_weights, SCORINGS.get(scoring), renormalise, scale)
        if r is not None:
            return _result_of(r)
    tokens, experts, stride, t = _matrix(logits, "logits")
    dev = logits.device
    if stream is not None or dev.index != torch.cuda.current_device():
        return _elsewhere(route_experts_grad, dev, stream, logits, route, grad_weights, scoring, renormalise, scale, out)
    k = route.experts.shape[-1]
    o = _opts(scoring, k, 1, 1, 1, renormalise, scale)
    pe, pw = _slots(route.experts, tokens, k, _i32, "route.experts", dev), _slots(grad_weights, tokens, k, _f32, "grad_weights", dev)
    out, gs, _ = _output(out, tokens, experts, logits.dtype, dev, same=True)
    rc = _library().dcr_route_grad(logits.data_ptr(), t, tokens, experts, stride, pe, pw, ctypes.byref(o), out.data_ptr(), gs,
                                   _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return out


def _output(out, rows, cols, dtype, dev, same=False):
    """A matrix to write to, its row stride and type code; same: of `dtype` only."""
    if out is None:
        t = DTYPES.get(dtype)
        if t is None:
            _refuse("dtype must be float32, bfloat16 or float16")
        return torch.empty((rows, cols), dtype=dtype, device=dev), cols, t
    r, c, stride, t = _matrix(out, "out")
    if (r, c) != (rows, cols) or out.device != dev or (same and out.dtype != dtype):
        _refuse("out must be [%d, %d]%s on the same device" % (rows, cols, " of %s" % dtype if same else ""))
    return out, stride, t


def experts_gather(x, route, weighted=False, dtype=None, out=None, stream=None):
    """dcr_experts_gather: the rows of x [tokens, cols] in the experts' order,
    [tokens * k, cols] in `dtype` (default: x's) or into `out` (which may
    overlap nothing that is read), times route.weights if weighted.  Rows behind
    the last expert's are left as they are."""
    if stream is None:
        r = _fast.gather(x, route.positions, route.weights if weighted else None, DTYPES.get(x.dtype if dtype is None else dtype), out)
        if r is not None:
            return _result_of(r)
    tokens, cols, stride, t = _matrix(x, "x")
    dev = x.device
    if stream is not None or dev.index != torch.cuda.current_device():
        return _elsewhere(experts_gather, dev, stream, x, route, weighted, dtype, out)
    k = route.positions.shape[-1]
    pp = _slots(route.positions, tokens, k, _i32, "route.positions", dev)
    pw = _slots(route.weights, tokens, k, _f32, "route.weights", dev) if weighted else None
    out, os, ot = _output(out, tokens * k, cols, x.dtype if dtype is None else dtype, dev)
    rc = _library().dcr_experts_gather(x.data_ptr(), t, tokens, cols, stride, pp, k, pw, out.data_ptr(), ot, tokens * k, os,
                                       _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return out


def experts_combine(y, route, weighted=True, dtype=None, out=None, stream=None):
    """dcr_experts_combine: for each token the sum of its rows of y [tokens * k,
    cols], times route.weights if weighted, [tokens, cols] in `dtype` (default:
    y's) or into `out` (which may overlap nothing that is read).  With
    weighted=False it is experts_gather's gradient."""
    if stream is None:
        r = _fast.combine(y, route.positions, route.weights if weighted else None, DTYPES.get(y.dtype if dtype is None else dtype), out)
        if r is not None:
            return _result_of(r)
    rows, cols, stride, t = _matrix(y, "y")
    dev = y.device
    if stream is not None or dev.index != torch.cuda.current_device():
        return _elsewhere(experts_combine, dev, stream, y, route, weighted, dtype, out)
    tokens, k = route.positions.shape
    if rows != tokens * k:
        _refuse("y must have %d rows" % (tokens * k))
    pp = _slots(route.positions, tokens, k, _i32, "route.positions", dev)
    pw = _slots(route.weights, tokens, k, _f32, "route.weights", dev) if weighted else None
    out, os, ot = _output(out, tokens, cols, y.dtype if dtype is None else dtype, dev)
    rc = _library().dcr_experts_combine(y.data_ptr(), t, rows, cols, stride, pp, pw, tokens, k, out.data_ptr(), ot, os,
                                        _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return out


def experts_combine_grad(y, route, grad, out=None, stream=None):
    """dcr_experts_combine_grad of experts_combine(y, route): from the gradient
    of its output, grad [tokens, cols], those by y (in y's type; into `out`,
    which may be y itself; rows behind the last expert's are left as they are) and by route.weights
    (float32 [tokens, k])."""
    if stream is None:
        r = _fast.combine_grad(y, route.positions, route.weights, grad, out)
        if r is not None:
            return _result_of(r)
    rows, cols, stride, t = _matrix(y, "y")
    dev = y.device
    if stream is not None or dev.index != torch.cuda.current_device():
        return _elsewhere(experts_combine_grad, dev, stream, y, route, grad, out)
    tokens, k = route.positions.shape
    if rows != tokens * k:
        _refuse("y must have %d rows" % (tokens * k))
    gr, gc, gs, gt = _matrix(grad, "grad")
    if (gr, gc) != (tokens, cols) or grad.device != dev:
        _refuse("grad must be [%d, %d] on the same device" % (tokens, cols))
    pp = _slots(route.positions, tokens, k, _i32, "route.positions", dev)
    pw = _slots(route.weights, tokens, k, _f32, "route.weights", dev)
    out, os, _ = _output(out, rows, cols, y.dtype, dev, same=True)
    by_weights = torch.empty((tokens, k), dtype=_f32, device=dev)
    rc = _library().dcr_experts_combine_grad(y.data_ptr(), t, rows, cols, stride, pp, pw, tokens, k, grad.data_ptr(), gt, gs, out.data_ptr(),
                                             os, by_weights.data_ptr(), _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return out, by_weights
