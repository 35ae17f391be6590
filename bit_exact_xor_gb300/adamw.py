"""The trainer's step (include/dcr_ops.h): the norm of all gradients, and AdamW
over many tensors at once.  Argument marshalling only, by the same rules as
ops.py."""
import ctypes
from typing import NamedTuple

import torch

from . import OK, check
from .ops import DTYPES, NONE, _elsewhere, _fast, _flat, _lib, _raw_stream, _refuse, _result_of

ADAMW_BLOCK = 256
NORM_WORKSPACE = 9728


class AdamState32(NamedTuple):
    """Moments of one tensor in 32 bits: m and v, float32 with its shape."""
    m: torch.Tensor
    v: torch.Tensor


class AdamState8(NamedTuple):
    """Moments of one tensor in 8 bits: m and v hold the e4m3 bytes of the first
    moment and of the second one's square root (uint8 or float8_e4m3fn, one
    for each value), m_scale and v_scale a float32 for every 256 consecutive
    values, the last of them for the rest."""
    m: torch.Tensor
    m_scale: torch.Tensor
    v: torch.Tensor
    v_scale: torch.Tensor


class _Grad(ctypes.Structure):
    _fields_ = [("values", ctypes.c_void_p), ("n", ctypes.c_uint64)]


class _Tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w", "grad", "m", "v", "m_scale", "v_scale", "copy")] + [("n", ctypes.c_uint64)]


class _Opts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay", "grad_scale", "max_norm")] + [
        ("step", ctypes.c_uint64), ("norm", ctypes.c_void_p), ("device_step", ctypes.c_void_p), ("device_lr", ctypes.c_void_p),
        ("seed", ctypes.c_uint32), ("state_bits", ctypes.c_uint32)]


_ops = None


def _library():
    global _ops
    if _ops is None:
        L = _lib()
        VP, U32 = ctypes.c_void_p, ctypes.c_uint32
        L.dcr_grad_norm.argtypes = [VP, U32, U32, VP, VP, VP]
        L.dcr_adamw.argtypes = [VP, U32, U32, U32, U32, VP, VP]
        _ops = L
    return _ops


def _list(tensors, what, like=None):
    """A list of contiguous tensors of one of DTYPES on one GPU; `like`: as many, of the same sizes, on the same device."""
    tensors = list(tensors)
    if like is not None and len(tensors) != len(like):
        _refuse("%s must have %d tensors" % (what, len(like)))
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous() or t.dtype != tensors[0].dtype or t.dtype not in DTYPES:
            _refuse("%s must be contiguous CUDA tensors, all float32, all bfloat16 or all float16" % what)
        other = tensors[0] if like is None else like[i]
        if t.device != other.device:
            _refuse("%s must lie on one device" % what)
        if like is not None and t.numel() != other.numel():
            _refuse("%s[%d] must have %d values" % (what, i, other.numel()))
    return tensors


def grad_norm(grads, stream=None):
    """dcr_grad_norm: a float32 scalar on the device, the 2-norm of all the
    tensors' values together (all float32, all bfloat16 or all float16)."""
    if stream is None:
        r = _fast.norm(grads)
        if r is not None:
            return _result_of(r)
    grads = _list(grads, "grads")
    if not grads:
        _refuse("grads must have at least one tensor")
    dev = grads[0].device
    if stream is not None or dev.index != torch.cuda.current_device():
        return _elsewhere(grad_norm, dev, stream, grads)
    table = (_Grad * len(grads))(*((t.data_ptr(), t.numel()) for t in grads))
    work = torch.empty(NORM_WORKSPACE, dtype=torch.uint8, device=dev)
    norm = torch.empty((), dtype=torch.float32, device=dev)
    rc = _library().dcr_grad_norm(table, len(grads), DTYPES[grads[0].dtype], work.data_ptr(), norm.data_ptr(), _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return norm


def adamw_states(weights, bits=32):
    """Moments of 0 for each of the weights, in 32 or in 8 bits."""
    if bits == 32:
        return [AdamState32(*(torch.zeros_like(w, dtype=torch.float32, memory_format=torch.contiguous_format) for _ in range(2))) for w in weights]
    if bits != 8:
        _refuse("bits must be 32 or 8")

    def part(w):
        return (torch.zeros_like(w, dtype=torch.uint8, memory_format=torch.contiguous_format),
                torch.zeros(-(-w.numel() // ADAMW_BLOCK), dtype=torch.float32, device=w.device))

    return [AdamState8(*part(w), *part(w)) for w in weights]


def _scalar(x, dtype, what, dev):
    """A number, or a tensor with one entry on the device: (number or 0, address or None)."""
    if isinstance(x, torch.Tensor):
        return 0, _flat(x, 1, dtype, what, dev)
    return x, None


_CODES = (torch.uint8, torch.float8_e4m3fn)


def adamw_step(weights, grads, states, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, copies=None, norm=None, max_norm=None,
               grad_scale=1.0, seed=0, stream=None):
    """dcr_adamw: one AdamW step over lists of tensors, in place.

    weights, grads and copies: contiguous tensors, each list of one type
    (float32, bfloat16 or float16); states: AdamState32 or AdamState8, one for
    each weight (adamw_states makes them).  copies receive the new weights in
    their own type, for example 16-bit views of the arena that a refit sends,
    beside a master in 32 bits.

    step: the number of this update, from 1; lr: the learning rate.  Either may
    be a tensor with one entry on the device (int64, float32), which the kernel
    reads, so that a captured graph can be replayed with other values.
    grad_scale multiplies every gradient; with norm (float32 on the device, as
    from grad_norm) and max_norm gradients are scaled down to that norm, and a
    norm that is not finite leaves the whole step out.  seed: for the rounding
    of 8-bit moments."""
    if max_norm is not None and not max_norm > 0:
        _refuse("max_norm must be positive")
    kind = type(states[0]) if states.__class__ is list and states else None
    if stream is None and (kind is AdamState32 or kind is AdamState8):
        r = _fast.adamw(weights, grads, states, 32 if kind is AdamState32 else 8, copies, norm, step, lr, betas[0], betas[1], eps, weight_decay,
                        max_norm or 0.0, grad_scale, seed & 0xFFFFFFFF)
        if r is not None:
            return None if r == OK else check(r)
    weights = _list(weights, "weights")
    if not weights:
        _refuse("weights must have at least one tensor")
    grads = _list(grads, "grads", weights)
    if copies is not None:
        copies = _list(copies, "copies", weights)
    dev = weights[0].device
    if stream is not None or dev.index != torch.cuda.current_device():
        return _elsewhere(adamw_step, dev, stream, weights, grads, states, step, lr, betas, eps, weight_decay, copies, norm, max_norm,
                          grad_scale, seed)
    states = list(states)
    if len(states) != len(weights):
        _refuse("states must have %d entries" % len(weights))
    kind = type(states[0])
    if kind not in (AdamState32, AdamState8) or any(type(s) is not kind for s in states):
        _refuse("states must be all AdamState32 or all AdamState8")
    table = (_Tensor * len(weights))()
    for i, (e, w, g, s) in enumerate(zip(table, weights, grads, states)):
        n = w.numel()
        e.w, e.grad, e.n = w.data_ptr(), g.data_ptr(), n
        if copies is not None:
            e.copy = copies[i].data_ptr()
        if kind is AdamState32:
            e.m, e.v = (_flat(x, n, torch.float32, "states", dev) for x in s)
        else:
            if s.m.dtype not in _CODES or s.v.dtype not in _CODES:
                _refuse("8-bit moments must be uint8 or float8_e4m3fn")
            blocks = -(-n // ADAMW_BLOCK)
            e.m, e.v = _flat(s.m, n, s.m.dtype, "states' m", dev), _flat(s.v, n, s.v.dtype, "states' v", dev)
            e.m_scale, e.v_scale = (_flat(x, blocks, torch.float32, "states' scales", dev) for x in (s.m_scale, s.v_scale))
    o = _Opts(beta1=betas[0], beta2=betas[1], eps=eps, weight_decay=weight_decay, grad_scale=grad_scale, max_norm=max_norm or 0.0,
              seed=seed & 0xFFFFFFFF, state_bits=32 if kind is AdamState32 else 8)
    o.step, o.device_step = _scalar(step, torch.int64, "step", dev)
    o.lr, o.device_lr = _scalar(lr, torch.float32, "lr", dev)
    if norm is not None:
        o.norm = _flat(norm, 1, torch.float32, "norm", dev)
    rc = _library().dcr_adamw(table, len(weights), DTYPES[weights[0].dtype], DTYPES[grads[0].dtype],
                              NONE if copies is None else DTYPES[copies[0].dtype], ctypes.byref(o), _raw_stream(dev.index))
    if rc != OK:
        check(rc)
