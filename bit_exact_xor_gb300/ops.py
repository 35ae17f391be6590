"""The operators around a refit (include/dcr_ops.h): NVFP4 quantisation, the
product of NVFP4 operands, and the policy loss.  Argument marshalling only, as
in the rest of the binding; tensors that are not given are allocated with
torch, and every call runs on `stream` (keyword; default: the current stream)
without waiting for it.  What a call allocates belongs to the stream that it
runs on; tensors handed in must be ready there.  A refused argument raises
DcrError.
"""
import ctypes
import functools
from typing import NamedTuple

import torch

from . import ERR_INVALID, DcrError, check, lib

F32, BF16, F16, NONE = 0, 1, 2, 3
SCALE_GIVEN, SCALE_TENSOR, SCALE_ROW = 0, 1, 2
MAX_EXPERTS = 1024
QUANT_PARTIALS = 1216
DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}

OP_EXPORTS = ["dcr_nvfp4_quantize", "dcr_nvfp4_matmul", "dcr_policy_loss", "dcr_token_logprobs",
              "dcr_ops_status"]


class Nvfp4(NamedTuple):
    """An NVFP4 matrix: codes [rows, cols / 2] uint8 (two e2m1 values a byte,
    the even column in the low four bits), scales [rows, cols / 16] uint8
    (e4m3) and scale, a float32 tensor with one entry, one per row, or (the
    weights of several experts) one per expert."""
    codes: torch.Tensor
    scales: torch.Tensor
    scale: torch.Tensor


class _Nvfp4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("scale_count", ctypes.c_uint64)]


class PolicyOpts(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float),
                ("kl_coef", ctypes.c_float)]


_ops = None


def _lib():
    global _ops
    if _ops is None:
        L = lib()
        P, VP, U32, U64 = ctypes.POINTER, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64
        L.dcr_nvfp4_quantize.argtypes = [VP, U32, U64, U64, U64, U32, VP, VP, VP, VP, U32, VP, VP]
        L.dcr_nvfp4_matmul.argtypes = [P(_Nvfp4), P(_Nvfp4), U64, U64, U64, VP, U32, VP, U32, U64, VP]
        L.dcr_policy_loss.argtypes = [VP, U32, U64, U64, U64, VP, VP, VP, VP, VP, P(PolicyOpts), VP, VP, VP, VP, U64, VP]
        L.dcr_token_logprobs.argtypes = [VP, U32, U64, U64, U64, VP, ctypes.c_float, VP, VP]
        L.dcr_ops_status.argtypes = [VP]
        _ops = L
    return _ops


def _need(ok, what):
    if not ok:
        raise DcrError(ERR_INVALID, what)


def _matrix(x, what, dtypes=DTYPES):
    _need(x.is_cuda, what + " must be a CUDA tensor")
    _need(x.dim() == 2, what + " must have two dimensions")
    _need(x.dtype in dtypes, what + " has an unsupported type")
    r, c = x.shape
    _need(c <= 1 or x.stride(1) == 1, what + " must be contiguous in its last dimension")
    # the stride of a single row says nothing
    stride = x.stride(0) if r > 1 else c
    _need(stride >= c, what + " has overlapping rows")
    return r, c, stride


def _flat(x, n, dtype, what, device):
    _need(x.device == device, what + " must be on the same device")
    _need(x.dtype == dtype, what + " has an unsupported type")
    _need(x.numel() == n and x.is_contiguous(), what + " must be contiguous with %d entries" % n)
    return x.data_ptr()


def _out(x, shape, dtype, what, device):
    """The caller's output, or a new one."""
    if x is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _flat(x, shape[0] * shape[1] if len(shape) == 2 else shape[0], dtype, what, device)
    return x


def _on_stream(f):
    """Runs f with `stream` current, so that what f allocates belongs to that
    stream, and with the device of its first tensor current."""
    @functools.wraps(f)
    def call(x, *args, stream=None, **kw):
        dev = getattr(x, "codes", x).device
        if stream is None:
            if dev.index is None or dev.index == torch.cuda.current_device():
                return f(x, *args, **kw)
            with torch.cuda.device(dev):
                return f(x, *args, **kw)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        with torch.cuda.stream(stream):
            return f(x, *args, **kw)
    return call


def _stream():
    return torch.cuda.current_stream().cuda_stream


@_on_stream
def nvfp4_quantize(x, scale=None, per_row=False, values=None, out=None):
    """dcr_nvfp4_quantize of x [rows, cols] (float32, bfloat16 or float16).

    The 32-bit scale is `scale` (one float32 value on the device) if given,
    else computed from all of x, or from each row with per_row=True.  `values`
    is a tensor [rows, cols], or a type to make one of, that receives what the
    codes stand for.  `out` is an Nvfp4 whose tensors are written (its scale
    is an output, too, unless `scale` is given), for example views of a
    trainer arena.  Returns (Nvfp4, values or None)."""
    rows, cols, stride = _matrix(x, "x")
    _need(cols % 16 == 0, "x must have a multiple of 16 columns")
    _need(not (per_row and scale is not None), "a given scale and per_row do not go together")
    dev = x.device
    codes, scales, sc = out if out is not None else (None, None, None)
    codes = _out(codes, (rows, cols // 2), torch.uint8, "codes", dev)
    scales = _out(scales, (rows, cols // 16), torch.uint8, "scales", dev)
    if scale is not None:
        _flat(scale, 1, torch.float32, "scale", dev)
        mode, sc = SCALE_GIVEN, scale
    else:
        mode = SCALE_ROW if per_row else SCALE_TENSOR
        if sc is not None:
            _flat(sc, rows if per_row else 1, torch.float32, "scale", dev)
        elif per_row:
            sc = torch.empty(rows, dtype=torch.float32, device=dev)
    work = None
    if mode == SCALE_TENSOR:
        work = torch.empty(QUANT_PARTIALS + 1, dtype=torch.float32, device=dev)
        sc = work[QUANT_PARTIALS:] if sc is None else sc
    vt = NONE
    if values is not None:
        if isinstance(values, torch.dtype):
            values = torch.empty((rows, cols), dtype=values, device=dev)
        vt = DTYPES.get(values.dtype)
        _need(vt is not None, "values has an unsupported type")
        _flat(values, rows * cols, values.dtype, "values", dev)
    check(_lib().dcr_nvfp4_quantize(x.data_ptr(), DTYPES[x.dtype], rows, cols, stride, mode, sc.data_ptr(),
                                    codes.data_ptr(), scales.data_ptr(),
                                    values.data_ptr() if values is not None else None, vt,
                                    work.data_ptr() if work is not None else None, _stream()))
    return Nvfp4(codes, scales, sc), values


def _nvfp4(a, what):
    rows, half, stride = _matrix(a.codes, what + ".codes", (torch.uint8,))
    _need(stride == half, what + ".codes must be contiguous")
    k = 2 * half
    _need(k > 0 and k % 32 == 0, what + " must have a positive multiple of 32 columns")
    dev = a.codes.device
    s = a.scales.view(torch.uint8) if a.scales.dtype == torch.float8_e4m3fn else a.scales
    return rows, k, _Nvfp4(a.codes.data_ptr(), _flat(s, rows * (k // 16), torch.uint8, what + ".scales", dev),
                           _flat(a.scale, a.scale.numel(), torch.float32, what + ".scale", dev), a.scale.numel())


@_on_stream
def nvfp4_matmul(x, w, offsets=None, dtype=torch.bfloat16, out=None):
    """dcr_nvfp4_matmul: y = x w^T of two Nvfp4 matrices, x [m, k] and w
    [n, k], in `dtype` (or into `out` [m, n]).

    offsets (int32, experts + 1 entries on the device, not decreasing): w is
    [experts * n, k], and rows offsets[e] to offsets[e + 1] of x are multiplied
    by expert e's matrix; rows that no expert has are not written."""
    m, k, cx = _nvfp4(x, "x")
    wrows, wk, cw = _nvfp4(w, "w")
    _need(k == wk, "x and w must have the same number of columns")
    dev = x.codes.device
    _need(w.codes.device == dev, "w must be on the same device")
    experts, po = 0, None
    if offsets is not None:
        experts = offsets.numel() - 1
        _need(1 <= experts <= MAX_EXPERTS, "offsets must have 2 to %d entries" % (MAX_EXPERTS + 1))
        _need(wrows % experts == 0, "w's rows must be a multiple of the number of experts")
        po = _flat(offsets, experts + 1, torch.int32, "offsets", dev)
    n = wrows // max(experts, 1)
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=dev)
        ys = n
    else:
        om, on, ys = _matrix(out, "out")
        _need((om, on) == (m, n) and out.device == dev, "out must be [%d, %d] on the same device" % (m, n))
    _need(out.dtype in DTYPES, "dtype is not supported")
    check(_lib().dcr_nvfp4_matmul(ctypes.byref(cx), ctypes.byref(cw), m, n, k, po, experts, out.data_ptr(),
                                  DTYPES[out.dtype], ys, _stream()))
    return out


@_on_stream
def nvfp4_linear(x, w, offsets=None, dtype=None, out=None):
    """y = x w^T for activations x [m, k] (float32, bfloat16 or float16): x is
    quantised with a scale per row, so that a row's result does not depend on
    the rows beside it, then multiplied as in nvfp4_matmul.  dtype defaults to
    x's type."""
    q, _ = nvfp4_quantize(x, per_row=True)
    return nvfp4_matmul(q, w, offsets, x.dtype if dtype is None else dtype, out)


@_on_stream
def policy_loss(logits, tokens, old_logp, advantages, weights, ref_logp=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                temperature=1.0, grad=True):
    """dcr_policy_loss.  logits [rows, vocab]; tokens int64 [rows]; old_logp,
    advantages, weights and ref_logp float32 [rows].  A row of weight 0 is left
    out; the weights carry the normalisation (1 / number of tokens, say).

    grad: True to make the gradient, False to leave it out, or a tensor to
    write it to (logits itself, to save the memory).  Returns (loss, logp,
    grad): a float32 scalar, float32 [rows], and the gradient by the logits in
    their type (or None), ready for logits.backward(grad)."""
    rows, vocab, stride = _matrix(logits, "logits")
    dev = logits.device
    f32 = torch.float32
    ptrs = [_flat(tokens, rows, torch.int64, "tokens", dev), _flat(old_logp, rows, f32, "old_logp", dev),
            None if ref_logp is None else _flat(ref_logp, rows, f32, "ref_logp", dev),
            _flat(advantages, rows, f32, "advantages", dev), _flat(weights, rows, f32, "weights", dev)]
    gs = 0
    if grad is True:
        grad = torch.empty((rows, vocab), dtype=logits.dtype, device=dev)
        gs = vocab
    elif grad is False or grad is None:
        grad = None
    else:
        gr, gc, gs = _matrix(grad, "grad")
        _need((gr, gc) == (rows, vocab) and grad.dtype == logits.dtype and grad.device == dev, "grad must be like logits")
    res = torch.empty(2 * rows + 1, dtype=f32, device=dev)
    loss, logp = res[2 * rows], res[:rows]
    base = res.data_ptr()
    opts = PolicyOpts(temperature, clip_low, clip_high, kl_coef)
    check(_lib().dcr_policy_loss(logits.data_ptr(), DTYPES[logits.dtype], rows, vocab, stride, *ptrs,
                                 ctypes.byref(opts), base + 8 * rows, base + 4 * rows, base,
                                 grad.data_ptr() if grad is not None else None, gs, _stream()))
    return loss, logp, grad


@_on_stream
def token_logprobs(logits, tokens, temperature=1.0, out=None):
    """dcr_token_logprobs: float32 [rows], the log-probability of each row's
    token under softmax(logits / temperature)."""
    rows, vocab, stride = _matrix(logits, "logits")
    dev = logits.device
    pt = _flat(tokens, rows, torch.int64, "tokens", dev)
    out = _out(out, (rows,), torch.float32, "out", dev)
    check(_lib().dcr_token_logprobs(logits.data_ptr(), DTYPES[logits.dtype], rows, vocab, stride, pt, temperature,
                                    out.data_ptr(), _stream()))
    return out


def ops_status(stream=None):
    """dcr_ops_status: waits for the stream and raises DcrError (TIMEOUT) if an
    operator gave up a wait on the device since the last call."""
    check(_lib().dcr_ops_status(_stream() if stream is None else getattr(stream, "cuda_stream", stream)))
