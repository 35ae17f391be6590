"""The operators around a refit (include/dcr_ops.h): NVFP4 quantisation, the
product of NVFP4 operands, and the policy loss.  Argument marshalling only, as
in the rest of the binding; tensors that are not given are allocated with
torch, and every call runs on `stream` (default: the current stream) without
waiting for it.  What a call allocates belongs to the stream that it runs on;
tensors handed in must be ready there, and are kept by the caller until the
call has run.  A refused argument raises DcrError.

The smallest of these operators take a few microseconds on the GPU, so their
common calls (tensors on the current device, new outputs, the current stream)
go through the compiled csrc/binding.cpp; it hands back what it does not
take, refusals among it, to the code below.  Where it is missing or was built
for another torch, a warning says so and every call takes that code.
"""
import ctypes
import warnings
from typing import NamedTuple

import torch

from . import ERR_INVALID, OK, DcrError, check, lib

F32, BF16, F16, NONE = 0, 1, 2, 3
SCALE_GIVEN, SCALE_TENSOR, SCALE_ROW = 0, 1, 2
MAX_EXPERTS = 1024
QUANT_PARTIALS = 1216
TEST_STALL = 0x80000000   # test only: a product whose waits run out
DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}

OP_EXPORTS = ["dcr_nvfp4_quantize", "dcr_nvfp4_matmul", "dcr_nvfp4_linear", "dcr_policy_loss", "dcr_token_logprobs",
              "dcr_ops_status"]


class Nvfp4(NamedTuple):
    """An NVFP4 matrix: codes [rows, cols / 2] uint8 (two e2m1 values a byte,
    the even column in the low four bits), scales [rows, cols / 16] (e4m3, as
    uint8 or float8_e4m3fn) and scale, a float32 tensor with one entry, one
    per row, or (the weights of several experts) one per expert."""
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
_empty, _f32, _u8 = torch.empty, torch.float32, torch.uint8
_SCALE_TYPES = (torch.uint8, torch.float8_e4m3fn)
_byref = ctypes.byref
_TYPES = (type(None), torch.dtype)


def _lib():
    global _ops
    if _ops is None:
        L = lib()
        P, VP, U32, U64 = ctypes.POINTER, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64
        L.dcr_nvfp4_quantize.argtypes = [VP, U32, U64, U64, U64, U32, VP, VP, VP, VP, U32, VP, VP]
        L.dcr_nvfp4_matmul.argtypes = [P(_Nvfp4), P(_Nvfp4), U64, U64, U64, VP, U32, VP, U32, U64, VP]
        L.dcr_nvfp4_linear.argtypes = [VP, U32, U64, P(_Nvfp4), U64, U64, U64, VP, U32, VP, U32, U64, VP, VP]
        L.dcr_policy_loss.argtypes = [VP, U32, U64, U64, U64, VP, VP, VP, VP, VP, P(PolicyOpts), VP, VP, VP, VP, U64, VP]
        L.dcr_token_logprobs.argtypes = [VP, U32, U64, U64, U64, VP, ctypes.c_float, VP, VP]
        L.dcr_ops_status.argtypes = [VP]
        _ops = L
    return _ops


def _refuse(what):
    raise DcrError(ERR_INVALID, what)


class _NoBinding:
    """In the compiled binding's place: takes no call, so that each goes on to
    the code below and through ctypes to the same kernels."""
    quantize = linear = loss = logprobs = staticmethod(lambda *args: None)


def _binding():
    """The compiled binding if it is there and was built for this torch."""
    try:
        from . import _binding as fast
        if fast.torch_version == torch.__version__:
            return fast
        why = "it was built for torch %s" % fast.torch_version
    except (ImportError, AttributeError) as e:
        why = str(e)
    warnings.warn("the operators' compiled binding is not used (%s): calls take a few microseconds more; "
                  "__graft_entry__.build() makes it" % why)
    return _NoBinding


_fast = _binding()


def _result_of(r):
    """What _fast returned: a status is raised."""
    if type(r) is int:
        check(r)
    return r


def _matrix(x, what):
    """Rows, columns, row stride and type code of a matrix of one of DTYPES."""
    if not x.is_cuda or x.dim() != 2:
        _refuse(what + " must be a CUDA tensor with two dimensions")
    r, c = x.shape
    t = DTYPES.get(x.dtype)
    if t is None:
        _refuse(what + " must be float32, bfloat16 or float16")
    stride, one = x.stride()
    if c > 1 and one != 1:
        _refuse(what + " must be contiguous in its last dimension")
    if r <= 1:
        stride = c          # the stride of a single row says nothing
    elif stride < c:
        _refuse(what + " has overlapping rows")
    return r, c, stride, t


def _flat(x, n, dtype, what, device):
    """Address of a contiguous tensor of n entries."""
    if x.dtype != dtype or x.numel() != n or not x.is_contiguous() or x.device != device:
        _refuse("%s must be contiguous %s with %d entries, on the same device" % (what, dtype, n))
    return x.data_ptr()


def _nvfp4(a, what):
    """Rows, columns, device and C form of an Nvfp4."""
    codes, scales, scale = a
    if codes.dtype != _u8 or codes.dim() != 2 or not codes.is_cuda or not codes.is_contiguous():
        _refuse(what + ".codes must be a contiguous uint8 CUDA matrix")
    rows, half = codes.shape
    dev = codes.device
    if half == 0 or half % 16:
        _refuse(what + " must have a positive multiple of 32 columns")
    if scales.dtype not in _SCALE_TYPES or scales.numel() != rows * (half // 8) or not scales.is_contiguous() or scales.device != dev:
        _refuse("%s.scales must be contiguous uint8 or float8_e4m3fn with %d entries, on the same device" % (what, rows * (half // 8)))
    n = scale.numel()
    if scale.dtype != _f32 or not scale.is_contiguous() or scale.device != dev:
        _refuse(what + ".scale must be contiguous float32, on the same device")
    return rows, 2 * half, dev, _Nvfp4(codes.data_ptr(), scales.data_ptr(), scale.data_ptr(), n)


def _elsewhere(f, device, stream, *args):
    """f on another stream or device than the current one: both are made
    current, so that what f allocates belongs to that stream."""
    with torch.cuda.device(device):
        if stream is None:
            return f(*args)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        with torch.cuda.stream(stream):
            return f(*args)


def _current_raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# the same without the Stream object (3 us less), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_raw_stream)
_current_device = torch.cuda.current_device



def nvfp4_quantize(x, scale=None, per_row=False, values=None, out=None, stream=None):
    """dcr_nvfp4_quantize of x [rows, cols] (float32, bfloat16 or float16).

    The 32-bit scale is `scale` (one float32 value on the device) if given,
    else computed from all of x, or from each row with per_row=True.  `values`
    is a tensor [rows, cols], or a type to make one of, that receives what the
    codes stand for.  `out` is an Nvfp4 whose tensors are written (its scale
    is an output, too, unless `scale` is given), for example views of a
    trainer arena.  Returns (Nvfp4, values or None); the computed scale of an
    empty matrix is 1."""
    if out is None and stream is None:
        r = _fast.quantize(x, scale, per_row, NONE if values is None else DTYPES.get(values, -1)) if values.__class__ in _TYPES else None
        if r is not None:
            codes, scales, sc, v = _result_of(r)
            return Nvfp4(codes, scales, sc), v
    rows, cols, stride, xt = _matrix(x, "x")
    dev = x.device
    if stream is not None or dev.index != _current_device():
        return _elsewhere(nvfp4_quantize, dev, stream, x, scale, per_row, values, out)
    if cols % 16:
        _refuse("x must have a multiple of 16 columns")
    if out is None:
        codes = _empty((rows, cols // 2), dtype=_u8, device=dev)
        scales = _empty((rows, cols // 16), dtype=_u8, device=dev)
        sc = None
    else:
        codes, scales, sc = out
        _flat(codes, rows * (cols // 2), _u8, "codes", dev)
        if scales.dtype not in _SCALE_TYPES:
            _refuse("scales must be uint8 or float8_e4m3fn")
        _flat(scales, rows * (cols // 16), scales.dtype, "scales", dev)
    work = None
    if scale is not None:
        if per_row:
            _refuse("a given scale and per_row do not go together")
        _flat(scale, 1, _f32, "scale", dev)
        mode, sc = SCALE_GIVEN, scale
    else:
        n = rows if per_row else 1
        mode = SCALE_ROW if per_row else SCALE_TENSOR
        if not per_row:
            work = _empty(QUANT_PARTIALS, dtype=_f32, device=dev)
        if sc is None:
            sc = _empty(n, dtype=_f32, device=dev)
        else:
            _flat(sc, n, _f32, "scale", dev)
        if x.numel() == 0:
            sc.fill_(1.0)    # the library launches nothing
    vt = NONE
    if values is not None:
        if isinstance(values, torch.dtype):
            values = _empty((rows, cols), dtype=values, device=dev)
        else:
            _flat(values, rows * cols, values.dtype, "values", dev)
        vt = DTYPES.get(values.dtype)
        if vt is None:
            _refuse("values must be float32, bfloat16 or float16")
    rc = _lib().dcr_nvfp4_quantize(x.data_ptr(), xt, rows, cols, stride, mode, sc.data_ptr(), codes.data_ptr(),
                                   scales.data_ptr(), None if values is None else values.data_ptr(), vt,
                                   None if work is None else work.data_ptr(), _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return Nvfp4(codes, scales, sc), values


def _experts(offsets, wrows, dev):
    """Number of experts and address of their offsets."""
    if offsets is None:
        return 0, None
    e = offsets.numel() - 1
    if not 1 <= e <= MAX_EXPERTS:
        _refuse("offsets must have 2 to %d entries" % (MAX_EXPERTS + 1))
    if wrows % e:
        _refuse("w's rows must be a multiple of the number of experts")
    return e, _flat(offsets, e + 1, torch.int32, "offsets", dev)


def _result(out, m, n, dtype, dev):
    """The result, its row stride and its type code."""
    if out is None:
        t = DTYPES.get(dtype)
        if t is None:
            _refuse("dtype must be float32, bfloat16 or float16")
        return _empty((m, n), dtype=dtype, device=dev), n, t
    om, on, ys, t = _matrix(out, "out")
    if om != m or on != n or out.device != dev:
        _refuse("out must be [%d, %d] on the same device" % (m, n))
    return out, ys, t


def nvfp4_matmul(x, w, offsets=None, dtype=torch.bfloat16, out=None, stream=None):
    """dcr_nvfp4_matmul: y = x w^T of two Nvfp4 matrices, x [m, k] and w
    [n, k], in `dtype` (or into `out` [m, n]).

    offsets (int32, experts + 1 entries on the device, not decreasing): w is
    [experts * n, k], and rows offsets[e] to offsets[e + 1] of x are multiplied
    by expert e's matrix; rows that no expert has are not written."""
    m, k, dev, cx = _nvfp4(x, "x")
    wrows, wk, wdev, cw = _nvfp4(w, "w")
    if k != wk or dev != wdev:
        _refuse("x and w must have the same number of columns, and the same device")
    if stream is not None or dev.index != _current_device():
        return _elsewhere(nvfp4_matmul, dev, stream, x, w, offsets, dtype, out)
    e, po = _experts(offsets, wrows, dev)
    n = wrows // e if e else wrows
    out, ys, t = _result(out, m, n, dtype, dev)
    rc = _lib().dcr_nvfp4_matmul(_byref(cx), _byref(cw), m, n, k, po, e, out.data_ptr(), t, ys, _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return out


def nvfp4_linear(x, w, offsets=None, dtype=None, out=None, stream=None):
    """dcr_nvfp4_linear: y = x w^T for activations x [m, k] (float32, bfloat16
    or float16), which are quantised with a scale per row, so that a row's
    codes do not depend on the rows beside it, then multiplied as in
    nvfp4_matmul.  dtype defaults to x's type."""
    if out is None and stream is None:
        t = DTYPES.get(x.dtype if dtype is None else dtype)
        r = None if t is None else _fast.linear(x, *w, offsets, t)
        if r is not None:
            return _result_of(r)
    m, k, xs, xt = _matrix(x, "x")
    wrows, wk, dev, cw = _nvfp4(w, "w")
    if k != wk or x.device != dev:
        _refuse("x and w must have the same number of columns, and the same device")
    if stream is not None or dev.index != _current_device():
        return _elsewhere(nvfp4_linear, dev, stream, x, w, offsets, dtype, out)
    e, po = _experts(offsets, wrows, dev)
    n = wrows // e if e else wrows
    out, ys, t = _result(out, m, n, x.dtype if dtype is None else dtype, dev)
    work = _empty(m * (k // 2 + k // 16 + 4) + 4, dtype=_u8, device=dev)
    rc = _lib().dcr_nvfp4_linear(x.data_ptr(), xt, xs, _byref(cw), m, n, k, po, e, out.data_ptr(), t, ys, work.data_ptr(),
                                 _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return out


def policy_loss(logits, tokens, old_logp, advantages, weights, ref_logp=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                temperature=1.0, grad=True, stream=None):
    """dcr_policy_loss.  logits [rows, vocab]; tokens int64 [rows]; old_logp,
    advantages, weights and ref_logp float32 [rows].  A row of weight 0 is left
    out; the weights carry the normalisation (1 / number of tokens, say).

    grad: True to make the gradient, False to leave it out, or a tensor to
    write it to (logits itself, to save the memory).  Returns (loss, logp,
    grad): a float32 scalar, float32 [rows], and the gradient by the logits in
    their type (or None), ready for logits.backward(grad)."""
    if stream is None and grad.__class__ is bool:
        r = _fast.loss(logits, tokens, old_logp, advantages, weights, ref_logp, clip_low, clip_high, kl_coef, temperature, grad)
        if r is not None:
            return _result_of(r)
    rows, vocab, stride, t = _matrix(logits, "logits")
    dev = logits.device
    if stream is not None or dev.index != _current_device():
        return _elsewhere(policy_loss, dev, stream, logits, tokens, old_logp, advantages, weights, ref_logp, clip_low, clip_high,
                          kl_coef, temperature, grad)
    pt = _flat(tokens, rows, torch.int64, "tokens", dev)
    po = _flat(old_logp, rows, _f32, "old_logp", dev)
    pr = None if ref_logp is None else _flat(ref_logp, rows, _f32, "ref_logp", dev)
    pa = _flat(advantages, rows, _f32, "advantages", dev)
    pw = _flat(weights, rows, _f32, "weights", dev)
    gs = 0
    if grad is True:
        grad = _empty((rows, vocab), dtype=logits.dtype, device=dev)
        gs = vocab
    elif grad is False or grad is None:
        grad = None
    else:
        gr, gc, gs, gt = _matrix(grad, "grad")
        if (gr, gc, gt) != (rows, vocab, t) or grad.device != dev:
            _refuse("grad must be like logits")
    loss = _empty((), dtype=_f32, device=dev)
    logp = _empty(rows, dtype=_f32, device=dev)
    work = _empty(rows, dtype=_f32, device=dev)
    rc = _lib().dcr_policy_loss(logits.data_ptr(), t, rows, vocab, stride, pt, po, pr, pa, pw,
                                _byref(PolicyOpts(temperature, clip_low, clip_high, kl_coef)), loss.data_ptr(), work.data_ptr(),
                                logp.data_ptr(), None if grad is None else grad.data_ptr(), gs, _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return loss, logp, grad


def token_logprobs(logits, tokens, temperature=1.0, out=None, stream=None):
    """dcr_token_logprobs: float32 [rows], the log-probability of each row's
    token under softmax(logits / temperature)."""
    if out is None and stream is None:
        r = _fast.logprobs(logits, tokens, temperature)
        if r is not None:
            return _result_of(r)
    rows, vocab, stride, t = _matrix(logits, "logits")
    dev = logits.device
    if stream is not None or dev.index != _current_device():
        return _elsewhere(token_logprobs, dev, stream, logits, tokens, temperature, out)
    pt = _flat(tokens, rows, torch.int64, "tokens", dev)
    if out is None:
        out = _empty(rows, dtype=_f32, device=dev)
    else:
        _flat(out, rows, _f32, "out", dev)
    rc = _lib().dcr_token_logprobs(logits.data_ptr(), t, rows, vocab, stride, pt, temperature, out.data_ptr(),
                                   _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return out


def ops_status(stream=None):
    """dcr_ops_status: waits for the stream (default: the current one) and
    raises DcrError (TIMEOUT) if an operator gave up a wait on the current
    device since the last call."""
    if stream is None:
        stream = torch.cuda.current_stream()
    check(_lib().dcr_ops_status(getattr(stream, "cuda_stream", stream)))
