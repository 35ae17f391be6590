"""Scores of given tokens (include/dcr_ops.h): log-probabilities, entropies,
likeliest alternatives, and the gradient of the first two.  Argument
marshalling only, by the same rules as ops.py."""
import ctypes
from typing import NamedTuple, Optional

import torch

from . import OK, check
from .ops import _elsewhere, _fast, _flat, _lib, _matrix, _raw_stream, _refuse, _result_of

MAX_TOP = 64
_f32 = torch.float32


class TokenScores(NamedTuple):
    """logp and entropy, float32 [rows]; top_logp float32 and top_tokens int64
    [rows, top], the likeliest first (None without alternatives); stats float32
    [rows, 3], which token_scores_grad takes."""
    logp: torch.Tensor
    entropy: torch.Tensor
    top_logp: Optional[torch.Tensor]
    top_tokens: Optional[torch.Tensor]
    stats: torch.Tensor


_ops = None


def _library():
    global _ops
    if _ops is None:
        L = _lib()
        VP, U32, U64, F = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float
        L.dcr_token_scores.argtypes = [VP, U32, U64, U64, U64, VP, F, U32, VP, VP, VP, VP, VP, VP]
        L.dcr_token_scores_grad.argtypes = [VP, U32, U64, U64, U64, VP, VP, VP, VP, F, VP, U64, VP]
        _ops = L
    return _ops


def token_scores(logits, tokens, top=0, temperature=1.0, stream=None):
    """dcr_token_scores of logits [rows, vocab] (float32, bfloat16 or float16)
    and tokens int64 [rows]: a TokenScores under softmax(logits / temperature).
    A row whose token lies outside [0, vocab) is left out (zeros, alternatives
    -1)."""
    if stream is None:
        r = _fast.scores(logits, tokens, top, temperature)
        if r is not None:
            return TokenScores(*_result_of(r))
    rows, vocab, stride, t = _matrix(logits, "logits")
    dev = logits.device
    if stream is not None or dev.index != torch.cuda.current_device():
        return _elsewhere(token_scores, dev, stream, logits, tokens, top, temperature)
    if not 0 <= top <= min(MAX_TOP, vocab):
        _refuse("top must be at most %d and the number of logits of a row" % MAX_TOP)
    pt = _flat(tokens, rows, torch.int64, "tokens", dev)
    logp, entropy = torch.empty(rows, dtype=_f32, device=dev), torch.empty(rows, dtype=_f32, device=dev)
    stats = torch.empty((rows, 3), dtype=_f32, device=dev)
    top_logp = top_tokens = None
    if top:
        top_logp, top_tokens = torch.empty((rows, top), dtype=_f32, device=dev), torch.empty((rows, top), dtype=torch.int64, device=dev)
    rc = _library().dcr_token_scores(logits.data_ptr(), t, rows, vocab, stride, pt, temperature, top, logp.data_ptr(), entropy.data_ptr(),
                                     top_logp.data_ptr() if top else None, top_tokens.data_ptr() if top else None, stats.data_ptr(),
                                     _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return TokenScores(logp, entropy, top_logp, top_tokens, stats)


def token_scores_grad(logits, tokens, stats, grad_logp=None, grad_entropy=None, temperature=1.0, out=None, stream=None):
    """dcr_token_scores_grad: the gradient by the logits, in their type, of a
    loss whose derivatives by token_scores' logp and entropy are grad_logp and
    grad_entropy (float32 [rows], either may be None).  stats and temperature
    are that call's; out: a matrix to write to (logits itself, to save the
    memory)."""
    if stream is None and out is None:
        r = _fast.scores_grad(logits, tokens, stats, grad_logp, grad_entropy, temperature)
        if r is not None:
            return _result_of(r)
    rows, vocab, stride, t = _matrix(logits, "logits")
    dev = logits.device
    if stream is not None or dev.index != torch.cuda.current_device():
        return _elsewhere(token_scores_grad, dev, stream, logits, tokens, stats, grad_logp, grad_entropy, temperature, out)
    pt = _flat(tokens, rows, torch.int64, "tokens", dev)
    ps = _flat(stats, rows * 3, _f32, "stats", dev)
    pl = None if grad_logp is None else _flat(grad_logp, rows, _f32, "grad_logp", dev)
    pe = None if grad_entropy is None else _flat(grad_entropy, rows, _f32, "grad_entropy", dev)
    if out is None:
        out, gs = torch.empty((rows, vocab), dtype=logits.dtype, device=dev), vocab
    else:
        gr, gc, gs, gt = _matrix(out, "out")
        if (gr, gc, gt) != (rows, vocab, t) or out.device != dev:
            _refuse("out must be like logits")
    rc = _library().dcr_token_scores_grad(logits.data_ptr(), t, rows, vocab, stride, pt, ps, pl, pe, temperature, out.data_ptr(), gs,
                                          _raw_stream(dev.index))
    if rc != OK:
        check(rc)
    return out
