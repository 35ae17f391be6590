"""Arguments that the operators refuse, at the C entries and in the binding,
before anything is launched (so on a machine without a GPU)."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

import bit_exact_xor_gb300 as dcr  # noqa: E402
from bit_exact_xor_gb300 import ops  # noqa: E402

P = 4096   # a well-aligned address that no refused call reads


def _quant(x=P, dtype=0, rows=2, cols=32, stride=32, mode=1, scale=P, codes=P, scales=P, values=None, vt=3, work=P):
    return ops._lib().dcr_nvfp4_quantize(x, dtype, rows, cols, stride, mode, scale, codes, scales, values, vt, work, None)


@pytest.mark.parametrize("kw,why", [
    (dict(dtype=3), "unknown dtype"), (dict(mode=3), "scale mode"), (dict(cols=24), "multiple of 16"),
    (dict(stride=16), "row_stride"), (dict(values=P), "values"), (dict(vt=1), "values"), (dict(x=None), "NULL"),
    (dict(scale=None), "NULL"), (dict(work=None), "NULL"), (dict(work=P + 2), "misaligned"), (dict(codes=None), "NULL"), (dict(scales=None), "NULL"), (dict(codes=P + 8), "misaligned"),
    (dict(values=P + 2, vt=1), "misaligned"), (dict(x=P + 2), "misaligned"), (dict(scale=P + 1), "misaligned"),
    (dict(rows=1 << 32), "too large"), (dict(cols=1 << 32, stride=1 << 32), "too large"),
])
def test_quantise(kw, why):
    assert _quant(**kw) == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()


def test_quantise_of_nothing_is_valid():
    assert _quant(rows=0, x=None, codes=None, scales=None) == dcr.OK
    assert _quant(cols=0, x=None) == dcr.OK


def _mat(codes=P, scales=P, scale=P, count=1):
    return ops._Nvfp4(codes, scales, scale, count)


def _matmul(x=None, w=None, m=4, n=8, k=64, offsets=None, experts=0, y=P, dtype=1, stride=8):
    x, w = x or _mat(), w or _mat()
    return ops._lib().dcr_nvfp4_matmul(ctypes.byref(x), ctypes.byref(w), m, n, k, offsets, experts, y, dtype, stride, None)


@pytest.mark.parametrize("kw,why", [
    (dict(dtype=3), "unknown dtype"), (dict(k=0), "multiple of 32"), (dict(k=48), "multiple of 32"),
    (dict(experts=1025, offsets=P), "experts"), (dict(experts=2), "offsets"), (dict(offsets=P), "offsets"),
    (dict(stride=7), "y_stride"), (dict(x=_mat(count=3)), "x needs"), (dict(w=_mat(count=4)), "w needs"),
    (dict(w=_mat(count=0)), "w needs"), (dict(x=_mat(codes=None)), "NULL"), (dict(w=_mat(scales=None)), "NULL"),
    (dict(x=_mat(scale=None)), "NULL"), (dict(y=None), "NULL"), (dict(x=_mat(codes=P + 8)), "misaligned"),
    (dict(w=_mat(codes=P + 4)), "misaligned"), (dict(y=P + 1), "misaligned"), (dict(m=1 << 31), "too large"),
    (dict(n=1 << 30, experts=4, offsets=P, stride=1 << 30), "too large"), (dict(k=1 << 31), "too large"),
    (dict(x=_mat(scale=P + 2)), "misaligned"), (dict(offsets=P + 2, experts=1), "misaligned"),
])
def test_matmul(kw, why):
    assert _matmul(**kw) == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()


def test_matmul_null_and_nothing():
    assert ops._lib().dcr_nvfp4_matmul(None, None, 1, 1, 32, None, 0, P, 0, 1, None) == dcr.ERR_INVALID
    assert _matmul(m=0, x=_mat(None, None, P, 1), y=None) == dcr.OK
    assert _matmul(n=0, w=_mat(None, None, P, 1), y=None, stride=0) == dcr.OK


def _linear(x=P, xdt=1, xs=64, w=None, m=4, n=8, k=64, offsets=None, experts=0, y=P, dtype=1, stride=8, work=P):
    w = w or _mat()
    return ops._lib().dcr_nvfp4_linear(x, xdt, xs, ctypes.byref(w), m, n, k, offsets, experts, y, dtype, stride, work, None)


@pytest.mark.parametrize("kw,why", [
    (dict(xdt=3), "unknown dtype"), (dict(dtype=4), "unknown dtype"), (dict(k=48), "multiple of 32"), (dict(xs=63), "x_stride"),
    (dict(x=None), "NULL"), (dict(work=None), "NULL"), (dict(w=_mat(codes=None)), "NULL"), (dict(work=P + 8), "misaligned"),
    (dict(x=P + 1), "misaligned"), (dict(w=_mat(codes=P + 8)), "misaligned"), (dict(experts=1), "offsets"),
    (dict(stride=7), "y_stride"), (dict(w=_mat(count=2)), "w needs"), (dict(n=1 << 31, stride=1 << 31), "too large"),
])
def test_linear(kw, why):
    assert _linear(**kw) == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()
    assert _linear(m=0, x=None, y=None, work=None) == dcr.OK


def _loss(logits=P, dtype=1, rows=4, vocab=10, stride=10, tokens=P, old=P, ref=P, adv=P, w=P, opts=(1.0, 0.2, 0.2, 0.1),
          loss=P, row_loss=P, logp=P, grad=2 * P, gstride=10):
    o = ctypes.byref(ops.PolicyOpts(*opts)) if opts else None
    return ops._lib().dcr_policy_loss(logits, dtype, rows, vocab, stride, tokens, old, ref, adv, w, o, loss, row_loss, logp,
                                      grad, gstride, None)


@pytest.mark.parametrize("kw,why", [
    (dict(dtype=7), "unknown dtype"), (dict(vocab=0), "vocab"), (dict(stride=9), "row_stride"), (dict(gstride=9), "grad_stride"),
    (dict(opts=None), "NULL"), (dict(loss=None), "NULL"), (dict(logits=None), "NULL"), (dict(tokens=None), "NULL"),
    (dict(old=None), "NULL"), (dict(adv=None), "NULL"), (dict(w=None), "NULL"), (dict(row_loss=None), "NULL"),
    (dict(logp=None), "NULL"), (dict(ref=None), "ref_logp"), (dict(opts=(0.0, 0.2, 0.2, 0.0)), "temperature"),
    (dict(opts=(-1.0, 0.2, 0.2, 0.0)), "temperature"), (dict(opts=(float("nan"), 0.2, 0.2, 0.0)), "temperature"),
    (dict(opts=(float("inf"), 0.2, 0.2, 0.0)), "temperature"), (dict(opts=(1.0, -0.1, 0.2, 0.0)), "clip_low"),
    (dict(opts=(1.0, 0.1, float("nan"), 0.0)), "clip_high"), (dict(opts=(1.0, 0.1, 0.2, -1.0)), "kl_coef"),
    (dict(grad=P, gstride=12), "same stride"), (dict(grad=P + 1), "misaligned"), (dict(logits=P + 1), "misaligned"),
    (dict(tokens=P + 4), "misaligned"), (dict(old=P + 2), "misaligned"), (dict(rows=1 << 28), "rows below"),
])
def test_policy_loss(kw, why):
    assert _loss(**kw) == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()


def test_token_logprobs():
    f = ops._lib().dcr_token_logprobs
    assert f(P, 1, 4, 0, 10, P, 1.0, P, None) == dcr.ERR_INVALID
    assert f(P, 1, 4, 10, 9, P, 1.0, P, None) == dcr.ERR_INVALID
    assert f(None, 1, 4, 10, 10, P, 1.0, P, None) == dcr.ERR_INVALID
    assert f(P, 1, 4, 10, 10, P, 0.0, P, None) == dcr.ERR_INVALID
    assert f(P, 1, 4, 10, 10, P, 1.0, P + 2, None) == dcr.ERR_INVALID
    assert f(P, 1, 0, 10, 10, None, 1.0, None, None) == dcr.OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 32)
    for call in (lambda: dcr.nvfp4_quantize(x), lambda: dcr.nvfp4_linear(x, dcr.Nvfp4(x, x, x)),
                 lambda: dcr.nvfp4_matmul(dcr.Nvfp4(x, x, x), dcr.Nvfp4(x, x, x)),
                 lambda: dcr.policy_loss(x, x, x, x, x), lambda: dcr.token_logprobs(x, x)):
        with pytest.raises(dcr.DcrError) as e:
            call()
        assert e.value.code == dcr.ERR_INVALID


def test_header_constants_and_exports():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(os.path.dirname(ops.__file__), "..", "include", "dcr_ops.h")).read(), flags=re.S)
    vals = {k: int(v) for k, v in re.findall(r"\bDCR_(\w+)\s*=\s*(\d+)", src)}
    assert vals and all(getattr(ops, k) == v for k, v in vals.items())
    assert int(re.search(r"DCR_QUANT_PARTIALS (\d+)u", src).group(1)) == ops.QUANT_PARTIALS
    assert int(re.search(r"DCR_MAX_EXPERTS (\d+)u", src).group(1)) == ops.MAX_EXPERTS
    assert int(re.search(r"DCR_TEST_STALL (0x\w+)u", src).group(1), 0) == ops.TEST_STALL
    assert "#define DCR_LINEAR_WORKSPACE(m, k) ((m) * ((k) / 2 + (k) / 16 + 4) + 4)" in src
    declared = set(re.findall(r"^int (dcr_\w+)\(", src, flags=re.M))
    assert declared == set(ops.OP_EXPORTS)
