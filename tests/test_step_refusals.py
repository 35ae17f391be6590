"""Arguments that the operators of a step refuse (token scores, routing, rows
by expert, AdamW), at the C entries and in the binding, before anything is
launched (so on a machine without a GPU)."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

import bit_exact_xor_gb300 as dcr  # noqa: E402
from bit_exact_xor_gb300 import adamw, experts, ops, scores  # noqa: E402

P = 4096   # a well-aligned address that no refused call reads


def _scores(x=P, dtype=1, rows=4, vocab=10, stride=10, tokens=P, temp=1.0, top=2, logp=P, entropy=P, tl=P, tt=P, stats=P):
    return scores._library().dcr_token_scores(x, dtype, rows, vocab, stride, tokens, temp, top, logp, entropy, tl, tt, stats, None)


@pytest.mark.parametrize("kw,why", [
    (dict(dtype=3), "unknown dtype"), (dict(vocab=0), "vocab"), (dict(vocab=1 << 31, stride=1 << 31), "vocab"), (dict(rows=1 << 28), "rows"),
    (dict(stride=9), "row_stride"), (dict(stride=1 << 40), "vocab"), (dict(x=None), "NULL"), (dict(tokens=None), "NULL"), (dict(tl=None), "NULL"),
    (dict(tt=None), "NULL"), (dict(top=65, vocab=100, stride=100), "top"), (dict(top=11), "top"), (dict(temp=0.0), "temperature"),
    (dict(temp=-1.0), "temperature"), (dict(temp=float("nan")), "temperature"), (dict(temp=float("inf")), "temperature"), (dict(x=P + 1), "misaligned"),
    (dict(tokens=P + 4), "misaligned"), (dict(logp=P + 2), "misaligned"), (dict(entropy=P + 1), "misaligned"), (dict(tl=P + 2), "misaligned"),
    (dict(tt=P + 4), "misaligned"), (dict(stats=P + 2), "misaligned")])
def test_token_scores(kw, why):
    assert _scores(**kw) == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()


def _scores_grad(x=P, dtype=1, rows=4, vocab=10, stride=10, tokens=P, stats=P, gl=P, ge=P, temp=1.0, grad=2 * P, gs=10):
    return scores._library().dcr_token_scores_grad(x, dtype, rows, vocab, stride, tokens, stats, gl, ge, temp, grad, gs, None)


@pytest.mark.parametrize("kw,why", [
    (dict(dtype=3), "unknown dtype"), (dict(stats=None), "NULL"), (dict(grad=None), "NULL"), (dict(gs=9), "grad_stride"),
    (dict(grad=P, gs=12), "same stride"), (dict(grad=P + 1), "misaligned"), (dict(stats=P + 2), "misaligned"), (dict(gl=P + 2), "misaligned"),
    (dict(ge=P + 2), "misaligned"), (dict(temp=0.0), "temperature")])
def test_token_scores_grad(kw, why):
    assert _scores_grad(**kw) == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()


def test_nothing_to_score_is_valid():
    assert _scores(rows=0, x=None, tokens=None, tl=None, tt=None) == dcr.OK
    assert _scores(top=0, logp=None, entropy=None, stats=None) == dcr.OK
    assert _scores_grad(rows=0, x=None, tokens=None, stats=None, grad=None) == dcr.OK


def _route(x=P, dtype=1, tokens=4, n=8, stride=8, bias=P, mask=P, opts=(0, 2, 2, 1, 2, 1, 1.0), chosen=P, weights=P, offsets=P, order=P, positions=P,
           work=P):
    o = ctypes.byref(experts._RouteOpts(*opts)) if opts else None
    return experts._library().dcr_route(x, dtype, tokens, n, stride, bias, mask, o, chosen, weights, offsets, order, positions, work, None)


@pytest.mark.parametrize("kw,why", [
    (dict(opts=None), "NULL"), (dict(dtype=3), "unknown dtype"), (dict(n=0), "experts"), (dict(n=1025, stride=1025), "experts"),
    (dict(opts=(2, 2, 1, 1, 1, 1, 1.0)), "scoring"), (dict(opts=(0, 0, 1, 1, 1, 1, 1.0)), "k must"), (dict(opts=(0, 9, 1, 1, 1, 1, 1.0)), "k must"),
    (dict(n=64, stride=64, opts=(0, 33, 1, 1, 1, 1, 1.0)), "k must"), (dict(opts=(0, 2, 0, 1, 1, 1, 1.0)), "groups"),
    (dict(opts=(0, 2, 3, 1, 1, 1, 1.0)), "groups"), (dict(n=66, stride=66, opts=(0, 2, 33, 1, 1, 1, 1.0)), "groups"),
    (dict(opts=(0, 2, 2, 0, 1, 1, 1.0)), "group_top"), (dict(opts=(0, 2, 2, 3, 1, 1, 1.0)), "group_top"), (dict(opts=(0, 2, 2, 1, 3, 1, 1.0)), "group_by"),
    (dict(opts=(0, 2, 2, 1, 0, 1, 1.0)), "group_by"), (dict(opts=(0, 3, 4, 1, 1, 1, 1.0)), "fewer than k"), (dict(opts=(0, 2, 1, 1, 1, 1, float("nan"))), "scale"),
    (dict(tokens=1 << 30), "2^31"), (dict(stride=7), "row_stride"), (dict(x=None), "NULL"), (dict(chosen=None), "NULL"), (dict(weights=None), "NULL"),
    (dict(offsets=None), "NULL"), (dict(order=None), "NULL"), (dict(positions=None), "NULL"), (dict(work=None), "NULL"), (dict(x=P + 1), "misaligned"),
    (dict(bias=P + 2), "misaligned"), (dict(chosen=P + 2), "misaligned"), (dict(weights=P + 2), "misaligned"), (dict(offsets=P + 2), "misaligned"),
    (dict(order=P + 2), "misaligned"), (dict(positions=P + 2), "misaligned"), (dict(work=P + 2), "misaligned")])
def test_route(kw, why):
    assert _route(**kw) == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()


def _route_grad(x=P, dtype=1, tokens=4, n=8, stride=8, chosen=P, gw=P, opts=(0, 2, 1, 1, 1, 1, 1.0), grad=2 * P, gs=8):
    o = ctypes.byref(experts._RouteOpts(*opts)) if opts else None
    return experts._library().dcr_route_grad(x, dtype, tokens, n, stride, chosen, gw, o, grad, gs, None)


@pytest.mark.parametrize("kw,why", [
    (dict(opts=None), "NULL"), (dict(n=1025, stride=1025), "experts"), (dict(x=None), "NULL"), (dict(chosen=None), "NULL"), (dict(gw=None), "NULL"),
    (dict(grad=None), "NULL"), (dict(gs=7), "grad_stride"), (dict(grad=P, gs=9), "same stride"), (dict(grad=P + 1), "misaligned"),
    (dict(chosen=P + 2), "misaligned"), (dict(gw=P + 2), "misaligned")])
def test_route_grad(kw, why):
    assert _route_grad(**kw) == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()
    assert _route_grad(tokens=0, x=None, chosen=None, gw=None, grad=None) == dcr.OK


def _gather(x=P, xt=1, tokens=4, cols=8, xs=8, pos=P, k=2, w=P, out=P, dtype=1, rows=8, stride=8):
    return experts._library().dcr_experts_gather(x, xt, tokens, cols, xs, pos, k, w, out, dtype, rows, stride, None)


def _combine(y=P, yt=1, rows=8, cols=8, ys=8, pos=P, w=P, tokens=4, k=2, out=P, dtype=1, stride=8):
    return experts._library().dcr_experts_combine(y, yt, rows, cols, ys, pos, w, tokens, k, out, dtype, stride, None)


def _combine_grad(y=P, yt=1, rows=8, cols=8, ys=8, pos=P, w=P, tokens=4, k=2, g=P, dtype=1, gs=8, gy=P, gys=8, gw=P):
    return experts._library().dcr_experts_combine_grad(y, yt, rows, cols, ys, pos, w, tokens, k, g, dtype, gs, gy, gys, gw, None)


@pytest.mark.parametrize("call,kw,why", [
    (c, kw, why) for c in (_gather, _combine, _combine_grad) for kw, why in [
        (dict(dtype=3), "unknown dtype"), (dict(k=0), "k must"), (dict(k=33), "k must"), (dict(tokens=1 << 30), "2^31"), (dict(rows=1 << 31), "2^31"),
        (dict(pos=None), "NULL"), (dict(pos=P + 2), "misaligned"), (dict(w=P + 2), "misaligned")]] + [
    (_gather, dict(xt=3), "unknown dtype"), (_gather, dict(xs=7), "stride of x"), (_gather, dict(stride=7), "stride of out"), (_gather, dict(x=None), "x is NULL"),
    (_gather, dict(out=None), "out is NULL"), (_gather, dict(x=P + 1), "x is misaligned"), (_gather, dict(out=P + 1), "out is misaligned"),
    (_combine, dict(yt=3), "unknown dtype"), (_combine, dict(ys=7), "stride of y"), (_combine, dict(stride=7), "stride of out"), (_combine, dict(y=None), "y is NULL"),
    (_combine, dict(out=None), "out is NULL"), (_combine, dict(y=P + 1), "y is misaligned"), (_combine_grad, dict(g=None), "grad is NULL"),
    (_combine_grad, dict(gs=7), "stride of grad"), (_combine_grad, dict(gys=7), "stride of grad_y"), (_combine_grad, dict(y=None), "y is NULL"),
    (_combine_grad, dict(gy=P + 1), "grad_y is misaligned"), (_combine_grad, dict(gw=P + 2), "misaligned")])
def test_exchange(call, kw, why):
    assert call(**kw) == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()


def test_nothing_to_exchange_is_valid():
    assert _gather(tokens=0, x=None, pos=None, rows=0, out=None) == dcr.OK
    assert _gather(cols=0, x=None, out=None) == dcr.OK
    assert _combine(tokens=0, pos=None, out=None) == dcr.OK
    assert _combine_grad(tokens=0, pos=None, g=None) == dcr.OK
    assert _combine_grad(gy=None, gw=None) == dcr.OK


def _norm(t=((P, 8),), dtype=1, work=P, norm=P):
    table = (adamw._Grad * max(1, len(t)))(*t)
    return adamw._library().dcr_grad_norm(table, len(t), dtype, work, norm, None)


@pytest.mark.parametrize("kw,why", [
    (dict(dtype=3), "unknown dtype"), (dict(work=None), "NULL"), (dict(norm=None), "NULL"), (dict(work=P + 4), "misaligned"), (dict(norm=P + 2), "misaligned"),
    (dict(t=((None, 8),)), "NULL"), (dict(t=((P, 8), (P + 1, 8))), "misaligned"), (dict(t=((P, 1 << 40),)), "too large")])
def test_norm(kw, why):
    assert _norm(**kw) == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()


M = 1 << 20


def _adamw(t=None, count=None, w=0, g=1, c=3, bits=32, **kw):
    t = t or [dict()]
    table = (adamw._Tensor * len(t))()
    for i, (e, x) in enumerate(zip(table, t)):
        base = dict(w=M, grad=2 * M, m=3 * M, v=4 * M, m_scale=5 * M, v_scale=6 * M, copy=7 * M if c != 3 else None, n=64)
        for name, value in dict(base, **x).items():
            setattr(e, name, value)
    o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, grad_scale=1.0, max_norm=0.0, step=1, state_bits=bits)
    return adamw._library().dcr_adamw(table, len(t), w, g, c, ctypes.byref(adamw._Opts(**dict(o, **kw))), None)


nan, inf = float("nan"), float("inf")


@pytest.mark.parametrize("kw,why", [
    (dict(w=3), "unknown dtype"), (dict(g=3), "unknown dtype"), (dict(c=4), "unknown dtype"), (dict(bits=16), "state_bits"), (dict(beta1=1.0), "betas"),
    (dict(beta1=-0.1), "betas"), (dict(beta2=nan), "betas"), (dict(lr=nan), "lr"), (dict(lr=-1.0), "lr"), (dict(eps=inf), "eps"), (dict(lr=1e39), "lr"), (dict(grad_scale=1e39), "grad_scale"), (dict(weight_decay=-1.0), "weight_decay"),
    (dict(grad_scale=inf), "grad_scale"), (dict(max_norm=1.0), "max_norm"), (dict(max_norm=nan, norm=P), "max_norm"), (dict(step=0), "step"),
    (dict(norm=P + 2), "misaligned"), (dict(device_step=P + 4), "misaligned"), (dict(device_lr=P + 2), "misaligned"),
    (dict(t=[dict(w=None)]), "NULL"), (dict(t=[dict(grad=None)]), "NULL"), (dict(t=[dict(m=None)]), "NULL"), (dict(t=[dict(v=None)]), "NULL"),
    (dict(bits=8, t=[dict(m_scale=None)]), "NULL"), (dict(bits=8, t=[dict(v_scale=None)]), "NULL"), (dict(c=1, t=[dict(copy=None)]), "NULL"),
    (dict(t=[dict(w=M + 2)]), "misaligned"), (dict(t=[dict(grad=2 * M + 1)]), "misaligned"), (dict(t=[dict(m=3 * M + 2)]), "misaligned"),
    (dict(bits=8, t=[dict(v_scale=M * 6 + 2)]), "misaligned"), (dict(t=[dict(n=1 << 40)]), "too large"),
    # the same tensor twice, moments of two tensors that overlap, a copy over the weights, a gradient that a copy is written over
    (dict(t=[dict(), dict()]), "overlap"), (dict(t=[dict(), dict(w=8 * M, v=9 * M, m=3 * M + 4 * 63)]), "overlap"),
    (dict(c=1, t=[dict(copy=M + 4 * 64 - 2)]), "overlap"), (dict(c=1, t=[dict(copy=2 * M + 2)]), "overlap"), (dict(t=[dict(m=4 * M)]), "overlap"),
    (dict(bits=8, t=[dict(m_scale=6 * M)]), "overlap")])
def test_adamw(kw, why):
    assert _adamw(**kw) == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()


def test_a_step_over_nothing_is_valid():
    assert adamw._library().dcr_adamw(None, 0, 0, 0, 3, ctypes.byref(adamw._Opts(lr=1e-3, step=1, state_bits=32)), None) == dcr.OK
    assert _adamw(t=[dict(n=0, w=None, grad=None, m=None, v=None)]) == dcr.OK
    assert adamw._library().dcr_adamw(None, 0, 0, 0, 3, None, None) == dcr.ERR_INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, t = torch.zeros(4, 32), torch.zeros(4, dtype=torch.int64)
    r = dcr.Route(*[torch.zeros(4, 2, dtype=torch.int32)] * 5)
    for call in (lambda: dcr.token_scores(x, t), lambda: dcr.token_scores_grad(x, t, x), lambda: dcr.route_experts(x, 2),
                 lambda: dcr.route_experts_grad(x, r, x), lambda: dcr.experts_gather(x, r), lambda: dcr.experts_combine(x, r),
                 lambda: dcr.experts_combine_grad(x, r, x), lambda: dcr.grad_norm([x]), lambda: dcr.grad_norm([]), lambda: dcr.adamw_states([x], 16),
                 lambda: dcr.adamw_step([x], [x], [dcr.AdamState32(x, x)], 1, 1e-3),
                 lambda: dcr.adamw_step([x], [x], [dcr.AdamState32(x, x)], 1, 1e-3, norm=x, max_norm=0.0), lambda: dcr.adamw_step([], [], [], 1, 1e-3)):
        with pytest.raises(dcr.DcrError) as e:
            call()
        assert e.value.code == dcr.ERR_INVALID


def test_header_constants():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(os.path.dirname(ops.__file__), "..", "include", "dcr_ops.h")).read(), flags=re.S)
    for module, names in ((scores, ["MAX_TOP"]), (experts, ["MAX_CHOSEN", "MAX_GROUPS", "ROUTE_PARTS"]), (adamw, ["ADAMW_BLOCK", "NORM_WORKSPACE"])):
        for n in names:
            assert int(re.search(r"DCR_%s (\d+)u" % n, src).group(1)) == getattr(module, n)
    assert "#define DCR_ROUTE_WORKSPACE(experts) (16ull * DCR_ROUTE_PARTS * (((experts) + 3) / 4))" in src


def test_no_block_reaches_into_another_before_the_cluster_runs():
    # every write to another block's shared memory comes behind a wait of the cluster's barrier, and another one follows it
    src = open(os.path.join(os.path.dirname(ops.__file__), "csrc", "token_scores.cu")).read()
    body = re.sub(r"//[^\n]*", "", src).split("scores_kernel(ScoreArgs A, uint32_t cluster)", 1)[1]
    first, last = body.index("to_first("), body.rindex("to_first(")
    assert body.index("barrier.cluster.arrive.relaxed") < body.index("barrier.cluster.wait.acquire") < first
    assert "barrier.cluster.arrive.release;\\nbarrier.cluster.wait.acquire" in body[last:]
