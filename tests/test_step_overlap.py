"""Operands that overlap: which do, against every byte of them, and which calls
of a step's operators are refused for it (before anything is launched)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

import bit_exact_xor_gb300 as dcr  # noqa: E402
from bit_exact_xor_gb300 import adamw, experts, scores  # noqa: E402

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_exact_xor_gb300", "csrc")
SOURCE = """
#include "overlap.h"
int dcr::set_error(int code, const char*, ...) { return code; }
extern "C" int meet(const uint64_t* a, const uint64_t* b)
{
    using dcr::Memory;
    return dcr::overlap(Memory("a", (const void*)a[0], uint32_t(a[1]), a[2], a[3], a[4]), Memory("b", (const void*)b[0], uint32_t(b[1]), b[2], b[3], b[4]));
}
"""


def _bytes(at, size, rows, cols, stride):
    return {at + (r * stride + c) * size + b for r in range(rows) for c in range(cols) for b in range(size)} if at else set()


def test_overlap_of_matrices(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    src, lib = tmp_path / "o.cpp", tmp_path / "o.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    meet = ctypes.CDLL(str(lib)).meet
    rng = random.Random(1)
    seen = [0, 0]

    def one(steps):
        cols = rng.randint(0, 6)
        return (rng.choice([0, 1, 1, 1]) * 2 * rng.randint(20, 60), rng.choice([1, 2, 4]), rng.randint(0, 7), cols, max(1, cols, rng.choice(steps)))

    for i in range(20000):
        steps = [rng.randint(1, 16)] if i % 2 else range(1, 17)
        a, b = one(steps), one(steps)
        exp = bool(_bytes(*a) & _bytes(*b))
        assert bool(meet((ctypes.c_uint64 * 5)(*a), (ctypes.c_uint64 * 5)(*b))) == exp, (a, b)
        seen[exp] += 1
    assert min(seen) > 2000, seen
    far = (4096, 4, 2 ** 31 - 1, 5, 2 ** 40 - 1)        # whose end no address reaches
    assert meet((ctypes.c_uint64 * 5)(*far), (ctypes.c_uint64 * 5)(4100, 4, 1, 1, 1)) and not meet((ctypes.c_uint64 * 5)(*far), (ctypes.c_uint64 * 5)(4116, 4, 1, 1, 1))


M = 1 << 20     # addresses that no refused call reads, far apart
A = [i * M for i in range(1, 16)]


def _refused(rc, why):
    assert rc == dcr.ERR_INVALID
    assert why in dcr.last_error(), dcr.last_error()


def _gather(x=A[0], cols=8, xs=8, pos=A[1], w=A[2], out=A[3], rows=8, stride=8):
    return experts._library().dcr_experts_gather(x, 1, 4, cols, xs, pos, 2, w, out, 1, rows, stride, None)


def _combine(y=A[0], cols=8, ys=8, pos=A[1], w=A[2], out=A[3], stride=8):
    return experts._library().dcr_experts_combine(y, 1, 8, cols, ys, pos, w, 4, 2, out, 1, stride, None)


def _combine_grad(y=A[0], ys=8, pos=A[1], w=A[2], g=A[3], gs=8, gy=A[4], gys=8, gw=A[5]):
    return experts._library().dcr_experts_combine_grad(y, 1, 8, 8, ys, pos, w, 4, 2, g, 1, gs, gy, gys, gw, None)


@pytest.mark.parametrize("call,kw,why", [
    (_gather, dict(out=A[0]), "out overlaps x"), (_gather, dict(out=A[0] - 2 * 8 * 8 + 2), "out overlaps x"), (_gather, dict(out=A[0] + 2 * 8 * 4 - 2), "out overlaps x"),
    # columns of one buffer, the last of the one the first of the other
    (_gather, dict(xs=15, stride=15, out=A[0] + 14), "out overlaps x"), (_gather, dict(xs=15, stride=15, out=A[0] - 14), "out overlaps x"),
    (_gather, dict(xs=24, stride=31, out=A[0] + 32), "out overlaps x"),
    (_gather, dict(out=A[1] + 16), "out overlaps positions"), (_gather, dict(out=A[2] + 16), "out overlaps weights"), (_gather, dict(pos=A[3] + 124), "out overlaps positions"),
    (_combine, dict(out=A[0]), "out overlaps y"), (_combine, dict(out=A[0] + 126), "out overlaps y"), (_combine, dict(out=A[1] + 28), "out overlaps positions"),
    (_combine, dict(out=A[2] - 62), "out overlaps weights"),
    (_combine_grad, dict(gy=A[3]), "grad_y overlaps grad"), (_combine_grad, dict(gy=A[1]), "grad_y overlaps positions"), (_combine_grad, dict(gy=A[2] - 4), "grad_y overlaps weights"),
    (_combine_grad, dict(gw=A[4] + 124), "grad_y overlaps grad_weights"), (_combine_grad, dict(gw=A[3] - 28), "grad_weights overlaps grad"),
    (_combine_grad, dict(gw=A[1]), "grad_weights overlaps positions"), (_combine_grad, dict(gw=A[0]), "grad_weights overlaps y"),
    # in the same place, but not the same rows; and beside it
    (_combine_grad, dict(gy=A[0], gys=9), "grad_y overlaps y"), (_combine_grad, dict(gy=A[0] + 16), "grad_y overlaps y"), (_combine_grad, dict(gw=A[2] + 4), "grad_weights overlaps weights")])
def test_exchange(call, kw, why):
    _refused(call(**kw), why)


def _scores(x=A[0], tokens=A[1], logp=A[2], entropy=A[3], tl=A[4], tt=A[5], stats=A[6], vocab=10, stride=10):
    return scores._library().dcr_token_scores(x, 1, 4, vocab, stride, tokens, 1.0, 2, logp, entropy, tl, tt, stats, None)


def _scores_grad(x=A[0], stride=10, tokens=A[1], stats=A[2], gl=A[3], ge=A[4], grad=A[5], gs=10):
    return scores._library().dcr_token_scores_grad(x, 1, 4, 10, stride, tokens, stats, gl, ge, 1.0, grad, gs, None)


@pytest.mark.parametrize("call,kw,why", [
    (_scores, dict(logp=A[0] + 76), "logp overlaps logits"), (_scores, dict(entropy=A[1] + 28), "entropy overlaps tokens"), (_scores, dict(tl=A[0]), "top_logp overlaps logits"),
    (_scores, dict(tt=A[1]), "top_tokens overlaps tokens"), (_scores, dict(stats=A[0] - 44), "stats overlaps logits"), (_scores, dict(entropy=A[2]), "logp overlaps entropy"),
    (_scores, dict(tt=A[4] + 24), "top_logp overlaps top_tokens"), (_scores, dict(stride=12, logp=A[0] + 16), "logp overlaps logits"),
    # one value or one row further on, and other strides
    (_scores_grad, dict(grad=A[0] + 2), "grad overlaps logits"), (_scores_grad, dict(grad=A[0] + 20), "grad overlaps logits"),
    (_scores_grad, dict(grad=A[0] - 2), "grad overlaps logits"), (_scores_grad, dict(stride=20, grad=A[0] + 18, gs=20), "grad overlaps logits"),
    (_scores_grad, dict(stride=12, grad=A[0] + 4, gs=10), "grad overlaps logits"), (_scores_grad, dict(grad=A[1] + 24), "grad overlaps tokens"),
    (_scores_grad, dict(grad=A[2] + 44), "grad overlaps stats"), (_scores_grad, dict(grad=A[3]), "grad overlaps grad_logp"), (_scores_grad, dict(grad=A[4]), "grad overlaps grad_entropy")])
def test_scores(call, kw, why):
    _refused(call(**kw), why)


def _route(x=A[0], stride=8, bias=A[1], mask=A[2], chosen=A[3], weights=A[4], offsets=A[5], order=A[6], positions=A[7], work=A[8]):
    o = ctypes.byref(experts._RouteOpts(0, 2, 1, 1, 1, 1, 1.0))
    return experts._library().dcr_route(x, 1, 4, 8, stride, bias, mask, o, chosen, weights, offsets, order, positions, work, None)


def _route_grad(x=A[0], stride=8, chosen=A[1], gw=A[2], grad=A[3], gs=8):
    return experts._library().dcr_route_grad(x, 1, 4, 8, stride, chosen, gw, ctypes.byref(experts._RouteOpts(0, 2, 1, 1, 1, 1, 1.0)), grad, gs, None)


@pytest.mark.parametrize("call,kw,why", [
    (_route, dict(chosen=A[0] + 60), "experts overlaps logits"), (_route, dict(weights=A[1] + 28), "weights overlaps bias"), (_route, dict(offsets=A[2] - 32), "offsets overlaps mask"),
    (_route, dict(order=A[0]), "order overlaps logits"), (_route, dict(positions=A[3]), "experts overlaps positions"), (_route, dict(positions=A[6] + 28), "order overlaps positions"),
    (_route, dict(work=A[5] - 16 * 152 * 2 + 16), "offsets overlaps workspace"), (_route, dict(work=A[0]), "workspace overlaps logits"),
    (_route_grad, dict(grad=A[0] + 2), "grad overlaps logits"), (_route_grad, dict(grad=A[0] - 16), "grad overlaps logits"),
    (_route_grad, dict(stride=16, grad=A[0] + 14, gs=16), "grad overlaps logits"), (_route_grad, dict(grad=A[1] + 28), "grad overlaps experts"), (_route_grad, dict(grad=A[2]), "grad overlaps grad_weights")])
def test_route(call, kw, why):
    _refused(call(**kw), why)


def _norm(work=A[0], norm=A[1], grads=((A[2], 8), (A[3], 8))):
    return adamw._library().dcr_grad_norm((adamw._Grad * len(grads))(*grads), len(grads), 1, work, norm, None)


def _adamw(**kw):
    table = (adamw._Tensor * 2)()
    for i, e in enumerate(table):
        e.w, e.grad, e.m, e.v, e.n = A[4 * i], A[4 * i + 1], A[4 * i + 2], A[4 * i + 3], 64
    o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, step=1, state_bits=32)
    return adamw._library().dcr_adamw(table, 2, 0, 1, 3, ctypes.byref(adamw._Opts(**dict(o, **kw))), None)


@pytest.mark.parametrize("call,kw,why", [
    (_norm, dict(norm=A[3] + 12), "norm overlaps a gradient"), (_norm, dict(work=A[2] - 9728 + 8), "workspace overlaps a gradient"), (_norm, dict(norm=A[0] + 9724), "norm overlaps workspace"),
    (_adamw, dict(norm=A[0] + 252), "overlap"), (_adamw, dict(norm=A[6]), "overlap"), (_adamw, dict(device_lr=A[3] + 4), "overlap"), (_adamw, dict(device_step=A[4] + 248), "overlap")])
def test_update(call, kw, why):
    _refused(call(**kw), why)
