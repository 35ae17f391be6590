"""Routing to experts and its gradient against 64 bits: choices, weights and
the experts' order."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402
import step_ref as R  # noqa: E402
from step_ref import DT, EPS, TINY  # noqa: E402


def _check(z, k, got, scoring="softmax", bias=None, groups=1, group_top=None, group_by=2, renormalise=True, scale=1.0, mask=None):
    tokens, experts = z.shape
    chosen = R.choose(z, k, scoring, bias, groups, groups if group_top is None else group_top, group_by, mask)
    assert torch.equal(got.experts.cpu().long(), chosen), (got.experts.cpu().long() != chosen).any(1).nonzero()[:5]
    offsets, order, positions = R.expert_order(chosen, experts)
    assert torch.equal(got.offsets.cpu().long(), offsets)
    assert torch.equal(got.order.cpu().long(), order)
    assert torch.equal(got.positions.cpu().long(), positions)
    w = R.weights(z.double(), chosen, scoring, renormalise, scale)
    # exponentials of 2 units and of a difference rounded by 2^-24 of it, sums of up to 37 terms one after another, two quotients
    finite = z.double()[torch.isfinite(z.double())]
    rel = (float(finite.max() - finite.min()) if finite.numel() else 0.0) * 2.0 ** -23 + 64 * 2.0 ** -24
    off = (got.weights.cpu().double() - w).abs()
    assert bool((off <= w.abs() * rel + TINY["f32"]).all()), float((off / w.abs()).nan_to_num(0).max())
    return chosen


def _router(tokens, experts, dtype, seed):
    return (torch.randn(tokens, experts, generator=torch.Generator().manual_seed(seed)) * 1.5).to(DT[dtype])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,k,dtype", [
    (0, 8, 2, "f32"), (1, 1, 1, "f32"), (1, 64, 8, "bf16"), (5, 2, 2, "f16"), (33, 60, 4, "f32"), (128, 64, 8, "f32"), (129, 64, 8, "bf16"),
    (700, 100, 6, "f16"), (65, 256, 32, "f32"), (300, 512, 8, "f32"), (257, 1000, 3, "bf16"), (40, 1024, 32, "f32"), (2500, 33, 1, "f32")])
def test_choice_and_order(tokens, experts, k, dtype, scoring):
    # bf16 logits: many equal ones
    z = _router(tokens, experts, dtype, tokens + experts)
    bias = torch.randn(experts, generator=torch.Generator().manual_seed(2)) * 0.05
    for b in (None, bias):
        for renormalise, scale in ((True, 1.0), (False, 2.5)):
            got = dcr.route_experts(z.cuda(), k, scoring=scoring, bias=None if b is None else b.cuda(), renormalise=renormalise, scale=scale)
            assert got.experts.dtype == got.offsets.dtype == got.order.dtype == got.positions.dtype == torch.int32
            _check(z, k, got, scoring, b, renormalise=renormalise, scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts", [1, 31, 33, 64, 127, 129, 256, 257, 511, 513, 777, 1023, 1024])
def test_few_and_many_tokens_over_any_number_of_experts(experts, dtype):
    # a batch in one launch, and just more than that
    k = min(experts, 8)
    bias = torch.randn(experts, generator=torch.Generator().manual_seed(2)) * 0.05
    for tokens in (1, 1024 // k, 1024 // k + 1):
        z = _router(tokens, experts, dtype, experts)
        _check(z, k, dcr.route_experts(z.cuda(), k, bias=bias.cuda()), bias=bias)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_by", [1, 2])
@pytest.mark.parametrize("tokens,experts,groups,group_top,k", [
    (70, 256, 8, 4, 8), (300, 64, 8, 2, 8), (9, 8, 8, 3, 3), (200, 60, 12, 5, 6), (130, 1024, 32, 1, 16), (64, 96, 3, 2, 32), (50, 160, 32, 32, 7),
    (40, 24, 2, 2, 24)])
def test_groups(tokens, experts, groups, group_top, k, group_by, scoring):
    z = _router(tokens, experts, "f32", experts)
    bias = torch.randn(experts, generator=torch.Generator().manual_seed(2)) * 0.05
    mask = torch.rand(tokens, generator=torch.Generator().manual_seed(3)) < 0.8
    for b in (None, bias):
        kw = dict(scoring=scoring, groups=groups, group_top=group_top, group_by=group_by)
        got = dcr.route_experts(z.cuda(), k, bias=None if b is None else b.cuda(), mask=mask.cuda(), **kw)
        _check(z, k, got, bias=b, mask=mask, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_scores_nearer_than_32_bits_tell(scoring, groups):
    # logits one unit of 2^-23 apart, in any order: scores of 32 bits are equal or in the wrong order
    tokens, experts, k = 40, 64, 7
    g = torch.Generator().manual_seed(8)
    z = torch.stack([1.0 + torch.randperm(experts, generator=g) * 2.0 ** -23 for _ in range(tokens)])
    bias = torch.zeros(experts)
    kw = dict(scoring=scoring, groups=groups, group_top=max(1, groups // 2), group_by=2)
    _check(z, k, dcr.route_experts(z.cuda(), k, bias=bias.cuda(), **kw), bias=bias, **kw)
    # scores that differ by less than a unit of 32 bits through a bias that nearly makes them equal
    x = torch.linspace(-1, 1, experts)
    s = torch.softmax(x.double(), 0) if scoring == "softmax" else torch.sigmoid(x.double())
    bias = (0.5 - s).float()
    z = x.expand(tokens, experts).contiguous()
    _check(z, k, dcr.route_experts(z.cuda(), k, bias=bias.cuda(), **kw), bias=bias, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_experts_and_tokens(scoring, renormalise, groups):
    tokens, experts, k = 9, 16, 4
    z = _router(tokens, experts, "f32", 5)
    z[0] = -math.inf                            # nothing to choose
    z[1, 2:] = -math.inf                        # fewer than k
    z[2, ::2] = float("nan")
    z[3] = float("nan")
    z[4, 3] = math.inf
    z[5] = torch.finfo(torch.float32).min       # all equal, and far away
    z[6] = 0.0
    z[7, :] = -200.0                            # scores that 32 bits cannot hold
    z[7, 5] = -190.0
    bias = torch.zeros(experts)
    bias[9] = -math.inf
    for b in (None, bias):
        for mask in (None, torch.tensor([1, 1, 1, 1, 1, 1, 1, 1, 0], dtype=torch.uint8)):
            kw = dict(scoring=scoring, groups=groups, group_top=max(1, groups // 2), renormalise=renormalise)
            got = dcr.route_experts(z.cuda(), k, bias=None if b is None else b.cuda(), mask=None if mask is None else mask.cuda(), **kw)
            assert bool((got.weights >= 0).all()) and bool(torch.isfinite(got.weights).all())
            chosen = R.choose(z, k, scoring, b, groups, kw["group_top"], 2, mask)
            assert torch.equal(got.experts.cpu().long(), chosen)
            assert bool((got.weights.cpu()[chosen < 0] == 0).all())
            keep = [i for i in range(tokens) if i != 4 and not (i == 7 and not renormalise)]
            w = R.weights(z[keep].double(), chosen[keep], scoring, renormalise, 1.0)
            off = (got.weights.cpu()[keep].double() - w).abs()
            assert bool((off <= w * 2.0 ** -16).all()), off
            grad = dcr.route_experts_grad(z.cuda(), got, torch.ones(tokens, k, device="cuda"), scoring=scoring, renormalise=renormalise).cpu()
            assert bool((grad[0] == 0).all()) and bool((grad[3] == 0).all()) and bool(torch.isfinite(grad[keep]).all())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("tokens,experts,k,dtype", [(1, 1, 1, "f32"), (5, 8, 2, "f32"), (200, 64, 8, "bf16"), (77, 100, 6, "f16"), (33, 1000, 32, "f32")])
def test_gradient(tokens, experts, k, dtype, renormalise, scoring):
    z = _router(tokens, experts, dtype, 4)
    mask = torch.arange(tokens) % 5 != 4
    d = torch.randn(tokens, k, generator=torch.Generator().manual_seed(6))
    got = dcr.route_experts(z.cuda(), k, scoring=scoring, renormalise=renormalise, scale=1.7, mask=mask.cuda())
    grad = dcr.route_experts_grad(z.cuda(), got, d.cuda(), scoring=scoring, renormalise=renormalise, scale=1.7)
    assert grad.dtype == z.dtype
    x = z.double().requires_grad_()
    chosen = got.experts.cpu().long()
    (R.weights(x, chosen, scoring, renormalise, 1.7) * d).sum().backward()
    # a difference of two sums of products, each with the weights' error
    size = (R.weights(z.double(), chosen, scoring, renormalise, 1.7) * d.abs()).sum(1, keepdim=True) + 1.7 * d.abs().amax(1, keepdim=True) * (
        torch.softmax(z.double(), 1) if scoring == "softmax" else 0.0)
    off = (grad.cpu().double() - x.grad).abs()
    bound = size * 2.0 ** -17 + x.grad.abs() * 1.01 * EPS[dtype] + TINY[dtype]
    assert bool((off <= bound).all()), float((off / bound).max())


def test_gradient_against_differences():
    tokens, experts, k = 3, 9, 3
    z = _router(tokens, experts, "f32", 7)
    d = torch.randn(tokens, k, generator=torch.Generator().manual_seed(8))
    for scoring in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            got = dcr.route_experts(z.cuda(), k, scoring=scoring, renormalise=renormalise)
            grad = dcr.route_experts_grad(z.cuda(), got, d.cuda(), scoring=scoring, renormalise=renormalise).cpu()
            chosen = got.experts.cpu().long()
            for i in range(tokens):
                for j in range(experts):
                    step = torch.zeros(tokens, experts, dtype=torch.float64)
                    step[i, j] = 1e-4
                    f = [float((R.weights(z.double() + s * step, chosen, scoring, renormalise, 1.0) * d).sum()) for s in (1, -1)]
                    assert abs((f[0] - f[1]) / 2e-4 - float(grad[i, j])) <= 1e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_streams_and_graphs(dtype):
    tokens, experts, k = 400, 40, 4
    z = _router(tokens, experts, dtype, 9)
    buf = torch.full((tokens, experts + 7), 50.0, dtype=DT[dtype], device="cuda")
    view = buf[:, 3:3 + experts]
    view.copy_(z)
    exp = dcr.route_experts(z.cuda(), k)
    got = dcr.route_experts(view, k)
    assert all(torch.equal(a, b) for a, b in zip(exp, got))
    d = torch.randn(tokens, k, generator=torch.Generator().manual_seed(8)).cuda()
    grad = dcr.route_experts_grad(z.cuda(), exp, d)
    assert torch.equal(dcr.route_experts_grad(view, exp, d, out=view), grad) and torch.equal(view, grad)
    assert bool((buf[:, :3] == 50).all()) and bool((buf[:, 3 + experts:] == 50).all())
    s = torch.cuda.Stream()
    zz = z.cuda()
    s.wait_stream(torch.cuda.current_stream())
    got = dcr.route_experts(zz, k, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(exp, got))
    # two graphs, each with its own workspace, replayed at the same time
    graphs, outs, ins = [], [], []
    for i in range(2):
        ins.append(zz.clone())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(dcr.route_experts(ins[i], k))
    ins[1].copy_(zz.flip(0))
    want = dcr.route_experts(ins[1], k)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], exp)) and all(torch.equal(a, b) for a, b in zip(outs[1], want))


def test_back_to_back_with_changing_logits():
    # the workspace of one call is the next one's
    zs = [_router(3000, 64, "f32", i).cuda() for i in range(4)]
    exp = [dcr.route_experts(z, 8) for z in zs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [dcr.route_experts(z, 8) for z in zs]
        for a, b in zip(got, exp):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_all_tokens_to_the_same_experts():
    z = torch.zeros(3000, 64)
    z[:, 5], z[:, 63] = 2.0, 1.0
    _check(z, 2, dcr.route_experts(z.cuda(), 2))


@pytest.mark.parametrize("experts,groups", [(64, 1), (256, 8), (60, 6), (1000, 4)])
def test_rows_without_a_difference(experts, groups):
    # padding that nothing masks: all logits of a row are equal, beside rows that are not; with all sorts of biases
    k, kw = 8, dict(groups=groups, group_top=max(2, groups // 2) if groups > 1 else 1)
    z = _router(300, experts, "f32", 11)
    z[::2] = 0.0
    z[1::10] = 3.5
    z[3::10] = -math.inf
    z[5::10, -1] = 0.1
    z[7::10] = float("nan")
    zero = torch.zeros(experts)
    some = zero.clone()
    some[3], some[-1] = -math.inf, 0.25
    for scoring in ("softmax", "sigmoid"):
        for bias in (None, zero, zero + 0.5, some, zero - math.inf):
            got = dcr.route_experts(z.cuda(), k, scoring=scoring, bias=None if bias is None else bias.cuda(), **kw)
            chosen = R.choose(z, k, scoring, bias, groups, kw["group_top"], 2, None)
            assert torch.equal(got.experts.cpu().long(), chosen)
            offsets, order, positions = R.expert_order(chosen, experts)
            assert torch.equal(got.offsets.cpu().long(), offsets) and torch.equal(got.order.cpu().long(), order)
            w = R.weights(z.double(), chosen, scoring, True, 1.0)
            # a few roundings: equal parts of 1, or the quotients of other tests
            assert bool(((got.weights.cpu().double() - w).abs() <= w * 2.0 ** -16).all())
