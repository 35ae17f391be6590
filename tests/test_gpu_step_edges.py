"""Rare inputs of a step's operators."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402
from bit_exact_xor_gb300 import experts  # noqa: E402
import step_ref as R  # noqa: E402
from step_ref import DT  # noqa: E402


def _rows_of_few_numbers(vocab):
    g = torch.Generator().manual_seed(3)
    z = torch.full((8, vocab), float("nan"))                            # the first: no number at all
    z[1, [5, vocab // 2, vocab - 1]] = torch.tensor([1.0, -2.0, 3.0])
    z[2, ::vocab // 30] = float("-inf")
    z[3] = z[2]
    z[3, 7:12] = torch.randn(5, generator=g)
    z[4, :600] = torch.randn(vocab, generator=g)[:600]
    z[5, 100:] = float("-inf")
    z[6, torch.randperm(vocab, generator=g)[:63]] = float("inf")
    z[7] = torch.randn(vocab, generator=g)                              # an ordinary one beside them
    return z


@pytest.mark.parametrize("rows,vocab,dtype", [(6, 40000, "f32"), (400, 40000, "f32"), (400, 40000, "bf16"), (1216, 20011, "f32"), (800, 9000, "f16"), (700, 200, "bf16")])
@pytest.mark.parametrize("top", [1, 8, 64])
def test_alternatives_of_rows_of_few_numbers(rows, vocab, dtype, top):
    z = _rows_of_few_numbers(vocab).to(DT[dtype])
    exp = R.top(z, top)
    at = torch.arange(rows) % len(z)
    got = dcr.token_scores(z[at].cuda(), torch.zeros(rows, dtype=torch.int64, device="cuda"), top=top)
    tokens = got.top_tokens.cpu()
    assert int(tokens.min()) >= 0 and int(tokens.max()) < vocab
    assert torch.equal(tokens, exp[at]), (tokens != exp[at]).any(1).nonzero()[:8, 0]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("large", [100.0, 1000.0, 65536.0])
@pytest.mark.parametrize("size", [2, 4, 6])
def test_groups_whose_biases_cancel(size, large, scoring):
    # the two best of a group have biases of opposite sign: their sum is far smaller than what it is the sum of
    tokens, groups = 2000, 4
    g = torch.Generator().manual_seed(size)
    bias = torch.tensor([large, -large] + [-4 * large] * (size - 2)).repeat(groups)
    z = torch.randn(tokens, 1, size, generator=g) + torch.randn(tokens, groups, size, generator=g) * 2e-5
    z = z.reshape(tokens, groups * size).contiguous()
    for group_top in (1, 2):
        kw = dict(scoring=scoring, groups=groups, group_top=group_top, group_by=2)
        got = dcr.route_experts(z.cuda(), 2, bias=bias.cuda(), **kw)
        exp = R.choose(z, 2, scoring, bias, groups, group_top, 2, None)
        assert torch.equal(got.experts.cpu().long(), exp), int((got.experts.cpu().long() != exp).any(1).sum())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_groups_whose_sums_pass_32_bits(scoring):
    # each score and bias is a finite number, and the sum of two is not one of 32 bits
    far = torch.tensor([-3.4e38, -3.4e38, -3e38, -3e38, -3.2e38, -3.2e38, 1.0, -math.inf])
    z = torch.randn(50, 8, generator=torch.Generator().manual_seed(4))
    for bias, group_top, k in ((far, 1, 1), (far, 2, 3), (far, 3, 5), (-far, 1, 2), (-far, 2, 4), (far.abs().clamp(max=3.4e38), 2, 3)):
        kw = dict(scoring=scoring, groups=4, group_top=group_top, group_by=2)
        got = dcr.route_experts(z.cuda(), k, bias=bias.cuda(), **kw)
        exp = R.choose(z, k, scoring, bias, 4, group_top, 2, None)
        assert torch.equal(got.experts.cpu().long(), exp), (got.experts[0].tolist(), exp[0].tolist())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_groups_whose_sums_pass_32_bits_and_that_are_chosen_from_again(scoring):
    # more experts of equal scores than a warp has lanes, which are decided one after another
    bias = torch.tensor([-3.4e38, -3e38, -3.2e38, -3.1e38]).repeat_interleave(40)
    z = torch.randn(50, 160, generator=torch.Generator().manual_seed(4))
    for group_top in (1, 2, 4):
        kw = dict(scoring=scoring, groups=4, group_top=group_top, group_by=2)
        got = dcr.route_experts(z.cuda(), 8, bias=bias.cuda(), **kw)
        exp = R.choose(z, 8, scoring, bias, 4, group_top, 2, None)
        assert torch.equal(got.experts.cpu().long(), exp), (got.experts[0].tolist(), exp[0].tolist())


@pytest.mark.parametrize("dtype,value", [("f32", 5e18), ("f32", 1e19), ("f32", 3e38), ("f32", 1e-22), ("f32", 1e-38), ("f32", 1e-44), ("bf16", 5e18),
                                         ("bf16", 1e38), ("bf16", 1e-22), ("bf16", 1e-39), ("f16", 6e-8)])
@pytest.mark.parametrize("n,gap", [(1, 0), (300, 1), (16384, 0), (100003, 3)])
def test_norm_of_squares_that_32_bits_do_not_hold(n, gap, dtype, value):
    g = (torch.randn(n + gap, generator=torch.Generator().manual_seed(1)).clamp(-1, 1) * value).to(DT[dtype])
    for x in (g, torch.full_like(g, value)):
        exp = math.sqrt(float((x[gap:].double() / value).square().sum())) * value
        got = float(dcr.grad_norm([x.cuda()[gap:]]))
        # at most 65 squares of 32 bits one after another, of which the root halves the error, and the result's own rounding
        assert abs(got - exp) <= exp * 70 * 2.0 ** -25 + 2.0 ** -150 or (exp > 3.4028235e38 and got == math.inf), (got, exp)


def test_norm_of_large_among_small():
    # one thread's squares do not fit 32 bits, the others' do not; what is not a number stays that
    x = torch.ones(100000)
    x[777], x[50001] = 1e30, 1e-30
    exp = math.sqrt(float(x.double().square().sum()))
    assert abs(float(dcr.grad_norm([torch.zeros(5000, device="cuda"), x.cuda()])) - exp) <= exp * 70 * 2.0 ** -25
    for bad in (math.inf, math.nan):
        x[99999] = bad
        norm = float(dcr.grad_norm([x.cuda()]))
        assert not math.isfinite(norm) and math.isnan(norm) == math.isnan(bad)
    assert float(dcr.grad_norm([torch.zeros(70001, dtype=torch.bfloat16, device="cuda"), -torch.zeros(3, dtype=torch.bfloat16, device="cuda")])) == 0.0


def test_moments_in_8_bits_near_the_smallest_number():
    # scales below the smallest normal number: they, and what the moments are divided by, have fewer digits
    n, blocks = 2 ** 20, 2 ** 12
    g = torch.Generator().manual_seed(6)
    size = torch.exp(torch.linspace(math.log(1e-36), math.log(1e-34), blocks))
    grad = (torch.rand(blocks, 256, generator=g) * 2 - 1) * size[:, None]
    grad[:, 0] = size                       # the block's largest
    grad[::2, ::3] = -size[::2, None]       # and many equal to it
    grad = grad.reshape(-1)
    w = torch.randn(n, generator=g)
    state = dcr.adamw_states([w.cuda()], 8)
    dev = w.cuda()
    dcr.adamw_step([dev], [grad.cuda()], state, 1, 1e-3, seed=11)
    zero = (torch.zeros(n, dtype=torch.uint8), torch.zeros(blocks))
    new, _, st = R.adamw(w, grad, zero + zero, None, 1, 1e-3, (0.9, 0.999), 1e-8, 0.0, bits=R.random_bits(11, 1, 0, n))
    assert float(st[1].min()) < 2.0 ** -126 < float(st[1].max())
    assert torch.equal(dev.cpu(), new)
    for a, b in zip(state[0], st):
        assert torch.equal(a.cpu(), b)
    assert not bool(((state[0].m & 127) == 127).any())


@pytest.mark.parametrize("tokens,experts,k", [(20000, 16, 8), (6000, 64, 32), (9800, 600, 32), (40000, 33, 8)])
def test_parts_of_several_rounds(tokens, experts, k):
    # a part of the batch holds more slots than the block that places them has threads
    z = torch.randn(tokens, experts, generator=torch.Generator().manual_seed(tokens))
    mask = torch.arange(tokens) % 7 != 3
    got = dcr.route_experts(z.cuda(), k, mask=mask.cuda())
    chosen = torch.where(mask[:, None], torch.sort(z, dim=1, descending=True, stable=True)[1][:, :k], -1)
    assert torch.equal(got.experts.cpu().long(), chosen)
    offsets, order, positions = R.expert_order(chosen, experts)
    assert torch.equal(got.offsets.cpu().long(), offsets)
    assert torch.equal(got.order.cpu().long(), order)
    assert torch.equal(got.positions.cpu().long(), positions)


@pytest.mark.parametrize("cols", [24, 515, 4096])
def test_exchange_within_one_buffer(cols):
    # inputs and outputs side by side in the columns of one buffer, and gradients in the place of what they are of
    tokens, k = 40, 2
    g = torch.Generator().manual_seed(2)
    chosen = torch.stack([torch.randperm(6, generator=g)[:k] for _ in range(tokens)])
    offsets, order, positions = R.expert_order(chosen, 6)
    r = dcr.Route(*(x.cuda() for x in (chosen.int(), torch.rand(tokens, k, generator=g), offsets.int(), order.int(), positions.int())))
    buf = torch.randn(tokens * k, 3 * cols + 8, generator=g).cuda()
    x, y, out, left = buf[:tokens, :cols], buf[:, cols:2 * cols], buf[:, 2 * cols:3 * cols], buf[:, 3 * cols:].clone()
    rows, sums = dcr.experts_gather(x.clone(), r), dcr.experts_combine(y.clone(), r)
    grads = dcr.experts_combine_grad(y.clone(), r, x.clone())
    assert torch.equal(dcr.experts_gather(x, r, out=out), rows)
    assert torch.equal(dcr.experts_combine(y, r, out=out[:tokens]), sums)
    with pytest.raises(dcr.DcrError, match="out overlaps y"):
        dcr.experts_combine(y, r, out=buf[:tokens, cols + 1:2 * cols + 1])
    with pytest.raises(dcr.DcrError, match="out overlaps x"):
        dcr.experts_gather(buf[:, :cols], dcr.Route(*(t[:, :1].contiguous() if t.dim() == 2 else t for t in r))._replace(
            positions=torch.arange(tokens * k, dtype=torch.int32, device="cuda").view(-1, 1)), out=buf[:, :cols])
    by_y, by_w = dcr.experts_combine_grad(y, r, x, out=y)
    assert torch.equal(y, grads[0]) and torch.equal(by_w, grads[1]) and torch.equal(buf[:, 3 * cols:], left)
    # the weights' gradient in the weights' place
    w, yy = r.weights.clone(), rows.clone()
    exp = dcr.experts_combine_grad(yy, r, sums)
    dcr.check(experts._library().dcr_experts_combine_grad(yy.data_ptr(), 0, tokens * k, cols, cols, r.positions.data_ptr(), w.data_ptr(), tokens, k,
                                                          sums.data_ptr(), 0, cols, None, cols, w.data_ptr(), torch.cuda.current_stream().cuda_stream))
    assert torch.equal(w, exp[1])


@pytest.mark.parametrize("vocab", [40, 9001])
def test_scores_within_one_buffer(vocab):
    # the gradient, and the outputs, in the columns beside the logits
    rows = 12
    z = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(2))
    tokens, one = torch.arange(rows).cuda(), torch.ones(rows, device="cuda")
    buf = torch.zeros(rows, 2 * vocab, device="cuda")
    left, right = buf[:, :vocab], buf[:, vocab:]
    left.copy_(z)
    s = dcr.token_scores(left, tokens)
    exp = dcr.token_scores_grad(left.contiguous(), tokens, s.stats, one, one)
    assert torch.equal(dcr.token_scores_grad(left, tokens, s.stats, one, one, out=right), exp)
    with pytest.raises(dcr.DcrError, match="grad overlaps logits"):
        dcr.token_scores_grad(left, tokens, s.stats, one, one, out=buf[:, 1:vocab + 1])


def test_routing_within_one_buffer():
    # the router's logits, and their gradient, beside what they are computed from
    tokens, n = 70, 24
    buf = torch.randn(tokens, 100 + n, generator=torch.Generator().manual_seed(2)).cuda()
    z, d = buf[:, 100:], torch.ones(tokens, 4, device="cuda")
    r, exp = dcr.route_experts(z, 4), dcr.route_experts(z.contiguous(), 4)
    assert all(torch.equal(a, b) for a, b in zip(r, exp))
    grad = dcr.route_experts_grad(z, r, d, renormalise=False)
    assert torch.equal(dcr.route_experts_grad(z, r, d, renormalise=False, out=buf[:, 100 - n:100]), grad)
    with pytest.raises(dcr.DcrError, match="grad overlaps logits"):
        dcr.route_experts_grad(z, r, d, out=buf[:, 99:99 + n])


def test_update_beside_its_numbers():
    # the norm, the rate and the step beside the tensors that are written, and the norm of a gradient that is the rate's neighbour
    n = 64
    buf = torch.zeros(4 * n + 8, device="cuda")
    w, m, v, g = (buf[i * n:(i + 1) * n] for i in range(4))
    norm, lr = buf[4 * n:4 * n + 1], buf[4 * n + 1:4 * n + 2]
    g.normal_()
    norm.copy_(dcr.grad_norm([g]))
    lr.fill_(0.5)
    dcr.adamw_step([w], [g], [dcr.AdamState32(m, v)], 1, lr, norm=norm, max_norm=1e6)
    assert bool(((w + 0.5 * torch.sign(g)).abs() < 1e-3).all())
    before = buf.clone()
    with pytest.raises(dcr.DcrError, match="overlap"):
        dcr.adamw_step([w], [g], [dcr.AdamState32(m, v)], 2, lr, norm=v[:1], max_norm=1e6)
    assert torch.equal(buf, before)
