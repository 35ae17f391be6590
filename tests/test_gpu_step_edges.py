"""Rare inputs of a step's operators."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402
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
