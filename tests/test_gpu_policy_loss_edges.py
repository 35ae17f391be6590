"""Policy loss and token log-probabilities where 32-bit arithmetic goes wrong
most easily: tokens that are nearly certain, logits far from zero, extreme
temperatures, ratios that overflow."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}


def _exact(z, tokens, temp):
    """In 64 bits and without a subtraction of near values: log-probabilities, 1 - p of the tokens, softmax."""
    z = z.double() / temp
    rows = torch.arange(len(tokens))
    rest = torch.exp(z - z[rows, tokens][:, None])
    rest[rows, tokens] = 0.0
    o = rest.sum(1)
    return -torch.log1p(o), o / (1 + o), torch.softmax(z, 1)


def _sum_error(z, temp):
    """A bound on the relative error of a row's sum of exponentials: two multiply-adds round an exponent (in units of
    log 2) of at most A by 2^-24 of it each, the rest of log2(e) / T is another such part; exponential, correction of the
    maximum's product and at most 48 additions one after another."""
    zz = z.double() / temp * 1.4426950408889634
    a = float((zz.amax(1) - zz.amin(1)).max())
    return 2.0 ** -21 + (3 * a + 48) * 2.0 ** -24


def _certain(rows, vocab, dtype, gap, seed):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, vocab, generator=g)
    tokens = torch.randint(0, vocab, (rows,), generator=g)
    tokens[0], tokens[-1] = 0, vocab - 1
    z[torch.arange(rows), tokens] += gap
    return z.to(DT[dtype]), tokens


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gap", [4.0, 8.0, 12.0])
@pytest.mark.parametrize("vocab", [2, 5, 40, 200, 2047, 7001, 33001, 280001])
def test_nearly_certain_tokens(dtype, gap, vocab):
    # the log-probability and the token's own gradient, c (1 - p), each to an error relative to itself
    rows, temp = 7, 0.8
    z, tokens = _certain(rows, vocab, dtype, gap, vocab)
    elp, eq, ep = _exact(z, tokens, temp)
    adv = torch.where(torch.arange(rows) % 2 == 0, 64.0, -64.0)
    old = elp.float()
    one = torch.ones(rows)
    loss, lp, grad = dcr.policy_loss(z.cuda(), tokens.cuda(), old.cuda(), adv.cuda(), one.cuda(), clip_low=0.5, clip_high=0.5,
                                     temperature=temp)
    r = _sum_error(z, temp)
    # the token is the largest or so near to it that nothing cancels: log1p of the others' sum, or the difference of two
    # rounded numbers of the size of lp
    top = z[torch.arange(rows), tokens] == z.amax(1)
    lp = lp.cpu().double()
    bound = torch.where(top, elp.abs() * (r + 2.0 ** -22), r + (elp.abs() + math.log(vocab) + 1) * 2.0 ** -21)
    assert bool(((lp - elp).abs() <= bound).all()), float(((lp - elp).abs() / bound).max())
    # the ratio carries lp's error, the rounding of lp - old, and the exponential's; then a few products and a quotient
    ratio = torch.exp(elp - old.double())
    c = -ratio * adv.double() / temp
    slope = bound + 2.0 ** -20
    got = grad.cpu().double()
    egrad = -c[:, None] * ep
    egrad[torch.arange(rows), tokens] = c * eq
    # a probability is the quotient of two such sums
    limit = egrad.abs() * (slope[:, None] + 2 * r + 2.0 ** -21 + 1.01 * EPS[dtype]) + TINY[dtype]
    bad = (got - egrad).abs() / limit
    assert float(bad.max()) <= 1.0, (float(bad.max()), float(bad[torch.arange(rows), tokens].max()))
    # the token's log-probability alone is the same
    assert torch.equal(dcr.token_logprobs(z.cuda(), tokens.cuda(), temperature=temp).cpu().double(), lp)


@pytest.mark.parametrize("vocab", [3, 130, 5000, 40000])
def test_token_that_is_nan_infinite_or_alone(vocab):
    z = torch.zeros(6, vocab, device="cuda")
    t = torch.tensor([0, 1, 2, vocab - 1, vocab // 2, 1], device="cuda")
    z[0, 0] = float("nan")                       # the token itself: not a number
    z[1, 1] = float("inf")                       # inf - inf
    z[2] = float("-inf")                         # alone: certain
    z[2, 2] = -3.0
    z[3, 0] = float("inf")                       # another one is infinite: impossible
    z[4, vocab // 2] = float("-inf")             # masked out
    z[5, 1] = 200.0                              # certain to 32 bits
    one = torch.ones(6, device="cuda")
    loss, lp, grad = dcr.policy_loss(z, t, torch.zeros(6, device="cuda"), one, one)
    lp, grad = lp.cpu(), grad.cpu()
    assert math.isnan(lp[0]) and math.isnan(lp[1]) and float(lp[2]) == 0.0
    assert float(lp[3]) == float("-inf") and float(lp[4]) == float("-inf") and float(lp[5]) == 0.0
    assert bool((grad[2] == 0).all()) and float(grad[5, 1]) == 0.0
    assert torch.equal(torch.isnan(dcr.token_logprobs(z, t).cpu()), torch.isnan(lp))


@pytest.mark.parametrize("dtype,vocab", [("f32", 8200), ("bf16", 40000), ("f16", 131072)])
def test_clusters_that_come_and_go(dtype, vocab):
    # rows of two to eight blocks, most of them left out and gone at once, on two streams: each block's part of the sum
    # reaches the others, whenever they start
    rows = 900
    g = torch.Generator().manual_seed(vocab)
    z = torch.randn(4, vocab, generator=g).to(DT[dtype])
    tokens = torch.randint(0, vocab, (rows,), generator=g)
    which = torch.arange(rows) % 4
    elp = torch.log_softmax(z.double(), 1)[which, tokens]
    w = (torch.rand(rows, generator=g) < 0.3).float()
    dev = z.cuda()[which.cuda()].contiguous()
    args = [t.cuda() for t in (tokens, elp.float(), torch.ones(rows), w)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [dcr.policy_loss(dev, *args, grad=i % 2 == 0, stream=streams[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    for loss, lp, grad in got:
        assert bool(((lp.cpu().double() - elp * (w != 0)).abs() <= 1e-5).all())
        assert torch.equal(lp, got[0][1]) and torch.equal(loss, got[0][0])
    assert all(torch.equal(g[2], got[0][2]) for g in got[::2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("temp", [1.0, 0.3, 0.1])
@pytest.mark.parametrize("vocab", [30, 5000, 70000])
def test_constant_rows_far_from_zero(dtype, vocab, temp):
    # softmax is uniform whatever the constant; log(V) has a few roundings, and the sum V + 2^-21 of it
    for v in (1e6, 1e8, 1e9, 5e9, 1e10, 1e12, 1e20, 1e30):
        for sign in (1, -1):
            z = torch.full((2, vocab), sign * v, dtype=DT[dtype], device="cuda")
            t = torch.tensor([0, vocab - 1], device="cuda")
            one = torch.ones(2, device="cuda")
            old = torch.full((2,), -math.log(vocab), device="cuda")
            loss, lp, grad = dcr.policy_loss(z, t, old, one, one, clip_high=1.0, clip_low=0.5, temperature=temp)
            assert float((lp + math.log(vocab)).abs().max()) <= 1e-5
            assert abs(float(loss) + 2) <= 1e-4
            exp = torch.full((2, vocab), 1.0 / vocab, dtype=torch.float64)
            exp[0, 0] -= 1
            exp[1, -1] -= 1
            exp /= temp
            err = (grad.cpu().double() - exp).abs() / exp.abs()
            assert float(err.max()) <= 1e-4 + 1.01 * EPS[dtype], (v, sign)


@pytest.mark.parametrize("temp", [1e-8, 1e-9, 1e-20, 1e-38, 1e-40, 1e-45])
@pytest.mark.parametrize("vocab", [30, 5000, 40000])
def test_temperatures_near_zero(vocab, temp):
    # ordinary logits: equal ones share the probability, and a larger one takes it all
    t = torch.tensor([3, 3, 4, 5], device="cuda")
    for v in (31.7, 20.0, -17.25, 1.0):
        z = torch.full((4, vocab), v, device="cuda")
        z[1:, 3] = v + 8
        z[3, 5] = v + 8
        lp = dcr.token_logprobs(z, t, temperature=temp).cpu()
        assert abs(float(lp[0]) + math.log(vocab)) <= 1e-5
        assert float(lp[1]) == 0.0
        assert float(lp[2]) <= -7.9 / temp * 0.999 or float(lp[2]) == float("-inf")
        assert abs(float(lp[3]) + math.log(2)) <= 1e-6


@pytest.mark.parametrize("vocab", [3, 5000, 40000])
def test_temperatures_near_the_largest(vocab):
    # z = x / T of ordinary size from logits near the type's largest
    for big, temp in ((1e38, 1e38), (1e37, 1e37), (3e30, 1e30)):
        z = torch.zeros(2, vocab, device="cuda")
        z[0, 0], z[0, 1], z[1, 2] = big, -big, -big
        t = torch.tensor([1, 0], device="cuda")
        exp = torch.log_softmax(z.cpu().double() / float(torch.tensor(temp)), 1)[torch.arange(2), t.cpu()]
        lp = dcr.token_logprobs(z, t, temperature=temp).cpu().double()
        assert float((lp - exp).abs().max()) <= 1e-5, (big, temp)


def test_overflowing_ratio_without_an_advantage():
    # exp(lp - old) passes the largest 32-bit number; times an advantage of 0 that is 0, as in 64 bits, and with an
    # advantage above 0 it is clipped
    z = torch.randn(3, 50, generator=torch.Generator().manual_seed(3)).cuda()
    t = torch.tensor([1, 2, 3], device="cuda")
    old = torch.tensor([-100.0, -2000.0, -100.0], device="cuda")
    adv = torch.tensor([0.0, 0.0, 0.5], device="cuda")
    loss, lp, grad = dcr.policy_loss(z, t, old, adv, torch.ones(3, device="cuda"), clip_high=0.25)
    assert abs(float(loss) + 1.25 * 0.5) <= 1e-6
    assert int(grad.count_nonzero()) == 0 and bool(torch.isfinite(grad).all())
