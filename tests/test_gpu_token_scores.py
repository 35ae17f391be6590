"""Token scores and their gradient against 64 bits: log-probabilities,
entropies, likeliest alternatives."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402
import step_ref as R  # noqa: E402
from step_ref import DT, EPS, TINY  # noqa: E402


def _rows(rows, vocab, dtype, seed, gap=0.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, vocab, generator=g) * 3
    tokens = torch.randint(0, vocab, (rows,), generator=g)
    if gap:
        z[torch.arange(rows), tokens] += gap + 12
    return z.to(DT[dtype]), tokens


def _check(z, tokens, temp, got, dtype):
    lp, h, p, d, mean, r = R.scores(z, tokens, temp)
    err = R.sum_error(z, temp)
    off = (got.logp.cpu().double() - lp).abs()
    is_max = z.double().gather(1, tokens[:, None])[:, 0] == z.double().amax(1)
    # -log(1 + r) alone, or a difference of two rounded numbers of the size of the result
    bound = torch.where(is_max, lp.abs() * (err + 2.0 ** -21) + TINY["f32"], err + (lp.abs() + math.log(z.shape[1]) + 1) * 2.0 ** -21)
    assert bool((off <= bound).all()), float((off / bound).max())
    # both parts are sums of one sign
    off = (got.entropy.cpu().double() - h).abs()
    bound = h * (2 * err + 2.0 ** -20) + TINY["f32"]
    assert bool((off <= bound).all()), float((off / bound).max())
    return p, d, mean, r, err


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gap", [0.0, 6.0])
@pytest.mark.parametrize("vocab", [1, 2, 5, 40, 257, 2047, 7001, 33001, 140001])
def test_scores_and_gradient(vocab, gap, dtype):
    rows, temp = 7, 0.8
    z, tokens = _rows(rows, vocab, dtype, vocab, gap)
    got = dcr.token_scores(z.cuda(), tokens.cuda(), temperature=temp)
    p, d, mean, r, err = _check(z, tokens, temp, got, dtype)
    assert got.top_logp is None and got.top_tokens is None
    g = torch.Generator().manual_seed(1)
    ga, gb = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    at = torch.arange(rows)
    for a, b in ((ga, gb), (ga, None), (None, gb)):
        grad = dcr.token_scores_grad(z.cuda(), tokens.cuda(), got.stats, None if a is None else a.cuda(), None if b is None else b.cuda(),
                                     temperature=temp)
        assert grad.dtype == z.dtype and grad.shape == z.shape
        a64 = torch.zeros(rows, 1, dtype=torch.float64) if a is None else a.double()[:, None]
        b64 = torch.zeros(rows, 1, dtype=torch.float64) if b is None else b.double()[:, None]
        other = -p * (a64 + b64 * (d + mean[:, None]))
        size = p * (a64.abs() + b64.abs() * (d.abs() + mean[:, None]))
        # 1 - p is r / (1 + r) for the largest, and not small for any other
        q = torch.where(d[at, tokens] == 0, r / (1 + r), 1 - p[at, tokens])
        mine = a64[:, 0] * q - b64[:, 0] * p[at, tokens] * (d[at, tokens] + mean)
        other[at, tokens] = mine
        size[at, tokens] = a64[:, 0].abs() * q + size[at, tokens]
        exp = other / temp
        bound = size / temp * (4 * err + 2.0 ** -19) + exp.abs() * 1.01 * EPS[dtype] + TINY[dtype]
        off = (grad.cpu().double() - exp).abs()
        assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,top", [(3, 1, 1), (5, 64, 64), (4, 65, 64), (9, 300, 5), (400, 300, 5), (5, 4099, 20), (6, 7000, 1),
                                            (3, 66001, 64), (310, 20011, 20)])
def test_alternatives(rows, vocab, top, dtype):
    z, tokens = _rows(rows, vocab, dtype, rows + vocab)
    got = dcr.token_scores(z.cuda(), tokens.cuda(), top=top, temperature=0.7)
    exp = torch.sort(z.float(), dim=1, descending=True, stable=True)[1][:, :top]
    assert torch.equal(got.top_tokens.cpu(), exp)
    _check(z, tokens, 0.7, got, dtype)
    same = dcr.token_scores(z.cuda(), tokens.cuda(), temperature=0.7)
    assert torch.equal(same.logp, got.logp) and torch.equal(same.entropy, got.entropy) and torch.equal(same.stats, got.stats)
    # an alternative's log-probability is what the token itself would have
    for i in {0, top // 2, top - 1}:
        each = dcr.token_scores(z.cuda(), got.top_tokens[:, i].contiguous(), temperature=0.7)
        assert torch.equal(each.logp, got.top_logp[:, i])


def _hard_rows(vocab):
    """Rows whose alternatives are hard to find."""
    g = torch.Generator().manual_seed(5)
    i = torch.arange(vocab)
    rows = [torch.zeros(vocab), torch.randint(0, 3, (vocab,), generator=g).float(), i.float() / vocab, -i.float() / vocab]
    for allowed in (0, 3, min(500, vocab), vocab // 2):             # masked: the rest is -inf, or the type's lowest
        for low in (-math.inf, torch.finfo(torch.float32).min):
            row = torch.full((vocab,), low)
            row[torch.randperm(vocab, generator=g)[:allowed]] = torch.randn(allowed, generator=g)
            if allowed or low != -math.inf:
                rows.append(row)
    warp = i // 4 // 32 % 8                             # of the thread that reads it, where rows are aligned
    for w in (0, 7):
        rows.append(torch.where(warp == w, torch.tensor(-5.0), torch.rand(vocab, generator=g)))
    rows.append(torch.where(i % 2 == 0, torch.tensor(0.0), torch.tensor(-0.0)))
    only = torch.full((vocab,), -3.0)
    only[-1] = 2.0
    rows.append(only)
    return torch.stack(rows)


@pytest.mark.parametrize("vocab,top", [(7000, 1), (7000, 20), (7000, 64), (40000, 20), (70, 64), (70, 5), (700, 20), (700, 32), (764, 1), (764, 33)])
@pytest.mark.parametrize("many", [False, True])
def test_alternatives_of_hard_rows(vocab, top, many):
    z = _hard_rows(vocab)
    n = len(z)
    if many:
        z = z.repeat(1 + 310 // n, 1)
    tokens = torch.zeros(len(z), dtype=torch.int64)
    got = dcr.token_scores(z.cuda(), tokens.cuda(), top=top)
    exp = torch.sort(z + 0.0, dim=1, descending=True, stable=True)[1][:, :top]
    assert torch.equal(got.top_tokens.cpu(), exp), (got.top_tokens.cpu() != exp).any(1).nonzero()[:, 0]


@pytest.mark.parametrize("vocab", [9, 5000, 40000])
def test_nan_and_infinities(vocab):
    z = torch.randn(6, vocab, generator=torch.Generator().manual_seed(2))
    t = torch.tensor([0, 1, 2, 3, 4, 5])
    z[0, 3] = float("nan")
    z[1] = float("nan")
    z[2, 2] = float("inf")
    z[3, 4] = float("inf")
    z[4] = float("-inf")
    z[5] = float("-inf")
    z[5, 5] = 1.5
    top = min(vocab, 8)
    got = dcr.token_scores(z.cuda(), t.cuda(), top=top)
    lp, h = got.logp.cpu(), got.entropy.cpu()
    assert math.isnan(lp[0]) and math.isnan(lp[1]) and math.isnan(lp[2]) and float(lp[3]) == -math.inf and math.isnan(lp[4])
    assert float(lp[5]) == 0.0 and float(h[5]) == 0.0 and all(math.isnan(h[i]) for i in range(5))
    assert torch.equal(got.top_tokens.cpu(), R.top(z, top))
    # the same as the other call's log-probabilities
    assert torch.equal(torch.isnan(dcr.token_logprobs(z.cuda(), t.cuda()).cpu()), torch.isnan(lp))
    one = torch.ones(6, device="cuda")
    grad = dcr.token_scores_grad(z.cuda(), t.cuda(), got.stats, one, one).cpu()
    assert bool((grad[5] == 0).all()) and bool(torch.isnan(grad[0]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [30, 5000, 70000])
@pytest.mark.parametrize("value,temp", [(1e6, 1.0), (-1e9, 0.3), (1e20, 0.1), (1e30, 1.0), (17.0, 1e-20), (3.0, 1e-45)])
def test_constant_rows_far_from_zero(dtype, vocab, value, temp):
    z = torch.full((2, vocab), value, dtype=DT[dtype], device="cuda")
    t = torch.tensor([0, vocab - 1], device="cuda")
    got = dcr.token_scores(z, t, top=2, temperature=temp)
    # 1 + r is the vocabulary's size after a few hundred roundings; then a logarithm
    bound = 192 * 2.0 ** -24 + math.log(vocab) * 2.0 ** -22
    assert float((got.logp.double() + math.log(vocab)).abs().max()) <= bound
    assert float((got.entropy.double() - math.log(vocab)).abs().max()) <= bound
    assert got.top_tokens.tolist() == [[0, 1]] * 2
    if temp >= 0.1:
        one = torch.ones(2, device="cuda")
        grad = dcr.token_scores_grad(z, t, got.stats, one, one, temperature=temp).cpu().double()
        exp = torch.full((2, vocab), -1.0 / vocab, dtype=torch.float64)
        exp[0, 0] += 1
        exp[1, -1] += 1
        exp /= temp
        # the entropy's part is log2 e of a sum of many roundings times p
        off = (grad - exp).abs()
        assert bool((off <= exp.abs() * (EPS[dtype] * 1.01 + 2.0 ** -14) + 2.0 ** -20 / vocab / temp).all()), float(off.max())


def test_rows_that_are_left_out():
    vocab = 1003
    z, tokens = _rows(6, vocab, "f32", 3)
    tokens[1], tokens[4] = -1, vocab
    z[1], z[4] = float("nan"), float("inf")
    got = dcr.token_scores(z.cuda(), tokens.cuda(), top=3)
    for i in (1, 4):
        assert float(got.logp[i]) == 0.0 and float(got.entropy[i]) == 0.0 and got.top_tokens[i].tolist() == [-1] * 3
        assert got.top_logp[i].tolist() == [0.0] * 3 and got.stats[i].tolist() == [0.0] * 3
    keep = [0, 2, 3, 5]
    # the others as in a batch that leaves none out, at the same places: which thread sums a value goes by its place in a word
    some = dcr.token_scores(z.cuda(), tokens.clamp(0, vocab - 1).cuda(), top=3)
    for a, b in zip(got, some):
        assert torch.equal(a[keep], b[keep])
    one = torch.ones(6, device="cuda")
    one[3] = 0
    grad = dcr.token_scores_grad(z.cuda(), tokens.cuda(), got.stats, one, one)
    assert int(grad[[1, 3, 4]].count_nonzero()) == 0 and bool((grad[[0, 2, 5]] != 0).any(1).all())


@pytest.mark.parametrize("dtype,skip,pad", [("bf16", 1, 7), ("f16", 3, 13), ("f32", 1, 2), ("bf16", 8, 8)])
@pytest.mark.parametrize("vocab", [3, 130, 9001])
def test_strides_and_offsets(vocab, dtype, skip, pad):
    z, tokens = _rows(5, vocab, dtype, 9)
    buf = torch.full((5, skip + vocab + pad), float("nan"), dtype=DT[dtype], device="cuda")
    view = buf[:, skip:skip + vocab]
    view.copy_(z)
    a, b = dcr.token_scores(view, tokens.cuda(), top=2), dcr.token_scores(z.cuda(), tokens.cuda(), top=2)
    # which thread sums a value goes by its place in a 16-byte word
    assert torch.equal(a.top_tokens, b.top_tokens)
    _check(z, tokens, 1.0, a, dtype)
    one = torch.ones(5, device="cuda")
    exp = dcr.token_scores_grad(z.cuda(), tokens.cuda(), b.stats, one, one)
    before = buf.clone()
    assert torch.equal(dcr.token_scores_grad(view, tokens.cuda(), b.stats, one, one), exp)
    # into another matrix with rows at another offset, then in place; what lies around stays as it was
    out = torch.full((5, vocab + 5), 7.0, dtype=DT[dtype], device="cuda")
    dcr.token_scores_grad(view, tokens.cuda(), b.stats, one, one, out=out[:, 2:2 + vocab])
    assert torch.equal(out[:, 2:2 + vocab], exp) and bool((out[:, :2] == 7).all()) and bool((out[:, 2 + vocab:] == 7).all())
    assert torch.equal(buf.nan_to_num(9.0), before.nan_to_num(9.0))
    dcr.token_scores_grad(view, tokens.cuda(), b.stats, one, one, out=view)
    assert torch.equal(view, exp)
    assert bool(torch.isnan(buf[:, :skip]).all()) and bool(torch.isnan(buf[:, skip + vocab:]).all())


def test_gradient_against_differences():
    # of sum_i a_i logp_i + b_i H_i, by central differences of the formulas in 64 bits
    rows, vocab, temp = 3, 11, 0.9
    z, tokens = _rows(rows, vocab, "f32", 4)
    a, b = torch.tensor([0.7, -1.2, 0.3]), torch.tensor([0.5, 0.9, -2.0])
    got = dcr.token_scores(z.cuda(), tokens.cuda(), temperature=temp)
    grad = dcr.token_scores_grad(z.cuda(), tokens.cuda(), got.stats, a.cuda(), b.cuda(), temperature=temp).cpu().double()

    def value(x):
        lp, h = R.scores(x, tokens, temp)[:2]
        return (a * lp + b * h).sum()

    for i in range(rows):
        for j in range(vocab):
            d = torch.zeros(rows, vocab, dtype=torch.float64)
            d[i, j] = 1e-4
            slope = float((value(z.double() + d) - value(z.double() - d)) / 2e-4)
            assert abs(slope - float(grad[i, j])) <= 1e-5


def test_empty_batches_and_large_offsets():
    z = torch.empty(0, 5, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    got = dcr.token_scores(z, t, top=2)
    assert got.logp.shape == (0,) and got.top_tokens.shape == (0, 2)
    assert dcr.token_scores_grad(z, t, got.stats).shape == (0, 5)
    buf = torch.empty(2 ** 31 + 6000, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(buf, (3, 5000), (2 ** 30, 1))
    z, tokens = _rows(3, 5000, "bf16", 8)
    view.copy_(z)
    a, b = dcr.token_scores(view, tokens.cuda(), top=4), dcr.token_scores(z.cuda(), tokens.cuda(), top=4)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    one = torch.ones(3, device="cuda")
    exp = dcr.token_scores_grad(z.cuda(), tokens.cuda(), b.stats, one, one)
    assert torch.equal(dcr.token_scores_grad(view, tokens.cuda(), b.stats, one, one, out=view), exp)


def test_streams_and_graphs():
    z, tokens = _rows(5, 40000, "bf16", 6)
    z, tokens, one = z.cuda(), tokens.cuda(), torch.ones(5, device="cuda")
    exp = dcr.token_scores(z, tokens, top=7)
    grad = dcr.token_scores_grad(z, tokens, exp.stats, one, one)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dcr.token_scores(z, tokens, top=7, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, exp))
    graph = torch.cuda.CUDAGraph()
    into = z.clone()
    with torch.cuda.graph(graph):
        got = dcr.token_scores(into, tokens, top=7)
        back = dcr.token_scores_grad(into, tokens, got.stats, one, one)
    for shift in (0.0, 1.0):
        into.copy_(z.roll(int(shift), 0))
        want = dcr.token_scores(into, tokens, top=7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(back, dcr.token_scores_grad(into, tokens, want.stats, one, one))
    assert torch.equal(dcr.token_scores_grad(z, tokens, exp.stats, one, one), grad)


@pytest.mark.parametrize("rows,vocab,dtype", [(2, 140001, "bf16"), (40, 70001, "f32"), (150, 33001, "f32")])
def test_clusters_that_come_and_go(rows, vocab, dtype):
    # rows of several blocks, most of them left out and gone at once, on two streams: each block's part reaches the first one
    z, tokens = _rows(rows, vocab, dtype, 2)
    every = dcr.token_scores(z.cuda(), tokens.cuda(), top=20)
    some = torch.where(torch.arange(rows) % 3 == 1, torch.full_like(tokens, -1), tokens).cuda()
    dev = z.cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [dcr.token_scores(dev, some, top=20, stream=streams[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    keep = (some >= 0).nonzero()[:, 0]
    for g in got:
        assert all(torch.equal(a[keep], b[keep]) for a, b in zip(g, every))
    exp = torch.sort(z.float(), dim=1, descending=True, stable=True)[1][:, :20]
    assert torch.equal(every.top_tokens.cpu(), exp)
