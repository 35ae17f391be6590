"""Policy loss, its gradient and token log-probabilities on the GPU against a
plain 64-bit form and against differences."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402
import ops_ref as R  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _case(rows, vocab, dtype, seed=0, pad=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    flat = (torch.randn(rows * (vocab + pad) + offset, generator=g) * 3).to(DT[dtype])
    z = flat.cuda()[offset:].reshape(rows, vocab + pad)[:, :vocab]
    tokens = torch.randint(0, vocab, (rows,), generator=g)
    lp = torch.log_softmax(z.cpu().double(), 1).gather(1, tokens[:, None])[:, 0]
    old = (lp + 0.3 * torch.randn(rows, generator=g)).float()
    ref = (lp + 0.3 * torch.randn(rows, generator=g)).float()
    adv = torch.randn(rows, generator=g)
    w = (torch.rand(rows, generator=g) >= 0.25).float() / max(rows, 1)
    return z, tokens, old, adv, w, ref


def _run(z, tokens, old, adv, w, ref, grad=True, lo=0.2, hi=0.3, kl=0.1, temp=1.0):
    dev = [t.cuda() if t is not None else None for t in (tokens, old, adv, w, ref)]
    out = dcr.policy_loss(z, dev[0], dev[1], dev[2], dev[3], ref_logp=dev[4], clip_low=lo, clip_high=hi, kl_coef=kl,
                          temperature=temp, grad=grad)
    torch.cuda.synchronize()
    return out


def _bounds(z, temp):
    """An absolute bound on the 32-bit log-probability: z / T and the logarithm round at their own size (a few units of
    2^-24 of the largest |z| / T and of lse), exponentials and their sum are relative errors of at most 2^-20 together."""
    big = float(z.double().abs().amax()) / temp
    return 2.0 ** -20 + 8 * 2.0 ** -24 * (big + math.log(z.shape[1]) + 1)


def _check(case, dtype, **kw):
    z, tokens, old, adv, w, ref = case
    temp, kl = kw.get("temp", 1.0), kw.get("kl", 0.1)
    loss, lp, grad = _run(*case, **kw)
    eloss, elp, egrad = R.policy(z.cpu(), tokens, old, adv, w, ref, kw.get("lo", 0.2), kw.get("hi", 0.3), kl, temp)
    b = _bounds(z.cpu(), temp)
    assert float((lp.cpu().double() - elp).abs().max()) <= b
    # the loss of a row moves by its slope times the error of lp, and by a few roundings of its terms
    ratio = torch.exp(elp - old.double()).clamp(max=1e6)
    size = w.double().abs() * (ratio * adv.double().abs() + kl * (torch.exp((ref.double() - elp)).clamp(max=1e6) + 2 + (ref.double() - elp).abs()) if ref is not None
                               else ratio * adv.double().abs())
    assert abs(float(loss) - float(eloss)) <= float(size.sum()) * (4 * b + 2.0 ** -20)
    if grad is not None:
        got = grad.cpu().double()
        # slope and probability each carry the error of lp; the type rounds once, and a sixteenth of its smallest normal
        tiny = {"f32": 1e-38, "bf16": 1e-38, "f16": 2.0 ** -25}[dtype]
        c = (size / temp)[:, None]
        p = egrad.abs() + 0
        bound = c * (4 * b + 2.0 ** -19) * (torch.softmax(z.cpu().double() / temp, 1) + (torch.arange(z.shape[1])[None] == tokens[:, None])) \
            + EPS[dtype] * 1.01 * p + tiny
        bad = (got - egrad).abs() > bound
        assert not bool(bad.any()), float(((got - egrad).abs() / bound).max())
        assert bool((got[w == 0] == 0).all())
    return loss, lp, grad


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (1, 2), (3, 7), (5, 31), (4, 33), (2, 256), (9, 1000), (17, 4099), (2, 8192),
                                        (3, 32771), (2, 65536), (1, 128256), (2, 131073)])
def test_sizes(dtype, rows, vocab):
    _check(_case(rows, vocab, dtype, rows + vocab), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [300001, 1200007])
def test_rows_too_long_for_the_chip(dtype, vocab):
    _check(_case(2, vocab, dtype, vocab), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 2), (8, 8), (5, 4), (2, 0)])
@pytest.mark.parametrize("vocab", [77, 2050, 9001])
def test_strides_and_alignment(dtype, pad, offset, vocab):
    _check(_case(6, vocab, dtype, pad + offset, pad=pad, offset=offset), dtype, temp=0.7)


@pytest.mark.parametrize("vocab", [50, 5003, 40000])
def test_gradient_in_place_and_into_strided_tensors(vocab):
    case = _case(6, vocab, "bf16", 4, pad=4)
    z = case[0]
    _, lp, grad = _run(*case)
    wide = torch.full((6, vocab + 3), 9.0, dtype=torch.bfloat16, device="cuda")
    _, _, g2 = _run(*case, grad=wide[:, 1:vocab + 1])
    assert torch.equal(g2, grad) and bool((wide[:, 0] == 9.0).all()) and bool((wide[:, vocab + 1:] == 9.0).all())
    _, lp3, none = _run(*case, grad=False)
    assert none is None and torch.equal(lp3, lp)
    _, lp4, g4 = _run(*case, grad=z)
    assert g4.data_ptr() == z.data_ptr() and torch.equal(z, grad) and torch.equal(lp4, lp)


def test_against_differences():
    z, tokens, old, adv, w, ref = _case(6, 23, "f32", 7)
    w[:] = 1.0
    adv[0], adv[1] = 2.0, -2.0
    _, _, grad = _run(z, tokens, old, adv, w, ref, temp=0.9)
    h = 1e-5
    zd = z.cpu().double()
    for i in range(6):
        for j in range(23):
            up, dn = zd.clone(), zd.clone()
            up[i, j] += h
            dn[i, j] -= h
            d = (R.policy(up, tokens, old, adv, w, ref, 0.2, 0.3, 0.1, 0.9)[0]
                 - R.policy(dn, tokens, old, adv, w, ref, 0.2, 0.3, 0.1, 0.9)[0]) / (2 * h)
            assert abs(float(grad[i, j]) - float(d)) <= 1e-5 * (1 + abs(float(d)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [40, 5000, 70001])
def test_left_out_rows_hold_anything(dtype, vocab):
    case = _case(8, vocab, dtype, 3)
    z, tokens, old, adv, w, ref = case
    w[:] = 0.5
    w[1], w[4] = 0.0, 0.0
    tokens[2], tokens[6] = -100, vocab
    before = _check(case, dtype)
    for bad in (float("nan"), float("inf"), float("-inf"), torch.finfo(DT[dtype]).min):
        for i in (1, 2, 4, 6):
            z[i] = bad
        old[1] = adv[1] = ref[4] = float("nan")
        after = _run(*case)
        assert all(torch.equal(a, b) for a, b in zip(before, after))
        assert bool((after[2][[1, 2, 4, 6]] == 0).all()) and bool((after[1][[1, 2, 4, 6]] == 0).all())
    # nothing left at all
    w[:] = 0
    loss, lp, grad = _run(*case)
    assert float(loss) == 0 and bool((lp == 0).all()) and int(grad.count_nonzero()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [33, 2049, 33000])
def test_masked_vocabulary(dtype, vocab):
    # -inf and the type's lowest value in most places, whole stretches among them; only the token left
    case = _case(5, vocab, dtype, 11)
    z, tokens = case[0], case[1]
    w = case[4]
    w[:] = 0.2
    low = torch.finfo(DT[dtype]).min
    keep = [z[i, tokens[i]].clone() for i in range(5)]
    z[0, vocab // 3:] = float("-inf")
    z[1, :vocab // 2] = low
    z[2, 1:] = float("-inf")
    z[3, ::2] = float("-inf")
    z[4] = float("-inf")
    for i in range(5):
        z[i, tokens[i]] = keep[i]
    loss, lp, grad = _run(*case, temp=1.0)
    eloss, elp, egrad = R.policy(z.cpu(), *case[1:], 0.2, 0.3, 0.1, 1.0)
    assert bool(torch.isfinite(lp).all()) and float(lp[4]) == 0.0
    assert float((lp.cpu().double() - elp).abs().max()) <= 2.0 ** -19 + 64 * 2.0 ** -24
    assert float((grad.cpu().double() - egrad).abs().max()) <= float(egrad.abs().max()) * (2.0 ** -18 + EPS[dtype])
    assert bool((grad.cpu()[torch.isneginf(z.cpu())] == 0).all())
    # the sampled token itself is masked out: its log-probability is -inf, as in 64 bits
    z[0, tokens[0]] = float("-inf")
    assert float(dcr.token_logprobs(z, tokens.cuda())[0]) == float("-inf")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [30, 5000, 70000])
def test_constant_rows_of_any_size(dtype, vocab):
    # the type's lowest and highest value, and others: softmax is uniform whatever the constant
    for v in (torch.finfo(DT[dtype]).min, torch.finfo(DT[dtype]).max, 0.0, -50.0):
        z = torch.full((2, vocab), v, dtype=DT[dtype], device="cuda")
        t = torch.tensor([0, vocab - 1], device="cuda")
        one = torch.ones(2, device="cuda")
        _, lp, grad = dcr.policy_loss(z, t, -one, one, one, clip_high=1e9)
        assert float((lp + math.log(vocab)).abs().max()) <= 1e-5
        assert bool(torch.isfinite(grad).all())


def test_non_finite_logits_show():
    for vocab in (64, 9000, 70000):
        z = torch.zeros(4, vocab, device="cuda")
        z[1, 5], z[2, 7], z[3] = float("nan"), float("inf"), float("-inf")
        t = torch.zeros(4, dtype=torch.int64, device="cuda")
        lp = dcr.token_logprobs(z, t).cpu()
        assert abs(float(lp[0]) + math.log(vocab)) <= 1e-5
        assert math.isnan(lp[1]) and float(lp[2]) == float("-inf") and math.isnan(lp[3])


def test_clipping_and_no_kl():
    z, tokens, old, adv, w, ref = _case(40, 100, "f32", 21)
    w[:] = 1.0 / 40
    old += torch.linspace(-1, 1, 40)       # ratios on both sides of the clip, with both signs of the advantage
    adv[::2] = adv[::2].abs()
    adv[1::2] = -adv[1::2].abs()
    case = (z, tokens, old, adv, w, None)
    loss, lp, grad = _check(case, "f32", kl=0.0, lo=0.1, hi=0.4)
    ratio = torch.exp(lp.cpu() - old)
    stopped = ((adv > 0) & (ratio > 1.41)) | ((adv < 0) & (ratio < 0.89))
    assert bool(stopped.any()) and bool((grad.cpu()[stopped] == 0).all())
    assert bool((grad.cpu()[~stopped & (ratio > 0.91) & (ratio < 1.39)].abs().amax(1) > 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab", [(1, 5), (1, 4096), (7, 32771), (64, 1000), (1, 128256), (8, 128256), (300, 17), (1, 900001)])
def test_token_logprobs(dtype, rows, vocab):
    z, tokens = _case(rows, vocab, dtype, vocab, pad=1)[:2]
    exp = torch.log_softmax(z.cpu().double() / 0.8, 1).gather(1, tokens[:, None])[:, 0]
    lp = dcr.token_logprobs(z, tokens.cuda(), temperature=0.8)
    assert float((lp.cpu().double() - exp).abs().max()) <= _bounds(z.cpu(), 0.8)
    t = tokens.clone()
    t[0] = vocab
    assert float(dcr.token_logprobs(z, t.cuda())[0]) == 0.0


def test_no_rows_and_many_rows():
    z = torch.empty(0, 50, device="cuda")
    e = torch.empty(0, device="cuda")
    loss, lp, grad = dcr.policy_loss(z, torch.empty(0, dtype=torch.int64, device="cuda"), e, e, e)
    assert float(loss) == 0.0 and lp.shape == (0,) and grad.shape == (0, 50)
    _check(_case(3001, 11, "bf16", 5), "bf16")


def test_past_32_bit_offsets():
    # 2^32 + vocab values: the last row's offset does not fit 32 bits
    rows, vocab = 32769, 131072
    z = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    z[-1] = torch.linspace(-4, 4, vocab, device="cuda").to(torch.bfloat16)
    tokens = torch.full((rows,), 5, dtype=torch.int64, device="cuda")
    w = torch.zeros(rows, device="cuda")
    w[-1] = w[0] = 1.0
    one, old = torch.ones(rows, device="cuda"), torch.full((rows,), -11.0, device="cuda")
    loss, lp, grad = dcr.policy_loss(z, tokens, old, one, w, grad=z)
    assert abs(float(lp[0]) + math.log(vocab)) <= 1e-5
    zl = torch.linspace(-4, 4, vocab).to(torch.bfloat16)[None]
    _, elp, egrad = R.policy(zl, tokens[:1], old[:1], one[:1], w[:1], None, 0.2, 0.2, 0.0, 1.0)
    assert abs(float(lp[-1]) - float(elp)) <= 1e-5
    assert float((z[-1:].cpu().double() - egrad).abs().max()) <= float(egrad.abs().max()) * 2.0 ** -8


def test_same_every_time_on_another_stream_and_in_a_graph():
    case = [t.cuda() for t in _case(50, 6000, "bf16", 2)]
    z, tokens, old, adv, w, ref = case
    call = lambda **kw: dcr.policy_loss(z, tokens, old, adv, w, ref_logp=ref, kl_coef=0.1, **kw)  # noqa: E731
    first = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for st in (None, s, s.cuda_stream):
        got = call(stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    adv.neg_()
    g.replay()
    again = call()
    assert all(torch.equal(a, b) for a, b in zip(out, again)) and not torch.equal(out[2], first[2])
