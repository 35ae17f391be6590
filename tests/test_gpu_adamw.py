"""The trainer's step: AdamW bit for bit against the same roundings on the CPU
and against 64 bits, moments in 8 bits, and the norm of all gradients."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402
import step_ref as R  # noqa: E402
from step_ref import DT, EPS  # noqa: E402

LR, BETAS, E, DECAY = 3e-4, (0.9, 0.999), 1e-8, 0.1


def _randn(n, seed, std=1.0):
    return torch.randn(n, generator=torch.Generator().manual_seed(seed)) * std


def _flat(sizes, dtype, seed, std, gap):
    """Tensors one behind another in a buffer, `gap` values apart."""
    buf = _randn(sum(sizes) + gap * (len(sizes) + 1), seed, std).to(dtype)
    out, at = [], gap
    for n in sizes:
        out.append(buf[at:at + n])
        at += n + gap
    return buf, out


def _on_gpu(buf, views):
    dev = buf.cuda()
    return dev, [dev[v.storage_offset():v.storage_offset() + v.numel()] for v in views]


def _states(sizes, bits, seed):
    """Moments as some steps leave them, on the CPU."""
    out = []
    for i, n in enumerate(sizes):
        m, v = _randn(n, seed + i, 1e-3), _randn(n, seed + 1000 + i, 1e-3).square()
        if bits == 32:
            out.append((m, v))
        else:
            half = torch.full((n,), 0x8000)
            out.append(R.to8(m, half, False) + R.to8(v.sqrt(), half, True))
    return out


def _gpu_states(states, bits, gap):
    if not gap:
        return [(dcr.AdamState32 if bits == 32 else dcr.AdamState8)(*(x.cuda() for x in s)) for s in states]
    # at odd places of a larger tensor
    def put(x):
        return torch.cat([x.new_zeros(gap), x]).cuda()[gap:]
    return [(dcr.AdamState32 if bits == 32 else dcr.AdamState8)(*(put(x) for x in s)) for s in states]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("w,g,c", [("f32", "bf16", "bf16"), ("f32", "f32", None), ("bf16", "f16", "f32"), ("f16", "f32", "f16"), ("f32", "f16", "f32")])
@pytest.mark.parametrize("sizes,gap", [([1], 0), ([256, 257, 255, 1, 2048], 0), ([70000, 0, 3, 511], 0), ([301, 64, 1000, 2049], 1), ([8, 4096], 8)])
def test_steps_bit_for_bit(sizes, gap, w, g, c, bits):
    wb, ws = _flat(sizes, DT[w], 1, 0.02, gap)
    gb, gs = _flat(sizes, DT[g], 2, 1e-3, gap)
    wd, wv = _on_gpu(wb, ws)
    gd, gv = _on_gpu(gb, gs)
    states = _states(sizes, bits, 3)
    dev = _gpu_states(states, bits, gap)
    cb = None if c is None else torch.full((len(wb),), 5.0, dtype=DT[c])
    cd, cv = (None, None) if c is None else _on_gpu(cb, [cb[x.storage_offset():x.storage_offset() + x.numel()] for x in ws])
    for step in (1, 2, 1000):
        dcr.adamw_step(wv, gv, dev, step, LR, betas=BETAS, eps=E, weight_decay=DECAY, copies=cv, seed=7)
        first = 0
        for i, n in enumerate(sizes):
            rnd = R.random_bits(7, step, first, n) if bits == 8 else None
            new, copy, states[i] = R.adamw(ws[i], gs[i], states[i], None if c is None else DT[c], step, LR, BETAS, E, DECAY, bits=rnd)
            ws[i].copy_(new)
            if c is not None:
                cb[ws[i].storage_offset():ws[i].storage_offset() + n] = copy
            first += n
        assert torch.equal(wd.cpu(), wb)          # the gaps stay as they were, too
        assert c is None or torch.equal(cd.cpu(), cb)
        for a, b in zip(dev, states):
            for x, y in zip(a, b):
                assert torch.equal(x.cpu(), y)
    assert torch.equal(gd.cpu(), gb)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_thousand_tensors(bits):
    sizes = [1 + i * 37 % 700 for i in range(1000)]
    wb, ws = _flat(sizes, torch.float32, 1, 0.02, 0)
    gb, gs = _flat(sizes, torch.bfloat16, 2, 1e-3, 0)
    wd, wv = _on_gpu(wb, ws)
    gd, gv = _on_gpu(gb, gs)
    states = _states(sizes, bits, 3)
    dev = _gpu_states(states, bits, 0)
    dcr.adamw_step(wv, gv, dev, 5, LR, betas=BETAS, eps=E, weight_decay=DECAY, seed=1)
    first = 0
    for i, n in enumerate(sizes):
        rnd = R.random_bits(1, 5, first, n) if bits == 8 else None
        new, _, s = R.adamw(ws[i], gs[i], states[i], None, 5, LR, BETAS, E, DECAY, bits=rnd)
        assert torch.equal(wv[i].cpu(), new) and all(torch.equal(a.cpu(), b) for a, b in zip(dev[i], s))
        first += n


def test_against_64_bits():
    n = 5000
    w, g = _randn(n, 1, 0.02), _randn(n, 2, 1e-3)
    m, v = _randn(n, 3, 1e-3), _randn(n, 4, 1e-3).square()
    wd = w.cuda()
    state = dcr.AdamState32(m.cuda(), v.cuda())
    dcr.adamw_step([wd], [g.cuda()], [state], 10, LR, betas=BETAS, eps=E, weight_decay=DECAY, grad_scale=0.5)
    g64 = g.double() * 0.5
    m64, v64 = BETAS[0] * m.double() + (1 - BETAS[0]) * g64, BETAS[1] * v.double() + (1 - BETAS[1]) * g64 ** 2
    step = m64 / (1 - BETAS[0] ** 10) / (torch.sqrt(v64 / (1 - BETAS[1] ** 10)) + E) * LR
    exp = w.double() * (1 - LR * DECAY) - step
    # each sum's parts are rounded three times at most
    size = BETAS[0] * m.double().abs() + (1 - BETAS[0]) * g64.abs()
    assert bool(((state.m.cpu().double() - m64).abs() <= size * 2.0 ** -22).all())
    assert bool(((state.v.cpu().double() - v64).abs() <= v64 * 2.0 ** -21).all())
    bound = w.double().abs() * 2.0 ** -22 + size / (1 - BETAS[0] ** 10) / (torch.sqrt(v64 / (1 - BETAS[1] ** 10)) + E) * LR * 2.0 ** -20
    assert bool(((wd.cpu().double() - exp).abs() <= bound).all())


def test_rounding_of_8_bit_moments_keeps_the_mean():
    # many rounds of one moment: the mean of what is read back is the moment; an error of at most one step of e4m3 (an eighth
    # of the value, and no less than 2^-9 of the scale) has a variance of at most a quarter of its square
    n, rounds = 512, 400
    m = _randn(n, 1, 1e-3)
    m[0] = 1e-2
    total = torch.zeros(n, dtype=torch.float64)
    zero8 = torch.zeros(n, dtype=torch.uint8)
    for seed in range(rounds):
        # beta1 = 0: the new first moment is the gradient itself
        s = dcr.AdamState8(zero8.cuda(), torch.zeros(2, device="cuda"), zero8.cuda(), torch.zeros(2, device="cuda"))
        dcr.adamw_step([torch.zeros(n, device="cuda")], [m.cuda()], [s], 1, LR, betas=(0.0, 0.9), seed=seed)
        total += R.from8(s.m.cpu(), s.m_scale.cpu()).double()
    scale = torch.stack([m[:256].abs().amax(), m[256:].abs().amax()]).repeat_interleave(256).double() / 448
    step = torch.maximum(m.double().abs() / 8, scale * 2.0 ** -9)
    off = (total / rounds - m.double()).abs()
    assert bool((off <= 6 * step / 2 / math.sqrt(rounds) + step * 2.0 ** -16).all()), float((off / step).max())


def test_8_bit_moments_move_by_less_than_a_step():
    # without gradients sqrt(v) falls by the square root of beta2 each time, far less than half a step of e4m3; over many
    # values it does so on average (the variance of a step's rounding is at most a quarter of the square of an eighth)
    n, steps = 1 << 16, 100
    v = torch.full((n,), 1e-3)
    v[::256] = 4e-3                        # the scale's; these are rounded like any other
    half = torch.full((n,), 0x8000)
    codes, scale = R.to8(v, half, True)
    start = R.from8(codes, scale).double()
    z8 = torch.zeros(n, dtype=torch.uint8).cuda()
    s = dcr.AdamState8(z8, torch.zeros(n // 256, device="cuda"), codes.cuda(), scale.cuda())
    w, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    for step in range(1, steps + 1):
        dcr.adamw_step([w], [g], [s], step, LR, betas=BETAS, seed=3)
    end = R.from8(s.v.cpu(), s.v_scale.cpu()).double()
    keep = torch.arange(n) % 256 != 0
    ratio = float(end[keep].sum() / start[keep].sum())
    exp = BETAS[1] ** (steps / 2)
    assert abs(ratio - exp) <= 6 * (1 / 16) * math.sqrt(steps / int(keep.sum())) + 1e-3, (ratio, exp)


def test_a_small_moment_never_makes_a_large_step():
    # second moments far below their block's largest: kept above 0, so that no step is first moment over eps
    n = 256
    m, v = torch.full((n,), 1e-9), torch.full((n,), 1e-9)
    m[0] = v[0] = 1.0
    half = torch.full((n,), 0x8000)
    state = dcr.AdamState8(*(x.cuda() for x in R.to8(m, half, False) + R.to8(v, half, True)))
    w = torch.zeros(n, device="cuda")
    g = torch.full((n,), 1e-9, device="cuda")
    for step in range(1, 30):
        dcr.adamw_step([w], [g], [state], 1000 + step, 1e-3, betas=BETAS, seed=step)
    # |m| / sqrt(v) <= (one step of m's block) / (one step of v's block) of equal scales, and the bias correction is near 1
    assert float(w.abs().max()) <= 30 * 1e-3 * 4
    assert bool((R.from8(state.v.cpu(), state.v_scale.cpu()) > 0).all())


def test_zero_and_nonfinite_gradients_in_8_bits():
    n = 600
    s = dcr.adamw_states([torch.zeros(n, device="cuda")], 8)
    assert type(s[0]) is dcr.AdamState8 and s[0].m_scale.numel() == 3
    w = torch.ones(n, device="cuda")
    dcr.adamw_step([w], [torch.zeros(n, device="cuda")], s, 1, LR, betas=BETAS)
    assert bool((w == 1).all()) and int(s[0].m.count_nonzero()) == 0 and int(s[0].v.count_nonzero()) == 0
    g = torch.zeros(n, device="cuda")
    g[300] = float("inf")
    dcr.adamw_step([w], [g], s, 2, LR, betas=BETAS)
    # the block of the infinite one reads back as NaN, the others go on
    m = R.from8(s[0].m.cpu(), s[0].m_scale.cpu())
    assert bool(torch.isnan(m[256:512]).all()) and bool((m[:256] == 0).all()) and bool((m[512:] == 0).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_norm_clips_or_leaves_the_step_out(bits):
    n = 3000
    g = _randn(n, 2)
    w = _randn(n, 1).cuda()
    norm = dcr.grad_norm([g.cuda()])
    state = dcr.adamw_states([w], bits)
    copy = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    a, b = w.clone(), w.clone()
    sa, sb = dcr.adamw_states([w], bits), dcr.adamw_states([w], bits)
    dcr.adamw_step([a], [g.cuda()], sa, 1, LR, norm=norm, max_norm=0.25)
    dcr.adamw_step([b], [g.cuda()], sb, 1, LR, grad_scale=float(torch.tensor(0.25) / norm.cpu()))
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(sa[0], sb[0]))
    # below the bound, or without one, the gradients stay as they are
    a, b = w.clone(), w.clone()
    sa, sb = dcr.adamw_states([w], bits), dcr.adamw_states([w], bits)
    dcr.adamw_step([a], [g.cuda()], sa, 1, LR, norm=norm, max_norm=1e6)
    dcr.adamw_step([b], [g.cuda()], sb, 1, LR, norm=norm)
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(sa[0], sb[0]))
    for bad in (float("nan"), float("inf")):
        g2 = g.clone()
        g2[1234] = bad
        norm = dcr.grad_norm([g2.cuda()])
        assert not math.isfinite(float(norm))
        before = w.clone()
        dcr.adamw_step([w], [g2.cuda()], state, 1, LR, weight_decay=DECAY, copies=[copy], norm=norm, max_norm=1.0)
        assert torch.equal(w, before) and int(copy.count_nonzero()) == 0 and all(int(x.count_nonzero()) == 0 for x in state[0])


@pytest.mark.parametrize("bits", [32, 8])
def test_step_and_rate_on_the_device_and_graphs(bits):
    n = 5000
    g, w0 = _randn(n, 2, 1e-3).cuda(), _randn(n, 1, 0.02).cuda()
    step, lr = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, device="cuda")
    w = w0.clone()
    state = dcr.adamw_states([w], bits)
    copy = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    step.fill_(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = dcr.grad_norm([g])
        dcr.adamw_step([w], [g], state, step, lr, betas=BETAS, weight_decay=DECAY, copies=[copy], norm=norm, max_norm=0.01, seed=5)
        step += 1
    w.copy_(w0)
    for x in state[0]:
        x.zero_()
    e, es = w0.clone(), dcr.adamw_states([w], bits)
    step.fill_(1)
    for i in range(1, 6):
        rate = LR / i
        lr.fill_(rate)
        graph.replay()
        dcr.adamw_step([e], [g], es, i, float(torch.tensor(rate)), betas=BETAS, weight_decay=DECAY, norm=dcr.grad_norm([g]), max_norm=0.01, seed=5)
        torch.cuda.synchronize()
        # the corrections are computed in 32 bits there: a few roundings of the step's own size
        off = (w - e).abs().double()
        assert float((off - (e.abs() * 2.0 ** -23 + i * LR * 4 * 2.0 ** -21)).max()) <= 0
        assert all(torch.equal(x, y) for x, y in zip(state[0], es[0]))
        assert torch.equal(copy, w.bfloat16())
    assert int(step) == 6


def test_streams():
    n = 40000
    g, w = _randn(n, 2, 1e-3).cuda(), _randn(n, 1, 0.02).cuda()
    a, b = w.clone(), w.clone()
    sa, sb = dcr.adamw_states([w], 8), dcr.adamw_states([w], 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    norm = dcr.grad_norm([g], stream=s)
    dcr.adamw_step([a], [g], sa, 1, LR, norm=norm, max_norm=0.1, stream=s)
    s.synchronize()
    dcr.adamw_step([b], [g], sb, 1, LR, norm=dcr.grad_norm([g]), max_norm=0.1)
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(sa[0], sb[0]))


def test_more_values_than_32_bits_count():
    n = 2 ** 32 + 777
    w, g = torch.empty(n, dtype=torch.bfloat16, device="cuda"), torch.empty(n, dtype=torch.bfloat16, device="cuda")
    ends = [slice(0, 1024), slice(2 ** 32 - 512, 2 ** 32 + 777)]
    w.fill_(0.5)
    g.fill_(1e-3)
    hw, hg = [], []
    for i, e in enumerate(ends):
        k = e.stop - e.start
        hw.append(_randn(k, i, 0.02).bfloat16())
        hg.append(_randn(k, 10 + i, 1e-3).bfloat16())
        w[e], g[e] = hw[-1].cuda(), hg[-1].cuda()
    s = dcr.adamw_states([w], 8)
    dcr.adamw_step([w], [g], s, 1, 1e-2, betas=BETAS, seed=9)
    for e, a, b in zip(ends, hw, hg):
        k, blocks = e.stop - e.start, slice(e.start // 256, -(-e.stop // 256))
        z = torch.zeros(k, dtype=torch.uint8)
        new, _, st = R.adamw(a, b, (z, torch.zeros(blocks.stop - blocks.start)) * 2, None, 1, 1e-2, BETAS, 1e-8, 0.0, bits=R.random_bits(9, 1, e.start, k))
        assert torch.equal(w[e].cpu(), new)
        assert torch.equal(s[0].m[e].cpu(), st[0]) and torch.equal(s[0].m_scale[blocks].cpu(), st[1])
        assert torch.equal(s[0].v[e].cpu(), st[2]) and torch.equal(s[0].v_scale[blocks].cpu(), st[3])
    del s, w
    g.fill_(1.0)
    # every square is 1, and the sum is exact
    assert float(dcr.grad_norm([g])) == float(torch.tensor(math.sqrt(n)))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes,gap", [([1], 0), ([0], 0), ([3, 0, 17], 1), ([16384, 16385, 5], 0), ([1000003], 3), ([100 + i for i in range(1500)], 1)])
def test_norm(sizes, gap, dtype):
    buf, views = _flat(sizes, DT[dtype], 4, 2.0, gap)
    _, dev = _on_gpu(buf, views)
    exp = math.sqrt(sum(float(v.double().square().sum()) for v in views))
    got = dcr.grad_norm(dev)
    assert got.shape == () and got.dtype == torch.float32
    # at most 64 squares of 32 bits one after another, of which the root halves the error
    assert abs(float(got) - exp) <= exp * 70 * 2.0 ** -25
    assert torch.equal(got, dcr.grad_norm(dev))
