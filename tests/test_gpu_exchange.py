"""Rows into the experts' order and back, and the gradients of both ways."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402
from step_ref import DT, EPS, TINY, expert_order  # noqa: E402


def _route(tokens, experts, k, seed, masked=0.0):
    """A Route on the CPU: distinct experts a token, some tokens and slots without."""
    g = torch.Generator().manual_seed(seed)
    chosen = torch.stack([torch.randperm(experts, generator=g)[:k] for _ in range(tokens)]) if tokens else torch.zeros(0, k, dtype=torch.int64)
    if masked:
        chosen[torch.rand(tokens, generator=g) < masked] = -1
        chosen[torch.rand(tokens, k, generator=g) < masked / 4] = -1
    weights = torch.where(chosen >= 0, torch.rand(tokens, k, generator=g), torch.zeros(tokens, k))
    offsets, order, positions = expert_order(chosen, experts)
    return dcr.Route(chosen.int(), weights, offsets.int(), order.int(), positions.int())


def _cuda(r):
    return dcr.Route(*(x.cuda() for x in r))


def _randn(rows, cols, dtype, seed):
    return torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])


SIZES = [(1, 1, 1, 1), (3, 4, 2, 7), (5, 8, 8, 8), (64, 64, 8, 100), (33, 40, 3, 2056), (130, 9, 1, 6144), (7, 33, 32, 515)]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32"), ("f32", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("tokens,experts,k,cols", SIZES)
def test_gather_and_combine(tokens, experts, k, cols, dtype, out):
    r = _route(tokens, experts, k, cols, masked=0.3)
    x, y = _randn(tokens, cols, dtype, 1), _randn(tokens * k, cols, dtype, 2)
    total = int(r.offsets[-1])
    slot = r.order[:total].long()
    y[total:] = float("nan")        # rows that no token has
    dev = _cuda(r)
    into = torch.full((tokens * k, cols), 7.0, dtype=DT[out], device="cuda")
    got = dcr.experts_gather(x.cuda(), dev, out=into)
    assert got is into
    assert torch.equal(got.cpu()[:total], x[slot // k].to(DT[out])) and bool((got[total:] == 7).all())
    got = dcr.experts_gather(x.cuda(), dev, weighted=True, dtype=DT[out]).cpu()[:total]
    assert torch.equal(got, (x[slot // k].float() * r.weights.reshape(-1)[slot][:, None]).to(DT[out]))
    for weighted in (True, False):
        got = dcr.experts_combine(y.cuda(), dev, weighted=weighted, dtype=DT[out])
        assert got.dtype == DT[out]
        w = r.weights.reshape(-1)[slot].double() if weighted else torch.ones(total, dtype=torch.float64)
        part = y[:total].double() * w[:, None]
        exp = torch.zeros(tokens, cols, dtype=torch.float64).index_add_(0, slot // k, part)
        size = torch.zeros(tokens, cols, dtype=torch.float64).index_add_(0, slot // k, part.abs())
        bound = size * k * 2.0 ** -24 + exp.abs() * 1.01 * EPS[out] + TINY[out]
        off = (got.cpu().double() - exp).abs()
        assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("dtype,grads", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("tokens,experts,k,cols", SIZES)
def test_gradients_of_combine(tokens, experts, k, cols, dtype, grads):
    r = _route(tokens, experts, k, cols, masked=0.3)
    y, g = _randn(tokens * k, cols, dtype, 2), _randn(tokens, cols, grads, 3)
    total = int(r.offsets[-1])
    slot = r.order[:total].long()
    y[total:] = float("nan")
    into = torch.full((tokens * k, cols), 7.0, dtype=DT[dtype], device="cuda")
    by_y, by_w = dcr.experts_combine_grad(y.cuda(), _cuda(r), g.cuda(), out=into)
    assert by_y is into and bool((by_y[total:] == 7).all())
    w = r.weights.reshape(-1)[slot]
    assert torch.equal(by_y.cpu()[:total], (g[slot // k].float() * w[:, None]).to(DT[dtype]))
    exp, size = (torch.zeros(tokens * k, dtype=torch.float64) for _ in range(2))
    exp[slot] = (y[:total].double() * g[slot // k].double()).sum(1)
    size[slot] = (y[:total].double() * g[slot // k].double()).abs().sum(1)
    # a thread adds up at most 8 products of every 2048 columns, then threads in pairs and warps
    bound = size * (8 * (cols // 2048 + 1) + 16) * 2.0 ** -24
    off = (by_w.cpu().double().reshape(-1) - exp).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    assert bool((by_w.cpu()[r.positions < 0] == 0).all())


@pytest.mark.parametrize("dtype,cols", [("bf16", 8192), ("bf16", 1000), ("f32", 333), ("f16", 8), ("f32", 4100)])
def test_gradients_of_combine_of_many_tokens(dtype, cols):
    # enough tokens for a warp each: a thread adds up at most 8 products of every 256 columns, then threads in pairs
    tokens, k = 2500, 2
    r = _route(tokens, 7, k, cols, masked=0.2)
    y, g = _randn(tokens * k, cols, dtype, 2), _randn(tokens, cols, dtype, 3)
    total = int(r.offsets[-1])
    slot = r.order[:total].long()
    y[total:] = float("nan")
    into = torch.full((tokens * k, cols), 7.0, dtype=DT[dtype], device="cuda")
    by_y, by_w = dcr.experts_combine_grad(y.cuda(), _cuda(r), g.cuda(), out=into)
    assert bool((by_y[total:] == 7).all())
    assert torch.equal(by_y.cpu()[:total], (g[slot // k].float() * r.weights.reshape(-1)[slot][:, None]).to(DT[dtype]))
    exp, size = (torch.zeros(tokens * k, dtype=torch.float64) for _ in range(2))
    part = y[:total].double() * g[slot // k].double()
    exp[slot], size[slot] = part.sum(1), part.abs().sum(1)
    off = (by_w.cpu().double().reshape(-1) - exp).abs()
    assert bool((off <= size * (8 * (cols // 256 + 1) + 8) * 2.0 ** -24).all())
    assert bool((by_w.cpu()[r.positions < 0] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [16, 40, 1001])
def test_strides(cols, dtype):
    # columns of wider buffers at odd offsets: the same values, and nothing else is touched
    tokens, k = 21, 4
    r = _cuda(_route(tokens, 8, k, 5))
    x, y, g = _randn(tokens, cols, dtype, 1).cuda(), _randn(tokens * k, cols, dtype, 2).cuda(), _randn(tokens, cols, dtype, 3).cuda()
    exp = dcr.experts_gather(x, r), dcr.experts_combine(y, r), dcr.experts_combine_grad(y, r, g)

    def wide(m, at):
        buf = torch.full((m.shape[0], cols + 11), 9.0, dtype=m.dtype, device="cuda")
        buf[:, at:at + cols] = m
        return buf, buf[:, at:at + cols]

    for at in (1, 8):
        bufs = [wide(m, at) for m in (x, y, g)]
        (_, vx), (_, vy), (_, vg) = bufs
        outs = [wide(torch.zeros_like(m), 3) for m in (y, x, y)]
        dcr.experts_gather(vx, r, out=outs[0][1])
        dcr.experts_combine(vy, r, out=outs[1][1])
        _, by_w = dcr.experts_combine_grad(vy, r, vg, out=outs[2][1])
        assert torch.equal(outs[0][1], exp[0]) and torch.equal(outs[1][1], exp[1]) and torch.equal(outs[2][1], exp[2][0])
        assert torch.allclose(by_w, exp[2][1], rtol=1e-4, atol=1e-4)
        for buf, v in outs:
            v.fill_(9.0)
            assert bool((buf == 9).all())


def test_positions_outside_are_passed_over():
    # what a wrong table holds is neither read nor written
    tokens, k, cols = 3, 2, 24
    r = _cuda(_route(tokens, 4, k, 1))
    bad = r.positions.clone()
    bad[0, 0], bad[1, 1], bad[2, 0] = tokens * k, -5, 2 ** 31 - 1
    q = r._replace(positions=bad)
    x, y = _randn(tokens, cols, "f32", 1).cuda(), _randn(tokens * k, cols, "f32", 2).cuda()
    out = dcr.experts_gather(x, q, out=torch.zeros(tokens * k, cols, device="cuda"))
    assert int(out.any(1).sum()) == 3
    s = dcr.experts_combine(y, q, weighted=False)
    exp = y[r.positions.long()]
    exp[0, 0] = exp[1, 1] = exp[2, 0] = 0
    assert torch.equal(s, exp.sum(1))


def test_empty_and_large():
    r = _cuda(_route(0, 4, 2, 1))
    assert dcr.experts_gather(torch.empty(0, 5, device="cuda"), r).shape == (0, 5)
    assert dcr.experts_combine(torch.empty(0, 5, device="cuda"), r).shape == (0, 5)
    r = _cuda(_route(3, 4, 2, 1))
    assert dcr.experts_combine(torch.empty(6, 0, device="cuda"), r).shape == (3, 0)
    by_y, by_w = dcr.experts_combine_grad(torch.empty(6, 0, device="cuda"), r, torch.empty(3, 0, device="cuda"))
    assert by_y.shape == (6, 0) and bool((by_w == 0).all())
    # rows whose offsets pass 32 bits
    tokens, k, cols = 9, 2, 1000
    r = _cuda(_route(tokens, 4, k, 1))
    buf = torch.zeros(2 ** 28 * (tokens * k - 1) + cols, dtype=torch.bfloat16, device="cuda")
    rows = torch.as_strided(buf, (tokens * k, cols), (2 ** 28, 1))
    x = _randn(tokens, cols, "bf16", 1).cuda()
    dcr.experts_gather(x, r, out=rows)
    assert torch.equal(rows, dcr.experts_gather(x, r))
    assert torch.equal(dcr.experts_combine(rows, r), dcr.experts_combine(rows.contiguous(), r))
    by_y, by_w = dcr.experts_combine_grad(rows.contiguous(), r, x)
    got = dcr.experts_combine_grad(rows, r, x, out=rows)
    assert torch.equal(got[0], by_y) and torch.equal(got[1], by_w)


def test_graphs_and_streams():
    r = _cuda(_route(50, 16, 4, 1))
    x, g = _randn(50, 512, "bf16", 1).cuda(), _randn(50, 512, "bf16", 2).cuda()

    def step():
        rows = dcr.experts_gather(x, r)
        return (rows, dcr.experts_combine(rows, r)) + dcr.experts_combine_grad(rows, r, g)

    exp = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, exp))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    rows = dcr.experts_gather(x, r, stream=s)
    out = dcr.experts_combine(rows, r, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(rows, exp[0]) and torch.equal(out, exp[1])
