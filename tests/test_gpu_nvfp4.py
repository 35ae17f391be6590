"""NVFP4 quantisation and products on the GPU against plain 64-bit forms."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402
import ops_ref as R  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# the most that rounding to a type of 24, 8 or 11 significant bits changes a value by, relative to it
EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _x(rows, cols, dtype, seed=0, std=1.0, pad=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    flat = torch.randn(rows * (cols + pad) + offset, generator=g) * std
    # the same layout on the device: rows cols + pad apart, from element `offset` on
    dev = flat.to(DT[dtype]).cuda()
    x = dev[offset:].reshape(rows, cols + pad)[:, :cols]
    return x


def _check(x, per_row=False, scale=None, values=None):
    q, v = dcr.nvfp4_quantize(x, scale=scale, per_row=per_row, values=None if values is None else DT[values])
    torch.cuda.synchronize()
    h = x.cpu()
    fin = torch.where(torch.isfinite(h.double()), h.double().abs(), 0.0)
    if scale is not None:
        t = scale.cpu().double()
    else:
        t = R.scale32(fin.amax(1) if per_row else fin.amax().reshape(1))
        assert torch.equal(q.scale.cpu().double(), t)
    codes, sb, val = R.quantize(h, t)
    assert torch.equal(q.scales.cpu(), sb)
    nan = (sb == 0x7F).repeat_interleave(16, 1)
    got = R.unpack(q.codes.cpu())
    assert torch.equal(got[~nan], codes[~nan])
    if values is not None:
        exp = val.float().to(DT[values])     # one rounding: a code times s t fits 64 bits, then 32, then the type
        assert torch.equal(torch.isnan(v.cpu()), nan)
        assert torch.equal(v.cpu()[~nan], exp[~nan])
    return q


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 48), (3, 32), (5, 1040), (33, 512), (2, 16384 + 16), (1, 65536), (700, 16)])
@pytest.mark.parametrize("per_row", [False, True])
def test_quantise_sizes(dtype, rows, cols, per_row):
    _check(_x(rows, cols, dtype, rows * cols), per_row=per_row, values="bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("values", [None, "f32", "bf16", "f16"])
def test_quantise_values_types(dtype, values):
    _check(_x(9, 272, dtype, 3), values=values)
    _check(_x(9, 272, dtype, 4), values=values, per_row=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 0), (4, 2), (16, 16), (0, 8)])
def test_quantise_strides_and_alignment(dtype, pad, offset):
    for per_row in (False, True):
        _check(_x(7, 544, dtype, pad + offset, pad=pad, offset=offset), per_row=per_row, values="f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantise_given_scale(dtype):
    x = _x(20, 128, dtype, 5)
    for t in (1.0, 2.0 ** -12, 1e-3, 1e-30, 1e30, 3e-45):
        _check(x, scale=torch.tensor([t], device="cuda"), values="f32")


def test_quantise_ties_and_every_scale():
    # with t = 1 and a block maximum of 6 s every e4m3 scale s occurs, and multiples of s / 4 hit every tie
    s = R.e4m3_table()[1:].float()
    step = torch.arange(16, dtype=torch.float32) * 0.25
    block = torch.cat([step[None, :15] * s[:, None], 6 * s[:, None]], 1)
    sign = torch.where(torch.arange(16) % 3 == 0, -1.0, 1.0)
    _check((block * sign).cuda().contiguous(), scale=torch.ones(1, device="cuda"), values="f32")


@pytest.mark.parametrize("per_row", [False, True])
def test_quantise_zeros_nan_inf_and_extremes(per_row):
    x = torch.randn(6, 96, generator=torch.Generator().manual_seed(1))
    x[0] = 0.0
    x[1, 3], x[1, 20], x[1, 40] = float("nan"), float("inf"), float("-inf")
    x[2] = float("nan")
    x[3] = float("inf")
    x[4] *= 1e-42
    x[5, :16], x[5, 16:32], x[5, 32] = -0.0, 1e-38, 3e38
    _check(x.cuda(), per_row=per_row, values="f32")
    _check(torch.zeros(4, 32, device="cuda"), per_row=per_row, values="bf16")
    _check(torch.full((2, 32), float("nan"), device="cuda"), per_row=per_row)
    _check(torch.full((2, 32), 1e-45, device="cuda"), per_row=per_row, values="f32")


def test_quantise_into_arena_views_and_empty():
    x = _x(64, 256, "bf16", 8)
    arena = torch.full((64 * 128 + 64 * 16 + 256,), 0xEE, dtype=torch.uint8, device="cuda")
    codes, scales = arena[:8192].view(64, 128), arena[8192:9216].view(64, 16)
    t = torch.empty(1, device="cuda")
    q, v = dcr.nvfp4_quantize(x, out=dcr.Nvfp4(codes, scales, t))
    ref, _ = dcr.nvfp4_quantize(x)
    assert v is None and q.codes.data_ptr() == arena.data_ptr()
    assert torch.equal(codes, ref.codes) and torch.equal(scales, ref.scales) and torch.equal(t, ref.scale)
    assert bool((arena[9216:] == 0xEE).all())
    q, v = dcr.nvfp4_quantize(torch.empty(0, 32, device="cuda"), values=torch.float32)
    assert q.codes.shape == (0, 16) and v.shape == (0, 32)


def test_quantise_past_32_bit_offsets():
    # 2^32 + 2^20 values: the last rows lie past 32-bit element offsets
    rows, cols = 4097, 1 << 20
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.linspace(-3, 3, cols, device="cuda").to(torch.bfloat16)
    for per_row in (False, True):
        q, _ = dcr.nvfp4_quantize(x, per_row=per_row)
        ref, _ = dcr.nvfp4_quantize(x[-1:].clone(), per_row=per_row)
        assert torch.equal(q.codes[-1], ref.codes[0]) and torch.equal(q.scales[-1], ref.scales[0])
        assert int(q.scales[:-1].count_nonzero()) == 0 and int(q.codes[:-1].count_nonzero()) == 0


# ---- products -----------------------------------------------------------------------------------------------------


def _operand(rows, k, seed, per_row=False, std=1.0):
    q, _ = dcr.nvfp4_quantize(_x(rows, k, "f32", seed, std), per_row=per_row)
    return q


def _product(x, w, offsets=None):
    """y in double and the sum of the products' magnitudes, for the bounds."""
    xs, ws = R.spread(x.codes.cpu(), x.scales.cpu()), R.spread(w.codes.cpu(), w.scales.cpu())
    tx, tw = x.scale.cpu().double().reshape(-1, 1), w.scale.cpu().double()
    if offsets is None:
        return (xs @ ws.T) * tx * tw, (xs.abs() @ ws.abs().T) * tx * tw
    e = len(offsets) - 1
    n = ws.shape[0] // e
    y, mag = (torch.zeros(xs.shape[0], n, dtype=torch.float64) for _ in range(2))
    for i in range(e):
        a, b = offsets[i], offsets[i + 1]
        t = tx[a:b] if len(tx) > 1 else tx
        t = t * (tw[i] if len(tw) > 1 else tw[0])
        y[a:b] = xs[a:b] @ ws[i * n:(i + 1) * n].T * t
        mag[a:b] = xs[a:b].abs() @ ws[i * n:(i + 1) * n].abs().T * t
    return y, mag


def _close(got, y, mag, k, dtype, rows=None):
    """A sum of k products, each exact in 32 bits, in any order: the error of 32-bit sums is at most k units of 2^-24
    of the magnitudes' sum; the two scales are three more roundings; the output's type rounds once."""
    got = got.cpu().double()
    bound = (k + 4) * 2.0 ** -24 * mag + EPS[dtype] * y.abs() * 1.01 + (2.0 ** -25 if dtype == "f16" else 1e-40)
    bad = (got - y).abs() > bound
    if rows is not None:
        bad = bad[rows]
    assert not bool(bad.any()), ((got - y).abs() / bound).max()


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 7, 64), (1, 129, 256), (2, 128, 96), (3, 200, 544), (8, 64, 1024),
                                   (9, 300, 160), (16, 130, 2048), (17, 127, 320), (33, 256, 512), (64, 640, 288),
                                   (65, 40, 1056), (127, 384, 256), (128, 128, 128), (129, 129, 384), (200, 333, 224),
                                   (257, 513, 736), (300, 1, 64), (513, 260, 1280)])
def test_product_sizes(m, n, k, out):
    x, w = _operand(m, k, m + k, per_row=True), _operand(n, k, n + k, std=0.05)
    y, mag = _product(x, w)
    _close(dcr.nvfp4_matmul(x, w, dtype=DT[out]), y, mag, k, out)


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(65, 9800, 32), (128, 9984, 256), (257, 5000, 96), (300, 5121, 544), (511, 5120, 1312),
                                   (700, 3333, 2080), (1030, 2048, 288)])
def test_product_of_many_tokens(m, n, k, out):
    # enough 256 by 256 tiles for the paired blocks; sizes around the tile's, odd row lengths (no 32-byte stores)
    x, w = _operand(m, k, m + k, per_row=True), _operand(n, k, n + k, std=0.05)
    y, mag = _product(x, w)
    _close(dcr.nvfp4_matmul(x, w, dtype=DT[out]), y, mag, k, out)


@pytest.mark.parametrize("counts", [[300, 0, 90, 257, 5], [256, 256, 0, 513], [0, 0, 700], [65] * 12])
def test_experts_of_many_tokens(counts):
    n, k, m, e = 2600, 416, sum(counts), len(counts)
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    x, w = _operand(m, k, m, per_row=True), _operand(e * n, k, e)
    w = dcr.Nvfp4(w.codes, w.scales, torch.linspace(0.5, 2.0, e, device="cuda"))
    y, mag = _product(x, w, off)
    for out in ("bf16", "f32"):
        got = dcr.nvfp4_matmul(x, w, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), dtype=DT[out])
        _close(got, y, mag, k, out)
        assert torch.equal(got, dcr.nvfp4_matmul(x, w, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), dtype=DT[out]))
    dcr.ops_status()


@pytest.mark.parametrize("m", [1, 5, 40, 150, 300])
def test_product_of_a_long_k(m):
    k = 16384 + 32
    x, w = _operand(m, k, m), _operand(136, k, 2)
    y, mag = _product(x, w)
    _close(dcr.nvfp4_matmul(x, w, dtype=torch.float32), y, mag, k, "f32")


@pytest.mark.parametrize("m", [1, 20, 140, 300])
def test_product_is_the_same_every_time_and_for_every_neighbour(m):
    # a row's result does not depend on the run, on the other rows' values, or on how they are spread over calls of that size
    k, n = 1536, 1000
    x, w = _operand(m, k, 1, per_row=True), _operand(n, k, 2)
    y = dcr.nvfp4_matmul(x, w, dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(y, dcr.nvfp4_matmul(x, w, dtype=torch.float32))
    f = torch.arange(m - 1, -1, -1, device="cuda")
    x2 = dcr.Nvfp4(x.codes[f].contiguous(), x.scales[f].contiguous(), x.scale[f].contiguous())
    assert torch.equal(y[f], dcr.nvfp4_matmul(x2, w, dtype=torch.float32))


@pytest.mark.parametrize("m,n", [(3, 50), (140, 136), (270, 300)])
def test_product_output_strides(m, n):
    x, w = _operand(m, 160, 3, per_row=True), _operand(n, 160, 4)
    y = dcr.nvfp4_matmul(x, w, dtype=torch.bfloat16)
    for pad, off in ((1, 0), (8, 8), (0, 3), (5, 1)):
        flat = torch.full((m * (n + pad) + off,), 7.0, dtype=torch.bfloat16, device="cuda")
        view = flat[off:].reshape(m, n + pad)
        got = dcr.nvfp4_matmul(x, w, out=view[:, :n])
        assert got.data_ptr() == view.data_ptr() and torch.equal(got, y)
        assert bool((view[:, n:] == 7.0).all()) and bool((flat[:off] == 7.0).all())


@pytest.mark.parametrize("counts", [[0], [1], [5, 0, 3], [0, 0, 0, 1], [130, 0, 257, 1, 64, 0], [300, 300], [1] * 40,
                                    [0] * 200 + [3] + [0] * 55])
@pytest.mark.parametrize("n,k", [(72, 96), (256, 512)])
def test_experts(counts, n, k):
    m, e = sum(counts), len(counts)
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    x = _operand(max(m, 1), k, m, per_row=True)
    w = _operand(e * n, k, e)
    w = dcr.Nvfp4(w.codes, w.scales, torch.linspace(0.5, 2.0, e, device="cuda"))
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    for out in ("bf16", "f32"):
        got = torch.full((max(m, 1), n), 3.0, dtype=DT[out], device="cuda")
        dcr.nvfp4_matmul(x, w, offsets=o, out=got)
        if m == 0:
            assert bool((got == 3.0).all())
            continue
        y, mag = _product(x, w, off)
        _close(got, y, mag, k, out)


def test_experts_leave_rows_outside_and_survive_bad_offsets():
    x, w = _operand(50, 64, 1, per_row=True), _operand(4 * 40, 64, 2)
    ref, mag = _product(x, w, [10, 20, 20, 35, 45])
    y = torch.full((50, 40), 3.0, device="cuda")
    dcr.nvfp4_matmul(x, w, offsets=torch.tensor([10, 20, 20, 35, 45], dtype=torch.int32, device="cuda"), out=y)
    _close(y, ref, mag, 64, "f32", slice(10, 45))
    assert bool((y[:10] == 3.0).all()) and bool((y[45:] == 3.0).all())
    # entries outside [0, m] are cut to it, and an expert whose end lies before its start has no rows
    ref, mag = _product(x, w, [0, 30, 30, 30, 50])
    y = torch.full((50, 40), 3.0, device="cuda")
    dcr.nvfp4_matmul(x, w, offsets=torch.tensor([-7, 30, 20, 30, 1000], dtype=torch.int32, device="cuda"), out=y)
    _close(y, ref, mag, 64, "f32", slice(0, 20))
    _close(y, ref, mag, 64, "f32", slice(30, 50))


def test_product_nan_and_zero_blocks():
    # a NaN block makes its own row (of x) or column (of w) NaN and no other value
    x, w = _operand(20, 512, 1, per_row=True), _operand(140, 512, 2)
    x.scales[3, 17] = 0x7F
    w.scales[130, 2] = 0x7F
    x.scales[5] = 0
    y = dcr.nvfp4_matmul(x, w, dtype=torch.float32).cpu()
    nan = torch.zeros(20, 140, dtype=torch.bool)
    nan[3], nan[:, 130] = True, True
    assert torch.equal(torch.isnan(y), nan)
    assert bool((y[5][~nan[5]] == 0).all())


def test_product_of_no_rows_and_wide_arena_offsets():
    w = _operand(40, 64, 1)
    e = dcr.Nvfp4(torch.empty(0, 32, dtype=torch.uint8, device="cuda"), torch.empty(0, 4, dtype=torch.uint8, device="cuda"),
                  torch.ones(1, device="cuda"))
    assert dcr.nvfp4_matmul(e, w).shape == (0, 40)
    # weights of more than 2^32 codes: the last expert lies past 32-bit offsets
    experts, n, k = 66, 8192, 8192
    codes = torch.zeros(experts * n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(experts * n, k // 16, dtype=torch.uint8, device="cuda")
    last = _operand(n, k, 5)
    codes[-n:], scales[-n:] = last.codes, last.scales
    x = _operand(3, k, 6, per_row=True)
    off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    off[-1] = 3
    got = dcr.nvfp4_matmul(x, dcr.Nvfp4(codes, scales, last.scale), offsets=off, dtype=torch.float32)
    y, mag = _product(x, last)
    _close(got, y, mag, k, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m", [1, 30, 150])
def test_linear_equals_quantise_then_product(dtype, m):
    x, w = _x(m, 480, dtype, 9, pad=3), _operand(200, 480, 2)
    q, _ = dcr.nvfp4_quantize(x, per_row=True)
    y = dcr.nvfp4_linear(x, w)
    assert y.dtype == DT[dtype]
    assert torch.equal(y, dcr.nvfp4_matmul(q, w, dtype=DT[dtype]))
    ref, mag = _product(q, w)
    _close(y, ref, mag, 480, dtype)


def test_calls_run_on_the_given_stream_and_in_a_graph():
    x, w = _x(40, 512, "bf16", 1), _operand(260, 512, 2)
    y = dcr.nvfp4_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for st in (s, s.cuda_stream):
        got = dcr.nvfp4_linear(x, w, stream=st)
        s.synchronize()
        assert torch.equal(got, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = dcr.nvfp4_linear(x, w)
    x.copy_(_x(40, 512, "bf16", 2))
    g.replay()
    assert torch.equal(out, dcr.nvfp4_linear(x, w)) and not torch.equal(out, y)


@pytest.mark.parametrize("m,n,k", [(16, 512, 2048), (300, 5000, 256)])
def test_a_wait_that_runs_out_is_reported(m, n, k):
    # no operand is ever loaded: every wait of the kernel gives up after about a second, the call's status says so,
    # and the device is as usable as before
    import ctypes
    from bit_exact_xor_gb300 import ops
    x, w = _operand(m, k, 1, per_row=True), _operand(n, k, 2)
    y = dcr.nvfp4_matmul(x, w, dtype=torch.float32)
    dcr.ops_status()
    out = torch.empty(m, n, device="cuda")
    cx, cw = ops._nvfp4(x, "x")[3], ops._nvfp4(w, "w")[3]
    rc = ops._lib().dcr_nvfp4_matmul(ctypes.byref(cx), ctypes.byref(cw), m, n, k, None, 0, out.data_ptr(), ops.F32 | ops.TEST_STALL, n,
                                     torch.cuda.current_stream().cuda_stream)
    assert rc == dcr.OK
    with pytest.raises(dcr.DcrError) as e:
        dcr.ops_status()
    assert e.value.code == dcr.ERR_TIMEOUT
    dcr.ops_status()
    assert torch.equal(y, dcr.nvfp4_matmul(x, w, dtype=torch.float32))
