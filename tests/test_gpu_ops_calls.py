"""The operators' calls as programs make them: linear layers with experts and
of every size through the compiled binding, back to back; from several
threads; without the compiled binding."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402
from bit_exact_xor_gb300 import ops  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _randn(rows, cols, dtype, seed):
    return torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).cuda()


def _weights(rows, k, seed):
    return dcr.nvfp4_quantize(_randn(rows, k, "f32", seed))[0]


@pytest.mark.parametrize("m,n", [(3, 200), (300, 5000)])
def test_first_call_of_a_thread(m, n):
    # a thread that has not used the device yet, as a C program's may be: nothing has made a context current there
    x, w = dcr.nvfp4_quantize(_randn(m, 96, "f32", 1), per_row=True)[0], _weights(n, 96, 2)
    exp = dcr.nvfp4_matmul(x, w)
    out = torch.empty_like(exp)
    torch.cuda.synchronize()
    args = (ctypes.byref(ops._nvfp4(x, "x")[3]), ctypes.byref(ops._nvfp4(w, "w")[3]), m, n, 96, None, 0, out.data_ptr(), ops.BF16, n, None)
    said = []

    def work():
        said.append(ops._lib().dcr_nvfp4_matmul(*args))
        said.append(dcr.last_error())

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert said[0] == dcr.OK, said
    assert torch.equal(out, exp)


@pytest.mark.parametrize("wide", [False, True])
def test_two_threads_with_and_without_experts(wide):
    # a product's shared memory grows with the number of experts: calls of both kinds at once, from C, each on its own
    # stream (ctypes lets go of the interpreter's lock)
    n, k, e = (256, 64, 1024) if wide else (16, 64, 1024)
    m = 20 * e if wide else e
    w, q = _weights(e * n, k, 1), dcr.nvfp4_quantize(_randn(m, k, "f32", 3), per_row=True)[0]
    off = torch.arange(0, m + 1, m // e, dtype=torch.int32, device="cuda")
    md, nd = (256, 256 * 80) if wide else (4, 64)
    wd, qd = _weights(nd, k, 2), dcr.nvfp4_quantize(_randn(md, k, "f32", 4), per_row=True)[0]
    jobs = [(q, w, m, n, off, e), (qd, wd, md, nd, None, 0)]
    exp = [dcr.nvfp4_matmul(x, y, offsets=o) for x, y, _, _, o, _ in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    call, codes, out = ops._lib().dcr_nvfp4_matmul, [[], []], [torch.empty_like(y) for y in exp]
    ready = threading.Barrier(2)

    def work(i):
        x, y, rows, cols, offsets, experts = jobs[i]
        args = (ctypes.byref(ops._nvfp4(x, "x")[3]), ctypes.byref(ops._nvfp4(y, "w")[3]), rows, cols, k,
                None if offsets is None else offsets.data_ptr(), experts, out[i].data_ptr(), ops.BF16, cols, streams[i].cuda_stream)
        ready.wait()
        codes[i] += [call(*args) for _ in range(10000)]

    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(before)
    torch.cuda.synchronize()
    for i in range(2):
        assert len(codes[i]) == 10000 and set(codes[i]) == {dcr.OK}, sum(c != dcr.OK for c in codes[i])
        assert torch.equal(out[i], exp[i])


def test_a_reported_error_is_not_reported_again():
    # a status call is not allowed while its stream is being captured: that call says so, and the next ones are good
    x, w = _randn(5, 64, "f32", 1), _weights(32, 64, 2)
    y = dcr.nvfp4_linear(x, w)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.capture_begin(capture_error_mode="relaxed")
        rc = ops._lib().dcr_ops_status(s.cuda_stream)
        try:
            g.capture_end()
        except RuntimeError:
            pass
    assert rc == dcr.ERR_CUDA, rc
    assert ops._lib().dcr_ops_status(torch.cuda.current_stream().cuda_stream) == dcr.OK
    # straight from C, and through the binding: nothing has cleared the thread's last error in between
    q = torch.empty(5 * 32, dtype=torch.uint8, device="cuda")
    sc, t = torch.empty(5 * 4, dtype=torch.uint8, device="cuda"), torch.empty(5, device="cuda")
    with torch.cuda.stream(s):
        g2 = torch.cuda.CUDAGraph()
        g2.capture_begin(capture_error_mode="relaxed")
        ops._lib().dcr_ops_status(s.cuda_stream)
        rc = ops._lib().dcr_nvfp4_quantize(x.data_ptr(), ops.F32, 5, 64, 64, ops.SCALE_ROW, t.data_ptr(), q.data_ptr(), sc.data_ptr(),
                                           None, ops.NONE, None, torch.cuda.default_stream().cuda_stream)
        try:
            g2.capture_end()
        except RuntimeError:
            pass
    assert rc == dcr.OK, dcr.last_error()
    assert torch.equal(dcr.nvfp4_linear(x, w), y)


def _then(x, w, offsets=None, dtype=None):
    q, _ = dcr.nvfp4_quantize(x, per_row=True)
    return dcr.nvfp4_matmul(q, w, offsets=offsets, dtype=dtype or x.dtype)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("m,n,k", [(1, 6000, 2048), (37, 9728, 96), (40, 9800, 544), (300, 5121, 544), (700, 3333, 2080),
                                   (257, 5000, 96)])
def test_linear_of_many_sizes_back_to_back(m, n, k, dtype, out):
    # the workspace of one call is the next one's: a product that read ahead of its quantisation would take the last one's
    w = _weights(n, k, 1)
    xs = [_randn(m, k, dtype, i) * (4.0 ** i) for i in range(5)]
    exp = [_then(x, w, dtype=DT[out]) for x in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [dcr.nvfp4_linear(x, w, dtype=DT[out]) for x in xs]
        assert all(torch.equal(a, b) for a, b in zip(got, exp))
    dcr.ops_status()


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("counts", [[3, 0, 1, 9, 0], [1] * 64, [0, 40, 0, 0, 17, 1, 0, 90], [300, 0, 90, 257, 5], [0, 0, 700], [1000] + [0] * 63])
@pytest.mark.parametrize("n,k", [(72, 96), (2601, 416)])
def test_linear_of_experts_back_to_back(counts, n, k, dtype, out):
    # offsets come from a kernel just ahead of the call, as from a router, and change from call to call
    e, m = len(counts), sum(counts)
    w = _weights(e * n, k, 2)
    w = dcr.Nvfp4(w.codes, w.scales, torch.linspace(0.5, 2.0, e, device="cuda"))
    xs = [_randn(m, k, dtype, i) * (4.0 ** i) for i in range(4)]
    each = [torch.tensor(counts[i:] + counts[:i], device="cuda") for i in range(4)]
    offs = [torch.cat([c.new_zeros(1), c.cumsum(0)]).to(torch.int32) for c in each]
    exp = [_then(x, w, o, DT[out]) for x, o in zip(xs, offs)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for x, c in zip(xs, each):
            off = torch.cat([c.new_zeros(1), c.cumsum(0)]).to(torch.int32)
            got.append(dcr.nvfp4_linear(x, w, offsets=off, dtype=DT[out]))
        assert all(torch.equal(a, b) for a, b in zip(got, exp))
    # through the call with every argument spelled out, too
    into = torch.empty(m, n, dtype=DT[out], device="cuda")
    assert torch.equal(dcr.nvfp4_linear(xs[0], w, offsets=offs[0], out=into), exp[0])
    dcr.ops_status()


def test_per_row_is_a_truth_value():
    x = _randn(5, 64, "f32", 1)
    for yes in (True, 1):
        assert dcr.nvfp4_quantize(x, per_row=yes)[0].scale.shape == (5,)
    for no in (False, 0):
        assert dcr.nvfp4_quantize(x, per_row=no)[0].scale.shape == (1,)


@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("shape", [(0, 32), (3, 0), (0, 0)])
def test_scale_of_an_empty_matrix_is_one(shape, per_row):
    # as of any matrix without a finite value other than 0
    junk = [torch.full((64,), 7.0, device="cuda") for _ in range(64)]   # what a new tensor may find in its memory
    del junk
    for out in (None, dcr.Nvfp4(torch.empty(shape[0], shape[1] // 2, dtype=torch.uint8, device="cuda"),
                                torch.empty(shape[0], shape[1] // 16, dtype=torch.uint8, device="cuda"),
                                torch.full((shape[0] if per_row else 1,), 7.0, device="cuda"))):
        q, _ = dcr.nvfp4_quantize(torch.empty(shape, device="cuda"), per_row=per_row, out=out)
        assert q.scale.shape == (shape[0] if per_row else 1,) and bool((q.scale == 1).all())


WITHOUT = """
import sys, warnings
warnings.simplefilter("ignore")
sys.modules["bit_exact_xor_gb300._binding"] = None    # as if it had not been built
import torch
import bit_exact_xor_gb300 as dcr
x = torch.randn(40, 512, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
w, v = dcr.nvfp4_quantize(torch.randn(96, 512, generator=torch.Generator().manual_seed(2)).cuda(), values=torch.float32)
y = dcr.nvfp4_linear(x, w)
t = torch.arange(40, device="cuda")
one = torch.ones(40, device="cuda")
lp = dcr.token_logprobs(y, t)
out = dcr.policy_loss(y, t, lp, one, one)
torch.save([a.cpu() for a in (w.codes, w.scales, w.scale, v, y, lp) + tuple(out)], sys.argv[1])
"""


def test_every_operator_without_the_compiled_binding(tmp_path):
    # the library's kernels run through ctypes then, with the same results
    got = []
    for i, code in enumerate((WITHOUT, WITHOUT.replace("sys.modules[", "dict()["))):
        path = str(tmp_path / ("%d.pt" % i))
        p = subprocess.run([sys.executable, "-c", code, path], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=600)
        assert p.returncode == 0, p.stdout.decode()[-2000:]
        got.append(torch.load(path))
    assert all(torch.equal(a, b) for a, b in zip(*got))
