"""The operators' calls as programs make them: linear layers with experts and
of every size through the compiled binding, back to back; from several
threads; without the compiled binding."""
import ctypes
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402
from bit_exact_xor_gb300 import ops  # noqa: E402

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
