"""What the operators' documentation promises of NVFP4, and what it does not."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402


def test_a_quantised_row_does_not_depend_on_its_batch():
    x = torch.randn(300, 1056, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    whole, _ = dcr.nvfp4_quantize(x, per_row=True)
    for at, n in ((0, 1), (7, 2), (100, 37), (299, 1), (43, 257)):
        part, _ = dcr.nvfp4_quantize(x[at:at + n], per_row=True)
        assert torch.equal(part.codes, whole.codes[at:at + n]) and torch.equal(part.scales, whole.scales[at:at + n])
        assert torch.equal(part.scale, whole.scale[at:at + n])


def test_products_of_the_same_row_in_any_batch_agree_to_the_sums_rounding():
    # the order of a row's sum goes by the batch; each order is within k 2^-24 of the magnitudes' sum
    k = 4096
    x = torch.randn(300, k, generator=torch.Generator().manual_seed(2)).cuda()
    w, wv = dcr.nvfp4_quantize(torch.randn(1000, k, generator=torch.Generator().manual_seed(3)).cuda(), values=torch.float32)
    xq, xv = dcr.nvfp4_quantize(x, per_row=True, values=torch.float32)
    mag = xv.double().abs() @ wv.double().abs().T
    whole = dcr.nvfp4_linear(x, w)
    for n in (1, 16, 40, 128):
        assert bool(((dcr.nvfp4_linear(x[:n], w) - whole[:n]).abs() <= 2 * (k + 4) * 2.0 ** -24 * mag[:n]).all())


@pytest.mark.parametrize("values", [torch.float32, torch.bfloat16])
def test_a_block_with_a_scale_among_the_smallest_may_saturate(values):
    # t = 1; a block's largest value 1.49 * 6 * 2^-9 wants a scale of 1.49 * 2^-9 and gets 2^-9, the smallest: 8.94 of it
    # becomes 6.  A block whose scale is a normal number keeps its largest value to a sixteenth.
    x = torch.zeros(1, 64, device="cuda")
    x[0, 0], x[0, 16], x[0, 17], x[0, 32] = 2688.0, 1.49 * 6 / 512, -4.0 / 512, 100.3
    q, v = dcr.nvfp4_quantize(x, values=values)
    assert float(q.scale) == 1.0 and int(q.scales[0, 1]) == 1
    assert float(v[0, 16]) == 6.0 / 512 and float(v[0, 17]) == -4.0 / 512
    assert abs(float(v[0, 32]) / 100.3 - 1) <= 1 / 16 + 2.0 ** -8 and float(v[0, 0]) == 2688.0
