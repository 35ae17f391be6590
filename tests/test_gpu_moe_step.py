"""examples/moe_step.py: runs as shipped (its own asserts check that the engine
computes the sender's logits after the refit), and its gradients are those of
the same model written plainly in 64 bits."""
import importlib.util
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EXAMPLE = os.path.join(ROOT, "examples", "moe_step.py")


def test_moe_step_parses():
    compile(open(EXAMPLE).read(), EXAMPLE, "exec")


@pytest.mark.gpu
def test_moe_step_runs():
    pytest.importorskip("torch")
    out = subprocess.run([sys.executable, EXAMPLE], stdout=subprocess.PIPE, stderr=subprocess.PIPE, timeout=600, cwd=ROOT)
    assert out.returncode == 0, out.stderr.decode()[-2000:]
    m = re.search(r"loss (-?[\d.]+); entropy ([\d.]+); gradient's norm ([\d.]+); (\d+) values changed; payload (\d+) bytes; logits moved by "
                  r"at most ([\d.]+)", out.stdout.decode())
    assert m, out.stdout.decode()
    assert float(m[2]) > 0 and float(m[3]) > 0 and int(m[4]) > 0 and int(m[5]) > 0 and float(m[6]) > 0


@pytest.mark.gpu
def test_moe_gradients():
    torch = pytest.importorskip("torch")
    import step_ref as R
    spec = importlib.util.spec_from_file_location("moe_step", EXAMPLE)
    M = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(M)
    g = torch.Generator().manual_seed(3)
    tokens, e, h, f, v, k = 40, M.EXPERTS, M.HIDDEN, M.FFN, M.VOCAB, M.CHOSEN
    shapes = dict(x=(tokens, h), router=(e, h), up=(e, f, h), down=(e, h, f), head=(v, h))
    std = dict(x=1.0, router=0.05, up=0.02, down=0.02, head=0.02)
    plain = {n: (torch.randn(*s, generator=g) * std[n]).double().requires_grad_() for n, s in shapes.items()}
    bias, keep = torch.randn(e, generator=g) * 0.01, torch.arange(tokens) < tokens - 5
    up = torch.randn(tokens, v, generator=g)
    # in 32 bits on the GPU
    dev = {n: t.detach().float().cuda().requires_grad_() for n, t in plain.items()}
    z = M.trainer_logits(**dev, bias=bias.cuda(), keep=keep.cuda())
    z.backward(up.cuda())
    # plainly: every token through its own experts; which ones is the same choice
    with torch.no_grad():
        logits32 = (dev["x"] @ dev["router"].T).cpu()
    chosen = R.choose(logits32, k, "sigmoid", bias, 4, 2, 2, keep)
    logits = plain["x"] @ plain["router"].T
    w = R.weights(logits, chosen, "sigmoid", True, 1.0)
    at = chosen.clamp(min=0)
    hidden = torch.nn.functional.silu(torch.einsum("th,tkfh->tkf", plain["x"], plain["up"][at]))
    out = torch.einsum("tkf,tkhf->tkh", hidden, plain["down"][at])
    exp = (plain["x"] + (out * w[:, :, None]).sum(1)) @ plain["head"].T
    exp.backward(up.double())
    # products of up to 2048 terms in 32 bits, four of them one after another, each off by at most about its length's root of
    # roundings: 2^-24 * 2^5.5 * 4 relative to the result's size, with room for a factor of 8
    for n in plain:
        a, b = dev[n].grad.cpu().double(), plain[n].grad
        assert float((a - b).norm() / b.norm()) <= 2.0 ** -13.5, n
    assert float((z.detach().cpu().double() - exp.detach()).norm() / exp.detach().norm()) <= 2.0 ** -13.5
