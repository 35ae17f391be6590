"""Calls of a step's operators as programs make them: from several threads,
back to back on changing inputs, and without the compiled binding."""
import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_exact_xor_gb300 as dcr  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _step(seed, tokens=300, experts=24, k=4, cols=136, vocab=5003):
    """All of a step's operators once; every output."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    r = dcr.route_experts(normal(tokens, experts), k, scoring="sigmoid", bias=normal(experts) * 0.05, groups=4, group_top=3)
    x = normal(tokens, cols).bfloat16()
    rows = dcr.experts_gather(x, r)
    y = dcr.experts_combine(rows, r)
    by_y, by_w = dcr.experts_combine_grad(rows, r, x)
    back = dcr.route_experts_grad(normal(tokens, experts), r, by_w, scoring="sigmoid")
    z, t = normal(tokens, vocab), torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
    s = dcr.token_scores(z, t, top=5)
    grad = dcr.token_scores_grad(z, t, s.stats, s.logp, s.entropy)
    w = [normal(1000), normal(77, 13)]
    gw = [normal(1000), normal(77, 13)]
    norm = dcr.grad_norm(gw)
    out = list(r) + [rows, y, by_y, by_w, back, grad, norm] + list(s)
    for bits in (32, 8):
        ww, states = [v.clone() for v in w], dcr.adamw_states(w, bits)
        copies = [torch.empty_like(v, dtype=torch.bfloat16) for v in w]
        dcr.adamw_step(ww, gw, states, 3, 1e-3, copies=copies, norm=norm, max_norm=0.5, seed=seed)
        out += ww + copies + [v for st in states for v in st]
    return out


def test_threads_on_their_own_streams():
    exp = [_step(i) for i in range(4)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = _step(i)
                s.synchronize()
                bad.extend((i, j) for j, (a, b) in enumerate(zip(got, exp[i])) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, sorted(set(bad))


def test_back_to_back_without_waiting():
    exp = [_step(i) for i in range(3)]
    torch.cuda.synchronize()
    got = [_step(i % 3) for i in range(12)]
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, exp[i % 3]))


WITHOUT = """
import sys, warnings
warnings.simplefilter("ignore")
sys.modules["bit_exact_xor_gb300._binding"] = None    # as if it had not been built
sys.path.insert(0, "tests")
import torch
import test_gpu_step_calls as t
torch.save([a.cpu() for a in t._step(1)], sys.argv[1])
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
