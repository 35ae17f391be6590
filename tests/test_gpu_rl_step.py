"""examples/rl_step.py runs as shipped: its own asserts check that the rollout
engine computes the sender's logits after the refit."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EXAMPLE = os.path.join(ROOT, "examples", "rl_step.py")


def test_rl_step_parses():
    compile(open(EXAMPLE).read(), EXAMPLE, "exec")


@pytest.mark.gpu
def test_rl_step_runs():
    pytest.importorskip("torch")
    out = subprocess.run([sys.executable, EXAMPLE], stdout=subprocess.PIPE, stderr=subprocess.PIPE, timeout=600, cwd=ROOT)
    assert out.returncode == 0, out.stderr.decode()[-2000:]
    m = re.search(r"loss (-?[\d.]+); (\d+) of (\d+) values changed; payload (\d+) bytes; logits moved by at most ([\d.]+)",
                  out.stdout.decode())
    assert m, out.stdout.decode()
    changed, total, size, moved = int(m[2]), int(m[3]), int(m[4]), float(m[5])
    assert 0 < changed < total and 0 < size < total and moved > 0
