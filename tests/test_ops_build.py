"""The library and the operators without the compiled binding: neither the
build nor a call depends on it."""
import os
import shutil
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from bit_exact_xor_gb300 import build as B  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALL = """
import sys, warnings
%s
import torch
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    import bit_exact_xor_gb300 as dcr
    try:
        dcr.nvfp4_quantize(torch.zeros(4, 32))
    except dcr.DcrError as e:
        assert e.code == dcr.ERR_INVALID and "CUDA tensor" in str(e), e
    else:
        raise AssertionError("a host tensor was taken")
print(len([w for w in said if "binding" in str(w.message)]))
"""


def _warnings(setup):
    p = subprocess.run([sys.executable, "-c", CALL % setup], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.PIPE, timeout=300)
    assert p.returncode == 0, p.stderr.decode()[-2000:]
    return int(p.stdout)


def test_operators_answer_without_the_binding():
    assert _warnings("sys.modules['bit_exact_xor_gb300._binding'] = None") == 1


def test_operators_answer_beside_a_binding_for_another_torch():
    # one that names another version, and one from before versions were named: neither is called
    for body in ("torch_version = '0.1'", "pass"):
        assert _warnings("import types\nm = types.ModuleType('_binding')\nexec(%r, m.__dict__)\n"
                         "import bit_exact_xor_gb300\nsys.modules['bit_exact_xor_gb300._binding'] = m\n"
                         "bit_exact_xor_gb300._binding = m" % body) == 1


@pytest.mark.skipif(shutil.which("nvcc") is None, reason="needs nvcc")
@pytest.mark.parametrize("how", ["no headers", "no torch", "no linking", "no compiler"])
def test_the_library_builds_where_the_binding_does_not(tmp_path, monkeypatch, how):
    def commands(bdir):
        if how == "no torch":
            raise ImportError("No module named 'torch'")
        if how == "no compiler":
            return ["/nonexistent/g++"], ["true"]
        return (["false"], ["true"]) if how == "no headers" else (["true"], ["false"])

    stale = tmp_path / "_binding.so"
    stale.write_bytes(b"an older one")
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "objects"), raising=False)
    monkeypatch.setattr(B, "OUT", str(tmp_path / "libdcr.so"))
    monkeypatch.setattr(B, "BINDING", str(stale))
    monkeypatch.setattr(B, "SOURCES", ["plan.cpp"])     # one of them, for time
    monkeypatch.setattr(B, "FLAGS", [f for f in B.FLAGS if f != "-O3"])
    monkeypatch.setattr(B, "binding_commands", commands)
    with pytest.warns(UserWarning, match="binding did not build"):
        B.build()
    assert os.path.getsize(B.OUT) > 0 and not stale.exists()


@pytest.mark.skipif(shutil.which("nvcc") is None, reason="needs nvcc")
def test_a_library_that_does_not_build_still_fails(tmp_path, monkeypatch):
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path), raising=False)
    monkeypatch.setattr(B, "OUT", str(tmp_path / "libdcr.so"))
    monkeypatch.setattr(B, "SOURCES", ["nothing.cpp"])
    monkeypatch.setattr(B, "binding_commands", lambda bdir: (["true"], ["true"]))
    with pytest.raises(RuntimeError, match="compiling failed"):
        B.build()
