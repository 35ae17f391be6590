"""Build libdcr.so in-tree: nvcc for sm_103a, one object per translation unit
compiled in parallel, then one shared-library link; and _binding.so, the
operators' common calls from Python, against torch's headers.  Nothing needs
the second one: where it does not build, that is said, and every call goes
through ctypes."""
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libdcr.so")
SOURCES = ["plan.cpp", "pipeline.cpp", "encode.cu", "apply.cu", "dense.cu", "nvfp4_quantize.cu", "nvfp4_matmul.cu",
           "policy_loss.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
BUILD_DIR = os.path.join(HERE, "_build")
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", os.path.join(HERE, "..", "include")]


BINDING = os.path.join(HERE, "_binding.so")


def binding_commands(bdir):
    """Compile and link commands of _binding.so."""
    import torch
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    obj = os.path.join(bdir, "binding.o")
    abi = ["-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, '-DDCR_TORCH_VERSION="%s"' % torch.__version__]
    cc = ["g++", "-O2", "-fPIC", "-std=c++17", "-w"] + abi + [x for i in inc for x in ("-isystem", i)] + [
        "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    lib = os.path.join(base, "lib")
    link = ["g++", "-shared", "-o", BINDING, obj, "-L" + HERE, "-l:libdcr.so", "-L" + lib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda",
            "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    return cc, link


def _start(cmd):
    return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _end(started, what):
    """What a started command said; RuntimeError if it failed."""
    cmd, p = started
    said = p.communicate()[0].decode()
    if p.returncode != 0:
        raise RuntimeError("%s failed: %s\n%s" % (what, " ".join(cmd), said))
    return said


def build(verbose=False):
    bdir = BUILD_DIR
    os.makedirs(bdir, exist_ok=True)
    procs, objs, binding, without = [], [], None, None
    for src in SOURCES:
        obj = os.path.join(bdir, src.rsplit(".", 1)[0] + ".o")
        procs.append(_start(["nvcc"] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose and src.endswith(".cu") else []) + [
            "-x", "cu" if src.endswith(".cu") else "c++", "-c", os.path.join(CSRC, src), "-o", obj]))
        objs.append(obj)
    try:
        cc, blink = binding_commands(bdir)
        binding = _start(cc)
    except Exception as e:      # no torch, or one laid out in another way
        without = e
    logs = [_end(p, "compiling") for p in procs]
    _end(_start(["nvcc"] + ARCH + ["-shared", "-o", OUT] + objs + ["-lcudart"]), "link")
    if binding:
        try:
            _end(binding, "compiling")
            _end(_start(blink), "link")
        except (RuntimeError, OSError) as e:
            without = e
    if without is not None:
        if os.path.exists(BINDING):
            os.remove(BINDING)      # an older one is for another source or another torch
        warnings.warn("the operators' compiled binding did not build; their calls go through ctypes, a few microseconds slower: %s" % without)
    return "".join(logs)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
