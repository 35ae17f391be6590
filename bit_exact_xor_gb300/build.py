"""Build libdcr.so in-tree: nvcc for sm_103a, one object per translation unit
compiled in parallel, then one shared-library link; and _binding.so, the
operators' common calls from Python, against torch's headers."""
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libdcr.so")
SOURCES = ["plan.cpp", "pipeline.cpp", "encode.cu", "apply.cu", "dense.cu", "nvfp4_quantize.cu", "nvfp4_matmul.cu",
           "policy_loss.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", os.path.join(HERE, "..", "include")]


BINDING = os.path.join(HERE, "_binding.so")


def binding_commands(bdir):
    """Compile and link commands of _binding.so."""
    import torch
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    obj = os.path.join(bdir, "binding.o")
    abi = "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI
    cc = ["g++", "-O2", "-fPIC", "-std=c++17", "-w", abi] + [x for i in inc for x in ("-isystem", i)] + [
        "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    lib = os.path.join(base, "lib")
    link = ["g++", "-shared", "-o", BINDING, obj, "-L" + HERE, "-l:libdcr.so", "-L" + lib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda",
            "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]
    return cc, link


def build(verbose=False):
    bdir = os.path.join(HERE, "_build")
    os.makedirs(bdir, exist_ok=True)
    objs, procs = [], []
    for src in SOURCES:
        obj = os.path.join(bdir, src.rsplit(".", 1)[0] + ".o")
        cmd = ["nvcc"] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose and src.endswith(".cu") else []) + [
            "-x", "cu" if src.endswith(".cu") else "c++", "-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    cc, blink = binding_commands(bdir)
    procs.append((cc, subprocess.Popen(cc, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    logs = []
    for cmd, p in procs:
        out, _ = p.communicate()
        logs.append(out.decode())
        if p.returncode != 0:
            raise RuntimeError("compiling failed: %s\n%s" % (" ".join(cmd), out.decode()))
    link = ["nvcc"] + ARCH + ["-shared", "-o", OUT] + objs + ["-lcudart"]
    p = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if p.returncode != 0:
        raise RuntimeError("link failed:\n" + p.stdout.decode())
    p = subprocess.run(blink, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if p.returncode != 0:
        raise RuntimeError("link failed:\n" + p.stdout.decode())
    return "".join(logs)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
