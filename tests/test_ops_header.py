"""include/dcr_ops.h as a C and a C++ program use it."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "dcr_ops.h"
#include <stdio.h>
int main(void)
{
    int m = 65536, k = 65536;
    uint32_t n = 131072, l = 65536;
    uint64_t a = 3, b = 96;
    printf("%llu %llu %llu %llu\\n", (unsigned long long)DCR_LINEAR_WORKSPACE(m, k), (unsigned long long)DCR_LINEAR_WORKSPACE(n, l),
           (unsigned long long)DCR_LINEAR_WORKSPACE(a, b), (unsigned long long)DCR_LINEAR_WORKSPACE(1 + 1, 32 + 32));
    return 0;
}
"""


@pytest.mark.parametrize("compiler,suffix,std", [("gcc", ".c", "c99"), ("g++", ".cpp", "c++17")])
def test_workspace_of_sizes_in_32_bit_types(tmp_path, compiler, suffix, std):
    if shutil.which(compiler) is None:
        pytest.skip("needs " + compiler)
    src, exe = tmp_path / ("w" + suffix), tmp_path / "w"
    src.write_text(SOURCE)
    subprocess.run([compiler, "-std=" + std, "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    said = subprocess.run([str(exe)], check=True, stdout=subprocess.PIPE).stdout.split()
    want = [m * (k // 2 + k // 16 + 4) + 4 for m, k in ((65536, 65536), (131072, 65536), (3, 96), (2, 64))]
    assert [int(x) for x in said] == want
