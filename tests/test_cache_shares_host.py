"""CPU test of the arithmetic that cuts the attention's stream of keys into shares, compiled from the kernels' own header."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
#include <stdio.h>
#include "tb_cache_internal.h"
int main() {
    unsigned long long units;
    unsigned budget;
    while (scanf("%llu %u", &units, &budget) == 2)
        printf("%llu\\n", (unsigned long long)tbk::units_of_share(units, budget));
    return 0;
}
"""


def test_shares_cover_the_stream(tmp_path):
    """A share is the stream's budget-th, rounded up, on both sides of 2^32 units."""
    if not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("HIP headers are not installed")
    (tmp_path / "shares.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "shares")
    subprocess.run([shutil.which("g++"), "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
                    "-I" + os.path.join(ROOT, "copy_reduce_amd", "csrc"), str(tmp_path / "shares.cpp"), "-o", exe], check=True)
    budgets = [1, 2, 3, 64, 255, 256, 768, 769, 1024, 4096]
    asked = [(u, b) for b in budgets for u in [1, 2, b - 1, b, b + 1, 10 ** 6 + 7, 2 ** 40] + [2 ** 32 + d for d in range(-b - 2, 3)] if u > 0]
    r = subprocess.run([exe], input="\n".join(f"{u} {b}" for u, b in asked), capture_output=True, text=True, check=True)
    assert [int(x) for x in r.stdout.split()] == [-(-u // b) for u, b in asked]
