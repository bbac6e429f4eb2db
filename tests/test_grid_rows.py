"""Host check of the grids of launches that take one workgroup per piece of
their input (`grid_rows` in csrc/rmoe_sched.h): every piece has its workgroup,
no row of workgroups is idle, and no dimension reaches 2^32 threads, which the
host would take modulo 2^32 without an error."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_routed_grouped_amd", "csrc")
PROGRAM = """
#include "rmoe_sched.h"
#include <stdio.h>
int main() {
    long long n;
    while (scanf("%lld", &n) == 1) {
        const rmoe::GridRows g = rmoe::grid_rows(n);
        printf("%u %u\\n", g.x, g.y);
    }
}
"""


def test_grid_rows(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "grid.cpp", tmp_path / "grid"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-O1", "-std=c++17", "-Wall", "-Werror", f"-I{CSRC}", "-o", str(exe), str(src)], check=True)
    row = 1 << 21
    edges = [m * row + d for m in (1, 2, 3, 7, 16) for d in (-1, 0, 1)]
    # tokens at which a workgroup per 64 or 32 of them passed 2^32 threads, and the largest counts
    wide = [2 ** 32 // 320 + 1, 2 ** 32 // 1024, 2 ** 32 // 1024 + 1, 2 ** 31 // 64, 2 ** 31 // 32]
    pieces = [1, 2, 255, 511, *edges, *wide]
    out = subprocess.run([str(exe)], input="\n".join(map(str, pieces)), capture_output=True, text=True, check=True).stdout
    grids = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert len(grids) == len(pieces)
    for n, (x, y) in zip(pieces, grids):
        assert x * y >= n > x * (y - 1), (n, x, y)
        assert x * 1024 < 2 ** 32 and y <= 65535, (n, x, y)
        assert y == 1 or x == row, (n, x, y)
