"""Where the kernels look for the scale of an MXFP8 element (csrc/mx_layout.h), against the layout's definition in
integers of any size, up to the largest matrices that the calls accept.  The header has no CUDA dependency on the host
side and is compiled here with the system's C++ compiler, signed overflow trapped."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "broadcast_implicit_gemm_gb300", "csrc")

CHECKER = r"""
#include <cstdio>
#include "mx_layout.h"
int main() {
    long long row, col, cols;
    while (scanf("%lld %lld %lld", &row, &col, &cols) == 3) {
        const int group = (int)col / bigemm::kMxGroup, blocks = (int)((cols + bigemm::kMxBlock - 1) / bigemm::kMxBlock);
        const long long apart = bigemm::mx_scale_row(row, blocks) + bigemm::mx_scale_group(group);
        if (apart != bigemm::mx_scale_offset(row, group, blocks)) return 1;
        printf("%lld\n", apart);
    }
    return 0;
}
"""

TOP = 1 << 30


def places():
    for cols in (1, 127, 128, 129, 5000, 1 << 20, (1 << 29) - 1, 1 << 29, (1 << 29) + 128, TOP - 1, TOP):
        for col in {0, 31, 32, 127, 128, cols // 2, cols - 129, cols - 1, 1 << 29, (1 << 29) + 127}:
            for row in (0, 1, 31, 32, 127, 128, 12345, 2 ** 31 - 1):
                if 0 <= col < cols:
                    yield row, col, cols


def test_offsets(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "chk.cc", tmp_path / "chk"
    src.write_text(CHECKER)
    subprocess.run([cxx, "-O1", "-ftrapv", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    asked = list(places())
    out = subprocess.run([str(exe)], input="\n".join("%d %d %d" % p for p in asked), capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stderr
    got = [int(v) for v in out.stdout.split()]
    want = [(r // 128 * -(-n // 128) + k // 128) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + k % 128 // 32 for r, k, n in asked]
    assert got == want
