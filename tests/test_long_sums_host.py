"""How long sums of the products' gradients are cut (csrc/matmul_back.cuh, csrc/matmul_back_run.cu): the shares of an axis
cover it once, none is empty, and none is longer than one accumulator takes."""
import os
import re
import subprocess

import pytest

import broadcast_implicit_gemm_gb300 as bg
from tests.test_train_host import lib  # noqa: F401

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "broadcast_implicit_gemm_gb300", "csrc")
LONGEST = 32768


@pytest.mark.parametrize("M,shares", [(32768, 0), (32769, 2), (131072, 4), (131073, 5), (2 ** 20, 32)])
def test_shares_of_many_tokens(lib, M, shares):
    """Through 4096 x 4096, where there are units enough without shares: dw's partial results beside what a call needs
    anyway (the sums over runs of rows)."""
    q = bg.matmul_backward_workspace_bytes
    own = q(4096, 4096, 4096, 256, 4096, 256, 4096, 256, 4096)
    assert q(M, 4096, 4096, 256, 4096, 256, 4096, 256, 4096) == shares * 4096 * 4096 * 4 + own
    q = bg.matmul_gated_backward_workspace_bytes
    both = q(4096, 4096, 4096, 256, 4096, 256, 4096, 256, 4096) - 2 * 4096 * 4096 * 2
    assert q(M, 4096, 4096, 256, 4096, 256, 4096, 256, 4096) == 2 * shares * 4096 * 4096 * 4 + 2 * M * 4096 * 2 + both


@pytest.mark.parametrize("N,plain,gated", [(16384, 0, 0), (16392, 0, 2), (32768, 0, 2), (32776, 2, 3), (65544, 3, 5)])
def test_shares_of_many_channels(lib, N, plain, gated):
    """dx of 4096 tokens, 4096 channels in, sums over N channels, of two products one after the other."""
    q = bg.matmul_backward_workspace_bytes
    M = K = 4096
    rows = -(-8 * 2 * 76 // -(-N // 256))                      # runs of rows of the sums over tokens, by their count
    got = q(M, N, K, 256, N, 256, K, 256, K)
    sums = [-(-r * N * 4 // 256) * 256 for r in range(1, rows + 2)]
    assert got - plain * M * K * 4 in sums
    q = bg.matmul_gated_backward_workspace_bytes
    got = q(M, N, K, 256, K, 256, K, 256, K) - -(-2 * M * N * 2 // 256) * 256
    assert got - gated * M * K * 4 in [-(-2 * r * N * 4 // 256) * 256 for r in range(1, rows + 2)]


PROGRAM = r'''
#include <cstdio>
#include <initializer_list>
#include "fastdiv.h"
using namespace bigemm;
%s
int main()
{
    const int blocks[] = {1, 2, 3, 4, 7, 64, 100, 511, 513, 2049, 40001, 1 << 20, (1 << 24) + 3, (1 << 25) - 1, 1 << 25};
    for (int b : blocks)
        for (int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 33, 500, 4097, 32767, 32768}) {
            if (s > b) continue;
            const UnitGrid g = make_unit_grid(3, 5, s, b);
            int at = 0;
            for (int i = 0; i < s; ++i) {
                const int k0 = share_start(g, i), k1 = share_start(g, i + 1);
                if (k0 != at || k1 <= k0 || k1 - k0 > (b + s - 1) / s || k0 != (long long)b * i / s)
                    return printf("%%d in %%d: share %%d is %%d to %%d\n", b, s, i, k0, k1), 1;
                at = k1;
            }
            if (at != b) return printf("%%d in %%d end at %%d\n", b, s, at), 1;
        }
    printf("ok\n");
    return 0;
}
'''


def test_shares_cover_the_axis_once(tmp_path):
    text = open(os.path.join(CSRC, "matmul_back.cuh")).read()
    part = re.search(r"struct UnitGrid \{.*?\n\}\n(?=\nstruct BackArgs)", text, re.S).group(0)
    src, exe = tmp_path / "shares.cpp", tmp_path / "shares"
    src.write_text(PROGRAM % part)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
