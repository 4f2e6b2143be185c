"""The walk of the gradients' products (csrc/back_walk.h), compiled for the host: every unit is taken exactly once, by
pairs that have their units one after the other, and long units do not leave pairs idle."""
import os
import subprocess


CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "broadcast_implicit_gemm_gb300", "csrc")
PROGRAM = r'''
#include <cstdio>
#include <vector>
#include "back_walk.h"
using namespace bigemm;
int main()
{
    const int sizes[] = {1, 2, 3, 16, 75, 76, 77, 151, 152, 153, 256, 300, 1000}, dws[] = {1, 2, 5, 60, 76, 100, 500, 2048};
    const int counts[] = {1, 2, 7, 76};
    const long long times[][2] = {{512, 64}, {10, 10}, {10, 500}, {70, 1}, {7, 3}};
    for (int dx : sizes) for (int dw : dws) for (int most : counts) for (auto &t : times) {
        const int pairs = most < dx + dw ? most : dx + dw;
        const BackWalk w = make_back_walk(dx, dw, pairs, t[0], t[1]);
        std::vector<int> seen(dx + dw, 0);
        long long longest = 0, all = dx * t[0] + dw * t[1], one = t[0] > t[1] ? t[0] : t[1];
        for (int p = 0; p < pairs; ++p) {
            long long time = 0;
            int turn = 0;
            for (;; ++turn) {
                const int u = back_unit(w, turn, p, pairs);
                if (u < 0) break;
                if (u >= dx + dw) return printf("out of range %d\n", u), 1;
                ++seen[u];
                time += u < dx ? t[0] : t[1];
            }
            for (int more = 1; more < 4; ++more)
                if (back_unit(w, turn + more, p, pairs) >= 0) return printf("%d %d %d: a unit after the end\n", dx, dw, pairs), 1;
            longest = time > longest ? time : longest;
        }
        for (int u = 0; u < dx + dw; ++u)
            if (seen[u] != 1) return printf("%d %d %d: unit %d %d times\n", dx, dw, pairs, u, seen[u]), 1;
        if (longest > all / pairs + one) return printf("%d %d %d: %lld of %lld\n", dx, dw, pairs, longest, all / pairs), 1;
    }
    printf("ok\n");
    return 0;
}
'''


def test_every_unit_once(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
