"""The grid of the norms' gradients of rows that a cluster of blocks shares: no more clusters than run at once, since each
walks over an equal share of the rows (a cluster that began when another had ended doubled the time)."""
import os
import subprocess
import sys

import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rows_of_sums(rows, cols, layer):
    """How many rows of partial sums a call leaves in its workspace: one for each cluster."""
    x, dx = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda"), torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    mean, rstd, dw, db = (torch.zeros(n, device="cuda") for n in (rows, rows, cols, cols))
    size = bg.norm_backward_workspace_bytes(rows, cols)
    space = torch.full((size // 4,), float("nan"), device="cuda")
    if layer:
        bg.layernorm_backward_run(rows, cols, bg.BF16, x, cols, x, cols, mean, rstd, None, None, 0, dx, cols, dw, db, space, size)
    else:
        bg.rmsnorm_backward_run(rows, cols, bg.BF16, x, cols, x, cols, None, 1e-6, None, 0, dx, cols, dw, space, size)
    torch.cuda.synchronize()
    left = int((~space.isnan()).sum())
    assert left % cols == 0 and bg.bigemm_last_device_error() == 0
    return left // cols // (2 if layer else 1)


@pytest.mark.parametrize("layer", [True, False])
def test_clusters(layer):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert rows_of_sums(400, 12000, layer) <= sms // 2
    assert rows_of_sums(400, 20000, layer) <= sms // 4
    # eight neighbours each: groups of SMs are no multiples of eight
    assert 8 <= rows_of_sums(400, 40000, layer) < sms // 8
    assert rows_of_sums(5, 40000, layer) == 5


FIRST_CALL = r'''
import torch
import broadcast_implicit_gemm_gb300 as bg
x, d, out = (torch.randn((300, 40000), device="cuda").bfloat16() for _ in range(3))
w, dw = torch.randn((64, 64), device="cuda").bfloat16(), torch.empty(40000, device="cuda")
bg.matmul(w, w)                  # the library knows the device
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    bg.rmsnorm_backward(d, x, dx=out, dweight=dw)
graph.replay()
want = bg.rmsnorm_backward(d, x)
assert torch.equal(out, want[0]) and torch.equal(dw, want[1]) and bg.bigemm_last_device_error() == 0
print("same")
'''


def test_a_first_call_that_is_captured():
    """How many clusters fit is asked for once, which may be while a stream is captured."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr
