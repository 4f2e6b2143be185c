"""The grid of the norms' gradients of rows that a cluster of blocks shares: no more clusters than run at once, since each
walks over an equal share of the rows (a cluster that began when another had ended doubled the time)."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

pytestmark = pytest.mark.gpu


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
