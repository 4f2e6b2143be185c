"""The norm where a block walks over more than one row: it loads the next row before it sums the present one, and takes
turns with two places for the warps' sums.  Each width has the threads per row that the name says, and enough rows for
three turns of all blocks on 152 SMs; on the 16-byte grid and off it, with the sum in place of either input."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg
from tests import layer_ref_gpu as lr

pytestmark = pytest.mark.gpu

TD, rand = lr.TD, lr.rand
# columns, rows
WALKS = {"a warp": (200, 15000), "a warp, two pieces": (500, 15000), "128": (1000, 4000), "128, two pieces": (2000, 4000),
         "256": (4000, 2000), "512": (8000, 1000), "1024": (16000, 500), "twice over": (20000, 300)}


def check(cols, rows, kind, out, residual, odd, place=None, seed=1):
    cols += odd
    pad = 8 * (1 - odd) + 2 * odd
    g = 1 + 0.2 * rand((cols,), seed)
    x = lr.strided(rand((rows, cols), seed + 1), pad, TD[kind])
    x *= torch.exp2((torch.arange(rows, device="cuda") % 7 - 3).float())[:, None].to(TD[kind])       # rows unlike each other
    r = lr.strided(rand((rows, cols), seed + 2), pad, TD[kind]) if residual else None
    h = x.double() + r.double() if residual else x.double()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * g.double()
    d = y.abs() * ((cols + 1) / 2 + 6) * 2.0 ** -23
    sums = {"x": x, "residual": r, None: lr.strided(torch.zeros((rows, cols), device="cuda"), pad, TD[kind])}[place] if residual else None
    odt = TD[kind] if out == "same" else TD[out]
    made = lr.strided(torch.zeros((rows, cols), device="cuda"), pad, odt)
    got = bg.rmsnorm(x, g, residual=r, sum_out=sums, out=made)
    got = got if isinstance(got, tuple) else (got,)
    torch.cuda.synchronize()
    assert got[0] is made and bg.bigemm_last_device_error() == 0
    if residual:
        assert got[-1] is sums
        lr.check_float(sums, h, 2.0 ** -24 * h.abs(), "sum")
        assert torch.isnan(sums._base[:, cols:]).all()
    if out == "mx":
        lr.check_mx(got[0], got[1], y, d, "norm")
    else:
        lr.check_float(got[0], y, d, "norm")
        assert torch.isnan(made._base[:, cols:]).all()


@pytest.mark.parametrize("walk", WALKS)
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("kind,out,residual", [("bf16", "same", True), ("f16", "mx", True), ("f16", "same", False), ("bf16", "mx", False),
                                               ("f16", "f32", True), ("f32", "same", True), ("f32", "mx", False)])
def test_rows(walk, odd, kind, out, residual):
    check(*WALKS[walk], kind, out, residual, odd)


@pytest.mark.parametrize("walk", WALKS)
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("place", ["x", "residual"])
@pytest.mark.parametrize("kind,out", [("bf16", "same"), ("f16", "mx"), ("f32", "same")])
def test_sum_in_place(walk, odd, place, kind, out):
    check(*WALKS[walk], kind, out, True, odd, place)


@pytest.mark.parametrize("walk", WALKS)
def test_nan_stays_in_its_row(walk):
    cols, rows = WALKS[walk]
    x = rand((rows, cols), 1).bfloat16()
    clean = bg.rmsnorm(x)
    bad = [rows // 3, rows // 2, rows - 1]
    x[bad, 17] = float("nan")
    got = bg.rmsnorm(x)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.isnan(got[bad]).all() and torch.equal(got[keep], clean[keep])
