"""Offsets past 2^31 elements, and more rows and tokens than a grid's wave, in the layer norm, the norms' gradients and
the products' gradients: all rows are zero but a few near both ends, so that the whole result is known from those."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg
from tests import train_ref as tr

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(BF)


def ends(rows, n=3):
    return [*range(n), *range(rows - n, rows)]


def quiet():
    torch.cuda.synchronize()
    assert bg.bigemm_last_device_error() == 0


@pytest.mark.parametrize("rows,cols", [(270_001, 8000), (1_200_003, 1801)])
def test_norm_of_many_elements(rows, cols):
    """2.16e9 elements, on the grid and off it."""
    assert rows * cols > 2 ** 31
    at = ends(rows)
    x = torch.zeros((rows, cols), dtype=BF, device="cuda")
    x[at] = rand((len(at), cols), 1)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    y = bg.layernorm(x, mean_out=mean, rstd_out=rstd)
    quiet()
    ref, ey, _, m, em, r, er = tr.layernorm64(x[at], None, None, None, 1e-5)
    tr.check(y[at], ref, ey, "y")
    tr.check(mean[at], m, em, "mean")
    assert not y[len(at): rows - len(at)].any()
    del y
    d = torch.zeros_like(x)
    d[at] = rand((len(at), cols), 2)
    dx, dw, db = bg.layernorm_backward(d, x, mean, rstd)
    quiet()
    ref = tr.layernorm_backward64(d[at], x[at], mean[at], rstd[at], None, None)
    tr.check(dx[at], *ref["dx"], "dx")
    assert not dx[len(at): rows - len(at)].any()
    # the other rows add zeros: the sums are these rows'
    tr.check(dw, *ref["dw"], "dw")
    tr.check(db, *ref["db"], "db")
    dx, dw = bg.rmsnorm_backward(d, x, dx=dx)
    quiet()
    ref = tr.rmsnorm_backward64(d[at], x[at], None, 1e-6, None)
    tr.check(dx[at], *ref["dx"], "dx")
    tr.check(dw, *ref["dw"], "dw")


def test_gated_layer_of_many_elements():
    """140 000 tokens by 16 384 channels, 2.3e9 elements."""
    M, N, K = 140_001, 16384, 64
    at = ends(M)
    x = torch.zeros((M, K), dtype=BF, device="cuda")
    x[at] = rand((len(at), K), 1)
    wg, wu = (rand((N, K), s) * 0.125 for s in (2, 3))
    g, u = torch.empty((M, N), dtype=BF, device="cuda"), torch.empty((M, N), dtype=BF, device="cuda")
    y = bg.matmul_gated(x, wg, wu, gate_out=g, up_out=u)
    quiet()
    ref = tr.gated64(x[at], wg, wu, None, None, "silu")
    for name, t in (("y", y), ("g", g), ("u", u)):
        tr.check(t[at], *ref[name], name)
        assert not t[len(at): M - len(at)].any()
    d = y.zero_()
    d[at] = rand((len(at), N), 4)
    dbg, dbu = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    dx, dwg, dwu = bg.matmul_gated_backward(d, x, wg, wu, g, u, dbias_gate=dbg, dbias_up=dbu)
    quiet()
    ref = tr.gated_backward64(d[at], x[at], wg, wu, g[at], u[at], "silu")
    tr.check(dx[at], *ref["dx"], "dx")
    assert not dx[len(at): M - len(at)].any()
    for name, t in (("dwg", dwg), ("dwu", dwu), ("dbg", dbg), ("dbu", dbu)):
        tr.check(t, *ref[name], name)
    dx, dw = bg.matmul_backward(d, x, wg, dbias=dbg)
    quiet()
    ref = tr.product_backward64(d[at], x[at], wg)
    tr.check(dx[at], *ref["dx"], "dx")
    tr.check(dw, *ref["dw"], "dw")
    tr.check(dbg, *ref["db"], "db")
