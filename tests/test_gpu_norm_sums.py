"""Sums over all rows in the norms' gradients, with a bound from how the kernels add (csrc/norm_back.cuh): U = 2^-24 of the
sum of magnitudes for each addition that a term passes through.

Up to 65536 columns a thread adds the rows of its walk, the four warps of a narrow row's block join (3), and each walk
leaves a row of sums: 152 blocks, or 76, at least 36 and at least 14 clusters of 2, 4 and 8 (groups of neighbouring SMs
decide how many fit), as many times over as blocks stand side by side.  Longer rows: runs of rows, five at 70 008 columns,
in pieces of 256 rows which are joined then.  In either case the rows of sums go to 64 threads (16 warps of 4 lanes to a
column) and are joined by 2 shuffles and 15 additions."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg
from tests import train_ref as tr

pytestmark = pytest.mark.gpu

U = tr.U


def adds(rows, cols):
    if cols > 65536:
        runs = max(1, min(rows, -(-1216 // -(-cols // 256))))
        mine = -(-rows // runs)
        return min(mine, 256) + -(-mine // 256) + runs / 64 + 18
    walks = 152 if cols <= 8192 else 76 if cols <= 16384 else 36 if cols <= 32768 else 14
    at_once = 4 if cols <= 256 else 1
    return rows / (min(walks, rows) * at_once) + 1 + 3 + 2432 / 64 + 18


def rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def expect(got, ref, bound, what):
    over = ((got.double() - ref).abs() / (bound + U * ref.abs() + 1e-300))
    assert bool(torch.isfinite(got).all()) and float(over.max()) <= 1, f"{what}: {float(over.max()):.3f} of the bound"


@pytest.mark.parametrize("rows,cols", [(10000, 512), (30000, 200), (6000, 1001), (4000, 8192), (4000, 12000), (4000, 20000),
                                       (4000, 40000), (4000, 70008), (700, 320000)])
def test_random_rows(rows, cols):
    x, d = rand((rows, cols), 1).bfloat16(), rand((rows, cols), 2).bfloat16()
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    bg.layernorm(x, mean_out=mean, rstd_out=rstd)
    _, dw, db = bg.layernorm_backward(d, x, mean, rstd)
    _, dwr = bg.rmsnorm_backward(d, x)
    n = adds(rows, cols)
    for c0 in range(0, cols, 4096):
        part = slice(c0, min(c0 + 4096, cols))
        xs, ds = x[:, part].double(), d[:, part].double()
        xh = (xs - mean.double()[:, None]) * rstd.double()[:, None]
        expect(db[part], ds.sum(0), n * U * ds.abs().sum(0), "db")
        # each term: a difference, two products
        expect(dw[part], (ds * xh).sum(0), (n + 4) * U * (ds * xh).abs().sum(0)
               + 2 * U * (ds * rstd.double()[:, None] * xs).abs().sum(0), "dw")
    # the root: a mean of squares (train_ref's row_adds for the sum), an addition, a reciprocal root of 2 ulp
    roots = torch.cat([1 / torch.sqrt((x[i: i + 500].double() ** 2).mean(-1) + 1e-6) for i in range(0, rows, 500)])
    e = (cols / 512 + 40) / 2 + 6
    for c0 in range(0, cols, 4096):
        part = slice(c0, min(c0 + 4096, cols))
        t = d[:, part].double() * x[:, part].double() * roots[:, None]
        expect(dwr[part], t.sum(0), (n + 4 + e) * U * t.abs().sum(0), "dw of rmsnorm")


def test_small_terms_behind_a_large_one():
    """One row of 2^24 at the head of each run of long rows and ones behind it: a single accumulator would lose every one."""
    rows, cols = 4000, 70008
    runs = 5
    d = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")
    heads = [rows * i // runs for i in range(runs)]
    d[heads] = 2.0 ** 24
    x = torch.ones_like(d)
    zeros, ones = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    _, dw, db = bg.layernorm_backward(d, x, zeros, ones)       # xh = 1
    want = runs * 2.0 ** 24 + rows - runs
    bound = adds(rows, cols) * U * want
    assert bound < rows / 2                                    # most of the small terms count
    for got in (dw, db):
        assert float((got.double() - want).abs().max()) <= bound
