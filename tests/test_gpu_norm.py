"""GPU parity of the RMS norm and of the MXFP8 quantisation against their 64-bit definitions."""
import numpy as np
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg
from tests import layer_ref as lr

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "mx": torch.float8_e4m3fn}


def rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def strided(t, pad, dtype, offset=0):
    big = torch.full((t.shape[0], t.shape[1] + pad + offset), float("nan")).to(dtype).cuda()
    big[:, offset: offset + t.shape[1]] = t.to(dtype).cuda()
    return big[:, offset: offset + t.shape[1]]


def f64(t):
    return t.cpu().double().numpy()


def norm64(x, r, g, eps):
    """Reference, sum, and the bound before the output's rounding: h is rounded once to fp32, the squares' sum is
    off by at most (cols + 1) ulp of fp32 for any order (half of it after the root), the root, quotient and two
    products by an ulp each."""
    h = x if r is None else x + r
    cols = x.shape[1]
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * (1.0 if g is None else g)
    return y, h, np.abs(y) * ((cols + 1) / 2 + 6) * 2.0 ** -23


def norm_case(rows, cols, kind="bf16", out="same", residual=True, weight=True, pad=0, offset=0, eps=1e-6, seed=1, size=1.0):
    x = strided(rand((rows, cols), seed) * size, pad, TD[kind], offset)
    r = strided(rand((rows, cols), seed + 1) * size, pad, TD[kind], offset) if residual else None
    g = (1 + 0.2 * rand((cols,), seed + 2)).cuda() if weight else None
    odt = TD[kind] if out == "same" else TD[out]
    h = strided(torch.zeros(rows, cols), pad, TD[kind], offset) if residual else None
    got = bg.rmsnorm(x, g, residual=r, eps=eps, out_dtype=odt, sum_out=h)
    torch.cuda.synchronize()
    ref, hs, d = norm64(f64(x), f64(r) if residual else None, f64(g) if weight else None, eps)
    what = f"{rows}x{cols} {kind}->{out}"
    if residual:
        lr.check_float(got[-1], hs, 2.0 ** -24 * np.abs(hs), what + " sum")
        if pad:
            assert torch.isnan(h._base[:, offset + cols:]).all()
    if out == "mx":
        lr.check_mx(got[0], got[1], ref, d, what)
        assert lr.padding_codes_are_zero(got[1], rows, cols)
    else:
        lr.check_float(got[0] if residual else got, ref, d, what)


@pytest.mark.parametrize("cols", [1, 2, 7, 8, 31, 32, 33, 127, 128, 255, 1000, 1023, 1024, 1025, 2049, 4096, 4104, 8192, 16384,
                                  16392, 20001])
@pytest.mark.parametrize("kind,out", [("bf16", "same"), ("f16", "mx"), ("bf16", "f32")])
def test_norm_widths(cols, kind, out):
    norm_case(5, cols, kind, out, seed=cols)


@pytest.mark.parametrize("rows", [1, 2, 31, 33, 127, 129, 300])
@pytest.mark.parametrize("out", ["same", "mx"])
def test_norm_rows(rows, out):
    norm_case(rows, 520, "bf16", out, seed=rows)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["same", "f32", "mx"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("weight", [False, True])
def test_norm_forms(kind, out, residual, weight):
    norm_case(9, 776, kind, out, residual, weight)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 8), (3, 1), (24, 16)])
@pytest.mark.parametrize("out", ["same", "mx", "f32"])
def test_norm_strides(pad, offset, out):
    norm_case(40, 648, "f16", out, pad=pad, offset=offset)


def test_norm_of_nothing_and_of_large_values():
    x = torch.zeros(3, 256, dtype=torch.float16, device="cuda")
    assert not bg.rmsnorm(x).any()
    q, s = bg.rmsnorm(x, out_dtype=torch.float8_e4m3fn)
    assert not q.float().any() and not s.view(torch.uint8).any()
    assert bg.rmsnorm(x[:0]).shape == (0, 256)
    norm_case(4, 512, "f16", "same", size=1e4)     # squares beyond f16's range
    norm_case(4, 512, "bf16", "mx", size=1e-3, eps=1e-12)


def test_norm_nan_stays_in_its_row():
    x = rand((6, 300), 1).bfloat16().cuda()
    clean = bg.rmsnorm(x)
    x[2, 17] = float("nan")
    got = bg.rmsnorm(x)
    keep = [0, 1, 3, 4, 5]
    assert torch.isnan(got[2]).all() and torch.equal(got[keep], clean[keep])


def test_norm_sum_in_place():
    x, r = rand((20, 768), 1).half().cuda(), rand((20, 768), 2).half().cuda()
    y, h = bg.rmsnorm(x, residual=r)
    y2, h2 = bg.rmsnorm(x, residual=r, sum_out=r)
    assert h2 is r and torch.equal(h, r) and torch.equal(y, y2)


# --------------------------------------------------------------------- quantisation

def quantize_case(x):
    q, s = bg.mx_quantize(x)
    torch.cuda.synchronize()
    rows, cols = x.shape
    ref = f64(x)
    assert np.array_equal(lr.codes_of(s, rows, cols), lr.code_of(lr.group_max(ref)))
    lr.check_mx(q, s, ref, np.zeros_like(ref))
    assert lr.padding_codes_are_zero(s, rows, cols)
    return q, s


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (1, 32), (2, 33), (5, 127), (129, 128), (300, 2056), (33, 4097), (260, 640)])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_quantize(rows, cols, kind, pad):
    spread = torch.exp2(torch.randint(-10, 10, (rows, cols), generator=torch.Generator().manual_seed(rows)).float())
    quantize_case(strided(rand((rows, cols), cols) * spread, pad, TD[kind]))


def test_quantize_at_the_steps():
    """Largest values at and beside 448 times a power of two, and powers of two from the smallest to the largest."""
    top = torch.tensor([448.0, 448.0 * (1 + 2 ** -23), 448.0 * (1 - 2 ** -24), 449.0, 256.0, 1.0, 1.75, 1.7500001])
    x = torch.zeros(8, 64)
    x[:, 5], x[:, 40] = top, top * 2.0 ** -30
    quantize_case(x.cuda())
    e = torch.arange(-148, 127).float()
    y = torch.zeros(len(e), 32)
    y[:, 3] = torch.exp2(e.double()).float()
    quantize_case(y.cuda())


def test_quantize_rounds_to_even():
    """Every midpoint of two neighbouring e4m3 values, at scale 1 (448 in the group)."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (codes[:-1] + codes[1:]) / 2
    x = torch.zeros(len(mid), 32)
    x[:, 0], x[:, 1], x[:, 2] = 448.0, mid, -mid
    q, s = bg.mx_quantize(x.cuda())
    want = torch.where(torch.arange(len(mid)) % 2 == 0, codes[:-1], codes[1:])
    assert (s.view(torch.uint8).cpu().reshape(-1)[0] == 127)
    assert torch.equal(q.float().cpu()[:, 1], want) and torch.equal(q.float().cpu()[:, 2], -want)


def test_quantize_infinities_and_nans():
    x = rand((3, 96), 1).cuda()
    clean, cs = bg.mx_quantize(x)
    x[1, 40], x[2, 70] = float("inf"), float("nan")
    q, s = bg.mx_quantize(x)
    code = lr.codes_of(s, 3, 96)
    assert code[1, 1] == 255 and code[2, 2] == 255 and (np.delete(code.reshape(-1), [4, 8]) < 255).all()
    assert torch.isnan(q.float()[1, 32:64]).all() and torch.isnan(q.float()[2, 64:]).all()
    assert torch.equal(q.float()[0], clean.float()[0]) and torch.equal(q.float()[1, :32], clean.float()[1, :32])
