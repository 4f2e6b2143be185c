"""Refusals of the layer norm, the norms' gradients and the products' gradients, without a GPU: every check comes before
any device work."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

F32, F16, BF16, MX = 0, 1, 2, 3
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from broadcast_implicit_gemm_gb300 import _build
    _build.build()
    return bg.load_library()


def layernorm(lib, rows=2, cols=8, dt=F16, x=256, ldx=8, r=None, ldr=0, g=None, b=None, h=None, ldh=0, out_dt=F16, out=256,
              ldo=8, s=None, mean=None, rstd=None):
    return lib.layernorm_run(rows, cols, dt, x, ldx, r, ldr, g, b, 1e-5, h, ldh, out_dt, out, ldo, s, mean, rstd, None)


def layer_back(lib, rows=2, cols=8, dt=F16, d=256, ldd=8, x=256, ldx=8, mean=256, rstd=256, w=None, s=None, lds=0, dx=256,
               ldo=8, dw=256, db=256, space=256, size=1 << 20):
    return lib.layernorm_backward_run(rows, cols, dt, d, ldd, x, ldx, mean, rstd, w, s, lds, dx, ldo, dw, db, space, size, None)


def rms_back(lib, rows=2, cols=8, dt=F16, d=256, ldd=8, x=256, ldx=8, w=None, s=None, lds=0, dx=256, ldo=8, dw=256, space=256,
             size=1 << 20):
    return lib.rmsnorm_backward_run(rows, cols, dt, d, ldd, x, ldx, w, 1e-6, s, lds, dx, ldo, dw, space, size, None)


@pytest.mark.parametrize("bad", [
    {"rows": -1}, {"cols": 0}, {"dt": 3}, {"dt": -1}, {"out_dt": 4}, {"x": None}, {"out": None}, {"ldx": 7}, {"ldo": 7},
    {"r": 256, "ldr": 7}, {"h": 256, "ldh": 7}, {"x": 257}, {"r": 257, "ldr": 8}, {"g": 258}, {"b": 257}, {"out_dt": MX},
    {"s": 256}, {"out_dt": MX, "s": 264}, {"mean": 258}, {"rstd": 257}])
def test_layernorm_refuses(lib, bad):
    assert layernorm(lib, **bad) == INVALID


def test_layernorm_refuses_another_16_bit_type_and_width(lib):
    assert layernorm(lib, dt=F16, out_dt=BF16) == UNSUPPORTED
    assert layernorm(lib, cols=2 ** 30 + 1, ldx=2 ** 31, ldo=2 ** 31) == UNSUPPORTED


BACK = [{"rows": -1}, {"cols": 0}, {"dt": 3}, {"dt": -1}, {"d": None}, {"x": None}, {"dx": None}, {"dw": None}, {"ldd": 7}, {"ldx": 7},
        {"ldo": 7}, {"s": 256, "lds": 7}, {"d": 257}, {"x": 257}, {"dx": 257}, {"s": 257, "lds": 8}, {"w": 258}, {"dw": 258},
        {"space": None}, {"space": 264}, {"size": 63}]


@pytest.mark.parametrize("bad", BACK + [{"db": None}, {"db": 257}, {"mean": None}, {"rstd": None}, {"mean": 258}, {"rstd": 258}])
def test_layernorm_backward_refuses(lib, bad):
    assert layer_back(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", BACK)
def test_rmsnorm_backward_refuses(lib, bad):
    assert rms_back(lib, **bad) == INVALID


def test_no_rows_is_no_norm(lib):
    assert layernorm(lib, rows=0) == 0


def test_norm_backward_workspace(lib):
    q = bg.norm_backward_workspace_bytes
    assert q(0, 8) == 0 and q(8, 0) == 0
    assert q(1, 8192) == 2 * 8192 * 4                          # a row of partial sums of each gradient
    assert q(10000, 8192) == 152 * 2 * 8192 * 4                # one of each block of a wave
    assert q(10000, 256) == 152 * 8 * 2 * 256 * 4
    assert q(5, 8193) == (5 * 2 * 8193 + 5) * 4                # and a root per row of long ones
    assert q(2 ** 31 - 1, 2 ** 30) == (2 * 2 ** 30 + 2 ** 31 - 1) * 4


def test_python_refusals():
    """The tensor forms check shapes, types and devices before they call the library."""
    x = torch.zeros(4, 16, dtype=torch.float16)
    v = torch.zeros(4)
    for call in (lambda: bg.layernorm(x), lambda: bg.layernorm_backward(x, x, v, v), lambda: bg.rmsnorm_backward(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
