"""Refusals of the transformer-layer entry points, without a GPU: every check comes before any device work."""
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


def matmul(lib, M=4, N=8, K=16, dt=F16, x=256, ldx=16, w=256, ldw=16, bias=None, act=0, comb=0, odt=F16, o=None, ldo2=0,
           out_dt=F16, out=256, ldo=8, ws=None):
    return lib.matmul_run(M, N, K, dt, x, ldx, w, ldw, bias, act, comb, odt, o, ldo2, out_dt, out, ldo, ws, 0, None)


def matmul_mx(lib, M=4, N=8, K=16, x=256, ldx=16, xs=256, w=256, ldw=16, ws=256, bias=None, act=0, comb=0, odt=F16, o=None,
              ldo2=0, out_dt=F16, out=256, ldo=8, outs=None):
    return lib.matmul_mx_run(M, N, K, x, ldx, xs, w, ldw, ws, bias, act, comb, odt, o, ldo2, out_dt, out, ldo, outs, None, 0, None)


def norm(lib, rows=2, cols=8, dt=F16, x=256, ldx=8, r=None, ldr=0, g=None, h=None, ldh=0, out_dt=F16, out=256, ldo=8, s=None):
    return lib.rmsnorm_run(rows, cols, dt, x, ldx, r, ldr, g, 1e-6, h, ldh, out_dt, out, ldo, s, None)


def quantize(lib, rows=2, cols=8, dt=F16, x=256, ldx=8, out=256, ldo=8, s=256):
    return lib.mx_quantize_run(rows, cols, dt, x, ldx, out, ldo, s, None)


@pytest.mark.parametrize("bad", [
    {"M": -1}, {"N": 0}, {"K": 0}, {"K": -5}, {"dt": 3}, {"dt": -1}, {"out_dt": 3}, {"out_dt": 9}, {"x": None}, {"w": None},
    {"out": None}, {"ldx": 15}, {"ldw": 15}, {"ldo": 7}, {"x": 257}, {"w": 257}, {"out": 257}, {"bias": 258}, {"act": 5},
    {"act": -1}, {"comb": 3}, {"comb": 1}, {"comb": 1, "o": 256, "ldo2": 7}, {"comb": 2, "o": 257, "ldo2": 8},
    {"comb": 1, "o": 256, "ldo2": 8, "odt": 3}, {"ws": 264}, {"ldx": 17}, {"w": 258}])
def test_matmul_refuses(lib, bad):
    assert matmul(lib, **bad) == INVALID


def test_matmul_refuses_32_bit_operands(lib):
    assert matmul(lib, dt=F32) == UNSUPPORTED


@pytest.mark.parametrize("bad", [
    {"M": -1}, {"N": 0}, {"K": 0}, {"xs": None}, {"ws": None}, {"xs": 264}, {"ws": 260}, {"out_dt": 4}, {"out_dt": MX},
    {"out_dt": F16, "outs": 256}, {"out_dt": MX, "outs": 264}, {"ldx": 15}, {"x": None}, {"bias": 257}])
def test_matmul_mx_refuses(lib, bad):
    assert matmul_mx(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    {"rows": -1}, {"cols": 0}, {"dt": 3}, {"out_dt": 4}, {"x": None}, {"out": None}, {"ldx": 7}, {"ldo": 7}, {"r": 256, "ldr": 7},
    {"h": 256, "ldh": 7}, {"x": 257}, {"r": 257, "ldr": 8}, {"g": 258}, {"out_dt": MX}, {"s": 256}, {"out_dt": MX, "s": 264}])
def test_norm_refuses(lib, bad):
    assert norm(lib, **bad) == INVALID


def test_norm_refuses_another_16_bit_type(lib):
    assert norm(lib, dt=F16, out_dt=BF16) == UNSUPPORTED


@pytest.mark.parametrize("bad", [{"rows": -1}, {"cols": 0}, {"dt": 3}, {"x": None}, {"out": None}, {"s": None}, {"ldx": 7}, {"ldo": 7},
                                 {"x": 257}, {"s": 264}])
def test_quantize_refuses(lib, bad):
    assert quantize(lib, **bad) == INVALID


def test_no_rows_is_no_work(lib):
    assert matmul(lib, M=0) == 0 and matmul_mx(lib, M=0) == 0 and norm(lib, rows=0) == 0 and quantize(lib, rows=0) == 0


def test_scale_bytes(lib):
    assert bg.bigemm_mx_scale_bytes(1, 1) == 512 and bg.bigemm_mx_scale_bytes(129, 4096) == 2 * 32 * 512
    assert bg.bigemm_mx_scale_bytes(0, 5) == 0 and bg.bigemm_mx_scale_bytes(2 ** 31 - 1, 2 ** 31 - 1) == (2 ** 24) ** 2 * 512
    assert bg.mx_scale_shape(129, 4096) == (2, 32, 32, 4, 4)


def test_python_refusals():
    """The tensor forms check shapes, types and devices before they call the library."""
    x = torch.zeros(4, 16, dtype=torch.float16)
    for call in (lambda: bg.matmul(x, x), lambda: bg.rmsnorm(x), lambda: bg.mx_quantize(x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_workspace_bytes(lib):
    """A copy of each operand off the 16-byte grid, its rows on it."""
    q = bg.matmul_workspace_bytes
    assert q(1000, 512, 256, F16, 256, 256, 256, 256) == 0
    assert q(1000, 512, 257, F16, 256, 257, 256, 264) == -(-1000 * 528 // 256) * 256
    assert q(1000, 512, 257, F16, 256, 264, 256, 257) == -(-512 * 528 // 256) * 256
    assert q(1000, 512, 256, F16, 258, 256, 258, 256) == 1000 * 512 + 512 * 512
    assert q(1000, 512, 250, MX, 256, 250, 256, 256) == 1000 * 256
    assert q(0, 5, 5, F16, 256, 5, 256, 5) == 0
