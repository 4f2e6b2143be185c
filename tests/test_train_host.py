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


def layernorm(lib, rows=2, cols=8, dt=F16, x=256, ldx=8, r=None, ldr=0, g=None, b=None, h=None, ldh=0, out_dt=F16, out=512,
              ldo=8, s=None, mean=None, rstd=None):
    return lib.layernorm_run(rows, cols, dt, x, ldx, r, ldr, g, b, 1e-5, h, ldh, out_dt, out, ldo, s, mean, rstd, None)


def layer_back(lib, rows=2, cols=8, dt=F16, d=256, ldd=8, x=256, ldx=8, mean=256, rstd=256, w=None, s=None, lds=0, dx=512,
               ldo=8, dw=1024, db=2048, space=256, size=1 << 20):
    return lib.layernorm_backward_run(rows, cols, dt, d, ldd, x, ldx, mean, rstd, w, s, lds, dx, ldo, dw, db, space, size, None)


def rms_back(lib, rows=2, cols=8, dt=F16, d=256, ldd=8, x=256, ldx=8, w=None, s=None, lds=0, dx=256, ldo=8, dw=256, space=256,
             size=1 << 20):
    return lib.rmsnorm_backward_run(rows, cols, dt, d, ldd, x, ldx, w, 1e-6, s, lds, dx, ldo, dw, space, size, None)


@pytest.mark.parametrize("bad", [
    {"rows": -1}, {"cols": 0}, {"dt": 3}, {"dt": -1}, {"out_dt": 4}, {"x": None}, {"out": None}, {"ldx": 7}, {"ldo": 7},
    {"r": 256, "ldr": 7}, {"h": 256, "ldh": 7}, {"x": 257}, {"r": 257, "ldr": 8}, {"g": 258}, {"b": 257}, {"out_dt": MX},
    {"s": 256}, {"out_dt": MX, "s": 264}, {"mean": 258}, {"rstd": 257}, {"mean": 1024, "rstd": 1024}, {"h": 512, "ldh": 8}])
def test_layernorm_refuses(lib, bad):
    assert layernorm(lib, **bad) == INVALID


def test_layernorm_refuses_another_16_bit_type_and_width(lib):
    assert layernorm(lib, dt=F16, out_dt=BF16) == UNSUPPORTED
    assert layernorm(lib, cols=2 ** 30 + 1, ldx=2 ** 31, ldo=2 ** 31) == UNSUPPORTED


BACK = [{"rows": -1}, {"cols": 0}, {"dt": 3}, {"dt": -1}, {"d": None}, {"x": None}, {"dx": None}, {"dw": None}, {"ldd": 7}, {"ldx": 7},
        {"ldo": 7}, {"s": 256, "lds": 7}, {"d": 257}, {"x": 257}, {"dx": 257}, {"s": 257, "lds": 8}, {"w": 258}, {"dw": 258},
        {"space": None}, {"space": 264}, {"size": 63}]


@pytest.mark.parametrize("bad", BACK + [{"db": None}, {"db": 257}, {"mean": None}, {"rstd": None}, {"mean": 258}, {"rstd": 258}, {"db": 1024}])
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
    assert q(10000, 256) == 152 * 4 * 2 * 256 * 4              # (blocks beside each other have four turns each)
    assert q(10000, 20000) == 38 * 2 * 20000 * 4               # or of a cluster of four
    assert q(5, 65537) == (5 * 2 * 65540 + 5) * 4              # and a root per row of longer ones
    assert q(2 ** 31 - 1, 2 ** 30) == (2 * 2 ** 30 + 2 ** 31 - 1) * 4


def test_python_refusals():
    """The tensor forms check shapes, types and devices before they call the library."""
    x = torch.zeros(4, 16, dtype=torch.float16)
    v = torch.zeros(4)
    for call in (lambda: bg.layernorm(x), lambda: bg.layernorm_backward(x, x, v, v), lambda: bg.rmsnorm_backward(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def gated(lib, M=4, N=8, K=16, dt=F16, x=256, ldx=16, wg=256, ldg=16, wu=256, ldu=16, bg_=None, bu=None, act=4, out=512, ldo=8,
          g=None, ldg2=0, u=None, ldu2=0, ws=None, size=0):
    return lib.matmul_gated_run(M, N, K, dt, x, ldx, wg, ldg, wu, ldu, bg_, bu, act, out, ldo, g, ldg2, u, ldu2, ws, size, None)


def linear_back(lib, M=4, N=8, K=16, dt=F16, d=256, ldd=8, x=256, ldx=16, w=256, ldw=16, dx=512, lddx=16, dw=1024, lddw=16, db=None,
                ws=256, size=1 << 20):
    return lib.matmul_backward_run(M, N, K, dt, d, ldd, x, ldx, w, ldw, dx, lddx, dw, lddw, db, ws, size, None)


def gated_back(lib, M=4, N=8, K=16, dt=F16, d=256, ldd=8, x=256, ldx=16, wg=256, ldg=16, wu=256, ldu=16, g=256, ldg2=8, u=256, ldu2=8,
               act=4, dx=512, lddx=16, dwg=1024, lddwg=16, dwu=2048, lddwu=16, dbg=None, dbu=None, ws=256, size=1 << 20):
    return lib.matmul_gated_backward_run(M, N, K, dt, d, ldd, x, ldx, wg, ldg, wu, ldu, g, ldg2, u, ldu2, act, dx, lddx, dwg, lddwg,
                                         dwu, lddwu, dbg, dbu, ws, size, None)


SIZES = [{"M": -1}, {"N": 0}, {"K": 0}, {"K": -5}, {"dt": 3}, {"dt": -1}, {"x": None}, {"ldx": 15}, {"x": 257}]


@pytest.mark.parametrize("bad", SIZES + [
    {"wg": None}, {"wu": None}, {"out": None}, {"ldg": 15}, {"ldu": 15}, {"ldo": 7}, {"wg": 257}, {"wu": 257}, {"out": 257},
    {"bg_": 258}, {"bu": 257}, {"act": 5}, {"act": -1}, {"g": 256, "ldg2": 7}, {"u": 256, "ldu2": 7}, {"g": 257, "ldg2": 8},
    {"u": 257, "ldu2": 8}, {"ws": 264}, {"ldx": 17}, {"wg": 258}, {"ldu": 17, "ws": 256, "size": 255},
    {"g": 512, "ldg2": 8}, {"g": 1024, "ldg2": 8, "u": 1024, "ldu2": 8}, {"u": 256, "ldu2": 8}])
def test_gated_refuses(lib, bad):
    assert gated(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", SIZES + [
    {"d": None}, {"w": None}, {"dx": None}, {"dw": None}, {"ldd": 7}, {"ldw": 15}, {"lddx": 15}, {"lddw": 15}, {"d": 257}, {"w": 257},
    {"dx": 257}, {"dw": 257}, {"db": 258}, {"ws": None}, {"ws": 264}, {"size": 255},
    {"dx": 256}, {"dw": 256}, {"dw": 512}, {"db": 1024}])
def test_matmul_backward_refuses(lib, bad):
    assert linear_back(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", SIZES + [
    {"d": None}, {"wg": None}, {"wu": None}, {"g": None}, {"u": None}, {"dx": None}, {"dwg": None}, {"dwu": None}, {"ldd": 7}, {"ldg": 15},
    {"ldu": 15}, {"ldg2": 7}, {"ldu2": 7}, {"lddx": 15}, {"lddwg": 15}, {"lddwu": 15}, {"d": 257}, {"wg": 257}, {"wu": 257}, {"g": 257},
    {"u": 257}, {"dx": 257}, {"dwg": 257}, {"dwu": 257}, {"dbg": 258}, {"dbu": 257}, {"act": 5}, {"act": -1}, {"ws": None}, {"ws": 264},
    {"size": 255}, {"dwg": 256}, {"dwu": 1024}, {"dx": 2048}, {"dbg": 4096, "dbu": 4096}])
def test_gated_backward_refuses(lib, bad):
    assert gated_back(lib, **bad) == INVALID


def test_products_refuse_32_bit_operands_and_huge_sizes(lib):
    for call in (gated, linear_back, gated_back):
        assert call(lib, dt=F32) == UNSUPPORTED
        assert call(lib, M=2 ** 30 + 1) == UNSUPPORTED


def test_no_tokens_is_no_gated_layer(lib):
    assert gated(lib, M=0) == 0


def test_product_workspaces(lib):
    """A copy of each operand off the 16-byte grid; the gradients' own: shares of dx, sums over runs of rows, and a gated
    layer's two gradients."""
    q = bg.matmul_gated_workspace_bytes
    assert q(1000, 512, 256, 256, 256, 256, 256, 256, 256) == 0
    assert q(1000, 512, 257, 256, 257, 256, 264, 256, 264) == -(-1000 * 528 // 256) * 256
    assert q(1000, 512, 257, 256, 264, 256, 257, 256, 257) == 2 * -(-512 * 528 // 256) * 256
    assert q(0, 5, 5, 256, 5, 256, 5, 256, 5) == 0
    q = bg.matmul_backward_workspace_bytes
    assert q(0, 5, 5, 256, 5, 256, 5, 256, 5) == 0 and q(2 ** 30 + 1, 5, 5, 256, 5, 256, 5, 256, 5) == 0
    plain = q(4096, 4096, 4096, 256, 4096, 256, 4096, 256, 4096)
    assert plain == 76 * 4096 * 4                              # tiles enough: no shares, runs of rows alone
    assert q(4096, 4096, 4096, 256, 4097, 256, 4096, 256, 4096) == plain + 4096 * 4096 * 2
    assert q(100, 4096, 4096, 256, 4096, 256, 4096, 256, 4096) > 100 * 4096 * 4
    q = bg.matmul_gated_backward_workspace_bytes
    assert q(4096, 4096, 4096, 256, 4096, 256, 4096, 256, 4096) == 2 * plain + 2 * 4096 * 4096 * 2


def test_python_refusals_of_products():
    x, w = torch.zeros(4, 16, dtype=torch.float16), torch.zeros(8, 16, dtype=torch.float16)
    d = torch.zeros(4, 8, dtype=torch.float16)
    for call in (lambda: bg.matmul_gated(x, w, w), lambda: bg.matmul_backward(d, x, w),
                 lambda: bg.matmul_gated_backward(d, x, w, w, d, d)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_what_is_no_tensor_or_has_no_memory():
    """Errors are Python's, also where torch's C++ side throws: a fake tensor has no address."""
    x = torch.zeros(4, 16, dtype=torch.float16)
    for bad in (None, 3, [1.0], "x"):
        with pytest.raises((TypeError, AttributeError)):
            bg.matmul(bad, x, out=x)
        with pytest.raises(TypeError, match="expected a tensor"):
            bg._layer().gated(bad, x, x, None, None, 0, x, None, None, None)
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        fake = torch.empty((4, 16), dtype=torch.float16, device="cuda")
        with pytest.raises((RuntimeError, ValueError)):
            bg.matmul(fake, fake, out=fake)
    for t in (torch.zeros(4, dtype=torch.float16), torch.zeros(2, 2, 2), torch.zeros(())):
        with pytest.raises(ValueError, match="2-D CUDA"):
            bg._layer().quantize(t, t, t, None)


def test_a_view_that_is_still_to_be_negated_is_refused():
    """Its memory holds the values' negatives."""
    x = torch._neg_view(torch.ones(2, 8))
    for call in (lambda: bg.layernorm(x), lambda: bg.rmsnorm(x), lambda: bg.matmul(x, torch.ones(3, 8))):
        with pytest.raises(ValueError, match="negated"):
            call()
