"""MXFP8 rows of more than 2^29 columns: their scales lie more than 2^31 bytes apart."""
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

pytestmark = pytest.mark.gpu

COLS = (1 << 29) + 256 + 40
MX = torch.float8_e4m3fn


def wide():
    """One row whose groups differ in size from their neighbours and from those 2^29 columns away."""
    n = torch.arange(COLS, dtype=torch.int32, device="cuda")
    x = torch.exp2((n // 32 % 13 - 6).float()).half()
    return (x * (1 + (n % 29).half() / 32) * (1 - 2 * (n % 3 == 0).half())).view(1, COLS)


def row_scales(s):
    """The codes of row 0, a group after the other."""
    return s.view(torch.uint8)[0, :, 0, 0, :].reshape(-1)


def test_quantize():
    x = wide()
    q, s = bg.mx_quantize(x)
    full = torch.zeros(s.shape[1] * 128, dtype=torch.float16, device="cuda")
    full[:COLS] = x[0]
    bits = full.view(-1, 32).abs().amax(-1).float().view(torch.int32)
    code = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp(min=0)
    assert torch.equal(row_scales(s), code.to(torch.uint8))
    assert not s.view(torch.uint8)[0, :, 1:].any() and not s.view(torch.uint8)[0, :, 0, 1:].any()
    for at in range(0, COLS, 1 << 27):
        part = slice(at, min(COLS, at + (1 << 27)))
        want = torch.ldexp(x[0, part].float(), 127 - code[at // 32: -(-part.stop // 32)].repeat_interleave(32)[: part.stop - at])
        assert torch.equal(q[0, part].view(torch.uint8), want.to(MX).view(torch.uint8))


def test_norm():
    x = wide()
    q, s = bg.rmsnorm(x, out_dtype=MX)
    p, t = bg.mx_quantize(bg.rmsnorm(x, out_dtype=torch.float32))
    assert torch.equal(s.view(torch.uint8), t.view(torch.uint8)) and torch.equal(q.view(torch.uint8), p.view(torch.uint8))
