"""The layer operators together: a gated MLP block against its 64-bit form.

Bounds, of the whole output's 2-norm: in 16 bits the stored intermediates (norm, up, gated product, output) are each
rounded once, for bfloat16 by 2^-8 at most and below 2^-9 in the 2-norm, four of them in sequence with gains near
one: below 4 * 2^-9.  MXFP8 rounds x's and each weight's elements to 4 significant bits, 2^-5 / sqrt 3 relative in the
mean for magnitudes spread over a binade, in the norm, the three weights and the gated product: five independent
contributions, below sqrt(5) * 2^-5, on the block's added part, which is less than the whole."""
import importlib.util
import os

import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mlp_block.py")
_spec = importlib.util.spec_from_file_location("mlp_block", _path)
mlp = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(mlp)


@pytest.mark.parametrize("tokens,hidden,inner", [(1, 256, 704), (70, 512, 1408), (300, 320, 1000), (520, 1024, 2816)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_block(tokens, hidden, inner, dtype):
    w = mlp.weights(hidden, inner, dtype, seed=tokens)
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x, r = torch.randn((2, tokens, hidden), generator=gen, device="cuda").to(dtype)
    ref = mlp.block64(x, r, w)
    got, h = mlp.block(x, r, w)
    assert torch.equal(h, (x.float() + r.float()).to(dtype))
    assert float((got.double() - ref).norm() / ref.norm()) < 4 * 2.0 ** -9
    got, h8 = mlp.block_mx(x, r, mlp.quantised(w))
    assert torch.equal(h8, h)
    assert float((got.double() - ref).norm() / ref.norm()) < 5 ** 0.5 * 2.0 ** -5
    assert bg.bigemm_last_device_error() == 0
