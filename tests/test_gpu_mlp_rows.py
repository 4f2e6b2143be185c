"""The gated MLP block row by row: every token's output against 64 bits, so that a few wrong tokens do not hide among the
others.  The bounds are those of test_gpu_mlp_block, which hold for each row (its elements' roundings are independent, 256
of them or more)."""
import importlib.util
import os

import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mlp_block.py")
_spec = importlib.util.spec_from_file_location("mlp_block_rows", _path)
mlp = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(mlp)


@pytest.mark.parametrize("tokens,hidden,inner", [(1, 256, 704), (70, 512, 1408), (300, 320, 1000), (2100, 2600, 4104), (9000, 520, 1041)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_row(tokens, hidden, inner, dtype):
    w = mlp.weights(hidden, inner, dtype, seed=tokens)
    x, r = torch.randn((2, tokens, hidden), generator=torch.Generator("cuda").manual_seed(tokens), device="cuda").to(dtype)
    ref = mlp.block64(x, r, w)
    for got, most in ((mlp.block(x, r, w)[0], 4 * 2.0 ** -9), (mlp.block_mx(x, r, mlp.quantised(w))[0], 5 ** 0.5 * 2.0 ** -5)):
        off = (got.double() - ref).norm(dim=1) / ref.norm(dim=1)
        assert float(off.max()) < most, f"row {int(off.argmax())}: {float(off.max()):.2e}"
    assert bg.bigemm_last_device_error() == 0
