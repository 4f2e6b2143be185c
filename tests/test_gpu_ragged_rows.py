"""16-bit outputs whose rows start on the 16-byte grid and end inside a 16-byte word: what lies behind a row's last element
in that word is the caller's, and stays (a TMA store is not exact to the element there)."""
import pytest

from tests import test_gpu_gated as gated
from tests import test_gpu_layernorm as norms

pytestmark = pytest.mark.gpu

WIDTHS = [1, 2, 3, 7, 9, 15, 23, 28, 31, 33, 39, 63, 65, 70, 71, 100, 127, 129, 199, 255, 257, 263, 300, 1001, 1007]


def to_grid(cols):
    """Columns behind the last that bring the next row to the 16-byte grid."""
    return -cols % 8 or 8


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("M", [3, 40, 300, 900])
def test_gated(cols, M):
    gated.gated_case(M, cols, 72, "bf16", bias=True, pad=to_grid(cols), seed=cols)


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("M,N", [(2, 40), (130, 72), (600, 520), (5, 3000)])
def test_gradients_of_a_product(cols, M, N):
    gated.linear_case(M, N, cols, "f16", pad=to_grid(cols), seed=cols)


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("M,N", [(2, 40), (130, 72), (600, 520), (5, 3000)])
def test_gradients_of_a_gated_layer(cols, M, N):
    gated.back_case(M, N, cols, "bf16", pad=to_grid(cols), seed=cols)


@pytest.mark.parametrize("cols", WIDTHS + [2047, 8199, 9001])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_norms(cols, kind):
    norms.norm_case(30, cols, kind, pad=to_grid(cols), seed=cols)
    for which in ("layer", "rms"):
        norms.back_case(which, 30, cols, kind, pad=to_grid(cols), seed=cols)
