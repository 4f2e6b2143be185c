"""Outputs of the layer norm and of the norms' gradients that are an input or another output: refused before any device
work, but for rows that take the place of rows of the same matrix."""
import pytest

from tests.test_train_host import BF16, F16, F32, INVALID, MX, layer_back, layernorm, lib, rms_back  # noqa: F401

# each argument a buffer of its own
APART = dict(d=4096, x=8192, mean=12288, rstd=16384, w=20480, s=24576, lds=8, dx=28672, dw=32768, db=36864, space=40960)
FORWARD = dict(x=4096, r=8192, ldr=8, g=12288, b=16384, h=20480, ldh=8, out=24576, mean=28672, rstd=32768)


@pytest.mark.parametrize("out", ["dw", "db"])
@pytest.mark.parametrize("same", ["d", "x", "mean", "rstd", "w", "s", "dx", "dw", "db"])
def test_sums_are_buffers_of_their_own(lib, out, same):
    if out == same:
        return
    assert layer_back(lib, **{**APART, out: APART[same]}) == INVALID
    if {out, same}.isdisjoint({"db", "mean", "rstd"}):
        rms = {k: v for k, v in APART.items() if k not in ("mean", "rstd", "db")}
        assert rms_back(lib, **{**rms, out: rms[same]}) == INVALID


@pytest.mark.parametrize("same", ["mean", "rstd", "w"])
def test_dx_is_no_vector(lib, same):
    assert layer_back(lib, **{**APART, "dt": F32, "dx": APART[same]}) == INVALID


@pytest.mark.parametrize("same,ld", [("d", "ldd"), ("x", "ldx"), ("s", "lds")])
def test_dx_in_place_has_the_same_rows(lib, same, ld):
    for call in (layer_back, rms_back):
        args = {**APART, "dx": APART[same], ld: 16}
        if call is rms_back:
            args = {k: v for k, v in args.items() if k not in ("mean", "rstd", "db")}
        assert call(lib, **args) == INVALID
        assert call(lib, **{**args, ld: 8, "ldo": 16}) == INVALID


@pytest.mark.parametrize("out", ["h", "out"])
@pytest.mark.parametrize("same,ld", [("x", "ldx"), ("r", "ldr")])
def test_the_forward_pass_in_place_has_the_same_rows(lib, out, same, ld):
    assert layernorm(lib, **{**FORWARD, out: FORWARD[same], ld: 16}) == INVALID


@pytest.mark.parametrize("dt,out_dt,scale", [(F16, F32, None), (BF16, F32, None), (F16, MX, 65536), (F32, MX, 65536)])
@pytest.mark.parametrize("same", ["x", "r"])
def test_out_of_another_type_is_not_in_place(lib, dt, out_dt, scale, same):
    assert layernorm(lib, **{**FORWARD, "dt": dt, "out_dt": out_dt, "s": scale, "out": FORWARD[same]}) == INVALID


@pytest.mark.parametrize("out", ["mean", "rstd", "out", "h"])
@pytest.mark.parametrize("same", ["x", "r", "g", "b", "mean", "rstd", "out", "h"])
def test_forward_outputs_are_buffers_of_their_own(lib, out, same):
    if out == same or (out in ("out", "h") and same in ("x", "r")):
        return
    assert layernorm(lib, **{**FORWARD, "dt": F32, "out_dt": F32, out: FORWARD[same]}) == INVALID
    if out == "out":
        assert layernorm(lib, **{**FORWARD, "dt": F32, "out_dt": MX, "s": FORWARD[same]}) == INVALID
