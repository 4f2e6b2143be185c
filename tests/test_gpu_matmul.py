"""GPU parity of the matrix products against their 64-bit definition: types, ragged sizes, strides, every activation
and combination, one token to several tiles, sums shared among CTAs, MXFP8 in and out."""
import numpy as np
import pytest
import torch

import broadcast_implicit_gemm_gb300 as bg
from tests import layer_ref as lr

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "mx": torch.float8_e4m3fn}


def rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g) * scale


def strided(t, pad, dtype):
    """The matrix as columns of a wider CUDA tensor (pad more elements per row)."""
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan")).to(dtype).cuda()
    big[:, : t.shape[1]] = t.to(dtype).cuda()
    return big[:, : t.shape[1]]


def f64(t):
    return t.cpu().double().numpy()


def run_case(M, N, K, kind="bf16", out="bf16", act="none", combine="none", bias=True, padx=0, padw=0, pado=0, other_kind=None,
             seed=1):
    x = strided(rand((M, K), seed), padx, TD[kind])
    w = strided(rand((N, K), seed + 1, K ** -0.5), padw, TD[kind])
    b = rand((N,), seed + 2).cuda() if bias else None
    o = strided(rand((M, N), seed + 3), pado, TD[other_kind or out]) if combine != "none" else None
    y = strided(torch.zeros((M, N)), pado, TD[out])
    y.fill_(float("nan"))
    r = bg.matmul(x, w, b, act=bg.ACT_NAMES[act], other=o, combine=bg.COMBINE_NAMES[combine], out=y)
    torch.cuda.synchronize()
    assert r is y and bg.bigemm_last_device_error() == 0
    ref, d = lr.product64(f64(x), f64(w), f64(b) if bias else None, act, f64(o) if o is not None else None, combine,
                          TD[out], False)
    lr.check_float(y, ref, d, f"{M}x{N}x{K} {kind}->{out} {act} {combine}")
    if pado:
        assert torch.isnan(y._base[:, N:]).all(), "written past the row"


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300])
@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f32")])
def test_token_counts(M, kind, out):
    run_case(M, 200, 320, kind, out, "gelu_tanh", "add", seed=M)


@pytest.mark.parametrize("N", [1, 7, 8, 31, 32, 127, 128, 129, 255, 384, 1000])
@pytest.mark.parametrize("M", [3, 150])
def test_channel_counts(M, N):
    run_case(M, N, 136, "f16", "f16", "silu", "mul", seed=N)


@pytest.mark.parametrize("K", [1, 2, 7, 8, 63, 64, 65, 128, 1000, 1024, 1025, 2048, 4097, 16384])
@pytest.mark.parametrize("M,kind,out", [(5, "bf16", "bf16"), (70, "f16", "f32"), (140, "f16", "f16")])
def test_lengths(M, K, kind, out):
    run_case(M, 160, K, kind, out, "none", "none", seed=K)


@pytest.mark.parametrize("act", list(bg.ACT_NAMES))
@pytest.mark.parametrize("combine", list(bg.COMBINE_NAMES))
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M", [4, 200])
def test_epilogues(act, combine, bias, M):
    run_case(M, 264, 192, "bf16", "bf16", act, combine, bias)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("other", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M", [9, 180])
def test_types(kind, out, other, M):
    run_case(M, 136, 200, kind, out, "relu", "add", other_kind=other)


@pytest.mark.parametrize("padx,padw,pado", [(8, 0, 0), (0, 8, 8), (1, 0, 0), (0, 1, 3), (4, 4, 1), (24, 40, 16)])
@pytest.mark.parametrize("M", [1, 33, 270])
def test_strides(M, padx, padw, pado):
    run_case(M, 130, 264, "bf16", "bf16", "gelu", "add", padx=padx, padw=padw, pado=pado)
    run_case(M, 130, 264, "f16", "f32", "none", "mul", padx=padx, padw=padw, pado=pado)


@pytest.mark.parametrize("M", [1, 40, 260])
def test_misaligned_bases(M):
    N, K = 96, 160
    wide = torch.randn(M * K + N * K + M * N + 3, device="cuda").to(torch.float16)
    x, w = wide[1: 1 + M * K].view(M, K), wide[1 + M * K: 1 + M * K + N * K].view(N, K) / K ** 0.5
    buf = torch.zeros(N * K + 1, dtype=torch.float16, device="cuda")
    w = buf[1:].view(N, K).copy_(w)
    y = torch.zeros(M * N + 1, dtype=torch.float16, device="cuda")[1:].view(M, N)
    bg.matmul(x, w, out=y)
    ref, d = lr.product64(f64(x), f64(w), None, "none", None, "none", torch.float16, False)
    lr.check_float(y, ref, d, "misaligned")


def test_many_channels_few_tokens_and_many_tokens_few_channels():
    run_case(2, 20000, 512, "bf16", "bf16", "none", "none", False)
    run_case(5000, 40, 96, "f16", "f16", "silu", "none", True)


@pytest.mark.parametrize("out", ["f16", "f32"])
def test_a_million_tokens(out):
    """More tiles of few tokens than a grid's second axis has places."""
    run_case(1_100_003, 8, 16, "f16", out, "relu", "add", True)


@pytest.mark.parametrize("M,N,K", [(300, 700, 520), (513, 1030, 264), (1024, 512, 1024), (777, 260, 4096)])
@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f32")])
def test_prompts(M, N, K, kind, out):
    run_case(M, N, K, kind, out, "gelu_tanh", "mul", seed=7)


def test_other_is_the_output():
    M, N, K = 70, 256, 128
    x, w = rand((M, K), 1).half().cuda(), rand((N, K), 2, K ** -0.5).half().cuda()
    y = rand((M, N), 3).half().cuda()
    o = f64(y)
    bg.matmul(x, w, other=y, out=y)
    ref, d = lr.product64(f64(x), f64(w), None, "none", o, "add", torch.float16, False)
    lr.check_float(y, ref, d, "in place")


def test_same_bits_every_time():
    x, w = rand((20, 4096), 1).bfloat16().cuda(), rand((512, 4096), 2, 1 / 64).bfloat16().cuda()
    first = bg.matmul(x, w, out_dtype=torch.float32)
    for _ in range(20):
        assert torch.equal(bg.matmul(x, w, out_dtype=torch.float32), first)


def test_another_stream_and_a_graph():
    x, w = rand((24, 512), 1).half().cuda(), rand((640, 512), 2, 0.05).half().cuda()
    want = bg.matmul(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = bg.matmul(x, w)
    named = torch.empty_like(want)
    bg.matmul(x, w, out=named, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(named, want)
    g, out = torch.cuda.CUDAGraph(), torch.zeros_like(want)
    with torch.cuda.graph(g):
        bg.matmul(x, w, out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_overlapping_streams():
    """Calls on two streams at once: no state is shared."""
    ss = [torch.cuda.Stream() for _ in range(3)]
    xs = [rand((16 + 30 * i, 2048), i).bfloat16().cuda() for i in range(3)]
    w = rand((4096, 2048), 9, 0.02).bfloat16().cuda()
    want = [bg.matmul(x, w) for x in xs]
    torch.cuda.synchronize()
    outs = [torch.empty_like(t) for t in want]
    for _ in range(10):
        for s, x, o in zip(ss, xs, outs):
            bg.matmul(x, w, out=o, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    assert bg.bigemm_last_device_error() == 0


def test_infinities_and_nans_stay_in_their_rows():
    M, N, K = 40, 200, 256
    x, w = rand((M, K), 1).half().cuda(), rand((N, K), 2, 0.05).half().cuda()
    clean = bg.matmul(x, w)
    x[3, 5], x[7, 9] = float("nan"), float("inf")
    got = bg.matmul(x, w)
    keep = [m for m in range(M) if m not in (3, 7)]
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[7]).any()
    assert torch.equal(got[keep], clean[keep])


def test_activations_far_out():
    """Large arguments: no NaN from an overflowing exponential, the limits are reached."""
    z = torch.tensor([-3e4, -1e3, -100, -88, -30, 0.0, 30, 88, 100, 1e3, 3e4])
    x, w = z[:, None].half().cuda(), torch.ones(1, 1).half().cuda()
    for act in ("gelu", "gelu_tanh", "silu"):
        y = bg.matmul(x, w, act=bg.ACT_NAMES[act], out_dtype=torch.float32)[:, 0].cpu().double().numpy()
        ref = lr.act64(act, f64(x)[:, 0])
        assert np.isfinite(y).all()
        assert np.all(np.abs(y - ref) <= 2.0 ** -19 * np.maximum(np.abs(ref), 1)), act


# --------------------------------------------------------------------- MXFP8

def mx_case(M, N, K, out="bf16", act="none", combine="none", bias=True, seed=1, loud=False):
    xf, wf = rand((M, K), seed).cuda(), rand((N, K), seed + 1, K ** -0.5).cuda()
    if loud:   # scales over a wide range
        xf *= torch.exp2(torch.randint(-12, 12, (M, 1), generator=torch.Generator().manual_seed(5))).cuda()
        wf *= torch.exp2(torch.randint(-8, 8, (1, -(-K // 32)), generator=torch.Generator().manual_seed(6))).cuda().repeat_interleave(32, 1)[:, :K]
    x, xs = bg.mx_quantize(xf)
    w, ws = bg.mx_quantize(wf)
    b = rand((N,), seed + 2).cuda() if bias else None
    side = torch.bfloat16 if out == "mx" else TD[out]
    o = rand((M, N), seed + 3).to(side).cuda() if combine != "none" else None
    got = bg.matmul_mx(x, xs, w, ws, b, act=bg.ACT_NAMES[act], other=o, combine=bg.COMBINE_NAMES[combine], out_dtype=TD[out])
    torch.cuda.synchronize()
    assert bg.bigemm_last_device_error() == 0
    ref, d = lr.product64(lr.decode(x, xs), lr.decode(w, ws), f64(b) if bias else None, act,
                          f64(o) if o is not None else None, combine, TD[out], True)
    what = f"mx {M}x{N}x{K} {out} {act} {combine}"
    if out == "mx":
        lr.check_mx(got[0], got[1], ref, d, what)
        assert lr.padding_codes_are_zero(got[1], M, N)
    else:
        lr.check_float(got, ref, d, what)


@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 64, 65, 100, 128, 129, 190, 256, 300])
@pytest.mark.parametrize("out", ["bf16", "mx"])
def test_mx_token_counts(M, out):
    mx_case(M, 200, 320, out, "gelu", "add", seed=M)


@pytest.mark.parametrize("N", [1, 31, 33, 128, 130, 1000])
@pytest.mark.parametrize("M,out", [(3, "mx"), (150, "f16"), (270, "mx")])
def test_mx_channel_counts(M, N, out):
    mx_case(M, N, 256, out, "silu", "mul", seed=N)


@pytest.mark.parametrize("K", [1, 16, 31, 32, 33, 127, 128, 130, 1024, 2056, 4112, 16384])
@pytest.mark.parametrize("M,out", [(5, "bf16"), (70, "f32"), (260, "f32")])
def test_mx_lengths(M, K, out):
    mx_case(M, 160, K, out, seed=K)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16", "mx"])
@pytest.mark.parametrize("M", [8, 200])
def test_mx_wide_scales(M, out):
    """Scales that differ from group to group and row to row: each has to meet its own elements."""
    if out == "f16":
        mx_case(M, 384, 640, "f16", seed=3)
    else:
        mx_case(M, 384, 640, out, seed=3, loud=True)


def test_mx_nan_scale_reaches_its_row_alone():
    M, N, K = 140, 130, 256
    x, xs = bg.mx_quantize(rand((M, K), 1).cuda())
    w, ws = bg.mx_quantize(rand((N, K), 2, 0.1).cuda())
    clean = bg.matmul_mx(x, xs, w, ws)
    xs.view(torch.uint8)[1, 0, 2, 0, 1] = 255      # row 130, group 1
    got = bg.matmul_mx(x, xs, w, ws)
    keep = [m for m in range(M) if m != 130]
    assert torch.isnan(got[130]).all() and torch.equal(got[keep], clean[keep])


# --------------------------------------------------------------------- refusals of the tensor calls

def test_tensor_refusals():
    x, w = torch.zeros(4, 32).half().cuda(), torch.zeros(8, 32).half().cuda()
    q, s = bg.mx_quantize(x)
    p, t = bg.mx_quantize(w)
    b = torch.zeros(8, device="cuda")
    for bad, call in (
            (ValueError, lambda: bg.matmul(x[0], w)),
            (ValueError, lambda: bg.matmul(x, w[:, :16])),
            (ValueError, lambda: bg.matmul(x.t(), w)),
            (ValueError, lambda: bg.matmul(x.expand(4, 32)[:, ::2], w[:, :16].contiguous())),
            (ValueError, lambda: bg.matmul(x, w.cpu())),
            (ValueError, lambda: bg.matmul(x, w, bias=b[:7])),
            (ValueError, lambda: bg.matmul(x, w, bias=b.double())),
            (ValueError, lambda: bg.matmul(x, w, bias=torch.zeros(16, device="cuda")[::2])),
            (ValueError, lambda: bg.matmul(x, w, combine=bg.COMBINE_ADD)),
            (ValueError, lambda: bg.matmul(x, w, other=torch.zeros(8, 4).half().cuda())),
            (ValueError, lambda: bg.matmul(x, w, out=torch.zeros(4, 9).half().cuda())),
            (TypeError, lambda: bg.matmul(x, w.bfloat16())),
            (TypeError, lambda: bg.matmul(x, w, out=torch.zeros(4, 8).half().cuda(), out_dtype=torch.float32)),
            (TypeError, lambda: bg.matmul(x, w, out=torch.zeros(4, 8, dtype=torch.int32, device="cuda"))),
            (TypeError, lambda: bg.matmul(q, p)),
            (TypeError, lambda: bg.matmul_mx(x, s, w, t)),
            (ValueError, lambda: bg.matmul_mx(q, s.reshape(-1)[:256], p, t)),
            (ValueError, lambda: bg.matmul_mx(q, s, p, None)),
            (ValueError, lambda: bg.matmul_mx(q, s.view(torch.uint8).float(), p, t)),
            (ValueError, lambda: bg.rmsnorm(x, weight=torch.ones(31, device="cuda"))),
            (ValueError, lambda: bg.rmsnorm(x, residual=x[:3])),
            (TypeError, lambda: bg.rmsnorm(x, residual=x.bfloat16())),
            (ValueError, lambda: bg.mx_quantize(x, scale=s.view(torch.uint8).reshape(-1)[1:])),
            (TypeError, lambda: bg.mx_quantize(x, out=torch.zeros(4, 32).half().cuda())),
    ):
        with pytest.raises(bad):
            call()
    with pytest.raises(bg.BigemmError):
        bg.matmul(x.float(), w.float())
    with pytest.raises(bg.BigemmError):
        bg.rmsnorm(q)
    with pytest.raises(bg.BigemmError):
        bg.rmsnorm(x, out_dtype=torch.bfloat16)
    assert bg.matmul(x[:0], w).shape == (0, 8)
    assert bg.matmul_mx(q[:0], s[:0], p, t).shape == (0, 8)
    assert bg.bigemm_last_device_error() == 0


# --------------------------------------------------------------------- far offsets

def test_offsets_past_32_bits():
    """Rows so far apart that element offsets pass 2^32: first, middle and last rows land where they should."""
    rows, cols, apart = 5, 64, (1 << 30) + 8
    base = torch.empty(4 * apart + cols, dtype=torch.float16, device="cuda")
    x = base.as_strided((rows, cols), (apart, 1))
    x.copy_(rand((rows, cols), 1).half())
    w = rand((72, cols), 2, 0.125).half().cuda()
    ref, d = lr.product64(f64(x), f64(w), None, "none", None, "none", torch.float16, False)
    lr.check_float(bg.matmul(x, w), ref, d, "far x")
    q, s = bg.mx_quantize(x)
    p, t = bg.mx_quantize(x.contiguous())
    assert torch.equal(q.view(torch.uint8), p.view(torch.uint8)) and torch.equal(s.view(torch.uint8), t.view(torch.uint8))
    assert torch.equal(bg.rmsnorm(x), bg.rmsnorm(x.contiguous()))
    y = base.as_strided((rows, 72), (apart - 8, 1))
    want = bg.matmul(x, w)
    x = x.contiguous()
    bg.matmul(x, w, out=y)
    assert torch.equal(y, want)
