"""The transformer-layer operators as they are measured: the matrix product with bias, activation and a residual or a
gate in its epilogue, the same product over MXFP8 operands, the root-mean-square norm with the residual's addition, and
the quantisation to MXFP8.

MXFP8: e4m3 elements with one power-of-two scale (E8M0) per 32 elements of a row.  Scales are kept in blocks of 128 rows
by 128 columns: scale[row // 128, col // 128, row % 32, (row // 32) % 4, (col // 32) % 4].
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "mx": torch.float8_e4m3fn}
BYTES = {"f16": 2, "bf16": 2, "f32": 4, "mx": 1 + 1 / 32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
MAX_FLOPS = 2 * 8192 * 16384 * 4096      # of the largest listed product
MAX_ELEMS = 8192 * 8192                  # of the largest listed norm


def listed():
    return [
        # one token through a layer's output projection, added to the residual stream
        {"name": "linear_token", "op": "matmul", "m": 1, "n": 4096, "k": 4096, "in": "bf16", "out": "bf16", "bias": False,
         "act": "none", "other": "add", "pad": 0},
        # a small serving batch of single tokens through an MLP's first product
        {"name": "linear_batch", "op": "matmul", "m": 27, "n": 16384, "k": 4096, "in": "f16", "out": "f16", "bias": True,
         "act": "gelu", "other": "none", "pad": 0},
        # a chunk of prompts, every size ragged, rows of a wider tensor, the gate of a gated MLP
        {"name": "linear_ragged", "op": "matmul", "m": 777, "n": 5001, "k": 1000, "in": "bf16", "out": "bf16", "bias": True,
         "act": "silu", "other": "mul", "pad": 24},
        # an MLP's second product with the residual kept in 32 bits
        {"name": "linear_down", "op": "matmul", "m": 2048, "n": 2048, "k": 8192, "in": "f16", "out": "f32", "bias": False,
         "act": "none", "other": "add", "pad": 0},
        # long prompts through an MLP's first product
        {"name": "linear_prompt", "op": "matmul", "m": 8192, "n": 16384, "k": 4096, "in": "bf16", "out": "bf16", "bias": True,
         "act": "gelu_tanh", "other": "none", "pad": 0},
        # a serving batch through an MLP's second product in 8 bits
        {"name": "mx_batch", "op": "matmul_mx", "m": 8, "n": 4096, "k": 16384, "out": "bf16", "bias": False, "act": "none",
         "other": "add"},
        # long prompts through an MLP's first product in 8 bits, its output quantised for the second
        {"name": "mx_prompt", "op": "matmul_mx", "m": 4096, "n": 8192, "k": 8192, "out": "mx", "bias": True, "act": "gelu",
         "other": "none"},
        # one token's norm, quantised for the product that follows
        {"name": "norm_token", "op": "rmsnorm", "m": 1, "k": 4096, "in": "bf16", "out": "mx", "residual": True, "pad": 0},
        # a chunk of prompts of an odd width
        {"name": "norm_ragged", "op": "rmsnorm", "m": 1537, "k": 2049, "in": "bf16", "out": "mx", "residual": False, "pad": 0},
        # long prompts, the norm in 16 bits
        {"name": "norm_prompt", "op": "rmsnorm", "m": 8192, "k": 8192, "in": "f16", "out": "f16", "residual": True, "pad": 0},
        # a chunk of activations of a width that ends inside a scale's block
        {"name": "quantize_ragged", "op": "quantize", "m": 300, "k": 2056, "in": "f16", "pad": 8},
        # a layer's weights
        {"name": "quantize_weights", "op": "quantize", "m": 16384, "k": 4096, "in": "bf16", "pad": 0},
    ]


def _size(rng, low, high):
    """A size spread over the logarithm: as it falls, or a multiple of 8 or of 128."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    to = rng.choice((1, 8, 128))
    return min(high, max(low, -(-n // to) * to)) if n >= to else n


def draw(rng):
    op = rng.choice(("matmul", "matmul", "matmul_mx", "rmsnorm", "quantize"))
    if op in ("matmul", "matmul_mx"):
        while True:
            m, n, k = _size(rng, 1, 8192), _size(rng, 64, 16384), _size(rng, 64, 16384)
            if 2 * m * n * k <= MAX_FLOPS:
                break
        case = {"op": op, "m": m, "n": n, "k": k, "bias": rng.random() < 0.5, "act": rng.choice(ACTS),
                "other": rng.choice(("none", "add", "mul"))}
        if op == "matmul":
            kind = rng.choice(("f16", "bf16"))
            return {**case, "in": kind, "out": rng.choice((kind, kind, "f32")), "pad": rng.choice((0, 0, 8, 24))}
        return {**case, "out": rng.choice(("f16", "bf16", "mx"))}
    while True:
        m, k = _size(rng, 1, 16384), _size(rng, 64, 16384)
        if m * k <= MAX_ELEMS:
            break
    case = {"op": op, "m": m, "k": k, "in": rng.choice(("f16", "bf16")), "pad": rng.choice((0, 0, 8, 24))}
    if op == "quantize":
        return case
    return {**case, "out": rng.choice((case["in"], "mx")), "residual": rng.random() < 0.7}


# ---------------------------------------------------------------- MXFP8 in elementary operations

def _blocks(rows, cols):
    return -(-rows // 128), -(-cols // 128)


def _scale_zeros(rows, cols):
    a, b = _blocks(rows, cols)
    return torch.zeros((a, b, 32, 4, 4), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)


def _quantize(y):
    """(e4m3 elements, blocked scales) of a 32-bit matrix: the smallest power of two s with amax <= 448 s."""
    rows, cols = y.shape
    a, b = _blocks(rows, cols)
    full = torch.zeros((a * 128, b * 128), dtype=torch.float32, device=y.device)
    full[:rows, :cols] = y
    groups = full.view(a * 128, b * 4, 32)
    bits = groups.abs().amax(-1).view(torch.int32)
    code = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)     # biased exponent of s: 448 = 1.75 * 2^8
    code = code.clamp(0, 254)
    q = torch.ldexp(groups, (127 - code)[..., None]).to(torch.float8_e4m3fn)
    q = q.view(a * 128, b * 128)[:rows, :cols].contiguous()
    code[rows:] = 0
    scale = code.to(torch.uint8).view(a, 4, 32, b, 4).permute(0, 3, 2, 1, 4).contiguous()
    return q, scale.view(torch.float8_e8m0fnu)


def _dequantize(q, scale):
    rows, cols = q.shape
    a, b = scale.shape[:2]
    code = scale.view(torch.uint8).permute(0, 3, 2, 1, 4).reshape(a * 128, b * 4)[:rows].to(torch.int32)
    code = code.repeat_interleave(32, dim=1)[:, :cols]
    return torch.ldexp(q.float(), code - 127)


# ---------------------------------------------------------------- inputs

def _activations(rows, cols, dtype, pad, gen):
    """Activations of a transformer: normal, with a few channels of much larger size; rows of a wider tensor if pad."""
    x = torch.randn((rows, cols + pad), generator=gen, device="cuda")
    loud = torch.rand((cols + pad,), generator=gen, device="cuda") < 0.005
    return (x * (1 + 15 * loud)).to(dtype)[:, :cols]


def _weights(rows, cols, gen):
    return torch.randn((rows, cols), generator=gen, device="cuda") / math.sqrt(cols)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    state = dict(case)
    if op in ("matmul", "matmul_mx"):
        n = case["n"]
        if op == "matmul":
            kind = DTYPES[case["in"]]
            state["x"] = _activations(m, k, kind, case["pad"], gen)
            state["w"] = _weights(n, k, gen).to(kind)
            side = DTYPES[case["out"]]
        else:
            state["x"], state["x_scale"] = _quantize(_activations(m, k, torch.float32, 0, gen))
            state["w"], state["w_scale"] = _quantize(_weights(n, k, gen))
            side = torch.bfloat16 if case["out"] == "mx" else DTYPES[case["out"]]
        state["b"] = torch.randn((n,), generator=gen, device="cuda") * 0.1 if case["bias"] else None
        state["o"] = torch.randn((m, n), generator=gen, device="cuda").to(side) if case["other"] != "none" else None
        state["out_dtype"] = DTYPES[case["out"]]
        state["y"] = torch.empty((m, n), dtype=state["out_dtype"], device="cuda")
        state["y_scale"] = _scale_zeros(m, n) if case["out"] == "mx" else None
        return state
    kind = DTYPES[case["in"]]
    state["x"] = _activations(m, k, kind, case["pad"], gen)
    if op == "rmsnorm":
        state["g"] = 1 + 0.1 * torch.randn((k,), generator=gen, device="cuda")
        state["r"] = _activations(m, k, kind, case["pad"], gen) if case["residual"] else None
        state["h"] = torch.empty((m, k), dtype=kind, device="cuda") if case["residual"] else None
        state["out_dtype"] = DTYPES[case["out"]]
    else:
        state["out_dtype"] = torch.float8_e4m3fn
    state["y"] = torch.empty((m, k), dtype=state["out_dtype"], device="cuda")
    state["y_scale"] = _scale_zeros(m, k) if state["out_dtype"] == torch.float8_e4m3fn else None
    return state


EPS = 1e-6


# ---------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _act(kind, z):
    if kind == "relu":
        return torch.maximum(z, torch.zeros((), device=z.device, dtype=z.dtype))
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _run_plain(state):
    op = state["op"]
    if op == "quantize":
        q, scale = _quantize(state["x"].float())
        return {"q": q, "scale": scale}
    if op == "rmsnorm":
        h = state["x"].float()
        if state["r"] is not None:
            h = h + state["r"].float()
        y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * state["g"]
        out = {"h": h.to(state["x"].dtype)} if state["r"] is not None else {}
        if state["out"] == "mx":
            out["q"], out["scale"] = _quantize(y)
        else:
            out["y"] = y.to(state["out_dtype"])
        return out
    if op == "matmul":
        z = state["x"].float() @ state["w"].float().t()
    else:
        z = _dequantize(state["x"], state["x_scale"]) @ _dequantize(state["w"], state["w_scale"]).t()
    if state["b"] is not None:
        z = z + state["b"]
    z = _act(state["act"], z)
    if state["other"] == "add":
        z = z + state["o"].float()
    elif state["other"] == "mul":
        z = z * state["o"].float()
    if state["out"] == "mx":
        q, scale = _quantize(z)
        return {"q": q, "scale": scale}
    return {"y": z.to(state["out_dtype"])}


def _run_own(state):
    import broadcast_implicit_gemm_gb300 as bg
    op = state["op"]
    if op == "quantize":
        q, scale = bg.mx_quantize(state["x"], out=state["y"], scale=state["y_scale"])
        return {"q": q, "scale": scale}
    if op == "rmsnorm":
        got = bg.rmsnorm(state["x"], state["g"], residual=state["r"], eps=EPS, out_dtype=state["out_dtype"],
                         out=state["y"], out_scale=state["y_scale"], sum_out=state["h"])
        out = {"h": state["h"]} if state["r"] is not None else {}
        if state["out"] == "mx":
            out["q"], out["scale"] = got[0], got[1]
        else:
            out["y"] = got if state["r"] is None else got[0]
        return out
    kw = {"bias": state["b"], "act": bg.ACT_NAMES[state["act"]], "other": state["o"],
          "combine": bg.COMBINE_NAMES[state["other"]], "out_dtype": state["out_dtype"], "out": state["y"]}
    if op == "matmul":
        return {"y": bg.matmul(state["x"], state["w"], **kw)}
    got = bg.matmul_mx(state["x"], state["x_scale"], state["w"], state["w_scale"], out_scale=state["y_scale"], **kw)
    return {"q": got[0], "scale": got[1]} if state["out"] == "mx" else {"y": got}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    if op == "quantize":
        return {"bytes": m * k * (BYTES[case["in"]] + BYTES["mx"]), "flops": 3 * m * k}
    if op == "rmsnorm":
        each = BYTES[case["in"]] * (3 if case["residual"] else 1) + BYTES[case["out"]]
        return {"bytes": m * k * each + 4 * k, "flops": 5 * m * k}
    n = case["n"]
    side = "bf16" if case["out"] == "mx" else case["out"]
    moved = (m * k + n * k) * BYTES[case["in"] if op == "matmul" else "mx"] + m * n * BYTES[case["out"]]
    moved += 4 * n if case["bias"] else 0
    moved += m * n * BYTES[side] if case["other"] != "none" else 0
    return {"bytes": moved, "flops": 2 * m * n * k}


# ---------------------------------------------------------------- the definition in 64 bits

def _decoded64(q, scale):
    """Each element times 2^(code - 127), the code looked up at the element's own place in the blocked scales."""
    rows, cols = q.shape
    row, col = torch.arange(rows, device=q.device)[:, None], torch.arange(0, cols, 32, device=q.device)[None, :]
    code = scale.view(torch.uint8)[row // 128, col // 128, row % 32, (row // 32) % 4, (col // 32) % 4]
    factor = torch.pow(2.0, code.double() - 127)
    return q.double() * factor.repeat_interleave(32, dim=1)[:, :cols]


def _encoded64(y):
    """MXFP8 of a 64-bit matrix: s = 2^ceil(log2(amax / 448)), q = y / s rounded to e4m3."""
    rows, cols = y.shape
    a, b = _blocks(rows, cols)
    fill = torch.zeros((rows, b * 128), dtype=torch.float64, device=y.device)
    fill[:, :cols] = y
    most = fill.view(rows, b * 4, 32).abs().amax(-1)
    mantissa, exponent = torch.frexp(most / 448)
    exponent = torch.where(mantissa == 0.5, exponent - 1, exponent).clamp(-127, 127)
    exponent = torch.where(most > 0, exponent, torch.full_like(exponent, -127))
    q = (fill.view(rows, b * 4, 32) * torch.pow(2.0, -exponent.double())[..., None]).float().to(torch.float8_e4m3fn)
    scale = torch.zeros((a, b, 32, 4, 4), dtype=torch.uint8, device=y.device)
    row, group = torch.arange(rows, device=y.device)[:, None], torch.arange(b * 4, device=y.device)[None, :]
    scale[row // 128, group // 4, row % 32, (row // 32) % 4, group % 4] = (exponent + 127).to(torch.uint8)
    return q.view(rows, b * 128)[:, :cols], scale.view(torch.float8_e8m0fnu)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        q, scale = _encoded64(s["x"].double())
        return {"q": q, "scale": scale}
    if op == "rmsnorm":
        h = s["x"].double() if s["r"] is None else s["x"].double() + s["r"].double()
        norm = torch.sqrt(torch.linalg.vecdot(h, h) / h.shape[1] + EPS)
        y = h / norm[:, None] * s["g"].double()
        out = {} if s["r"] is None else {"h": h}
        if case["out"] == "mx":
            out["q"], out["scale"] = _encoded64(y)
        else:
            out["y"] = y
        return out
    if op == "matmul":
        z = torch.mm(s["x"].double(), s["w"].double().T)
    else:
        z = torch.mm(_decoded64(s["x"], s["x_scale"]), _decoded64(s["w"], s["w_scale"]).T)
    if s["b"] is not None:
        z += s["b"].double()
    if case["act"] == "relu":
        z = z.clamp(min=0)
    elif case["act"] == "gelu":
        z = z * torch.special.ndtr(z)
    elif case["act"] == "gelu_tanh":
        z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    elif case["act"] == "silu":
        z = z * torch.sigmoid(z)
    if case["other"] == "add":
        z = z + s["o"].double()
    elif case["other"] == "mul":
        z = z * s["o"].double()
    if case["out"] == "mx":
        q, scale = _encoded64(z)
        return {"q": q, "scale": scale}
    return {"y": z}
