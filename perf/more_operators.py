"""What training a transformer's feed-forward block takes, and its layer norm, as they are measured: the layer norm with
the residual's addition, the gradients of the layer norm and of the root-mean-square norm with the sums over all rows that
make the weight's gradient, the two products of a gated layer with the activation and the multiplication, its gradients,
and the gradients of a plain product.

Weights are [out features, in features], as in the forward calls.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
ACTS = ("silu", "gelu", "gelu_tanh", "relu", "none")
NORMS = ("layernorm", "layernorm_back", "rmsnorm_back")
MAX_FLOPS = 8 * 4096 * 16384 * 4096      # of the largest listed products
MAX_ELEMS = 8192 * 8192                  # of the largest listed norm
LN_EPS, RMS_EPS = 1e-5, 1e-6


def listed():
    return [
        # one token's norm before a layer, added to the residual stream
        {"name": "ln_token", "op": "layernorm", "m": 1, "k": 4096, "in": "bf16", "residual": True, "affine": True,
         "stats": False, "pad": 0},
        # a long batch in training: the sum and the statistics are kept for the gradient
        {"name": "ln_long", "op": "layernorm", "m": 8192, "k": 8192, "in": "f16", "residual": True, "affine": True,
         "stats": True, "pad": 0},
        # a batch of ragged prompts of an odd width
        {"name": "ln_back_ragged", "op": "layernorm_back", "m": 1537, "k": 2049, "in": "bf16", "residual": False, "affine": True,
         "pad": 0},
        # a long batch in training, with the residual stream's gradient
        {"name": "ln_back_long", "op": "layernorm_back", "m": 8192, "k": 8192, "in": "bf16", "residual": True, "affine": True,
         "pad": 0},
        # a small fine-tuning batch of a small model in 32 bits
        {"name": "rms_back_small", "op": "rmsnorm_back", "m": 64, "k": 1000, "in": "f32", "residual": False, "affine": True,
         "pad": 0},
        # a long batch in training, with the residual stream's gradient
        {"name": "rms_back_long", "op": "rmsnorm_back", "m": 16384, "k": 4096, "in": "f16", "residual": True, "affine": True,
         "pad": 0},
        # one token in serving
        {"name": "gated_token", "op": "gated", "m": 1, "n": 16384, "k": 4096, "in": "bf16", "bias": False, "act": "silu",
         "keep": False, "pad": 0},
        # a long batch in training: both products are kept for the gradient
        {"name": "gated_long", "op": "gated", "m": 8192, "n": 16384, "k": 4096, "in": "bf16", "bias": False, "act": "silu",
         "keep": True, "pad": 0},
        # a ragged batch with an inner width off every grid, with biases
        {"name": "gated_back_ragged", "op": "gated_back", "m": 777, "n": 5001, "k": 1000, "in": "f16", "bias": True,
         "act": "gelu", "pad": 24},
        # a long batch in training
        {"name": "gated_back_long", "op": "gated_back", "m": 4096, "n": 16384, "k": 4096, "in": "bf16", "bias": False,
         "act": "silu", "pad": 0},
        # a fine-tuning batch of few tokens through a square product
        {"name": "linear_back_few", "op": "linear_back", "m": 100, "n": 4096, "k": 4096, "in": "f16", "bias": True, "pad": 0},
        # a long batch through a feed-forward block's second product
        {"name": "linear_back_long", "op": "linear_back", "m": 8192, "n": 4096, "k": 16384, "in": "bf16", "bias": False,
         "pad": 0},
    ]


def _size(rng, low, high):
    """A size spread over the logarithm: as it falls, or a multiple of 8 or of 128."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    to = rng.choice((1, 8, 128))
    return min(high, max(low, -(-n // to) * to)) if n >= to else n


FLOPS = {"gated": 4, "gated_back": 8, "linear_back": 4}


def draw(rng):
    op = rng.choice(NORMS + ("gated", "gated_back", "linear_back"))
    if op in NORMS:
        while True:
            m, k = _size(rng, 1, 16384), _size(rng, 64, 16384)
            if m * k <= MAX_ELEMS:
                break
        case = {"op": op, "m": m, "k": k, "in": rng.choice(("f16", "bf16", "f32")), "residual": rng.random() < 0.6,
                "affine": rng.random() < 0.8, "pad": rng.choice((0, 0, 8, 24, 3))}
        return {**case, "stats": rng.random() < 0.5} if op == "layernorm" else case
    while True:
        m, n, k = _size(rng, 1, 8192), _size(rng, 64, 16384), _size(rng, 64, 16384)
        if FLOPS[op] * m * n * k <= MAX_FLOPS:
            break
    case = {"op": op, "m": m, "n": n, "k": k, "in": rng.choice(("f16", "bf16")), "bias": rng.random() < 0.4,
            "pad": rng.choice((0, 0, 8, 24))}
    if op != "linear_back":
        case["act"] = rng.choice(ACTS)
    return {**case, "keep": rng.random() < 0.5} if op == "gated" else case


# ---------------------------------------------------------------- inputs

def _activations(rows, cols, dtype, pad, gen):
    """Activations of a transformer: normal, off-centre, with a few channels of much larger size; rows of a wider tensor
    if pad."""
    x = torch.randn((rows, cols + pad), generator=gen, device="cuda")
    loud = torch.rand((cols + pad,), generator=gen, device="cuda") < 0.005
    return ((x + 0.1) * (1 + 15 * loud)).to(dtype)[:, :cols]


def _gradients(rows, cols, dtype, pad, gen):
    """Gradients under a loss scale: normal, of small size, tokens of different weight."""
    d = torch.randn((rows, cols + pad), generator=gen, device="cuda")
    return (d * (0.05 * torch.rand((rows, 1), generator=gen, device="cuda") + 0.01)).to(dtype)[:, :cols]


def _weights(rows, cols, dtype, gen):
    return (torch.randn((rows, cols), generator=gen, device="cuda") / math.sqrt(cols)).to(dtype)


def _bias(n, gen):
    return torch.randn((n,), generator=gen, device="cuda") * 0.1


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, m, k, pad = case["op"], case["m"], case["k"], case["pad"]
    kind = DTYPES[case["in"]]
    state = dict(case)
    state["x"] = _activations(m, k, kind, pad, gen)
    if op in NORMS:
        state["w"] = 1 + 0.1 * torch.randn((k,), generator=gen, device="cuda") if case["affine"] else None
        if op == "layernorm":
            state["b"] = _bias(k, gen) if case["affine"] else None
            state["r"] = _activations(m, k, kind, pad, gen) if case["residual"] else None
            state["h"] = torch.empty((m, k), dtype=kind, device="cuda") if case["residual"] else None
            state["y"] = torch.empty((m, k), dtype=kind, device="cuda")
            state["mean"] = torch.empty((m,), device="cuda") if case["stats"] else None
            state["rstd"] = torch.empty((m,), device="cuda") if case["stats"] else None
            return state
        state["d"] = _gradients(m, k, kind, pad, gen)
        state["s"] = _gradients(m, k, kind, pad, gen) if case["residual"] else None
        if op == "layernorm_back":
            # kept by the forward pass
            h = state["x"].double()
            state["mean"] = h.mean(-1).float()
            state["rstd"] = (1 / torch.sqrt(h.var(-1, correction=0) + LN_EPS)).float()
            state["db"] = torch.empty((k,), device="cuda")
        state["dx"] = torch.empty((m, k), dtype=kind, device="cuda")
        state["dw"] = torch.empty((k,), device="cuda")
        return state
    n = case["n"]
    if op == "linear_back":
        state["w"] = _weights(n, k, kind, gen)
        state["d"] = _gradients(m, n, kind, pad, gen)
        state["dx"] = torch.empty((m, k), dtype=kind, device="cuda")
        state["dw"] = torch.empty((n, k), dtype=kind, device="cuda")
        state["db"] = torch.empty((n,), device="cuda") if case["bias"] else None
        return state
    state["wg"], state["wu"] = _weights(n, k, kind, gen), _weights(n, k, kind, gen)
    bg, bu = (_bias(n, gen), _bias(n, gen)) if case["bias"] else (None, None)
    if op == "gated":
        state["bg"], state["bu"] = bg, bu
        for name in ("y", "g", "u"):
            state[name] = torch.empty((m, n), dtype=kind, device="cuda") if name == "y" or case["keep"] else None
        return state
    # kept by the forward pass
    for name, w, b in (("g", state["wg"], bg), ("u", state["wu"], bu)):
        z = state["x"] @ w.t()
        state[name] = z if b is None else (z + b).to(kind)
    state["d"] = _gradients(m, n, kind, pad, gen)
    state["dx"] = torch.empty((m, k), dtype=kind, device="cuda")
    state["dwg"], state["dwu"] = (torch.empty((n, k), dtype=kind, device="cuda") for _ in range(2))
    state["dbg"], state["dbu"] = (torch.empty((n,), device="cuda") if case["bias"] else None for _ in range(2))
    return state


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


def _act_slope(kind, z):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if kind == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _run_plain(state):
    op, kind = state["op"], DTYPES[state["in"]]
    if op == "layernorm":
        h = state["x"].float()
        if state["r"] is not None:
            h = h + state["r"].float()
        mean = h.mean(-1, keepdim=True)
        d = h - mean
        rstd = torch.rsqrt((d * d).mean(-1, keepdim=True) + LN_EPS)
        y = d * rstd
        if state["w"] is not None:
            y = y * state["w"] + state["b"]
        out = {"y": y.to(kind)}
        if state["r"] is not None:
            out["h"] = h.to(kind)
        if state["stats"]:
            out["mean"], out["rstd"] = mean[:, 0], rstd[:, 0]
        return out
    if op in NORMS:
        h, d = state["x"].float(), state["d"].float()
        g = d if state["w"] is None else d * state["w"]
        if op == "layernorm_back":
            rstd = state["rstd"][:, None]
            xh = (h - state["mean"][:, None]) * rstd
            dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
        else:
            rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + RMS_EPS)
            xh = h * rstd
            dx = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
        if state["s"] is not None:
            dx = dx + state["s"].float()
        out = {"dx": dx.to(kind), "dw": (d * xh).sum(0)}
        if op == "layernorm_back":
            out["db"] = d.sum(0)
        return out
    x = state["x"].float()
    if op == "linear_back":
        d = state["d"].float()
        out = {"dx": (d @ state["w"].float()).to(kind), "dw": (d.t() @ x).to(kind)}
        if state["bias"]:
            out["db"] = d.sum(0)
        return out
    wg, wu = state["wg"].float(), state["wu"].float()
    if op == "gated":
        g, u = x @ wg.t(), x @ wu.t()
        if state["bg"] is not None:
            g, u = g + state["bg"], u + state["bu"]
        out = {"y": (_act(state["act"], g) * u).to(kind)}
        if state["keep"]:
            out["g"], out["u"] = g.to(kind), u.to(kind)
        return out
    d, g, u = state["d"].float(), state["g"].float(), state["u"].float()
    dg, du = d * u * _act_slope(state["act"], g), d * _act(state["act"], g)
    out = {"dx": (dg @ wg + du @ wu).to(kind), "dwg": (dg.t() @ x).to(kind), "dwu": (du.t() @ x).to(kind)}
    if state["bias"]:
        out["dbg"], out["dbu"] = dg.sum(0), du.sum(0)
    return out


def _run_own(state):
    import broadcast_implicit_gemm_gb300 as bg
    op = state["op"]
    if op == "layernorm":
        bg.layernorm(state["x"], state["w"], state["b"], residual=state["r"], eps=LN_EPS, out=state["y"], sum_out=state["h"],
                     mean_out=state["mean"], rstd_out=state["rstd"])
        out = {"y": state["y"]}
        if state["r"] is not None:
            out["h"] = state["h"]
        if state["stats"]:
            out["mean"], out["rstd"] = state["mean"], state["rstd"]
        return out
    if op == "layernorm_back":
        dx, dw, db = bg.layernorm_backward(state["d"], state["x"], state["mean"], state["rstd"], state["w"], dsum=state["s"],
                                           dx=state["dx"], dweight=state["dw"], dbias=state["db"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "rmsnorm_back":
        dx, dw = bg.rmsnorm_backward(state["d"], state["x"], state["w"], eps=RMS_EPS, dsum=state["s"], dx=state["dx"],
                                     dweight=state["dw"])
        return {"dx": dx, "dw": dw}
    if op == "linear_back":
        dx, dw = bg.matmul_backward(state["d"], state["x"], state["w"], dx=state["dx"], dw=state["dw"], dbias=state["db"])
        return {"dx": dx, "dw": dw, **({"db": state["db"]} if state["bias"] else {})}
    act = bg.ACT_NAMES[state["act"]]
    if op == "gated":
        y = bg.matmul_gated(state["x"], state["wg"], state["wu"], state["bg"], state["bu"], act=act, out=state["y"],
                            gate_out=state["g"], up_out=state["u"])
        return {"y": y, **({"g": state["g"], "u": state["u"]} if state["keep"] else {})}
    dx, dwg, dwu = bg.matmul_gated_backward(state["d"], state["x"], state["wg"], state["wu"], state["g"], state["u"], act=act,
                                            dx=state["dx"], dw_gate=state["dwg"], dw_up=state["dwu"],
                                            dbias_gate=state["dbg"], dbias_up=state["dbu"])
    out = {"dx": dx, "dwg": dwg, "dwu": dwu}
    if state["bias"]:
        out["dbg"], out["dbu"] = state["dbg"], state["dbu"]
    return out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, m, k, es = case["op"], case["m"], case["k"], BYTES[case["in"]]
    vector = 4 * k if case.get("affine") else 0
    if op == "layernorm":
        moved = m * k * es * (4 if case["residual"] else 2) + 2 * vector + (8 * m if case["stats"] else 0)
        return {"bytes": moved, "flops": 8 * m * k}
    if op in NORMS:
        moved = m * k * es * (4 if case["residual"] else 3) + vector + 4 * k * (2 if op == "layernorm_back" else 1)
        return {"bytes": moved + (8 * m if op == "layernorm_back" else 0), "flops": 14 * m * k}
    n, bias = case["n"], 4 * case["n"] if case["bias"] else 0
    flops = FLOPS[op] * m * n * k
    if op == "linear_back":
        return {"bytes": (2 * m * k + 2 * n * k + m * n) * es + bias, "flops": flops}
    if op == "gated":
        return {"bytes": (m * k + 2 * n * k + m * n * (3 if case["keep"] else 1)) * es + 2 * bias, "flops": flops}
    return {"bytes": (2 * m * k + 4 * n * k + 3 * m * n) * es + 2 * bias, "flops": flops}


# ---------------------------------------------------------------- the definition in 64 bits

def _act64(kind, z):
    """(act(z), its derivative)."""
    if kind == "relu":
        return z.clamp(min=0), torch.where(z > 0, 1.0, 0.0).double()
    if kind == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, torch.addcmul(phi, z, torch.exp(z.square() / -2) * (0.5 / math.pi) ** 0.5)
    if kind == "gelu_tanh":
        # z sigmoid(t), t = 2 sqrt(2/pi) (z + 0.044715 z^3)
        c = math.sqrt(8 / math.pi)
        p = torch.sigmoid(c * torch.addcmul(z, z.pow(3), torch.tensor(0.044715, dtype=z.dtype, device=z.device)))
        return z * p, p + z * p * (1 - p) * c * (1 + 0.134145 * z.square())
    if kind == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    x = s["x"].double()
    if op == "layernorm":
        h = x if s["r"] is None else x + s["r"].double()
        var, mean = torch.var_mean(h, -1, correction=0, keepdim=True)
        std = torch.sqrt(var + LN_EPS)
        y = (h - mean) / std
        if s["w"] is not None:
            y = torch.addcmul(s["b"].double(), y, s["w"].double())
        return {"y": y, **({"h": h} if s["r"] is not None else {}),
                **({"mean": mean[:, 0], "rstd": 1 / std[:, 0]} if case["stats"] else {})}
    if op in NORMS:
        d, k = s["d"].double(), x.shape[1]
        w = torch.ones(k, dtype=torch.float64, device=x.device) if s["w"] is None else s["w"].double()
        if op == "layernorm_back":
            std = 1 / s["rstd"].double()[:, None]
            n = (x - s["mean"].double()[:, None]) / std
            level = (d @ w)[:, None] / k
        else:
            std = torch.sqrt(torch.linalg.vecdot(x, x)[:, None] / k + RMS_EPS)
            n, level = x / std, 0
        dx = (d * w - level - n * (torch.linalg.vecdot(d * n, w.expand_as(n))[:, None] / k)) / std
        out = {"dx": dx if s["s"] is None else dx + s["s"].double(), "dw": torch.einsum("rk,rk->k", d, n)}
        if op == "layernorm_back":
            out["db"] = torch.ones(x.shape[0], dtype=torch.float64, device=x.device) @ d
        return out
    if op == "linear_back":
        d = s["d"].double()
        out = {"dx": torch.mm(d, s["w"].double()), "dw": torch.mm(d.T, x)}
        if case["bias"]:
            out["db"] = torch.ones(x.shape[0], dtype=torch.float64, device=x.device) @ d
        return out
    if op == "gated":
        both = []
        for w, b in ((s["wg"], s["bg"]), (s["wu"], s["bu"])):
            z = torch.mm(x, w.double().T)
            both.append(z if b is None else z.add_(b.double()))
        out = {"y": _act64(case["act"], both[0])[0].mul_(both[1])}
        if case["keep"]:
            out["g"], out["u"] = both
        return out
    a, slope = _act64(case["act"], s["g"].double())
    d = s["d"].double()
    du, dg = a.mul_(d), slope.mul_(d).mul_(s["u"].double())
    out = {"dx": torch.mm(dg, s["wg"].double()).addmm_(du, s["wu"].double()), "dwg": torch.mm(dg.T, x), "dwu": torch.mm(du.T, x)}
    if case["bias"]:
        one = torch.ones(x.shape[0], dtype=torch.float64, device=x.device)
        out["dbg"], out["dbu"] = one @ dg, one @ du
    return out
