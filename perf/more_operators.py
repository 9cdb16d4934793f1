"""The operators of a feed-forward block around and within its products: what is measured of them, and their plain forms.

Four operators:

* root-mean-square norm with the residual's addition, its output in its own type or in 8 bits with scales, and its gradient;
* the gated product act(X Wg^T) * (X Wu^T), and its gradients;
* the product of 8-bit (e4m3) matrices with a scale for each 128 elements along K;
* the conversion of a matrix to 8 bits with such scales, as it stands or transposed.

A case names one call of one of them ("op") with its sizes, types and options.  ``run`` makes that call: in elementary
torch operations in 32 bits where ``own`` is false, through this package's public entry points where it is true.
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4}
_FP8 = torch.float8_e4m3fn

_EPS = 1e-5
_GROUP = 128             # elements that share a scale
_TOP = 448.0             # the largest e4m3 number
_LEAST = 2.0 ** -126     # the smallest scale
_LARGEST = 8192 * 16384 * 4096     # rows x columns x K of the largest product


def listed():
    return [
        # the norm before the products of a single token, with the residual's addition: latency
        {"name": "rms_fwd_token", "op": "rms_fwd", "rows": 1, "cols": 4096, "pad": 0, "type": "bf16", "weight": "bf16",
         "residual": True, "fp8": False},
        # the norm of a batch of prompts before an 8-bit product, 32-bit weights
        {"name": "rms_fwd_fp8_batch", "op": "rms_fwd", "rows": 16384, "cols": 4096, "pad": 0, "type": "bf16", "weight": "f32",
         "residual": True, "fp8": True},
        # gradients of a wide norm in a training step, with the gradient along the residual
        {"name": "rms_bwd_batch", "op": "rms_bwd", "rows": 8192, "cols": 8192, "pad": 0, "type": "bf16", "weight": "bf16",
         "residual": True},
        # one token's gated projections: the weights' bytes
        {"name": "gated_fwd_token", "op": "gated_fwd", "M": 1, "F": 8192, "K": 4096, "type": "bf16", "act": "silu",
         "keep": False},
        # a ragged batch of a narrow model in fp16
        {"name": "gated_fwd_ragged", "op": "gated_fwd", "M": 1023, "F": 4104, "K": 2056, "type": "f16", "act": "gelu",
         "keep": False},
        # a training micro-batch's forward pass, which keeps both projections for the gradients
        {"name": "gated_fwd_batch", "op": "gated_fwd", "M": 8192, "F": 16384, "K": 4096, "type": "bf16", "act": "silu",
         "keep": True},
        # gradients of a training micro-batch
        {"name": "gated_bwd_batch", "op": "gated_bwd", "M": 4096, "F": 8192, "K": 4096, "type": "bf16", "act": "silu"},
        # a decoding step of a small batch through an 8-bit layer: the weights' bytes
        {"name": "fp8_step", "op": "fp8", "M": 16, "N": 8192, "K": 4096, "type": "bf16", "b_scales": "square"},
        # a ragged weight gradient: both sides are activations with scales along the tokens
        {"name": "fp8_ragged", "op": "fp8", "M": 1000, "N": 2056, "K": 4112, "type": "f16", "b_scales": "row"},
        # a batch of prompts through a large 8-bit layer
        {"name": "fp8_batch", "op": "fp8", "M": 8192, "N": 8192, "K": 8192, "type": "bf16", "b_scales": "square"},
        # a batch's activations to 8 bits
        {"name": "quantize_rows", "op": "quantize", "rows": 8192, "cols": 8192, "pad": 0, "type": "bf16", "block": "row",
         "transpose": False},
        # a ragged 32-bit weight to 8 bits, transposed for the gradient's product
        {"name": "quantize_squares_transposed", "op": "quantize", "rows": 4099, "cols": 1000, "pad": 5, "type": "f32",
         "block": "square", "transpose": True},
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One case of the listed ones' ranges: any type and option, sizes from a single row up, odd ones among them."""
    op = rng.choice(["rms_fwd", "rms_fwd", "rms_bwd", "gated_fwd", "gated_fwd", "gated_bwd", "fp8", "fp8", "quantize"])
    up = lambda n, m: -(-n // m) * m  # noqa: E731
    if op in ("rms_fwd", "rms_bwd", "quantize"):
        kind = rng.choice(["f16", "bf16", "bf16", "f32"])
        cols = _log_int(rng, 8, 16384)
        if rng.random() < 0.6:               # most programs have sizes of whole 16-byte vectors
            cols = up(cols, 8)
        case = {"op": op, "rows": _log_int(rng, 1, min(65536, (1 << 26) // cols)), "cols": cols,
                "pad": rng.choice([0, 0, 8, 3]), "type": kind}
        if op == "quantize":
            return case | {"block": rng.choice(["row", "square"]), "transpose": rng.random() < 0.5}
        case |= {"weight": rng.choice([kind, "f32"]), "residual": rng.random() < 0.6}
        return case | {"fp8": rng.random() < 0.5} if op == "rms_fwd" else case
    kind = rng.choice(["f16", "bf16"])
    rows = rng.choice([_log_int(rng, 1, 128), _log_int(rng, 128, 8192)])     # decoding steps, batches
    k = up(_log_int(rng, 64, 8192), 16)
    n = up(_log_int(rng, 64, min(16384, _LARGEST // (rows * k))), 8)
    if op == "fp8":
        return {"op": op, "M": rows, "N": n, "K": k, "type": kind, "b_scales": rng.choice(["square", "square", "row"])}
    case = {"op": op, "M": rows, "F": n if op == "gated_fwd" else min(n, up(_LARGEST // (2 * rows * k), 8)), "K": k, "type": kind,
            "act": rng.choice(["silu", "silu", "gelu", "relu", "none"])}
    return case | {"keep": rng.random() < 0.5} if op == "gated_fwd" else case


# ---------------------------------------------------------------- inputs

def _padded(rows, cols, pad, dtype):
    """A rows x cols matrix whose rows stand cols + pad elements apart."""
    return torch.zeros(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]


def _hidden(rows, cols, g):
    """Hidden states: columns of different size, a few of them large."""
    size = torch.exp(0.3 * torch.randn(cols, generator=g, device="cuda"))
    size = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.002, size * 20, size)
    return torch.randn(rows, cols, generator=g, device="cuda") * size


def _groups(n):
    return -(-n // _GROUP)


def _rms_inputs(case, g):
    kind, rows, cols, pad = _TYPES[case["type"]], case["rows"], case["cols"], case["pad"]
    x = _hidden(rows, cols, g)
    if rows > 1:
        x[torch.rand(rows, generator=g, device="cuda") < 0.01] = 0          # rows of padding
    weight = _TYPES[case["weight"]]
    state = {"x": _padded(rows, cols, pad, kind).copy_(x), "residual": None, "total": None, "dtotal": None,
             "gamma": (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(weight)}
    if case["op"] == "rms_fwd":
        if case["residual"]:
            state["residual"] = _padded(rows, cols, pad, kind).copy_(2 * _hidden(rows, cols, g))
            state["total"] = _padded(rows, cols, pad, kind)
        state["rstd"] = torch.empty(rows, device="cuda")
        if case["fp8"]:
            state["q"] = torch.empty(rows, cols, dtype=_FP8, device="cuda")
            state["scales"] = torch.empty(rows, _groups(cols), device="cuda")
        else:
            state["y"] = _padded(rows, cols, pad, kind)
        return state
    state["rstd"] = 1 / torch.sqrt(state["x"].float().square().mean(1) + _EPS)
    state["dy"] = _padded(rows, cols, pad, kind).copy_(torch.randn(rows, cols, generator=g, device="cuda") * 1e-2)
    if case["residual"]:
        state["dtotal"] = _padded(rows, cols, pad, kind).copy_(torch.randn(rows, cols, generator=g, device="cuda") * 1e-2)
    state["dx"] = _padded(rows, cols, pad, kind)
    state["dgamma"] = torch.empty(cols, dtype=weight, device="cuda")
    return state


def _gated_inputs(case, g):
    kind, m, f, k = _TYPES[case["type"]], case["M"], case["F"], case["K"]
    state = {"X": torch.randn(m, k, generator=g, device="cuda").to(kind),
             "W": (torch.randn(2 * f, k, generator=g, device="cuda") / math.sqrt(k)).to(kind)}
    if case["op"] == "gated_fwd":
        state["H"] = torch.empty(m, f, dtype=kind, device="cuda")
        state["gate_up"] = torch.empty(m, 2 * f, dtype=kind, device="cuda") if case["keep"] else None
        return state
    state["gate_up"] = torch.randn(m, 2 * f, generator=g, device="cuda").to(kind)
    state["dH"] = (torch.randn(m, f, generator=g, device="cuda") * 1e-1).to(kind)
    state["dgate_up"] = torch.empty(m, 2 * f, dtype=kind, device="cuda")
    state["dX"], state["dW"] = (torch.empty_like(state[n]) for n in ("X", "W"))
    return state


def _by_rows(x):
    """(8-bit values, scales) of a 32-bit matrix, a scale for each 128 elements of a row."""
    rows, cols = x.shape
    groups = torch.nn.functional.pad(x, (0, -cols % _GROUP)).view(rows, -1, _GROUP)
    scales = (groups.abs().amax(2) * (1 / _TOP)).clamp_min(_LEAST)
    q = (groups * scales.reciprocal()[:, :, None]).clamp(-_TOP, _TOP).view(rows, -1)[:, :cols]
    return q.to(_FP8), scales


def _by_squares(x):
    """(8-bit values, scales) of a 32-bit matrix, a scale for each 128 x 128 elements."""
    rows, cols = x.shape
    blocks = torch.nn.functional.pad(x, (0, -cols % _GROUP, 0, -rows % _GROUP)).view(_groups(rows), _GROUP, -1, _GROUP)
    scales = (blocks.abs().amax((1, 3)) * (1 / _TOP)).clamp_min(_LEAST)
    q = (blocks * scales.reciprocal()[:, None, :, None]).clamp(-_TOP, _TOP)
    return q.view(_groups(rows) * _GROUP, -1)[:rows, :cols].to(_FP8), scales


def _fp8_inputs(case, g):
    m, n, k = case["M"], case["N"], case["K"]
    state = {"C": torch.empty(m, n, dtype=_TYPES[case["type"]], device="cuda")}
    a, a_scales = _by_rows(_hidden(m, k, g))
    if case["b_scales"] == "square":
        b, b_scales = _by_squares(torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k))
    else:
        b, b_scales = _by_rows(_hidden(n, k, g) / math.sqrt(k))
    state["A"], state["B"] = a.contiguous(), b.contiguous()
    state["a_scales"], state["b_scales"] = a_scales.contiguous(), b_scales.contiguous()
    return state


def _quantize_inputs(case, g):
    rows, cols = case["rows"], case["cols"]
    shape = (cols, rows) if case["transpose"] else (rows, cols)
    scales = (_groups(shape[0]) if case["block"] == "square" else shape[0], _groups(shape[1]))
    return {"x": _padded(rows, cols, case["pad"], _TYPES[case["type"]]).copy_(_hidden(rows, cols, g)),
            "q": torch.empty(shape, dtype=_FP8, device="cuda"), "scales": torch.empty(scales, device="cuda")}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    make = {"rms": _rms_inputs, "gated": _gated_inputs, "fp8": _fp8_inputs, "quantize": _quantize_inputs}
    state = make[case["op"].split("_")[0]](case, g)
    state["case"] = case
    if own:
        import dense_gemm_hgemm_gb300 as gb
        if case["op"].startswith("rms"):
            state["plan"] = gb.RmsNormPlan(case["rows"], case["cols"], case["type"], weight=case["weight"])
        elif case["op"].startswith("gated"):
            state["plan"] = gb.GatedPlan(case["M"], case["F"], case["K"], case["type"], act=case["act"])
        elif case["op"] == "fp8":
            state["plan"] = gb.Fp8Plan(case["M"], case["N"], case["K"], case["type"], b_scales=case["b_scales"])
    return state


# ---------------------------------------------------------------- one pass

def _rms_fwd(s, case):
    out = {}
    t = s["x"].float()
    if s["residual"] is not None:
        out["total"] = (t + s["residual"].float()).to(s["x"].dtype)
        t = out["total"].float()
    out["rstd"] = 1 / torch.sqrt(t.square().mean(1) + _EPS)
    y = t * out["rstd"][:, None] * s["gamma"].float()
    if case["fp8"]:
        out["q"], out["scales"] = _by_rows(y)
    else:
        out["y"] = y.to(s["x"].dtype)
    return out


def _rms_bwd(s, case):
    rstd, dy = s["rstd"][:, None], s["dy"].float()
    hat = s["x"].float() * rstd
    g = dy * s["gamma"].float()
    dx = rstd * (g - hat * (g * hat).mean(1, keepdim=True))
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * hat).sum(0).to(s["gamma"].dtype)}


def _act(g, act):
    """(act(g), act'(g))"""
    if act == "silu":
        half = 1 / (1 + torch.exp(-g))
        return g * half, half * (1 + g * (1 - half))
    if act == "gelu":
        phi = 0.5 * (1 + torch.erf(g / math.sqrt(2)))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if act == "relu":
        return torch.where(g > 0, g, 0.0), (g > 0).float()
    return g, torch.ones_like(g)


def _gated_fwd(s, case):
    gate_up = s["X"].float() @ s["W"].float().t()
    g, u = gate_up.split(case["F"], 1)
    out = {"H": (_act(g, case["act"])[0] * u).to(s["X"].dtype)}
    if case["keep"]:
        out["gate_up"] = gate_up.to(s["X"].dtype)
    return out


def _gated_bwd(s, case):
    kind = s["X"].dtype
    g, u = s["gate_up"].float().split(case["F"], 1)
    dh = s["dH"].float()
    value, slope = _act(g, case["act"])
    dgate_up = torch.cat([dh * u * slope, dh * value], 1)
    return {"dgate_up": dgate_up.to(kind), "dX": (dgate_up @ s["W"].float()).to(kind),
            "dW": (dgate_up.t() @ s["X"].float()).to(kind)}


def _spread(scales, rows, cols, square, dtype=torch.float32):
    """A rows x cols matrix of the scales of its elements."""
    scales = scales.to(dtype).repeat_interleave(_GROUP, 1)[:, :cols]
    return scales.repeat_interleave(_GROUP, 0)[:rows] if square else scales


def _fp8(s, case):
    a = s["A"].float() * _spread(s["a_scales"], case["M"], case["K"], False)
    b = s["B"].float() * _spread(s["b_scales"], case["N"], case["K"], case["b_scales"] == "square")
    return (a @ b.t()).to(s["C"].dtype)


def _quantize(s, case):
    x = s["x"].float()
    q, scales = (_by_rows if case["block"] == "row" else _by_squares)(x.t() if case["transpose"] else x)
    return {"q": q.contiguous(), "scales": scales}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        plain = {"rms_fwd": _rms_fwd, "rms_bwd": _rms_bwd, "gated_fwd": _gated_fwd, "gated_bwd": _gated_bwd, "fp8": _fp8,
                 "quantize": _quantize}
        return plain[op](s, case)
    if op == "quantize":
        import dense_gemm_hgemm_gb300 as gb
        gb.fp8_quantize(s["x"], s["q"], s["scales"], block=case["block"], transpose=case["transpose"])
        return {"q": s["q"], "scales": s["scales"]}
    plan = s["plan"]
    if op == "rms_fwd":
        more = {"rstd": s["rstd"], "residual": s["residual"], "total": s["total"], "eps": _EPS}
        out = {"rstd": s["rstd"]}
        if case["fp8"]:
            plan.forward_fp8(s["x"], s["gamma"], s["q"], s["scales"], **more)
            out |= {"q": s["q"], "scales": s["scales"]}
        else:
            plan.forward(s["x"], s["gamma"], s["y"], **more)
            out["y"] = s["y"]
        if case["residual"]:
            out["total"] = s["total"]
        return out
    if op == "rms_bwd":
        plan.backward(s["x"], s["gamma"], s["rstd"], s["dy"], s["dx"], s["dgamma"], dtotal=s["dtotal"])
        return {"dx": s["dx"], "dgamma": s["dgamma"]}
    if op == "gated_fwd":
        plan.forward(s["X"], s["W"], s["H"], gate_up=s["gate_up"])
        return {"H": s["H"], "gate_up": s["gate_up"]} if case["keep"] else {"H": s["H"]}
    if op == "gated_bwd":
        plan.backward(s["X"], s["W"], s["gate_up"], s["dH"], s["dgate_up"], s["dX"], s["dW"])
        return {"dgate_up": s["dgate_up"], "dX": s["dX"], "dW": s["dW"]}
    plan.run(s["A"], s["a_scales"], s["B"], s["b_scales"], s["C"])
    return s["C"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, e = case["op"], _BYTES[case["type"]]
    if op in ("rms_fwd", "rms_bwd"):
        n, r = case["rows"] * case["cols"], 2 if case["residual"] else 0
        weights = case["cols"] * _BYTES[case["weight"]]
        if op == "rms_bwd":
            return {"bytes": (3 + r / 2) * n * e + 2 * weights + 4 * case["rows"], "flops": 12 * n}
        out = n + 4 * case["rows"] * _groups(case["cols"]) if case["fp8"] else n * e
        return {"bytes": (1 + r) * n * e + out + weights + 4 * case["rows"], "flops": 6 * n}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        scales = n // _GROUP if case["block"] == "row" else n // _GROUP ** 2
        return {"bytes": n * (e + 1) + 4 * scales, "flops": 3 * n}
    m, k = case["M"], case["K"]
    if op == "fp8":
        n = case["N"]
        scales = (m + (n if case["b_scales"] == "row" else _groups(n))) * _groups(k)
        return {"bytes": (m + n) * k + m * n * e + 4 * scales, "flops": 2 * m * n * k}
    f = case["F"]
    if op == "gated_fwd":
        return {"bytes": ((m + 2 * f) * k + m * f * (3 if case["keep"] else 1)) * e, "flops": 4 * m * f * k}
    return {"bytes": (2 * (m + 2 * f) * k + 5 * m * f) * e, "flops": 8 * m * f * k}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _exact_scales(y, square):
    """The scales of a 64-bit matrix and, unrounded, what its 8-bit values stand for over them."""
    rows, cols = y.shape
    down = _GROUP if square else 1
    high = torch.zeros(-(-rows // down) * down, _groups(cols) * _GROUP, dtype=torch.float64, device="cuda")
    high[:rows, :cols] = y.abs()
    scales = (high.view(-1, down, _groups(cols), _GROUP).amax((1, 3)) / _TOP).clamp_min(_LEAST)
    return scales, y / _spread(scales, rows, cols, square, torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rms_fwd":
        t, out = s["x"].double(), {}
        if case["residual"]:
            # the sum as it is kept: the norm is of what the next layer reads (the 32-bit sum's own rounding is far below)
            t = (t + s["residual"].double()).to(s["x"].dtype).double()
            out["total"] = t
        out["rstd"] = torch.rsqrt((t * t).sum(1) / case["cols"] + _EPS)
        y = t * (out["rstd"][:, None] * s["gamma"].double()[None, :])
        if case["fp8"]:
            out["scales"], out["q"] = _exact_scales(y, False)
        else:
            out["y"] = y
        return out
    if op == "rms_bwd":
        t, dy, rstd = s["x"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        up = dy * s["gamma"].double()
        along = torch.einsum("ij,ij->i", up, t)[:, None]
        dx = rstd * up - rstd ** 3 * t * along / case["cols"]
        if case["residual"]:
            dx += s["dtotal"].double()
        return {"dx": dx, "dgamma": torch.einsum("ij,ij,i->j", dy, t, rstd[:, 0])}
    if op == "quantize":
        y = s["x"].double()
        scales, q = _exact_scales(y.t() if case["transpose"] else y, case["block"] == "square")
        return {"scales": scales, "q": q}
    if op == "fp8":
        a = s["A"].double() * _spread(s["a_scales"], case["M"], case["K"], False, torch.float64)
        b = s["B"].double() * _spread(s["b_scales"], case["N"], case["K"], case["b_scales"] == "square", torch.float64)
        return torch.mm(a, b.T)
    f = case["F"]
    x, w = s["X"].double(), s["W"].double()
    gate_up = s["gate_up"].double() if op == "gated_bwd" else torch.mm(x, w.T)
    g, u = gate_up[:, :f], gate_up[:, f:]
    if case["act"] == "silu":
        half = torch.sigmoid(g)
        value, slope = half * g, half + half * g * torch.sigmoid(-g)
    elif case["act"] == "gelu":
        half = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        value, slope = half * g, half + g * torch.exp(-g.square() / 2) * (1 / math.sqrt(2 * math.pi))
    elif case["act"] == "relu":
        value, slope = g.clamp_min(0), torch.heaviside(g, torch.zeros((), dtype=g.dtype, device="cuda"))
    else:
        value, slope = g, torch.ones_like(g)
    if op == "gated_fwd":
        return {"H": value * u, "gate_up": gate_up} if case["keep"] else {"H": value * u}
    dh = s["dH"].double()
    dgate_up = torch.cat([slope * u * dh, value * dh], 1)
    return {"dgate_up": dgate_up, "dX": torch.mm(dgate_up, w), "dW": torch.mm(dgate_up.T, x)}
