"""The operators around the products of a training step: what is measured of them, and their plain forms.

Three operators, each with its gradient:

* the embedding lookup with a scale, and the gradient of its table;
* layer norm, and its gradient with the reduction of the weight's and the bias' gradients;
* the distillation loss against a teacher's top logits: forward, backward, and both in one call.

A case names one call of one of them ("op") with its sizes, types and options.  ``run`` makes that call: in elementary
torch operations in 32 bits where ``own`` is false, through this package's public entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4, "i32": 4, "i64": 8}
_INDEX = {"i32": torch.int32, "i64": torch.int64}

_PAD_SHARE = 0.03        # share of padding tokens in a batch of token ids
_PADDING = 0             # the padding token's id
_LEFT_OUT = 0.06         # share of loss rows without teacher entries (prompt and padding positions)
_EPS = 1e-5


def listed():
    return [
        # the tokens of one decoding step of a small batch: latency
        {"name": "embed_fwd_step", "op": "embed_fwd", "tokens": 8, "vocab": 32000, "dim": 4096, "type": "bf16",
         "index": "i64", "scale": 64.0},
        # the tokens of one training micro-batch
        {"name": "embed_fwd_batch", "op": "embed_fwd", "tokens": 16384, "vocab": 128000, "dim": 4096, "type": "bf16",
         "index": "i32", "scale": 64.0},
        # the same batch's table gradient, written whole (most of the table's rows are zeros)
        {"name": "embed_bwd_dense", "op": "embed_bwd", "tokens": 16384, "vocab": 64000, "dim": 4096, "type": "bf16",
         "grad": "bf16", "index": "i64", "scale": 64.0, "accumulate": False},
        # gradient accumulation into a 32-bit table: an odd vocabulary, a ragged batch, rows of 1000 elements
        {"name": "embed_bwd_accumulate", "op": "embed_bwd", "tokens": 4099, "vocab": 50021, "dim": 1000, "type": "f16",
         "grad": "f32", "index": "i32", "scale": 1.0, "accumulate": True},
        # one row: the norm before the product of a single token, latency
        {"name": "norm_fwd_token", "op": "norm_fwd", "rows": 1, "cols": 4096, "pad": 0, "type": "bf16", "weight": "bf16"},
        # the norm before the FFN product of a training micro-batch, 32-bit weights
        {"name": "norm_fwd_batch", "op": "norm_fwd", "rows": 16384, "cols": 4096, "pad": 0, "type": "bf16",
         "weight": "f32"},
        # gradients of a wide norm
        {"name": "norm_bwd_batch", "op": "norm_bwd", "rows": 8192, "cols": 8192, "pad": 0, "type": "bf16",
         "weight": "bf16"},
        # a ragged micro-batch of a narrow model, rows of 1000 elements inside wider ones
        {"name": "norm_bwd_ragged", "op": "norm_bwd", "rows": 1023, "cols": 1000, "pad": 24, "type": "f16",
         "weight": "f32"},
        # the validation loss of a few rows in 32 bits: fewer rows than multiprocessors
        {"name": "distill_fwd_few", "op": "distill_fwd", "rows": 33, "vocab": 32000, "pad": 0, "top": 20, "type": "f32",
         "teacher": "f32", "index": "i64", "temperature": 1.0, "teacher_lse": False},
        # the validation loss of a batch over a large vocabulary
        {"name": "distill_fwd_batch", "op": "distill_fwd", "rows": 4096, "vocab": 128000, "pad": 0, "top": 64,
         "type": "bf16", "teacher": "f16", "index": "i32", "temperature": 2.0, "teacher_lse": False},
        # the loss' gradient alone (its upstream gradient known later), logits padded to the product's eight columns
        {"name": "distill_bwd_padded", "op": "distill_bwd", "rows": 2048, "vocab": 50021, "pad": 3, "top": 32,
         "type": "f16", "teacher": "f32", "index": "i32", "temperature": 1.0, "teacher_lse": True},
        # loss and gradient of a training micro-batch in one call
        {"name": "distill_step_batch", "op": "distill_step", "rows": 4096, "vocab": 64000, "pad": 0, "top": 64,
         "type": "bf16", "teacher": "bf16", "index": "i64", "temperature": 2.0, "teacher_lse": False},
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One case of the listed ones' ranges: any type and option, sizes from a single row up, odd ones among them."""
    op = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd", "distill_fwd", "distill_bwd", "distill_step"])
    kind = rng.choice(["f16", "bf16", "bf16", "f32"])
    index = rng.choice(["i32", "i64"])
    even = rng.random() < 0.6                # most programs have sizes of whole 16-byte vectors
    size = lambda lo, hi: _log_int(rng, lo, hi) if not even else -(-_log_int(rng, lo, hi) // 8) * 8  # noqa: E731
    if op.startswith("embed"):
        dim = size(8, 8192)
        case = {"op": op, "tokens": _log_int(rng, 1, min(32768, (1 << 26) // dim)),
                "vocab": _log_int(rng, 16, min(128000, (1 << 27) // dim)), "dim": dim, "type": kind, "index": index,
                "scale": rng.choice([1.0, math.sqrt(dim)])}
        if op == "embed_bwd":
            case["grad"] = rng.choice([kind, "f32"])
            case["accumulate"] = rng.random() < 0.5
        return case
    if op.startswith("norm"):
        cols = size(8, 16384)
        return {"op": op, "rows": _log_int(rng, 1, min(65536, (1 << 26) // cols)), "cols": cols,
                "pad": rng.choice([0, 0, 8, 3]), "type": kind, "weight": rng.choice([kind, "f32"])}
    vocab = size(100, 128000)
    return {"op": op, "rows": _log_int(rng, 1, min(16384, 120_000_000 // vocab)), "vocab": vocab,
            "pad": rng.choice([0, -vocab % 8, 5]), "top": _log_int(rng, 1, 90), "type": kind,
            "teacher": rng.choice(["f16", "bf16", "f32"]), "index": index,
            "temperature": rng.choice([1.0, 2.0, rng.uniform(0.7, 4.0)]), "teacher_lse": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

def _padded(rows, cols, pad, dtype):
    """A rows x cols matrix whose rows stand cols + pad elements apart."""
    return torch.zeros(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]


def _token_ids(case, g):
    """Token ids as text has them: the n-th most frequent one about 1/n as often, the frequent ones anywhere in the
    table, and some padding."""
    n, vocab = case["tokens"], case["vocab"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)).long() - 1).clamp(0, vocab - 1)
    ids = (rank * 7919 + 13) % vocab
    pad = torch.rand(n, generator=g, device="cuda") < _PAD_SHARE
    return torch.where(pad, torch.full_like(ids, _PADDING), ids).to(_INDEX[case["index"]])


def _embed_inputs(case, g):
    kind, n, vocab, dim = _TYPES[case["type"]], case["tokens"], case["vocab"], case["dim"]
    state = {"ids": _token_ids(case, g)}
    if case["op"] == "embed_fwd":
        state["table"] = (torch.randn(vocab, dim, generator=g, device="cuda") * 0.02).to(kind)
        state["out"] = torch.empty(n, dim, dtype=kind, device="cuda")
    else:
        state["dout"] = (torch.randn(n, dim, generator=g, device="cuda") * 1e-2).to(kind)
        shape, grad = (vocab, dim), _TYPES[case["grad"]]
        state["dtable"] = ((torch.randn(shape, generator=g, device="cuda") * 1e-2).to(grad) if case["accumulate"]
                           else torch.empty(shape, dtype=grad, device="cuda"))
    return state


def _norm_inputs(case, g):
    kind, rows, cols, pad = _TYPES[case["type"]], case["rows"], case["cols"], case["pad"]
    # hidden states: columns of different size, a few of them large, and some rows of padding that are all zeros
    size = torch.exp(0.3 * torch.randn(cols, generator=g, device="cuda"))
    size = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.002, size * 20, size)
    x = torch.randn(rows, cols, generator=g, device="cuda") * size + 0.1
    if rows > 1:
        x[torch.rand(rows, generator=g, device="cuda") < 0.01] = 0
    weight = _TYPES[case["weight"]]
    state = {"x": _padded(rows, cols, pad, kind).copy_(x),
             "gamma": (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(weight)}
    if case["op"] == "norm_fwd":
        state["beta"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(weight)
        state["y"] = _padded(rows, cols, pad, kind)
        state["mean"], state["rstd"] = (torch.empty(rows, device="cuda") for _ in range(2))
    else:
        x = state["x"].float()
        state["mean"] = x.mean(1)
        state["rstd"] = 1 / torch.sqrt((x - state["mean"][:, None]).square().mean(1) + _EPS)
        state["dy"] = _padded(rows, cols, pad, kind).copy_(torch.randn(rows, cols, generator=g, device="cuda") * 1e-2)
        state["dx"] = _padded(rows, cols, pad, kind)
        state["dgamma"], state["dbeta"] = (torch.empty(cols, dtype=weight, device="cuda") for _ in range(2))
    return state


def _distill_inputs(case, g):
    kind, rows, vocab, top = _TYPES[case["type"]], case["rows"], case["vocab"], case["top"]
    masked = min(16, vocab // 100)           # the table's last rows are no tokens: their logits are masked
    tokens = vocab - masked
    uniform = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    # the teacher's top entries: distinct tokens, falling logits; a tenth of the rows has fewer, some have none
    start = (uniform(rows, 1) * tokens).long()
    step = 1 + (uniform(rows, 1) * (tokens // top - 1)).long()
    at = torch.arange(top, device="cuda")
    ids = (start + step * at) % tokens
    gaps = -torch.log(uniform(rows, top).clamp_min(1e-6)) * (6.0 / top)
    values = (12 - torch.cumsum(gaps, 1)).to(_TYPES[case["teacher"]])
    count = torch.where(uniform(rows) < 0.1, (uniform(rows) * top).long() + 1, top)
    if rows > 1:
        count = torch.where(uniform(rows) < _LEFT_OUT, 0, count)
        count[0] = top
    logits = _padded(rows, vocab, case["pad"], kind)
    logits.copy_(torch.randn(rows, vocab, generator=g, device="cuda") * 1.5)
    logits.scatter_add_(1, ids, (values.float() - 5 + torch.randn(rows, top, generator=g, device="cuda")).to(kind))
    if masked:
        logits[:, tokens:] = -math.inf
    state = {"logits": logits, "values": values, "teacher_lse": None,
             "ids": torch.where(at < count[:, None], ids, -1).to(_INDEX[case["index"]]),
             "loss": torch.empty(rows, device="cuda"), "lse": torch.empty(rows, device="cuda")}
    if case["teacher_lse"]:                  # the teacher's whole distribution has some more mass than its top
        state["teacher_lse"] = torch.logsumexp(values.float() / case["temperature"], 1) + 0.2 * uniform(rows)
    if case["op"] != "distill_fwd":
        scale = 512.0 if case["type"] == "f16" else 1.0      # the usual loss scale of 16-bit gradients
        state["dloss"] = (0.5 + uniform(rows)) * scale
        state["dlogits"] = _padded(rows, vocab, case["pad"], kind)
    if case["op"] == "distill_bwd":
        lse = torch.empty(rows, device="cuda")
        for r in range(0, rows, 1024):
            lse[r:r + 1024] = torch.logsumexp(logits[r:r + 1024].float() / case["temperature"], 1)
        state["lse"] = torch.where(count > 0, lse, -math.inf)
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    make = {"embed": _embed_inputs, "norm": _norm_inputs, "distill": _distill_inputs}[case["op"].split("_")[0]]
    state = make(case, g)
    state["case"] = case
    if own:
        import dense_gemm_hgemm_gb300 as gb
        if case["op"].startswith("embed"):
            state["plan"] = gb.EmbedPlan(case["vocab"], case["dim"], case["tokens"], case["type"],
                                         grad=case.get("grad", case["type"]))
        elif case["op"].startswith("norm"):
            state["plan"] = gb.NormPlan(case["rows"], case["cols"], case["type"], weight=case["weight"])
        else:
            state["plan"] = gb.DistillPlan(case["rows"], case["vocab"], case["top"], case["type"])
    return state


# ---------------------------------------------------------------- one pass

def _embed_fwd(s, case):
    ids = s["ids"].long()
    rows = s["table"][ids].float() * case["scale"]
    return torch.where((ids != _PADDING)[:, None], rows, 0.0).to(s["table"].dtype)


def _embed_bwd(s, case):
    ids = s["ids"].long()
    rows = s["dout"].float() * case["scale"]
    rows = torch.where((ids != _PADDING)[:, None], rows, 0.0)
    total = torch.zeros(case["vocab"], case["dim"], device="cuda").index_add_(0, ids, rows)
    if case["accumulate"]:
        return s["dtable"].copy_(s["dtable"].float() + total)
    return total.to(s["dtable"].dtype)


def _norm_fwd(s, case):
    x = s["x"].float()
    mean = x.mean(1)
    x = x - mean[:, None]
    rstd = 1 / torch.sqrt((x * x).mean(1) + _EPS)
    y = x * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _norm_bwd(s, case):
    x, dy = s["x"].float(), s["dy"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["gamma"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    weight = s["gamma"].dtype
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum(0).to(weight), "dbeta": dy.sum(0).to(weight)}


def _teacher(s, case, dtype=torch.float32):
    """The teacher's probabilities p, log p, and which entries there are."""
    there = s["ids"] >= 0
    v = torch.where(there, s["values"].to(dtype) / case["temperature"], -math.inf)
    if s["teacher_lse"] is not None:
        norm = s["teacher_lse"].to(dtype)[:, None]
    else:
        high = v.max(1, keepdim=True).values
        high = torch.where(high > -math.inf, high, 0.0)
        norm = high + torch.log(torch.exp(v - high).sum(1, keepdim=True))
    logp = torch.where(there, v - norm, -math.inf)
    return torch.exp(logp), logp, there


def _distill_loss(s, case, scaled, p, logp, there):
    """(loss, lse) from the logits over the temperature."""
    high = scaled.max(1, keepdim=True).values
    safe = torch.where(high > -math.inf, high, 0.0)
    lse = (safe + torch.log(torch.exp(scaled - safe).sum(1, keepdim=True)))[:, 0]
    kept = there.any(1) & (lse > -math.inf)
    at = scaled.gather(1, s["ids"].long().clamp_min(0))
    terms = torch.where(p > 0, p * (logp - at + lse[:, None]), 0.0)
    loss = torch.where(kept, case["temperature"] ** 2 * terms.sum(1), 0.0)
    return loss, torch.where(kept, lse, -math.inf)


def _distill_grad(s, case, scaled, lse, p, there):
    kept = lse > -math.inf
    grad = torch.exp(scaled - torch.where(kept, lse, 0.0)[:, None]) * p.sum(1, keepdim=True)
    grad = grad.scatter_add_(1, s["ids"].long().clamp_min(0), torch.where(there, -p, 0.0))
    grad = grad * (case["temperature"] * s["dloss"])[:, None]
    return torch.where(kept[:, None], grad, 0.0).to(s["logits"].dtype)


def _distill(s, case):
    scaled = s["logits"].float() / case["temperature"]
    p, logp, there = _teacher(s, case)
    if case["op"] == "distill_bwd":
        return {"dlogits": _distill_grad(s, case, scaled, s["lse"], p, there)}
    loss, lse = _distill_loss(s, case, scaled, p, logp, there)
    out = {"loss": loss, "lse": lse}
    if case["op"] == "distill_step":
        out["dlogits"] = _distill_grad(s, case, scaled, lse, p, there)
    return out


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        plain = {"embed_fwd": _embed_fwd, "embed_bwd": _embed_bwd, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd}
        return plain.get(op, _distill)(s, case)
    plan = s["plan"]
    if op == "embed_fwd":
        plan.forward(s["ids"], s["table"], s["out"], scale=case["scale"], padding=_PADDING)
        return s["out"]
    if op == "embed_bwd":
        plan.backward(s["ids"], s["dout"], s["dtable"], scale=case["scale"], padding=_PADDING,
                      accumulate=case["accumulate"])
        return s["dtable"]
    if op == "norm_fwd":
        plan.forward(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], eps=_EPS)
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_bwd":
        plan.backward(s["x"], s["gamma"], s["mean"], s["rstd"], s["dy"], s["dx"], s["dgamma"], s["dbeta"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    more = {"temperature": case["temperature"], "teacher_lse": s["teacher_lse"]}
    if op == "distill_fwd":
        plan.forward(s["logits"], s["ids"], s["values"], s["loss"], s["lse"], **more)
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "distill_bwd":
        plan.backward(s["logits"], s["ids"], s["values"], s["lse"], s["dlogits"], dloss=s["dloss"], **more)
        return {"dlogits": s["dlogits"]}
    plan.forward_backward(s["logits"], s["ids"], s["values"], s["loss"], s["lse"], s["dlogits"], dloss=s["dloss"],
                          **more)
    return {"loss": s["loss"], "lse": s["lse"], "dlogits": s["dlogits"]}


# ---------------------------------------------------------------- what a pass cannot do without

def _distinct(case):
    """How many different tokens a batch has, by the frequencies of _token_ids (without the padding)."""
    v = np.arange(case["vocab"], dtype=np.float64)
    share = np.log((v + 2) / (v + 1)) / math.log(case["vocab"] + 1) * (1 - _PAD_SHARE)
    return float((1 - (1 - share) ** case["tokens"]).sum())


def work(case):
    op, e = case["op"], _BYTES[case["type"]]
    if op.startswith("embed"):
        n, dim, vocab = case["tokens"], case["dim"], case["vocab"]
        ids = n * _BYTES[case["index"]]
        if op == "embed_fwd":
            return {"bytes": ids + n * dim * e + _distinct(case) * dim * e, "flops": n * dim}
        grads = (2 * _distinct(case) if case["accumulate"] else vocab) * dim * _BYTES[case["grad"]]
        return {"bytes": ids + n * (1 - _PAD_SHARE) * dim * e + grads, "flops": n * dim}
    if op.startswith("norm"):
        n = case["rows"] * case["cols"]
        weights = case["cols"] * _BYTES[case["weight"]]
        if op == "norm_fwd":
            return {"bytes": 2 * n * e + 2 * weights + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 3 * weights + 8 * case["rows"], "flops": 16 * n}
    rows, vocab = case["rows"], case["vocab"]
    kept = rows * (1 - _LEFT_OUT) if rows > 1 else 1
    teacher = rows * case["top"] * (_BYTES[case["index"]] + _BYTES[case["teacher"]]) + 12 * rows
    if op == "distill_fwd":
        return {"bytes": kept * vocab * e + teacher, "flops": 4 * kept * vocab}
    return {"bytes": (kept + rows) * vocab * e + teacher, "flops": (4 if op == "distill_bwd" else 8) * kept * vocab}


# ---------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed_fwd":
        out = s["table"].double().index_select(0, s["ids"].long()) * case["scale"]
        out[s["ids"] == _PADDING] = 0
        return out
    if op == "embed_bwd":
        kept = s["ids"] != _PADDING
        out = (s["dtable"].double() if case["accumulate"]
               else torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda"))
        return out.index_add_(0, s["ids"][kept].long(), s["dout"][kept].double(), alpha=case["scale"])
    if op == "norm_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = torch.rsqrt(var + _EPS)
        hat = (x - mean[:, None]) * rstd[:, None]
        return {"y": hat * s["gamma"].double() + s["beta"].double(), "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        hat = (s["x"].double() - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
        dy, cols = s["dy"].double(), case["cols"]
        up = dy * s["gamma"].double()
        along = (up * hat).sum(1, keepdim=True)
        dx = (cols * up - up.sum(1, keepdim=True) - hat * along) / cols * s["rstd"].double()[:, None]
        return {"dx": dx, "dgamma": torch.einsum("ij,ij->j", dy, hat), "dbeta": dy.sum(0)}
    tau, rows, vocab = case["temperature"], case["rows"], case["vocab"]
    loss, lses, grads = [], [], []
    block = max(1, (1 << 26) // vocab)
    for r in range(0, rows, block):
        logits = s["logits"][r:r + block].double() / tau
        ids, values = s["ids"][r:r + block].long(), s["values"][r:r + block].double() / tau
        values = values.masked_fill(ids < 0, -math.inf)
        whole = s["teacher_lse"][r:r + block].double() if s["teacher_lse"] is not None else values.logsumexp(1)
        some = (ids >= 0).any(1)
        p = torch.exp(values - torch.where(some, whole, 0.0)[:, None])
        lse = logits.logsumexp(1)
        if op == "distill_bwd":
            lse = s["lse"][r:r + block].double()
        else:
            logq = (logits - lse[:, None]).gather(1, ids.clamp_min(0))
            loss.append((torch.xlogy(p, p) - torch.where(p > 0, p * logq, 0.0)).sum(1) * tau * tau)
            lse = lse.masked_fill(~some, -math.inf)
        lses.append(lse)
        if op != "distill_fwd":
            q = torch.exp(logits - torch.where(some, lse, 0.0)[:, None]) * p.sum(1, keepdim=True)
            one = torch.arange(ids.shape[0], device="cuda")[:, None].expand_as(ids)
            q.index_put_((one, ids.clamp_min(0)), -p, accumulate=True)
            grads.append(q * (tau * some * s["dloss"][r:r + block].double())[:, None])
    out = {}
    if op != "distill_bwd":
        out = {"loss": torch.cat(loss), "lse": torch.cat(lses)}
    if op != "distill_fwd":
        out["dlogits"] = torch.cat(grads)
    return out
