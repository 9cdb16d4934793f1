"""64-bit definitions of the operators around a training step's products (CPU, numpy),
and the error bounds that their tests hold the kernels to.

Bounds.  A kernel's result is an fp32 evaluation of the formula, rounded once to its type.
With u = 2^-24 the fp32 unit roundoff:
  * rounding to the result's type costs u_T * |value| (2^-11 fp16, 2^-8 bf16, 2^-24 fp32;
    fp16 also half its smallest subnormal, 2^-25);
  * a sum of n terms by at least 32 lanes with a tree over the lanes costs at most
    (n / 32 + 16) * u times the sum of the magnitudes, a sum in any order n * u times it;
  * every further operation costs u times its result.
Each bound below adds these up for the terms of the formula.
"""
import numpy as np

U = 2.0 ** -24
ROUND = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 0.0, "f32": 0.0}


def rounded(value, elem):
    """The cost of rounding `value` to the type."""
    return ROUND[elem] * np.abs(value) + TINY[elem]


def lanes(n):
    return (n / 32 + 16) * U


# ---- layer norm

def norm_forward(x, gamma, beta, eps):
    mean = x.mean(1)
    var = np.square(x - mean[:, None]).mean(1)
    rstd = 1 / np.sqrt(var + eps)
    hat = (x - mean[:, None]) * rstd[:, None]
    return hat * gamma + beta, mean, rstd


def norm_forward_bounds(x, gamma, beta, eps, elem):
    """Bounds of (y, mean, rstd).  mean: a sum.  var: a sum of squares about a mean that is off by
    dm <= lanes * mean|x| (which adds dm^2, as the sum about the true mean is zero, and the roundings of
    x - mean, u * (|x| + |mean|) each)."""
    y, mean, rstd = norm_forward(x, gamma, beta, eps)
    n = x.shape[1]
    size = np.abs(x).mean(1)
    dm = (lanes(n) + U) * size
    d = np.abs(x - mean[:, None])
    each = U * (d + np.abs(mean)[:, None]) + dm[:, None]     # the error of one x - mean
    # d(var) <= mean(2 d u(d + |mean|)) + dm^2 + lanes * var;   rstd changes by half of that over var + eps
    dvar = (2 * d * U * (d + np.abs(mean)[:, None])).mean(1) + np.square(each).mean(1) + (lanes(n) + 4 * U) * np.square(d).mean(1)
    rel = 0.5 * dvar * np.square(rstd) + 4 * U
    hat = d * rstd[:, None]
    dy = np.abs(gamma) * (each * rstd[:, None] + hat * (rel[:, None] + 4 * U)) + U * np.abs(beta) + U * np.abs(y)
    return dy * 1.01 + rounded(y, elem), dm * 1.01 + U * np.abs(mean), rel * rstd * 1.01


def norm_backward(x, gamma, mean, rstd, dy):
    hat = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - hat * (g * hat).mean(1, keepdims=True))
    return dx, (dy * hat).sum(0), dy.sum(0)


def norm_backward_bounds(x, gamma, mean, rstd, dy, elem, weight):
    dx, dgamma, dbeta = norm_backward(x, gamma, mean, rstd, dy)
    rows, n = x.shape
    hat = np.abs((x - mean[:, None]) * rstd[:, None])
    g = np.abs(dy * gamma)
    few = 8 * U
    a, b = g.mean(1, keepdims=True), (g * hat).mean(1, keepdims=True)
    ddx = rstd[:, None] * (few * g + (lanes(n) + few) * a + hat * (lanes(n) + few) * b)
    dg = (rows * U + few) * (np.abs(dy) * hat).sum(0)
    db = (rows * U + few) * np.abs(dy).sum(0)
    return (ddx * 1.01 + rounded(dx, elem), dg * 1.01 + rounded(dgamma, weight),
            db * 1.01 + rounded(dbeta, weight))


# ---- embedding

def embed_forward(ids, padding, table, scale):
    out = np.zeros((len(ids), table.shape[1]))
    for t, v in enumerate(ids):
        if v != padding and 0 <= v < len(table):
            out[t] = scale * table[v]
    return out


def embed_backward(ids, padding, dout, scale, vocab, start=None):
    """(gradient, bound's sum): the second is the sum of magnitudes times the number of terms."""
    grad = np.zeros((vocab, dout.shape[1])) if start is None else start.copy()
    size, count = np.abs(grad), np.zeros(vocab)
    for t, v in enumerate(ids):
        if v != padding and 0 <= v < vocab:
            grad[v] += scale * dout[t]
            size[v] += abs(scale) * np.abs(dout[t])
            count[v] += 1
    return grad, size * (count[:, None] + 4) * U


# ---- distillation

def teacher(ids, values, tau, teacher_lse=None):
    """(p, log p) with p = 0, log p = -inf where there is no entry."""
    v = np.where(ids >= 0, values / tau, -np.inf)
    if teacher_lse is None:
        high = v.max(1, keepdims=True) if v.shape[1] else np.full((len(v), 1), -np.inf)
        high = np.where(high == -np.inf, 0, high)
        with np.errstate(divide="ignore"):
            norm = high + np.log(np.exp(v - high).sum(1, keepdims=True))
    else:
        norm = teacher_lse[:, None]
    with np.errstate(invalid="ignore"):
        logp = np.where(v == -np.inf, -np.inf, v - norm)
    return np.exp(logp), logp


def distill(logits, ids, values, tau, teacher_lse=None, dloss=None):
    """(loss, lse, dlogits)."""
    rows, vocab = logits.shape
    s = logits / tau
    p, logp = teacher(ids, values, tau, teacher_lse)
    high = s.max(1, keepdims=True)
    high0 = np.where(high == -np.inf, 0, high)
    with np.errstate(divide="ignore"):
        lse = (high0 + np.log(np.exp(s - high0).sum(1, keepdims=True)))[:, 0]
    keep = (p.sum(1) > 0) & (lse > -np.inf)
    loss, grad = np.zeros(rows), np.zeros((rows, vocab))
    for r in np.flatnonzero(keep):
        some = p[r] > 0
        loss[r] = tau * tau * (p[r][some] * (logp[r][some] - s[r][ids[r][some]] + lse[r])).sum()
        grad[r] = p[r].sum() * np.exp(s[r] - lse[r])
        np.add.at(grad[r], ids[r][ids[r] >= 0], -p[r][ids[r] >= 0])
        grad[r] *= tau * (1.0 if dloss is None else dloss[r])
    return loss, np.where(keep, lse, -np.inf), grad


def distill_bounds(logits, ids, values, tau, elem, teacher_lse=None, dloss=None):
    """Bounds of (loss, lse, dlogits).

    An exponent is formed from s / tau with three roundings of values up to the largest magnitude A of the
    row's s / tau, v / tau and log-sum-exps, and exp2 adds two units: `e` is its absolute error, which is the
    relative error of an exponential.  Left-out rows have to be exact."""
    rows, vocab = logits.shape
    loss, lse, grad = distill(logits, ids, values, tau, teacher_lse, dloss)
    p, logp = teacher(ids, values, tau, teacher_lse)
    s = logits / tau
    keep = lse > -np.inf
    fin = lambda a: np.where(np.isfinite(a), np.abs(a), 0.0)  # noqa: E731
    most = lambda a: fin(a).max(1) if a.shape[1] else np.zeros(len(a))  # noqa: E731
    large = most(s) + most(np.where(ids >= 0, values / tau, 0)) + fin(lse) + most(logp) + np.log(vocab + 1.0)
    if teacher_lse is not None:
        large = large + np.abs(teacher_lse)
    e = 4 * U * large + 8 * U
    dlse = e + lanes(vocab) + U * fin(lse)
    mass = p.sum(1)
    dp = 2 * e + lanes(p.shape[1])                             # relative error of p
    terms = np.zeros(rows)
    for r in np.flatnonzero(keep):
        some = p[r] > 0
        t = np.abs(logp[r][some]) + np.abs(s[r][ids[r][some]]) + abs(lse[r])
        terms[r] = (p[r][some] * ((dp[r] + lanes(p.shape[1]) + 4 * U) * t + dp[r] + e[r] + dlse[r])).sum()
    dloss_bound = tau * tau * terms * 1.02
    scale = tau * (np.ones(rows) if dloss is None else np.abs(dloss))
    q = np.where(keep[:, None], np.exp(s - np.where(keep, lse, 0)[:, None]), 0.0)
    own = np.zeros((rows, vocab))
    for r in np.flatnonzero(keep):
        np.add.at(own[r], ids[r][ids[r] >= 0], p[r][ids[r] >= 0])
    rel = (dp + e + dlse + 8 * U + lanes(p.shape[1]))[:, None]
    dgrad = scale[:, None] * (mass[:, None] * q + own) * rel * 1.02
    return dloss_bound, np.where(keep, dlse * 1.02, 0.0), np.where(keep[:, None], dgrad + rounded(grad, elem), 0.0)
