"""64-bit definitions of the operators of a feed-forward block (CPU, torch), and the error bounds
that their tests hold the kernels to.

Bounds.  A kernel's result is an fp32 evaluation of the formula, rounded once to its type.  With
U = 2^-24 the fp32 unit roundoff:
  * rounding to the result's type costs half a step, ROUND * |value| (TINY: half the smallest subnormal);
  * a sum of n terms by at least 16 lanes with a tree over the lanes costs at most (n / 16 + 16) * U times the
    sum of the magnitudes, a sum of n terms in any order n * U times it;
  * every further operation costs U times its result.
Each bound below adds these up for the terms of the formula.
"""
import math

import torch

U = 2.0 ** -24
ROUND = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 0.0, "f32": 0.0}
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 128


def rounded(value, elem):
    """The cost of rounding `value` to the type."""
    return ROUND[elem] * value.abs() + TINY[elem]


def lanes(n):
    return (n / 16 + 16) * U


def groups(n):
    return -(-n // GROUP)


# ---- RMS norm

def rms_total(x, residual):
    """x + residual as it is kept: an fp32 sum, rounded to the type."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def rms_forward(t, gamma, eps):
    t = t.double()
    rstd = 1 / torch.sqrt(t.square().mean(1) + eps)
    return t * rstd[:, None] * gamma.double(), rstd


def rms_error(n):
    """The relative error of rstd: half that of the mean square plus eps, and five operations."""
    return 0.5 * (lanes(n) + 4 * U) + 5 * U


def rms_backward(t, gamma, rstd, dy, dtotal):
    t, dy, rstd = t.double(), dy.double(), rstd.double()[:, None]
    hat, g = t * rstd, dy * gamma.double()
    dx = rstd * (g - hat * (g * hat).mean(1, keepdim=True))
    if dtotal is not None:
        dx = dx + dtotal.double()
    return dx, (dy * hat).sum(0)


def rms_backward_bounds(t, gamma, rstd, dy, dtotal, elem, weight):
    n = t.shape[1]
    dx, dgamma = rms_backward(t, gamma, rstd, dy, dtotal)
    hat, g, r = t.double() * rstd.double()[:, None], dy.double() * gamma.double(), rstd.double()[:, None]
    size = (g * hat).abs().mean(1, keepdim=True)
    ddx = r * (3 * U * g.abs() + hat.abs() * size * (lanes(n) + 8 * U)) + U * dx.abs()
    dg = (t.shape[0] + 4) * U * (dy.double() * hat).abs().sum(0)
    return ddx * 1.01 + rounded(dx, elem), dg * 1.01 + rounded(dgamma, weight)


# ---- 8 bits

def quantize(x, square):
    """(e4m3 values, scales) in the fp32 arithmetic that the definition names."""
    rows, cols = x.shape
    down = GROUP if square else 1
    high = torch.zeros(-(-rows // down) * down, groups(cols) * GROUP)
    high[:rows, :cols] = torch.where(x.isnan(), 0.0, x.abs())
    high = high.view(-1, down, groups(cols), GROUP).amax((1, 3))
    scales = (high * torch.tensor(1 / 448.0)).clamp_min(2.0 ** -126)
    return (x * spread(1 / scales, rows, cols, square)).clamp(-448, 448).to(torch.float8_e4m3fn), scales


def spread(scales, rows, cols, square):
    """The scale of each element."""
    scales = scales.repeat_interleave(GROUP, 1)[:, :cols]
    return scales.repeat_interleave(GROUP, 0)[:rows] if square else scales


def stands_for(q, scales, square):
    """The numbers that an 8-bit matrix stands for, in 64 bits."""
    return q.double() * spread(scales.double(), *q.shape, square)


def conversion_bound(value, scales, square):
    """Half a step of e4m3: 2^-4 of the value, and half the smallest subnormal, 2^-10, times the scale."""
    return 2.0 ** -4 * value.abs() + 2.0 ** -10 * spread(scales.double(), *value.shape, square)


# ---- products

def act(g, kind):
    """(act(g), act'(g)) in 64 bits."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if kind == "gelu":
        phi = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if kind == "relu":
        return g.clamp_min(0), (g > 0).double()
    return g, torch.ones_like(g)


def mma_error(k, step):
    """The error of a sum of k products by tensor cores, over the sum of the magnitudes: each instruction adds `step`
    products and the sum so far, and loses at worst a whole unit (2 U) at each of its additions; the products are exact.
    An instruction aligns its terms and adds them at once, so the running sum is cut once an instruction."""
    return (k / step + step) * 2 * U


def fp8_product(a, a_scales, b, b_scales, square):
    """(C, bound before rounding) of an 8-bit product: per group of 128 an exact-product sum, then the scales' product
    (U), a fused multiply-add (U) and a sum over the groups."""
    x, w = stands_for(a, a_scales, False), stands_for(b, b_scales, square)
    size = x.abs() @ w.abs().t()
    return x @ w.t(), (mma_error(GROUP, 32) + (groups(a.shape[1]) + 4) * U) * size


LIPSCHITZ = 1.13      # of the activations
ACT_ERROR = 2.0 ** -18    # relative, of the fp32 activation with its fast exponential and quotient, for sizes up to 90
# In the lower tails exp and erfc fall below the smallest normal fp32 number (at g = -30 erfc is 1e-197), which no
# fp32 value can stand for: what is below 2^-126 may be taken as zero, and g (up to 2^7) multiplies it.
ACT_TINY = 2.0 ** -119


def gated_forward(x, w, kind):
    """(H, bound, gate_up, bound) before rounding."""
    x, w = x.double(), w.double()
    gu, size = x @ w.t(), x.abs() @ w.abs().t()
    off = mma_error(x.shape[1], 16) * size
    f = w.shape[0] // 2
    g, u, dg, du = gu[:, :f], gu[:, f:], off[:, :f], off[:, f:]
    a = act(g, kind)[0]
    bound = LIPSCHITZ * dg * (u.abs() + du) + a.abs() * du + ACT_ERROR * (a * u).abs() + ACT_TINY * u.abs()
    return a * u, bound, gu, off


def gate_gradient(gate_up, dh, kind):
    """(dgate_up, bound before rounding)"""
    f = dh.shape[1]
    g, u, dh = gate_up.double()[:, :f], gate_up.double()[:, f:], dh.double()
    a, slope = act(g, kind)
    want = torch.cat([dh * u * slope, dh * a], 1)
    # act' is a sum of two terms, each of at most 1.2 in size
    bound = torch.cat([(dh * u).abs() * (2.5 * ACT_ERROR + ACT_TINY), (dh * a).abs() * ACT_ERROR + dh.abs() * ACT_TINY], 1)
    return want, bound
