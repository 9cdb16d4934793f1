"""A feed-forward block's training step, and a projection in 8 bits, on the library's kernels alone.

The block, with the residual around it:

    t = x + r ; y = norm(t)                      (RmsNormPlan, one call)
    h = silu(y Wg^T) * (y Wu^T)                  (GatedPlan, one call, which keeps both products)
    out = h Wd^T                                 (Plan, TN)

and its gradients: the down product's (Plan NN and NT), the gated product's, the norm's with the
gradient that comes along the residual.

The projection c = norm(x + r) W^T in 8 bits (e4m3) with a scale for each 128 elements: the norm's
results come as 8-bit rows (RmsNormPlan.forward_fp8), the weights are converted once by squares
(fp8_quantize), and so are, transposed, what the gradients' two products take (Fp8Plan).

    python examples/ffn_block.py [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_hgemm_gb300 as g  # noqa: E402

BF16 = {"dtype": torch.bfloat16, "device": "cuda"}


class Block:
    """Weights, buffers and plans of one batch size."""

    def __init__(self, tokens=512, dim=256, inner=704, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, std):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()
        self.gamma = torch.ones(dim, device="cuda")
        self.gate_up = weight(2 * inner, dim, std=dim ** -0.5)
        self.down = weight(dim, inner, std=inner ** -0.5)
        new = lambda *s: torch.empty(*s, **BF16)  # noqa: E731
        self.total, self.normed, self.out = (new(tokens, dim) for _ in range(3))
        self.products, self.h = new(tokens, 2 * inner), new(tokens, inner)
        self.rstd = torch.empty(tokens, device="cuda")
        self.d_products, self.d_h, self.d_normed, self.d_x = new(tokens, 2 * inner), new(tokens, inner), new(tokens, dim), new(tokens, dim)
        self.grad = {"gamma": torch.empty_like(self.gamma), "gate_up": torch.empty_like(self.gate_up),
                     "down": torch.empty_like(self.down)}
        self.norm = g.RmsNormPlan(tokens, dim, "bf16", weight="f32")
        self.gated = g.GatedPlan(tokens, inner, dim, "bf16", act="silu")
        self.product = g.Plan(tokens, dim, inner, "bf16", layout="TN")       # out = h . down^T
        self.to_input = g.Plan(tokens, inner, dim, "bf16", layout="NN")      # d_h = d_out . down
        self.to_weight = g.Plan(dim, inner, tokens, "bf16", layout="NT")     # d_down = d_out^T . h

    def forward(self, x, residual):
        """The block's result in self.out, the sum for the next residual in self.total."""
        self.norm.forward(x, self.gamma, self.normed, self.rstd, residual=residual, total=self.total)
        self.gated.forward(self.normed, self.gate_up, self.h, gate_up=self.products)
        self.product.run(self.h, self.down, self.out)

    def backward(self, d_out, d_total):
        """The gradients of the weights in self.grad, of x (and of the residual) in self.d_x."""
        self.to_input.run(d_out, self.down, self.d_h)
        self.to_weight.run(d_out, self.h, self.grad["down"])
        self.gated.backward(self.normed, self.gate_up, self.products, self.d_h, self.d_products, self.d_normed,
                            self.grad["gate_up"])
        self.norm.backward(self.total, self.gamma, self.rstd, self.d_normed, self.d_x, self.grad["gamma"], dtotal=d_total)

    def check(self):
        """Raises what the kernels have to report."""
        for plan in (self.gated, self.product, self.to_input, self.to_weight):
            plan.check()

    def close(self):
        for plan in (self.norm, self.gated, self.product, self.to_input, self.to_weight):
            plan.close()


class Projection:
    """c = norm(x + residual) W^T with 8-bit operands, and its gradients."""

    def __init__(self, weight, tokens):
        out, dim = weight.shape
        groups = lambda n: -(-n // 128)  # noqa: E731

        def held(rows, cols, square=False):
            return (torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda"),
                    torch.empty(groups(rows) if square else rows, groups(cols), device="cuda"))

        def along_tokens(rows):
            # (the product's K is a multiple of 16: zeros stand behind the last token)
            whole = torch.zeros(rows, -(-tokens // 16) * 16, device="cuda").to(torch.float8_e4m3fn)
            return whole, whole[:, :tokens], torch.empty(rows, groups(tokens), device="cuda")
        self.gamma = torch.ones(dim, device="cuda")
        self.w, self.w_turned = held(out, dim, True), held(dim, out, True)
        g.fp8_quantize(weight, *self.w, block="square")
        g.fp8_quantize(weight, *self.w_turned, block="square", transpose=True)
        self.y, self.d = held(tokens, dim), held(tokens, out)
        self.y_turned, self.d_turned = along_tokens(dim), along_tokens(out)
        self.total, self.normed, self.d_normed = (torch.empty(tokens, dim, **BF16) for _ in range(3))
        self.rstd, self.c = torch.empty(tokens, device="cuda"), torch.empty(tokens, out, **BF16)
        self.d_weight = torch.empty(out, dim, **BF16)
        self.norm = g.RmsNormPlan(tokens, dim, "bf16", weight="f32")
        self.product = g.Fp8Plan(tokens, out, dim, "bf16")
        self.to_input = g.Fp8Plan(tokens, dim, out, "bf16")
        self.to_weight = g.Fp8Plan(out, dim, self.d_turned[0].shape[1], "bf16", b_scales="row")

    def forward(self, x, residual):
        self.norm.forward_fp8(x, self.gamma, *self.y, self.rstd, residual=residual, total=self.total)
        self.product.run(*self.y, *self.w, self.c)

    def backward(self, d_c):
        """d_normed and d_weight.  (The weight's gradient runs along the tokens: both operands are converted
        with scales along them, from 16 bits.)"""
        g.fp8_quantize(d_c, *self.d)
        self.to_input.run(*self.d, *self.w_turned, self.d_normed)
        self.norm.forward(self.total, self.gamma, self.normed)
        (d, d_tokens, d_scales), (y, y_tokens, y_scales) = self.d_turned, self.y_turned
        g.fp8_quantize(d_c, d_tokens, d_scales, transpose=True)
        g.fp8_quantize(self.normed, y_tokens, y_scales, transpose=True)
        self.to_weight.run(d, d_scales, y, y_scales, self.d_weight)

    def check(self):
        for plan in (self.product, self.to_input, self.to_weight):
            plan.check()

    def close(self):
        for plan in (self.norm, self.product, self.to_input, self.to_weight):
            plan.close()


def train(steps=20, rate=0.3, tokens=512, dim=256, seed=0):
    """The mean square of each step's distance from a fixed map of the input, by plain gradient descent."""
    block = Block(tokens, dim, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    goal = torch.randn(dim, dim, generator=gen, device="cuda") * dim ** -0.5
    nothing = torch.zeros(tokens, dim, **BF16)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, dim, generator=gen, device="cuda").bfloat16()
        block.forward(x, nothing)
        off = block.out.float() - x.float() @ goal
        losses.append(off.square().mean())
        block.backward((off * (2 / tokens)).bfloat16(), nothing)
        for name, d in block.grad.items():
            getattr(block, name).sub_(d.to(getattr(block, name).dtype), alpha=rate)
    block.check()
    block.close()
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    g.build_library()
    for n, value in enumerate(train(ap.parse_args().steps)):
        print("step %3d  mean square %.4f" % (n, value))
