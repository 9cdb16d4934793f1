"""A student's training steps from a teacher's top logits, on the library's kernels alone:

    tokens -> embedding (EmbedPlan) -> layer norm (NormPlan) -> head product (Plan, TN)
           -> distillation loss and its gradient (DistillPlan, one call)
           -> the product's gradients (Plan NN for its input, Plan NT for its weight)
           -> norm's gradients -> the embedding table's gradient, all written into kept buffers.

The vocabulary is not a multiple of 8: the head has a few more rows, and the logits' rows
are as wide; the loss works on the first `vocab` columns in place.  The optimiser is plain
gradient descent on 32-bit weights, of which the products take bf16 copies.

    python examples/distill_head.py [--steps 40]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_hgemm_gb300 as g  # noqa: E402


class Student:
    """Weights, buffers and plans of one batch size."""

    def __init__(self, tokens=512, vocab=1003, dim=256, top=16, temperature=2.0, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.temperature, self.scale = vocab, temperature, dim ** 0.5
        wide = -(-vocab // 8) * 8                       # the head's rows, with the padding
        bf16 = {"dtype": torch.bfloat16, "device": "cuda"}

        def weight(*shape, std=0.02):
            return torch.randn(*shape, generator=gen, device="cuda") * std
        self.master = {"table": weight(vocab, dim), "gamma": torch.ones(dim, device="cuda"),
                       "beta": torch.zeros(dim, device="cuda"), "head": weight(wide, dim)}
        self.grad = {k: torch.zeros_like(v) for k, v in self.master.items() if k != "head"}
        self.grad["head"] = torch.zeros(wide, dim, **bf16)
        self.table, self.head = (self.master[k].to(torch.bfloat16) for k in ("table", "head"))
        self.hidden, self.normed, self.d_hidden, self.d_normed = (torch.empty(tokens, dim, **bf16) for _ in range(4))
        self.logits, self.d_logits = (torch.zeros(tokens, wide, **bf16) for _ in range(2))
        self.mean, self.rstd, self.loss, self.lse = (torch.empty(tokens, device="cuda") for _ in range(4))
        self.embed = g.EmbedPlan(vocab, dim, tokens, "bf16", grad="f32")
        self.norm = g.NormPlan(tokens, dim, "bf16", weight="f32")
        self.distill = g.DistillPlan(tokens, vocab, top, "bf16")
        self.product = g.Plan(tokens, wide, dim, "bf16", layout="TN")        # logits = normed . head^T
        self.to_input = g.Plan(tokens, dim, wide, "bf16", layout="NN")       # d_normed = d_logits . head
        self.to_weight = g.Plan(wide, dim, tokens, "bf16", layout="NT")      # d_head = d_logits^T . normed

    def gradients(self, ids, top_ids, top_values, weights):
        """The loss of each token in self.loss, the gradients of sum(weights * loss) in self.grad."""
        m, d = self.master, self.grad
        self.embed.forward(ids, self.table, self.hidden, scale=self.scale)
        self.norm.forward(self.hidden, m["gamma"], m["beta"], self.normed, self.mean, self.rstd)
        self.product.run(self.normed, self.head, self.logits)
        self.distill.forward_backward(self.logits[:, :self.vocab], top_ids, top_values, self.loss, self.lse,
                                      self.d_logits[:, :self.vocab], dloss=weights, temperature=self.temperature)
        self.to_input.run(self.d_logits, self.head, self.d_normed)
        self.to_weight.run(self.d_logits, self.normed, d["head"])
        self.norm.backward(self.hidden, m["gamma"], self.mean, self.rstd, self.d_normed, self.d_hidden, d["gamma"],
                           d["beta"])
        self.embed.backward(ids, self.d_hidden, d["table"], scale=self.scale)

    def step(self, rate):
        for k, w in self.master.items():
            w.sub_(self.grad[k], alpha=rate)
        self.table.copy_(self.master["table"])
        self.head.copy_(self.master["head"])

    def check(self):
        """Raises what the kernels have to report."""
        for plan in (self.embed, self.norm, self.distill, self.product, self.to_input, self.to_weight):
            plan.check()

    def close(self):
        for plan in (self.embed, self.norm, self.distill, self.product, self.to_input, self.to_weight):
            plan.close()


def batch(tokens, vocab, top, gen):
    """Token ids and what a teacher would say of each: entries that depend on the token alone."""
    ids = torch.randint(vocab, (tokens,), generator=gen, device="cuda")
    at = torch.arange(top, device="cuda")
    return ids, (ids[:, None] * 31 + at * at + 7 * at) % vocab, (3.0 - 0.4 * at).expand(tokens, top).contiguous()


def train(steps=40, rate=20.0, tokens=512, vocab=1003, dim=256, top=16, seed=0):
    """The mean loss of each step."""
    student = Student(tokens, vocab, dim, top, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    weights = torch.full((tokens,), 1.0 / tokens, device="cuda")
    losses = []
    for _ in range(steps):
        student.gradients(*batch(tokens, vocab, top, gen), weights)
        student.step(rate)
        losses.append(student.loss.mean())
    student.check()
    student.close()
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    g.build_library()
    for n, value in enumerate(train(ap.parse_args().steps)):
        if n % 5 == 0:
            print("step %3d  loss %.4f" % (n, value))
