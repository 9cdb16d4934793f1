"""The operators and the products together: the example's student against the same student
in 64-bit torch autograd, and its training."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import distill_head  # noqa: E402

pytestmark = pytest.mark.gpu


def _reference(student, ids, top_ids, values, weights):
    m = {k: v.double().requires_grad_() for k, v in student.master.items()}
    # the kernels take bf16 copies of these two
    table = m["table"] + (student.table.double() - m["table"]).detach()
    head = (m["head"] + (student.head.double() - m["head"]).detach())[:student.vocab]
    hidden = table[ids] * student.scale
    normed = torch.nn.functional.layer_norm(hidden, hidden.shape[1:], m["gamma"], m["beta"], 1e-5)
    tau = student.temperature
    logq = torch.log_softmax(normed @ head.T / tau, 1).gather(1, top_ids)
    p = torch.softmax(values.double() / tau, 1)
    loss = tau * tau * (p * (p.log() - logq)).sum(1)
    (loss * weights.double()).sum().backward()
    return loss.detach(), {k: v.grad for k, v in m.items()}


def test_step_gradients(gemm_lib):
    """Every gradient within 2 % of the 64-bit one in the norm of the difference.  Five tensors on the way are
    rounded to bf16 (2^-9 each in the mean square, at most 2^-8): hidden, normed, logits, the logits' gradient
    and normed's; logits of size ~1 moved by 2^-9 move the probabilities by as much.  Five times 2^-8 is 2 %."""
    student = distill_head.Student(tokens=384, vocab=1003, dim=128)
    gen = torch.Generator(device="cuda").manual_seed(4)
    ids, top_ids, values = distill_head.batch(384, 1003, 16, gen)
    weights = torch.rand(384, generator=gen, device="cuda") / 384
    student.gradients(ids, top_ids, values, weights)
    student.check()
    loss, want = _reference(student, ids, top_ids, values, weights)
    assert float((student.loss.double() - loss).norm() / loss.norm()) < 0.02
    for name, w in want.items():
        off = float((student.grad[name].double() - w).norm() / w.norm())
        assert off < 0.02, (name, off)
    student.close()


def test_training_lowers_the_loss(gemm_lib):
    losses = distill_head.train(steps=40)
    assert losses[-1] < 0.5 * losses[0], losses
