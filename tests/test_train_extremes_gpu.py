"""Distillation and layer norm at values far from one, where a formula's steps can leave fp32
although its result does not."""
import math

import numpy as np
import pytest
import torch

import test_train_ops_gpu as ops
import train_oracle as to

pytestmark = pytest.mark.gpu


# few and many short rows; rows in pieces, a cluster's each; the pipeline, by one block and by clusters; wide rows
SIZES = [(3, 40), (700, 40), (3, 9000), (700, 9000), (160, 66000), (1, 850000)]


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_distillation_of_shifted_rows(gemm_lib, rows, vocab, tau):
    """A number added to all of a row's logits changes its log-sum-exp alone.  The logits are multiples of 1/8, so they
    and the shift add exactly; the bounds are those of the rows before the shift."""
    tau = float(np.float32(tau))
    c = ops._distill_case(rows, vocab, 9, "f32", "f32", "i64", 0, 0, False, tau)
    near = torch.round(c["logits"] * 8) / 8
    c["logits"] = near
    args = (ops._f64(near), c["ids"].cpu().numpy(), ops._f64(c["values"]), tau)
    want = to.distill(*args, dloss=ops._f64(c["dloss"]))
    bound = to.distill_bounds(*args, "f32", dloss=ops._f64(c["dloss"]))
    with gemm_lib.DistillPlan(rows, vocab, 9, "f32") as plan:
        for shift in (0.0, 2.0 ** 20, -2.0 ** 20):
            far = near + shift
            far[near == -math.inf] = -math.inf
            for both in (False, True):
                c["loss"].fill_(7.0)
                if both:
                    plan.forward_backward(far, c["ids"], c["values"], c["loss"], c["lse"], c["dlogits"], dloss=c["dloss"],
                                          temperature=tau)
                    ops._within(c["dlogits"], want[2], bound[2], "dlogits of rows moved by %g" % shift)
                else:
                    plan.forward(far, c["ids"], c["values"], c["loss"], c["lse"], temperature=tau)
                ops._within(c["loss"], want[0], bound[0], "loss of rows moved by %g" % shift)
                ops._within(c["lse"], want[1] + shift / tau, bound[1] + 4 * to.U * abs(shift / tau),
                            "lse of rows moved by %g" % shift)


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("elem", ["f32", "bf16"])
@pytest.mark.parametrize("tau", [1.0, 0.5, 0.7, 30.0])
@pytest.mark.parametrize("level", [-1e9, -3e9, -1e10, -1e20, 1e15])
def test_distillation_of_level_rows(gemm_lib, rows, vocab, elem, tau, level):
    """Rows whose logits are all one large number (a mask that leaves nothing and is no infinity): uniform."""
    tau = float(np.float32(tau))
    ids, values = torch.tensor([[1, 5]], device="cuda").repeat(rows, 1), torch.zeros(rows, 2, device="cuda")
    loss, lse = torch.full((rows,), 7.0, device="cuda"), torch.empty(rows, device="cuda")
    logits = torch.full((rows, vocab), level, device="cuda").to(ops.TYPES[elem])
    level = float(logits[0, 0])
    grad = torch.full((rows, vocab), 7.0, device="cuda").to(ops.TYPES[elem])
    # p = 1/2 twice, q = 1 / vocab: some roundings of numbers up to the logarithms; the sum of vocab ones
    few = 64 * to.U + to.lanes(vocab)
    want = tau * tau * math.log(vocab / 2)
    q = torch.full((vocab,), 1.0 / vocab, device="cuda", dtype=torch.float64)
    q[[1, 5]] -= 0.5
    with gemm_lib.DistillPlan(rows, vocab, 2, elem) as plan:
        for both in (False, True):
            if both:
                plan.forward_backward(logits, ids, values, loss, lse, grad, temperature=tau)
                off = (grad.double() - tau * q).abs()
                assert bool((off <= tau * few * (1.0 / vocab + 0.5 * (q < 0)) + to.ROUND[elem] * tau * q.abs()).all())
            else:
                plan.forward(logits, ids, values, loss, lse, temperature=tau)
            assert bool(((loss - want).abs() <= few * tau * tau * (math.log(vocab) + 1)).all())
            assert bool(((lse - level / tau).abs() <= 4 * to.U * abs(level / tau) + math.log(vocab)).all())
        # log(vocab) is below the unit of such a log-sum-exp: what the gradient makes of it is finite
        plan.backward(logits, ids, values, lse, grad, temperature=tau)
        assert bool((grad.abs() <= tau).all())


@pytest.mark.parametrize("rows,vocab", [(3, 40), (3, 9000), (700, 9000), (700, 40)])
def test_distillation_limit_of_masks(gemm_lib, rows, vocab):
    """A logit below -1e30 times the temperature is a mask, one above it is a logit: a row that has only such
    ones is uniform.  (At this temperature the scale of the exponents is exactly one.)"""
    tau = float(np.float32(1.4426950408889634))
    kept, masked = -1.2e30, -1.5e30
    ids, values = torch.tensor([[1, 5]], device="cuda").repeat(rows, 1), torch.zeros(rows, 2, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    grad = torch.empty(rows, vocab, device="cuda")
    with gemm_lib.DistillPlan(rows, vocab, 2, "f32") as plan:
        for level in (kept, masked):
            logits = torch.full((rows, vocab), level, device="cuda")
            for both in (False, True):
                loss.fill_(7.0)
                grad.fill_(7.0)
                if both:
                    plan.forward_backward(logits, ids, values, loss, lse, grad, temperature=tau)
                else:
                    plan.forward(logits, ids, values, loss, lse, temperature=tau)
                if level == masked:
                    assert not bool(loss.any()) and bool((lse == -math.inf).all())
                    assert not both or not bool(grad.any())
                    continue
                # p = 1/2 twice, q = 1 / vocab: a few roundings of numbers up to log(vocab)
                want = tau * tau * math.log(vocab / 2)
                assert bool(((loss - want).abs() <= 64 * to.U * want).all())
                assert bool(((lse - kept / tau).abs() <= 4 * to.U * -kept).all())
                if both:
                    q = torch.full((vocab,), 1.0 / vocab, device="cuda", dtype=torch.float64)
                    q[[1, 5]] -= 0.5
                    assert bool(((grad.double() - tau * q).abs() <= 64 * to.U * (1.0 / vocab + 0.5 * (q < 0))).all())


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_distillation_of_shifted_teachers(gemm_lib, rows, vocab, tau):
    """A number added to all of a row's teacher values changes nothing where they add exactly (multiples of 1/8)."""
    tau = float(np.float32(tau))
    c = ops._distill_case(rows, vocab, 9, "f32", "f32", "i64", 0, 0, False, tau)
    near = torch.round(c["values"] * 8) / 8
    args = (ops._f64(c["logits"]), c["ids"].cpu().numpy(), ops._f64(near), tau)
    want = to.distill(*args, dloss=ops._f64(c["dloss"]))
    bound = to.distill_bounds(*args, "f32", dloss=ops._f64(c["dloss"]))
    with gemm_lib.DistillPlan(rows, vocab, 9, "f32") as plan:
        for shift in (0.0, 2.0 ** 20, -2.0 ** 20):
            more = {"temperature": tau}
            plan.forward(c["logits"], c["ids"], near + shift, c["loss"], c["lse"], **more)
            ops._within(c["loss"], want[0], bound[0], "loss of a teacher moved by %g" % shift)
            plan.backward(c["logits"], c["ids"], near + shift, c["lse"], c["dlogits"], dloss=c["dloss"], **more)
            ops._within(c["dlogits"], want[2], bound[2], "dlogits of a teacher moved by %g" % shift)
            plan.forward_backward(c["logits"], c["ids"], near + shift, c["loss"], c["lse"], c["dlogits"], dloss=c["dloss"], **more)
            ops._within(c["loss"], want[0], bound[0], "both: loss of a teacher moved by %g" % shift)
            ops._within(c["dlogits"], want[2], bound[2], "both: dlogits of a teacher moved by %g" % shift)


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("value,level", [("f32", -3.4028234663852886e38), ("f32", -1e10), ("bf16", -3e38), ("f16", -65504.0)])
@pytest.mark.parametrize("tau", [1.0, 0.7, 4.0])
def test_distillation_of_level_teachers(gemm_lib, rows, vocab, value, level, tau):
    """Only infinities have no mass: four entries of any one value, the type's lowest too, are 1/4 each."""
    tau = float(np.float32(tau))
    c = ops._distill_case(rows, vocab, 4, "f32", value, "i64", 0, 0, False, tau, mask=False)
    args = (ops._f64(c["logits"]), c["ids"].cpu().numpy(), np.zeros((rows, 4)), tau)
    want = to.distill(*args, dloss=ops._f64(c["dloss"]))
    bound = to.distill_bounds(*args, "f32", dloss=ops._f64(c["dloss"]))
    c["values"].fill_(level)
    with gemm_lib.DistillPlan(rows, vocab, 4, "f32") as plan:
        plan.forward_backward(c["logits"], c["ids"], c["values"], c["loss"], c["lse"], c["dlogits"], dloss=c["dloss"],
                              temperature=tau)
        ops._within(c["loss"], want[0], bound[0], "loss")
        ops._within(c["dlogits"], want[2], bound[2], "dlogits")


@pytest.mark.parametrize("rows,cols", [(5, 200), (3000, 333), (1300, 1024), (400, 8192), (320, 8200), (320, 12000), (320, 12003), (3, 17000)])
@pytest.mark.parametrize("elem", ["f32", "bf16"])
@pytest.mark.parametrize("exponent", [-76, 70])
def test_norm_of_small_and_large_rows(gemm_lib, rows, cols, elem, exponent):
    """Rows times a power of two, without eps: rstd is divided by it, and dx times rstd's change.  The square of either
    leaves fp32; neither result does.  The bounds are those of the scaled rows."""
    c = ops._norm_case(rows, cols, elem, "f32", 0, 0, seed=9)
    scale = 2.0 ** exponent
    c["x"][1] = torch.randn(cols, device="cuda").to(ops.TYPES[elem])     # (a row without variance has no norm without eps)
    c["x"].mul_(scale)
    c["dy"].mul_(2.0 ** -20)
    with gemm_lib.NormPlan(rows, cols, elem, weight="f32") as plan:
        x = c["x"].double()
        mean = x.mean(1)
        c["mean"].copy_(mean)
        c["rstd"].copy_(1 / (x - mean[:, None]).square().mean(1).sqrt())
        plan.backward(c["x"], c["gamma"], c["mean"], c["rstd"], c["dy"], c["dx"], c["dgamma"], c["dbeta"])
        args = (ops._f64(c["x"]), ops._f64(c["gamma"]), ops._f64(c["mean"]), ops._f64(c["rstd"]), ops._f64(c["dy"]))
        want, bound = to.norm_backward(*args), to.norm_backward_bounds(*args, elem, "f32")
        for k, name in enumerate(("dx", "dgamma", "dbeta")):
            ops._within(c[name], want[k], bound[k], name)
        plan.check()
