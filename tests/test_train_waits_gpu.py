"""Waits that run out in the operators' kernels, without faulting or hanging the GPU.

A plan's wait-test hook makes copies wait for bytes that never come; with a limit of 20 ms the
bounded waits run out, the kernel lets its own copies land (bounded as well) and returns, and the
plan's check reports GEMM_ERR_DEVICE_TIMEOUT.  The same plan then computes a right result."""
import time

import pytest

import test_train_ops_gpu as ops

pytestmark = pytest.mark.gpu

LIMIT = 20_000_000       # ns


def _times_out(gemm_lib, plan, call):
    call()
    with pytest.raises(gemm_lib.GemmError) as e:
        plan.check()
    assert e.value.status == 9
    plan.check()                         # reported once


def _distill_calls(plan, c):
    return {"forward": lambda: plan.forward(c["logits"], c["ids"], c["values"], c["loss"], c["lse"]),
            "backward": lambda: plan.backward(c["logits"], c["ids"], c["values"], c["lse"], c["dlogits"], dloss=c["dloss"]),
            "both": lambda: plan.forward_backward(c["logits"], c["ids"], c["values"], c["loss"], c["lse"], c["dlogits"],
                                                  dloss=c["dloss"])}


@pytest.mark.parametrize("rows,vocab,elem", [(1, 4200, "bf16"), (3, 20011, "f32"), (5, 50000, "bf16"), (40, 9001, "f16")])
@pytest.mark.parametrize("name", ["forward", "backward", "both"])
@pytest.mark.parametrize("every", [1, 2])
def test_distillation_of_few_rows(gemm_lib, rows, vocab, elem, name, every):
    """Rows by one block per piece (two to eight), which share a row in a cluster: all of the blocks, or every second."""
    c = ops._distill_case(rows, vocab, 9, elem, "f32", "i64", 0, 0, False, 1.0)
    with gemm_lib.DistillPlan(rows, vocab, 9, elem) as plan:
        calls = _distill_calls(plan, c)
        calls["forward"]()
        plan.set_timeout(LIMIT)
        plan.set_wait_test(16, every)
        _times_out(gemm_lib, plan, calls[name])
        plan.set_wait_test(0)
        plan.set_timeout(0)
        calls["forward"]()
        calls["backward"]()
        ops._check_distill(c, elem, 1.0)
        calls["both"]()
        ops._check_distill(c, elem, 1.0, what="both: ")
        plan.check()


@pytest.mark.parametrize("rows,vocab,elem", [(700, 9001, "f32"), (480, 20011, "bf16"), (200, 40000, "f16"), (160, 66000, "bf16"),
                                             (330, 70000, "f32"), (90, 150000, "bf16")])
@pytest.mark.parametrize("name", ["forward", "both"])
@pytest.mark.parametrize("every", [1, 2, 5])
def test_distillation_pipeline(gemm_lib, rows, vocab, elem, name, every):
    """Many rows, many of them without entries, by one block or by a cluster each: the waits of all blocks, or those of
    some of a cluster's blocks, run out; then the others wait for their numbers in vain."""
    c = ops._distill_case(rows, vocab, 9, elem, "f32", "i64", 0, 0, False, 1.0)
    c["ids"][::3] = -1
    with gemm_lib.DistillPlan(rows, vocab, 9, elem) as plan:
        calls = _distill_calls(plan, c)
        calls[name]()
        plan.check()
        plan.set_timeout(LIMIT)
        plan.set_wait_test(16, every)
        began = time.perf_counter()
        _times_out(gemm_lib, plan, calls[name])
        # a wait or two of each block, one of the next, and what is left behind: each 20 ms at most
        assert time.perf_counter() - began < 2.0
        plan.set_wait_test(0)
        plan.set_timeout(0)
        calls["forward"]()
        calls["backward"]()
        ops._check_distill(c, elem, 1.0)
        calls["both"]()
        ops._check_distill(c, elem, 1.0, what="both: ")
        plan.check()


@pytest.mark.parametrize("rows,cols,elem,weight", [
    (1300, 4096, "bf16", "f32"), (5200, 1000, "f16", "f16"), (1301, 4090, "bf16", "bf16"), (3000, 333, "f32", "f32"),
    (650, 12000, "bf16", "bf16"), (320, 16384, "f16", "f16")])
@pytest.mark.parametrize("name", ["forward", "backward"])
@pytest.mark.parametrize("every", [1, 7])
def test_norm_rings(gemm_lib, rows, cols, elem, weight, name, every):
    """Rings of whole rows, of rows off the boundaries in packs and in single elements, and of wide rows."""
    c = ops._norm_case(rows, cols, elem, weight, 0, 0)
    with gemm_lib.NormPlan(rows, cols, elem, weight=weight) as plan:
        calls = {"forward": lambda: plan.forward(c["x"], c["gamma"], c["beta"], c["y"], c["mean"], c["rstd"]),
                 "backward": lambda: plan.backward(c["x"], c["gamma"], c["mean"], c["rstd"], c["dy"], c["dx"], c["dgamma"],
                                                   c["dbeta"])}
        calls["forward"]()
        plan.check()
        plan.set_timeout(LIMIT)
        plan.set_wait_test(16, every)
        began = time.perf_counter()
        _times_out(gemm_lib, plan, calls[name])
        assert time.perf_counter() - began < 2.0
        plan.set_wait_test(0)
        plan.set_timeout(0)
        calls["forward"]()
        calls["backward"]()
        ops._check_norm(c, elem, weight)
        plan.check()


@pytest.mark.parametrize("make", [lambda g: g.DistillPlan(4, 5000, 3, "f32"), lambda g: g.NormPlan(4, 5000, "f32")])
def test_wait_test_hook_validates(gemm_lib, make):
    with make(gemm_lib) as plan:
        for bad in ((7, 1), (8192, 1), (16, 0)):
            with pytest.raises(gemm_lib.GemmError) as e:
                plan.set_wait_test(*bad)
            assert e.value.status == 1
