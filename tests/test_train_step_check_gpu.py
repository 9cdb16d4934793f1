"""What the example's student reports of its plans."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import distill_head  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["norm", "distill"])
def test_student_reports_waits_that_ran_out(gemm_lib, name):
    import torch
    student = distill_head.Student(tokens=1536, vocab=5003, dim=1024)
    gen = torch.Generator(device="cuda").manual_seed(4)
    args = (*distill_head.batch(1536, 5003, 16, gen), torch.full((1536,), 1.0 / 1536, device="cuda"))
    student.gradients(*args)
    student.check()
    plan = getattr(student, name)
    plan.set_timeout(20_000_000)
    plan.set_wait_test(16)
    student.gradients(*args)
    with pytest.raises(gemm_lib.GemmError) as e:
        student.check()
    assert e.value.status == 9
    plan.set_wait_test(0)
    plan.set_timeout(0)
    student.gradients(*args)
    student.check()
    assert bool(torch.isfinite(student.loss).all())
    student.close()
