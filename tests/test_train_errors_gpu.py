"""What the plans of the operators report, whatever else the GPU is doing."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["embed", "distill"])
def test_errors_of_a_plan_made_while_the_default_stream_is_busy(gemm_lib, kind):
    """The plan's error word is cleared when the plan is made, not when the default stream comes to it."""
    g = gemm_lib
    ids = torch.tensor([1, 2, 100, 3], device="cuda")
    table, out = torch.randn(100, 64, device="cuda"), torch.empty(4, 64, device="cuda")
    loss, lse = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    values = torch.ones(4, 1, device="cuda")

    def make():
        return g.EmbedPlan(100, 64, 4, "f32") if kind == "embed" else g.DistillPlan(4, 64, 1, "f32")

    def call(plan, stream):
        if kind == "embed":
            plan.forward(ids, table, out, stream=stream)
        else:
            plan.forward(out, ids[:, None], values, loss, lse, stream=stream)

    side = torch.cuda.Stream()
    with make() as plan:                             # (what a first call loads is loaded)
        call(plan, side)
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)               # about a tenth of a second
        with make() as late:
            call(late, side)
            side.synchronize()
            torch.cuda.synchronize()
            with pytest.raises(g.GemmError) as e:
                late.check(side)
            assert e.value.status == 12
            late.check(side)                         # reported once


@pytest.mark.parametrize("temperature", [float("inf"), float("nan"), 0.0, -1.0, 1e-40])
@pytest.mark.parametrize("call", ["forward", "backward", "forward_backward"])
def test_temperatures_that_are_no_normal_numbers_are_refused(gemm_lib, temperature, call):
    x, w = torch.zeros(4, 64, device="cuda"), torch.zeros(4, device="cuda")
    ids, values = torch.zeros(4, 3, dtype=torch.int64, device="cuda"), torch.zeros(4, 3, device="cuda")
    args = {"forward": (x, ids, values, w, w), "backward": (x, ids, values, w, x), "forward_backward": (x, ids, values, w, w, x)}
    with gemm_lib.DistillPlan(4, 64, 3, "f32") as plan:
        with pytest.raises(gemm_lib.GemmError) as e:
            getattr(plan, call)(*args[call], temperature=temperature)
        assert e.value.status == 1
    torch.cuda.synchronize()
    assert not bool(x.any()) and not bool(w.any())
