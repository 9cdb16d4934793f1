"""NULL handles of the plans' further functions (no GPU needed)."""


def test_null_handles_of_checks_and_hooks(gemm_lib):
    lib = gemm_lib.library()
    for kind in ("norm", "embed", "distill"):
        assert getattr(lib, "gemm_%s_plan_check" % kind)(None, None) == 1
    for kind in ("norm", "distill"):
        assert getattr(lib, "gemm_%s_plan_set_timeout" % kind)(None, 1) == 1
        assert getattr(lib, "gemm_%s_plan_set_wait_test" % kind)(None, 16, 1) == 1
