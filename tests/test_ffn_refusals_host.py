"""Calls without a tensor, or with one of other dimensions, raise GemmError (no GPU needed)."""
import pytest
import torch


def _plan(cls, **fields):
    """A plan of the class without its C handle: its calls stop at the arguments."""
    plan = object.__new__(cls)
    plan.handle = None
    for name, value in fields.items():
        setattr(plan, name, value)
    return plan


def test_missing_tensors_and_other_dimensions(gemm_lib):
    ffn, elem = gemm_lib.ffn, gemm_lib.ELEMS["bf16"]
    gemm_lib.train._torch_types()
    m, scalar, rows = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros((), dtype=torch.bfloat16), torch.zeros(3)
    norm = _plan(ffn.RmsNormPlan, max_rows=4, cols=8, _elem=elem, _weight=elem, _enter_forward=None, _enter_fp8=None,
                 _enter_backward=None)
    product = _plan(ffn.Fp8Plan, M=4, N=8, K=16, _elem=elem, _scales=1, _enter_run=None)
    for bad in (None, scalar, rows, torch.zeros(2, 2, 2)):
        for call in (lambda: norm.forward(bad, None, m), lambda: norm.forward_fp8(bad, None, m, m),
                     lambda: norm.backward(bad, None, None, m), lambda: ffn.fp8_quantize(bad, m, m)):
            with pytest.raises(gemm_lib.GemmError) as e:
                call()
            assert e.value.status == 1
    for call in (lambda: norm.forward(m, None, None), lambda: norm.forward_fp8(m, None, None, None),
                 lambda: norm.backward(m, None, None, None), lambda: product.run(None, None, None, None, None)):
        with pytest.raises(gemm_lib.GemmError) as e:
            call()
        assert e.value.status == 1
