"""An 8-bit projection and its gradients over numbers of tokens that are no multiple of 16."""
import os
import sys

import pytest
import torch

import ffn_oracle as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import ffn_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,dim,out", [(1, 128, 64), (15, 256, 144), (1000, 640, 512), (385, 1024, 256), (127, 128, 128)])
def test_weight_gradient_over_any_number_of_tokens(gemm_lib, tokens, dim, out):
    """The product of what the 8-bit matrices stand for, tokens alone, within the product's own bound; and the example's
    calls together with the formula (its bound is derived in test_ffn_step_gpu.py)."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    weight, x, residual, d_c = (r(out, dim) * dim ** -0.5).bfloat16(), r(tokens, dim).bfloat16(), r(tokens, dim).bfloat16(), r(tokens, out).bfloat16()
    layer = ffn_block.Projection(weight, tokens)
    layer.forward(x, residual)
    layer.backward(d_c)
    layer.check()
    want, bound = ref.fp8_product(layer.d_turned[1], layer.d_turned[2], layer.y_turned[1], layer.y_turned[2], False)
    assert ((layer.d_weight.double() - want).abs() <= bound + ref.rounded(want, "bf16") * 1.01).all()
    for whole, front, _ in (layer.d_turned, layer.y_turned):
        assert (whole.view(torch.uint8)[:, tokens:] == 0).all()
    full = d_c.double().t() @ layer.normed.double()
    assert float((layer.d_weight.double() - full).norm() / full.norm()) < 0.13
    layer.close()
