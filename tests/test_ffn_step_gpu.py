"""The feed-forward block's operators together, as the example runs them: against the same block and the same
projection in 64-bit torch autograd, in a CUDA graph, and what they report."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import ffn_block  # noqa: E402

pytestmark = pytest.mark.gpu


def _inputs(tokens, dim, seed, count):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(tokens, dim, generator=gen, device="cuda").bfloat16() for _ in range(count)]


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


def _norm(x, r, gamma):
    # (the sum is kept in bf16, and the norm is of what is kept)
    t = x.double() + r.double()
    t = t + (t.float().bfloat16().double() - t).detach()
    return t, t / torch.sqrt(t.square().mean(1, keepdim=True) + 1e-5) * gamma


@pytest.mark.parametrize("tokens,dim,inner", [(384, 128, 264), (100, 256, 704), (1, 512, 1000)])
def test_block_gradients(gemm_lib, tokens, dim, inner):
    """Results and gradients within 2.5 % of the 64-bit ones in the norm of the difference.  Tensors rounded to bf16 on
    the way (2^-9 each in the mean square, at most 2^-8): normed, h, both products kept for the gradients, d_h,
    d_products and d_normed, and the result's own rounding.  Six times 2^-8 is 2.4 %."""
    block = ffn_block.Block(tokens, dim, inner)
    x, r, d_out, d_total = _inputs(tokens, dim, 3, 4)
    block.gamma.uniform_(0.8, 1.2)
    block.forward(x, r)
    block.backward(d_out, d_total)
    block.check()
    w = {k: getattr(block, k).double().requires_grad_() for k in block.grad}
    xd = x.double().requires_grad_()
    t, y = _norm(xd, r, w["gamma"])
    g, u = (y @ w["gate_up"].t()).split(inner, 1)
    out = (torch.nn.functional.silu(g) * u) @ w["down"].t()
    ((out * d_out.double()).sum() + (t * d_total.double()).sum()).backward()
    assert torch.equal(block.total, t.detach().bfloat16())
    assert _off(block.out, out.detach()) < 0.025
    assert _off(block.d_x, xd.grad) < 0.025
    for name, d in block.grad.items():
        assert _off(d, w[name].grad) < 0.025, name
    block.close()


@pytest.mark.parametrize("tokens,dim,out", [(384, 256, 512), (48, 640, 144), (16, 1024, 2048)])
def test_projection_gradients(gemm_lib, tokens, dim, out):
    """Within 13 % in the norm of the difference: both operands of a product are rounded to e4m3, by at most 2^-4 of a
    value each (6.25 %; 2.6 % in the mean square), and a result of independent terms is off by no more than its
    operands together; bf16 roundings and values below the smallest normal add less than 1 %."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    weight = (torch.randn(out, dim, generator=gen, device="cuda") * dim ** -0.5).bfloat16()
    layer = ffn_block.Projection(weight, tokens)
    x, r = _inputs(tokens, dim, 6, 2)
    d_c = _inputs(tokens, out, 7, 1)[0]
    layer.forward(x, r)
    layer.backward(d_c)
    layer.check()
    w = weight.double().requires_grad_()
    y = _norm(x, r, 1.0)[1].requires_grad_()
    c = y @ w.t()
    (c * d_c.double()).sum().backward()
    assert _off(layer.c, c.detach()) < 0.13
    assert _off(layer.d_normed, y.grad) < 0.13
    assert _off(layer.d_weight, w.grad) < 0.13
    layer.close()


def test_a_captured_step_repeats_itself(gemm_lib):
    block, layer = ffn_block.Block(200, 256, 320), None
    x, r, d_out, d_total = _inputs(200, 256, 8, 4)
    layer = ffn_block.Projection(block.gate_up, 200 - 200 % 16)
    outs = [block.out, block.d_x, layer.c, layer.d_weight, *block.grad.values()]

    def step():
        block.forward(x, r)
        block.backward(d_out, d_total)
        layer.forward(block.out[:192], block.total[:192])
        layer.backward(block.products[:192])
    step()
    torch.cuda.synchronize()
    want = [v.clone() for v in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for v in outs:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(v, w) for v, w in zip(outs, want))
    block.check()
    layer.check()
    block.close()
    layer.close()


def test_block_reports_a_wait_that_ran_out(gemm_lib):
    block = ffn_block.Block(300, 512, 1024)
    x, r, d_out, d_total = _inputs(300, 512, 9, 4)
    block.forward(x, r)
    block.check()
    want = block.out.clone()
    block.gated.set_timeout(20_000_000)
    block.gated.set_wait_test(16)
    block.forward(x, r)
    with pytest.raises(gemm_lib.GemmError) as e:
        block.check()
    assert e.value.status == 9
    block.gated.set_wait_test(0)
    block.gated.set_timeout(0)
    block.forward(x, r)
    block.check()
    assert torch.equal(block.out, want)
    block.close()


def test_training_runs(gemm_lib):
    losses = ffn_block.train(steps=10)
    assert len(losses) == 10 and all(v == v and v < float("inf") for v in losses)
