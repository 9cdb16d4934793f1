"""The norm's numbers do not depend on where its results go: inputs on the 16-byte boundaries, results on and off them."""
import pytest
import torch

import ffn_oracle as ref

pytestmark = pytest.mark.gpu
T = ref.TYPES
FP8 = torch.float8_e4m3fn


def _room(rows, cols, first, pad, dtype):
    """A matrix `first` elements behind a boundary, its rows `pad` elements apart, and its buffer, of sevens."""
    whole = torch.full((first + rows * (cols + pad) + 8,), 7.0, device="cuda").to(dtype)
    return whole.as_strided((rows, cols), (cols + pad, 1), first), whole


def _bits(t):
    return t.contiguous().view(torch.uint8)


def _only_in(m, whole):
    """Whether nothing but the matrix was written."""
    m.copy_(torch.full((), 7.0, device="cuda").to(m.dtype))
    return bool((whole.float() == 7).all())


@pytest.mark.parametrize("cols", [8, 64, 1000, 2048, 4096, 5120, 8192, 12288, 16384, 16392, 20000])
@pytest.mark.parametrize("elem,weight", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_results_off_the_boundaries_have_the_same_bits(gemm_lib, cols, elem, weight):
    rows = 331 if cols < 5000 else 170
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, r, dy, dt = (torch.randn(rows, cols, generator=g, device="cuda").to(T[elem]) for _ in range(4))
    gamma = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(T[weight])
    total, y, dx = (torch.empty_like(x) for _ in range(3))
    rstd, rstd2 = (torch.empty(rows, device="cuda") for _ in range(2))
    dgamma, dgamma2 = torch.empty_like(gamma), torch.empty_like(gamma)
    groups = ref.groups(cols)
    q, scales = torch.empty(rows, cols, dtype=FP8, device="cuda"), torch.empty(rows, groups, device="cuda")
    with gemm_lib.RmsNormPlan(rows, cols, elem, weight=weight) as plan:
        for residual in (r, None):
            plan.forward(x, gamma, y, rstd, residual=residual, total=total)
            plan.forward_fp8(x, gamma, q, scales, residual=residual)
            plan.backward(total, gamma, rstd, dy, dx, dgamma, dtotal=residual)
            for first, pad in ((1, 0), (0, 3), (3, 5), (4, 8)):
                (t2, t_all), (y2, y_all), (dx2, dx_all) = (_room(rows, cols, first, pad, T[elem]) for _ in range(3))
                q2, q_all = _room(rows, cols, first, pad, FP8)
                s2, s_all = _room(rows, groups, first, pad, torch.float32)
                # each result alone off the boundaries, then all of them
                plan.forward(x, gamma, y2, rstd2, residual=residual, total=torch.empty_like(total))
                assert torch.equal(rstd, rstd2) and torch.equal(_bits(y), _bits(y2))
                y3 = torch.empty_like(y)
                plan.forward(x, gamma, y3, rstd2, residual=residual, total=t2)
                assert torch.equal(rstd, rstd2) and torch.equal(_bits(y), _bits(y3)) and torch.equal(_bits(total), _bits(t2))
                t2.zero_()
                y2.zero_()
                plan.forward(x, gamma, y2, rstd2, residual=residual, total=t2)
                assert torch.equal(rstd, rstd2) and torch.equal(_bits(y), _bits(y2)) and torch.equal(_bits(total), _bits(t2))
                t2.zero_()
                plan.forward_fp8(x, gamma, q2, s2, rstd2, residual=residual, total=t2)
                assert torch.equal(rstd, rstd2) and torch.equal(_bits(q), _bits(q2)) and torch.equal(scales, s2)
                assert torch.equal(_bits(total), _bits(t2))
                plan.backward(total, gamma, rstd, dy, dx2, dgamma2, dtotal=residual)
                assert torch.equal(_bits(dx), _bits(dx2)) and torch.equal(dgamma, dgamma2)
                plan.backward(total, gamma, rstd, dy, None, dgamma2, dtotal=residual)
                assert torch.equal(dgamma, dgamma2)
                assert all(_only_in(*v) for v in ((t2, t_all), (y2, y_all), (dx2, dx_all), (q2, q_all), (s2, s_all)))
