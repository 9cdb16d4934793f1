"""The 64-bit definitions against differences of themselves and against closed forms (no GPU)."""
import numpy as np
import pytest

import train_oracle as to


def _difference(f, x, direction, h=1e-5):
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


def test_norm_gradient_is_the_derivative():
    rng = np.random.default_rng(1)
    x, dy = rng.normal(size=(3, 17)), rng.normal(size=(3, 17))
    gamma, beta, eps = rng.normal(size=17), rng.normal(size=17), 1e-3
    _, mean, rstd = to.norm_forward(x, gamma, beta, eps)
    dx, dgamma, dbeta = to.norm_backward(x, gamma, mean, rstd, dy)
    for _ in range(5):
        d = rng.normal(size=x.shape)
        assert abs(_difference(lambda v: (to.norm_forward(v, gamma, beta, eps)[0] * dy).sum(), x, d) - (dx * d).sum()) < 1e-7
        w = rng.normal(size=17)
        assert abs(_difference(lambda v: (to.norm_forward(x, v, beta, eps)[0] * dy).sum(), gamma, w) - (dgamma * w).sum()) < 1e-7
        assert abs(_difference(lambda v: (to.norm_forward(x, gamma, v, eps)[0] * dy).sum(), beta, w) - (dbeta * w).sum()) < 1e-7


def test_embedding_gradient_is_the_derivative():
    rng = np.random.default_rng(2)
    ids = np.array([3, 0, 3, 5, 1, 3, 5])
    table, dout = rng.normal(size=(6, 4)), rng.normal(size=(7, 4))
    grad, _ = to.embed_backward(ids, 1, dout, 2.5, 6)
    d = rng.normal(size=table.shape)
    assert abs(_difference(lambda w: (to.embed_forward(ids, 1, w, 2.5) * dout).sum(), table, d) - (grad * d).sum()) < 1e-8
    assert not grad[1].any() and not grad[2].any() and not grad[4].any()


@pytest.mark.parametrize("tau", [1.0, 2.5])
@pytest.mark.parametrize("given", [False, True])
def test_distillation_gradient_is_the_derivative(tau, given):
    rng = np.random.default_rng(3)
    logits, values = rng.normal(size=(4, 11)), rng.normal(size=(4, 3)) + 2
    ids = np.array([[1, 5, 7], [2, -1, 2], [-1, -1, -1], [10, 0, -1]])
    lse = rng.normal(size=4) + 5 if given else None
    dloss = rng.uniform(0.5, 2, size=4)
    f = lambda s: (to.distill(s, ids, values, tau, lse)[0] * dloss).sum()  # noqa: E731
    grad = to.distill(logits, ids, values, tau, lse, dloss)[2]
    for _ in range(5):
        d = rng.normal(size=logits.shape)
        assert abs(_difference(f, logits, d) - (grad * d).sum()) < 1e-8
    assert not grad[2].any()


def test_distillation_of_the_whole_vocabulary_is_the_divergence():
    """With every token among the entries the loss is KL(teacher || student), zero for equal logits."""
    rng = np.random.default_rng(4)
    logits, values = rng.normal(size=(2, 6)), rng.normal(size=(2, 6))
    ids = np.tile(np.arange(6), (2, 1))
    p = np.exp(values) / np.exp(values).sum(1, keepdims=True)
    q = np.exp(logits) / np.exp(logits).sum(1, keepdims=True)
    loss, _, grad = to.distill(logits, ids, values, 1.0)
    assert np.allclose(loss, (p * np.log(p / q)).sum(1)) and np.allclose(grad, q - p)
    assert np.allclose(to.distill(values, ids, values, 3.0)[0], 0)


def test_left_out_rows():
    logits = np.array([[0.0, 1.0], [-np.inf, -np.inf], [0.0, -np.inf]])
    ids, values = np.array([[-1], [0], [0]]), np.array([[1.0], [1.0], [-np.inf]])
    loss, lse, grad = to.distill(logits, ids, values, 1.0)
    assert not loss.any() and not grad.any() and (lse == -np.inf).all()


@pytest.mark.parametrize("planted", ["no mean term", "no hat term", "one term less"])
def test_bounds_find_planted_mistakes(planted):
    """A gradient with a term left out is outside the bounds that the kernels are held to."""
    rng = np.random.default_rng(5)
    x, dy, gamma = rng.normal(size=(64, 96)), rng.normal(size=(64, 96)), rng.normal(size=96)
    _, mean, rstd = to.norm_forward(x, gamma, np.zeros(96), 1e-5)
    hat, g = (x - mean[:, None]) * rstd[:, None], dy * gamma
    dx, dgamma, _ = to.norm_backward(x, gamma, mean, rstd, dy)
    bx, bg, _ = to.norm_backward_bounds(x, gamma, mean, rstd, dy, "bf16", "f32")
    if planted == "no mean term":
        assert (np.abs(dx - rstd[:, None] * (g - hat * (g * hat).mean(1, keepdims=True))) > bx).any()
    elif planted == "no hat term":
        assert (np.abs(dx - rstd[:, None] * (g - g.mean(1, keepdims=True))) > bx).any()
    else:
        assert (np.abs(dgamma - (dy * hat)[1:].sum(0)) > bg).all()
