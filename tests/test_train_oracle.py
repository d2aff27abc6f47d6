"""The oracle of the node-side operators against differences (CPU): every
gradient it gives is the derivative of the forward it gives."""
import numpy as np
import pytest

from tests import train_oracle as T


def _directional(f, v, d, h=1e-5):
    return (f(v + h * d) - f(v - h * d)) / (2 * h)


def test_embed_gradient_against_differences():
    rng = np.random.default_rng(0)
    ids = np.array([3, 0, -1, 3, 7, 2, 3, 9])
    table, g = rng.standard_normal((8, 5)), rng.standard_normal((8, 5))
    d = rng.standard_normal(table.shape)
    want = _directional(lambda t: (g * T.embed_fwd(ids, t, 1.5)).sum(), table, d)
    assert np.isclose((T.embed_bwd(ids, g, 8, 1.5) * d).sum(), want, rtol=1e-8)


@pytest.mark.parametrize("kind", ["none", "silu", "tanh"])
def test_norm_gradients_against_differences(kind):
    rng = np.random.default_rng(1)
    ptr, groups, C = np.array([0, 4, 4, 5, 11]), 3, 12
    x, gamma, beta, g = (rng.standard_normal(s) for s in ((11, C), C, C, (11, C)))
    grads = T.norm_bwd(x, gamma, beta, g, ptr, groups, 1e-3, kind)
    for k, (v, got) in enumerate(zip((x, gamma, beta), grads)):
        d = rng.standard_normal(v.shape)
        args = [x, gamma, beta]

        def f(w):
            args[k] = w
            return (g * T.norm_fwd(*args, ptr, groups, 1e-3, kind)[0]).sum()

        assert np.isclose((got * d).sum(), _directional(f, v, d), rtol=1e-6), k


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (1, 4), (6, 6)])
def test_orthogonalize_is_the_matrix_iteration(shape):
    """The singular-value form equals the iteration by matrix products."""
    rng = np.random.default_rng(4)
    G, (a, b, c) = rng.standard_normal(shape), (3.4445, -4.7750, 2.0315)
    X = G / (np.linalg.norm(G) + 1e-7)
    for _ in range(5):
        A = X @ X.T
        X = a * X + (b * A + c * A @ A) @ X
    got, norms = T.orthogonalize(G, 5, (a, b, c), 1e-7, 2.0)
    assert np.allclose(got, 2.0 * X, rtol=1e-10, atol=1e-10)
    assert np.isclose(norms[-1], np.linalg.norm(X))
    # a cubic that converges gives the nearest orthogonal matrix
    U, _, Vt = np.linalg.svd(G, full_matrices=False)
    assert np.allclose(T.orthogonalize(G, 60, (1.5, -0.5, 0.0), 0.0, 1.0)[0], U @ Vt, atol=1e-9)


def test_bf16_rounding():
    v = np.array([1.0, 1.00390625, 1.01171875, -3.14159, 0.0, 1e-30], np.float32)
    import torch
    assert np.array_equal(T.bf16(v), torch.from_numpy(v).bfloat16().float().numpy())
