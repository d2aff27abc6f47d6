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


def test_bf16_rounding():
    v = np.array([1.0, 1.00390625, 1.01171875, -3.14159, 0.0, 1e-30], np.float32)
    import torch
    assert np.array_equal(T.bf16(v), torch.from_numpy(v).bfloat16().float().numpy())
