"""The training example: its parameters' gradients are the derivatives of its
loss, and training lowers the loss."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.fixture(scope="module")
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, EXAMPLES)
    try:
        import train_potential
    finally:
        sys.path.remove(EXAMPLES)
    return torch, train_potential


def test_gradients_against_differences(example):
    """The whole chain (embedding, convolution, mixing, normalisation) against
    central differences of its fp32 loss.  A step h along a direction of norm
    |d| changes a loss of order 1 by h <g, d>: rounding (about 1e-6 of the loss,
    divided by 2 h) and the third-order term (about h^2) stay below 1e-2 of the
    gradient's scale at h = 1e-2."""
    torch, ex = example
    dev = torch.device("cuda:0")
    b = ex.batch(12, 3, dev)
    model = ex.Potential(32, 48, 6, dev, seed=2)
    model.params["gamma"].add_(0.1 * torch.randn_like(model.params["gamma"]))

    def loss():
        return float(((model.forward(b)[0] - b["energy"]).double() ** 2).mean())

    energy, kept = model.forward(b)
    error = energy - b["energy"]
    grads = model.backward(b, 2 * error / error.numel(), kept)
    for name, g in grads.items():
        d = g / g.norm()                     # the steepest direction: the derivative is |g|
        w = model.params[name]
        at, h = w.clone(), 1e-2
        w.copy_(at + h * d)
        up = loss()
        w.copy_(at - h * d)
        down = loss()
        w.copy_(at)
        want = float(g.double().norm())
        got = (up - down) / (2 * h)
        print(f"[example] {name}: |g| {want:.5f}, by differences {got:.5f}", flush=True)
        assert abs(got - want) <= 1e-2 * max(want, 1.0), name


def test_training_lowers_the_loss(example):
    _, ex = example
    losses = ex.train(steps=40, channels=32, out_channels=32, groups=4, structures=32, log=None)
    assert all(v == v for v in losses)
    assert sum(losses[-4:]) <= 0.7 * sum(losses[:4]), losses


def test_gradients_along_random_directions(example):
    """As above but relative to each gradient: its derivative along its own
    direction and along one with a random part.  The differences at h and h / 2
    are extrapolated, which leaves the h^4 term; rounding of the loss (1e-6 over
    2 h, h = 1e-2) is below 2e-4, so a gradient of norm 0.05 or more is checked
    to 1 part in 100."""
    torch, ex = example
    dev = torch.device("cuda:0")
    b = ex.batch(12, 5, dev)
    model = ex.Potential(32, 48, 6, dev, seed=4)
    gen = torch.Generator(device=dev)
    gen.manual_seed(11)
    rnd = lambda t: torch.randn(t.shape, generator=gen, device=dev)  # noqa: E731
    model.params["gamma"].add_(0.1 * rnd(model.params["gamma"]))

    def loss():
        return float(((model.forward(b)[0] - b["energy"]).double() ** 2).mean())

    energy, kept = model.forward(b)
    error = energy - b["energy"]
    grads = model.backward(b, 2 * error / error.numel(), kept)
    for name, g in grads.items():
        size = float(g.double().norm())
        assert size >= 0.05, (name, size)
        w, v = model.params[name], rnd(g)
        for d in (g / g.norm(), 0.8 * g / g.norm() + 0.6 * v / v.norm()):
            at = w.clone()

            def slope(h):
                w.copy_(at + h * d)
                up = loss()
                w.copy_(at - h * d)
                down = loss()
                w.copy_(at)
                return (up - down) / (2 * h)

            got = (4 * slope(0.5e-2) - slope(1e-2)) / 3
            want = float((g.double() * d.double()).sum())
            print(f"[example] {name}: |g| {size:.5f}, along d {want:.5f}, by differences {got:.5f}", flush=True)
            assert abs(got - want) <= 1e-2 * size, name
