"""The dense operators as a potential uses them, with the convolution, the
normalisation and the embedding: a radial network (two products) makes the
convolution's edge weights from functions of the distance, and the atoms'
invariant rows are updated by a block with normalisation, two products, dropout
and a residual.  The gradients of all parameters against differences, the
whole step captured and replayed, and a few steps of training on it."""
import pytest

pytestmark = pytest.mark.gpu
SPECIES, BASIS, HIDDEN, C = 5, 8, 48, 32
DROP = dict(p_drop=0.2, seed=2**40 + 3)


@pytest.fixture(scope="module")
def tt():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch, torch.device("cuda:0")


class Model:
    def __init__(self, torch, dev, atoms=60):
        import clebsch_gordan_tensor_cgtp_amd as cg
        self.torch, self.cg = torch, cg
        g = torch.Generator(device=dev)
        g.manual_seed(3)
        rnd = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
        self.plan = cg.Plan(0, 1, 1, C)
        P = self.plan.num_paths
        self.params = {"table": rnd(SPECIES, C), "W1": rnd(BASIS, HIDDEN) / BASIS ** 0.5, "b1": 0.1 * rnd(HIDDEN),
                       "W2": rnd(HIDDEN, P * C) / HIDDEN ** 0.5, "gamma": 1 + 0.1 * rnd(C), "beta": 0.1 * rnd(C),
                       "W3": rnd(C, 4 * C) / C ** 0.5, "b3": 0.1 * rnd(4 * C), "W4": rnd(4 * C, C) / (4 * C) ** 0.5,
                       "w_out": rnd(C) / C ** 0.5}
        # a ring: every atom sees the three before and the three behind it
        steps = torch.tensor([-3, -2, -1, 1, 2, 3], device=dev)
        self.src = ((torch.arange(atoms, device=dev)[:, None] + steps) % atoms).int().view(-1)
        self.row_ptr = (6 * torch.arange(atoms + 1, device=dev)).int()
        self.r = rnd(6 * atoms, 3)
        dist = self.r.norm(dim=1, keepdim=True)
        self.basis = torch.exp(-(dist - torch.linspace(0.3, 3.0, BASIS, device=dev)) ** 2)
        self.species = torch.randint(0, SPECIES, (atoms,), generator=g, device=dev, dtype=torch.int32)
        self.seg = torch.tensor([0, atoms // 3, atoms // 2, atoms], dtype=torch.int32, device=dev)
        self.Y = self.plan.sh(self.r)
        self.ws = self.plan.graph_prepare(self.row_ptr, self.src)

    def forward(self, step=None):
        cg, p = self.cg, self.params
        h, z1 = cg.linear_act_fwd(self.basis, p["W1"], p["b1"], "silu")
        W, _ = cg.linear_act_fwd(h, p["W2"], act="none")
        W = W.view(-1, self.plan.num_paths, C)
        x = cg.embed_fwd(self.species, p["table"])
        out = self.plan.conv_fwd(self.row_ptr, self.src, x.view(-1, 1, C), self.Y, W, self.ws)
        s = out[:, 0, :]
        n, mean, rstd = cg.norm_act_fwd(s, p["gamma"], p["beta"], 4, self.seg, act="none")
        u, z3 = cg.linear_act_fwd(n, p["W3"], p["b3"], "tanh", offset=0, step=step, **DROP)
        y, _ = cg.linear_act_fwd(u, p["W4"], act="none", residual=s, offset=1 << 33, step=step, **DROP)
        y = cg.dropout(y, 0.1, 11, 5, step)
        return y @ p["w_out"], (h, z1, W, x, out, n, mean, rstd, u, z3, y)

    def backward(self, grad, kept, step=None):
        cg, p = self.cg, self.params
        h, z1, W, x, out, n, mean, rstd, u, z3, y = kept
        g = {"w_out": y.t().contiguous() @ grad}
        gy = cg.dropout(grad[:, None] * p["w_out"], 0.1, 11, 5, step)
        gu, g["W4"], _ = cg.linear_act_bwd(u, p["W4"], None, gy, "none", offset=1 << 33, step=step, want=("x", "W"), **DROP)
        gn, g["W3"], g["b3"] = cg.linear_act_bwd(n, p["W3"], z3, gu, "tanh", offset=0, step=step, **DROP)
        gs, g["gamma"], g["beta"] = cg.norm_act_bwd(out[:, 0, :], mean, rstd, p["gamma"], p["beta"], gn, 4, self.seg, act="none")
        gout = self.torch.zeros_like(out)
        gout[:, 0, :] = gs + gy
        gx, gW, _ = self.plan.conv_bwd(self.row_ptr, self.src, x.view(-1, 1, C), self.Y, W, gout, self.ws, want=("dx", "dW"))
        g["table"] = cg.embed_bwd(self.species, gx[:, 0, :], SPECIES)
        gh, g["W2"], _ = cg.linear_act_bwd(h, p["W2"], None, gW.view(gW.shape[0], -1), "none", want=("x", "W"))
        _, g["W1"], g["b1"] = cg.linear_act_bwd(self.basis, p["W1"], z1, gh, "silu", want=("W", "bias"))
        return g


def test_gradients_of_a_potential_against_differences(tt):
    """The derivative of sum(e^2) / 2 of the atoms' energies along each gradient and along one with a
    random part, by differences at h and h / 2, extrapolated: fp32 rounding of a loss of order |e|^2
    (1e-6 of it over 2 h, h = 1e-2) and the h^4 term stay below 1 part in 100 of |g|."""
    torch, dev = tt
    model = Model(torch, dev)
    loss = lambda: float((model.forward()[0].double() ** 2).sum() / 2)  # noqa: E731
    e, kept = model.forward()
    grads = model.backward(e, kept)
    gen = torch.Generator(device=dev)
    gen.manual_seed(8)
    scale = loss()
    for name, g in grads.items():
        w, v = model.params[name], torch.randn(g.shape, generator=gen, device=dev)
        size = float(g.double().norm())
        for d in (g / g.norm(), 0.8 * g / g.norm() + 0.6 * v / v.norm()):
            at = w.clone()

            def slope(h):
                w.copy_(at + h * d)
                up = loss()
                w.copy_(at - h * d)
                down = loss()
                w.copy_(at)
                return (up - down) / (2 * h)

            got, want = (4 * slope(0.5e-2) - slope(1e-2)) / 3, float((g.double() * d.double()).sum())
            print(f"[together] {name}: |g| {size:.5f}, along d {want:.5f}, by differences {got:.5f}", flush=True)
            assert abs(got - want) <= 1e-2 * size + 2e-4 * scale, name


def test_training_step_in_a_graph(tt):
    """Forward, backward and the update of the step counter, captured once: replays between eager
    steps on changed parameters give the eager gradients of that counter, bit for bit."""
    torch, dev = tt
    model = Model(torch, dev)
    step = torch.zeros(1, dtype=torch.int64, device=dev)

    def run(at):
        e, kept = model.forward(at)
        return model.backward(e, kept, at)

    run(step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run(step)
        step.add_(1)
    seen = []
    for k in range(3):
        model.params["W3"].mul_(0.9)
        at = torch.full((1,), k, dtype=torch.int64, device=dev)
        graph.replay()
        eager = run(at)
        torch.cuda.synchronize()
        for name, g in eager.items():
            assert torch.equal(g, kept[name]), (k, name)
        seen.append(kept["W4"].clone())
    assert int(step) == 3 and not torch.equal(seen[0], seen[1])


def test_training_steps_run(tt):
    torch, dev = tt
    model = Model(torch, dev)
    target = torch.randn(60, device=dev)
    for k in range(5):
        step = torch.full((1,), k, dtype=torch.int64, device=dev)
        e, kept = model.forward(step)
        grads = model.backward((e - target) / 60, kept, step)
        assert sorted(grads) == sorted(model.params)
        for name, g in grads.items():
            assert torch.isfinite(g).all(), name
            assert g.shape == model.params[name].shape, name
            w = model.params[name]
            w.sub_(0.05 * (model.cg.orthogonalize(g) if g.dim() == 2 else g))
