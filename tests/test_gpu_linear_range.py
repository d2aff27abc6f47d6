"""Operands whose neighbours differ by up to 60 decades, in every form of the product: each
element keeps its own precision whatever stands beside it, in both directions.

One operand holds elements of 1e-30 to 1e30 in no order, the other picks one of them for each
result (a single 1 to a row or column of the contraction), so that a result is one element: an fp32
one as its three bf16 numbers, which hold it but for what lies below 2^-126 (twice that at most),
added in fp32: 2 u of it, u = 2^-24; a bf16 one as it is."""
import numpy as np
import pytest

from tests import test_gpu_linear as G

pytestmark = pytest.mark.gpu
U = G.U


@pytest.fixture(scope="module")
def tt():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch, torch.device("cuda:0")


def scattered(torch, gen, dev, dt, *shape):
    e = torch.rand(shape, generator=gen, device=dev) * 60 - 30
    return (torch.randn(shape, generator=gen, device=dev).double() * 10.0 ** e.double()).to(dt)


def single(torch, dev, dt, rows, cols, at):
    """[rows][cols] of zeros but for a 1 in column at[r] of row r."""
    t = torch.zeros(rows, cols, device=dev, dtype=dt)
    t[torch.arange(rows, device=dev), at] = 1.0
    return t


def near(torch, name, got, want):
    off = (got.double() - want.double()).abs()
    tol = 2 * U * want.double().abs() + 2.0 ** -125 if got.dtype == torch.float32 else 0.0 * want.double().abs()
    assert (off <= tol).all(), (name, float((off / want.double().abs().clamp_min(1e-300)).max()), int((off > tol).sum()))


# few rows; rows in registers; tiles; planes with rows behind the last tile; narrow gradients; dx and dW of
# few inputs in registers (from 40000, 32768 and 8192 rows)
SHAPES = [(2, 600, 72), (16, 1024, 40), (300, 64, 136), (260, 120, 33), (40, 300, 200), (130, 200, 264), (1100, 1024, 1032),
          (4097, 512, 4096), (3000, 128, 128), (301, 61, 127), (40000, 24, 136), (32768, 72, 136), (9001, 40, 264), (8193, 64, 131)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,M", SHAPES)
def test_elements_keep_their_own_precision(tt, N, K, M, dtype):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[range] N={N} K={K} M={M} {dtype}", flush=True)
    dt = G._dt(torch, dtype)
    gen = torch.Generator(device=dev)
    gen.manual_seed(N + K + M)
    rnd = lambda *s: scattered(torch, gen, dev, dt, *s)  # noqa: E731
    pick = lambda n, lim: torch.randint(lim, (n,), generator=gen, device=dev)  # noqa: E731
    x, W, g = rnd(N, K), rnd(K, M), rnd(N, M)
    k_of_n, k_of_m, m_of_k, m_of_n = pick(N, K), pick(M, K), pick(K, M), pick(N, M)
    n_of_k, n_of_m = torch.randperm(N, generator=gen, device=dev), torch.randperm(N, generator=gen, device=dev)
    # y: an element of x, an element of W
    near(torch, "y of x", cg.linear_act_fwd(x, single(torch, dev, dt, M, K, k_of_m).t().contiguous(), act="none")[0], x[:, k_of_m])
    near(torch, "y of W", cg.linear_act_fwd(single(torch, dev, dt, N, K, k_of_n), W, act="none")[0], W[k_of_n])
    # dx: an element of g, an element of W
    back = lambda x, W, g, want: cg.linear_act_bwd(x, W, None, g, "none", want=(want,))["xW".index(want)]  # noqa: E731
    near(torch, "dx of g", back(x, single(torch, dev, dt, K, M, m_of_k), g, "x"), g[:, m_of_k])
    near(torch, "dx of W", back(x, W, single(torch, dev, dt, N, M, m_of_n), "x"), W[:, m_of_n].t())
    # dW: an element of g for each input that has a row, an element of x for each output that has one
    ks, ms = min(N, K), min(N, M)
    one = torch.zeros(N, K, device=dev, dtype=dt)
    one[n_of_k[:ks], torch.arange(ks, device=dev)] = 1.0
    dW = back(one, W, g, "W")
    near(torch, "dW of g", dW[:ks], g[n_of_k[:ks]])
    assert not dW[ks:].any()
    one = torch.zeros(N, M, device=dev, dtype=dt)
    one[n_of_m[:ms], torch.arange(ms, device=dev)] = 1.0
    dW = back(x, W, one, "W")
    near(torch, "dW of x", dW[:, :ms], x[n_of_m[:ms]].t())
    assert not dW[:, ms:].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,M", [(32768, 72, 136), (40000, 24, 136), (32801, 128, 264)])
def test_infinities_reach_only_their_results(tt, N, K, M, dtype):
    """Of the gradients from rows in registers: the same as of the other forms."""
    G.test_infinities_reach_only_their_results(tt, N, K, M, dtype)
