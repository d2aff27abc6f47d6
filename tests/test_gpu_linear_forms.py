"""The forms of the product at the sizes that take them: their results against the
oracle in 64 bits (the bounds of the product's own tests), and where one gives way to another."""
import numpy as np
import pytest

from tests import dense_oracle as D
from tests import test_gpu_linear as G
from tests import train_oracle as T

pytestmark = pytest.mark.gpu
U = G.U


@pytest.fixture(scope="module")
def tt():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch, torch.device("cuda:0")


# dx of few inputs over many outputs, from rows of g in registers: whole and ragged blocks, outputs that end inside a step
DX = [(32768, 128, 136, "silu", 0.0), (32801, 72, 264, "tanh", 0.1), (33000, 65, 200, "none", 0.0), (40000, 64, 136, "none", 0.0),
      (40100, 24, 264, "none", 0.25), (40003, 8, 144, "silu", 0.1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,M,act,p", DX)
def test_dx_of_few_inputs(tt, N, K, M, act, p, dtype):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[forms] N={N} K={K} M={M} {act} p={p} {dtype}", flush=True)
    rng = np.random.default_rng(N + K)
    q = T.bf16 if dtype == "bf16" else (lambda v: v.astype(np.float32))
    W, z, g = q(rng.standard_normal((K, M)) / K ** 0.5), q(rng.standard_normal((N, M))), q(rng.standard_normal((N, M)))
    m = D.mask(N, M, p, 11, 12)
    to = lambda v: torch.from_numpy(v).to(dev).to(G._dt(torch, dtype))  # noqa: E731
    x = torch.empty(N, K, dtype=G._dt(torch, dtype), device=dev)
    gx, whole = G.rows(torch, dev, np.zeros((N, K)), 2, dtype, fill=7.0)
    dx, _, _ = cg.linear_act_bwd(x, to(W), None if act == "none" else to(z), to(g), act, p_drop=p, seed=11, offset=12,
                                 want=("x",), grad_x=gx)
    assert dx is gx and (whole[:, 0] == 7.0).all()
    want, _, _, dz = D.linear_bwd(np.zeros((N, K)), W, z, g, act, m)
    aW = np.abs(W).astype(np.float64).T
    e = np.abs(dz) * 2 * U + (0 if act == "none" else 16 * U * (1 + np.abs(z)) * np.abs(g) * m)
    tol = e @ aW + (12 * M + 4) * U * (np.abs(dz) @ aW)
    G.near("dx", dx, want, tol + (G.HALF[dtype] + 2 * U) * np.abs(want), dtype, M, extra=16 * U)


def test_dx_of_some_thousand_rows_fills_the_chip(tt):
    """A sixteenth of the rows takes a small part of the time: 65536 rows move 2.1 GB, 0.27 ms at least,
    4096 of them 0.13 GB.  (One block to 256 rows, each through all 4096 outputs, would take
    three quarters of it.)  The shortest of five runs of each."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    K, M = 64, 4096
    W = torch.randn(K, M, device=dev)

    def shortest(N):
        x, z, g = torch.empty(N, K, device=dev), torch.randn(N, M, device=dev), torch.randn(N, M, device=dev)
        us = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            cg.linear_act_bwd(x, W, z, g, want=("x",))
            a.record()
            for _ in range(10):
                cg.linear_act_bwd(x, W, z, g, want=("x",))
            b.record()
            b.synchronize()
            us.append(a.elapsed_time(b) * 100)
        return min(us)

    few, many = shortest(4096), shortest(65536)
    print(f"[forms] dx of 4096 rows {few:.0f} us, of 65536 {many:.0f} us", flush=True)
    assert few <= 0.35 * many
