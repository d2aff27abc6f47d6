"""What the products hold between their operands and their results: the gradient
dz = drop(g) act'(z) keeps fp32's bits whatever the arrays' type, and each result
is rounded once.  u = 2^-24.

dz's bits are seen where what a shorter number would hold of them cancels: with a = g act'(z)
from 64 bits, the gradients -bf16(a) and -bf16(a - bf16(a)) at two places whose slope is 1 (z = 24:
1 + exp(-24) is 1 in fp32) leave what is below a's first 16 bits.

The bound, in the 2-norm over all results, relative to |a| times the other operand.  With E = exp(-z),
0.5 <= z <= 2.5, E is within (|z| + 2) u of itself, 1 + E adds u and the reciprocal 2 u, so that
s = 1 / (1 + E) is within 4 u; 1 - s within 4 u s, z (1 - s) within 8.4 u, two more products and a sum
u each: the slope is within 14 u at most, and a third of that, 5 u, is what independent roundings leave.
The three terms are nine products of bf16 numbers (18 and more for fp32, the others' terms zero),
exact, added with at most 2 u of a partial sum each were it a truncation: sqrt(9) 2 u / sqrt(3) = 3.5 u.
Together 6 u, and twice that is allowed.  a in 16 bits is off by 2^-17 of its binade at most,
in the mean 37 u of a; in eight bits by 2^-8 at most."""
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


# rows, inputs, outputs, probability: tiles, narrow gradients, dx from rows in registers, planes (with rows behind the last tile)
SHAPES = [(300, 130, 200, 0.0), (16, 512, 520, 0.25), (63, 131, 203, 0.0), (3000, 128, 128, 0.25), (500, 40, 64, 0.0),
          (2000, 300, 72, 0.0), (901, 61, 127, 0.5), (5000, 64, 264, 0.25), (4500, 120, 200, 0.0), (1100, 1024, 1032, 0.0),
          (810, 520, 512, 0.25), (4097, 512, 4096, 0.0), (32768, 72, 136, 0.25), (33001, 128, 264, 0.0)]


def cancelling(rng, n, dtype):
    """n slopes' arguments and gradients whose product a keeps 24 bits, a, and the two gradients that leave its last eight."""
    q = T.bf16 if dtype == "bf16" else (lambda v: v.astype(np.float32))
    z, g = q(rng.uniform(0.5, 2.5, n)).astype(np.float64), q(rng.uniform(1, 2, n) * rng.choice([-1, 1], n)).astype(np.float64)
    a = g * T.act_slope("silu", z)
    h = T.bf16(a).astype(np.float64)
    m = T.bf16(a - h).astype(np.float64)
    return z, g, a, -h, -m


def run(torch, dev, dtype, x, W, z, g, p, want):
    import clebsch_gordan_tensor_cgtp_amd as cg
    to = lambda v: torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(dev).to(G._dt(torch, dtype))  # noqa: E731
    return cg.linear_act_bwd(to(x), to(W), to(z), to(g), "silu", p_drop=p, seed=3, offset=5, want=want)


def places(rng, kept):
    """Three different columns of each row among those kept; rows that have fewer take none."""
    order = np.argsort(np.where(kept, rng.random(kept.shape), 2.0), axis=1)[:, :3]
    return order, kept.sum(1) >= 3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_gradients_hold_fp32(tt, k, dtype):
    torch, dev = tt
    N, K, M, p = SHAPES[k]
    print(f"[precision] N={N} K={K} M={M} p={p} {dtype}", flush=True)
    rng = np.random.default_rng(k)
    m = D.mask(N, M, p, 3, 5)
    # dx: three outputs of each row, every output's weight alike; dW: three rows of each output, every row alike
    for want in ("x", "W"):
        kept = m != 0 if want == "x" else (m != 0).T
        z, g = np.full(kept.shape, 1.0), np.zeros(kept.shape)
        at, some = places(rng, kept)
        zt, gt, a, h, l = cancelling(rng, kept.shape[0], dtype)
        i = np.arange(kept.shape[0])[some]
        assert i.size
        for j, (zj, gj) in enumerate(((zt, gt), (24.0 + 0 * zt, h), (24.0 + 0 * zt, l))):
            z[i, at[i, j]], g[i, at[i, j]] = zj[i], gj[i]
        other = T.bf16(rng.uniform(0.5, 1.0, K)).astype(np.float64)
        if want == "x":
            x, W = np.ones((N, K)), np.repeat(other[:, None], M, 1)
        else:
            z, g = z.T, g.T
            x, W = np.repeat(other[None, :], N, 0), np.ones((K, M))
        wdx, wdW, _, _ = D.linear_bwd(x, W, z, g, "silu", m)
        got, exact = run(torch, dev, dtype, x, W, z, g, p, (want,)), {"x": wdx, "W": wdW}[want]
        got = G.host(got[0] if want == "x" else got[1])
        size = np.linalg.norm(other) * np.linalg.norm(a[i]) * m.max()
        off = np.linalg.norm(got - exact) / size / U
        print(f"[precision] d{want}: {off:.2f} u", flush=True)
        assert off <= 12, want


@pytest.mark.parametrize("k", [k for k in range(len(G.CASES)) if k % 3 != 2])
def test_bf16_gradients_are_rounded_once(tt, k):
    """v, what a gradient is before it is rounded, is within e of the exact w; the distance to the
    nearest bf16 number changes by no more than v does, so that the result is within d(w) + 2 e of w,
    d(w) the distance of w itself: elementwise with the bound of e, in the 2-norm with what is
    expected of it (the fp32 products' bounds, of bf16 operands times dz in three numbers)."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    N, K, M, pitch, p, _, _ = G.CASES[k]
    act = ("silu", "tanh")[k % 3]
    print(f"[precision] rounded once N={N} K={K} M={M} p={p} {act}", flush=True)
    x, W, b, _, g, seed, offset, m = G.inputs(k, "bf16")
    z = T.bf16(D.linear_fwd(x, W, b, None, act, m)[1].astype(np.float32))
    tx, tg = G.rows(torch, dev, x, pitch, "bf16")[0], G.rows(torch, dev, g, pitch, "bf16")[0]
    tW, tz = (torch.from_numpy(v).to(dev).bfloat16() for v in (W, z))
    dx, dW, _ = cg.linear_act_bwd(tx, tW, tz, tg, act=act, p_drop=p, seed=seed, offset=offset)
    wdx, wdW, _, dz = D.linear_bwd(x, W, z, g, act, m)
    e = np.abs(dz) * 2 * U + 16 * U * (1 + np.abs(z)) * np.abs(g) * m
    aW, ax = np.abs(W).astype(np.float64).T, np.abs(x).astype(np.float64).T
    for name, got, want, n, tol in (
            ("dx", dx, wdx, M, e @ aW + (6 * M + 4) * U * (np.abs(dz) @ aW)),
            ("dW", dW, wdW, N, ax @ e + (6 * N + 4) * U * (ax @ np.abs(dz)))):
        d = np.abs(T.bf16(want).astype(np.float64) - want)
        err = np.abs(G.host(got) - want)
        tol = tol + 2 * U * np.abs(want)
        assert np.all(err <= d + 2 * tol), (name, float((err / np.maximum(d + 2 * tol, 1e-300)).max()))
        size = np.linalg.norm(want)
        if want.size >= 64 and size > 0:
            expected = (2 * (4 + (6 * n) ** 0.5) + 16) * U * size
            assert np.linalg.norm(err) <= np.linalg.norm(d) + 2 * expected, (name, np.linalg.norm(err) / size, np.linalg.norm(d) / size)
