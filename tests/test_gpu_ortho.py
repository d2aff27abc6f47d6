"""GPU parity of the orthogonalised update against the singular-value form in
64 bits.

Tolerance.  A step's rounding (products that carry 24 bits, fp32 sums) disturbs
its result by about u (|a| + |b| + |c|) ||X||_F, u = 2^-24, at the step's
iterate X; the later steps magnify that by at most their largest slope, a each.
Four times the sum over the steps is allowed, in the Frobenius norm (which also
bounds every element), and bf16's unit roundoff, 2^-8 of the result's norm, for
bf16 results.
"""
import numpy as np
import pytest

from tests import train_oracle as T

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
QUINTIC, CUBIC = (3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0)


@pytest.fixture(scope="module")
def tt():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch, torch.device("cuda:0")


def tolerance(norms, coeffs, scale, dtype):
    a, steps = abs(coeffs[0]), len(norms) - 1
    size = sum(abs(v) for v in coeffs)
    t = 4 * U * scale * size * sum(norms[k] * a ** (steps - 1 - k) for k in range(steps))
    return t + (2.0 ** -8 if dtype == "bf16" else U) * scale * norms[-1]


def gradient(rng, B, m, n, kind):
    G = rng.standard_normal((B, m, n))
    if kind == "spectrum":      # a few strong directions over noise
        r = max(1, min(m, n) // 8)
        G = 0.3 * G + (rng.standard_normal((B, m, r)) * np.exp(-3 * np.arange(r) / r)) @ rng.standard_normal((B, r, n))
    if kind == "rank one":
        G = rng.standard_normal((B, m, 1)) @ rng.standard_normal((B, 1, n))
    return G.astype(np.float32)


CASES = [(1, 1, 1, "noise"), (3, 1, 70, "noise"), (2, 70, 1, "noise"), (15, 128, 128, "spectrum"),
         (4, 64, 200, "noise"), (3, 200, 64, "noise"), (5, 5, 7, "noise"), (2, 33, 31, "spectrum"),
         (34, 64, 64, "noise"), (2, 127, 129, "spectrum"), (2, 130, 126, "noise"), (1, 128, 1024, "spectrum"),
         (1, 257, 300, "spectrum"), (2, 300, 150, "noise"), (1, 8, 3000, "noise"), (1, 3000, 8, "noise"),
         (6, 10, 25, "spectrum"), (3, 16, 16, "noise"), (2, 16, 2048, "spectrum"), (2, 3900, 8, "noise"),
         (1, 16, 2049, "noise"), (2, 17, 40, "noise"), (1, 520, 520, "spectrum"), (2, 96, 96, "rank one"), (1, 1100, 1030, "noise"), (1, 1030, 2100, "spectrum"),
         (3, 1100, 1030, "spectrum")]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,m,n,kind", CASES)
def test_orthogonalize(tt, B, m, n, kind, dtype):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[ortho] {B} x {m} x {n} {kind} {dtype}", flush=True)
    rng = np.random.default_rng(m * 7 + n)
    G = gradient(rng, B, m, n, kind)
    G *= np.exp(rng.uniform(-8, 8, (B, 1, 1))).astype(np.float32)      # the matrices' own magnitudes do not matter
    G = T.bf16(G) if dtype == "bf16" else G
    coeffs, steps, scale = ((QUINTIC, 5, 1.0), (CUBIC, 4, 0.2), (QUINTIC, 1, 3.0))[(m + n) % 3]
    t = torch.from_numpy(G).to(dev).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    out = cg.orthogonalize(t, steps, coeffs, 1e-7, scale)
    assert out.dtype == t.dtype and out.shape == t.shape
    got = out.double().cpu().numpy()
    for b in range(B):
        want, norms = T.orthogonalize(G[b], steps, coeffs, 1e-7, scale)
        err, tol = np.linalg.norm(got[b] - want), tolerance(norms, coeffs, scale, dtype)
        assert err <= tol, (b, float(err / tol))
    assert torch.equal(out, cg.orthogonalize(t, steps, coeffs, 1e-7, scale))


@pytest.mark.parametrize("m,n", [(40, 48), (128, 300), (200, 160), (12, 31)])
def test_orthogonalize_special_matrices(tt, m, n):
    """Zero, tiny, huge and non-finite matrices of one stack do not touch each
    other."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    g = torch.randn(7, m, n, device=dev)
    plain = cg.orthogonalize(g)
    s = g.clone()
    s[0] = 0.0
    s[1, 3, 4] = float("nan")
    s[2, m - 1, n - 1] = float("inf")
    s[3] *= 1e30
    s[4] *= 1e-30                       # far below eps: eps decides
    s[5] = 0.0
    s[5, 1, 2] = -4.0                   # one entry: one singular value
    out = cg.orthogonalize(s)
    assert (out[0] == 0).all() and torch.isnan(out[1]).all() and torch.isnan(out[2]).all()
    assert torch.equal(out[6], plain[6])
    for b in (3, 4, 5):
        want, norms = T.orthogonalize(s[b].cpu().numpy(), 5, QUINTIC, 1e-7, 1.0)
        err = np.linalg.norm(out[b].double().cpu().numpy() - want)
        assert err <= tolerance(norms, QUINTIC, 1.0, "f32"), b


def test_orthogonalize_makes_orthogonal_rows(tt):
    """A convergent cubic ends at the nearest matrix with orthonormal rows."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    g = torch.randn(2, 60, 90, device=dev)
    q = cg.orthogonalize(g, steps=30, coeffs=CUBIC).double()
    eye = torch.eye(60, dtype=torch.float64, device=dev)
    assert max((v @ v.t().contiguous() - eye).norm() for v in q) <= 30 * 4 * U * 2 * 60 ** 0.5


def test_orthogonalize_empty_stack(tt):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    assert cg.orthogonalize(torch.zeros(0, 5, 6, device=dev)).shape == (0, 5, 6)


@pytest.mark.parametrize("m,n", [(128, 128), (64, 500), (300, 260), (9, 20)])
def test_orthogonalize_on_another_stream_and_in_a_graph(tt, m, n):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    g = torch.randn(3, m, n, device=dev)
    want = cg.orthogonalize(g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cg.orthogonalize(g)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(g)
    with torch.cuda.graph(graph):
        cg.orthogonalize(g, out=out)
    for k in range(3):
        g.copy_(torch.randn(3, m, n, device=dev))
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, cg.orthogonalize(g)), k


def products32(G, steps, coeffs, eps, scale):
    """The iteration by plain fp32 products, on the CPU."""
    import torch
    a, b, c = coeffs
    X = torch.from_numpy(np.ascontiguousarray(G, np.float32))
    X = X / (X.norm() + eps)
    tall = X.shape[0] > X.shape[1]
    X = X.t().contiguous() if tall else X
    for _ in range(steps):
        A = X @ X.t().contiguous()
        X = a * X + (b * A + c * (A @ A)) @ X
    return (scale * (X.t() if tall else X)).double().numpy()


STEEP = (4.0848, -6.8946, 2.9270)   # a steeper quintic: a step's error grows faster


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("coeffs,steps", [(QUINTIC, 5), (QUINTIC, 10), (QUINTIC, 20), (STEEP, 5)])
@pytest.mark.parametrize("B,m,n,kind", [(1, 64, 64, "noise"), (1, 128, 128, "spectrum"), (1, 300, 260, "noise"),
                                        (1, 128, 1024, "spectrum"), (1, 500, 64, "noise"), (3, 1100, 1030, "noise"),
                                        (1, 12, 400, "noise"), (1, 12, 2730, "noise"), (1, 12, 2740, "noise"),
                                        (1, 9000, 5, "spectrum"), (1, 3, 20000, "noise")])
def test_orthogonalize_is_as_exact_as_fp32_products(tt, B, m, n, kind, coeffs, steps, dtype):
    """Against the same iteration by fp32 products on the CPU, whose error in
    the Frobenius norm is e32: within 4 e32, whatever the type, steps and
    coefficients, for every form.  A bf16 result is rounded once: rounding is
    an element's distance to a grid, which changes by at most what the element
    changes, so the error is at most that of rounding the exact result plus
    twice 4 e32."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[ortho] {B} x {m} x {n} {kind} {coeffs} x {steps} {dtype}", flush=True)
    G = gradient(np.random.default_rng(m + n + steps), B, m, n, kind)
    G = T.bf16(G) if dtype == "bf16" else G
    t = torch.from_numpy(G).to(dev).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    got = cg.orthogonalize(t, steps, coeffs, 1e-7, 0.5)[0].double().cpu().numpy()
    want, norms = T.orthogonalize(G[0], steps, coeffs, 1e-7, 0.5)
    e32 = np.linalg.norm(products32(G[0], steps, coeffs, 1e-7, 0.5) - want)
    err, tol = np.linalg.norm(got - want), 4 * e32
    if dtype == "bf16":
        tol = np.linalg.norm(T.bf16(want.astype(np.float32)) - want) + 2 * tol
    print(f"[ortho] error {err / norms[-1]:.3e} of the result, allowed {tol / norms[-1]:.3e}", flush=True)
    assert err <= tol, float(err / tol)


@pytest.mark.parametrize("B,m,n,kind", [(2, 64, 64, "noise"), (15, 128, 128, "spectrum"), (3, 90, 120, "noise"),
                                        (4, 128, 1000, "noise"), (2, 500, 64, "noise"), (1, 300, 260, "noise"),
                                        (3, 1100, 1030, "noise")])
def test_orthogonalize_bf16_is_the_fp32_result_rounded(tt, B, m, n, kind):
    """bf16 matrices are fp32 matrices too, and take the same arithmetic: the
    results differ by the last rounding alone (from 17 rows up; below, fp64
    sums are rounded to either type)."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[ortho] {B} x {m} x {n} {kind}", flush=True)
    t = torch.from_numpy(T.bf16(gradient(np.random.default_rng(m + 2 * n), B, m, n, kind))).to(dev)
    assert torch.equal(cg.orthogonalize(t.bfloat16()), cg.orthogonalize(t).bfloat16())


def test_orthogonalize_short_rows_are_rounded_once(tt):
    """Matrices of few rows in fp64, one step, bf16: the definition followed in
    64 bits (X held as fp32, as the kernel does) and rounded once gives the same
    bits, but where the exact value is within 2^-40 of the middle of two bf16
    numbers.  Through fp32 about one element in 2^17 would differ, a dozen here."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    rng = np.random.default_rng(17)
    a, b, c = QUINTIC
    G = T.bf16(rng.standard_normal((100000, 1, 16)).astype(np.float32))
    t = torch.from_numpy(G).to(dev).bfloat16()
    got = cg.orthogonalize(t, 1, QUINTIC, 2.0, 0.75).float().cpu().numpy().ravel()
    g = G.astype(np.float64)
    inv = 1.0 / (np.sqrt((g * g).sum((1, 2), keepdims=True)) + 2.0)
    x = (g * inv).astype(np.float32).astype(np.float64)
    A = (x * x).sum(2, keepdims=True)
    want = ((a * x + (b * A + c * A * A) * x) * 0.75).ravel()
    # bf16 by its definition: 2^7 steps in each power of two
    f, e = np.frexp(want)
    n = np.ldexp(f, 8)
    clear = np.abs(np.abs(n - np.floor(n)) - 0.5) > 2.0 ** -32
    exact = np.ldexp(np.rint(n), e - 8)
    assert clear.mean() > 0.999
    wrong = (got != exact)[clear].sum()
    assert wrong == 0, wrong


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,m,n,steps", [(100, 128, 300, 5), (200, 300, 60, 2), (300, 40, 200, 5), (90, 100, 520, 1),
                                         (2, 20, 65536, 3), (2, 128, 33000, 5)])
def test_orthogonalize_several_chunks_to_a_block(tt, B, m, n, steps, dtype):
    """Short sides of up to 128 with more chunks of 128 columns than blocks, so
    that a block takes several chunks in turn."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[ortho] chunks {B} x {m} x {n} {dtype}", flush=True)
    G = gradient(np.random.default_rng(B + m), B, m, n, "noise")
    G = T.bf16(G) if dtype == "bf16" else G
    t = torch.from_numpy(G).to(dev).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    out = cg.orthogonalize(t, steps)
    got = out.double().cpu().numpy()
    for b in (0, B // 2, B - 1):
        want, norms = T.orthogonalize(G[b], steps, QUINTIC, 1e-7, 1.0)
        err, tol = np.linalg.norm(got[b] - want), tolerance(norms, QUINTIC, 1.0, dtype)
        assert err <= tol, (b, float(err / tol))
    assert torch.equal(out, cg.orthogonalize(t, steps))
    few = cg.orthogonalize(t[:1], steps)        # the same matrix by more blocks: the partial sums differ in order
    want, norms = T.orthogonalize(G[0], steps, QUINTIC, 1e-7, 1.0)
    assert np.linalg.norm(few[0].double().cpu().numpy() - want) <= tolerance(norms, QUINTIC, 1.0, dtype)


def test_orthogonalize_offsets_beyond_32_bits(tt):
    """A stack of more than 2^31 elements (matrices by tiles, by chunks, and one
    per block): the last matrix as by itself, from the same form, or within the
    tolerance."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    for B, m, n in ((9, 15000, 16200), (260, 128, 1 << 16), (131500, 128, 128)):
        print(f"[ortho] beyond 32 bits {B} x {m} x {n}", flush=True)
        assert B * m * n > 1 << 31
        t = torch.zeros(B, m, n, device=dev, dtype=torch.bfloat16)
        last = gradient(np.random.default_rng(5), 1, min(m, 40), min(n, 300), "noise")[0]
        t[-1, :last.shape[0], :last.shape[1]] = torch.from_numpy(last).to(dev)
        last = t[-1, :last.shape[0], :last.shape[1]].float().cpu().numpy()
        out = cg.orthogonalize(t, 1)
        assert not out[:-1].any()
        got = out[-1]
        want, norms = T.orthogonalize(last, 1, QUINTIC, 1e-7, 1.0)     # zero rows and columns stay zero
        err = np.linalg.norm(got[:last.shape[0], :last.shape[1]].double().cpu().numpy() - want)
        assert err <= tolerance(norms, QUINTIC, 1.0, "bf16")
        assert not got[last.shape[0]:].any() and not got[:, last.shape[1]:].any()
        del t, out, got
