"""GPU parity of the product with bias, activation, dropout and residual, and
of its gradients, against the oracle in 64 bits.

Tolerances, with u = 2^-24 and the half steps h (fp32 2^-24, bf16 2^-8).
An fp32 product of k terms: each operand is three bf16 numbers that hold it
exactly; the terms left out are at most 2^-25 of a term; the six products are
exact in fp32 and added with at most one rounding each (2 u of the partial sum, were it
a truncation), the parts' sums in fp64: elementwise at most (12 k + 4) u S, S the
sum of the terms' magnitudes.  In the 2-norm the roundings are independent: 6 k of
them, each at most u of a partial sum that grows like its square root, so that
sqrt(6 k) u of the result's norm bounds what is expected; 4 u more for the
terms left out and the last rounding, and twice that is allowed (a missing
remainder of an operand would leave 2^-18, 64 u).  bf16 products are exact: the same with k for 6 k.
y = r + s act(z) moves by 1.1 s times z's error, 8 u max(1, |z|) s for the activation's own, and u of
each term.  dz carries 16 u (1 + |z|) |g| s of its slope, and for bf16 is rounded to half a step before
the products (not before the bias' sum, which is fp64).  Each result is rounded once."""
import numpy as np
import pytest

from tests import dense_oracle as D
from tests import train_oracle as T

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def tt():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch, torch.device("cuda:0")


def _dt(torch, dtype):
    return torch.float32 if dtype == "f32" else torch.bfloat16


def rows(torch, dev, v, pitch, dtype, fill=float("nan")):
    """v [N][C] as every pitch-th row of a wider array of `fill`."""
    t = torch.full((v.shape[0], pitch, v.shape[1]), fill, dtype=_dt(torch, dtype), device=dev)
    t[:, pitch - 1, :] = torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(dev)
    return t[:, pitch - 1, :], t


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def steps(dtype):
    return 12 if dtype == "f32" else 2


def near(name, got, want, tol, dtype, k, extra=0.0):
    """Elementwise, and for fp32 in the 2-norm."""
    got = host(got)
    err = np.abs(got - want)
    assert np.all(err <= tol), (name, float((err / np.maximum(tol, 1e-300)).max()))
    size = np.linalg.norm(want)
    if dtype == "f32" and want.size >= 64 and size > 0:
        rel = np.linalg.norm(got - want) / size
        assert rel <= 2 * U * (4 + (6 * k) ** 0.5) + extra, (name, rel / U)


# rows, inputs, outputs, stride of rows, probability, bias, residual
CASES = [(1, 1, 1, 1, 0.0, True, True), (1, 8, 8, 1, 0.0, True, False), (2, 3, 5, 1, 0.5, True, True),
         (3, 5, 7, 2, 0.0, False, True), (17, 33, 65, 1, 0.1, True, True), (64, 64, 64, 1, 0.0, False, False),
         (65, 8, 64, 1, 0.1, True, False), (130, 128, 128, 9, 0.1, True, True), (500, 24, 1920, 1, 0.0, False, False),
         (129, 129, 130, 3, 0.25, True, True), (33, 4096, 40, 1, 0.0, True, True), (2000, 128, 128, 9, 0.1, True, True),
         (5000, 16, 24, 1, 0.5, True, False), (257, 72, 200, 1, 0.1, True, True), (1, 1000, 520, 1, 0.0, True, True),
         (4, 2048, 96, 1, 0.1, True, True), (7, 40, 4104, 2, 0.0, True, False), (9000, 136, 264, 1, 0.1, True, True),
         (40000, 8, 64, 1, 0.0, True, False), (12, 30, 2050, 1, 0.9, True, True), (300, 2056, 1000, 1, 0.0, True, False),
         (16, 512, 512, 1, 0.0, True, True), (1029, 520, 776, 1, 0.1, True, True), (100, 1, 300, 1, 0.0, True, True),
         (100, 300, 1, 1, 0.0, True, True), (8, 1001, 64, 1, 0.0, False, False),
         # products of planes: contractions that are whole steps and not, cut and not, tiles that end inside
         (1025, 1000, 1032, 1, 0.1, True, True), (4100, 264, 1000, 2, 0.0, True, False),
         (300, 2056, 2000, 1, 0.5, False, True), (2050, 1024, 512, 1, 0.0, False, False),
         (256, 4096, 1024, 1, 0.1, True, True), (16500, 256, 264, 1, 0.0, True, False),
         (1100, 1024, 1024, 3, 0.0, True, True), (4352, 512, 4096, 1, 0.1, True, False),
         # narrow gradients: slabs of inputs or outputs, a chunk to a block and several, ragged ends
         (70000, 128, 128, 1, 0.1, True, False), (40001, 64, 64, 2, 0.0, True, False), (3001, 300, 72, 1, 0.5, True, True),
         (3001, 72, 300, 1, 0.5, True, True), (20000, 120, 56, 1, 0.0, True, False), (64, 128, 128, 1, 0.0, True, True),
         (63, 61, 127, 1, 0.1, True, True), (65, 129, 128, 1, 0.1, True, True), (5001, 1000, 8, 1, 0.0, True, False),
         # few inputs over many outputs: rows of g and columns of x and g in registers
         (9001, 64, 200, 1, 0.0, True, False), (8200, 40, 1000, 2, 0.0, True, False), (8193, 7, 136, 1, 0.0, True, True),
         (5000, 120, 264, 1, 0.1, True, False), (12345, 50, 131, 1, 0.0, False, False), (20000, 64, 1920, 1, 0.0, False, False),
         (8192, 64, 136, 1, 0.5, True, False),
         (1300, 1000, 1032, 1, 0.1, True, True), (1400, 1032, 1000, 2, 0.0, False, False), (810, 520, 512, 1, 0.1, True, True),
         # rows behind the last whole tile that go by themselves
         (4097, 512, 4096, 1, 0.1, True, True), (16390, 1032, 264, 1, 0.5, True, True),
         (16448, 264, 1024, 2, 0.1, True, False)]


def inputs(k, dtype):
    N, K, M, pitch, p, bias, residual = CASES[k]
    rng = np.random.default_rng(100 + k)
    q = T.bf16 if dtype == "bf16" else (lambda v: v.astype(np.float32))
    x, W = q(rng.standard_normal((N, K))), q(rng.standard_normal((K, M)) / K ** 0.5)
    b = rng.standard_normal(M).astype(np.float32) if bias else None
    r = q(rng.standard_normal((N, M))) if residual else None
    seed, offset = int(rng.integers(0, 2**64, dtype=np.uint64)), int(rng.integers(0, 2**40))
    return x, W, b, r, q(rng.standard_normal((N, M))), seed, offset, D.mask(N, M, p, seed, offset)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", range(len(CASES)))
def test_linear_forward(tt, k, dtype):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    N, K, M, pitch, p, bias, residual = CASES[k]
    act = ("silu", "tanh", "none")[k % 3]
    print(f"[linear] forward N={N} K={K} M={M} pitch={pitch} p={p} {act} {dtype}", flush=True)
    x, W, b, r, _, seed, offset, m = inputs(k, dtype)
    tx, tr = rows(torch, dev, x, pitch, dtype)[0], None if r is None else rows(torch, dev, r, pitch, dtype)[0]
    tW = torch.from_numpy(W).to(dev).to(tx.dtype)
    tb = None if b is None else torch.from_numpy(b).to(dev)
    out, whole = rows(torch, dev, np.zeros((N, M)), pitch, dtype, fill=7.0)
    args = dict(residual=tr, p_drop=p, seed=seed, offset=offset)
    y, z = cg.linear_act_fwd(tx, tW, tb, act, out=out, **args)
    assert y is out and (z is None) == (act == "none")
    wy, wz = D.linear_fwd(x, W, b, r, act, m)
    S = np.abs(x).astype(np.float64) @ np.abs(W).astype(np.float64)
    tz = (steps(dtype) * K + 4) * U * S + 2 * U * np.abs(wz)
    ty = 1.1 * m * tz + 8 * U * m * np.maximum(1, np.abs(wz)) + 3 * U * (np.abs(wy) + (0 if r is None else np.abs(r)))
    # (the residual's part of y hides the product's in the norm; the activation adds its own 8 u)
    near("y", y, wy, ty + HALF[dtype] * np.abs(wy), dtype, K, extra=16 * U)
    if z is not None:
        near("z", z, wz, tz + HALF[dtype] * np.abs(wz), dtype, K)
    assert pitch == 1 or (whole[:, :pitch - 1] == 7.0).all()
    again, none = cg.linear_act_fwd(tx, tW, tb, act, save=False, **args)
    assert none is None and torch.equal(again, y) and again.is_contiguous()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", range(len(CASES)))
def test_linear_backward(tt, k, dtype):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    N, K, M, pitch, p, _, _ = CASES[k]
    act = ("silu", "tanh", "none")[k % 3]
    print(f"[linear] backward N={N} K={K} M={M} pitch={pitch} p={p} {act} {dtype}", flush=True)
    x, W, b, _, g, seed, offset, m = inputs(k, dtype)
    q = T.bf16 if dtype == "bf16" else (lambda v: v.astype(np.float32))
    z = q(D.linear_fwd(x, W, b, None, act, m)[1].astype(np.float32))
    tx, tg = rows(torch, dev, x, pitch, dtype)[0], rows(torch, dev, g, pitch, dtype)[0]
    tW = torch.from_numpy(W).to(dev).to(tx.dtype)
    tz = torch.from_numpy(z).to(dev).to(tx.dtype) if act != "none" else None
    gx, whole = rows(torch, dev, np.zeros((N, K)), pitch, dtype, fill=7.0)
    args = dict(act=act, p_drop=p, seed=seed, offset=offset)
    dx, dW, db = cg.linear_act_bwd(tx, tW, tz, tg, grad_x=gx, **args)
    assert dx is gx and dW.dtype == tW.dtype and db.dtype == torch.float32
    wdx, wdW, wdb, dz = D.linear_bwd(x, W, z, g, act, m)
    e = np.abs(dz) * 2 * U + (0 if act == "none" else 16 * U * (1 + np.abs(z)) * np.abs(g) * m)
    rounded = e + (HALF["bf16"] * np.abs(dz) if dtype == "bf16" and act != "none" else 0)
    aW, ax = np.abs(W).astype(np.float64).T, np.abs(x).astype(np.float64).T
    tdx = rounded @ aW + (steps(dtype) * M + 4) * U * (np.abs(dz) @ aW)
    tdW = ax @ rounded + (steps(dtype) * N + 4) * U * (ax @ np.abs(dz))
    near("dx", dx, wdx, tdx + (HALF[dtype] + 2 * U) * np.abs(wdx), dtype, M, extra=16 * U)
    near("dW", dW, wdW, tdW + (HALF[dtype] + 2 * U) * np.abs(wdW), dtype, N, extra=16 * U)
    near("db", db, wdb, e.sum(0) + 2 * U * np.abs(wdb) + N * 2.0 ** -53 * np.abs(dz).sum(0), "bf16", N)
    assert pitch == 1 or (whole[:, :pitch - 1] == 7.0).all()
    for want in (("x",), ("W",), ("bias",), ("x", "bias"), ("W", "bias"), ()):
        got = cg.linear_act_bwd(tx, tW, tz, tg, want=want, **args)
        for name, u, v in zip(("x", "W", "bias"), got, (dx, dW, db)):
            assert (u is None) == (name not in want)
            assert u is None or torch.equal(u, v), (want, name)


@pytest.mark.parametrize("act", ["none", "silu", "tanh"])
def test_linear_gradients_against_differences(tt, act):
    """Central differences of <G, y> in fp32 along random directions of norm d,
    extrapolated from h and h / 2: the h^4 term at h = 0.02 is below 1e-5 of
    derivatives of order |G|, and rounding leaves 4 u sqrt(N M) |y| / h, below 1e-4."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    N, K, M = 200, 72, 120
    gen = torch.Generator(device=dev)
    gen.manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    a = {"x": rnd(N, K), "W": rnd(K, M) / K ** 0.5, "bias": rnd(M), "residual": rnd(N, M)}
    G = rnd(N, M)
    drop = dict(p_drop=0.2, seed=4, offset=11)

    def forward(**change):
        v = {**a, **change}
        return cg.linear_act_fwd(v["x"], v["W"], v["bias"], act, residual=v["residual"], **drop)

    _, z = forward()
    gx, gW, gb = cg.linear_act_bwd(a["x"], a["W"], z, G, act, **drop)
    for name, g in (("x", gx), ("W", gW), ("bias", gb), ("residual", G)):
        d = rnd(*g.shape)
        d /= d.norm()
        loss = lambda h: float((G.double() * forward(**{name: a[name] + h * d})[0].double()).sum())  # noqa: E731
        slope = lambda h: (loss(h) - loss(-h)) / (2 * h)  # noqa: E731
        got, want = (4 * slope(0.01) - slope(0.02)) / 3, float((g.double() * d.double()).sum())
        print(f"[linear] {act} {name}: {want:.5f}, by differences {got:.5f}", flush=True)
        assert abs(got - want) <= 2e-2 * max(1.0, float(g.norm()) / g.numel() ** 0.5), name


def test_linear_dropout_is_dropout_of_the_product(tt):
    """One mask: the epilogue's is that of the call by itself, forward and back, for
    whole tiles, odd widths, few rows and contractions that are cut."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    for N, K, M in ((300, 64, 128), (37, 19, 61), (3, 256, 96), (40, 4096, 24), (6, 5, 9)):
        x, W, r = torch.randn(N, K, device=dev), torch.randn(K, M, device=dev), torch.randn(N, M, device=dev)
        y, z = cg.linear_act_fwd(x, W, act="tanh")
        got, z2 = cg.linear_act_fwd(x, W, act="tanh", residual=r, p_drop=0.3, seed=8, offset=2**35)
        assert torch.equal(z, z2) and torch.equal(got, cg.dropout(y, 0.3, 8, 2**35, residual=r)), (N, K, M)
        keep = torch.from_numpy(D.mask(N, M, 0.3, 8, 2**35) != 0).to(dev)
        g = torch.randn(N, M, device=dev)
        spoilt = torch.where(keep, g, float("nan"))      # what is dropped is not looked at
        zs = torch.where(keep, z, float("inf"))
        a = cg.linear_act_bwd(x, W, zs, spoilt, "tanh", p_drop=0.3, seed=8, offset=2**35)
        b = cg.linear_act_bwd(x, W, z, g, "tanh", p_drop=0.3, seed=8, offset=2**35)
        assert all(torch.equal(u, v) for u, v in zip(a, b)), (N, K, M)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_of_no_rows(tt, dtype):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    x, W = torch.zeros(0, 24, device=dev, dtype=_dt(torch, dtype)), torch.ones(24, 40, device=dev, dtype=_dt(torch, dtype))
    y, z = cg.linear_act_fwd(x, W)
    assert y.shape == (0, 40) and z.shape == (0, 40)
    dx, dW, db = cg.linear_act_bwd(x, W, z, y)
    assert dx.shape == (0, 24) and dW.shape == (24, 40) and (dW == 0).all() and (db == 0).all()
    dW = cg.linear_act_bwd(x[:, :3], W[:3, :1].contiguous(), z[:, :1].contiguous(), y[:, :1])[1]
    assert dW.shape == (3, 1) and (dW == 0).all()


def test_linear_of_three_axes_and_rows_of_features(tt):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    x, W, r = torch.randn(5, 60, 40, device=dev), torch.randn(40, 56, device=dev), torch.randn(5, 60, 56, device=dev)
    y, z = cg.linear_act_fwd(x, W, residual=r)
    flat = cg.linear_act_fwd(x.view(300, 40), W, residual=r.view(300, 56))
    assert y.shape == (5, 60, 56) and torch.equal(y.view(300, 56), flat[0]) and torch.equal(z.view(300, 56), flat[1])
    g = cg.linear_act_bwd(x, W, z, r)
    f = cg.linear_act_bwd(x.view(300, 40), W, flat[1], r.view(300, 56))
    assert g[0].shape == x.shape and torch.equal(g[0].view(300, 40), f[0]) and torch.equal(g[1], f[1])


def test_infinities_and_nan_stay_in_their_rows(tt):
    """A row of x that holds an infinity or a NaN gives results that are not finite; the
    other rows are what they are without it.  (The gradient of W sums over all rows.)"""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    for dt in (torch.float32, torch.bfloat16):
        for N, K, M in ((200, 72, 136), (5, 200, 48), (70, 33, 35)):
            x, W = torch.randn(N, K, device=dev, dtype=dt), torch.randn(K, M, device=dev, dtype=dt)
            y = cg.linear_act_fwd(x, W, act="none")[0]
            for bad in (float("inf"), float("-inf"), float("nan")):
                s = x.clone()
                s[3, K // 2] = bad
                got = cg.linear_act_fwd(s, W, act="none")[0]
                assert not torch.isfinite(got[3]).any()
                got[3] = y[3]
                assert torch.equal(got, y)


def test_wide_range_of_magnitudes(tt):
    """fp32 operands keep their own precision whatever stands beside them: a column of W
    that spans 60 decades against rows that pick one element each.  (A remainder below fp32's
    smallest normal number 2^-126 counts as zero in the matrix instructions: an element's second
    and third number are each lost where they are below it, together less than 2 x 2^-126.)"""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    K = 64
    W = torch.logspace(-30, 30, K, device=dev, dtype=torch.float64).float()[:, None] * torch.randn(K, 40, device=dev)
    x = torch.eye(K, device=dev)
    y = cg.linear_act_fwd(x, W, act="none")[0]
    assert ((y - W).abs() <= 2 * U * W.abs() + 2.0 ** -125).all()
    y = cg.linear_act_fwd(torch.cat([x] * 3), W, act="none")[0]      # by tiles, whatever few rows take
    assert ((y - torch.cat([W] * 3)).abs() <= 2 * U * torch.cat([W] * 3).abs() + 2.0 ** -125).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_in_a_captured_graph(tt, dtype):
    """A forward and backward step, captured with its own workspaces and replayed between
    eager steps on other data, gives the eager results each time; the masks follow the step."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    dt = _dt(torch, dtype)
    N, K, M = 3000, 64, 200
    x, W, b = torch.randn(N, K, device=dev).to(dt), torch.randn(K, M, device=dev).to(dt), torch.randn(M, device=dev)
    g, step = torch.randn(N, M, device=dev).to(dt), torch.zeros(1, dtype=torch.int64, device=dev)

    def run(offset=0, at=step):
        y, z = cg.linear_act_fwd(x, W, b, p_drop=0.2, seed=3, offset=offset, step=at)
        return (y, z) + cg.linear_act_bwd(x, W, z, g, p_drop=0.2, seed=3, offset=offset, step=at)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
        step.add_(1)
    for k in range(4):
        x.copy_(torch.randn(N, K, device=dev))
        graph.replay()
        eager = run(offset=k, at=None)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(kept, eager)), k


def test_linear_on_two_streams(tt):
    """Calls with their own workspaces on two streams at once."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    x, W = [torch.randn(20000, 64, device=dev) for _ in range(2)], torch.randn(64, 96, device=dev)
    z = [cg.linear_act_fwd(v, W)[1] for v in x]
    want = [cg.linear_act_bwd(v, W, u, u) for v, u in zip(x, z)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(cg.linear_act_bwd(x[i], W, z[i], z[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for v in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(v, want[i]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_offsets_beyond_32_bits(tt, dtype):
    """y of more than 2^31 elements, and rows of x more than 2^32 bytes from its start."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    N, K, M = (1 << 20) + 77, 16, 2056
    print(f"[linear] beyond 32 bits {dtype}", flush=True)
    dt = _dt(torch, dtype)
    gen = torch.Generator(device=dev)
    gen.manual_seed(1)
    wide = torch.zeros(N, 2304, device=dev, dtype=dt)
    x = wide[:, 2288:]
    x.copy_(torch.randn(N, K, generator=gen, device=dev))
    W = (torch.randn(K, M, generator=gen, device=dev) / 4).to(dt)
    y = cg.linear_act_fwd(x, W, act="none")[0]
    at = torch.tensor([0, 1, N // 2, N - 130, N - 2, N - 1], device=dev)
    want = host(x[at]) @ host(W)
    S = np.abs(host(x[at])) @ np.abs(host(W))
    assert np.all(np.abs(host(y[at]) - want) <= 12 * 17 * U * S + HALF[dtype] * np.abs(want))
    # one row of the gradient alone: dx has that row, dW its outer product
    y.zero_()
    row = torch.randn(M, generator=gen, device=dev).to(dt)
    for n in (N - 1, N // 2):
        y[n] = row
        dx, dW, db = cg.linear_act_bwd(x, W, None, y, act="none")
        h = host(row)
        want, S = h @ host(W).T, np.abs(h) @ np.abs(host(W)).T
        assert np.all(np.abs(host(dx[n]) - want) <= 12 * (M + 1) * U * S + HALF[dtype] * np.abs(want))
        want = host(x[n])[:, None] * h[None, :]
        assert np.all(np.abs(host(dW) - want) <= (2 * U + HALF[dtype]) * np.abs(want))
        assert np.array_equal(host(db), h)
        y[n] = 0
        dx[n] = 0
        assert not dx.any()


# every form of the product, its rows on odd addresses
ODD = [(3, 600, 72), (300, 64, 128), (40, 3000, 24), (1100, 1024, 1032), (5000, 72, 264), (9000, 48, 200),
       (3000, 96, 40), (700, 300, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", range(len(ODD)))
def test_linear_on_odd_addresses(tt, k, dtype):
    """Arrays that begin one element behind a 16-byte boundary, their rows an odd number of elements apart."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    N, K, M = ODD[k]
    print(f"[linear] odd addresses N={N} K={K} M={M} {dtype}", flush=True)
    dt, rng = _dt(torch, dtype), np.random.default_rng(k)
    q = T.bf16 if dtype == "bf16" else (lambda v: v.astype(np.float32))

    def rows_at(v, gap):
        """v as rows `gap` elements apart more than their width, from an odd element on"""
        n, c = v.shape
        flat = torch.full((n * (c + gap) + 9,), float("nan"), dtype=dt, device=dev)
        t = flat[1:1 + n * (c + gap)].view(n, c + gap)[:, :c]
        t.copy_(torch.from_numpy(v.astype(np.float32)).to(dev))
        return t, flat

    x, W, r, g = (q(rng.standard_normal(s)) for s in ((N, K), (K, M), (N, M), (N, M)))
    W = q(W / K ** 0.5)
    b = rng.standard_normal(M).astype(np.float32)
    m = D.mask(N, M, 0.2, 7, 9)
    tx, tW, tr, tg = rows_at(x, 3)[0], rows_at(W, 0)[0], rows_at(r, 5)[0], rows_at(g, 1)[0]
    tb = torch.cat([torch.zeros(1), torch.from_numpy(b)]).to(dev)[1:]
    out, flat = rows_at(np.zeros((N, M)), 1)
    cg.linear_act_fwd(tx, tW, tb, "tanh", residual=tr, p_drop=0.2, seed=7, offset=9, out=out, save=False)
    wy, wz = D.linear_fwd(x, W, b, r, "tanh", m)
    tz = (steps(dtype) * K + 4) * U * (np.abs(x).astype(np.float64) @ np.abs(W).astype(np.float64)) + 2 * U * np.abs(wz)
    ty = 1.1 * m * tz + 8 * U * m * np.maximum(1, np.abs(wz)) + 3 * U * (np.abs(wy) + np.abs(r))
    near("y", out, wy, ty + HALF[dtype] * np.abs(wy), dtype, K, extra=16 * U)
    assert int(torch.isnan(flat).sum()) == flat.numel() - N * M
    z = q(wz.astype(np.float32))
    zt = rows_at(z, 0)[0]
    gx, flat = rows_at(np.zeros((N, K)), 1)
    dx, dW, db = cg.linear_act_bwd(tx, tW, zt, tg, "tanh", p_drop=0.2, seed=7, offset=9, grad_x=gx)
    wdx, wdW, wdb, dz = D.linear_bwd(x, W, z, g, "tanh", m)
    e = np.abs(dz) * 2 * U + 16 * U * (1 + np.abs(z)) * np.abs(g) * m
    rounded = e + (HALF["bf16"] * np.abs(dz) if dtype == "bf16" else 0)
    aW, ax = np.abs(W).astype(np.float64).T, np.abs(x).astype(np.float64).T
    near("dx", dx, wdx, rounded @ aW + (steps(dtype) * M + 4) * U * (np.abs(dz) @ aW) + (HALF[dtype] + 2 * U) * np.abs(wdx),
         dtype, M, extra=16 * U)
    near("dW", dW, wdW, ax @ rounded + (steps(dtype) * N + 4) * U * (ax @ np.abs(dz)) + (HALF[dtype] + 2 * U) * np.abs(wdW),
         dtype, N, extra=16 * U)
    near("db", db, wdb, e.sum(0) + 2 * U * np.abs(wdb) + N * 2.0 ** -53 * np.abs(dz).sum(0), "bf16", N)
    assert int(torch.isnan(flat).sum()) == flat.numel() - N * K


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,M", [(3, 65536, 8), (40, 65536, 24), (5, 8, 65536), (300, 16, 65536), (260, 65536, 16)])
def test_linear_widest(tt, N, K, M, dtype):
    """The largest widths: rows that pick one input each give that row of W, and one output's
    gradient gives that column (exact: one term of each product is not zero)."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[linear] widest N={N} K={K} M={M} {dtype}", flush=True)
    dt = _dt(torch, dtype)
    W = torch.randn(K, M, device=dev).to(dt)
    at = (torch.arange(N, device=dev) * 7919 + K - 1) % K
    x = torch.zeros(N, K, device=dev, dtype=dt)
    x[torch.arange(N, device=dev), at] = 1.0
    assert torch.equal(cg.linear_act_fwd(x, W, act="none")[0], W[at])
    to = (torch.arange(N, device=dev) * 4001 + M - 1) % M
    g = torch.zeros(N, M, device=dev, dtype=dt)
    g[torch.arange(N, device=dev), to] = 1.0
    dx, dW, db = cg.linear_act_bwd(x, W, None, g, act="none")
    assert torch.equal(dx, W.t()[to])
    want = torch.zeros(K, M, device=dev).index_put_((at, to), torch.ones(N, device=dev), accumulate=True)
    assert torch.equal(dW.float(), want) and torch.equal(db, g.float().sum(0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,M", [(4, 600, 72), (300, 64, 136), (40, 200, 48), (1100, 1024, 1032), (5000, 72, 264),
                                   (9000, 48, 200), (700, 300, 128), (70, 33, 35)])
def test_infinities_reach_only_their_results(tt, N, K, M, dtype):
    """An infinity or NaN in a column of W spoils that column of y and that input's dx; in x, that row of y
    and that row of dW; in the gradient, that row of dx, that column of dW and that sum: all else is what it was."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    dt = _dt(torch, dtype)
    print(f"[linear] infinities N={N} K={K} M={M} {dtype}", flush=True)
    x, W, g = (torch.randn(*s, device=dev).to(dt) for s in ((N, K), (K, M), (N, M)))
    run = lambda x, W, g: (cg.linear_act_fwd(x, W, act="none")[0],) + cg.linear_act_bwd(x, W, None, g, act="none")  # noqa: E731
    clean = run(x, W, g)
    n, k, c = N - 2, K // 2, M - 3
    for bad in (float("inf"), float("nan")):
        for which in "xWg":
            a = {"x": x.clone(), "W": W.clone(), "g": g.clone()}
            a[which][{"x": (n, k), "W": (k, c), "g": (n, c)}[which]] = bad
            hit = [torch.zeros_like(v, dtype=torch.bool) for v in clean]     # y, dx, dW, db
            if which == "x":
                hit[0][n], hit[2][k] = True, True
            elif which == "W":
                hit[0][:, c], hit[1][:, k] = True, True
            else:
                hit[1][n], hit[2][:, c], hit[3][c] = True, True, True
            for name, u, v, h in zip(("y", "dx", "dW", "db"), run(a["x"], a["W"], a["g"]), clean, hit):
                assert torch.equal(u[~h], v[~h]), (which, bad, name)
                assert not torch.isfinite(u[h]).any(), (which, bad, name)
