"""GPU parity of the group normalisation with an activation, forward and
backward, against the oracle in 64 bits.

Tolerances, in units u = 2^-24.  mean and rstd are fp64 sums rounded once:
mean within 2 u |mean| (+ 2 u), rstd within 2 u rstd plus the fp64
cancellation.  An element passes through x - mean (the rounded mean is off by
u |mean|), two products, an addition and an activation with slope at most 1.1
whose own evaluation is good to about 8 u max(1, |z|): in all at most
16 u (|gamma| (1 + |xhat| + |mean| rstd) + |beta| + 1).  dx goes through the
same chain times |dy| and rstd, plus the group means: 32 u rstd (|h| + |s1| +
|xhat s2| + the mean term).  The channel sums add n such terms in fp64.  bf16
results carry 2^-9 relative on top.
"""
import numpy as np
import pytest

from tests import train_oracle as T

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def tt():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch, torch.device("cuda:0")


def lengths(rng, kind, N, B):
    if kind == "equal":
        assert N % B == 0
        return np.full(B, N // B)
    if kind == "one":
        v = np.zeros(B, np.int64)
        v[B // 2] = N
        return v
    w = rng.random(B) ** 4 + 1e-9
    w[rng.random(B) < 0.3] = 0
    w[0] += 1e-9
    cut = np.floor(np.cumsum(w) / w.sum() * N).astype(np.int64)
    cut[-1] = N
    return np.diff(np.concatenate([[0], cut]))


def bounds(x, gamma, beta, grad, ptr, G, eps, kind):
    """(tolerances of y, of dx, of dgamma and of dbeta before rounding to bf16)"""
    C = x.shape[1]
    mean, rstd = T.norm_stats(x, ptr, G, eps)
    mu, rs = T._spread(mean, ptr, C), T._spread(rstd, ptr, C)
    xhat = np.abs((x - mu) * rs)
    off = 1 + xhat + np.abs(mu) * rs
    ty = 16 * U * (np.abs(gamma) * off + np.abs(beta) + 1)
    e = np.abs(grad) * (1 + ty / U / 16)     # |dz| and what an error of z does to it
    h = e * np.abs(gamma)
    s = np.zeros_like(h)
    for i, j in zip(ptr, ptr[1:]):
        if j > i:
            hs, xs = (v[i:j].reshape(j - i, G, C // G) for v in (h, off))
            s[i:j] = (hs.mean((0, 2), keepdims=True) + xs * (hs * xs).mean((0, 2), keepdims=True)).reshape(j - i, C)
    return ty, 32 * U * rs * (h * off + s), 32 * U * (e * off).sum(0), 32 * U * e.sum(0)


CASES = [("equal", 1, 1, 1, 1, 1), ("equal", 4, 4, 8, 2, 1), ("equal", 6, 2, 128, 8, 1), ("one", 2000, 1, 128, 8, 9),
         ("ragged", 2500, 100, 128, 8, 1), ("ragged", 777, 300, 96, 32, 4), ("ragged", 3000, 3, 40, 8, 1),
         ("ragged", 500, 7, 6, 2, 1), ("ragged", 401, 5, 30, 10, 2), ("equal", 35000, 5, 16, 1, 1),
         ("ragged", 300, 4, 1536, 3, 1), ("ragged", 200, 3, 2050, 2, 1), ("ragged", 90, 2, 4104, 1, 1),
         ("one", 70, 2000, 24, 4, 1), ("ragged", 1, 3, 8, 8, 1), ("ragged", 65000, 30, 8, 8, 1),
         ("ragged", 2048, 1500, 64, 64, 1), ("equal", 300, 3, 333, 9, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", range(len(CASES)))
def test_norm(tt, k, dtype):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    kind, N, B, C, G, pitch = CASES[k]
    act, eps = ("none", "silu", "tanh")[k % 3], 1e-5
    print(f"[norm] {kind} N={N} B={B} C={C} G={G} pitch={pitch} {act} {dtype}", flush=True)
    rng = np.random.default_rng(k)
    ptr = np.concatenate([[0], np.cumsum(lengths(rng, kind, N, B))])
    q = T.bf16 if dtype == "bf16" else (lambda v: v.astype(np.float32))
    x = q(rng.standard_normal((N, C)) * (0.5 + rng.random(C)) + 2 * rng.standard_normal(C))
    grad = q(rng.standard_normal((N, C)))
    gamma, beta = ((1 + 0.3 * rng.standard_normal(C)).astype(np.float32), rng.standard_normal(C).astype(np.float32))
    dt = torch.float32 if dtype == "f32" else torch.bfloat16

    def rows(v):        # every pitch-th row of a wider array
        t = torch.full((N, pitch, C), float("nan"), dtype=dt, device=dev)
        t[:, 0, :] = torch.from_numpy(v).to(dev)
        return t[:, 0, :]

    tx, tg = rows(x), rows(grad)
    seg = torch.from_numpy(ptr.astype(np.int32)).to(dev)
    if kind == "equal":
        tx, tg, seg = tx.view(B, N // B, C), tg.view(B, N // B, C), None
    tgm, tbt = torch.from_numpy(gamma).to(dev), torch.from_numpy(beta).to(dev)
    y, mean, rstd = cg.norm_act_fwd(tx, tgm, tbt, G, seg, eps, act)
    dx, dg, db = cg.norm_act_bwd(tx, mean, rstd, tgm, tbt, tg, G, seg, act)
    wy, wm, wr = T.norm_fwd(x, gamma, beta, ptr, G, eps, act)
    wdx, wdg, wdb = T.norm_bwd(x, gamma, beta, grad, ptr, G, eps, act)
    ty, tdx, tdg, tdb = bounds(x.astype(np.float64), gamma, beta, grad, ptr, G, eps, act)
    r = 2.0 ** -8 if dtype == "bf16" else 2 * U
    for name, got, want, tol in (("mean", mean, wm, 2 * U * np.abs(wm) + 2 * U), ("rstd", rstd, wr, 4 * U * wr),
                                 ("y", y, wy, ty + r * np.abs(wy)), ("dx", dx, wdx, tdx + r * np.abs(wdx)),
                                 ("dgamma", dg, wdg, tdg + 2 * U * np.abs(wdg)),
                                 ("dbeta", db, wdb, tdb + 2 * U * np.abs(wdb))):
        g = got.float().cpu().numpy().astype(np.float64).reshape(want.shape)
        err = np.abs(g - want)
        assert np.all(err <= tol), (name, float((err / np.maximum(tol, 1e-300)).max()))
    again = cg.norm_act_bwd(tx, mean, rstd, tgm, tbt, tg, G, seg, act)
    assert torch.equal(y, cg.norm_act_fwd(tx, tgm, tbt, G, seg, eps, act)[0])
    assert all(torch.equal(u, v) for u, v in zip((dx, dg, db), again))


def test_norm_without_affine_and_partial_gradients(tt):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    x, g = torch.randn(300, 64, device=dev), torch.randn(300, 64, device=dev)
    one, zero = torch.ones(64, device=dev), torch.zeros(64, device=dev)
    y, m, r = cg.norm_act_fwd(x, None, None, 4)
    assert torch.equal(y, cg.norm_act_fwd(x, one, zero, 4)[0])
    full = cg.norm_act_bwd(x, m, r, one, zero, g, 4)
    for want in (("x",), ("gamma",), ("beta",), ("x", "beta"), ()):
        got = cg.norm_act_bwd(x, m, r, None, None, g, 4, want=want)
        for name, a, b in zip(("x", "gamma", "beta"), got, full):
            assert (a is None) == (name not in want)
            assert a is None or torch.equal(a, b), name


def test_norm_of_no_rows(tt):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    x, w = torch.zeros(0, 16, device=dev), torch.ones(16, device=dev)
    seg = torch.zeros(4, dtype=torch.int32, device=dev)
    y, m, r = cg.norm_act_fwd(x, w, w, 2, seg, eps=0.25)
    assert y.shape == (0, 16) and (m == 0).all() and (r == 2).all()
    dx, dg, db = cg.norm_act_bwd(x, m, r, w, w, x, 2, seg)
    assert dx.shape == (0, 16) and (dg == 0).all() and (db == 0).all()
    y, m, r = cg.norm_act_fwd(x, w, w, 2, seg[:1])
    assert y.shape == (0, 16) and m.shape == (0, 2)
    assert all((t == 0).all() for t in cg.norm_act_bwd(x, m, r, w, w, x, 2, seg[:1])[1:])


def test_norm_keeps_nonfinite_values_in_their_group(tt):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    x = torch.randn(90, 32, device=dev)
    seg = torch.tensor([0, 30, 60, 90], dtype=torch.int32, device=dev)
    w = torch.ones(32, device=dev)
    ref, rm, rr = cg.norm_act_fwd(x, w, w, 4, seg)
    x[40, 9], x[70, 31] = float("nan"), float("inf")
    y, m, r = cg.norm_act_fwd(x, w, w, 4, seg)
    hit = torch.zeros(90, 32, dtype=torch.bool, device=dev)
    hit[30:60, 8:16] = True
    hit[60:90, 24:32] = True
    assert torch.equal(y[~hit], ref[~hit]) and torch.isnan(y[30:60, 8:16]).all() and torch.isnan(y[60:90, 24:32]).all()
    bad = torch.zeros(3, 4, dtype=torch.bool, device=dev)
    bad[1, 1] = bad[2, 3] = True
    assert torch.equal(m[~bad], rm[~bad]) and torch.equal(r[~bad], rr[~bad])


def test_norm_large_offset(tt):
    """Values far from zero beside their spread: the variance is formed in 64
    bits, so only the mean's own rounding is lost."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    rng = np.random.default_rng(8)
    x = (1000 + 0.01 * rng.standard_normal((512, 16))).astype(np.float32)
    one = np.ones(16)
    y, m, r = cg.norm_act_fwd(torch.from_numpy(x).to(dev), None, None, 2, act="none", eps=1e-8)
    wy, wm, wr = T.norm_fwd(x, one, 0 * one, np.array([0, 512]), 2, 1e-8, "none")
    assert np.abs(r.cpu().numpy() / wr - 1).max() <= 4 * U + 512 * 8 * 2.0 ** -53 * 1e6 / 1e-4
    err = np.abs(y.cpu().numpy() - wy)
    assert np.all(err <= 16 * U * (2 + np.abs(wy) + np.abs(wm).max() * wr.max()))


def test_norm_malformed_offsets_stay_in_bounds(tt):
    """Offsets that break the precondition (unsorted, beyond the rows,
    negative): every index is clamped, the call returns."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    x, w = torch.randn(200, 32, device=dev), torch.ones(32, device=dev)
    for bad in ([0, 150, 50, 200], [0, 500, 700, 900], [-5, -3, 10, 2000], [200, 200, 200, 200], [0, 0, 0, 0]):
        seg = torch.tensor(bad, dtype=torch.int32, device=dev)
        y, m, r = cg.norm_act_fwd(x, w, w, 4, seg)
        cg.norm_act_bwd(x, torch.zeros(3, 4, device=dev), torch.ones(3, 4, device=dev), w, w, x, 4, seg)
        torch.cuda.synchronize()
        assert y.shape == x.shape


def test_norm_gradient_against_differences(tt):
    """The GPU gradients' product with a direction is the difference quotient
    of the oracle's forward along it (step 1e-5 in 64 bits: error about 1e-9)."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    rng = np.random.default_rng(21)
    ptr, G, C = np.array([0, 50, 50, 51, 140]), 4, 32
    x, g = (rng.standard_normal((140, C)).astype(np.float32) for _ in range(2))
    gamma, beta = (rng.standard_normal(C).astype(np.float32) for _ in range(2))
    t = [torch.from_numpy(v).to(dev) for v in (x, gamma, beta, g, ptr.astype(np.int32))]
    y, m, r = cg.norm_act_fwd(t[0], t[1], t[2], G, t[4], 1e-3, "silu")
    grads = cg.norm_act_bwd(t[0], m, r, t[1], t[2], t[3], G, t[4], "silu")
    _, tdx, tdg, tdb = bounds(x.astype(np.float64), gamma, beta, g, ptr, G, 1e-3, "silu")
    for k, (got, tol) in enumerate(zip(grads, (tdx, tdg, tdb))):
        args = [v.astype(np.float64) for v in (x, gamma, beta)]
        d, at, h = rng.standard_normal(args[k].shape), args[k], 1e-5

        def f(v):
            args[k] = v
            return (g.astype(np.float64) * T.norm_fwd(*args, ptr, G, 1e-3, "silu")[0]).sum()

        want = (f(at + h * d) - f(at - h * d)) / (2 * h)
        assert abs((got.double().cpu().numpy() * d).sum() - want) <= (tol * np.abs(d)).sum() + 1e-6 * abs(want), k


def test_norm_on_another_stream_and_in_a_graph(tt):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    x, g = torch.randn(1000, 64, device=dev), torch.randn(1000, 64, device=dev)
    w = torch.randn(64, device=dev)
    seg = torch.tensor([0, 10, 10, 700, 1000], dtype=torch.int32, device=dev)
    step = lambda: (lambda y, m, r: (y, m, r) + cg.norm_act_bwd(x, m, r, w, w, g, 8, seg))(  # noqa: E731
        *cg.norm_act_fwd(x, w, w, 8, seg))
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(3):
        x.copy_(torch.randn(1000, 64, device=dev) + k)
        seg.copy_(torch.tensor([0, 300 * k, 900, 900, 1000], dtype=torch.int32, device=dev))
        for o in outs:
            o.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, step())), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,C,G", [(3, 60, 32, 4), (1, 2000, 128, 8), (2, 40000, 32, 4), (1, 30001, 24, 3)])
def test_norm_of_values_whose_squares_leave_fp32(tt, B, N, C, G, dtype):
    """Values of up to 1e20 or so, whose squares fp32 does not hold: statistics
    and results as for any other magnitude, in segments that a block takes
    whole and in those cut into runs.  (Tolerances as above; the mean, a sum
    that nearly cancels, to fp64's roundoff of the deviation too.)"""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[norm] large values {B} {N} {C} {G} {dtype}", flush=True)
    rng = np.random.default_rng(N)
    q = T.bf16 if dtype == "bf16" else (lambda v: v.astype(np.float32))
    x = q(3e19 * (rng.standard_normal((N, C)) + rng.standard_normal(C)))
    gamma, beta = ((1 + 0.3 * rng.standard_normal(C)).astype(np.float32), rng.standard_normal(C).astype(np.float32))
    t = torch.from_numpy(x).to(dev).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    y, mean, rstd = cg.norm_act_fwd(t.view(B, N // B, C), torch.from_numpy(gamma).to(dev),
                                    torch.from_numpy(beta).to(dev), G, act="none")
    ptr = np.arange(B + 1) * (N // B)
    wy, wm, wr = T.norm_fwd(x, gamma, beta, ptr, G, 1e-5, "none")
    ty = bounds(x.astype(np.float64), gamma, beta, np.zeros_like(x), ptr, G, 1e-5, "none")[0]
    r = 2.0 ** -8 if dtype == "bf16" else 2 * U
    host = lambda v: v.double().cpu().numpy()  # noqa: E731
    assert np.all(np.abs(host(rstd) - wr) <= 4 * U * wr)
    assert np.all(np.abs(host(mean) - wm) <= 2 * U * np.abs(wm) + 2.0 ** -40 / wr)
    assert np.all(np.abs(host(y).reshape(N, C) - wy) <= ty + r * np.abs(wy))


@pytest.mark.parametrize("N,C,G", [(20000, 16, 2), (30001, 30, 3)])
def test_norm_large_offset_in_long_segments(tt, N, C, G):
    """As test_norm_large_offset, in a segment that is cut into runs: at most 512
    lane sums and 1024 runs' sums are added after a lane's own, each to fp64's
    roundoff of the squared mean."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    x = (1000 + 0.01 * np.random.default_rng(9).standard_normal((N, C))).astype(np.float32)
    one = np.ones(C)
    y, m, r = cg.norm_act_fwd(torch.from_numpy(x).to(dev), None, None, G, act="none", eps=1e-8)
    wy, wm, wr = T.norm_fwd(x, one, 0 * one, np.array([0, N]), G, 1e-8, "none")
    off = 1536 * 2.0 ** -53 * 1e6 / 1e-4
    assert np.abs(r.cpu().numpy() / wr - 1).max() <= 4 * U + off
    assert np.abs(m.cpu().numpy() / wm - 1).max() <= 2 * U
    err = np.abs(y.cpu().numpy() - wy)
    assert np.all(err <= 16 * U * (2 + np.abs(wy) + np.abs(wm).max() * wr.max()) + off * np.abs(wy))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,C,G", [(3, 60, 32, 4), (40, 4000, 64, 8), (1, 2000, 128, 8), (1, 40000, 16, 2),
                                     (2, 30002, 30, 3)])
def test_norm_gradient_sums_are_64_bit(tt, B, N, C, G, dtype):
    """Rows of 2^30, -2^30 and 1 in turn at random: fp64 holds every partial sum
    exactly, so what is left is the number of ones, where fp32 would lose a
    one beside a large row.  (mean 0 and rstd 1 are given and x is 1, so that
    xhat is 1 and both sums have the same terms.)"""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[norm] sums {B} {N} {C} {G} {dtype}", flush=True)
    rng = np.random.default_rng(N + C)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    ones = N // 5 + N % 2               # the others in pairs
    ones += (N - ones) % 2
    row = np.concatenate([np.ones(ones), np.repeat([2.0 ** 30, -2.0 ** 30], (N - ones) // 2)])
    g = np.stack([rng.permutation(row) for _ in range(C)], axis=1)
    tg = torch.from_numpy(g).to(dev).to(dt).view(B, N // B, C)
    x = torch.ones(B, N // B, C, device=dev, dtype=dt)
    mean, rstd = torch.zeros(B, G, device=dev), torch.ones(B, G, device=dev)
    for want in (("x", "gamma", "beta"), ("gamma", "beta")):
        _, dg, db = cg.norm_act_bwd(x, mean, rstd, None, None, tg, G, act="none", want=want)
        assert (db == ones).all() and (dg == ones).all(), (want, db[:4].tolist(), ones)
    # the group means of dx: of a row of ones, 1 - 2 mean
    dx = cg.norm_act_bwd(x, mean, rstd, None, None, tg, G, act="none")[0].double().cpu().numpy().reshape(g.shape)
    s = g.reshape(B, N // B, G, C // G).mean((1, 3), keepdims=True)
    w = np.broadcast_to(1 - 2 * s, (B, N // B, G, C // G)).reshape(N, C)
    at = g == 1
    r = 2.0 ** -8 if dtype == "bf16" else 4 * U
    assert np.all(np.abs(dx - w)[at] <= (r * np.abs(w) + 4 * U * np.abs(1 - w))[at])


def mixed_lengths(rng, kind, N, B, longest):
    """Lengths of B segments of N rows together, where blocks take segments of up
    to `longest` rows (the backward; the forward twice that) and runs the others."""
    run = max(16, -(-N // 1024))
    v = rng.integers(1, 40, B)
    v[rng.random(B) < 0.1] = 0
    if kind == "one":                       # one long structure holds nearly all rows
        v[B // 3] = 0
        v[B // 3] = N - v.sum()
    elif kind == "several":                 # from a run's first row, next to each other, either side of the limit
        before = v[:3].sum()
        v[3] = -before % run                # the next begins with a run
        v[4:10] = longest + 1, longest, 5 * run, longest + 1 + run, 2 * longest, 2 * longest + 1
        v[-1] = longest + 2
        v[B // 2] = 0
        v[B // 2] = N - v.sum()
    else:                                   # none is long: the runs find nothing
        v = np.full(B, N // B)
        v[rng.permutation(B)[:N - v.sum()]] += 1
    assert v.sum() == N and v.min() >= 0
    return v


# Rows of C channels that together pass 32 MB, so that whole segments and runs go out in one call: in both directions,
# but the last two in the backward alone.  C = 250: no wide accesses.  B = 3000: short segments, several to a block.
MIXED = [("one", 17000, 300, 512, 8, "silu", "f32"), ("several", 17000, 300, 512, 8, "tanh", "f32"),
         ("none", 16500, 400, 512, 8, "silu", "f32"), ("several", 34000, 400, 250, 5, "silu", "f32"),
         ("one", 70000, 3000, 128, 8, "silu", "f32"), ("several", 34000, 400, 512, 32, "silu", "bf16"),
         ("one", 9000, 256, 512, 4, "none", "f32"), ("several", 18000, 300, 512, 8, "silu", "bf16")]


@pytest.mark.parametrize("kind,N,B,C,G,act,dtype", MIXED)
def test_norm_whole_segments_beside_runs(tt, kind, N, B, C, G, act, dtype):
    """Ragged batches in which blocks take the short segments and runs the long
    ones: every result against the oracle, each gradient asked for alone."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[norm] mixed {kind} N={N} B={B} C={C} G={G} {act} {dtype}", flush=True)
    rng = np.random.default_rng(N + B + C)
    es = 4 if dtype == "f32" else 2
    lens = mixed_lengths(rng, kind, N, B, (1 << 20) // (C * es * 2))
    ptr = np.concatenate([[0], np.cumsum(lens)])
    q = T.bf16 if dtype == "bf16" else (lambda v: v.astype(np.float32))
    x = q(rng.standard_normal((N, C)) * (0.5 + rng.random(C)) + 2 * rng.standard_normal(C))
    grad = q(rng.standard_normal((N, C)))
    gamma, beta = ((1 + 0.3 * rng.standard_normal(C)).astype(np.float32), rng.standard_normal(C).astype(np.float32))
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    tx, tg = (torch.from_numpy(v).to(dev).to(dt) for v in (x, grad))
    tgm, tbt, seg = (torch.from_numpy(v).to(dev) for v in (gamma, beta, ptr.astype(np.int32)))
    y, mean, rstd = cg.norm_act_fwd(tx, tgm, tbt, G, seg, act=act)
    dx, dg, db = cg.norm_act_bwd(tx, mean, rstd, tgm, tbt, tg, G, seg, act)
    wy, wm, wr = T.norm_fwd(x, gamma, beta, ptr, G, 1e-5, act)
    wdx, wdg, wdb = T.norm_bwd(x, gamma, beta, grad, ptr, G, 1e-5, act)
    ty, tdx, tdg, tdb = bounds(x.astype(np.float64), gamma, beta, grad, ptr, G, 1e-5, act)
    r = 2.0 ** -8 if dtype == "bf16" else 2 * U
    for name, got, want, tol in (("mean", mean, wm, 2 * U * np.abs(wm) + 2 * U), ("rstd", rstd, wr, 4 * U * wr),
                                 ("y", y, wy, ty + r * np.abs(wy)), ("dx", dx, wdx, tdx + r * np.abs(wdx)),
                                 ("dgamma", dg, wdg, tdg + 2 * U * np.abs(wdg)),
                                 ("dbeta", db, wdb, tdb + 2 * U * np.abs(wdb))):
        err = np.abs(got.float().cpu().numpy().astype(np.float64) - want)
        assert np.all(err <= tol), (name, float((err / np.maximum(tol, 1e-300)).max()))
    for want in (("x",), ("gamma", "beta"), ("beta",)):
        for name, a, b in zip(("x", "gamma", "beta"), cg.norm_act_bwd(tx, mean, rstd, tgm, tbt, tg, G, seg, act, want),
                              (dx, dg, db)):
            assert torch.equal(a, b) if name in want else a is None, name
    again = cg.norm_act_fwd(tx, tgm, tbt, G, seg, act=act)
    assert all(torch.equal(a, b) for a, b in zip((y, mean, rstd), again))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,B,C,pitch", [(300, 20, 64, 4), (2000, 1, 128, 9), (40000, 2, 64, 3), (17000, 300, 512, 2),
                                         (500, 7, 30, 5)])
def test_norm_gradient_into_rows_of_a_wider_array(tt, N, B, C, pitch, dtype):
    """grad_x as every pitch-th row of an array: the same values as by itself,
    the other rows left alone; whole segments, runs, and both (the rows of all
    cases begin on the same boundaries as by themselves, so that the same
    kernels run)."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[norm] grad_x {N} {B} {C} {pitch} {dtype}", flush=True)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    ptr = np.concatenate([[0], np.cumsum(lengths(np.random.default_rng(N), "ragged" if B > 1 else "one", N, B))])
    seg = torch.from_numpy(ptr.astype(np.int32)).to(dev)
    x, g = torch.randn(N, C, device=dev).to(dt), torch.randn(N, C, device=dev).to(dt)
    w = torch.randn(C, device=dev)
    y, m, r = cg.norm_act_fwd(x, w, w, 2, seg)
    want = cg.norm_act_bwd(x, m, r, w, w, g, 2, seg)
    full = torch.full((N, pitch, C), 7.0, device=dev, dtype=dt)
    for k in range(pitch):
        full.fill_(7.0)
        got = cg.norm_act_bwd(x, m, r, w, w, g, 2, seg, grad_x=full[:, k, :])
        assert got[0].data_ptr() == full[:, k, :].data_ptr()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
        assert (full[:, [q for q in range(pitch) if q != k], :] == 7.0).all(), k
    none = cg.norm_act_bwd(x, m, r, w, w, g, 2, seg, want=("gamma",), grad_x=full[:, 0, :])
    assert none[0] is None and (full[:, 0, :] == 7.0).all() and torch.equal(none[1], want[1])


@pytest.mark.parametrize("long", [False, True])
def test_norm_offsets_beyond_32_bits(tt, long):
    """Rows that together pass 2^31 elements, short segments throughout or one
    long one before them: the last segments against the oracle, and the sums
    over all rows from rows that are alike."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[norm] beyond 32 bits, long {long}", flush=True)
    C, G, S, tail = 128, 4, 40, 25
    B = (1 << 24) // S + 2 * tail           # 2.15e9 elements
    N, last = B * S, tail * S
    rng = np.random.default_rng(3)
    part, dpart = (T.bf16(rng.standard_normal((last, C)).astype(np.float32)) for _ in range(2))
    x = torch.ones(N, C, device=dev, dtype=torch.bfloat16)
    x[1::2] = -1.0                          # mean 0, deviation 1 in every even-sized segment
    g = torch.zeros_like(x)
    x[-last:] = torch.from_numpy(part).to(dev)
    g[-last:] = torch.from_numpy(dpart).to(dev)
    ptr = np.arange(B + 1, dtype=np.int64) * S
    if long:
        ptr = np.concatenate([[0], ptr[-tail - 1:]])
    seg = torch.from_numpy(ptr.astype(np.int32)).to(dev)
    gamma, beta = (rng.standard_normal(C).astype(np.float32) for _ in range(2))
    tgm, tbt = torch.from_numpy(gamma).to(dev), torch.from_numpy(beta).to(dev)
    y, m, r = cg.norm_act_fwd(x, tgm, tbt, G, seg, act="silu")
    end = np.arange(tail + 1) * S
    wy, wm, wr = T.norm_fwd(part, gamma, beta, end, G, 1e-5, "silu")
    ty, tdx, tdg, tdb = bounds(part.astype(np.float64), gamma, beta, dpart, end, G, 1e-5, "silu")
    host = lambda v: v.double().cpu().numpy()  # noqa: E731
    assert np.all(np.abs(host(y[-last:]) - wy) <= ty + 2.0 ** -8 * np.abs(wy))
    assert np.all(np.abs(host(m[-tail:]) - wm) <= 2 * U * np.abs(wm) + 2 * U)
    assert np.all(np.abs(host(r[-tail:]) - wr) <= 4 * U * wr)
    assert (m[:-tail] == 0).all() and (r[:-tail] == r[0]).all()
    for k in (0, 1):                        # all rows alike are the same bits
        rows = y[k:N - last:2]
        assert (rows == rows[0]).all()
    del y, rows
    dx, dg, db = cg.norm_act_bwd(x, m, r, tgm, tbt, g, G, seg, act="silu")
    wdx, wdg, wdb = T.norm_bwd(part, gamma, beta, dpart, end, G, 1e-5, "silu")
    assert np.all(np.abs(host(dx[-last:]) - wdx) <= tdx + 2.0 ** -8 * np.abs(wdx))
    assert np.all(np.abs(host(dg) - wdg) <= tdg + 2 * U * np.abs(wdg))
    assert np.all(np.abs(host(db) - wdb) <= tdb + 2 * U * np.abs(wdb))
    assert not dx[:-last].any()
