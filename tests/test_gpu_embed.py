"""GPU parity of the embedding and of its table's gradient against the oracle
in 64 bits.

Tolerances, with the unit roundoffs 2^-24 of fp32 and 2^-8 of bf16.  Forward:
one fp32 product, rounded once more to bf16.  Gradient: fp64 sums of the given
values, one rounding to fp32 (the scaled sum) and one more to bf16, plus the
fp64 sum's own error, at most n 2^-53 times the sum of the magnitudes.  Two
fp32 roundoffs and one of bf16 are allowed (2 EPS below), and twice the sum's.
"""
import numpy as np
import pytest

from tests import train_oracle as T

pytestmark = pytest.mark.gpu
EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -9 + 2.0 ** -24}


@pytest.fixture(scope="module")
def tt():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch, torch.device("cuda:0")


def _dt(torch, dtype):
    return torch.float32 if dtype == "f32" else torch.bfloat16


def draw_ids(rng, kind, N, V):
    if kind == "uniform":
        return rng.integers(0, V, N).astype(np.int32)
    if kind == "one":
        return np.full(N, V - 1, np.int32)
    if kind == "few":
        return (rng.integers(0, 5, N) ** 2 % V).astype(np.int32)
    if kind == "sorted":
        return np.sort(rng.integers(0, V, N)).astype(np.int32)
    if kind == "padding":
        return rng.choice(np.array([-1, -2**31, V, 2**31 - 1], np.int64), N).astype(np.int32)
    # half padding, a hot id, the rest anywhere
    v = rng.integers(0, V, N)
    v[rng.random(N) < 0.4] = V // 2
    v[rng.random(N) < 0.5] = -1
    return v.astype(np.int32)


def check(got, want, mass, n, dtype):
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - want)
    tol = 2 * (EPS[dtype] * np.abs(want) + n * 2.0 ** -53 * mass) + 1e-38
    assert np.all(err <= tol), float((err / tol).max())


CASES = [("uniform", 1, 1, 1, 1), ("uniform", 0, 7, 8, 1), ("uniform", 2, 300, 3, 2), ("one", 65, 1, 128, 1),
         ("few", 2000, 89, 128, 9), ("mixed", 2047, 89, 130, 1), ("mixed", 2049, 255, 64, 1),
         ("uniform", 4097, 256, 40, 1), ("one", 5000, 257, 17, 3), ("sorted", 3001, 65536, 33, 1),
         ("mixed", 16385, 70001, 96, 1), ("padding", 999, 50, 24, 1), ("uniform", 33, 2**24 + 3, 1, 1),
         ("few", 300, 11, 2056, 1), ("mixed", 70, 9, 4100, 2), ("one", 100003, 3, 8, 1),
         # either side of what the gradient does in one launch; narrow rows, many groups to a block
         ("mixed", 4096, 4096, 36, 1), ("mixed", 4097, 4096, 36, 1), ("uniform", 4096, 4097, 20, 1),
         ("few", 3999, 4097, 128, 4), ("sorted", 4095, 700, 8, 1), ("one", 4096, 511, 7, 1), ("sorted", 257, 512, 16, 1),
         ("few", 30000, 70000, 8, 1), ("mixed", 20000, 300, 4, 1), ("sorted", 9000, 5000, 3, 2),
         ("sorted", 26001, 900, 12, 1),
         # ids that span some hundred runs
         ("one", 6000, 5000, 1024, 1), ("few", 9000, 7, 1024, 1), ("sorted", 5000, 3, 1032, 1),
         # few ids, wide rows of either access
         ("few", 409, 138, 1778, 1), ("mixed", 3000, 60, 4104, 2), ("mixed", 1500, 200, 1027, 1), ("sorted", 4096, 40, 8200, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,N,V,C,pitch", CASES)
def test_embed(tt, kind, N, V, C, pitch, dtype):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[embed] {kind} N={N} V={V} C={C} pitch={pitch} {dtype}", flush=True)
    rng = np.random.default_rng(N + V + C)
    ids = draw_ids(rng, kind, N, V)
    ti = torch.from_numpy(ids).to(dev)
    scale = float(np.float32(1.7))
    table = torch.randn(V, C, device=dev).to(_dt(torch, dtype))
    wide = torch.full((N, pitch, C), 7.0, device=dev, dtype=table.dtype)
    out = cg.embed_fwd(ti, table, scale, out=wide[:, 0, :])
    want = T.embed_fwd(ids, table.float().cpu().numpy(), scale)
    check(out, want, 0.0, 0, dtype)
    assert (wide[:, 1:, :] == 7.0).all()
    g = torch.randn(N, pitch, C, device=dev).to(table.dtype)[:, pitch - 1, :]
    got = cg.embed_bwd(ti, g, V, scale)
    gh = g.float().cpu().numpy()
    want = T.embed_bwd(ids, gh, V, scale)
    check(got, want, T.embed_bwd(ids, np.abs(gh), V, scale), N, dtype)
    assert torch.equal(got, cg.embed_bwd(ti, g, V, scale))      # the same bits every time


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_embed_unaligned_rows(tt, dtype):
    """Arrays aligned to their elements only: one element into an allocation,
    and a row stride that is no multiple of 16 bytes."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    rng = np.random.default_rng(5)
    N, V, C = 517, 40, 32
    ids = draw_ids(rng, "mixed", N, V)
    ti = torch.from_numpy(ids).to(dev)
    table = torch.randn(V * C + 1, device=dev).to(_dt(torch, dtype))[1:].view(V, C)
    out = torch.zeros(N, C + 1, device=dev, dtype=table.dtype)[:, 1:]
    cg.embed_fwd(ti, table, 0.5, out=out)
    check(out, T.embed_fwd(ids, table.float().cpu().numpy(), 0.5), 0.0, 0, dtype)
    g = torch.randn(N, C + 3, device=dev).to(table.dtype)[:, 2:-1]
    gt = torch.empty(V * C + 1, device=dev, dtype=table.dtype)[1:].view(V, C)
    cg.embed_bwd(ti, g, V, 0.5, grad_table=gt)
    gh = g.float().cpu().numpy()
    check(gt, T.embed_bwd(ids, gh, V, 0.5), T.embed_bwd(ids, np.abs(gh), V, 0.5), N, dtype)


def test_embed_nonfinite_values_stay_in_their_rows(tt):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    ids = torch.tensor([0, 2, -1, 2, 1], dtype=torch.int32, device=dev)
    g = torch.ones(5, 8, device=dev)
    g[2] = float("nan")                 # a padded row: ignored
    g[0, 0], g[1, 1], g[3, 1] = float("inf"), float("inf"), float("-inf")
    got = cg.embed_bwd(ids, g, 4, 2.0).cpu()
    assert got[0, 0] == float("inf") and torch.isnan(got[2, 1])
    assert torch.isfinite(got).sum() == 4 * 8 - 2
    assert (got[3] == 0).all() and (got[1] == 2).all()
    table = torch.full((3, 8), float("nan"), device=dev)
    assert (cg.embed_fwd(torch.full((3,), 3, dtype=torch.int32, device=dev), table) == 0).all()


def test_embed_gradient_against_differences(tt):
    """The gradient's product with a direction is the difference quotient of
    the oracle's forward along it (linear: exact up to rounding)."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    rng = np.random.default_rng(11)
    ids = draw_ids(rng, "mixed", 700, 30)
    g = rng.standard_normal((700, 24)).astype(np.float32)
    d = rng.standard_normal((30, 24))
    got = cg.embed_bwd(torch.from_numpy(ids).to(dev), torch.from_numpy(g).to(dev), 30, 3.0).double().cpu().numpy()
    f = lambda t: (g.astype(np.float64) * T.embed_fwd(ids, t, 3.0)).sum()  # noqa: E731
    want = (f(d) - f(-d)) / 2
    mass = (np.abs(got) * np.abs(d)).sum()
    assert abs((got * d).sum() - want) <= 2 * EPS["f32"] * mass


def test_embed_on_another_stream_and_in_a_graph(tt):
    """The calls run on the current stream and replay from a captured graph:
    every replay, between eager calls, equals the eager result."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    rng = np.random.default_rng(3)
    N, V, C = 3000, 500, 64
    ids = torch.from_numpy(draw_ids(rng, "mixed", N, V)).to(dev)
    table, g = torch.randn(V, C, device=dev), torch.randn(N, C, device=dev)
    want = cg.embed_fwd(ids, table, 2.0), cg.embed_bwd(ids, g, V, 2.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, gt = torch.empty(N, C, device=dev), torch.empty(V, C, device=dev)
    ws = torch.empty(cg.embed_bwd_workspace_size(torch.float32, N, V, C), dtype=torch.uint8, device=dev)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cg.embed_fwd(ids, table, 2.0, out=out)
        cg.embed_bwd(ids, g, V, 2.0, grad_table=gt, ws=ws)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(gt, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cg.embed_fwd(ids, table, 2.0, out=out)
        cg.embed_bwd(ids, g, V, 2.0, grad_table=gt, ws=ws)
    for k in range(3):
        g.copy_(torch.randn(N, C, device=dev))
        ids.copy_(torch.from_numpy(draw_ids(rng, ("few", "one", "uniform")[k], N, V)).to(dev))
        out.zero_()
        gt.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, cg.embed_fwd(ids, table, 2.0)), k
        assert torch.equal(gt, cg.embed_bwd(ids, g, V, 2.0)), k


@pytest.mark.parametrize("N,V,C", [(3, 5, 8), (3000, 90, 24), (6000, 5000, 16), (6000, 5000, 1032), (30000, 70000, 3),
                                   (70001, 70000, 8)])
def test_embed_gradient_is_rounded_once(tt, N, V, C):
    """1 + 2^-8 + 2^-30 lies just above the middle of two bf16 numbers: rounded
    once it is 1 + 2^-7; through fp32, where it is the middle, it would be 1.
    Mirrored below zero, and 1 + 2^-8 - 2^-30 the other way.  One id's rows lie
    together, another's span the whole batch."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[embed] rounding {N} {V} {C}", flush=True)
    g = np.zeros((N, C))
    ids = np.full(N, V - 1, np.int32)       # a hot id
    ids[:3] = 0                             # three rows of their own
    terms = np.array([1.0, 2.0 ** -8, 2.0 ** -30])[:, None] * np.where(np.arange(C) % 2, -1.0, 1.0)
    terms[2] *= np.where(np.arange(C) % 3 == 2, -1.0, 1.0)
    g[:3] = terms
    if N > 3:
        g[[3, N // 2, N - 1]] = terms
    want = np.where(np.arange(C) % 3 == 2, 1.0, 1 + 2.0 ** -7) * np.where(np.arange(C) % 2, -1.0, 1.0)
    got = cg.embed_bwd(torch.from_numpy(ids).to(dev), torch.from_numpy(g).to(dev).bfloat16(), V).float().cpu().numpy()
    assert np.array_equal(got[0], want) and (N == 3 or np.array_equal(got[V - 1], want))
    big = torch.full((2, C), 3.38e38, device=dev).bfloat16()
    got = cg.embed_bwd(torch.zeros(2, dtype=torch.int32, device=dev), big, 2)
    assert torch.isinf(got[0]).all() and (got[1] == 0).all()     # beyond the type: infinity


# Sorts by tiles of 1024 ids: up to 64 tiles (65536 ids) and more, more than 256 of them (262144 ids, whose counts are
# summed in several rounds), one, two and three passes of 9 bits, and many digits in use in each.
TILED = [("uniform", 65536, 300, 4, 1), ("uniform", 65537, 300, 4, 1), ("mixed", 70001, 70000, 8, 1),
         ("uniform", 270000, 600, 8, 1), ("uniform", 300001, 100000, 4, 1), ("mixed", 270001, 400, 3, 2),
         ("sorted", 262145, 511, 4, 1), ("few", 300000, 2 ** 20, 4, 1), ("uniform", 66000, 2 ** 19, 4, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,N,V,C,pitch", TILED)
def test_embed_gradient_of_many_ids(tt, kind, N, V, C, pitch, dtype):
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[embed] many {kind} N={N} V={V} C={C} pitch={pitch} {dtype}", flush=True)
    rng = np.random.default_rng(N + V)
    ids = draw_ids(rng, kind, N, V)
    ti = torch.from_numpy(ids).to(dev)
    g = torch.randn(N, pitch, C, device=dev).to(_dt(torch, dtype))[:, pitch - 1, :]
    got = cg.embed_bwd(ti, g, V, 0.5)
    gh = g.float().cpu().numpy()
    check(got, T.embed_bwd(ids, gh, V, 0.5), T.embed_bwd(ids, np.abs(gh), V, 0.5), N, dtype)
    assert torch.equal(got, cg.embed_bwd(ti, g, V, 0.5))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_embed_offsets_beyond_32_bits(tt, dtype):
    """Tables and rows of more than 2^31 elements: the last rows are read and
    written at their own places."""
    torch, dev = tt
    import clebsch_gordan_tensor_cgtp_amd as cg
    print(f"[embed] beyond 32 bits {dtype}", flush=True)
    V, C, N = (1 << 22) + 37, 520, 3000     # a table of 2.18e9 elements
    rng = np.random.default_rng(1)
    ids = np.concatenate([[0, V - 1, V, -1, V - 2, 1 << 21], rng.integers(V - 500, V, N - 6)]).astype(np.int32)
    ti = torch.from_numpy(ids).to(dev)
    table = torch.zeros(V, C, device=dev, dtype=_dt(torch, dtype))
    table[V - 500:] = torch.randn(500, C, device=dev)
    table[0], table[1 << 21] = 3.0, 5.0
    rows = np.unique(ids[(ids >= 0) & (ids < V)])
    at = {int(v): k for k, v in enumerate(rows)}
    small = np.array([at.get(int(i), -1) for i in ids], np.int32)
    tr = torch.from_numpy(rows).to(dev).long()
    out = cg.embed_fwd(ti, table, 0.5)
    check(out, T.embed_fwd(small, table[tr].float().cpu().numpy(), 0.5), 0.0, 0, dtype)
    del table
    g = torch.randn(N, C, device=dev).to(_dt(torch, dtype))
    got = cg.embed_bwd(ti, g, V, 0.5)
    gh = g.float().cpu().numpy()
    check(got[tr], T.embed_bwd(small, gh, len(rows), 0.5), T.embed_bwd(small, np.abs(gh), len(rows), 0.5), N, dtype)
    got[tr] = 0
    assert not got.any()
    del got
    # rows of 2^23 elements apart
    n = 300
    wide = torch.full((n, 1 << 23), 7.0, device=dev, dtype=g.dtype)
    few = torch.randn(9, 64, device=dev).to(g.dtype)
    ids = rng.integers(0, 9, n).astype(np.int32)
    cg.embed_fwd(torch.from_numpy(ids).to(dev), few, 2.0, out=wide[:, :64])
    check(wide[:, :64], T.embed_fwd(ids, few.float().cpu().numpy(), 2.0), 0.0, 0, dtype)
    assert (wide[:, 64:] == 7.0).all()
    gh = wide[:, :64].float().cpu().numpy()
    got = cg.embed_bwd(torch.from_numpy(ids).to(dev), wide[:, :64], 9, 1.0)
    check(got, T.embed_bwd(ids, gh, 9, 1.0), T.embed_bwd(ids, np.abs(gh), 9, 1.0), n, dtype)
