"""Host-side checks of dropout and of the product with its epilogue (no GPU):
the oracle's generator gives the published values and its gradients are the
derivatives of its forward, and bad arguments are refused before any HIP call."""
import ctypes

import numpy as np
import pytest
import torch

from tests import dense_oracle as D

BIG = 1 << 40
FAKE, ODD, WS, WS_ODD = (ctypes.c_void_p(v) for v in (4096, 4097, 1 << 20, (1 << 20) + 64))  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from clebsch_gordan_tensor_cgtp_amd import _lib
    _lib.lib()
    return _lib


def test_generator_gives_the_published_values():
    """The known answers of Philox4x32-10 for counters and keys of zeros, of ones and
    of the digits of pi."""
    f = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((f, f, f, f), (f, f), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(int(v) for v in D.philox(counter, key)) == want


def test_mask_keeps_the_mean():
    """Over n kept-or-dropped elements the mean of the mask is 1 within five
    deviations, sqrt(p / (1 - p) / n)."""
    for p in (0.1, 0.5, 0.9):
        m = D.mask(500, 203, p, 12345678901234567890, 7)
        assert abs(m.mean() - 1.0) <= 5 * (p / (1 - p) / m.size) ** 0.5
        assert not np.array_equal(m, D.mask(500, 203, p, 12345678901234567890, 8))


@pytest.mark.parametrize("kind", ["none", "silu", "tanh"])
def test_oracle_gradients_are_the_derivatives(kind):
    """Central differences of <G, y> along random directions, extrapolated: the
    fourth-order term at h = 1e-3 is below 1e-9 of values of order 10."""
    rng = np.random.default_rng(3)
    N, K, M = 7, 5, 11
    x, W, b, G, r = (rng.standard_normal(s) for s in ((N, K), (K, M), (M,), (N, M), (N, M)))
    m = D.mask(N, M, 0.3, 5, 1 << 40)
    z = D.linear_fwd(x, W, b, r, kind, m)[1]
    dx, dW, db, _ = D.linear_bwd(x, W, z, G, kind, m)
    for which, g in (("x", dx), ("W", dW), ("b", db), ("r", G)):
        d = rng.standard_normal(g.shape)

        def loss(h):
            a = {"x": x, "W": W, "b": b, "r": r}
            a[which] = a[which] + h * d
            return (G * D.linear_fwd(a["x"], a["W"], a["b"], a["r"], kind, m)[0]).sum()

        slope = lambda h: (loss(h) - loss(-h)) / (2 * h)  # noqa: E731
        got = (4 * slope(0.5e-3) - slope(1e-3)) / 3
        assert abs(got - (g * d).sum()) <= 1e-8 * (1 + abs(got)), which


def test_dropout_refusals(L):
    lib, bad, uns = L.lib(), L.CGTP_ERR_INVALID_ARG, L.CGTP_ERR_UNSUPPORTED

    def call(d=0, N=4, C=8, p=0.1, step=None, x=FAKE, ldx=8, r=None, ldr=8, out=FAKE, ldo=8):
        return lib.cgtp_dropout(d, N, C, p, 1, 2, step, x, ldx, r, ldr, out, ldo, None)

    assert call(N=0, x=None, out=None) == L.CGTP_OK
    assert call(d=2) == bad and call(d=-1) == bad and call(N=-1) == bad and call(N=2**31 - 1) == bad and call(C=0) == bad
    assert call(C=(1 << 20) + 1, ldx=1 << 21, ldo=1 << 21) == uns
    for p in (-0.1, 1.0, 1.5, float("nan"), float("inf")):
        assert call(p=p) == bad, p
    assert call(step=ctypes.c_void_p(4100)) == bad
    for k in ("x", "out"):
        assert call(**{k: None}) == bad and call(**{k: ODD}) == bad, k
    assert call(r=ODD) == bad and call(r=FAKE, ldr=7) == bad
    assert call(ldx=7) == bad and call(ldo=7) == bad and call(ldx=1 << 50) == bad


def test_linear_refusals(L):
    lib, bad, uns = L.lib(), L.CGTP_ERR_INVALID_ARG, L.CGTP_ERR_UNSUPPORTED
    nan = float("nan")

    def fwd(d=0, act=1, N=4, K=8, M=16, x=FAKE, ldx=8, W=FAKE, b=None, r=None, ldr=16, p=0.0, step=None, z=None,
            y=FAKE, ldy=16, ws=None, n=0):
        return lib.cgtp_linear_act_fwd(d, act, N, K, M, x, ldx, W, b, r, ldr, p, 1, 2, step, z, y, ldy, ws, n, None)

    assert fwd(N=0, x=None, W=None, y=None) == L.CGTP_OK
    assert fwd(d=2) == bad and fwd(act=3) == bad and fwd(act=-1) == bad
    assert fwd(N=-1) == bad and fwd(K=0) == bad and fwd(M=0) == bad
    assert fwd(N=1 << 30) == uns and fwd(K=(1 << 16) + 1) == uns and fwd(M=(1 << 16) + 1) == uns
    assert fwd(p=1.0) == bad and fwd(p=-0.5) == bad and fwd(p=nan) == bad and fwd(step=ODD) == bad
    for k in ("x", "W", "y"):
        assert fwd(**{k: None}) == bad and fwd(**{k: ODD}) == bad, k
    for k in ("b", "r", "z"):
        assert fwd(**{k: ODD}) == bad, k
    assert fwd(ldx=7) == bad and fwd(ldy=15) == bad and fwd(r=FAKE, ldr=15) == bad
    long = dict(N=100, K=40000, M=16, ldx=40000)        # a contraction that is cut: these need a workspace
    assert fwd(**long) == L.CGTP_ERR_WORKSPACE and fwd(**long, ws=WS, n=64) == L.CGTP_ERR_WORKSPACE
    assert fwd(**long, ws=WS_ODD, n=BIG) == bad

    def bwd(act=1, N=4, x=FAKE, ldx=8, W=FAKE, z=FAKE, g=FAKE, ldg=16, p=0.0, dx=FAKE, ldd=8, dW=FAKE, db=FAKE, ws=WS,
            n=BIG):
        return lib.cgtp_linear_act_bwd(0, act, N, 8, 16, x, ldx, W, z, g, ldg, p, 1, 2, None, dx, ldd, dW, db, ws, n,
                                       None)

    assert bwd(dx=None, dW=None, db=None, g=None, ws=None) == L.CGTP_OK     # nothing wanted
    for k in ("x", "W", "z", "g"):
        assert bwd(**{k: None}) == bad and bwd(**{k: ODD}) == bad, k
    for k in ("dx", "dW", "db"):
        assert bwd(**{k: ODD}) == bad, k
    assert bwd(ldx=7) == bad and bwd(ldg=15) == bad and bwd(ldd=7) == bad and bwd(p=1.0) == bad and bwd(act=7) == bad
    assert bwd(N=100000, ws=None) == L.CGTP_ERR_WORKSPACE and bwd(N=100000, n=64) == L.CGTP_ERR_WORKSPACE
    assert bwd(N=100000, ws=WS_ODD) == bad
    b = ctypes.c_size_t()
    size = lambda *a: (lib.cgtp_linear_act_workspace_size(*a, ctypes.byref(b)), b.value)  # noqa: E731
    assert size(0, 0, 8, 16, 0) == (L.CGTP_OK, 0) and size(0, 0, 8, 16, 1) == (L.CGTP_OK, 0)
    assert size(0, 100000, 64, 64, 1)[1] > 64 * 64 * 4
    assert size(0, -1, 8, 16, 0)[0] == bad and size(2, 4, 8, 16, 0)[0] == bad and size(0, 1 << 30, 8, 16, 0)[0] == uns
    assert size(0, (1 << 30) - 1, 1 << 16, 1 << 16, 0)[0] == uns       # more tiles than a launch holds
    assert lib.cgtp_linear_act_workspace_size(0, 4, 8, 16, 0, None) == bad


def test_dense_binding_refusals(L):
    import clebsch_gordan_tensor_cgtp_amd as cg
    x, W = torch.zeros(6, 8), torch.zeros(8, 16)
    with pytest.raises(ValueError, match="GPU"):
        cg.dropout(x, 0.1, 0)
    with pytest.raises(ValueError, match="probability"):
        cg.dropout(x, 1.0, 0)
    with pytest.raises(ValueError, match="2\\^64"):
        cg.dropout(x, 0.1, -1)
    with pytest.raises(ValueError, match="2\\^64"):
        cg.dropout(x, 0.1, 0, 1 << 64)
    with pytest.raises(TypeError, match="int64"):
        cg.dropout(x, 0.1, 0, step=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="shape"):
        cg.dropout(x, 0.1, 0, residual=torch.zeros(6, 7))
    with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
        cg.dropout(x.double(), 0.1, 0)
    with pytest.raises(ValueError, match=r"\[N\]\[C\]"):
        cg.dropout(torch.zeros(8), 0.1, 0)
    with pytest.raises(ValueError, match="channels must be contiguous"):
        cg.dropout(torch.zeros(8, 6).t(), 0.1, 0)
    with pytest.raises(ValueError, match="GPU"):
        cg.linear_act_fwd(x, W)
    with pytest.raises(ValueError, match="W has shape"):
        cg.linear_act_fwd(x, torch.zeros(7, 16))
    with pytest.raises(TypeError, match="W must be torch.float32"):
        cg.linear_act_fwd(x, W.bfloat16())
    with pytest.raises(ValueError, match="W must be contiguous"):
        cg.linear_act_fwd(x, torch.zeros(16, 8).t())
    with pytest.raises(TypeError, match=r"\[in\]\[out\]"):
        cg.linear_act_fwd(x, torch.zeros(8))
    with pytest.raises(ValueError, match="bias has shape"):
        cg.linear_act_fwd(x, W, torch.zeros(8))
    with pytest.raises(TypeError, match="bias must be torch.float32"):
        cg.linear_act_fwd(x.bfloat16(), W.bfloat16(), torch.zeros(16).bfloat16())
    with pytest.raises(ValueError, match="act must be"):
        cg.linear_act_fwd(x, W, act="relu")
    with pytest.raises(ValueError, match="residual has shape"):
        cg.linear_act_fwd(x, W, residual=x)
    with pytest.raises(ValueError, match="out has shape"):
        cg.linear_act_fwd(x, W, out=x)
    with pytest.raises(TypeError, match="z must be a torch.Tensor"):
        cg.linear_act_bwd(x, W, None, torch.zeros(6, 16))
    with pytest.raises(ValueError, match="grad_y has shape"):
        cg.linear_act_bwd(x, W, None, x, act="none")
    with pytest.raises(ValueError, match="grad_x has shape"):
        cg.linear_act_bwd(x, W, None, torch.zeros(6, 16), act="none", grad_x=torch.zeros(6, 16))
