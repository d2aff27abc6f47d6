"""Host-side checks of the node-side operators (no GPU): the library exports
what include/cgtp_train.h declares with as many arguments, workspaces grow
with the sizes, and bad arguments are refused before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 1 << 40
FAKE, ODD, WS, WS_ODD = (ctypes.c_void_p(v) for v in (4096, 4097, 1 << 20, (1 << 20) + 64))  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from clebsch_gordan_tensor_cgtp_amd import _lib
    _lib.lib()
    return _lib


def _declared():
    text = open(os.path.join(ROOT, "include", "cgtp_train.h")).read()
    return re.findall(r"^cgtp_status_t\s+(cgtp_\w+)\(([^)]*)\);", text, re.M)


def test_exports_and_argument_counts(L):
    names = [n for n, _ in _declared()]
    assert "cgtp_embed_fwd" in names and "cgtp_norm_act_bwd" in names
    for name, params in _declared():
        assert hasattr(L.lib(), name), name
        assert len(L.SIGNATURES[name][1]) == len([p for p in params.split(",") if p.strip()]), name


def test_header_compiles_as_c(tmp_path):
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "cgtp_train.h"\nint main(void) { return CGTP_F32; }\n')
    subprocess.run(["gcc", "-std=c99", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    "/opt/rocm/include", "-fsyntax-only", str(src)], check=True)


def test_embed_refusals(L):
    lib, bad, uns = L.lib(), L.CGTP_ERR_INVALID_ARG, L.CGTP_ERR_UNSUPPORTED
    fwd = lambda d=0, N=4, V=5, C=8, ids=FAKE, t=FAKE, o=FAKE, ld=8: lib.cgtp_embed_fwd(d, N, V, C, ids, t, 1.0, o, ld, None)
    assert fwd(N=0, ids=None, t=None, o=None) == L.CGTP_OK
    assert fwd(d=2) == bad and fwd(d=-1) == bad
    assert fwd(N=-1) == bad and fwd(V=0) == bad and fwd(C=0) == bad and fwd(N=2**31 - 1) == bad and fwd(V=2**31) == bad
    assert fwd(C=(1 << 20) + 1, ld=1 << 21) == uns
    assert fwd(ids=None) == bad and fwd(t=None) == bad and fwd(o=None) == bad
    assert fwd(ids=ODD) == bad and fwd(t=ODD) == bad and fwd(o=ODD) == bad
    assert fwd(ld=7) == bad and fwd(ld=1 << 50) == bad
    bwd = lambda d=0, N=4, V=5, C=8, ids=FAKE, g=FAKE, ld=8, t=FAKE, ws=WS, n=BIG: lib.cgtp_embed_bwd(
        d, N, V, C, ids, g, ld, 1.0, t, ws, n, None)
    assert bwd(t=None) == bad and bwd(t=ODD) == bad and bwd(g=None) == bad and bwd(ld=7) == bad and bwd(ids=ODD) == bad
    assert bwd(ws=None) == L.CGTP_ERR_WORKSPACE and bwd(n=16) == L.CGTP_ERR_WORKSPACE and bwd(ws=WS_ODD) == bad
    b = ctypes.c_size_t()
    size = lambda *a: (lib.cgtp_embed_bwd_workspace_size(*a, ctypes.byref(b)), b.value)
    assert size(0, 0, 5, 8)[0] == L.CGTP_OK
    small, large = size(0, 1000, 5, 8)[1], size(0, 100000, 5, 8)[1]
    assert 16 * 1000 <= small < large
    assert size(0, -1, 5, 8)[0] == bad and lib.cgtp_embed_bwd_workspace_size(0, 4, 5, 8, None) == bad


def test_norm_refusals(L):
    lib, bad, uns = L.lib(), L.CGTP_ERR_INVALID_ARG, L.CGTP_ERR_UNSUPPORTED

    def fwd(d=0, act=1, N=6, B=2, C=8, G=4, seg=FAKE, eps=1e-5, x=FAKE, ldx=8, gm=FAKE, bt=FAKE, y=FAKE, ldy=8,
            mean=FAKE, rstd=FAKE, ws=WS, n=BIG):
        return lib.cgtp_norm_act_fwd(d, act, N, B, C, G, seg, eps, x, ldx, gm, bt, y, ldy, mean, rstd, ws, n, None)

    assert fwd(N=0, B=0, x=None, y=None, mean=None, rstd=None, ws=None) == L.CGTP_OK
    assert fwd(d=5) == bad and fwd(act=3) == bad and fwd(act=-1) == bad
    assert fwd(N=-1) == bad and fwd(B=-1) == bad and fwd(C=0) == bad and fwd(G=0) == bad and fwd(G=3) == bad
    assert fwd(B=0) == bad                              # rows but no segment
    assert fwd(seg=None, N=7) == bad                    # equal segments need a multiple
    assert fwd(C=1 << 17, G=1, ldx=1 << 17, ldy=1 << 17) == uns
    assert fwd(eps=0.0) == bad and fwd(eps=-1.0) == bad and fwd(eps=float("inf")) == bad and fwd(eps=float("nan")) == bad
    for k in ("x", "y", "mean", "rstd"):
        assert fwd(**{k: None}) == bad and fwd(**{k: ODD}) == bad, k
    for k in ("seg", "gm", "bt"):
        assert fwd(**{k: ODD}) == bad, k
    assert fwd(ldx=7) == bad and fwd(ldy=7) == bad
    large = dict(N=400000, B=2)     # segments that no block takes whole: these need a workspace
    assert fwd(**large, ws=None) == L.CGTP_ERR_WORKSPACE and fwd(**large, n=64) == L.CGTP_ERR_WORKSPACE
    assert fwd(**large, ws=WS_ODD) == bad
    b = ctypes.c_size_t()
    size = lambda *a: (lib.cgtp_norm_act_workspace_size(*a, ctypes.byref(b)), b.value)  # noqa: E731
    assert size(0, 6, 2, 8, 4, 1, 0) == (L.CGTP_OK, 0) and size(0, 6, 2, 8, 4, 1, 1)[1] > 0
    assert size(0, 400000, 2, 8, 4, 1, 0)[1] > 0 and size(0, 6, 2, 8, 3, 1, 0)[0] == bad
    assert lib.cgtp_norm_act_workspace_size(0, 6, 2, 8, 4, 1, 0, None) == bad

    def bwd(x=FAKE, mean=FAKE, rstd=FAKE, gm=FAKE, dy=FAKE, ldy=8, dx=FAKE, ldd=8, dg=FAKE, db=FAKE, ws=WS, n=BIG):
        return lib.cgtp_norm_act_bwd(0, 1, 6, 2, 8, 4, FAKE, x, 8, mean, rstd, gm, FAKE, dy, ldy, dx, ldd, dg, db, ws,
                                     n, None)

    assert bwd(dx=None, dg=None, db=None, ws=None) == L.CGTP_OK     # nothing wanted
    for k in ("x", "mean", "rstd", "dy"):
        assert bwd(**{k: None}) == bad and bwd(**{k: ODD}) == bad, k
    for k in ("gm", "dx", "dg", "db"):
        assert bwd(**{k: ODD}) == bad, k
    assert bwd(ldy=7) == bad and bwd(ldd=7) == bad
    assert bwd(n=64) == L.CGTP_ERR_WORKSPACE and bwd(ws=None) == L.CGTP_ERR_WORKSPACE


def test_orthogonalize_refusals(L):
    lib, bad, uns = L.lib(), L.CGTP_ERR_INVALID_ARG, L.CGTP_ERR_UNSUPPORTED
    nan, inf = float("nan"), float("inf")

    def call(d=0, B=2, m=4, n=6, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, scale=1.0, G=FAKE, out=FAKE, ws=WS,
             size=BIG):
        return lib.cgtp_orthogonalize(d, B, m, n, steps, a, b, c, eps, scale, G, out, ws, size, None)

    assert call(B=0, G=None, out=None, ws=None) == L.CGTP_OK
    assert call(d=3) == bad and call(B=-1) == bad and call(m=0) == bad and call(n=0) == bad
    assert call(m=(1 << 16) + 1) == uns and call(m=1 << 16, n=1 << 16) == uns and call(B=1 << 40) == uns
    assert call(steps=0) == bad and call(steps=65) == bad and call(eps=-1e-7) == bad and call(eps=nan) == bad
    assert call(scale=inf) == bad and call(a=nan) == bad and call(b=inf) == bad
    assert call(a=30.0, b=0.0, c=20.0) == bad           # grows without bound
    assert call(a=1.0, b=0.0, c=0.0) == bad             # no product at all
    assert call(m=200, n=300, a=1.5, b=-0.5, c=0.0, ws=None) == L.CGTP_ERR_WORKSPACE      # the cubic is fine
    assert call(G=None) == bad and call(out=None) == bad and call(G=ODD) == bad and call(out=ODD) == bad
    large = dict(m=200, n=300)      # a matrix that no block holds: these need a workspace
    assert call(**large, ws=None) == L.CGTP_ERR_WORKSPACE and call(**large, size=64) == L.CGTP_ERR_WORKSPACE
    assert call(**large, ws=WS_ODD) == bad
    b = ctypes.c_size_t()
    size = lambda *a: (lib.cgtp_orthogonalize_workspace_size(*a, ctypes.byref(b)), b.value)  # noqa: E731
    assert size(0, 15, 128, 128) == (L.CGTP_OK, 0)
    assert 0 < size(0, 1, 128, 1024)[1] < size(0, 15, 128, 1024)[1] < size(1, 15, 512, 1024)[1]
    assert size(0, 1, 0, 8)[0] == bad and lib.cgtp_orthogonalize_workspace_size(0, 1, 8, 8, None) == bad


def test_binding_refusals(L):
    import clebsch_gordan_tensor_cgtp_amd as cg
    ids, table = torch.zeros(4, dtype=torch.int32), torch.zeros(5, 8)
    with pytest.raises(ValueError, match="GPU"):
        cg.embed_fwd(ids, table)
    with pytest.raises(TypeError, match="int32"):
        cg.embed_fwd(ids.long(), table)
    with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
        cg.embed_fwd(ids, table.double())
    with pytest.raises(ValueError, match="shape"):
        cg.embed_fwd(ids, table, out=torch.zeros(3, 8))
    with pytest.raises(ValueError, match="contiguous"):
        cg.embed_fwd(ids, table.t())
    with pytest.raises(ValueError, match="channels must be contiguous"):
        cg.embed_bwd(ids, torch.zeros(8, 4).t(), 5)
    with pytest.raises(ValueError, match="overlap"):
        cg.embed_bwd(ids, torch.zeros(1, 8).expand(4, 8), 5)
    x, w = torch.zeros(6, 8), torch.ones(8)
    with pytest.raises(ValueError, match="contiguous"):
        cg.orthogonalize(torch.zeros(8, 4).t())
    with pytest.raises(ValueError, match="rows, cols"):
        cg.orthogonalize(torch.zeros(8))
    with pytest.raises(ValueError, match="at least 1"):
        cg.orthogonalize(torch.zeros(3, 0, 8))
    with pytest.raises(ValueError, match="GPU"):
        cg.orthogonalize(torch.zeros(3, 4, 8))
    with pytest.raises(ValueError, match="does not divide"):
        cg.norm_act_fwd(x, w, w, 3)
    with pytest.raises(ValueError, match="act must be"):
        cg.norm_act_fwd(x, w, w, 4, act="relu")
    with pytest.raises(TypeError, match="int32"):
        cg.norm_act_fwd(x, w, w, 4, torch.tensor([0, 6]))
    with pytest.raises(ValueError, match="shape"):
        cg.norm_act_fwd(x, w[:4], w, 4)
    with pytest.raises(ValueError, match="equally spaced"):
        cg.norm_act_fwd(torch.zeros(3, 5, 8)[:, :2], w, w, 4)
    with pytest.raises(ValueError, match="shape"):
        cg.norm_act_bwd(x, torch.zeros(2, 4), torch.zeros(1, 4), w, w, x, 4)


def test_norm_gradient_output_refusals(L):
    import clebsch_gordan_tensor_cgtp_amd as cg
    x, w, s = torch.zeros(6, 8), torch.ones(8), torch.zeros(1, 4)
    call = lambda g: cg.norm_act_bwd(x, s, s, w, w, x, 4, grad_x=g)  # noqa: E731
    for bad in (torch.zeros(5, 8), torch.zeros(6, 3, 8)):
        with pytest.raises(ValueError, match="grad_x has shape"):
            call(bad)
    with pytest.raises(TypeError, match="grad_x must be torch.float32"):
        call(torch.zeros(6, 8).bfloat16())
    with pytest.raises(TypeError, match="torch.Tensor"):
        call([0.0])
    with pytest.raises(ValueError, match="channels must be contiguous"):
        call(torch.zeros(8, 6).t())
    with pytest.raises(ValueError, match="overlap"):
        call(torch.zeros(1, 8).expand(6, 8))
    with pytest.raises(ValueError, match="GPU"):
        call(torch.zeros(6, 2, 8)[:, 0])
