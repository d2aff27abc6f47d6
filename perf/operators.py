"""What is measured of the node-side operators of a training step: the species
(token) embedding and its gradient, the group normalisation with an activation
over ragged segments of channels-last rows and its gradient, and the
orthogonalised update of a stack of weight matrices.

``listed`` and ``draw`` name the cases, ``prepare`` makes a case's inputs,
``run`` makes one pass (the plain form in torch, or the package's operators
where ``own`` is true), ``exact`` gives the outputs from the definitions in 64
bits and ``work`` the bytes and operations that a pass cannot do without.
"""
import math

import numpy as np
import torch

own = False

# the quintic a x + b x^3 + c x^5 of five Newton-Schulz steps, and the norm's offset
COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
NS_EPS = 1e-7
NORM_EPS = 1e-5

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ---- cases ---------------------------------------------------------------------
def _embed(name, op, rows, table, channels, dtype, pitch=1, pad=0.0, zipf=False):
    return {"name": name, "op": op, "rows": rows, "table": table, "channels": channels, "dtype": dtype,
            "pitch": pitch, "pad": pad, "zipf": zipf}


def _norm(name, op, segments, rows, channels, groups, dtype, act, ragged, pitch=1):
    return {"name": name, "op": op, "segments": segments, "rows": rows, "channels": channels, "groups": groups,
            "dtype": dtype, "act": act, "ragged": ragged, "pitch": pitch}


def _ortho(name, batch, rows, cols, dtype):
    return {"name": name, "op": "ortho", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype}


def listed():
    return [
        # the invariant features of one 2000-atom layer at 128 channels, one row per chemical element
        _embed("embed_fwd_layer", "embed_fwd", 2000, 89, 128, "f32"),
        # its gradient, taken from the l = 0 row of the convolution's [N][9][128] input gradient; few species
        _embed("embed_bwd_layer", "embed_bwd", 2000, 89, 128, "f32", pitch=9),
        # the 50000-atom structure: half a dozen species hold all the rows
        _embed("embed_bwd_large", "embed_bwd", 50000, 89, 128, "f32"),
        # a padded batch of tokens over a large table, with the usual skew of token counts
        _embed("embed_fwd_vocabulary", "embed_fwd", 16385, 65536, 1024, "bf16", pad=0.05, zipf=True),
        _embed("embed_bwd_vocabulary", "embed_bwd", 16385, 65536, 1024, "bf16", pad=0.05, zipf=True),
        # the invariant rows (l = 0) of one 2000-atom layer's [N][9][128] features, one structure: the smallest calls
        _norm("norm_fwd_layer", "norm_fwd", 1, 2000, 128, 8, "f32", "silu", True, pitch=9),
        # a training batch of small molecules, 20-odd atoms each
        _norm("norm_fwd_molecules", "norm_fwd", 1024, 25000, 128, 8, "bf16", "silu", True),
        _norm("norm_bwd_molecules", "norm_bwd", 1024, 25000, 128, 8, "f32", "silu", True),
        # eight equal images or grids of channels-last values
        _norm("norm_bwd_large", "norm_bwd", 8, 400008, 256, 32, "bf16", "silu", False),
        # the mixing matrices of all fifteen paths at degree 2 and 128 channels
        _ortho("ortho_paths", 15, 128, 128, "f32"),
        # the same paths mixed into the largest supported output width
        _ortho("ortho_paths_wide", 15, 128, 1024, "bf16"),
        # one large square matrix
        _ortho("ortho_square", 1, 2048, 2048, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 5e12, w["flops"] / 1e14)


def draw(rng):
    """One more case over the listed ones' ranges: every operator, both types, sizes from a single row to the largest
    listed, odd ones among them."""
    family = lambda op: op.split("_")[0]  # noqa: E731
    top = {}
    for c in listed():
        top[family(c["op"])] = max(top.get(family(c["op"]), 0.0), _cost(c))
    op = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd", "ortho"])
    while True:
        dtype = rng.choice(["f32", "bf16"])
        if op.startswith("embed"):
            zipf = rng.random() < 0.5
            case = _embed("", op, _log(rng, 1, 400000), _log(rng, 300, 130000) if zipf else _log(rng, 1, 300),
                          _log(rng, 8, 2048), dtype, rng.choice([1, 1, 4, 9]) if op == "embed_bwd" else 1,
                          rng.choice([0.0, 0.1]), zipf)
        elif op.startswith("norm"):
            groups, per = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 3, 4, 8, 16, 32, 40, 64])
            ragged = rng.random() < 0.7
            segments, rows = _log(rng, 1, 3000), _log(rng, 1, 500000)
            rows = rows if ragged else max(1, rows // segments) * segments
            if rows // segments * per < 8:   # a group of one or two values has nothing to normalise
                continue
            case = _norm("", op, segments, rows, groups * per, groups, dtype, rng.choice(["none", "silu", "tanh"]),
                         ragged, rng.choice([1, 1, 4, 9]) if ragged else 1)
        else:
            case = _ortho("", _log(rng, 1, 64), _log(rng, 8, 3000), _log(rng, 8, 3000), dtype)
            if min(case["rows"], case["cols"]) > 2048:
                continue
        case.pop("name")
        values = case["rows"] * case.get("channels", 1) * case.get("pitch", 1)
        if _cost(case) <= top[family(op)] and values <= 1 << 28:
            return case


# ---- inputs --------------------------------------------------------------------
def _ids(case, g, dev):
    """Token ids with the skew of real ones: a large table's by rank (Zipf), a small one's from at most six kinds;
    a share `pad` of them is -1 (padding)."""
    N, V = case["rows"], case["table"]
    if case["zipf"]:
        p = 1.0 / (torch.arange(V, device=dev, dtype=torch.float64) + 2.7) ** 1.05
        p = p[torch.randperm(V, generator=g, device=dev)]
    else:
        p = torch.zeros(V, device=dev, dtype=torch.float64)
        k = min(6, V)
        p[torch.randperm(V, generator=g, device=dev)[:k]] = 0.5 ** torch.arange(k, device=dev, dtype=torch.float64)
    c = torch.cumsum(p / p.sum(), 0)
    ids = torch.searchsorted(c, torch.rand(N, generator=g, device=dev, dtype=torch.float64)).clamp_(max=V - 1)
    ids[torch.rand(N, generator=g, device=dev) < case["pad"]] = -1
    return ids.to(torch.int32)


def _segments(case, g, dev):
    """Offsets of the ragged segments: spread lengths, about one in fifty empty."""
    B, N = case["segments"], case["rows"]
    w = torch.exp(0.6 * torch.randn(B, generator=g, device=dev, dtype=torch.float64))
    w[torch.rand(B, generator=g, device=dev) < 0.02] = 0.0
    w[0] += 1e-9
    ptr = torch.zeros(B + 1, dtype=torch.int64, device=dev)
    ptr[1:] = torch.floor(torch.cumsum(w, 0) / w.sum() * N).to(torch.int64).clamp_(max=N)
    ptr[B] = N
    return ptr.to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]
    rnd = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    op = case["op"]
    s = {"case": case}
    if op.startswith("embed"):
        s["ids"] = _ids(case, g, dev)
        s["scale"] = math.sqrt(case["channels"])
        if op == "embed_fwd":
            s["table"] = (0.02 * rnd(case["table"], case["channels"])).to(dt)
        else:  # the gradient's rows may be every pitch-th row of a wider tensor
            s["grad"] = rnd(case["rows"], case["pitch"], case["channels"]).to(dt)[:, 0, :]
    elif op.startswith("norm"):
        N, B, C, G = case["rows"], case["segments"], case["channels"], case["groups"]
        x = rnd(N, case["pitch"], C)[:, 0, :] * (0.5 + torch.rand(C, generator=g, device=dev)) + 0.7 * rnd(C)
        full = torch.zeros((N, case["pitch"], C), dtype=dt, device=dev)
        full[:, 0, :] = x.to(dt)
        s["x"] = full[:, 0, :] if case["ragged"] else full.view(B, N // B, C)
        s["ptr"] = _segments(case, g, dev) if case["ragged"] else None
        s["gamma"], s["beta"] = 1.0 + 0.2 * rnd(C), 0.2 * rnd(C)
        if op == "norm_bwd":  # what the forward pass left behind
            s["grad"] = rnd(*s["x"].shape).to(dt)
            s["mean"], s["rstd"] = _stats64(s["x"], _bounds(s), G)
    else:
        B, m, n = case["batch"], case["rows"], case["cols"]
        # a gradient's spectrum: a few strong directions over a floor of noise
        r = max(1, min(m, n) // 8)
        decay = torch.exp(-3.0 * torch.arange(r, device=dev) / r)
        low = torch.matmul(rnd(B, m, r) * decay, rnd(B, r, n)) / math.sqrt(r)
        s["grad"] = (1e-3 * (low + 0.3 * rnd(B, m, n))).to(dt)
    return s


# ---- one pass ------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import clebsch_gordan_tensor_cgtp_amd as cg
        if op == "embed_fwd":
            return cg.embed_fwd(s["ids"], s["table"], s["scale"])
        if op == "embed_bwd":
            return cg.embed_bwd(s["ids"], s["grad"], case["table"], s["scale"])
        if op == "norm_fwd":
            return cg.norm_act_fwd(s["x"], s["gamma"], s["beta"], case["groups"], s["ptr"], NORM_EPS, case["act"])
        if op == "norm_bwd":
            return cg.norm_act_bwd(s["x"], s["mean"], s["rstd"], s["gamma"], s["beta"], s["grad"], case["groups"],
                                   s["ptr"], case["act"])
        return cg.orthogonalize(s["grad"], STEPS, COEFFS, NS_EPS)
    return {"embed_fwd": _embed_fwd, "embed_bwd": _embed_bwd, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd,
            "ortho": _orthogonalize}[op](s)


def _embed_fwd(s):
    ids, table = s["ids"], s["table"]
    inside = (ids >= 0) & (ids < table.shape[0])
    rows = table[torch.where(inside, ids, 0)].float() * s["scale"]
    return torch.where(inside[:, None], rows, 0.0).to(table.dtype)


def _embed_bwd(s):
    ids, grad, V = s["ids"], s["grad"], s["case"]["table"]
    total = torch.zeros((V + 1, grad.shape[1]), device=grad.device)   # row V takes what is outside the table
    total.index_add_(0, torch.where((ids >= 0) & (ids < V), ids, V), grad.float())
    return (total[:V] * s["scale"]).to(grad.dtype)


def _act(z, act):
    return z if act == "none" else z * torch.sigmoid(z) if act == "silu" else torch.tanh(z)


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "silu":
        e = torch.sigmoid(z)
        return e * (1.0 + z * (1.0 - e))
    return 1.0 - torch.tanh(z) ** 2


class _Rows:
    """Sums over the rows of each segment and their way back, for ragged segments (offsets) and for equal ones."""

    def __init__(self, s):
        case = s["case"]
        self.B, self.N, self.ptr = case["segments"], case["rows"], s["ptr"]
        if self.ptr is not None:
            at = torch.arange(self.N, device=self.ptr.device, dtype=torch.int32)
            self.of = torch.searchsorted(self.ptr[1:].contiguous(), at, right=True)
            self.count = (self.ptr[1:] - self.ptr[:-1]).float()[:, None]
        else:
            self.count = float(self.N // self.B)

    def total(self, v):      # [N][K] -> [B][K]
        if self.ptr is None:
            return v.view(self.B, -1, v.shape[1]).sum(1)
        return torch.zeros((self.B, v.shape[1]), device=v.device).index_add_(0, self.of, v)

    def spread(self, v):     # [B][K] -> [N][K]
        if self.ptr is None:
            return v[:, None, :].expand(-1, self.N // self.B, -1).reshape(self.N, -1)
        return v[self.of]

    def values(self, per):   # values in each segment's groups, at least one
        return (self.count * per).clamp(min=1.0) if self.ptr is not None else max(self.count * per, 1.0)


def _norm_fwd(s):
    case = s["case"]
    N, C, G = case["rows"], case["channels"], case["groups"]
    R = _Rows(s)
    x = s["x"].reshape(N, G, C // G).float()
    mean = R.total(x.sum(2)) / R.values(C // G)
    d = x - R.spread(mean)[:, :, None]
    rstd = 1.0 / torch.sqrt(R.total((d * d).sum(2)) / R.values(C // G) + NORM_EPS)
    z = (d * R.spread(rstd)[:, :, None]).view(N, C) * s["gamma"] + s["beta"]
    return _act(z, case["act"]).to(s["x"].dtype).view(s["x"].shape), mean, rstd


def _norm_bwd(s):
    case = s["case"]
    N, C, G = case["rows"], case["channels"], case["groups"]
    R = _Rows(s)
    x, dy = s["x"].reshape(N, G, C // G).float(), s["grad"].reshape(N, C).float()
    rstd = R.spread(s["rstd"])[:, :, None]
    xhat = ((x - R.spread(s["mean"])[:, :, None]) * rstd).view(N, C)
    dz = dy * _act_grad(xhat * s["gamma"] + s["beta"], case["act"])
    h = dz * s["gamma"]
    one, two = h.view(N, G, -1).sum(2), (h * xhat).view(N, G, -1).sum(2)
    one, two = (R.spread(R.total(v) / R.values(C // G))[:, :, None] for v in (one, two))
    dx = rstd * (h.view(N, G, -1) - one - xhat.view(N, G, -1) * two)
    return dx.to(s["x"].dtype).view(s["x"].shape), (dz * xhat).sum(0), dz.sum(0)


def _orthogonalize(s):
    G = s["grad"]
    a, b, c = COEFFS
    X = G.float()
    X = X / (torch.sqrt((X * X).sum((1, 2), keepdim=True)) + NS_EPS)
    tall = X.shape[1] > X.shape[2]
    X = X.transpose(1, 2).contiguous() if tall else X
    for _ in range(STEPS):
        A = torch.matmul(X, X.transpose(1, 2).contiguous())
        X = a * X + torch.matmul(b * A + c * torch.matmul(A, A), X)
    return (X.transpose(1, 2) if tall else X).to(G.dtype).contiguous()


# ---- the definitions in 64 bits ------------------------------------------------
def _bounds(s):
    case = s["case"]
    if s["ptr"] is not None:
        return s["ptr"].tolist()
    return [k * (case["rows"] // case["segments"]) for k in range(case["segments"] + 1)]


def _stats64(x, bounds, groups):
    """Mean and 1/deviation of each segment's groups in 64 bits, kept in 32."""
    C = x.shape[-1]
    x = x.reshape(-1, groups, C // groups)
    mean = torch.zeros((len(bounds) - 1, groups), dtype=torch.float64, device=x.device)
    var = torch.zeros_like(mean)
    for k, (i, j) in enumerate(zip(bounds, bounds[1:])):
        if j > i:
            v = x[i:j].double()
            mean[k], var[k] = v.mean((0, 2)), v.var((0, 2), unbiased=False)
    return mean.float(), (1.0 / torch.sqrt(var + NORM_EPS)).float()


def _exact_embed(s, op):
    case = s["case"]
    ids = s["ids"].cpu().numpy().astype(np.int64)
    V, C = case["table"], case["channels"]
    inside = (ids >= 0) & (ids < V)
    if op == "embed_fwd":
        out = np.zeros((ids.size, C))
        out[inside] = s["table"].double().cpu().numpy()[ids[inside]] * s["scale"]
        return out
    g = s["grad"].double().cpu().numpy()[inside]
    order = np.argsort(ids[inside], kind="stable")
    kind, first = np.unique(ids[inside][order], return_index=True)
    out = np.zeros((V, C))
    if kind.size:
        out[kind] = np.add.reduceat(g[order], first, axis=0) * s["scale"]
    return out


def _exact_norm(s, op):
    case = s["case"]
    C, G, act = case["channels"], case["groups"], case["act"]
    bounds = _bounds(s)
    x = s["x"].reshape(-1, C)
    gamma, beta = s["gamma"].double(), s["beta"].double()
    mean = torch.zeros((len(bounds) - 1, G), dtype=torch.float64, device=x.device)
    rstd = torch.full_like(mean, NORM_EPS ** -0.5)
    rows = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    dgamma, dbeta = torch.zeros_like(gamma), torch.zeros_like(beta)
    dy = s["grad"].reshape(-1, C) if op == "norm_bwd" else None
    for k, (i, j) in enumerate(zip(bounds, bounds[1:])):
        if j == i:
            continue
        v = x[i:j].double().view(j - i, G, C // G)
        var, mu = torch.var_mean(v, (0, 2), unbiased=False)
        mean[k], rstd[k] = mu, (var + NORM_EPS) ** -0.5
        n = (v - mu[:, None]) * rstd[k][:, None]
        z = n.view(-1, C) * gamma + beta
        p = torch.sigmoid(z)
        if op == "norm_fwd":
            rows[i:j] = {"none": lambda: z, "silu": lambda: z * p, "tanh": lambda: torch.tanh(z)}[act]()
            continue
        slope = {"none": lambda: torch.ones_like(z), "silu": lambda: p + z * p * (1 - p),
                 "tanh": lambda: torch.cosh(z) ** -2}[act]()
        d = dy[i:j].double() * slope
        dgamma += (d * n.view(-1, C)).sum(0)
        dbeta += d.sum(0)
        d = (d * gamma).view(n.shape)
        rows[i:j] = (rstd[k][:, None] * (d - d.mean((0, 2))[:, None] - n * (d * n).mean((0, 2))[:, None])).view(-1, C)
    rows = rows.view(s["x"].shape)
    return (rows, mean, rstd) if op == "norm_fwd" else (rows, dgamma, dbeta)


def _exact_ortho(s):
    """By the eigenvalues of the smaller Gram matrix: every step multiplies a singular value x by a + b x^2 + c x^4."""
    a, b, c = COEFFS
    out = []
    for G in s["grad"].double().cpu().numpy():
        X = G / (np.linalg.norm(G) + NS_EPS)
        tall = X.shape[0] > X.shape[1]
        X = X.T if tall else X
        lam, U = np.linalg.eigh(X @ X.T)
        lam, q = np.maximum(lam, 0.0), np.ones_like(lam)
        for _ in range(STEPS):
            f = a + lam * (b + c * lam)
            q, lam = q * f, lam * f * f
        O = (U * q) @ (U.T @ X)
        out.append(O.T if tall else O)
    return np.stack(out)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("embed"):
        return _exact_embed(s, op)
    if op.startswith("norm"):
        return _exact_norm(s, op)
    return _exact_ortho(s)


# ---- what a pass cannot do without ---------------------------------------------
def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op.startswith("embed"):
        N, V, C = case["rows"], case["table"], case["channels"]
        if op == "embed_fwd":   # ids, the rows used (once each), the output
            return {"bytes": 4 * N + e * C * (min(N, V) + N), "flops": N * C}
        return {"bytes": 4 * N + e * C * (N + V), "flops": N * C + V * C}
    if op.startswith("norm"):
        N, C, B, G = case["rows"], case["channels"], case["segments"], case["groups"]
        small = 8 * C + 8 * B * G + (4 * (B + 1) if case["ragged"] else 0)
        if op == "norm_fwd":
            return {"bytes": 2 * e * N * C + small, "flops": 12 * N * C}
        return {"bytes": 3 * e * N * C + small + 8 * C, "flops": 25 * N * C}
    # per step one Gram matrix and one square of it (symmetric: half the products) and one full product
    m, n = sorted((case["rows"], case["cols"]))
    return {"bytes": 2 * e * case["batch"] * m * n, "flops": case["batch"] * STEPS * (3.0 * m * m * n + m ** 3)}
