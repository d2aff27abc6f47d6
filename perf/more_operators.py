"""What is measured of the dense operators beside the convolution: the product
of rows with a weight matrix with bias, activation, dropout and residual in its
epilogue (the radial network of the edges, the update block of the atoms'
invariant rows) and its gradients, and dropout from a counter-based generator
by itself.

``listed`` and ``draw`` name the cases, ``prepare`` makes a case's inputs,
``run`` makes one pass (the plain form in torch, or the package's operators
where ``own`` is true), ``exact`` gives the outputs from the definitions in 64
bits and ``work`` the bytes and operations that a pass cannot do without.

Element (n, c) of dropped rows is kept where field c mod 8 (16 bits each, from
the lowest) of the 128 bits of Philox4x32-10 at the counter (c div 8, n, offset
low, offset high) and the key (seed low, seed high) is at least t =
min(floor(65536 p + 1/2), 65535), and then multiplied by 1 / (1 - t / 65536).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ---- cases ---------------------------------------------------------------------
def _linear(name, op, rows, cin, cout, dtype, act, bias=True, residual=False, drop=0.0, save=True, pitch=1):
    """save: the forward keeps what the backward needs; pitch: x's rows are every pitch-th row of a wider array."""
    return {"name": name, "op": op, "rows": rows, "cin": cin, "cout": cout, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "drop": drop, "save": save, "pitch": pitch}


def _dropout(name, rows, channels, dtype, drop, residual=False, pitch=1):
    return {"name": name, "op": "dropout", "rows": rows, "cin": channels, "cout": channels, "dtype": dtype,
            "drop": drop, "residual": residual, "pitch": pitch}


def listed():
    return [
        # the update of the invariant (l = 0) rows of one 2000-atom layer's [N][9][128] features: the smallest step
        _linear("linear_fwd_layer", "linear_fwd", 2000, 128, 128, "f32", "silu", residual=True, drop=0.1, pitch=9),
        _linear("linear_bwd_layer", "linear_bwd", 2000, 128, 128, "f32", "silu", drop=0.1, pitch=9),
        # one row, as a model answers with it: latency and the weights' bytes
        _linear("linear_fwd_token", "linear_fwd", 1, 1024, 4096, "bf16", "silu", save=False),
        # the radial network of the 2000-atom layer's 105730 edges: eight distance functions to its hidden width
        _linear("linear_fwd_radial_in", "linear_fwd", 105730, 8, 64, "f32", "silu"),
        # and from there to the convolution's edge weights, fifteen paths of 128 channels; their gradients
        _linear("linear_fwd_radial_out", "linear_fwd", 105730, 64, 1920, "f32", "none", bias=False),
        _linear("linear_bwd_radial_out", "linear_bwd", 105730, 64, 1920, "f32", "none", bias=False),
        # the gradients of an update block over a training batch of small molecules
        _linear("linear_bwd_molecules", "linear_bwd", 25000, 128, 128, "bf16", "tanh"),
        # a batch of tokens through the first layer of a wide block, odd in its rows
        _linear("linear_fwd_tokens", "linear_fwd", 16385, 1024, 4096, "bf16", "silu", drop=0.1),
        _linear("linear_bwd_tokens", "linear_bwd", 16385, 1024, 4096, "bf16", "silu", drop=0.1),
        # dropout by itself: the invariant rows of a layer, a batch of tokens, a large batch joined to its residual
        _dropout("dropout_layer", 2000, 128, "f32", 0.1, pitch=9),
        _dropout("dropout_tokens", 16385, 1024, "bf16", 0.5),
        _dropout("dropout_residual", 400008, 256, "f32", 0.1, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 5e12, w["flops"] / 1e14)


def draw(rng):
    """One more case over the listed ones' ranges: both directions, both types, sizes from a single row to the largest
    listed, odd ones among them."""
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    op = rng.choice(["linear_fwd", "linear_bwd", "dropout"])
    while True:
        dtype, drop = rng.choice(["f32", "bf16"]), rng.choice([0.0, 0.1, 0.5])
        rows, pitch = _log(rng, 1, 400000), rng.choice([1, 1, 1, 4])
        if op == "dropout":
            case = _dropout("", rows, _log(rng, 8, 4096), dtype, drop or 0.25, rng.random() < 0.5, pitch)
        else:
            cin, cout = _log(rng, 8, 4096), _log(rng, 8, 4096)
            if rng.random() < 0.6:   # most widths are whole vectors
                cin, cout = -(-cin // 8) * 8, -(-cout // 8) * 8
            case = _linear("", op, rows, cin, cout, dtype, rng.choice(["none", "silu", "tanh"]), rng.random() < 0.7,
                           op == "linear_fwd" and rng.random() < 0.5, drop, rng.random() < 0.7, pitch)
        case.pop("name")
        if _cost(case) <= top[op] and rows * max(case["cin"] * pitch, case["cout"]) <= 1 << 28:
            return case


# ---- inputs --------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]
    N, K, M = case["rows"], case["cin"], case["cout"]
    rnd = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    # the program's seed, and how far its earlier calls have moved the generator
    s = {"case": case, "seed": (seed * 0x9E3779B97F4A7C15 + 0x1234567) % 2 ** 63, "offset": 2 ** 33 + 5 * seed}
    wide = rnd(N, case["pitch"], K).to(dt)
    s["x"] = wide[:, 0, :]
    s["residual"] = rnd(N, M).to(dt) if case["residual"] else None
    if case["op"] == "dropout":
        return s
    s["W"] = (rnd(K, M) / math.sqrt(K)).to(dt)
    s["bias"] = 0.2 * rnd(M) if case["bias"] else None
    if case["op"] == "linear_bwd":   # what the forward pass left behind
        s["z"] = _preactivation(s).to(dt) if case["act"] != "none" else None
        s["grad"] = rnd(N, M).to(dt)
    return s


# ---- one pass ------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import clebsch_gordan_tensor_cgtp_amd as cg
        if op == "dropout":
            return cg.dropout(s["x"], case["drop"], s["seed"], s["offset"], residual=s["residual"])
        if op == "linear_fwd":
            return cg.linear_act_fwd(s["x"], s["W"], s["bias"], case["act"], residual=s["residual"],
                                     p_drop=case["drop"], seed=s["seed"], offset=s["offset"], save=case["save"])
        want = ("x", "W", "bias") if case["bias"] else ("x", "W")
        return cg.linear_act_bwd(s["x"], s["W"], s["z"], s["grad"], case["act"], p_drop=case["drop"], seed=s["seed"],
                                 offset=s["offset"], want=want)
    return {"dropout": _drop_rows, "linear_fwd": _linear_fwd, "linear_bwd": _linear_bwd}[op](s)


def _threshold(p):
    return min(int(math.floor(65536.0 * p + 0.5)), 65535)


def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011) on int64 tensors of 32-bit values."""
    low = 0xFFFFFFFF
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57      # modulo 2^64: their halves are what is wanted
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _kept(s, rows, width, device):
    """Whether each element of [rows][width] is kept."""
    blocks = -(-width // 8)
    n = torch.arange(rows, device=device)[:, None].expand(rows, blocks)
    b = torch.arange(blocks, device=device)[None, :].expand(rows, blocks)
    offset = torch.full_like(n, s["offset"])
    words = torch.stack(_philox(b, n, offset & 0xFFFFFFFF, offset >> 32, s["seed"] & 0xFFFFFFFF, s["seed"] >> 32), -1)
    fields = torch.stack([words & 0xFFFF, words >> 16], -1).view(rows, 8 * blocks)
    return fields[:, :width] >= _threshold(s["case"]["drop"])


def _drop(s, v):
    p = s["case"]["drop"]
    if p == 0.0:
        return v
    scale = 1.0 / (1.0 - _threshold(p) / 65536.0)
    return torch.where(_kept(s, v.shape[0], v.shape[1], v.device), v * scale, 0.0)


def _joined(s, v):
    r = s["residual"]
    return (v if r is None else v + r.float()).to(s["x"].dtype)


def _drop_rows(s):
    return _joined(s, _drop(s, s["x"].float()))


def _preactivation(s):
    z = torch.matmul(s["x"].float(), s["W"].float())
    return z if s["bias"] is None else z + s["bias"]


def _act(z, act):
    return z if act == "none" else z * torch.sigmoid(z) if act == "silu" else torch.tanh(z)


def _act_grad(z, act):
    if act == "silu":
        e = torch.sigmoid(z)
        return e * (1.0 + z * (1.0 - e))
    return 1.0 - torch.tanh(z) ** 2


def _linear_fwd(s):
    case = s["case"]
    z = _preactivation(s)
    y = _joined(s, _drop(s, _act(z, case["act"])))
    return y, z.to(y.dtype) if case["save"] and case["act"] != "none" else None


def _linear_bwd(s):
    case, dt = s["case"], s["x"].dtype
    dz = _drop(s, s["grad"].float())
    if case["act"] != "none":
        dz = dz * _act_grad(s["z"].float(), case["act"])
    dx = torch.matmul(dz, s["W"].float().t().contiguous())
    dW = torch.matmul(s["x"].float().t().contiguous(), dz)
    return dx.to(dt), dW.to(dt), dz.sum(0) if case["bias"] else None


# ---- the definitions in 64 bits ------------------------------------------------
def _mask64(case, seed, offset):
    """1 / (1 - t / 65536) where an element is kept and 0 where not, in numpy."""
    rows, width = case["rows"], case["cout"]
    out = np.ones((rows, width))
    if case["drop"] == 0.0:
        return out
    t = min(round(case["drop"] * 65536), 65535)
    blocks = (width + 7) // 8
    u, half = np.uint64, np.uint64(32)
    some = max(1, 65536 // blocks)                   # rows at a time, so that arrays stay in a cache
    for n0 in range(0, rows, some):
        n = np.arange(n0, min(n0 + some, rows), dtype=u)
        x = [np.tile(np.arange(blocks, dtype=u), n.size), np.repeat(n, blocks), np.full(n.size * blocks, offset % 2 ** 32, u),
             np.full(n.size * blocks, offset // 2 ** 32, u)]
        for r in range(10):
            k = [(seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
            p, q = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
            x = [(q >> half) ^ x[1] ^ u(k[0]), q & u(2 ** 32 - 1), (p >> half) ^ x[3] ^ u(k[1]), p & u(2 ** 32 - 1)]
        bits = np.stack(x, 1).astype("<u4").view("<u2").reshape(n.size, 8 * blocks)[:, :width]
        out[n0:n0 + some] = np.where(bits >= t, 1.0 / (1.0 - t / 65536.0), 0.0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    mask = torch.from_numpy(_mask64(case, s["seed"], s["offset"])).to(s["x"].device)
    x = s["x"].double()
    r = 0.0 if s["residual"] is None else s["residual"].double()
    if case["op"] == "dropout":
        return r + mask * x
    W, act = s["W"].double(), case["act"]
    slope = {"none": lambda z: 1.0, "tanh": lambda z: torch.cosh(z) ** -2,
             "silu": lambda z: (1 + torch.exp(-z) * (1 + z)) / (1 + torch.exp(-z)) ** 2}[act]
    value = {"none": lambda z: z, "tanh": torch.tanh, "silu": lambda z: z / (1 + torch.exp(-z))}[act]
    if case["op"] == "linear_fwd":
        z = x @ W + (0.0 if s["bias"] is None else s["bias"].double())
        return r + mask * value(z), z if case["save"] and act != "none" else None
    dz = s["grad"].double() * mask
    if act != "none":
        dz = dz * slope(s["z"].double())
    return dz @ W.t(), x.t() @ dz, dz.sum(0) if case["bias"] else None


# ---- what a pass cannot do without ---------------------------------------------
def work(case):
    N, K, M, e = case["rows"], case["cin"], case["cout"], SIZE[case["dtype"]]
    if case["op"] == "dropout":
        return {"bytes": e * N * M * (3 if case["residual"] else 2), "flops": 2 * N * M}
    z = case["act"] != "none"
    small = 4 * M if case["bias"] else 0
    if case["op"] == "linear_fwd":   # x, W and the residual read, y and what is kept written
        arrays = 1 + int(case["residual"]) + int(z and case["save"])
        return {"bytes": e * (N * K + K * M + N * M * arrays) + small, "flops": 2 * N * K * M}
    # the gradient and what was kept, x and W read; the gradients of x, W and the bias written
    return {"bytes": e * (N * M * (1 + int(z)) + 2 * N * K + 2 * K * M) + small, "flops": 4 * N * K * M}
