"""The node-side operators' definitions in numpy and 64 bits, written for
clarity: loops over ids and segments, sums of whole arrays, singular values."""
import numpy as np


def bf16(a):
    """a rounded to bfloat16 (nearest even), as float32."""
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


def embed_fwd(ids, table, scale):
    table = np.asarray(table, np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    for n, i in enumerate(ids):
        if 0 <= i < table.shape[0]:
            out[n] = scale * table[i]
    return out


def embed_bwd(ids, grad, rows, scale):
    grad = np.asarray(grad, np.float64)
    out = np.zeros((rows, grad.shape[1]))
    inside = (ids >= 0) & (ids < rows)
    np.add.at(out, ids[inside], grad[inside])
    return scale * out


def act(kind, z):
    if kind == "none":
        return z
    return z / (1.0 + np.exp(-z)) if kind == "silu" else np.tanh(z)


def act_slope(kind, z):
    if kind == "none":
        return np.ones_like(z)
    if kind == "silu":
        e = np.exp(-z)
        return (1.0 + e + z * e) / (1.0 + e) ** 2
    return 1.0 / np.cosh(z) ** 2


def norm_stats(x, ptr, groups, eps):
    x = np.asarray(x, np.float64)
    B = len(ptr) - 1
    mean, rstd = np.zeros((B, groups)), np.full((B, groups), eps ** -0.5)
    for b in range(B):
        v = x[ptr[b]:ptr[b + 1]].reshape(-1, groups, x.shape[1] // groups)
        if v.shape[0]:
            mean[b] = v.mean((0, 2))
            rstd[b] = 1.0 / np.sqrt(((v - mean[b][None, :, None]) ** 2).mean((0, 2)) + eps)
    return mean, rstd


def _spread(v, ptr, C):
    """[B][G] -> [N][C]"""
    return np.repeat(np.repeat(v, np.diff(ptr), axis=0), C // v.shape[1], axis=1)


def norm_fwd(x, gamma, beta, ptr, groups, eps, kind):
    mean, rstd = norm_stats(x, ptr, groups, eps)
    C = x.shape[1]
    z = (np.asarray(x, np.float64) - _spread(mean, ptr, C)) * _spread(rstd, ptr, C) * gamma + beta
    return act(kind, z), mean, rstd


def norm_bwd(x, gamma, beta, grad, ptr, groups, eps, kind):
    mean, rstd = norm_stats(x, ptr, groups, eps)
    C = x.shape[1]
    xhat = (np.asarray(x, np.float64) - _spread(mean, ptr, C)) * _spread(rstd, ptr, C)
    dz = np.asarray(grad, np.float64) * act_slope(kind, xhat * gamma + beta)
    h = dz * gamma
    dx = np.zeros_like(xhat)
    for b in range(len(ptr) - 1):
        i, j = ptr[b], ptr[b + 1]
        hs, xs = (v[i:j].reshape(j - i, groups, C // groups) for v in (h, xhat))
        if j > i:
            one, two = hs.mean((0, 2), keepdims=True), (hs * xs).mean((0, 2), keepdims=True)
            dx[i:j] = (rstd[b][None, :, None] * (hs - one - xs * two)).reshape(j - i, C)
    return dx, (dz * xhat).sum(0), dz.sum(0)


def orthogonalize(G, steps, coeffs, eps, scale):
    """By the singular values: x -> a x + b x^3 + c x^5, `steps` times.  Also
    the Frobenius norm of every iterate."""
    a, b, c = coeffs
    G = np.asarray(G, np.float64)
    U, x, Vt = np.linalg.svd(G / (np.linalg.norm(G) + eps), full_matrices=False)
    norms = [np.linalg.norm(x)]
    for _ in range(steps):
        x = a * x + b * x ** 3 + c * x ** 5
        norms.append(np.linalg.norm(x))
    return scale * (U * x) @ Vt, norms
