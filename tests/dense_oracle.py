"""The dense operators' definitions in numpy and 64 bits, written for clarity:
the generator on Python integers' arithmetic, the products as whole matrices."""
import numpy as np

from tests.train_oracle import act, act_slope

LOW = np.uint64(0xFFFFFFFF)
M0, M1, W0, W1 = np.uint64(0xD2511F53), np.uint64(0xCD9E8D57), 0x9E3779B9, 0xBB67AE85


def philox(counter, key):
    """Philox4x32-10 of Salmon, Moraes, Dror and Shaw (2011): counter, four
    arrays of 32-bit values (as uint64), key, two integers; four arrays."""
    x0, x1, x2, x3 = (np.asarray(c, np.uint64) for c in counter)
    for r in range(10):
        k0 = np.uint64((key[0] + r * W0) & 0xFFFFFFFF)
        k1 = np.uint64((key[1] + r * W1) & 0xFFFFFFFF)
        p, q = M0 * x0, M1 * x2
        x0, x1, x2, x3 = (q >> np.uint64(32)) ^ x1 ^ k0, q & LOW, (p >> np.uint64(32)) ^ x3 ^ k1, p & LOW
    return x0, x1, x2, x3


def threshold(p):
    return min(int(np.floor(65536 * p + 0.5)), 65535)


def mask(rows, channels, p, seed, offset):
    """1 / (1 - t / 65536) where (n, c) is kept and 0 where not."""
    t = threshold(p)
    if t == 0:
        return np.ones((rows, channels))
    blocks = (channels + 7) // 8
    n, b = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    offset %= 1 << 64
    words = philox((b, n, np.full(b.shape, offset & 0xFFFFFFFF), np.full(b.shape, offset >> 32)),
                   (seed & 0xFFFFFFFF, seed >> 32))
    out = np.empty((rows, blocks, 8))
    for j in range(8):
        out[:, :, j] = (words[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xFFFF)
    keep = out.reshape(rows, 8 * blocks)[:, :channels] >= t
    return np.where(keep, 1.0 / (1.0 - t / 65536.0), 0.0)


def masked(m, v):
    """v times the mask; zero where it is zero, whatever v holds there."""
    return np.where(m == 0.0, 0.0, m * np.where(m == 0.0, 0.0, v))


def linear_fwd(x, W, bias, residual, kind, m):
    z = np.asarray(x, np.float64) @ np.asarray(W, np.float64) + (0.0 if bias is None else bias)
    return masked(m, act(kind, z)) + (0.0 if residual is None else residual), z


def linear_bwd(x, W, z, grad, kind, m):
    dz = masked(m, np.asarray(grad, np.float64) * act_slope(kind, np.asarray(z, np.float64)))
    return dz @ np.asarray(W, np.float64).T, np.asarray(x, np.float64).T @ dz, dz.sum(0), dz
