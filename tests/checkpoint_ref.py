"""Checkpoints in 64 bits (numpy), written from the format: e4m3 elements, a power of
two for 32 rows of a column.

Bounds of a sum over rows on the tensor cores (e = 2^-24): products of two e4m3 values and of
powers of two are exact.  A step of 32 rows adds 32 products and the sum so far with at
least fp32's bits, none rounded up: it loses at most 4 e of their magnitudes together; 64 steps
at most follow one another before the sum is added to others, in fp32 (at most 64 of these
here).  So a sum is off by at most (4 * 64 + 64 + 16) e times the sum of its terms'
magnitudes.
"""
import numpy as np

E = 2.0 ** -24
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": E}
SUM = (4 * 64 + 64 + 16) * E


def e4m3_values():
    """The value of every byte."""
    b = np.arange(256)
    exp, man = (b >> 3) & 15, b & 7
    v = np.where(exp > 0, (8 + man) * np.exp2(exp - 10.0), man * 2.0 ** -9)
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >> 7, -v, v)


def exponent(top):
    """The smallest integer e >= -127 with top <= 448 2^e."""
    if top == 0:
        return -127
    e = -127
    while top > 448.0 * 2.0 ** e:
        e += 1
    return e


def store(x, one=False):
    """Bytes [rows, width] and exponents [blocks, width]."""
    x = np.asarray(x, np.float64)
    if one:
        x = np.concatenate([x, np.ones((len(x), 1))], 1)
    rows, width = x.shape
    q = np.zeros((rows, width), np.uint8)
    ex = np.zeros((-(-rows // 32), width), np.int64)
    grid = e4m3_values()[:127]  # 0 .. 448, ascending with the byte
    mid = (grid[1:] + grid[:-1]) / 2
    for t in range(len(ex)):
        b = x[32 * t:32 * t + 32]
        top = np.where(np.isfinite(b), np.abs(b), 0).max(0)
        for c in range(width):
            e = exponent(top[c])
            ex[t, c] = e
            y = np.abs(b[:, c]) * 2.0 ** -e
            if e == 120:
                y = np.minimum(y, 240.0)
            n = np.searchsorted(mid, y, side="left")                 # ties: the lower one ...
            tie = (n < len(mid)) & (mid[np.minimum(n, len(mid) - 1)] == y)
            n = np.where(tie & (n % 2 == 1), n + 1, n)               # ... unless its byte is odd
            n = np.where(np.isfinite(b[:, c]), n, 127)
            q[32 * t:32 * t + 32, c] = np.where(np.signbit(b[:, c]) & np.isfinite(b[:, c]), n + 128, n)
    return q, ex


def values(q, ex):
    return e4m3_values()[q] * np.exp2(np.repeat(ex, 32, 0)[:len(q)].astype(np.float64))


def place(rows, t, c):
    """Where the exponent of block t of column c is."""
    return ((c // 128) * -(-rows // 128) + t // 4) * 512 + c % 32 * 16 + c % 128 // 32 * 4 + t % 4


def scale_bytes(ex, rows):
    width = ex.shape[1]
    out = np.zeros(-(-rows // 128) * -(-width // 128) * 512, np.uint8)
    for t in range(ex.shape[0]):
        c = np.arange(width)
        out[place(rows, t, c)] = ex[t] + 127
    return out


def weight_grad(g, a, alpha, beta=0.0, old=None):
    """beta old + alpha g^T a, and its bound without the last rounding."""
    out, size = alpha * (g.T @ a), abs(alpha) * (np.abs(g).T @ np.abs(a))
    if beta:
        out = out + beta * old
        size = size + abs(beta * old)
    return out, SUM * size
