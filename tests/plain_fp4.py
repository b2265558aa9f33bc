"""The 4-bit floating-point formats in float64: values of codes and placed scales, rows quantised by the written formulas."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
BLOCK = {"mx": 32, "nv": 16}
E4M3_NAN, E8M0_NAN = 0x7F, 0xFF


def e4m3_values():
    """The value of every non-negative E4M3 byte (0..126), by its fields."""
    b = np.arange(127)
    e, m = b >> 3, b & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def scale_bytes(rows, D, fmt):
    blocks = D // BLOCK[fmt]
    return -(-rows // 128) * -(-blocks // 4) * 512


def scale_index(rows, D, fmt):
    """Where the scale of each row and block lies, [rows][blocks]."""
    blocks = D // BLOCK[fmt]
    pieces = -(-blocks // 4)
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None, :]
    return ((r // 128) * pieces + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4


def scale_values(placed, rows, D, fmt):
    """Scales [rows][blocks] of a buffer (NaN bytes give NaN)."""
    b = np.asarray(placed)[scale_index(rows, D, fmt)].astype(np.int64)
    if fmt == "mx":
        return np.where(b == E8M0_NAN, np.nan, 2.0 ** (b - 127.0))
    table = np.append(e4m3_values(), np.nan)
    return np.concatenate([table, -table])[b]


def code_values(codes, rows, D):
    c = np.asarray(codes).reshape(rows, D // 2)
    c = np.stack([c & 15, c >> 4], axis=-1).reshape(rows, D)
    return np.where(c > 7, -1.0, 1.0) * GRID[c & 7]


def values(codes, placed, rows, D, fmt):
    s = scale_values(placed, rows, D, fmt)
    return code_values(codes, rows, D) * np.repeat(s, BLOCK[fmt], axis=1)


def hadamard(n):
    i = np.arange(n)
    bits = i[:, None] & i[None, :]
    return (1 - 2 * (np.array([bin(v).count("1") for v in bits.ravel()]).reshape(n, n) % 2)) / np.sqrt(n)


def rotate(x, g):
    if not g:
        return np.asarray(x, dtype=np.float64)
    return (np.asarray(x, dtype=np.float64).reshape(-1, g) @ hadamard(g)).reshape(x.shape)


def distance(z, grid):
    """Of each |z|, the distance to the nearest number of an ascending grid (beyond its end: to the end)."""
    z = np.abs(z)
    i = np.clip(np.searchsorted(grid, z), 1, len(grid) - 1)
    return np.where(z > grid[-1], z - grid[-1], np.minimum(np.abs(z - grid[i - 1]), np.abs(grid[i] - z)))


def quantised(x, fmt, factor=1.0):
    """(scales, codes' values) of rows by the formulas; ties to even."""
    v = x.reshape(x.shape[0], -1, BLOCK[fmt]) / (factor if fmt == "nv" else 1.0)
    m = np.abs(v).max(axis=-1)
    if fmt == "mx":
        s = np.where(m >= 2.0 ** -100, 2.0 ** (np.floor(np.log2(np.maximum(m, 2.0 ** -100))) - 2), 0.0)
    else:
        r = np.minimum(m / 6, 448.0)
        step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(r, 2.0 ** -30))), -6) - 3)
        s = np.minimum(np.round(r / step) * step, 448.0)
    z = np.abs(np.divide(v, s[..., None], out=np.zeros_like(v), where=s[..., None] > 0))
    step = np.where(z < 2, 0.5, np.where(z < 4, 1.0, 2.0))
    q = np.minimum(np.round(z / step) * step, 6.0) * np.sign(v)
    return s, q.reshape(x.shape)
