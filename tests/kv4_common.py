"""The 4-bit cache's format and the rotation, written down a second time in numpy
and 64 bits, for the tests to hold the kernels to."""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                 for e in range(16) for m in range(8)][:127])


def nearest(x, values):
    """Index of the nearest of `values` (ascending) to x >= 0; halfway cases to the even one."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    below, above = x - values[lo], values[hi] - x
    return np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def f32(x):
    return np.asarray(x).astype(np.float32).astype(np.float64)


def quantise(x, unit):
    """x [..., kv_heads, head_dim] (fp32 values): codes [..., head_dim] and scale bytes
    [..., head_dim / 16], by the definition."""
    y = f32(np.asarray(x, np.float64) / np.asarray(unit, np.float64)[:, None])
    y = y.reshape(*y.shape[:-1], y.shape[-1] // 16, 16)
    sb = nearest(f32(np.abs(y).max(-1) / 6.0), E4M3)
    s = E4M3[sb][..., None]
    code = nearest(np.where(s > 0, f32(np.abs(y) / np.where(s > 0, s, 1.0)), 0.0), E2M1)
    code = code + 8 * ((y < 0) & (s > 0))
    return code.reshape(x.shape).astype(np.uint8), sb.astype(np.uint8)


def dequantise(code, sb, unit):
    number = np.concatenate([E2M1, -E2M1])[code].reshape(*code.shape[:-1], code.shape[-1] // 16, 16)
    width = np.concatenate([E4M3, np.full(129, np.nan)])
    return (number * width[sb][..., None]).reshape(code.shape) * \
        np.asarray(unit, np.float64)[:, None]


def split_pool(pool, head_dim):
    """Views of a pool's bytes [blocks + 1, kv_heads, 9 * head_dim]: number pairs
    [.., 16, head_dim / 2] and scales [.., 16, head_dim / 16]."""
    n, h = pool.shape[:2]
    return (pool[..., :8 * head_dim].reshape(n, h, 16, head_dim // 2),
            pool[..., 8 * head_dim:].reshape(n, h, 16, head_dim // 16))


def pool_values(pool, unit):
    """64-bit values [blocks + 1, kv_heads, 16, head_dim] of a pool's bytes (numpy)."""
    data, sb = split_pool(pool, pool.shape[2] // 9)
    code = np.stack([data & 15, data >> 4], -1).reshape(*data.shape[:-1], -1)
    v = dequantise(np.moveaxis(code, 1, -2), np.moveaxis(sb, 1, -2), unit)
    return np.moveaxis(v, -2, 1)


def rotate(x, positions, table, interleaved, rounded):
    """x [tokens, heads, head_dim] rotated in 64 bits; rounded: each product and sum to
    fp32, as the kernels have it."""
    keep = f32 if rounded else (lambda y: y)
    x = np.asarray(x, np.float64).copy()
    row = np.asarray(table, np.float64)[np.asarray(positions)][:, None]
    half = row.shape[-1] // 2
    c, s = row[..., :half], row[..., half:]
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = keep(keep(a * c) - keep(b * s))
    x[..., ib] = keep(keep(b * c) + keep(a * s))
    return x


def table(positions, rotary_dim, base=10000.0):
    half = rotary_dim // 2
    angle = np.arange(positions)[:, None] * base ** (-np.arange(half) / half)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
