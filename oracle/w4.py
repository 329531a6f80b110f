"""64-bit oracle of the products over 4-bit weights -- TEST INFRASTRUCTURE ONLY, in plain numpy,
sharing no code with the HIP path.

A canonical weight: u (K/2 x N bytes), s (groups x N 16-bit patterns), z (groups x N bytes, or None).
"""
from __future__ import annotations

import numpy as np

F16, BF16 = 0, 1


def scale_values(s, fmt):
    if fmt == F16:
        return s.view(np.float16).astype(np.float64)
    return (s.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def nibbles(u):
    """K x N values of 0 .. 15."""
    v = np.empty((2 * u.shape[0], u.shape[1]), np.int64)
    v[0::2], v[1::2] = u & 15, u >> 4
    return v


def points(z, groups, n):
    return np.full((groups, n), 8, np.int64) if z is None else z.astype(np.int64)


def weight(u, s, z, fmt, group):
    """K x N values in 64 bits."""
    v = nibbles(u)
    sc = scale_values(s, fmt)
    row = np.arange(v.shape[0]) // group
    return (v - points(z, *s.shape)[row]) * sc[row]


def product(x, u, s, z, fmt, group):
    """(y, worst, spread) of bf16 rows x (as fp64): the product, the most that fp32 sums may be off, and
    the root mean square that independent roundings of them have.

    The kernels add x (16 + u) and subtract (16 + z) sum x, both in fp32: with A = sum |x| (32 + u + z)
    of a group, every partial sum is below A, there are at most 2 group + 8 of them, and each rounding
    (or cut) is below 2^-23 of it.  The scaled sums join in groups + 32 additions (groups, waves,
    splits, epilogue) of at most sum |s| A."""
    v, sc, zp = nibbles(u), scale_values(s, fmt), points(z, *s.shape)
    K, n = v.shape
    y, size, square = (np.zeros((x.shape[0], n)) for _ in range(3))
    ax = np.abs(x)
    for j in range(s.shape[0]):
        a, b = j * group, min(K, (j + 1) * group)
        y += (x[:, a:b] @ v[a:b] - x[:, a:b].sum(1, keepdims=True) * zp[j]) * sc[j]
        t = (ax[:, a:b] @ (v[a:b] + 32) + ax[:, a:b].sum(1, keepdims=True) * zp[j]) * np.abs(sc[j])
        size += t
        square += t * t
    groups = s.shape[0]
    eps = 2.0 ** -23
    return y, eps * (2 * group + 8 + groups + 32) * size, \
        eps * np.sqrt((2 * group + 8) * square + (groups + 32) * np.square(np.abs(y) + np.sqrt(square)))


def product_q8(xq, dx, u, s, z, fmt, group):
    """The same of int8 rows xq with scales dx (m x K/32): a block's dot is exact; its scaling takes at
    most four fp32 roundings, and the blocks' sum K/32 + 32 additions."""
    v, sc, zp = nibbles(u), scale_values(s, fmt), points(z, *s.shape)
    K, n = v.shape
    y, size, square = (np.zeros((xq.shape[0], n)) for _ in range(3))
    for b in range(K // 32):
        rows = slice(32 * b, 32 * b + 32)
        j = 32 * b // group
        d = xq[:, rows].astype(np.float64) @ (v[rows] - zp[j])
        t = d * dx[:, b:b + 1].astype(np.float64) * sc[j]
        y += t
        size += np.abs(t)
        square += t * t
    eps = 2.0 ** -23
    return y, eps * (K // 32 + 36) * size, eps * np.sqrt(8 * square + (K // 32 + 32) * np.square(np.abs(y) + np.sqrt(square)))
