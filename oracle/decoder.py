"""64-bit oracle of what runs between a layer's q/k/v product and its output product -- TEST
INFRASTRUCTURE ONLY, in plain numpy, sharing no code with the HIP path: a step's page tables, the
rotary frequencies, head norms with rotation, the cache layout, and attention over it.

A cache buffer is an array of bytes; ``layout`` gives, for one buffer, the index arrays of a
(slot, head, dim) value, and ``write_rows`` / ``read_rows`` move canonical rows (tokens x heads x
dim) in and out of it.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np

BF16, Q8_0 = 0, 1


def bf16_round(a):
    """Nearest bf16 values (ties to even) of fp32 values, as fp32; finite inputs."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    u = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return u.astype(np.uint32).view(np.float32)


def bf16_bits(a):
    return (bf16_round(a).view(np.uint32) >> 16).astype(np.uint16)


# ---- a step's tables ---------------------------------------------------------------

def kv_step(lens, new, table, free, count, page, m):
    """(table, free, count, lens, row_start, positions, slots, status) after one step, sequence by
    sequence as the definition reads."""
    table, free = np.array(table), np.array(free)
    n, most = table.shape
    ceil = lambda a: -(-a // page)  # noqa: E731
    for i in range(n):
        if new[i] < 0:
            for j in range(ceil(lens[i])):
                if count < len(free):
                    free[count] = table[i, j]
                    count += 1
    have = count
    lens_out = np.zeros(n, np.int32)
    start = np.zeros(n + 1, np.int32)
    positions, slots = np.zeros(m, np.int32), np.full(m, -1, np.int32)
    row = asked = refused = 0
    for i in range(n):
        rows = max(int(new[i]), 0)
        first, row = row, row + rows
        start[i + 1] = min(row, m)
        if new[i] < 0:
            continue
        held, total = ceil(lens[i]), ceil(lens[i] + rows)
        fits = total <= most and row <= m
        need = total - held if fits else 0
        asked += need
        lens_out[i] = lens[i]
        if not fits or (need > 0 and asked > have):
            refused += 1
            continue
        for j in range(held, total):
            count -= 1
            table[i, j] = free[count]
        lens_out[i] += rows
        for r in range(rows):
            p = int(lens[i]) + r
            positions[first + r] = p
            slots[first + r] = table[i, p // page] * page + p % page
    return (table, free, count, lens_out, start, positions, slots,
            np.array([refused, max(0, asked - have)], np.int32))


# ---- heads --------------------------------------------------------------------------

def rope_freqs(base, rot, scaling=0, factor=1.0, low=1.0, high=4.0, original=8192):
    out = []
    for p in range(rot // 2):
        f = base ** (-2.0 * p / rot)
        if scaling == 0:
            keep = 1.0
        elif scaling == 1:
            keep = 0.0
        elif scaling == 2:
            turns = original * f / (2 * math.pi)
            keep = min(max((turns - low) / (high - low), 0.0), 1.0)
        else:
            at = lambda t: rot * math.log(original / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
            a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
            keep = 1.0 - min(max((p - a) / max(b - a, 0.001), 0.0), 1.0)
        out.append(f * keep + f / factor * (1.0 - keep))
    return np.array(out)


def heads(x, norm, eps, freqs, positions, layout, attn_factor):
    """(y, bound): rows x heads x dim in 64 bits, and for each value what its fp32 error scales with:
    the sizes of the two normed values that it mixes."""
    x = np.asarray(x, np.float64)
    if norm is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * norm
    y, bound = x.copy(), np.abs(x)
    half = len(freqs)
    if half:
        i = np.arange(half)
        a, b = (i, i + half) if layout == 0 else (2 * i, 2 * i + 1)
        angle = np.asarray(positions, np.float64)[:, None, None] * freqs
        c, s = np.cos(angle) * attn_factor, np.sin(angle) * attn_factor
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        size = (np.abs(x[..., a]) + np.abs(x[..., b])) * max(1.0, abs(attn_factor))
        bound[..., a] = bound[..., b] = size
    return y, bound


# ---- the cache ----------------------------------------------------------------------

@dataclass(frozen=True)
class Layout:
    fmt: int
    heads: int
    dim: int
    page: int

    @property
    def record(self):
        return self.page * self.dim * 2 if self.fmt == BF16 else self.page * self.dim // 8 * 9

    def nbytes(self, pages):
        return pages * self.heads * self.record

    def value_at(self, which, slots):
        """Byte offsets, tokens x heads x dim."""
        slots = np.asarray(slots, np.int64)
        page, t = slots // self.page, slots % self.page
        d = np.arange(self.dim)[None, None, :]
        h = np.arange(self.heads)[None, :, None]
        t = t[:, None, None]
        inner = (d // 8 * self.page + t) * 8 + d % 8 if which == "k" else (t // 8 * self.dim + d) * 8 + t % 8
        return (page[:, None, None] * self.heads + h) * self.record + inner * (2 if self.fmt == BF16 else 1)

    def scale_at(self, slots):
        """Byte offsets of the fp32 scales, tokens x heads x dim/32."""
        slots = np.asarray(slots, np.int64)
        page, t = slots // self.page, slots % self.page
        b = np.arange(self.dim // 32)[None, None, :]
        h = np.arange(self.heads)[None, :, None]
        return ((page[:, None, None] * self.heads + h) * self.record + self.page * self.dim
                + (b * self.page + t[:, None, None]) * 4)


def write_rows(lay, buf, which, slots, rows):
    """Writes fp32 rows (tokens x heads x dim) into the byte array ``buf`` in the cache's format;
    returns the values that the cache then stands for, in 64 bits."""
    at = lay.value_at(which, slots)
    if lay.fmt == BF16:
        bits = bf16_bits(rows)
        buf[at], buf[at + 1] = (bits & 255).astype(np.uint8), (bits >> 8).astype(np.uint8)
        return bf16_round(rows).astype(np.float64)
    from . import quantize_rows_f32
    flat = np.ascontiguousarray(rows, np.float32).reshape(len(rows), lay.heads * lay.dim)
    code, d = quantize_rows_f32(flat)
    code, d = code.reshape(rows.shape), d.reshape(*rows.shape[:2], lay.dim // 32)
    buf[at] = code.view(np.uint8)
    raw = d.astype(np.float32).view(np.uint8).reshape(*d.shape, 4)
    for e in range(4):
        buf[lay.scale_at(slots) + e] = raw[..., e]
    return code.astype(np.float64) * np.repeat(d.astype(np.float64), 32, -1)


def read_rows(lay, buf, which, slots):
    at = lay.value_at(which, slots)
    if lay.fmt == BF16:
        u = buf[at].astype(np.uint32) << 16 | buf[at + 1].astype(np.uint32) << 24
        return u.view(np.float32).astype(np.float64)
    sc = lay.scale_at(slots)
    raw = np.stack([buf[sc + e] for e in range(4)], -1)
    d = np.ascontiguousarray(raw).view(np.float32)[..., 0]
    return buf[at].view(np.int8).astype(np.float64) * np.repeat(d.astype(np.float64), 32, -1)


# ---- attention ------------------------------------------------------------------------

def attention(q, k, v, positions, scale, window=0, sinks=0, present=None):
    """(o, bound, spread, size) in 64 bits of rows q (rows x heads x dim) at their positions over the
    tokens k, v (tokens x kv_heads x dim); present: which tokens exist.  bound = sum of p |v|, what
    roundings of the probabilities scale with at the worst; spread = sqrt(sum of (p v)^2), what they
    scale with when they are independent; size = for each (row, head) the largest |scale| sum |q k| of
    a token that it sees."""
    rows, hq, dim = q.shape
    group = hq // k.shape[1] if len(k) else 1
    o, bound, spread = (np.zeros((rows, hq, dim)) for _ in range(3))
    size = np.zeros((rows, hq))
    t = np.arange(len(k))
    for r in range(rows):
        see = t <= positions[r]
        if window:
            see &= (t > positions[r] - window) | (t < sinks)
        if present is not None:
            see &= present
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[see, h // group], v[see, h // group]
            s = scale * (kk @ q[r, h])
            size[r, h] = (abs(scale) * (np.abs(kk) @ np.abs(q[r, h]))).max()
            p = np.exp(s - s.max())
            p /= p.sum()
            o[r, h], bound[r, h] = p @ vv, p @ np.abs(vv)
            spread[r, h] = np.sqrt((p * p) @ (vv * vv))
    return o, bound, spread, size
