"""64-bit oracle of the rules on logits and of the drawn token -- TEST INFRASTRUCTURE ONLY, in plain
numpy, row by row as the definitions read, sharing no code with the HIP path."""
from __future__ import annotations

import math

import numpy as np


def rules(x, tokens=(), prompt=0, repetition=1.0, presence=0.0, frequency=0.0, biases=(), mask=None):
    """(values in 64 bits, the most that their fp32 roundings may be off) of one row.  ``biases``: pairs
    (token, value); ``mask``: 32-bit words or None."""
    y = x.astype(np.float64)
    v = len(y)
    off = np.zeros(v)
    step = 2.0 ** -23

    def past_range(t):
        """A value that rounds past fp32's largest is infinite."""
        if math.isfinite(y[t]) and abs(y[t]) >= 2.0 ** 128 * (1 - 2.0 ** -25):
            y[t] = math.copysign(math.inf, y[t])

    here = [t for t in tokens if 0 <= t < v]
    for t in set(here):
        if repetition != 1.0:
            y[t] = y[t] / np.float64(np.float32(repetition)) if y[t] > 0 else y[t] * np.float64(np.float32(repetition))
            past_range(t)
            off[t] += step * abs(y[t])
    made, count = np.unique([t for t in list(tokens)[max(prompt, 0):] if 0 <= t < v], return_counts=True)
    for t, c in zip(made.astype(int), count):
        a, b = float(np.float32(frequency)) * c, float(np.float32(presence))
        off[t] += 3 * step * (abs(y[t]) + abs(a) + abs(b))
        y[t] = y[t] - a - b
        past_range(t)
    for t, value in dict((t, w) for t, w in biases).items():
        if 0 <= t < v:
            y[t] += float(np.float32(value))
            past_range(t)
            off[t] += 2 * step * (abs(y[t]) + abs(value))
    if mask is not None:
        for t in range(v):
            if not int(mask[t // 32]) >> (t % 32) & 1:
                y[t] = -math.inf
                off[t] = 0.0
    return y, off


def logprob(x, token):
    """Log-probability of a token of the row, in 64 bits."""
    x = x.astype(np.float64)
    x = np.where(np.isnan(x), -math.inf, x)
    top = x.max()
    if top == -math.inf:
        return -math.inf
    with np.errstate(invalid="ignore"):
        e = np.where(x == top, 1.0, np.exp(x - top))
        return (0.0 if x[token] == top else x[token] - top) - math.log(e.sum())


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The tokens that may be drawn: one, or where u (or top_p's cut) lies within the weights' own
    precision of a boundary, those on both sides.  A weight is rounded to a multiple of 2^-sh of the
    largest and computed to 1e-13, so a sum of them is off by at most V 2^-(sh+1) + 1e-13 W; twice that
    where two sums are compared, and 2^-51 W for the comparison in fp64."""
    x = x.astype(np.float64)
    x = np.where(np.isnan(x), -math.inf, x)
    v = len(x)
    top = x.max()
    if top == -math.inf:
        return {-1}
    if not temperature > 0:
        return {int(x.argmax())}
    with np.errstate(invalid="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / float(np.float32(temperature))))
    w[x == -math.inf] = 0.0
    sh = min(51, 62 - v.bit_length())
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -math.inf]
    mass = np.cumsum(w[order])
    eps = 2 * (v * 2.0 ** -(sh + 1) + 1e-13 * mass[-1]) + 2.0 ** -51 * mass[-1]
    p = float(np.float32(top_p))
    n = len(order) if not 0 < top_k < v else min(top_k, len(order))
    cuts = {n}
    if p < 1:
        cuts = {min(n, max(1, 1 + int(np.searchsorted(mass, p * mass[-1] + d, side="left")))) for d in (-eps, 0.0, eps)}
    low = min(1.0, float(np.float32(min_p)))
    found = set()
    for n in cuts:
        kept = np.zeros(v, bool)
        kept[order[:n]] = True
        cdf = np.cumsum(np.where(kept & (w >= low), w, 0.0))
        at = min(max(u, 0.0), 1.0) * cdf[-1]
        for d in (-eps, 0.0, eps):
            t = int(np.searchsorted(cdf, max(at + d, 0.0), side="right"))
            found.add(min(t, int(np.flatnonzero(kept & (w >= low)).max())))
    return found
