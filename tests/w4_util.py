"""Helpers of the 4-bit weight's GPU tests: canonical weights, their packed form, calls."""
import numpy as np
import torch

import block_quantized_weight_02_amd as q8
from oracle import decoder as dec
from oracle import w4
from tests import gpu_util as g

BF16, Q8 = q8.Q8_ACT_BF16, q8.Q8_ACT_Q8_0


def scale_bits(values, fmt):
    if fmt == w4.F16:
        return values.astype(np.float16).view(np.uint16)
    return dec.bf16_bits(values.astype(np.float32))


class Weight:
    """A canonical weight drawn from a seed (exact: scales of powers of two), packed on the GPU."""

    def __init__(self, K, N, group, zeros, fmt, seed, exact=False, points=(5, 11)):
        r = np.random.default_rng([seed, K, N, group, int(zeros), fmt])
        self.K, self.N, self.group, self.fmt = K, N, group, fmt
        groups = -(-K // group)
        self.u = r.integers(0, 256, (K // 2, N), dtype=np.uint8)
        s = 2.0 ** r.integers(-3, 1, (groups, N)) if exact else \
            np.exp(0.4 * r.standard_normal((groups, N))) * 0.2 / np.sqrt(K)
        s = np.where(r.random((groups, N)) < 0.1, -s, s)
        self.s = scale_bits(s, fmt)
        self.z = r.integers(*points, (groups, N), dtype=np.int64).astype(np.uint8) if zeros else None
        self.canonical = (self.u, self.s, self.z, fmt, group)

    def pack(self):
        zeros = self.z is not None
        self.values = g.empty_bytes(q8.q8_w4_values_bytes(self.K, self.N))
        self.scales = g.empty_bytes(q8.q8_w4_scales_bytes(self.K, self.N, self.group, zeros))
        self.values.fill_(0xA5)
        self.scales.fill_(0xA5)
        self.w = q8.make_w4_weight(self.values, self.scales, self.K, self.N, self.group, self.fmt, zeros)
        q8.q8_w4_repack(g.dev(self.u), g.dev(self.s.view(np.int16)),
                        g.dev(self.z) if zeros else None, self.w)
        return self


class Act:
    """Rows of bf16 (or of their quantized form) and their 64-bit values."""

    def __init__(self, m, K, act, seed, exact=False):
        r = np.random.default_rng([seed, m, K])
        x = r.integers(-8, 9, (m, K)).astype(np.float32) if exact else r.standard_normal((m, K))
        if exact:
            x[:, ::32] = 127.0            # a quantized block's scale is then 1
        bits = dec.bf16_bits(x.astype(np.float32))
        self.m, self.K, self.act = m, K, act
        self.x = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        if act == Q8:
            self.dev = g.quantize(bits)
            self.q, self.d = g.act_host(self.dev, m, K)
        else:
            self.dev = g.dev(bits.view(np.int16))

    def times(self, weight):
        if self.act == Q8:
            return w4.product_q8(self.q, self.d, *weight.canonical)
        return w4.product(self.x, *weight.canonical)


def blank(m, N):
    return torch.full((m, q8.q8_padded_cols(N)), float("nan"), dtype=torch.float32, device=g.DEV)


def workspace(m, w, act, pair=False):
    need = (q8.q8_w4_glu_workspace_bytes if pair else q8.q8_w4_gemv_workspace_bytes)(m, w.w, act)
    return (torch.zeros(need, dtype=torch.uint8, device=g.DEV) if need else None), need


def gemv(a, w, ep=None, y=None, ws=None, stream=None):
    y = blank(a.m, w.N) if y is None else y
    buf, need = ws or workspace(a.m, w, a.act)
    q8.q8_w4_gemv(a.dev, w.w, y, a.m, a.act, ep, stream, buf, need)
    return y


def gemm(a, w):
    y = blank(a.m, w.N)
    q8.q8_w4_gemm(a.dev, w.w, y, a.m, a.act)
    return y


def pair(a, wg, wu, ep=None, many=False, y=None):
    y = blank(a.m, wg.N) if y is None else y
    if many:
        q8.q8_w4_gemm_glu(a.dev, wg.w, wu.w, y, a.m, a.act, ep)
    else:
        buf, need = workspace(a.m, wg, a.act, True)
        q8.q8_w4_gemv_glu(a.dev, wg.w, wu.w, y, a.m, a.act, ep, None, buf, need)
    return y


def real(y, N):
    """The N columns of an output on the host; its pad columns are +0."""
    y = y.cpu().numpy()
    assert (y[:, N:].view(np.uint32) == 0).all(), "pad columns"
    return y[:, :N].astype(np.float64)


def compare(got, want, what):
    y, worst, spread = want
    err = np.abs(got - y)
    limit = worst + np.abs(y) * 2.0 ** -23 + 1e-30
    assert np.isfinite(got).all(), what
    assert (err <= limit).all(), (what, float((err / limit).max()))
    rms = lambda a: float(np.sqrt(np.mean(a * a)))  # noqa: E731
    assert rms(err) <= rms(spread) + 1e-30, (what, rms(err), rms(spread))
