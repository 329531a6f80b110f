"""The products over 4-bit weights against the 64-bit oracle, through the C ABI.

Exact cases (small integers, scales of powers of two) have sums that fp32 holds whatever their order:
they are compared bit for bit.  Random cases lie within the oracle's worst case of fp32 sums, and their
root mean square within that of independent roundings (both derived beside the oracle).  The pair's
tolerance follows from its products' through silu(g) * u, |silu'| < 1.1, and 8 fp32 steps of the result.
"""
import numpy as np
import pytest
import torch

import block_quantized_weight_02_amd as q8
import oracle
from oracle import w4

pytestmark = pytest.mark.gpu

from tests import gpu_util as g  # noqa: E402
from tests import w4_util as u  # noqa: E402
from tests.w4_util import BF16, Q8, Act, Weight  # noqa: E402

FORMS = [(32, False, 0), (32, True, 1), (64, False, 1), (64, True, 0), (128, False, 0), (128, True, 1)]
SHAPES = [(32, 1), (96, 65), (416, 130), (512, 64)]


@pytest.mark.parametrize("group,zeros,fmt", FORMS)
@pytest.mark.parametrize("K,N", [(32, 1), (160, 70), (512, 200), (1120, 129)])
def test_repack_and_back(K, N, group, zeros, fmt):
    w = Weight(K, N, group, zeros, fmt, 1, points=(0, 256)).pack()
    back = g.empty_bytes(K // 2 * N), g.empty_bytes(w.s.size * 2), g.empty_bytes(w.s.size)
    q8.q8_w4_unpack(w.w, back[0], back[1], back[2] if zeros else None)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(back[0].cpu().numpy()[:w.u.size].reshape(w.u.shape), w.u)
    np.testing.assert_array_equal(back[1].cpu().numpy()[:2 * w.s.size].view(np.uint16).reshape(w.s.shape), w.s)
    if zeros:
        np.testing.assert_array_equal(back[2].cpu().numpy()[:w.z.size].reshape(w.z.shape), w.z)


def test_packed_layout():
    """A dword holds rows 8q .. 8q+7 of a column: row 2p as nibble p, row 2p + 1 as nibble p + 4."""
    K, N, group = 64, 70, 32
    w = Weight(K, N, group, False, 0, 3).pack()
    v = np.zeros((K, 128), np.uint32)
    v[:, :N] = w4.nibbles(w.u)
    got = w.values.cpu().numpy()[:K * 64].view(np.uint32).reshape(2, K // 32, 64, 4)
    for t, b, lane, grp in ((0, 0, 0, 0), (0, 1, 37, 2), (1, 0, 5, 0), (1, 1, 63, 3)):
        c, row = 64 * t + 16 * grp + lane % 16, 32 * b + 8 * (lane // 16)
        want = 0
        for p in range(4):
            want |= int(v[row + 2 * p, c]) << (4 * p) | int(v[row + 2 * p + 1, c]) << (16 + 4 * p)
        assert got[t, b, lane, grp] == want
    s = w.scales.cpu().numpy()[:2 * 256].view(np.uint16).reshape(2, 16, 2, 4)   # tile, lane, group, column
    pad = np.zeros((2, 128), np.uint16)
    pad[:, :N] = w.s
    np.testing.assert_array_equal(s, pad.reshape(2, 2, 4, 16).transpose(1, 3, 0, 2))


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("group,zeros,fmt", FORMS)
@pytest.mark.parametrize("m", [1, 3, 4, 5, 16, 17, 32])
def test_exact(m, group, zeros, fmt, act):
    for K, N in SHAPES:
        w = Weight(K, N, group, zeros, fmt, 5, exact=True).pack()
        a = Act(m, K, act, 7, exact=True)
        got = u.real(u.gemv(a, w), N)
        np.testing.assert_array_equal(got, a.times(w)[0], err_msg=f"{m}x{K}x{N}")


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("group,zeros,fmt", FORMS)
@pytest.mark.parametrize("m", [33, 65, 128, 200])
def test_exact_many_rows(m, group, zeros, fmt, act):
    for K, N in SHAPES:
        w = Weight(K, N, group, zeros, fmt, 5, exact=True).pack()
        a = Act(m, K, act, 9, exact=True)
        got = u.real(u.gemm(a, w), N)
        np.testing.assert_array_equal(got, a.times(w)[0], err_msg=f"{m}x{K}x{N}")


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("group,zeros,fmt", FORMS)
@pytest.mark.parametrize("m", [6, 8, 9, 18, 23, 24, 25])
def test_exact_part_filled_row_groups(m, group, zeros, fmt, act):
    for K, N in ((160, 65), (1120, 130), (64, 24600)):
        w = Weight(K, N, group, zeros, fmt, 5, exact=True).pack()
        a = Act(m, K, act, 7, exact=True)
        np.testing.assert_array_equal(u.real(u.gemv(a, w), N), a.times(w)[0], err_msg=f"{m}x{K}x{N}")


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("group,zeros,fmt", FORMS)
def test_exact_with_as_many_tiles_as_cus_and_more(group, zeros, fmt, act):
    """256 tiles of columns and 258, where the launch takes another shape."""
    for K, N in ((160, 16384), (576, 16449)):
        w = Weight(K, N, group, zeros, fmt, 5, exact=True).pack()
        for m in (1, 4, 7, 13, 17, 24, 32):
            a = Act(m, K, act, 7, exact=True)
            np.testing.assert_array_equal(u.real(u.gemv(a, w), N), a.times(w)[0], err_msg=f"{m}x{K}x{N}")


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("m,K,N,group,zeros,fmt", [
    (1, 4096, 1024, 128, False, 0), (1, 4096, 40, 32, True, 0), (2, 1024, 9000, 64, False, 1),
    (8, 14336, 512, 64, True, 1), (16, 4096, 320, 128, True, 0), (27, 2080, 1000, 32, False, 0),
    (32, 5120, 257, 128, False, 1), (1, 16384, 64, 32, False, 0)])
def test_random(m, K, N, group, zeros, fmt, act):
    w = Weight(K, N, group, zeros, fmt, 11).pack()
    a = Act(m, K, act, 13)
    first = u.gemv(a, w)
    u.compare(u.real(first, N), a.times(w), (m, K, N, group, zeros))
    assert torch.equal(first, u.gemv(a, w)), "two calls differ"


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("m,K,N,group,zeros,fmt", [
    (33, 1056, 300, 64, True, 0), (100, 2048, 640, 128, False, 1), (129, 1024, 1000, 32, True, 0),
    (512, 512, 2000, 128, True, 0), (300, 4096, 130, 64, False, 0), (1024, 256, 4100, 32, False, 1),
    (5, 1024, 100, 128, False, 0)])
def test_random_many_rows(m, K, N, group, zeros, fmt, act):
    w = Weight(K, N, group, zeros, fmt, 17).pack()
    a = Act(m, K, act, 19)
    first = u.gemm(a, w)
    u.compare(u.real(first, N), a.times(w), (m, K, N, group, zeros))
    assert torch.equal(first, u.gemm(a, w)), "two calls differ"


# Sizes with more than 1280 tiles of 64 x 64 (the pair's of 32 x 64): the blocks of 128 rows.
@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("group,zeros,fmt", FORMS)
@pytest.mark.parametrize("m,K,N", [(1025, 32, 5129), (1087, 416, 5000), (4100, 96, 1300)])
def test_exact_blocks(m, K, N, group, zeros, fmt, act):
    w = Weight(K, N, group, zeros, fmt, 5, exact=True).pack()
    a = Act(m, K, act, 9, exact=True)
    np.testing.assert_array_equal(u.real(u.gemm(a, w), N), a.times(w)[0])


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("m,K,N,group,zeros,fmt", [
    (1100, 1056, 4993, 64, True, 0), (1030, 2048, 5100, 128, False, 1), (1281, 544, 4100, 32, True, 1),
    (2000, 1184, 2700, 32, False, 0)])
def test_random_blocks(m, K, N, group, zeros, fmt, act):
    w = Weight(K, N, group, zeros, fmt, 17).pack()
    a = Act(m, K, act, 19)
    first = u.gemm(a, w)
    u.compare(u.real(first, N), a.times(w), (m, K, N, group, zeros))
    assert torch.equal(first, u.gemm(a, w)), "two calls differ"


def test_a_row_of_infinities_stays_in_its_row_of_a_block():
    m, K, N = 1025, 96, 5129
    w = Weight(K, N, 128, False, 0, 31, exact=True).pack()
    a = Act(m, K, BF16, 37, exact=True)
    want = a.times(w)[0]
    bad = [1, 127, 512, m - 1]
    for r in bad:
        a.dev[r] = 0x7F80                          # infinity
    got = u.gemm(a, w).cpu().numpy()[:, :N]
    assert not np.isfinite(got[bad]).any()
    good = np.setdiff1d(np.arange(m), bad)
    np.testing.assert_array_equal(got[good].astype(np.float64), want[good])


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("m", [2, 16, 40])
def test_zero_points_of_a_whole_byte(m, act):
    K, N = 288, 66
    w = Weight(K, N, 32, True, 0, 23, exact=True, points=(0, 256)).pack()
    a = Act(m, K, act, 29, exact=True)
    got = u.real(u.gemv(a, w) if m <= 32 else u.gemm(a, w), N)
    np.testing.assert_array_equal(got, a.times(w)[0])


@pytest.mark.parametrize("m", [3, 20, 70, 130, 290])
def test_a_row_of_infinities_stays_in_its_row(m):
    """K of an odd number of blocks: a stage's reads past a row's end meet the next row."""
    for K, N in ((96, 70), (160, 64), (1056, 320)):
        w = Weight(K, N, 128, False, 0, 31, exact=True).pack()
        a = Act(m, K, BF16, 37, exact=True)
        want = a.times(w)[0]
        bad = [r for r in (1, m // 2, m - 1)]
        for r in bad:
            a.dev[r] = 0x7F80                      # infinity
        got = (u.gemv(a, w) if m <= 32 else u.gemm(a, w)).cpu().numpy()[:, :N]
        for r in range(m):
            if r in bad:
                assert not np.isfinite(got[r]).any()
            else:
                np.testing.assert_array_equal(got[r].astype(np.float64), want[r], err_msg=f"row {r}")


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("m,K,N", [(1, 512, 40), (5, 256, 200), (17, 512, 130), (32, 96, 64), (3, 512, 9000)])
def test_epilogue_exact(m, K, N, act):
    """Bias, residual and the quantized output, bit for bit; the residual may be y."""
    r = np.random.default_rng([m, K, N])
    Npad = q8.q8_padded_cols(N)
    w = Weight(K, N, 64, True, 1, 41, exact=True).pack()
    a = Act(m, K, act, 43, exact=True)
    bias = (r.integers(-64, 65, N) / 8).astype(np.float32)
    res = np.zeros((m, Npad), np.float32)
    res[:, :N] = r.integers(-640, 641, (m, N)) / 8
    want = (a.times(w)[0] + bias + res[:, :N]).astype(np.float32)
    z = np.zeros((m, Npad), np.float32)
    z[:, :N] = want
    codes, scales = oracle.quantize_rows_f32(z)
    y, bias_d, res_d = g.dev(res), g.dev(bias), g.dev(res)
    yq = g.empty_bytes(q8.q8_act_bytes(m, Npad))
    u.gemv(a, w, q8.make_epilogue(bias_d, y, yq), y)
    np.testing.assert_array_equal(u.real(y, N), want.astype(np.float64))
    only = g.empty_bytes(q8.q8_act_bytes(m, Npad))
    u.gemv(a, w, q8.make_epilogue(bias_d, res_d, only, write_y=False))
    for buf in (yq, only):
        c, s = g.act_host(buf, m, Npad)
        np.testing.assert_array_equal(c, codes)
        np.testing.assert_array_equal(s, scales)
        np.testing.assert_array_equal(g.act_view(buf, m, Npad), oracle.act_view_ref(codes))


def pair_tolerance(gate, up, bg, bu):
    G, U = gate[0] + bg, up[0] + bu
    step = 2.0 ** -23
    tg = gate[1] + step * (np.abs(G) + np.abs(bg))
    tu = up[1] + step * (np.abs(U) + np.abs(bu))
    sig = 1 / (1 + np.exp(-G))
    out = G * sig * U
    worst = 1.1 * tg * (np.abs(U) + tu) + (np.abs(G * sig) + 1.1 * tg) * tu + 8 * step * np.abs(out) + 1e-30
    spread = 1.1 * gate[2] * np.abs(U) + np.abs(G * sig) * up[2] + 8 * step * np.abs(out) + 1e-30
    return out, worst, spread


PAIRS = [(1, 32, 1, 32, False, 0), (1, 4096, 1000, 64, False, 0), (4, 1056, 130, 128, True, 1),
         (16, 2048, 9000, 32, True, 0), (29, 1024, 200, 64, True, 1), (32, 512, 64, 128, False, 0),
         (7, 1024, 300, 32, True, 1), (8, 512, 5000, 128, False, 0), (23, 2048, 130, 32, False, 0),
         (24, 544, 9000, 64, True, 0), (40, 512, 300, 32, False, 1), (128, 1024, 200, 128, True, 0),
         (257, 288, 520, 64, False, 0), (600, 544, 4470, 128, True, 0), (1030, 160, 2600, 64, False, 1),
         (641, 288, 4200, 32, True, 1)]


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("m,K,N,group,zeros,fmt,many", [(*p, b) for p in PAIRS for b in (False, True)
                                                        if b or p[0] <= q8.Q8_MAX_ROWS])
def test_pair(m, K, N, group, zeros, fmt, many, act):
    wg, wu = (Weight(K, N, group, zeros, fmt, s).pack() for s in (47, 53))
    a = Act(m, K, act, 59)
    r = np.random.default_rng([m, K, N])
    bias = [r.standard_normal(N).astype(np.float32) for _ in range(2)]
    bg, bu = (g.dev(b) for b in bias)
    gate, up = a.times(wg), a.times(wu)
    y = u.pair(a, wg, wu, None, many)
    u.compare(u.real(y, N), pair_tolerance(gate, up, 0.0, 0.0), "plain")
    Npad = q8.q8_padded_cols(N)
    yq = g.empty_bytes(q8.q8_act_bytes(m, Npad))
    yq.fill_(0x5A)
    y = u.pair(a, wg, wu, q8.make_glu_epilogue(bg, bu, yq), many)
    want = pair_tolerance(gate, up, bias[0].astype(np.float64), bias[1].astype(np.float64))
    got = u.real(y, N)
    u.compare(got, want, "biases")
    # the quantized output is that of the fp32 rows, bit for bit
    z = y.cpu().numpy()
    codes, scales = oracle.quantize_rows_f32(z)
    c, s = g.act_host(yq, m, Npad)
    np.testing.assert_array_equal(c, codes)
    np.testing.assert_array_equal(s, scales)
    np.testing.assert_array_equal(g.act_view(yq, m, Npad), oracle.act_view_ref(codes))
    only = g.empty_bytes(q8.q8_act_bytes(m, Npad))
    untouched = u.blank(m, N)
    u.pair(a, wg, wu, q8.make_glu_epilogue(bg, bu, only, write_y=False), many, untouched)
    c, s = g.act_host(only, m, Npad)
    np.testing.assert_array_equal(c, codes)
    assert torch.isnan(untouched).all()


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
def test_weights_that_end_with_their_allocation(group, zeros, act):
    """Five blocks of 32 rows, no whole stage of any kernel, and values of exactly 10 MiB, which the
    allocator gives an allocation of their own: a stage's loads stay within the last tile."""
    K, N = 160, 1 << 17
    w = Weight(K, N, group, zeros, 0, 113, exact=True)
    torch.cuda.empty_cache()
    w.pack()
    assert w.values.numel() == 10 << 20
    for m in (1, 7, 16, 32, 64, 130):
        a = Act(m, K, act, 109, exact=True)
        got = u.real(u.gemv(a, w) if m <= 32 else u.gemm(a, w), N)
        np.testing.assert_array_equal(got, a.times(w)[0], err_msg=f"{m} rows")


@pytest.mark.parametrize("m", [2, 20, 70, 1025])
def test_large_activations(m):
    """Rows at the header's bound on a bf16 activation, 2^112 (the exact case's largest value is 127)."""
    for zeros in (False, True):
        K, N = 160, 5129 if m > 1000 else 130
        w = Weight(K, N, 128, zeros, 1, 97, exact=True, points=(0, 256)).pack()
        a = Act(m, K, BF16, 101, exact=True)
        want = a.times(w)[0]
        a.dev.copy_(torch.where(a.dev == 0, a.dev, a.dev + (105 << 7)))       # times 2^105
        got = (u.gemv(a, w) if m <= 32 else u.gemm(a, w)).cpu().numpy()[:, :N].astype(np.float64)
        np.testing.assert_array_equal(got * 2.0 ** -105, want)


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("m", [3, 24, 100, 1025])
def test_smallest_scales(m, act):
    """fp16 scales below its normal range (2^-24 .. 2^-21) are exact."""
    K, N = 96, 5129 if m > 1000 else 70
    w = Weight(K, N, 32, False, 0, 103, exact=True)
    w.s = scale_bits_of(w.s, 2.0 ** -21)
    w.canonical = (w.u, w.s, w.z, w.fmt, w.group)
    w.pack()
    a = Act(m, K, act, 107, exact=True)
    got = u.real(u.gemv(a, w) if m <= 32 else u.gemm(a, w), N)
    np.testing.assert_array_equal(got, a.times(w)[0])


@pytest.mark.parametrize("act", [BF16, Q8])
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("m", [3, 24, 100, 1025])
def test_largest_scales(m, group, zeros, act):
    """bf16 scales of 2^123 .. 2^126 over an activation of 2^-110, the product and the pair: nothing on the
    way to an output is larger than it."""
    K, N = 96, 5129 if m > 1000 else 70
    w = Weight(K, N, group, zeros, 1, 127, exact=True)
    w.s = (w.s + (126 << 7)).astype(np.uint16)
    w.canonical = (w.u, w.s, w.z, w.fmt, w.group)
    w.pack()
    a = Act(m, K, act, 131, exact=True)
    x = a.x * 2.0 ** -110
    bits = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    a.dev = g.quantize(bits) if act == Q8 else g.dev(bits.view(np.int16))
    a.x, a.d = x, getattr(a, "d", np.ones(1)) * 2.0 ** -110
    want = a.times(w)[0]
    got = u.real(u.gemv(a, w) if m <= 32 else u.gemm(a, w), N)
    np.testing.assert_array_equal(got, want)
    y = u.real(u.pair(a, w, w, many=m > 32), N)
    with np.errstate(over="ignore"):
        u.compare(y, pair_tolerance((want, 0, 0), (want, 0, 0), 0.0, 0.0), "pair")


def scale_bits_of(bits, factor):
    return (bits.view(np.float16) * np.float16(factor)).view(np.uint16)


def test_one_workspace_serves_every_shape():
    """Splits over one zeroed workspace, products and pairs in turn: its counters end at zero."""
    cases = [(1, 4096, 40), (32, 2048, 300), (7, 1024, 900), (16, 4096, 130)]
    ws = [(Weight(K, N, 128, False, 0, 61).pack(), Weight(K, N, 128, False, 0, 67).pack(), Act(m, K, BF16, 71))
          for m, K, N in cases]
    need = max(max(q8.q8_w4_gemv_workspace_bytes(a.m, w.w, BF16), q8.q8_w4_glu_workspace_bytes(a.m, w.w, BF16))
               for w, _, a in ws)
    buf = torch.zeros(need, dtype=torch.uint8, device=g.DEV)
    for _ in range(3):
        for w, v, a in ws:
            y = u.blank(a.m, w.N)
            q8.q8_w4_gemv(a.dev, w.w, y, a.m, BF16, None, None, buf, need)
            assert torch.equal(y, u.gemv(a, w))
            q8.q8_w4_gemv_glu(a.dev, w.w, v.w, y, a.m, BF16, None, None, buf, need)
            assert torch.equal(y, u.pair(a, w, v))
    assert int(buf[:4 << 20].count_nonzero()) == 0


def test_captured_and_on_another_stream():
    w, v = (Weight(2048, 200, 64, True, 0, s).pack() for s in (73, 79))
    a = Act(4, 2048, BF16, 83)
    want, want2 = u.gemv(a, w), u.pair(a, w, v)
    buf, need = u.workspace(4, w, BF16, True)
    y, y2 = u.blank(4, 200), u.blank(4, 200)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        q8.q8_w4_gemv(a.dev, w.w, y, 4, BF16, None, None, buf, need)
        q8.q8_w4_gemv_glu(a.dev, w.w, v.w, y2, 4, BF16, None, None, buf, need)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(y2, want2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        q8.q8_w4_gemv(a.dev, w.w, y, 4, BF16, None, None, buf, need)
        q8.q8_w4_gemv_glu(a.dev, w.w, v.w, y2, 4, BF16, None, None, buf, need)
    for k in range(4):
        b = Act(4, 2048, BF16, 89 + k)
        a.dev.copy_(b.dev)
        y.zero_()
        y2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, u.gemv(b, w)) and torch.equal(y2, u.pair(b, w, v))
