"""Attention over the paged cache -- one row a sequence and chunks of rows -- against the 64-bit oracle
on a GPU: formats, shapes, lengths and masks where it can go wrong, and a layer's calls together."""
import numpy as np
import pytest
import torch

import block_quantized_weight_02_amd as q8
from block_quantized_weight_02_amd import inputs
from oracle import decoder as dec

pytestmark = pytest.mark.gpu

from tests import gpu_util as g  # noqa: E402
from tests import decoder_util as u  # noqa: E402

BF16, Q8 = q8.Q8_KV_BF16, q8.Q8_KV_Q8_0


def want_of(s, q, counts, scale, window=0, sinks=0, present=None):
    """The oracle over every sequence's rows, its last ones."""
    none = np.zeros((0,) + q.shape[1:])
    out, at = [(none, none, none, none[..., 0])], 0
    for i, c in enumerate(counts):
        pos = np.arange(s.lens[i] - c, s.lens[i])
        out.append(dec.attention(q[at:at + c], s.k[i], s.v[i], pos, scale, window, sinks,
                                 None if present is None else present[i]))
        at += c
    return tuple(np.concatenate([o[j] for o in out]) for j in range(4))


def queries(s, m, group, seed, big=1.0):
    q = np.random.default_rng(seed).standard_normal((m, s.lay.heads * group, s.lay.dim)) * big
    return dec.bf16_round(q.astype(np.float32)).astype(np.float64)


def check_decode(s, group, window=0, sinks=0, scale=None, seed=1, big=1.0, present=None, what=""):
    dim = s.lay.dim
    scale = dim ** -0.5 if scale is None else scale
    q = queries(s, s.n, group, seed, big)
    qd = u.bf16_dev(q)
    o = torch.full((s.n, q.shape[1], dim), 7.0, dtype=torch.bfloat16, device=g.DEV)
    oq = g.empty_bytes(q8.q8_act_bytes(s.n, q.shape[1] * dim))
    attn = q8.make_attn(scale, window, sinks)
    ws = s.workspace(0, q.shape[1])
    u.decode(s, qd, attn, o, oq, ws=ws)
    only, onlyq = torch.zeros_like(o), torch.zeros_like(oq)
    u.decode(s, qd, attn, only, None, ws=ws)
    u.decode(s, qd, attn, None, onlyq, ws=ws)
    torch.cuda.synchronize()
    assert not ws[0][:4 << 20].any()
    assert torch.equal(o, only)                              # the same again, whatever is asked for
    want = want_rows(s, q, scale, window, sinks, present)
    u.compare(u.host(o), want, int(s.lens.max()), dim, what)
    assert (u.host(o)[s.lens == 0] == 0).all()
    xq, dx = u.compare_q8(oq, want, int(s.lens.max()), dim, what)
    for a, b in zip((xq, dx), g.act_host(onlyq, s.n, q.shape[1] * dim)):
        np.testing.assert_array_equal(a, b)
    return u.host(o)


def want_rows(s, q, scale, window, sinks, present):
    out = [dec.attention(q[i:i + 1], s.k[i], s.v[i], [s.lens[i] - 1], scale, window, sinks,
                         None if present is None else present[i]) for i in range(s.n)]
    return tuple(np.concatenate([o[j] for o in out]) for j in range(4))


def check_rows(s, group, counts, window=0, sinks=0, scale=None, seed=1, big=1.0, present=None, pad=3, what=""):
    dim = s.lay.dim
    scale = dim ** -0.5 if scale is None else scale
    m = int(sum(counts))
    q = queries(s, m + pad, group, seed, big)
    q[m:] = np.nan                                           # rows behind the last sequence: not read into any
    qd = u.bf16_dev(np.nan_to_num(q))
    qd[m:] = float("nan")
    start = g.dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    o = torch.full((m + pad, q.shape[1], dim), 7.0, dtype=torch.bfloat16, device=g.DEV)
    K = q.shape[1] * dim
    oq = torch.full((q8.q8_act_bytes(m + pad, K),), 91, dtype=torch.uint8, device=g.DEV)
    attn = q8.make_attn(scale, window, sinks)
    ws = s.workspace(m + pad, q.shape[1])
    u.rows(s, qd, start, attn, o, oq, ws=ws)
    only, onlyq = torch.full_like(o, 7.0), torch.full_like(oq, 91)
    u.rows(s, qd, start, attn, only, None, ws=ws)
    u.rows(s, qd, start, attn, None, onlyq, ws=ws)
    torch.cuda.synchronize()
    assert ws[0] is None or not ws[0][:4 << 20].any()
    assert torch.equal(o, only) and torch.equal(oq, onlyq)
    want = want_of(s, q[:m], counts, scale, window, sinks, present)
    u.compare(u.host(o)[:m], want, int(s.lens.max()), dim, what)
    assert (u.host(o)[m:] == 7.0).all()
    # the quantized rows: compared as a buffer of m + pad rows whose last ones were left alone
    xq, dx = u.compare_q8(oq, want, int(s.lens.max()), dim, what, pad)
    assert (xq[m:].view(np.uint8) == 91).all() and (dx[m:].view(np.uint8) == 91).all()
    return u.host(o)[:m]


# ---- one row a sequence -----------------------------------------------------------------

@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 256])
def test_decode(fmt, dim, page):
    s = u.Scene(fmt, 2, dim, page, [1, 0, 2, 31, 32, 33, 65, 300, 16, 17], seed=dim + page).to_device()
    check_decode(s, 4)


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (1, 8), (2, 7), (1, 16), (2, 17), (1, 40), (8, 5), (128, 8)])
def test_decode_heads(fmt, heads, group):
    s = u.Scene(fmt, heads, 64, 16, [40, 3, 129], seed=heads * group).to_device()
    check_decode(s, group)
    if heads < 4:
        s = u.Scene(fmt, heads, 128, 64, [70, 0, 200], seed=heads * group).to_device()
        check_decode(s, group)


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("dim,lens", [(128, [5000]), (64, [4097, 1]), (128, [1, 2, 9001, 3, 700]), (256, [3000, 64]),
                                      (128, [777] * 9)])
def test_decode_split(fmt, dim, lens):
    """Long sequences: their pieces meet through the workspace."""
    s = u.Scene(fmt, 2, dim, 16 if dim != 256 else 64, lens, seed=len(lens) + dim).to_device()
    check_decode(s, 4)


def test_decode_many_sequences():
    r = np.random.default_rng(3)
    lens = r.integers(0, 40, 1000)
    lens[r.random(1000) < 0.2] = 0
    check_decode(u.Scene(BF16, 1, 64, 16, lens.tolist(), seed=3).to_device(), 2)
    lens = r.integers(0, 90, 300)
    check_decode(u.Scene(Q8, 2, 128, 32, lens.tolist(), seed=4).to_device(), 2)
    lens = np.zeros(8192, int)
    lens[[0, 77, 4000, 8191]] = [9, 1, 50, 33]
    check_decode(u.Scene(BF16, 1, 64, 16, lens.tolist(), seed=5).to_device(), 1)
    check_decode(u.Scene(BF16, 1, 64, 16, [0, 0, 0], seed=6).to_device(), 4)


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 3), (100, 4), (33, 40), (500, 0), (64, 10 ** 6),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
def test_decode_window(fmt, window, sinks):
    s = u.Scene(fmt, 2, 128, 16, [1, 16, 17, 33, 100, 101, 499, 500, 1300], seed=window % 1000).to_device()
    check_decode(s, 4, window, sinks)


@pytest.mark.parametrize("fmt", [BF16, Q8])
def test_decode_counts_every_token_once(fmt):
    """Equal scores: every probability is the same power of two of the largest, and the values are small
    whole numbers, so a sum of them is exact and only the division and the last rounding are not."""
    r = np.random.default_rng(8)
    for dim, page, lens in ((128, 16, [1, 45, 1001, 64]), (64, 64, [777, 63, 64, 65]), (256, 32, [513, 31])):
        s = u.Scene(fmt, 2, dim, page, lens, seed=dim)
        for i, l in enumerate(lens):
            # a block's largest is 127, so that Q8_0 codes are the values
            v = r.integers(-100, 101, (l, 2, dim)).astype(np.float32)
            v[..., ::32] = 127.0
            s.v[i] = s.put("v", i, v)
            np.testing.assert_array_equal(s.v[i], v)
        s.to_device()
        qd = torch.zeros((s.n, 8, dim), dtype=torch.bfloat16, device=g.DEV)
        for window, sinks in ((0, 0), (40, 3)):
            o = torch.zeros_like(qd)
            u.decode(s, qd, q8.make_attn(1.0, window, sinks), o)
            orows = torch.zeros_like(qd)
            u.rows(s, qd, g.dev(np.arange(s.n + 1, dtype=np.int32)), q8.make_attn(1.0, window, sinks), orows)
            torch.cuda.synchronize()
            want = want_rows(s, np.zeros((s.n, 8, dim)), 1.0, window, sinks, None)[0]
            for got in (o, orows):
                assert (np.abs(u.host(got) - want) <= np.abs(want) * u.HALF_BF16 + 127 * 8 * u.EPS32).all()


@pytest.mark.parametrize("fmt", [BF16, Q8])
def test_scales_of_either_sign(fmt):
    s = u.Scene(fmt, 2, 128, 16, [100, 1, 37, 300], seed=12).to_device()
    for scale in (-0.1, 0.0, 1.0, 1e-30):
        check_decode(s, 4, scale=scale, what=scale)
        check_rows(s, 4, [50, 1, 20, 3], scale=scale, what=scale)
    # scores of some thousands: one token takes nearly all
    check_decode(s, 4, scale=4.0, big=16.0)
    check_rows(s, 4, [50, 1, 20, 3], scale=4.0, big=16.0)


def leading(s, i, positions, score, window, sinks):
    """The mean value of the seen tokens of the largest score: what the softmax of scores too far apart
    to share leaves.  score: one number a token."""
    t = np.arange(s.lens[i])
    out = np.zeros((len(positions), s.lay.heads, s.lay.dim))
    for j, p in enumerate(positions):
        see = t <= p
        if window:
            see &= (t > p - window) | (t < sinks)
        out[j] = s.v[i][see & (score == score[see].max())].mean(0)
    return out


def check_far_scores(fmt, dim, scales):
    """Scores of the scales' size and either sign: the largest of a row counts in full, so equal ones share
    evenly and smaller ones, this far apart, count nothing.  Every token's key is +-1.015625 in dim 0 and 0
    elsewhere, the queries 1.0078125 there, so a product has bits that its fp32 score rounds away.

    All tokens that count have the same probability, rounded to bf16 once; the values are whole numbers to
    127, so a sum of n of them is off by at most n roundings of it; the output is rounded once."""
    r = np.random.default_rng(dim)
    lens, counts, group = [1, 2, 40, 700], [1, 2, 33, 300], 4
    odd = [None, None, 3, 399]                     # a token of the other sign, near its sequence's first rows
    for far in (False, True):
        s = u.Scene(fmt, 2, dim, 16, lens, seed=dim)
        score = []
        for i, l in enumerate(lens):
            v = r.integers(-100, 101, (l, 2, dim)).astype(np.float32)
            v[..., ::32] = 127.0                   # Q8_0 codes are the values
            s.v[i] = s.put("v", i, v)
            k = np.zeros((l, 2, dim), np.float32)
            k[..., 0] = 1.015625
            if far and odd[i] is not None:
                k[odd[i], :, 0] = -1.015625
            s.k[i] = s.put("k", i, k)
            score.append(np.sign(k[:, 0, 0]))
        s.to_device()
        m = sum(counts)
        q = torch.zeros((m, 2 * group, dim), dtype=torch.bfloat16, device=g.DEV)
        q[..., 0] = 1.0078125
        start = g.dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
        for scale in scales:
            for sign in (1, -1):
                for window, sinks in ((0, 0), (40, 3)):
                    attn = q8.make_attn(sign * scale, window, sinks)
                    o, one = torch.zeros_like(q), torch.zeros_like(q[:4])
                    u.rows(s, q, start, attn, o)
                    u.decode(s, q[:4], attn, one)
                    torch.cuda.synchronize()
                    for got, rows in ((u.host(o), counts), (u.host(one), [1] * 4)):
                        at = 0
                        for i, c in enumerate(rows):
                            pos = np.arange(lens[i] - c, lens[i])
                            want = np.repeat(leading(s, i, pos, sign * score[i], window, sinks), group, 1)
                            tol = np.abs(want) * u.HALF_BF16 * (2 + u.HALF_BF16) + (lens[i] + 8) * 127 * u.EPS32
                            err = np.abs(got[at:at + c] - want)
                            assert (err <= tol).all(), (far, sign * scale, window, i, c, float(np.nanmax(err)))
                            at += c


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scores_of_any_size(fmt, dim):
    """Also scores whose fp32 rounding is many powers of two."""
    check_far_scores(fmt, dim, (3e6, 7e7, 1e9, 3e15, 1e38))


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scores_near_the_lowest(fmt, dim):
    """Rows whose every score, in powers of two, lies between -3.4e38 and -3e38."""
    check_far_scores(fmt, dim, (2.2e38,))



def poison(s, which, i, first, end, kind):
    """Bytes of tokens first .. end of sequence i: NaN, infinities or the types' largest values."""
    buf = s.kbuf if which == "k" else s.vbuf
    at = s.lay.value_at(which, s.slots(i, first, end))
    value = {"nan": np.float32(np.nan), "inf": np.float32(np.inf), "ninf": np.float32(-np.inf),
             "huge": np.float32(3.3e38)}[kind]
    bits = value.view(np.uint32) >> 16
    if s.lay.fmt == BF16:
        buf[at], buf[at + 1] = bits & 255, bits >> 8
    else:
        sc = s.lay.scale_at(s.slots(i, first, end))
        for b in range(4):
            buf[sc + b] = np.float32(value).view(np.uint32) >> (8 * b) & 255
        buf[at] = 127


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scores_of_minus_infinity(fmt, dim):
    """Tokens with such scores count nothing; rows that see no others get zeros."""
    s = u.Scene(fmt, 2, dim, 16, [70, 300], seed=dim)
    poison(s, "k", 0, 0, 70, "ninf")
    poison(s, "k", 1, 0, 250, "ninf")
    s.k[1][:250] = 0.0
    s.to_device()
    counts, seen = [40, 100], [np.zeros(70, bool), np.arange(300) >= 250]
    q = np.ones((140, 8, dim))
    o, one = (torch.full((r, 8, dim), 7.0, dtype=torch.bfloat16, device=g.DEV) for r in (140, 2))
    attn = q8.make_attn(dim ** -0.5)
    u.rows(s, u.bf16_dev(q), g.dev(np.array([0, 40, 140], np.int32)), attn, o)
    u.decode(s, u.bf16_dev(q[:2]), attn, one)
    u.compare(u.host(o), want_of(s, q, counts, dim ** -0.5, present=seen), 300, dim, "rows")
    u.compare(u.host(one), want_rows(s, q[:2], dim ** -0.5, 0, 0, seen), 300, dim, "decode")
    assert (u.host(o)[:90] == 0).all() and (u.host(one)[0] == 0).all()


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("kind", ["nan", "inf", "ninf", "huge"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_masked_tokens_hold_anything(fmt, kind, dim):
    """Tokens outside the window of every row, in either buffer."""
    s = u.Scene(fmt, 2, dim, 16, [100, 333, 40, 1500], seed=21)
    window, sinks = 30, 5
    counts = [7, 3, 10, 9]
    for i, l in enumerate(s.lens):
        for which in "kv":
            poison(s, which, i, sinks, l - counts[i] + 1 - window, kind)
    s.to_device()
    seen = [np.arange(l) >= 0 for l in s.lens]
    for i, l in enumerate(s.lens):
        seen[i][sinks:l - counts[i] + 1 - window] = False
    check_decode(s, 4, window, sinks, present=seen)
    check_rows(s, 4, counts, window, sinks, present=seen)


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("kind", ["nan", "inf"])
def test_tokens_ahead_hold_anything(fmt, kind):
    """A row is not touched by what the rows after it put into the cache; rows that see a NaN have one."""
    for dim in (64, 128, 256):
        s = u.Scene(fmt, 2, dim, 16, [90, 700], seed=31)
        clean = u.Scene(fmt, 2, dim, 16, [90, 700], seed=31).to_device()
        for which in "kv":
            poison(s, which, 0, 80, 81, kind)
            poison(s, which, 1, 650, 653, kind)
        s.to_device()
        q = queries(s, 360, 4, 5)
        start = g.dev(np.array([0, 60, 360], np.int32))
        outs = []
        for x in (s, clean):
            o = torch.zeros((360, 8, dim), dtype=torch.bfloat16, device=g.DEV)
            u.rows(x, u.bf16_dev(q), start, q8.make_attn(dim ** -0.5), o)
            torch.cuda.synchronize()
            outs.append(u.host(o))
        a, b = outs
        sees = np.concatenate([np.arange(30, 90) >= 80, np.arange(400, 700) >= 650])
        np.testing.assert_array_equal(a[~sees], b[~sees])
        assert (~np.isfinite(a[sees])).any(-1).all()
        # and the token's own row in a single-token call
        o = torch.zeros((2, 8, dim), dtype=torch.bfloat16, device=g.DEV)
        u.decode(s, u.bf16_dev(q[:2]), q8.make_attn(dim ** -0.5), o)
        assert (~np.isfinite(u.host(o))).any(-1).all()


@pytest.mark.parametrize("fmt", [BF16, Q8])
def test_bad_queries_stay_in_their_row(fmt):
    s = u.Scene(fmt, 2, 128, 16, [90, 700, 33], seed=41).to_device()
    q = u.bf16_dev(queries(s, 200, 4, 6))
    start = g.dev(np.array([0, 40, 190, 200], np.int32))
    attn = q8.make_attn(0.1)
    bad = q.clone()
    for r, h, x in ((3, 2, float("nan")), (100, 7, float("inf")), (195, 0, float("-inf"))):
        bad[r, h, 5] = x
    outs = [torch.zeros_like(q) for _ in range(2)]
    for x, o in zip((q, bad), outs):
        u.rows(s, x, start, attn, o)
    a, b = (u.host(o) for o in outs)
    other = np.ones(a.shape[:2], bool)
    for r, h in ((3, 2), (100, 7), (195, 0)):
        other[r, h] = False
    np.testing.assert_array_equal(a[other], b[other])
    outs = [torch.zeros((3, 8, 128), dtype=torch.bfloat16, device=g.DEV) for _ in range(2)]
    bad = q[:3].clone()
    bad[1, 3] = float("nan")
    for x, o in zip((q[:3].contiguous(), bad), outs):
        u.decode(s, x, attn, o)
    a, b = (u.host(o) for o in outs)
    a[1, 3] = b[1, 3] = 0
    np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("page", [16, 64])
def test_bad_pages_are_not_seen(fmt, page):
    for dim in (64, 128, 256):
        s = u.Scene(fmt, 2, dim, page, [300, 17, 1, 129, 2000], seed=51, extra=2)
        seen = [np.ones(l, bool) for l in s.lens]
        for i, j, bad in ((0, 1, -1), (0, 3, s.pages), (1, 0, -2 ** 31), (2, 0, 2 ** 31 - 1), (4, 0, -7),
                          (4, (1999 // page), s.pages + 5)):
            s.table[i, j] = bad
            seen[i][j * page:(j + 1) * page] = False
        s.to_device()
        check_decode(s, 4, present=seen)
        check_decode(s, 4, 40, 3, present=seen)
        counts = [100, 17, 1, 3, 70]
        check_rows(s, 4, counts, present=seen)
        check_rows(s, 4, counts, 40, 3, present=seen)


def test_lengths_out_of_range():
    s = u.Scene(BF16, 2, 64, 16, [64, 64, 64], seed=61).to_device()
    q = u.bf16_dev(queries(s, 3, 4, 7))
    attn = q8.make_attn(0.125)
    want = torch.zeros_like(q)
    u.decode(s, q, attn, want)
    s.lens_d = g.dev(np.array([2 ** 31 - 1, -5, 65], np.int32))
    for call in (lambda o: u.decode(s, q, attn, o),
                 lambda o: u.rows(s, q, g.dev(np.arange(4, dtype=np.int32)), attn, o)):
        o = torch.full_like(q, 7.0)
        call(o)
        assert (u.host(o)[1] == 0).all()
        err = np.abs(u.host(o) - u.host(want))[[0, 2]]
        assert (err <= 4 * u.HALF_BF16 * np.abs(u.host(want)).max()).all()


# ---- chunks of rows ------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 128])
def test_rows(fmt, dim, page):
    lens = [1, 0, 40, 65, 130, 257, 3, 64]
    counts = [1, 0, 40, 1, 66, 100, 0, 64]
    check_rows(u.Scene(fmt, 2, dim, page, lens, seed=dim + page).to_device(), 4, counts)


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (2, 3), (1, 16), (1, 33), (2, 80), (16, 2)])
def test_rows_heads(fmt, heads, group):
    s = u.Scene(fmt, heads, 64, 16, [77, 9, 200], seed=heads * group).to_device()
    check_rows(s, group, [33, 9, 50])
    if heads < 4:
        s = u.Scene(fmt, heads, 128, 16, [150, 9], seed=heads * group).to_device()
        check_rows(s, group, [20, 5])


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("dim,lens,counts", [(128, [3000], [5]), (64, [2500, 30], [20, 3]), (256, [1800], [9]),
                                             (128, [700, 1, 1200, 40], [1, 1, 1, 1]), (128, [900], [300])])
def test_rows_split(fmt, dim, lens, counts):
    s = u.Scene(fmt, 2, dim, 32, lens, seed=dim + len(lens)).to_device()
    check_rows(s, 4, counts)
    check_rows(s, 4, counts, 100, 7)


def test_rows_without_split():
    """Blocks of columns enough that each takes its whole context; the longest refills its list of pages."""
    for lens, counts, group in (([290], [290], 1), ([9000], [3], 2)):
        s = u.Scene(BF16, 128, 64, 64, lens, seed=lens[0]).to_device()
        assert s.workspace(sum(counts) + 3, 128 * group)[1] == 0
        check_rows(s, group, counts)
    s = u.Scene(BF16, 2, 128, 64, [1100], seed=71).to_device()
    check_rows(s, 2, [1100], pad=0)
    s = u.Scene(BF16, 2, 64, 16, [600, 620], seed=72).to_device()
    check_rows(s, 2, [600, 500])


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (16, 0), (33, 70), (100, 4), (64, 0), (10 ** 6, 3),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
def test_rows_window(fmt, window, sinks):
    s = u.Scene(fmt, 2, 128, 16, [1, 100, 333, 64], seed=window % 1000).to_device()
    check_rows(s, 4, [1, 90, 200, 64], window, sinks)
    s = u.Scene(fmt, 2, 64, 32, [500], seed=window % 1000).to_device()
    check_rows(s, 2, [400], window, sinks)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(300, 0), (300, 70), (512, 4), (1000, 0), (1000, 130)])
def test_rows_long_window(dim, window, sinks):
    """Windows that leave whole stages of keys between their edge and a block's first row, behind first
    tokens that are kept: a few rows split along the tokens, and enough blocks that each takes its whole
    window."""
    s = u.Scene(BF16, 2, dim, 16, [1500, 3000], seed=window + sinks).to_device()
    check_rows(s, 4, [130, 70], window, sinks)
    s = u.Scene(BF16, 8, dim, 64, [1700], seed=window).to_device()
    assert s.workspace(523, 64)[1] == 0
    check_rows(s, 8, [520], window, sinks)


@pytest.mark.parametrize("fmt", [BF16, Q8])
def test_rows_one_long_among_many(fmt):
    """A mixed step: single rows of many short sequences, one of a long one, and a chunk of a prompt."""
    r = np.random.default_rng(13)
    lens = r.integers(1, 60, 33).tolist()
    lens[20], lens[30] = 9001, 400
    counts = [1] * 33
    counts[7], counts[30] = 0, 150
    s = u.Scene(fmt, 2, 128, 16, lens, seed=14).to_device()
    check_rows(s, 4, counts)
    check_rows(s, 4, counts, 500, 4)


def test_rows_many_sequences():
    r = np.random.default_rng(3)
    lens = r.integers(0, 30, 500)
    counts = np.minimum(lens, r.integers(0, 4, 500))
    check_rows(u.Scene(BF16, 1, 64, 16, lens.tolist(), seed=3).to_device(), 2, counts)
    lens = np.zeros(8192, int)
    lens[[0, 5000, 8191]] = [40, 33, 9]
    counts = np.zeros(8192, int)
    counts[[0, 5000, 8191]] = [3, 33, 9]
    check_rows(u.Scene(Q8, 1, 128, 16, lens.tolist(), seed=4).to_device(), 4, counts)
    # none of the rows belongs to a sequence
    check_rows(u.Scene(BF16, 1, 64, 16, [5, 0], seed=5).to_device(), 4, [0, 0])


def test_rows_more_than_tokens():
    """Rows before the first token of a sequence see none and get zeros."""
    s = u.Scene(BF16, 2, 128, 16, [3, 0], seed=81).to_device()
    q = u.bf16_dev(queries(s, 9, 4, 8))
    o = torch.full_like(q, 7.0)
    u.rows(s, q, g.dev(np.array([0, 5, 9], np.int32)), q8.make_attn(0.1), o)
    got = u.host(o)
    assert (got[:2] == 0).all() and (got[5:] == 0).all() and (got[2:5] != 0).any((1, 2)).all()


@pytest.mark.parametrize("fmt", [BF16, Q8])
def test_one_row_of_either_call(fmt):
    """The two calls agree on single rows, up to their roundings of the same sum."""
    s = u.Scene(fmt, 4, 128, 16, [1, 50, 64, 700], seed=91).to_device()
    a = check_decode(s, 4)
    q = queries(s, 4, 4, 1)
    o = torch.zeros((4, 16, 128), dtype=torch.bfloat16, device=g.DEV)
    u.rows(s, u.bf16_dev(q), g.dev(np.arange(5, dtype=np.int32)), q8.make_attn(128 ** -0.5), o)
    assert np.abs(u.host(o) - a).max() <= 4 * u.HALF_BF16 * max(np.abs(v).max() for v in s.v)


@pytest.mark.parametrize("fmt", [BF16, Q8])
def test_pages_past_4_gib(fmt):
    """A cache of 5 GiB a buffer: the attentions, the heads' rows and rows read back equal those of a small
    cache of the same pages."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB of device memory")
    hkv, group, dim, page = 4, 4, 128, 256
    s = u.Scene(fmt, hkv, dim, page, [700, 513, 30], seed=7, spare=1).to_device()
    per_page = s.lay.nbytes(1)
    pages = (5 << 30) // per_page
    far = np.linspace(pages - 1, pages // 2, s.pages).astype(np.int64)   # where each page goes
    big = [torch.empty(pages * per_page, dtype=torch.uint8, device=g.DEV) for _ in "kv"]
    for b, small in zip(big, (s.kd, s.vd)):
        for i, p in enumerate(far):
            b[p * per_page:(p + 1) * per_page] = small[i * per_page:(i + 1) * per_page]
    cache = q8.make_kv_cache(*big, pages, fmt, hkv, dim, page)
    table = g.dev(np.where(s.table >= 0, far[s.table], -1).astype(np.int32))
    q = u.bf16_dev(queries(s, 93, group, 5))
    start = g.dev(np.array([0, 40, 63, 93], np.int32))
    x = torch.randn((37, (hkv * group + 2 * hkv) * dim), device=g.DEV)
    ld, free = x.shape[1], int(s.free[0])
    heads = q8.make_heads(None, None, 0.0, None, 0, 0)
    pos = torch.zeros(37, dtype=torch.int32, device=g.DEV)
    outs = []
    for c, t, at in ((s.cache, s.table_d, free), (cache, table, int(far[free]))):
        slots = g.dev(np.array([at * page + 3 + i for i in range(37)], np.int32))
        o, one, qo = torch.zeros_like(q), torch.zeros_like(q[:3]), torch.zeros_like(q[:37])
        back = [torch.zeros((37, hkv, dim), dtype=torch.bfloat16, device=g.DEV) for _ in "kv"]
        ws = s.workspace(93, hkv * group), s.workspace(0, hkv * group)
        q8.q8_attn_rows(q, 93, hkv * group, c, t, s.max_pages, s.lens_d, start, 3, q8.make_attn(0.09), o, None, None,
                        *ws[0])
        q8.q8_attn_decode(q, hkv * group, c, t, s.max_pages, s.lens_d, 3, q8.make_attn(0.09), one, None, None, *ws[1])
        q8.q8_qkv_heads(x, ld, x[:, hkv * group * dim:], ld, x[:, hkv * (group + 1) * dim:], ld, 37, hkv * group, heads,
                        pos, slots, qo, c)
        q8.q8_kv_gather(c, slots, 37, *back)
        torch.cuda.synchronize()
        outs.append((o, one, qo, *back))
    for a, b in zip(*outs):
        assert a.any() and torch.equal(a, b)


# ---- streams, graphs, workspaces ------------------------------------------------------------------

def test_two_streams():
    """Calls at once on two streams, a workspace each, equal the same calls in turn."""
    scenes = [u.Scene(BF16, 2, 128, 16, [3000, 5, 900], seed=101).to_device(),
              u.Scene(Q8, 2, 128, 16, [2000, 77], seed=102).to_device()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    work = []
    for s in scenes:
        q = u.bf16_dev(queries(s, s.n, 4, 9))
        start = g.dev(np.arange(s.n + 1, dtype=np.int32))
        work.append((s, q, start, s.workspace(0, 8), s.workspace(s.n, 8)))
    attn = q8.make_attn(0.1)

    def run(k, st):
        s, q, start, wd, wr = work[k]
        a, b = torch.zeros_like(q), torch.zeros_like(q)
        st and st.wait_stream(torch.cuda.default_stream())
        for _ in range(4):
            u.decode(s, q, attn, a, None, st.cuda_stream if st else None, wd)
            u.rows(s, q, start, attn, b, None, st.cuda_stream if st else None, wr)
        return a, b

    want = [run(k, None) for k in (0, 1)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [run(k, streams[k]) for k in (0, 1)]
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("fmt", [BF16, Q8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_replays_follow_the_lengths(fmt, dim):
    """Both calls captured over one workspace; between the replays the lengths, rows and pages change and
    the workspace serves eager calls; every replay equals the eager calls on the same state."""
    s = u.Scene(fmt, 2, dim, 16, [900, 40, 0, 333], seed=111).to_device()
    q = u.bf16_dev(queries(s, 60, 4, 3))
    start = g.dev(np.array([0, 20, 25, 25, 60], np.int32))
    attn = q8.make_attn(0.1, 200, 4)
    b = max(s.workspace(0, 8)[1], s.workspace(60, 8)[1])
    ws = torch.zeros(b, dtype=torch.uint8, device=g.DEV), b
    bufs = [torch.zeros((r, 8, dim), dtype=torch.bfloat16, device=g.DEV) for r in (4, 60)]

    def run(o, p):
        u.decode(s, q[:4], attn, o, None, ws=ws)
        u.rows(s, q, start, attn, p, None, ws=ws)

    run(*bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*bufs)
    order = np.random.default_rng(5)
    for lens, starts in (([900, 40, 0, 333], [0, 20, 25, 25, 60]), ([899, 39, 0, 1], [0, 0, 39, 39, 40]),
                         ([31, 32, 0, 300], [0, 31, 40, 40, 60]), ([0, 0, 0, 0], [0, 0, 0, 0, 0]),
                         ([900, 1, 0, 333], [0, 1, 2, 2, 3])):
        s.lens_d.copy_(torch.tensor(lens))
        start.copy_(torch.tensor(starts))
        s.table[0, :56] = s.table[0, order.permutation(56)]
        s.table_d.copy_(torch.from_numpy(s.table))
        for o in bufs:
            o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        want = [torch.full_like(o, 7.0) for o in bufs]
        run(*want)
        torch.cuda.synchronize()
        for x, y in zip(bufs, want):
            assert torch.equal(x, y), lens
        assert (u.host(bufs[1])[starts[-1]:] == 7.0).all()
        assert not ws[0][:4 << 20].any()


def test_layer_replayed():
    """A step's calls as a serving loop captures them: tables, the q/k/v product, heads, attention and the
    output product, replayed while the cache grows, each replay against the same calls run eagerly from
    the same state, and the attention of the first steps against the oracle."""
    hq, hkv, dim, page, n, K = 8, 2, 64, 16, 5, 512
    N = (hq + 2 * hkv) * dim
    rng = np.random.default_rng(7)
    x, q, sc = inputs.random_case(n, K, N, seed=1)
    Wq, Ws = g.pack(q, sc)
    _, q2, sc2 = inputs.random_case(1, hq * dim, K, seed=2)
    W2, Ws2 = g.pack(q2, sc2)
    Npad, Kpad = q8.q8_padded_cols(N), q8.q8_padded_cols(K)
    xd = g.dev(x.view(np.int16))
    lay = dec.Layout(BF16, hkv, dim, page)
    pages, most = 40, 8
    lens0 = np.array([0, 15, 16, 33, 100], np.int32)
    held = -(-lens0 // page)
    table0 = np.full((n, most), -1, np.int32)
    order = rng.permutation(pages).astype(np.int32)
    at = 0
    for i in range(n):
        table0[i, :held[i]] = order[at:at + held[i]]
        at += held[i]
    free0 = np.zeros(pages, np.int32)
    free0[:pages - at] = order[at:]
    ws_bytes = max(q8.q8_attn_workspace_bytes(0, n, hq, q8.make_kv_cache(1 << 20, 1 << 20, pages, 0, hkv, dim, page)),
                   q8.q8_plan_workspace_bytes(q8.q8_gemv_default_plan(n, K, N, q8.Q8_ACT_BF16), n, K, N),
                   q8.q8_plan_workspace_bytes(q8.q8_gemv_default_plan(n, hq * dim, K, q8.Q8_ACT_Q8_0), n, hq * dim, K))

    class State:
        def __init__(self):
            i32 = lambda a: g.dev(np.array(a, np.int32))  # noqa: E731
            self.k = torch.full((lay.nbytes(pages),), 255, dtype=torch.uint8, device=g.DEV)
            self.v = self.k.clone()
            kv = np.random.default_rng(8)
            for b in (self.k, self.v):
                h = b.cpu().numpy()
                for i in range(n):
                    t = np.arange(lens0[i])
                    slots = table0[i, t // page] * page + t % page
                    if len(t):
                        dec.write_rows(lay, h, "k" if b is self.k else "v", slots,
                                       kv.standard_normal((len(t), hkv, dim)).astype(np.float32))
                b.copy_(torch.from_numpy(h))
            self.lens, self.table, self.free, self.count = i32(lens0), i32(table0), i32(free0), i32([pages - at])
            self.new, self.start, self.pos, self.slots, self.status = (
                i32([1] * n), i32([0] * (n + 1)), i32([0] * n), i32([0] * n), i32([0, 0]))
            self.y = torch.zeros((n, Npad), device=g.DEV)
            self.qo = torch.zeros((n, hq, dim), dtype=torch.bfloat16, device=g.DEV)
            self.o = torch.zeros_like(self.qo)
            self.oq = g.empty_bytes(q8.q8_act_bytes(n, hq * dim))
            self.out = torch.zeros((n, Kpad), device=g.DEV)
            self.ws = torch.zeros(ws_bytes, dtype=torch.uint8, device=g.DEV)
            self.freqs = torch.zeros(dim // 2, dtype=torch.float64, device=g.DEV)
            q8.q8_rope_freqs(q8.make_rope(10000.0, dim), self.freqs)
            self.norm = torch.ones(dim, device=g.DEV)
            self.cache = q8.make_kv_cache(self.k, self.v, pages, BF16, hkv, dim, page)
            self.heads = q8.make_heads(self.norm, self.norm, 1e-6, self.freqs, dim, q8.Q8_ROPE_HALF)
            self.step = q8.make_kv_step(self.lens, self.new, n, self.table, most, page, self.free, pages, self.count,
                                        self.lens, self.count, self.start, self.pos, self.slots, n, self.status)

        def run(self):
            q8.q8_kv_step(self.step)
            q8.q8_gemv_ws(xd, Wq, Ws, self.y, n, K, N, q8.Q8_ACT_BF16, None, self.ws, ws_bytes)
            q8.q8_qkv_heads(self.y, Npad, self.y[:, hq * dim:], Npad, self.y[:, (hq + hkv) * dim:], Npad, n, hq,
                            self.heads, self.pos, self.slots, self.qo, self.cache)
            q8.q8_attn_decode(self.qo, hq, self.cache, self.table, most, self.lens, n, q8.make_attn(dim ** -0.5),
                              self.o, self.oq, None, self.ws, ws_bytes)
            q8.q8_gemv_ws(self.oq, W2, Ws2, self.out, n, hq * dim, K, q8.Q8_ACT_Q8_0, None, self.ws, ws_bytes)

        def result(self):
            torch.cuda.synchronize()
            return [t.clone() for t in (self.lens, self.table, self.count, self.qo, self.o, self.out, self.k, self.v)]

    warm = State()
    warm.run()
    a, b = State(), State()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    torch.cuda.synchronize()
    for step in range(20):
        b.run()
        want = b.result()
        graph.replay()
        got = a.result()
        for x0, y0 in zip(want, got):
            assert torch.equal(x0.view(torch.uint8), y0.view(torch.uint8)), step
        if step in (0, 1, 17):
            lens = got[0].cpu().numpy()
            np.testing.assert_array_equal(lens, lens0 + step + 1)
            table = got[1].cpu().numpy()
            qh = u.host(got[3])
            res = []
            for i in range(n):
                t = np.arange(lens[i])
                slots = table[i, t // page].astype(np.int64) * page + t % page
                k = dec.read_rows(lay, got[6].cpu().numpy(), "k", slots)
                v = dec.read_rows(lay, got[7].cpu().numpy(), "v", slots)
                res.append(dec.attention(qh[i:i + 1], k, v, [lens[i] - 1], dim ** -0.5))
            u.compare(u.host(got[4]), tuple(np.concatenate([r[j] for r in res]) for j in range(4)), int(lens.max()),
                      dim, step)
    assert not a.ws[:4 << 20].any()


def test_prompt_and_step_of_one_cache():
    """A prompt in chunks and then steps: the rows of a chunk equal those of one whole call."""
    hq, hkv, dim, page, total = 8, 2, 128, 32, 150
    rng = np.random.default_rng(17)
    lay = dec.Layout(Q8, hkv, dim, page)
    pages = 7
    cacheb = [torch.full((lay.nbytes(pages),), 255, dtype=torch.uint8, device=g.DEV) for _ in "kv"]
    cache = q8.make_kv_cache(*cacheb, pages, Q8, hkv, dim, page)
    table = rng.permutation(pages).astype(np.int32)[None, :5].copy()
    x = rng.standard_normal((total, (hq + 2 * hkv) * dim)).astype(np.float32)
    freqs = g.dev(dec.rope_freqs(10000.0, dim))
    heads = q8.make_heads(None, None, 0.0, freqs, dim, 1)
    table_d = g.dev(table)
    attn = q8.make_attn(dim ** -0.5)
    out = np.zeros((total, hq, dim))
    qrows = np.zeros((total, hq, dim))
    done = 0
    for rows in (70, 1, 33, 1, 1, 44):
        pos = np.arange(done, done + rows)
        slots = (table[0, pos // page] * page + pos % page).astype(np.int32)
        xd = g.dev(x[done:done + rows])
        ld = x.shape[1]
        qo = torch.zeros((rows, hq, dim), dtype=torch.bfloat16, device=g.DEV)
        q8.q8_qkv_heads(xd, ld, xd[:, hq * dim:], ld, xd[:, (hq + hkv) * dim:], ld, rows, hq, heads,
                        g.dev(pos.astype(np.int32)), g.dev(slots), qo, cache)
        done += rows
        o = torch.zeros_like(qo)
        lens = g.dev(np.array([done], np.int32))
        b = q8.q8_attn_workspace_bytes(0 if rows == 1 else rows, 1, hq, cache)
        ws = torch.zeros(max(b, 16), dtype=torch.uint8, device=g.DEV)
        if rows == 1:
            q8.q8_attn_decode(qo, hq, cache, table_d, 5, lens, 1, attn, o, None, None, ws, b)
        else:
            q8.q8_attn_rows(qo, rows, hq, cache, table_d, 5, lens, g.dev(np.array([0, rows], np.int32)), 1, attn, o,
                            None, None, ws if b else None, b)
        torch.cuda.synchronize()
        out[done - rows:done], qrows[done - rows:done] = u.host(o), u.host(qo)
    t = np.arange(total)
    slots = table[0, t // page].astype(np.int64) * page + t % page
    k, v = (dec.read_rows(lay, c.cpu().numpy(), w, slots) for c, w in zip(cacheb, "kv"))
    u.compare(out, dec.attention(qrows, k, v, t, dim ** -0.5), total, dim, "chunks")
    # and the whole chain in 64 bits: queries and keys rotated from the fp32 rows, the cache's rounding known
    f = dec.rope_freqs(10000.0, dim)
    q64, _ = dec.heads(x[:, :hq * dim].reshape(total, hq, dim), None, 0.0, f, t, 1, 1.0)
    k64, _ = dec.heads(x[:, hq * dim:(hq + hkv) * dim].reshape(total, hkv, dim), None, 0.0, f, t, 1, 1.0)
    v64 = x[:, (hq + hkv) * dim:].reshape(total, hkv, dim).astype(np.float64)
    exact = dec.attention(q64, k64, v64, t, dim ** -0.5)
    # a score moves by at most its terms' size times the queries' rounding, and by |q| times half a step of
    # the keys' codes; a probability by twice that; a value by half a step of its codes
    half = np.abs(k64).max() / 254
    ds = exact[3] * u.HALF_BF16 + dim ** -0.5 * np.abs(q64).sum(-1) * half
    tol = exact[1] * (np.exp(2 * ds)[..., None] - 1 + u.HALF_BF16) + np.abs(v64).max() / 254 * 1.1 + \
        np.abs(exact[0]) * u.HALF_BF16 * 1.1
    assert (np.abs(out - exact[0]) <= tol).all()
