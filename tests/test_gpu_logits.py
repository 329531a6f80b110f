"""The rules on logits and the drawn token against the 64-bit oracle, through the C ABI."""
import math

import numpy as np
import pytest
import torch

import block_quantized_weight_02_amd as q8
from oracle import logits as ol

pytestmark = pytest.mark.gpu

from tests import gpu_util as g  # noqa: E402
from tests import w4_util as w4u  # noqa: E402

INF = math.inf


def ld_of(v):
    return -(-v // 64) * 64


# ---- rules ---------------------------------------------------------------------------

class Rules:
    """The rules of m rows: per row a history, its prompt's length, penalties, biases, a mask's row."""

    def __init__(self, m, v, seed, held=0, biases=0, masks=0, width=None, spread=None):
        r = np.random.default_rng([seed, m, v])
        self.m, self.v, self.r = m, v, r
        self.tokens = [list(r.integers(0, spread or v, r.integers(0, held + 1))) for _ in range(m)] if held else [[]] * m
        self.prompt = [int(r.integers(0, len(t) + 1)) for t in self.tokens]
        self.rep = (1 + r.random(m) * r.integers(0, 2, m)).astype(np.float32)
        self.pres = r.standard_normal(m).astype(np.float32)
        self.freq = r.standard_normal(m).astype(np.float32)
        self.bias = [[(int(t), np.float32(b)) for t, b in zip(r.integers(0, v, n), r.standard_normal(n))]
                     for n in r.integers(0, biases + 1, m)] if biases else [[]] * m
        words = (v + 31) // 32 + 1
        self.masks = r.integers(0, 1 << 32, (max(masks, 1), words), dtype=np.uint32)
        self.mask_row = r.integers(-1, masks + 1, m) if masks else np.full(m, -1)
        self.held, self.biases, self.n_masks, self.words = held, biases, masks, words
        self.width = width or max(1, max(len(t) for t in self.tokens) + 3)

    def device(self, **change):
        m = self.m
        tok = np.full((m, self.width), -7, np.int32)
        for i, t in enumerate(self.tokens):
            tok[i, :len(t)] = t
        start = np.concatenate([[0], np.cumsum([len(b) for b in self.bias])]).astype(np.int32)
        flat = [e for b in self.bias for e in b]
        i32 = lambda a: g.dev(np.asarray(a, np.int32))  # noqa: E731
        f = {}
        if self.held:
            f |= dict(tokens=i32(tok), ld_tokens=self.width, lens=i32([len(t) for t in self.tokens]),
                      prompt_lens=i32(self.prompt), repetition=g.dev(self.rep), presence=g.dev(self.pres),
                      frequency=g.dev(self.freq))
        if self.biases:
            f |= dict(bias_start=i32(start), bias_token=i32([t for t, _ in flat] or [0]),
                      bias_value=g.dev(np.array([b for _, b in flat] or [0], np.float32)), bias_entries=len(flat))
        if self.n_masks:
            f |= dict(mask=g.dev(self.masks.view(np.int32)), ld_mask=self.words, mask_row=i32(self.mask_row),
                      mask_rows=self.n_masks)
        self.keep = f | change
        return q8.make_logit_rules(**self.keep)

    def want(self, x, i):
        mr = int(self.mask_row[i])
        return ol.rules(x, self.tokens[i], self.prompt[i], self.rep[i] if self.held else 1.0, self.pres[i],
                        self.freq[i], self.bias[i], self.masks[mr] if 0 <= mr < self.n_masks else None)


def check_rules(s, x, rules, in_place=False, pad=0):
    m, v = s.m, s.v
    ld = ld_of(v)
    rows = np.full((m, ld), np.nan, np.float32)
    rows[:, :v] = x
    src = g.dev(rows)
    out = src if in_place else torch.full((m, ld + pad), -5.0, device=g.DEV)
    q8.q8_logits_rules(src, ld, m, v, rules, out, out.shape[1])
    got = out.cpu().numpy()
    rest = got[:, v:]
    assert np.isnan(rest).all() if in_place else (rest == -5.0).all(), "columns past V"
    if not in_place:
        np.testing.assert_array_equal(src.cpu().numpy(), rows)
    for i in range(m):
        want, off = s.want(x[i], i)
        np.testing.assert_array_equal(np.isnan(got[i, :v]), np.isnan(want))
        fine = np.isfinite(want)
        np.testing.assert_array_equal(got[i, :v][~fine], want[~fine].astype(np.float32))
        assert (np.abs(got[i, :v][fine] - want[fine]) <= off[fine]).all(), i


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("held,biases,masks", [(0, 0, 2), (40, 0, 0), (0, 9, 0), (30, 12, 3), (0, 0, 0)])
@pytest.mark.parametrize("m,v", [(1, 1), (2, 3), (3, 31), (4, 33), (5, 1000), (2, 4097), (3, 9001)])
def test_rules(m, v, held, biases, masks, in_place):
    s = Rules(m, v, 3, held, biases, masks)
    x = (s.r.standard_normal((m, v)) * 4).astype(np.float32)
    check_rules(s, x, s.device(), in_place, pad=4)


@pytest.mark.parametrize("in_place", [False, True])
def test_rules_over_infinities_and_nan(in_place):
    s = Rules(4, 777, 5, 500, 20, 2)
    x = (s.r.standard_normal((4, 777)) * 4).astype(np.float32)
    x[0, ::5], x[1, ::7], x[2, ::3] = np.nan, INF, -INF
    x[3] = np.finfo(np.float32).min
    s.freq[:] = np.abs(s.freq)                  # (the type's lowest value less a penalty stays finite)
    s.pres[:] = 0
    check_rules(s, x, s.device(), in_place)


def test_rules_of_a_long_history():
    """More tokens than threads, most of them few words; every slice of the vocabulary."""
    s = Rules(3, 20000, 7, 30000, 300, 1, spread=12000)
    x = s.r.standard_normal((3, 20000)).astype(np.float32)
    check_rules(s, x, s.device())


def test_rules_of_the_longest_history():
    """2^31 - 1 tokens, of which the first and the last few count."""
    n, v = 2 ** 31 - 1, 8
    tokens = torch.full((1, n), -1, dtype=torch.int32, device=g.DEV)
    tokens[0, 0], tokens[0, n - 3:] = 2, torch.tensor([5, 5, 7], dtype=torch.int32, device=g.DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=g.DEV)
    freq = torch.ones(1, device=g.DEV)
    x = torch.zeros((1, 64), device=g.DEV)
    q8.q8_logits_rules(x, 64, 1, v, q8.make_logit_rules(tokens=tokens, ld_tokens=n, lens=lens, frequency=freq), x, 64)
    assert x[0, :v].tolist() == [0, 0, -1, 0, 0, -2, 0, -1]


def test_rules_bounds():
    """Lengths outside the row, tokens outside the vocabulary, biases past the entries, prompt lengths
    past the history, and a width of no multiple of four."""
    m, v = 4, 130
    s = Rules(m, v, 9, 13, 6, 2, width=13)
    s.tokens = [list(s.r.integers(-50, v + 50, 13)) for _ in range(m)]
    s.prompt = [-5, 99, 0, 4]
    x = s.r.standard_normal((m, v)).astype(np.float32)
    dev = s.device(lens=g.dev(np.array([13, 1 << 30, 13, -4], np.int32)))
    s.tokens[3] = []
    check_rules(s, x, dev)
    entries = sum(len(b) for b in s.bias)
    start = np.array([0, entries + 1000, 0, 5, 2], np.int32)     # too far, falling, again falling
    flat = [e for b in s.bias for e in b]
    s.bias = [flat, [], flat[0:5], []]
    check_rules(s, x, s.device(lens=g.dev(np.array([13, 13, 13, 0], np.int32)), bias_start=g.dev(start),
                               bias_token=g.dev(np.array([t for t, _ in flat], np.int32)),
                               bias_value=g.dev(np.array([b for _, b in flat], np.float32)), bias_entries=entries))


@pytest.mark.parametrize("held", [0, 13])
def test_rules_of_biases_that_end_below_zero(held):
    """A start below 0 is 0: a row that ends there has no biases, with a history and without one, and
    the next row's begin at 0."""
    m, v = 5, 130
    s = Rules(m, v, 13, held, 6, 2)
    flat = [(int(t), np.float32(b)) for t, b in zip(s.r.integers(0, v, 9), s.r.standard_normal(9))]
    start = np.array([-3, -1, 4, -2 ** 31, -7, 9], np.int32)
    s.bias = [[], flat[0:4], [], [], flat]
    x = s.r.standard_normal((m, v)).astype(np.float32)
    check_rules(s, x, s.device(bias_start=g.dev(start),
                               bias_token=g.dev(np.array([t for t, _ in flat], np.int32)),
                               bias_value=g.dev(np.array([b for _, b in flat], np.float32)), bias_entries=9))


def test_rules_without_optional_arrays():
    """Every token made, no penalties but one; masks by row."""
    s = Rules(3, 200, 11, 20, 0, 3)
    s.prompt, s.mask_row = [0] * 3, np.arange(3)
    s.rep[:], s.freq[:] = 1.0, 0.0
    dev = s.device(prompt_lens=None, repetition=None, frequency=None, mask_row=None)
    check_rules(s, s.r.standard_normal((3, 200)).astype(np.float32), dev)


# ---- the draw ------------------------------------------------------------------------

def draw(x, u, temperature=None, top_k=None, top_p=None, min_p=None, logprob=True, stream=None):
    m, v = x.shape
    ld = ld_of(v)
    rows = np.full((m, ld), 1e30, np.float32)      # past V nothing counts
    rows[:, :v] = x
    f = lambda a: None if a is None else g.dev(np.array(np.broadcast_to(np.asarray(a, np.float32), m)))  # noqa: E731
    keep = [g.dev(rows), g.dev(np.array(np.broadcast_to(np.asarray(u, np.float64), m))), f(temperature),
            None if top_k is None else g.dev(np.array(np.broadcast_to(np.asarray(top_k, np.int32), m))), f(top_p), f(min_p)]
    token = torch.full((m,), -9, dtype=torch.int32, device=g.DEV)
    lp = torch.full((m,), float("nan"), device=g.DEV) if logprob else None
    need = q8.q8_sample_workspace_bytes(m, v)
    ws = torch.zeros(need, dtype=torch.uint8, device=g.DEV) if need else None
    q8.q8_sample(keep[0], ld, m, v, q8.make_sampling(keep[1], *keep[2:]), token, lp, stream, ws, need)
    torch.cuda.synchronize()
    return token.cpu().numpy(), lp.cpu().numpy() if logprob else None


def check_draw(x, u, **limits):
    m = x.shape[0]
    token, lp = draw(x, u, **limits)
    at = lambda a, i: np.broadcast_to(a, m)[i]  # noqa: E731
    for i in range(m):
        one = {k: at(a, i) for k, a in limits.items()}
        want = ol.sample(x[i], float(at(u, i)), **{k: (int(a) if k == "top_k" else float(a)) for k, a in one.items()})
        assert int(token[i]) in want, (i, one, float(at(u, i)), int(token[i]), want)
        p = ol.logprob(x[i], token[i])
        # fp32 sums of up to V / 1024 + 6 terms of at most two steps each, the exponents rounded
        tol = (x.shape[1] / 1024 + 16) * 2.0 ** -22 + 2.0 ** -23 * abs(p)
        assert lp[i] == p or abs(lp[i] - p) <= tol, (i, lp[i], p)
    again, lp2 = draw(x, u, **limits)
    np.testing.assert_array_equal(token, again)
    np.testing.assert_array_equal(lp, lp2)
    return token


LIMITS = [{}, dict(temperature=0.0), dict(temperature=0.3), dict(top_k=1), dict(top_k=7), dict(top_p=0.9),
          dict(top_p=0.0), dict(min_p=0.1), dict(temperature=1.7, top_k=40, top_p=0.8, min_p=0.01),
          dict(temperature=0.7, top_p=0.5), dict(top_k=200, top_p=0.999), dict(min_p=2.0)]
SIZES = [1, 2, 5, 64, 1000, 1024, 1025, 5000]


@pytest.mark.parametrize("limits", LIMITS)
@pytest.mark.parametrize("v", SIZES)
def test_draw(v, limits):
    r = np.random.default_rng([13, v])
    x = (r.standard_normal((12, v)) * 3).astype(np.float32)
    check_draw(x, r.random(12), **limits)


@pytest.mark.parametrize("kind", ["equal", "two", "narrow", "steps", "wide", "outlier", "ties", "zeros"])
@pytest.mark.parametrize("limits", LIMITS[4:6] + LIMITS[8:11] + [dict(top_k=3000), dict(top_k=2500, top_p=0.7)])
def test_draw_of_crowded_rows(kind, limits):
    """Rows whose cut falls among many equal or nearly equal logits, or far from the largest."""
    v = 6001
    r = np.random.default_rng([17, v])
    n = r.standard_normal((4, v))
    x = {"equal": np.full((4, v), 1.5), "two": np.where(n > 1.0, 2.0, 1.0), "narrow": 7 + n * 1e-6,
         "steps": np.round(n * 2), "wide": n * 1000, "outlier": np.where(np.arange(v) == 77, 1e30, n),
         "ties": np.round(n * 40) / 40, "zeros": np.where(n > 0, 0.0, -0.0) - (n > 1.5)}[kind]
    check_draw(x.astype(np.float32), r.random(4), **limits)


@pytest.mark.parametrize("limits", [LIMITS[i] for i in (0, 1, 4, 5, 8)])
def test_draw_over_masked_rows(limits):
    """-infinity, NaN and infinity among the logits; a row of nothing, of one token, of lowest values."""
    v = 3001
    r = np.random.default_rng(19)
    x = (r.standard_normal((9, v)) * 3).astype(np.float32)
    x[0] = -INF
    x[1] = np.nan
    x[2] = -INF
    x[2, 2048] = -3e38
    x[3, r.random(v) < 0.99] = -INF
    x[4, r.random(v) < 0.5] = np.nan
    x[5, 17] = x[5, 2999] = INF
    x[6] = np.finfo(np.float32).min
    x[7] = INF
    x[8, :] = -INF
    x[8, -1] = 4.0
    token = check_draw(x, r.random(9), **limits)
    assert token[0] == token[1] == -1 and token[2] == 2048 and token[8] == v - 1
    assert token[5] in (17, 2999)


# rows of two tiles a wave in one workgroup, rows in slices, and four tiles a wave (from 96 rows)
LONG = [(6, 20001), (6, 40001), (97, 33333), (3, 131073)]


@pytest.mark.parametrize("limits", LIMITS)
@pytest.mark.parametrize("m,v", LONG)
def test_draw_of_long_rows(m, v, limits):
    r = np.random.default_rng([41, v])
    x = (r.standard_normal((m, v)) * r.choice([0.3, 1, 3, 10], (m, 1))).astype(np.float32)
    check_draw(x, r.random(m), **limits)


@pytest.mark.parametrize("kind", ["equal", "two", "narrow", "steps", "wide", "outlier", "ties"])
@pytest.mark.parametrize("limits", LIMITS[4:6] + LIMITS[8:11] + [dict(top_k=3000), dict(top_k=15000, top_p=0.7)])
@pytest.mark.parametrize("m,v", LONG[:3])
def test_draw_of_crowded_long_rows(m, v, kind, limits):
    """More tokens in the step of the cut than are ordered at once, counted (top_k) or not (top_p)."""
    r = np.random.default_rng([43, v])
    m = min(m, 4) if m < 96 else m
    n = r.standard_normal((4, v))
    x = {"equal": np.full((4, v), 1.5), "two": np.where(n > 1.0, 2.0, 1.0), "narrow": 7 + n * 1e-6,
         "steps": np.round(n * 2), "wide": n * 1000, "outlier": np.where(np.arange(v) == 77, 1e30, n),
         "ties": np.round(n * 40) / 40}[kind].astype(np.float32)
    # (of 97 rows the oracle looks at these four, and the last)
    rows, u = x[np.arange(m) % 4], r.random(m)
    token, lp = draw(rows, u, **limits)
    for i in (0, 1, 2, 3, m - 1):
        one = {k: (int(a) if k == "top_k" else float(a)) for k, a in limits.items()}
        assert int(token[i]) in ol.sample(rows[i], float(u[i]), **one), (i, limits, float(u[i]), int(token[i]))
    again, lp2 = draw(rows, u, **limits)
    np.testing.assert_array_equal(token, again)
    np.testing.assert_array_equal(lp, lp2)


@pytest.mark.parametrize("limits", [LIMITS[i] for i in (0, 1, 4, 5, 8)])
@pytest.mark.parametrize("m,v", LONG[:3])
def test_draw_over_masked_long_rows(m, v, limits):
    r = np.random.default_rng([47, v])
    m = max(m, 9)
    x = (r.standard_normal((m, v)) * 3).astype(np.float32)
    x[0] = -INF
    x[1] = np.nan
    x[2] = -INF
    x[2, 2048] = -3e38
    x[3, r.random(v) < 0.999] = -INF
    x[4, r.random(v) < 0.5] = np.nan
    x[5, 17] = x[5, v - 2] = INF
    x[6] = np.finfo(np.float32).min
    x[7] = INF
    x[8, :] = -INF
    x[8, -1] = 4.0
    token = check_draw(x, r.random(m), **limits)
    assert token[0] == token[1] == -1 and token[2] == 2048 and token[8] == v - 1
    assert token[5] in (17, v - 2)


@pytest.mark.parametrize("temperature", [0.05, 0.2])
@pytest.mark.parametrize("top_k", [1, 50, 200, 1500])
@pytest.mark.parametrize("m,v", LONG)
def test_top_k_at_low_temperatures(m, v, top_k, temperature):
    r = np.random.default_rng([67, v])
    x = (r.standard_normal((m, v)) * 2.5).astype(np.float32)
    x[:, ::500] += (r.random((m, -(-v // 500))) * 12).astype(np.float32)
    check_draw(x, r.random(m), temperature=temperature, top_k=top_k)


def test_top_k_takes_no_longer_at_a_low_temperature():
    """The order that top_k cuts does not depend on the temperature, nor does the time by much (a row whose
    cut lies behind all the steps is read again by one workgroup, three times as long in all)."""
    v, n = 131072, 20
    r = np.random.default_rng(71)
    x = r.standard_normal((1, v)) * 2.5
    x += (r.random((1, v)) < 0.001) * r.random((1, v)) * 12
    x = g.dev(x.astype(np.float32))
    u, k = torch.full((1,), 0.5, dtype=torch.float64, device=g.DEV), torch.full((1,), 50, dtype=torch.int32, device=g.DEV)
    need = q8.q8_sample_workspace_bytes(1, v)
    ws = torch.zeros(need, dtype=torch.uint8, device=g.DEV)
    token = torch.zeros(1, dtype=torch.int32, device=g.DEV)
    heat = [torch.full((1,), t, device=g.DEV) for t in (0.05, 1.0)]
    times = [[], []]
    for _ in range(10):
        for i, t in enumerate(heat):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            sampling = q8.make_sampling(u, temperature=t, top_k=k)
            begin.record()
            for _ in range(n):
                q8.q8_sample(x, v, 1, v, sampling, token, None, None, ws, need)
            end.record()
            torch.cuda.synchronize()
            times[i].append(begin.elapsed_time(end))
    assert min(times[0]) < 1.7 * min(times[1]), times


@pytest.mark.parametrize("v", [20001, 40001])
def test_a_row_is_drawn_alike_alone_and_in_a_batch(v):
    r = np.random.default_rng([53, v])
    x = (r.standard_normal((100, v)) * 3).astype(np.float32)
    u = r.random(100)
    for limits in ({}, dict(top_p=0.9), dict(top_k=40, top_p=0.95, min_p=0.01)):
        token, _ = draw(x, u, **limits)
        for i in (0, 57, 99):
            assert draw(x[i:i + 1], u[i:i + 1], **limits)[0][0] == token[i]


@pytest.mark.parametrize("m,v", [(3, 1000), (2, 32769), (95, 40001), (96, 40001), (40, 65536), (5, 65537),
                                 (170, 70001)])
def test_draw_within_its_workspace(m, v):
    """Draws over a workspace of exactly the bytes asked for, and of those of more rows: nothing behind
    them is written, nor the counters in front, and the tokens are the same."""
    r = np.random.default_rng([61, v])
    x = (r.standard_normal((m, v)) * 3).astype(np.float32)
    u = r.random(m)
    limits = dict(top_k=r.choice([0, 50], m).astype(np.int32), top_p=r.choice([1.0, 0.9], m))
    want, want_lp = draw(x, u, **limits)
    rows = torch.zeros((m, ld_of(v)), device=g.DEV)
    rows[:, :v] = g.dev(x)
    keep = [g.dev(u), g.dev(limits["top_k"]), g.dev(limits["top_p"].astype(np.float32))]
    for need in (q8.q8_sample_workspace_bytes(m, v), q8.q8_sample_workspace_bytes(m + 1, v + 5)):
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=g.DEV)
        token = torch.zeros(m, dtype=torch.int32, device=g.DEV)
        lp = torch.zeros(m, device=g.DEV)
        q8.q8_sample(rows, ld_of(v), m, v, q8.make_sampling(keep[0], top_k=keep[1], top_p=keep[2]), token, lp,
                     None, ws, need)
        torch.cuda.synchronize()
        assert (ws[:4 << 20] == 0xA5).all() and (ws[need:] == 0xA5).all()
        np.testing.assert_array_equal(token.cpu().numpy(), want)
        np.testing.assert_array_equal(lp.cpu().numpy(), want_lp)


def test_draw_at_the_ends_of_u():
    x = np.zeros((6, 40), np.float32)
    x[:, :8] = -INF
    u = np.array([0.0, 1.0 - 2.0 ** -53, 1.0, -1.0, np.nan, 7.0])
    token, _ = draw(x, u)
    np.testing.assert_array_equal(token, [8, 39, 39, 8, 8, 39])


@pytest.mark.parametrize("temperature", [1e-45, 1e-3, 1e3, 3e38, INF, np.nan, -1.0, -INF])
def test_draw_at_extreme_temperatures(temperature):
    r = np.random.default_rng(23)
    x = (r.standard_normal((8, 2000)) * 5).astype(np.float32)
    x[0, 5] = x[0, 900] = 50.0
    check_draw(x, r.random(8), temperature=temperature)
    check_draw(x, r.random(8), temperature=temperature, top_k=50, top_p=0.9)


def test_draw_of_a_batch():
    """Every kind of row in one call, more rows than CUs, a large vocabulary."""
    m, v = 300, 20011
    r = np.random.default_rng(29)
    x = (r.standard_normal((m, v)) * r.choice([0.3, 1, 3, 10], (m, 1))).astype(np.float32)
    x[::4] += (r.random((75, v)) < 0.001) * r.random((75, v)) * 12
    check_draw(x, r.random(m), temperature=r.choice([0.0, 0.5, 1.0, 2.0], m), top_k=r.choice([0, 1, 50, 1500], m),
               top_p=r.choice([1.0, 0.95, 0.3], m), min_p=r.choice([0.0, 0.05], m))


def test_draw_of_the_largest_vocabulary():
    v = q8.Q8_MAX_VOCAB
    r = np.random.default_rng(31)
    x = (r.standard_normal((4, v)) * 2).astype(np.float32)
    check_draw(x, r.random(4), top_p=[1.0, 0.9, 1.0, 0.99], top_k=[0, 0, 100, 0], temperature=[1, 1, 1, 0])


def test_draws_follow_the_weights():
    """Over a grid of u each token's share is its weight, to the grid's step."""
    x = np.log(np.array([0.5, 0.125, 0.25, 0.0625, 0.0625], np.float32))
    n = 1600
    token, _ = draw(np.tile(x, (n, 1)), (np.arange(n) + 0.5) / n)
    np.testing.assert_array_equal(np.bincount(token, minlength=5), [800, 200, 400, 100, 100])
    token, _ = draw(np.tile(x, (n, 1)), (np.arange(n) + 0.5) / n, top_k=3)
    np.testing.assert_allclose(np.bincount(token, minlength=5) / n, [4 / 7, 1 / 7, 2 / 7, 0, 0], atol=1.01 / n)


@pytest.mark.parametrize("d", [4, 8, 14, 20])
@pytest.mark.parametrize("v", [1000, 20001, 40001])
def test_log_probabilities_near_zero(v, d):
    """One token d above all others: -log(1 + (V - 1) exp(-d)), relative to itself.  A term's exponent is
    rounded thrice (difference, product, constant), each d 2^-24 of it, the exponential by at most two
    steps of 2^-24, the result once more."""
    x = np.full((3, v), -float(d), np.float32)
    x[np.arange(3), [0, v // 2, v - 1]] = 0.0
    token, lp = draw(x, 0.5, temperature=0.0)
    np.testing.assert_array_equal(token, [0, v // 2, v - 1])
    want = -math.log1p((v - 1) * math.exp(-d))
    assert (np.abs(lp - want) <= (3 * d + 4) * 2.0 ** -24 * -want).all(), (lp, want)


def logprob_bound(x, p):
    """The most that a log-probability may be off.  A term exp(-d) below its slice's largest has an exponent
    rounded thrice in fp32 (difference, product, constant), each d 2^-24 of it at most, and an exponential
    within two steps of 2^-24; the largest terms are 1, and sums and logarithm are fp64 (a hundredth of a
    step over all).  The result is rounded once."""
    x = x.astype(np.float64)
    d = x.max() - x
    w = np.exp(-d)
    return 2.0 ** -24 * (1.01 * float((w * np.where(d > 0, 3 * np.minimum(d, 800) + 2, 0)).sum() / w.sum()) + 1.01 * abs(p))


@pytest.mark.parametrize("limits", [{}, dict(temperature=0.0), dict(temperature=1.3, top_k=300, top_p=0.9)])
@pytest.mark.parametrize("kind", ["spread", "two", "steps", "narrow", "far", "outlier"])
@pytest.mark.parametrize("m,v", [(4, 1000), *LONG])
def test_log_probabilities(m, v, kind, limits):
    """Rows of one launch and of slices, whose maxima differ ("far": all of them 15 and more below one
    token); drawn tokens and the largest."""
    r = np.random.default_rng([73, v])
    n = r.standard_normal((4, v))
    far = -20 + 0.5 * n - 5 * np.sin(np.arange(v) // 4096)
    far[np.arange(4), r.integers(0, v, 4)] = 0.0
    x = {"spread": n * np.array([[0.3], [1], [3], [10]]), "two": np.where(n > 1.0, 2.0, 1.0), "steps": np.round(n * 2),
         "narrow": 7 + n * 1e-6, "far": far, "outlier": np.where(np.arange(v) == 77, 1e30, n)}[kind].astype(np.float32)
    rows = x[np.arange(m) % 4]
    token, lp = draw(rows, r.random(m), **limits)
    for i in {0, 1, 2, 3, m - 1} & set(range(m)):
        p = ol.logprob(rows[i], token[i])
        assert abs(lp[i] - p) <= logprob_bound(rows[i], p), (i, lp[i], p)
        if kind == "far":
            assert token[i] == rows[i].argmax() and -1e-2 < lp[i] < 0


def test_draw_without_logprob():
    r = np.random.default_rng(37)
    x = r.standard_normal((3, 500)).astype(np.float32)
    u = r.random(3)
    for limits in ({}, dict(temperature=0.0), dict(top_k=5)):
        np.testing.assert_array_equal(draw(x, u, logprob=False, **limits)[0], draw(x, u, **limits)[0])


@pytest.mark.parametrize("m,v", [(5, 20001), (5, 40001), (97, 33333)])
def test_draws_captured_and_on_two_streams(m, v):
    """Replays over new logits and numbers, and two calls at once, each with a workspace of its own."""
    r = np.random.default_rng([59, v])
    ld = ld_of(v)
    x = [torch.zeros((m, ld), device=g.DEV) for _ in range(2)]
    u = [torch.zeros(m, dtype=torch.float64, device=g.DEV) for _ in range(2)]
    top_p, top_k = torch.full((m,), 0.9, device=g.DEV), torch.full((m,), 40, dtype=torch.int32, device=g.DEV)
    top_k[::2] = 0
    need = q8.q8_sample_workspace_bytes(m, v)
    ws = [torch.empty(need, dtype=torch.uint8, device=g.DEV).fill_(0xA5) for _ in range(2)]
    out = [(torch.zeros(m, dtype=torch.int32, device=g.DEV), torch.zeros(m, device=g.DEV)) for _ in range(2)]
    sampling = [q8.make_sampling(n, top_p=top_p, top_k=top_k) for n in u]
    side = [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side[0]):
        q8.q8_sample(x[0], ld, m, v, sampling[0], *out[0], None, ws[0], need)
    for _ in range(4):
        rows = [(r.standard_normal((m, v)) * 3).astype(np.float32) for _ in range(2)]
        nums = [r.random(m) for _ in range(2)]
        for k in range(2):
            x[k][:, :v].copy_(torch.from_numpy(rows[k]))
            u[k].copy_(torch.from_numpy(nums[k]))
        want = [draw(rows[k], nums[k], top_p=0.9, top_k=top_k.cpu().numpy()) for k in range(2)]
        with torch.cuda.stream(side[0]):
            graph.replay()
        with torch.cuda.stream(side[1]):
            q8.q8_sample(x[1], ld, m, v, sampling[1], *out[1], None, ws[1], need)
        torch.cuda.synchronize()
        for k in range(2):
            np.testing.assert_array_equal(out[k][0].cpu().numpy(), want[k][0])
            np.testing.assert_array_equal(out[k][1].cpu().numpy(), want[k][1])


# ---- together ------------------------------------------------------------------------

def test_a_step_from_activation_to_token_captured():
    """The last product over a 4-bit weight, the rules on its rows in place, the draw, captured once and
    replayed over changing activations, histories and random numbers: each replay is the eager step."""
    m, K, v = 3, 512, 1000
    ld = q8.q8_padded_cols(v)
    w = w4u.Weight(K, v, 64, True, 0, 41).pack()
    r = np.random.default_rng(43)
    x = torch.empty((m, K), dtype=torch.int16, device=g.DEV)
    tokens = torch.zeros((m, 16), dtype=torch.int32, device=g.DEV)
    lens = torch.zeros(m, dtype=torch.int32, device=g.DEV)
    ones = torch.ones(m, device=g.DEV)
    rep, pres = ones * 1.3, ones * 0.5
    mask = g.dev(r.integers(0, 1 << 32, (m, -(-v // 32)), dtype=np.uint32).view(np.int32))
    rules = q8.make_logit_rules(tokens=tokens, ld_tokens=16, lens=lens, repetition=rep, presence=pres, mask=mask,
                                ld_mask=mask.shape[1], mask_rows=m)
    u = torch.zeros(m, dtype=torch.float64, device=g.DEV)
    top_p = ones * 0.9
    sampling = q8.make_sampling(u, top_p=top_p)
    need = max(16, q8.q8_w4_gemv_workspace_bytes(m, w.w, w4u.BF16), q8.q8_sample_workspace_bytes(m, v))
    ws = torch.zeros(need, dtype=torch.uint8, device=g.DEV)

    def step(y, token, logprob):
        q8.q8_w4_gemv(x, w.w, y, m, w4u.BF16, None, None, ws, need)
        q8.q8_logits_rules(y, ld, m, v, rules, y, ld)
        q8.q8_sample(y, ld, m, v, sampling, token, logprob, None, ws, need)

    out = [torch.zeros((m, ld), device=g.DEV), torch.zeros(m, dtype=torch.int32, device=g.DEV),
           torch.zeros(m, device=g.DEV)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(*out)
    for k in range(6):
        a = w4u.Act(m, K, w4u.BF16, 47 + k)
        x.copy_(a.dev)
        u.copy_(torch.from_numpy(r.random(m)))
        graph.replay()
        torch.cuda.synchronize()
        eager = [torch.zeros_like(t) for t in out]
        step(*eager)
        for got, want in zip(out, eager):
            assert torch.equal(got, want)
        # and the step is the operators' definitions, one after the other
        y = out[0].cpu().numpy()[:, :v]
        for i in range(m):
            assert int(out[1][i]) in ol.sample(y[i], float(u[i]), top_p=0.9)
            held = tokens[i, :int(lens[i])].cpu().numpy()
            want, off = ol.rules(a.times(w)[0][i].astype(np.float32), held, 0, 1.3, 0.5, 0.0, (),
                                 mask[i].cpu().numpy().view(np.uint32))
            slack = 1.3 * (a.times(w)[1][i] + 2.0 ** -23 * np.abs(a.times(w)[0][i]))
            fine = np.isfinite(want)
            np.testing.assert_array_equal(np.isfinite(y[i]), fine)
            assert (np.abs(y[i][fine] - want[fine]) <= (off + slack)[fine]).all()
        tokens.scatter_(1, lens.long()[:, None], out[1][:, None])      # the drawn token joins the history
        lens += 1
