"""The logits' calls on the host: the arguments they refuse before any device work, and the oracle."""
import math
import os

import numpy as np
import pytest

import block_quantized_weight_02_amd as q8
from block_quantized_weight_02_amd import binding
from oracle import logits as ol

pytestmark = pytest.mark.skipif(not os.path.exists(binding.LIB_PATH), reason="libq8gemv.so not built")

A, S0 = 1 << 20, 0     # an aligned address that is never read; the null stream, never reached


def refuse(status, fn, *args, part=""):
    with pytest.raises(q8.Q8Error) as e:
        fn(*args)
    assert e.value.status == status, e.value
    assert part in e.value.message


def rules(logits=A, ld=128, m=2, v=100, r=None, out=A + 4096, ld_out=128, **fields):
    r = q8.make_logit_rules(**fields) if r is None else r
    q8.q8_logits_rules(logits, ld, m, v, r, out, ld_out, S0)


def sample(logits=A, ld=128, m=2, v=100, token=A, logprob=A, ws=A, ws_bytes=1 << 30, **fields):
    q8.q8_sample(logits, ld, m, v, q8.make_sampling(fields.pop("u", A), **fields), token, logprob, S0, ws, ws_bytes)


@pytest.mark.parametrize("call", [rules, sample])
def test_sizes_are_refused(call):
    for bad, part in ((dict(m=0), "m ="), (dict(m=8193), "m ="), (dict(v=0), "V ="), (dict(v=-1), "V ="),
                      (dict(v=(1 << 20) + 1, ld=1 << 21), "V ="), (dict(ld=99), "ld ="), (dict(ld=102), "ld ="),
                      (dict(ld=1 << 32), "ld =")):
        refuse(1, lambda b=bad: call(**b), part=part)
    refuse(3, lambda: call(logits=None), part="logits")
    refuse(4, lambda: call(logits=A + 4), part="logits")


def test_rules_refuse():
    refuse(1, lambda: rules(ld_out=100 - 4), part="ld_out")
    refuse(1, lambda: rules(out=A, ld_out=256), part="in place")
    refuse(3, lambda: rules(out=None), part="out")
    refuse(3, lambda: q8.q8_logits_rules(A, 128, 2, 100, None, A + 4096, 128, S0), part="rules")
    refuse(3, lambda: rules(tokens=A, ld_tokens=4), part="lens")
    refuse(1, lambda: rules(tokens=A, lens=A), part="ld_tokens")
    for k in ("repetition", "presence", "frequency"):
        refuse(3, lambda k=k: rules(**{k: A}), part="tokens")
        refuse(4, lambda k=k: rules(tokens=A, lens=A, ld_tokens=4, **{k: A + 4}), part=k)
    refuse(4, lambda: rules(tokens=A, lens=A, ld_tokens=4, prompt_lens=A + 8), part="prompt_lens")
    refuse(1, lambda: rules(bias_start=A, bias_entries=-1), part="bias_entries")
    refuse(3, lambda: rules(bias_start=A, bias_entries=3), part="bias_token")
    refuse(3, lambda: rules(bias_start=A, bias_entries=3, bias_token=A), part="bias_value")
    refuse(1, lambda: rules(mask=A, ld_mask=3, mask_rows=2), part="ld_mask")
    refuse(1, lambda: rules(mask=A, ld_mask=4, mask_rows=1), part="mask_rows")
    refuse(1, lambda: rules(mask=A, ld_mask=4, mask_rows=-1, mask_row=A), part="mask_rows")


def test_sample_refuses():
    refuse(3, lambda: sample(u=None), part="u is NULL")
    refuse(3, lambda: sample(token=None), part="token")
    refuse(3, lambda: q8.q8_sample(A, 128, 2, 100, None, A, A, S0), part="sampling")
    for k in ("temperature", "top_k", "top_p", "min_p", "u", "token", "logprob", "ws"):
        refuse(4, lambda k=k: sample(**{k: A + 4}))


def test_sample_workspace():
    need = q8.q8_sample_workspace_bytes(2, 100)
    assert need > 4 << 20 and need % 256 == 0
    assert q8.q8_sample_workspace_bytes(256, 131072) > need
    assert q8.q8_sample_workspace_bytes(0, 100) == 0 and q8.q8_sample_workspace_bytes(1, (1 << 20) + 1) == 0
    refuse(5, lambda: sample(ws=None), part="needed")
    refuse(5, lambda: sample(ws_bytes=need - 1), part="needed")


VOCABULARIES = (1, 1000, 32000, 32768, 32769, 50001, 65536, 65537, 131072, 1 << 20)


def test_a_sample_workspace_serves_smaller_calls():
    """Bytes never fall with the rows or the vocabulary."""
    rows = [*range(1, 400), 511, 512, 513, 1023, 1024, 1025, 4000, 8192]
    last = {m: 0 for m in rows}
    for v in VOCABULARIES:
        need = {m: q8.q8_sample_workspace_bytes(m, v) for m in rows}
        for a, b in zip(rows, rows[1:]):
            assert need[a] <= need[b], (a, b, v)
        for m in rows:
            assert need[m] >= last[m], (m, v)
        last = need


def test_rows_drawn_by_one_launch_ask_for_no_slices():
    """Rows of up to 32768 logits: no more than the counters' 4 MiB and a little; longer ones for the
    slices of fewer than 96 rows where more are drawn by one launch."""
    for m, v in ((1, 100), (8192, 32000), (300, 32768)):
        assert q8.q8_sample_workspace_bytes(m, v) <= (4 << 20) + 4096
    assert q8.q8_sample_workspace_bytes(8192, 50001) == q8.q8_sample_workspace_bytes(95, 50001) > 8 << 20


def test_oracle_of_the_rules():
    x = np.array([1.0, -1.0, 2.0, 3.0, 4.0], np.float32)
    y, _ = ol.rules(x, [0, 1, 3, 3, 9, -1], 2, 2.0, 0.5, 0.25, [(2, 1.0), (2, 5.0), (7, 1.0)], np.array([0b01111]))
    np.testing.assert_array_equal(y, [0.5, -2.0, 7.0, 1.5 - 0.5 - 0.5, -math.inf])


def test_oracle_of_the_draw():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3])).astype(np.float32)
    assert [ol.sample(x, u) for u in (0.05, 0.2, 0.6, 0.9)] == [{0}, {1}, {2}, {3}]
    assert ol.sample(x, 0.99, top_k=2) == {3} and ol.sample(x, 0.5, top_k=2) == {1}
    assert ol.sample(x, 0.99, top_p=0.39) == {1} and ol.sample(x, 0.99, top_p=0.41) == {3}
    assert ol.sample(x, 0.0, min_p=0.6) == {1} and ol.sample(x, 0.99, min_p=0.6) == {3}
    assert ol.sample(x, 0.3, temperature=0.0) == {1}
    assert ol.sample(np.full(4, -np.inf, np.float32), 0.5) == {-1}
    assert ol.sample(np.zeros(4, np.float32), 0.25) == {0, 1}          # on the boundary itself
    assert ol.logprob(x, 1) == pytest.approx(math.log(0.4), abs=1e-6)
