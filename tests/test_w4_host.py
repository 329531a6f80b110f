"""The 4-bit weight's calls on the host: sizes, and the arguments they refuse before any device work."""
import os

import numpy as np
import pytest

import block_quantized_weight_02_amd as q8
from block_quantized_weight_02_amd import binding
from oracle import w4

pytestmark = pytest.mark.skipif(not os.path.exists(binding.LIB_PATH), reason="libq8gemv.so not built")

A, S0 = 1 << 20, 0     # an aligned address that is never read; the null stream, never reached


def refuse(status, fn, *args, part=""):
    with pytest.raises(q8.Q8Error) as e:
        fn(*args)
    assert e.value.status == status, e.value
    assert part in e.value.message
    return e.value.message


def weight(K=64, N=8, group=32, fmt=0, zeros=False, values=A, scales=A):
    return q8.make_w4_weight(values, scales, K, N, group, fmt, zeros)


def test_sizes():
    assert q8.q8_w4_values_bytes(4096, 14336) == 4096 * 14336 // 2
    assert q8.q8_w4_values_bytes(96, 40) == 48 * 64
    assert q8.q8_w4_scales_bytes(4096, 14336, 128, False) == 32 * 14336 * 2
    assert q8.q8_w4_scales_bytes(4096, 14336, 128, True) == 32 * 14336 * 3
    assert q8.q8_w4_scales_bytes(96, 40, 32, False) == 4 * 64 * 2       # three groups as two pairs
    assert q8.q8_w4_scales_bytes(160, 40, 128, True) == 2 * 64 * 3      # the last group is shorter
    for bad in ((0, 8, 32), (48, 8, 32), (64, 0, 32), (64, 8, 16), (64, 8, 0), (1 << 25, 8, 32)):
        assert q8.q8_w4_scales_bytes(*bad, False) == 0
    assert q8.q8_w4_values_bytes(33, 8) == 0
    assert q8.q8_w4_values_bytes(1 << 24, 1 << 24) == 0


def test_workspace_sizes():
    wide, narrow = weight(4096, 14336, 128), weight(4096, 1024, 128)
    assert q8.q8_w4_gemv_workspace_bytes(32, wide, 0) == 0
    one = q8.q8_w4_gemv_workspace_bytes(1, narrow, 0)
    assert one > 4 << 20 and one % 256 == 0
    assert q8.q8_w4_gemv_workspace_bytes(32, narrow, 1) > one
    assert q8.q8_w4_glu_workspace_bytes(1, narrow, 0) >= one
    for m, w, act in ((0, narrow, 0), (33, narrow, 0), (1, narrow, 2), (1, None, 0), (1, weight(40), 0)):
        assert q8.q8_w4_gemv_workspace_bytes(m, w, act) == 0
        assert q8.q8_w4_glu_workspace_bytes(m, w, act) == 0


CALLS = {
    "gemv": lambda w, m=1, x=A, y=A, act=0, ws=None, n=0: q8.q8_w4_gemv(x, w, y, m, act, None, S0, ws, n),
    "gemm": lambda w, m=1, x=A, y=A, act=0: q8.q8_w4_gemm(x, w, y, m, act, S0),
    "pair": lambda w, m=1, x=A, y=A, act=0: q8.q8_w4_gemv_glu(x, w, w, y, m, act, None, S0),
    "pairs": lambda w, m=1, x=A, y=A, act=0: q8.q8_w4_gemm_glu(x, w, w, y, m, act, None, S0),
}


@pytest.mark.parametrize("call", CALLS)
def test_products_refuse(call):
    f = CALLS[call]
    most = 32 if call in ("gemv", "pair") else 8192
    for m in (0, -1, most + 1):
        refuse(1, f, weight(), m, part="m =")
    for bad in (dict(K=0), dict(K=-32), dict(N=0), dict(K=1 << 25), dict(N=(1 << 24) + 1), dict(group=16),
                dict(group=256)):
        refuse(1, f, weight(**bad))
    assert "bound 64" in refuse(1, f, weight(K=40))
    refuse(1, f, weight(K=1 << 24, N=1 << 24), part="2^40")
    refuse(2, f, weight(fmt=2), part="scale_fmt")
    for act in (2, 3, -1):
        refuse(2, lambda w: f(w, act=act), weight(), part="act_fmt")
    refuse(3, f, None)
    refuse(3, f, weight(values=None), part="values")
    refuse(3, f, weight(scales=None), part="scales")
    refuse(4, f, weight(values=A + 8))
    refuse(4, f, weight(scales=A + 4))
    refuse(3, lambda w: f(w, x=None), weight(), part="x is NULL")
    refuse(3, lambda w: f(w, y=None), weight(), part="y is NULL")
    refuse(4, lambda w: f(w, x=A + 2), weight())
    refuse(4, lambda w: f(w, y=A + 4), weight())


def test_long_quantized_rows_are_refused():
    w = weight(K=1 << 24, N=64, group=128)
    refuse(1, q8.q8_w4_gemm, A, w, A, 512, 1, S0, part="too large")


def test_workspace_refusals():
    w = weight(4096, 1024, 128)
    need = q8.q8_w4_gemv_workspace_bytes(1, w, 0)
    refuse(5, q8.q8_w4_gemv, A, w, A, 1, 0, None, S0, None, 0)
    refuse(5, q8.q8_w4_gemv, A, w, A, 1, 0, None, S0, A, need - 1)
    refuse(4, q8.q8_w4_gemv, A, w, A, 1, 0, None, S0, A + 8, need)
    refuse(5, q8.q8_w4_gemv_glu, A, w, w, A, 1, 0, None, S0, A,
           q8.q8_w4_glu_workspace_bytes(1, w, 0) - 1)


def test_epilogue_refusals():
    w = weight()
    refuse(3, q8.q8_w4_gemv, A, w, A, 1, 0, q8.make_epilogue(write_y=False), S0, part="neither")
    refuse(3, q8.q8_w4_gemv, A, w, None, 1, 0, q8.make_epilogue(y_q8=A), S0)
    for k in ("bias", "residual", "y_q8"):
        refuse(4, q8.q8_w4_gemv, A, w, A, 1, 0, q8.make_epilogue(**{k: A + 4}), S0, part=k)
    for call in (q8.q8_w4_gemv_glu, q8.q8_w4_gemm_glu):
        refuse(3, call, A, w, w, A, 1, 0, q8.make_glu_epilogue(write_y=False), S0, part="neither")
        for k in ("bias_g", "bias_u", "y_q8"):
            refuse(4, call, A, w, w, A, 1, 0, q8.make_glu_epilogue(**{k: A + 4}), S0, part=k)


@pytest.mark.parametrize("other", [dict(K=96), dict(N=9), dict(group=64), dict(fmt=1), dict(zeros=True)])
def test_a_pair_of_unlike_weights_is_refused(other):
    for call in (q8.q8_w4_gemv_glu, q8.q8_w4_gemm_glu):
        refuse(1, call, A, weight(), weight(**other), A, 1, 0, None, S0, part="differ")


def test_repack_refusals():
    for call in (lambda u, s, z, w: q8.q8_w4_repack(u, s, z, w, S0),
                 lambda u, s, z, w: q8.q8_w4_unpack(w, u, s, z, S0)):
        refuse(3, call, None, A, None, weight(), part="u_kn")
        refuse(3, call, A, None, None, weight(), part="s_kn")
        refuse(3, call, A, A, None, weight(zeros=True), part="z_kn")
        refuse(4, call, A, A, A + 1, weight(zeros=True), part="z_kn")
        refuse(1, call, A, A, None, weight(K=33))
        refuse(2, call, A, A, None, weight(fmt=7))


def test_oracle_forms_agree():
    """The product's two ways of summing, and the weight's values, on a small case by hand."""
    u = np.array([[0x5F], [0x80]] * 8, np.uint8)          # rows 15, 5, 0, 8, ...
    s = np.array([[0x3C00]], np.uint16)                   # 1 in fp16
    x = np.arange(1.0, 33.0)[None, :]
    w = w4.weight(u, s, None, 0, 32)
    np.testing.assert_array_equal(w[:4, 0], [7, -3, -8, 0])
    assert w4.product(x, u, s, None, 0, 32)[0][0, 0] == (x @ w)[0, 0]
    z = np.array([[3]], np.uint8)
    assert w4.weight(u, s, z, 0, 32)[0, 0] == 12
    assert w4.scale_values(np.array([0x3F80], np.uint16), 1)[0] == 1.0
