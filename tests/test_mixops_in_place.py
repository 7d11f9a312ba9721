"""Outputs on top of inputs, at the C entries and on the CPU: refused where the
input's rows lie elsewhere than the output's, so nothing here reaches the GPU."""
import ctypes

import pytest

from gated_delta_product_amd import binding as B

INV, OK = B.GDP_ERR_INVALID, B.GDP_OK
BIG = 1 << 40
X, G, Y = 0x1000000, 0x2000000, 0x3000000


def rec(**kw):
    base = dict(B=2, T=10, C=64, dtype=B.GDP_BF16, g_dtype=B.GDP_BF16, decay=0, complement=0, cu_seqlens=None, num_seqs=0,
                x=X, x_b_stride=640, x_t_stride=64, g=G, g_b_stride=640, g_t_stride=64, h0=None, y=Y, ht=None)
    base.update(kw)
    return B.LinrecArgs(**base)


@pytest.mark.parametrize("kw", [
    dict(y=X, x_t_stride=128, x_b_stride=1280), dict(y=X, x_b_stride=1280), dict(y=X, x_b_stride=0), dict(y=X, B=1, x_t_stride=0),
    dict(y=G, g_t_stride=128, g_b_stride=1280), dict(y=G, g_dtype=B.GDP_F32), dict(y=X, B=3, T=1, x_b_stride=128)])
def test_recurrence(kw):
    assert B.lib().gdp_linrec_fwd(ctypes.byref(rec(**kw)), 0x100, BIG, None) == INV
    assert B.lib().gdp_last_error()


@pytest.mark.parametrize("kw", [
    dict(y=X, x_t_stride=128, x_n_stride=256), dict(y=X, x_n_stride=256), dict(y=X, x_t_stride=0),
    dict(y=X, S=1, x_n_stride=128)])
def test_steps(kw):
    shared = dict(n=3, S=2, C=64, dtype=B.GDP_BF16, pool=4, x=X, x_n_stride=128, x_t_stride=64, state=0x30000, slots=None, y=Y)
    r = dict(g_dtype=B.GDP_BF16, decay=1, complement=1, g=G, g_n_stride=128, g_t_stride=64)
    c = dict(W=4, activation=1, w=0x20000, b=None)
    assert B.lib().gdp_conv_decode(ctypes.byref(B.ConvDecodeArgs(**{**shared, **c, **kw})), None) == INV
    assert B.lib().gdp_linrec_decode(ctypes.byref(B.LinrecDecodeArgs(**{**shared, **r, **kw})), None) == INV
    on_g = {k.replace("x_", "g_"): v for k, v in kw.items()}
    on_g["y"] = G
    assert B.lib().gdp_linrec_decode(ctypes.byref(B.LinrecDecodeArgs(**{**shared, **r, **on_g})), None) == INV
    assert B.lib().gdp_linrec_decode(ctypes.byref(B.LinrecDecodeArgs(**{**shared, **r, "y": G, "g_dtype": B.GDP_F32})), None) == INV
