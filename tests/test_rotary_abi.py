"""Further refusals of gdp_rotary on the CPU: nothing here reaches the GPU."""
import ctypes

import pytest

from gated_delta_product_amd import binding as B

INV, UNS = B.GDP_ERR_INVALID, B.GDP_ERR_UNSUPPORTED


def rot(**kw):
    base = dict(B=1, T=10, H=2, HK=0, D=80, R=20, dtype=B.GDP_BF16, interleaved=0, inverse=0, scale=1.0, cu_seqlens=None,
                num_seqs=0, positions=None, pos_b_stride=10, pos_t_stride=1, offsets=None, freq=0x9000, q=0x10000,
                q_b_stride=1600, q_t_stride=160, k=None, k_b_stride=0, k_t_stride=0, qo=0x10000, qo_b_stride=1600,
                qo_t_stride=160, ko=None, ko_b_stride=0, ko_t_stride=0)
    base.update(kw)
    return B.RotaryArgs(**base)


@pytest.mark.parametrize("kw", [
    dict(T=1 << 28),  # 8 tokens of 140 pieces a block
    dict(T=1 << 28, D=4096, R=4096, q_t_stride=8192, qo_t_stride=8192),  # 2 of them, by their cosines
    dict(T=1 << 30, H=1, D=64, R=64, q_t_stride=64, qo_t_stride=64, dtype=B.GDP_F32, q=0x10004, qo=0x10004),
], ids=["pieces", "cosines", "elements"])
def test_too_many_threads_for_one_launch(kw):
    assert B.lib().gdp_rotary(ctypes.byref(rot(**kw)), None) == UNS
    assert b"too large" in B.lib().gdp_last_error()


@pytest.mark.parametrize("kw", [
    dict(B=2, q_b_stride=160, qo_b_stride=160),                      # row 1 is row 0 one token on
    dict(B=2, q_b_stride=1600 - 160, qo_b_stride=1600 - 160),        # its first token is row 0's last
    dict(B=3, q_b_stride=80 + 1600, qo_b_stride=80 + 1600, q_t_stride=320, qo_t_stride=320),  # between tokens, and into one
    dict(B=9, T=9, q_b_stride=7 * 160, qo_b_stride=7 * 160),
    dict(B=2, T=1, q_b_stride=100, qo_b_stride=100),
], ids=["same", "last", "between", "seven", "one token"])
def test_rows_of_an_output_that_overlap(kw):
    assert B.lib().gdp_rotary(ctypes.byref(rot(**kw)), None) == INV
    assert b"overlap" in B.lib().gdp_last_error()


@pytest.mark.parametrize("kw", [dict(qo=0x40000, ko=0x10000), dict(ko=0x10000), dict(qo=0x40000), dict(qo=0x50000, ko=0x50000)],
                         ids=["swapped", "k' on q", "q' on k", "k' on q'"])
def test_an_output_on_another_tensor(kw):
    both = dict(HK=2, k=0x40000, k_b_stride=1600, k_t_stride=160, ko=0x60000, ko_b_stride=1600, ko_t_stride=160)
    assert B.lib().gdp_rotary(ctypes.byref(rot(**{**both, **kw})), None) == INV
    assert B.lib().gdp_last_error()
