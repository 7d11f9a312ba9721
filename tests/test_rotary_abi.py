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
