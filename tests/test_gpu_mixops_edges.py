"""Calls without rows, and positions given for packed requests."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from mixref import rotate, worst

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", [16, 7])
def test_no_rows(C, dtype):
    """States pass through sequences of no tokens, forwards and backwards; sums over none are zero."""
    x, s = torch.zeros(3, 0, C, dtype=dtype, device=DEV), torch.randn(3, C, device=DEV)
    y, ht = G.linrec_fwd(x, x, initial_state=s, output_final_state=True)
    assert y.shape == x.shape and torch.equal(ht, s)
    dx, dg, dh0 = G.linrec_bwd(x, x, x, initial_state=s, dht=s + 1)
    assert dx.shape == x.shape and dg.shape == x.shape and torch.equal(dh0, s + 1)
    assert not G.linrec_fwd(x, x, output_final_state=True)[1].any()
    w, b = torch.randn(C, 4, device=DEV), torch.randn(C, device=DEV)
    s = torch.randn(3, 3, C, device=DEV).to(dtype)
    y, ht = G.conv_fwd(x, w, b, initial_state=s, output_final_state=True)
    assert y.shape == x.shape and torch.equal(ht, s)
    dx, dw, db, dh0 = G.conv_bwd(x, x, w, b, initial_state=s, dht=s + 1)
    assert dx.shape == x.shape and not dw.any() and not db.any() and torch.equal(dh0, s + 1)
    q = torch.zeros(2, 0, 2, 16, dtype=dtype, device=DEV)
    assert G.rotary(q, None, torch.zeros(8, dtype=torch.float64, device=DEV))[0].shape == q.shape


def test_positions_of_packed_requests():
    """Given positions count, and rows outside every request stay as they were; heads of k alone, a scale of zero."""
    T, D = 50, 32
    x = torch.randn(1, T, 2, D)
    pos = torch.randint(0, 10000, (1, T), dtype=torch.int32)
    freq, _ = G.rotary_freq(D)
    cu = torch.tensor([3, 20, 41], dtype=torch.int32, device=DEV)
    out = (torch.full((1, T, 2, D), 7.0, device=DEV), torch.full((1, T, 2, D), 7.0, device=DEV))
    q, k = G.rotary(x.to(DEV), x.to(DEV), freq.to(DEV), positions=pos.to(DEV), cu_seqlens=cu, out=out)
    want, err = rotate(x[0], pos[0], freq)
    assert torch.equal(q, k)
    assert worst("q", q[0, 3:41].cpu(), want[3:41], err[3:41]) <= 1
    assert (q[0, :3] == 7).all() and (q[0, 41:] == 7).all()
    assert not G.rotary(x.to(DEV), None, freq.to(DEV), scale=0.0)[0].any()
