"""Layouts of rotary positions' outputs: any whose rows do not overlap."""
import pytest
import torch

from gated_delta_product_amd import binding as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("B,T,bs,ts", [
    (3, 7, 1, 3), (7, 3, 1, 7),        # tokens first
    (2, 2, 3, 2), (2, 9, 3, 2),        # batch rows between each other's tokens
    (4, 5, 6, 30), (5, 1, 2, 1), (1, 5, 0, 2)])
def test_batch_rows_among_tokens(B, T, bs, ts):
    H, D = 2, 16
    q = torch.randn(B, T, H, D, device=DEV)
    freq, _ = G.rotary_freq(D, device=DEV)
    want, _ = G.rotary(q, None, freq)
    wide = torch.full((B * bs + T * ts + 1, H, D), 3.0, device=DEV)
    out = wide.as_strided((B, T, H, D), (bs * H * D, ts * H * D, D, 1))
    places = {b * bs + t * ts for b in range(B) for t in range(T)}
    if len(places) < B * T:
        with pytest.raises(G.GdpError):
            G.rotary(q, None, freq, out=(out, None))
        return
    G.rotary(q, None, freq, out=(out, None))
    assert torch.equal(out, want)
    rest = [i for i in range(wide.shape[0]) if i not in places]
    assert (wide[rest] == 3).all()
    out.copy_(q)
    G.rotary(out, None, freq, out=(out, None))  # where they lie
    assert torch.equal(out, want)


def test_swapped_outputs_are_refused():
    q, k = (torch.randn(1, 5, 2, 16, device=DEV) for _ in range(2))
    freq, _ = G.rotary_freq(16, device=DEV)
    keep = q.clone(), k.clone()
    for out in ((k, q), (k, torch.empty_like(k)), (torch.empty_like(q), q)):
        with pytest.raises(G.GdpError):
            G.rotary(q, k, freq, out=out)
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1])
