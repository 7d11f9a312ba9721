"""Steps and prompts whose outputs take the place of their inputs."""
import pytest
import torch

from gated_delta_product_amd import binding as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,S,C", [(3, 1, 40), (2, 5, 7), (1, 4, 64)])
def test_steps(n, S, C, dtype):
    x, g = (torch.randn(n, S, C, device=DEV).to(dtype) for _ in range(2))
    state, taps = torch.randn(n, C, device=DEV), torch.randn(C, 4, device=DEV)
    rows = torch.randn(n, 3, C, device=DEV).to(dtype)
    want_state, want_rows = state.clone(), rows.clone()
    how = dict(decay="sigmoid", complement=True)
    want = G.linrec_decode(x, g, want_state, **how)
    conv = G.conv_decode(x, want_rows, taps)
    for i in range(2):
        pair, s = [x.clone(), g.clone()], state.clone()
        assert G.linrec_decode(*pair, s, y=pair[i], **how) is pair[i]
        assert torch.equal(pair[i], want) and torch.equal(s, want_state) and torch.equal(pair[1 - i], (x, g)[1 - i])
    y, r = x.clone(), rows.clone()
    G.conv_decode(y, r, taps, y=y)
    assert torch.equal(y, conv) and torch.equal(r, want_rows)


def test_an_output_across_its_input_is_refused():
    wide = torch.randn(1, 20, 64, device=DEV)
    x, y, keep = wide[:, ::2], wide[:, :10], wide.clone()
    for call in (lambda: G.linrec_fwd(x, x, y=y), lambda: G.linrec_decode(x, x, torch.zeros(1, 64, device=DEV), y=y),
                 lambda: G.conv_decode(x, torch.zeros(1, 3, 64, device=DEV), torch.zeros(64, 4, device=DEV), y=y)):
        with pytest.raises(G.GdpError):
            call()
    assert torch.equal(wide, keep)
