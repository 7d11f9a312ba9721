"""Refusals of the linear-attention and group-norm calls through the Python
binding, on the CPU: the tensors are host tensors and every call is refused
before anything is launched."""
import pytest
import torch

from gated_delta_product_amd import binding as B


@pytest.fixture
def host(monkeypatch):
    """The binding's checks and the library's, without a device."""
    def call(dev, fn, *args):
        B._check(fn(*args, None))

    monkeypatch.setattr(B, "_need_cuda", lambda *ts: torch.device("cpu"))
    monkeypatch.setattr(B, "_call", call)


def lin(K=64, V=64, T=3, H=1, HV=1):
    return [torch.zeros(1, T, h, d) for h, d in ((H, K), (H, K), (HV, V))]


@pytest.mark.parametrize("name,call,status", [
    ("prompt, K=96", lambda: B.linattn_fwd(*lin(K=96)), B.GDP_ERR_UNSUPPORTED),
    ("gradients, V=512", lambda: B.linattn_bwd(lin(V=512)[2], *lin(V=512)), B.GDP_ERR_UNSUPPORTED),
    ("step, K=96", lambda: B.linattn_decode(*lin(K=96), torch.zeros(1, 1, 64, 96)), B.GDP_ERR_UNSUPPORTED),
    ("prompt, HV % H", lambda: B.linattn_fwd(*lin(H=2, HV=3)), B.GDP_ERR_INVALID),
    ("norm, D=5000", lambda: B.group_norm_fwd(torch.zeros(2, 5000), 1), B.GDP_ERR_UNSUPPORTED),
    ("norm gradients, D=5000", lambda: B.group_norm_bwd(torch.zeros(2, 5000), torch.zeros(2, 5000), 1,
                                                        torch.ones(5000)), B.GDP_ERR_UNSUPPORTED),
    ("norm gradients, eps", lambda: B.group_norm_bwd(torch.zeros(2, 64), torch.zeros(2, 64), 1, torch.ones(64),
                                                     eps=-1.0), B.GDP_ERR_INVALID),
], ids=lambda x: x if isinstance(x, str) else "")
def test_refusals_keep_the_library_s_status(host, name, call, status):
    with pytest.raises(B.GdpError) as e:
        call()
    assert e.value.status == status, str(e.value)
    assert "workspace" not in str(e.value)


@pytest.mark.parametrize("T,H,HV,K,V", [(100, 1, 2, 64, 64), (9000, 32, 32, 64, 64), (8192, 8, 32, 128, 256)])
def test_workspace_without_g_serves_every_decay(T, H, HV, K, V):
    """Asked before the tensors exist, the size covers a decay per token and one per head."""
    import ctypes
    L = B.lib()

    def need(**kw):
        a = B.LinattnArgs(B=1, T=T, H=H, HV=HV, K=K, V=V, dtype=B.GDP_BF16, **kw)
        return L.gdp_linattn_workspace_bytes(ctypes.byref(a), 1)

    before, token, head = need(), need(g=0x1000), need(g_head=0x1000)
    assert before == head >= token > 0
    assert need(h0=0x1000) > before
