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
