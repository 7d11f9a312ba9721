"""Refusals and sizes of the linear-attention and group-norm entry points on
the CPU: every call here fails validation (or has nothing to launch), so
nothing reaches the GPU."""
import ctypes
import os
import subprocess

import pytest
import torch

from gated_delta_product_amd import binding as B
from linref import Linear, decay_matrix

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS = B.GDP_ERR_INVALID, B.GDP_ERR_UNSUPPORTED


@pytest.mark.parametrize("cls,cname", [
    (B.LinattnArgs, "gdp_linattn_args"), (B.LinattnGrads, "gdp_linattn_grads"),
    (B.LinattnDecodeArgs, "gdp_linattn_decode_args"), (B.GroupNormArgs, "gdp_group_norm_args"),
    (B.GroupNormGrads, "gdp_group_norm_grads")])
def test_struct_layout_matches_c(tmp_path, cls, cname):
    fields = [f for f, _ in cls._fields_]
    prog = '#include <stdio.h>\n#include <stddef.h>\n#include "gdp.h"\nint main(void){\n'
    prog += 'printf("%%zu\\n", sizeof(%s));\n' % cname
    prog += "".join('printf("%%zu\\n", offsetof(%s, %s));\n' % (cname, f) for f in fields)
    c = tmp_path / "layout.c"
    c.write_text(prog + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)])
    vals = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert vals == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


def lin(**kw):
    base = dict(B=1, T=128, H=2, HV=4, K=64, V=128, scale=0.0, dtype=B.GDP_BF16, cu_seqlens=None, num_seqs=0,
                q=0x10000, q_b_stride=128 * 128, q_t_stride=128, k=0x20000, k_b_stride=128 * 128, k_t_stride=128,
                v=0x30000, v_b_stride=128 * 512, v_t_stride=512, g=0x50000, g_b_stride=512, g_t_stride=4,
                g_head=None, h0=0x60000, o=0x70000, ht=0x80000)
    base.update(kw)
    return B.LinattnArgs(**base)


BAD_LIN = [
    ("K=96", dict(K=96), UNS), ("V=512", dict(V=512), UNS), ("HV % H", dict(H=3), INV), ("H=0", dict(H=0), INV),
    ("dtype", dict(dtype=9), INV), ("B<0", dict(B=-1), INV), ("T<0", dict(T=-1), INV),
    ("scale", dict(scale=float("inf")), INV), ("cu with B=2", dict(B=2, cu_seqlens=0x1000, num_seqs=2), INV),
    ("num_seqs<0", dict(cu_seqlens=0x1000, num_seqs=-1), INV), ("two decays", dict(g_head=0x51000), INV),
    ("g stride", dict(g_t_stride=-4), INV), ("g alignment", dict(g=0x50002), INV), ("q NULL", dict(q=None), INV),
    ("k alignment", dict(k=0x20008), INV), ("v token stride", dict(v_t_stride=516), INV),
    ("q batch stride", dict(q_b_stride=-16), INV), ("far tokens", dict(v_t_stride=1 << 25), UNS),
    ("h0 alignment", dict(h0=0x60004), INV), ("HV", dict(HV=1 << 17, H=1 << 17), UNS),
    ("too many tokens", dict(T=1 << 32), UNS), ("too many walks", dict(T=1 << 30, B=60), UNS),
    ("cu alignment", dict(cu_seqlens=0x1001, num_seqs=1), INV),
]


@pytest.mark.parametrize("name,kw,status", BAD_LIN, ids=[c[0] for c in BAD_LIN])
def test_linattn_rejects(name, kw, status):
    a = lin(**kw)
    d = B.LinattnGrads(dout=0x90000, do_b_stride=128 * 512, do_t_stride=512, dq=0xA0000, dk=0xB0000, dv=0xC0000)
    L = B.lib()
    big = 1 << 40
    assert L.gdp_linattn_fwd(ctypes.byref(a), 0x1000000, big, None) == status
    assert L.gdp_last_error()
    assert L.gdp_linattn_bwd(ctypes.byref(a), ctypes.byref(d), 0x1000000, big, None) == status
    assert L.gdp_last_error()


def test_linattn_rejects_outputs_and_workspaces():
    L = B.lib()
    ok = lin(T=4096)
    need = L.gdp_linattn_workspace_bytes(ctypes.byref(ok), 0)
    assert need > 0
    for a, ws, n in ((lin(o=None), 0, 0), (lin(o=0x70004), 0, 0), (lin(ht=0x80008), 0, 0), (ok, 0, need),
                     (ok, 0x1000000, need - 1), (ok, 0x1000010, need)):
        assert L.gdp_linattn_fwd(ctypes.byref(a), ws, n, None) == INV
    assert L.gdp_linattn_fwd(None, None, 0, None) == INV
    need = L.gdp_linattn_workspace_bytes(ctypes.byref(ok), 1)
    good = dict(dout=0x90000, do_b_stride=128 * 512, do_t_stride=512, dq=0xA0000, dk=0xB0000, dv=0xC0000)
    for kw in (dict(dout=None), dict(dq=None), dict(dk=0xB0004), dict(dv=None), dict(dg_head=0xD0000),
               dict(dg=0xD0001), dict(dht=0xD0008), dict(dh0=0x60000), dict(dh0=0xE0000, dht=0xE0000),
               dict(do_t_stride=3)):
        d = B.LinattnGrads(**{**good, **kw})
        assert L.gdp_linattn_bwd(ctypes.byref(ok), ctypes.byref(d), 0x1000000, need, None) == INV, kw
    d = B.LinattnGrads(**good)
    assert L.gdp_linattn_bwd(ctypes.byref(ok), ctypes.byref(d), 0x1000000, need - 1, None) == INV
    assert L.gdp_linattn_bwd(ctypes.byref(ok), None, 0x1000000, need, None) == INV
    no_h0 = lin(h0=None, g=None, g_head=0x50000)
    for kw in (dict(dh0=0xE0000), dict(dg=0xE0000)):
        d = B.LinattnGrads(**{**good, **kw})
        assert L.gdp_linattn_bwd(ctypes.byref(no_h0), ctypes.byref(d), 0x1000000, 1 << 40, None) == INV, kw


@pytest.mark.parametrize("kw", [
    dict(B=1 << 20, T=1, H=64, HV=64), dict(cu_seqlens=0x1000, num_seqs=1 << 20, T=1 << 20, H=64, HV=64),
    dict(B=1 << 19, T=600, H=4, HV=32, V=256)], ids=["rows of one token", "packed", "V=256"])
def test_linattn_refuses_launches_over_2_32_threads(kw):
    L = B.lib()
    w, v = kw["H"] * 64, kw["HV"] * kw.get("V", 128)
    a = lin(q_t_stride=w, k_t_stride=w, v_t_stride=v, **kw)
    d = B.LinattnGrads(dout=0x90000, do_t_stride=v, dq=0xA0000, dk=0xB0000, dv=0xC0000)
    assert L.gdp_linattn_fwd(ctypes.byref(a), 0x1000000, 1 << 60, None) == UNS
    assert b"one launch" in L.gdp_last_error()
    assert L.gdp_linattn_bwd(ctypes.byref(a), ctypes.byref(d), 0x1000000, 1 << 60, None) == UNS
    assert L.gdp_linattn_workspace_bytes(ctypes.byref(a), 0) == -1


def test_strides_of_single_elements_do_not_matter():
    """One token or one row: its stride may be anything (the calls get as far as the missing output)."""
    L = B.lib()
    odd = dict(q_t_stride=3, k_t_stride=1 << 40, v_t_stride=0, q_b_stride=5, o=None)
    for a in (lin(T=1, B=1, **odd), lin(T=128, B=1, q_b_stride=7, k_b_stride=1, o=None)):
        assert L.gdp_linattn_fwd(ctypes.byref(a), None, 0, None) == INV
        assert b"o is NULL" in L.gdp_last_error()
    a = dec(S=1, q_t_stride=3, k_t_stride=1 << 40, v_t_stride=1, o=None)
    assert L.gdp_linattn_decode(ctypes.byref(a), None) == INV
    assert b"o is NULL" in L.gdp_last_error()
    for kw in (dict(T=2, B=1, q_t_stride=132), dict(T=1, B=2, v_b_stride=12)):
        assert L.gdp_linattn_fwd(ctypes.byref(lin(o=None, **kw)), None, 0, None) == INV
        assert b"aligned" in L.gdp_last_error()


def test_linattn_nothing_to_do():
    L = B.lib()
    assert L.gdp_linattn_fwd(ctypes.byref(lin(B=0)), None, 0, None) == B.GDP_OK
    assert L.gdp_linattn_fwd(ctypes.byref(lin(T=0, ht=None)), None, 0, None) == B.GDP_OK
    assert L.gdp_linattn_fwd(ctypes.byref(lin(cu_seqlens=0x1000, num_seqs=0)), None, 0, None) == B.GDP_OK
    assert L.gdp_linattn_workspace_bytes(ctypes.byref(lin(K=7)), 0) == -1
    assert L.gdp_linattn_workspace_bytes(None, 1) == -1


def dec(**kw):
    base = dict(n=3, S=2, H=2, HV=4, K=128, V=64, scale=0.0, dtype=B.GDP_BF16, pool=4, q=0x10000, q_n_stride=512,
                q_t_stride=256, k=0x20000, k_n_stride=512, k_t_stride=256, v=0x30000, v_n_stride=512, v_t_stride=256,
                g=0x40000, g_n_stride=8, g_t_stride=4, g_head=None, state=0x50000, slots=0x60000, o=0x70000)
    base.update(kw)
    return B.LinattnDecodeArgs(**base)


@pytest.mark.parametrize("name,kw,status", [
    ("K", dict(K=32), UNS), ("V", dict(V=96), UNS), ("HV", dict(HV=5), INV), ("dtype", dict(dtype=5), INV),
    ("n<0", dict(n=-1), INV), ("S", dict(S=5000), UNS), ("n", dict(n=1 << 30), UNS), ("threads", dict(n=1 << 21), UNS), ("pool", dict(pool=-1), INV),
    ("pool without slots", dict(pool=2, slots=None), INV), ("two decays", dict(g_head=0x41000), INV),
    ("state NULL", dict(state=None), INV), ("state alignment", dict(state=0x50004), INV), ("o", dict(o=None), INV),
    ("q", dict(q=0x10002), INV), ("k stride", dict(k_n_stride=4), INV), ("v", dict(v=None), INV),
    ("slots alignment", dict(slots=0x60002), INV), ("g stride", dict(g_n_stride=-1), INV),
    ("scale", dict(scale=float("nan")), INV)])
def test_decode_rejects(name, kw, status):
    assert B.lib().gdp_linattn_decode(ctypes.byref(dec(**kw)), None) == status
    assert B.lib().gdp_last_error()


def test_decode_nothing_to_do():
    assert B.lib().gdp_linattn_decode(ctypes.byref(dec(n=0)), None) == B.GDP_OK
    assert B.lib().gdp_linattn_decode(ctypes.byref(dec(S=0)), None) == B.GDP_OK
    assert B.lib().gdp_linattn_decode(None, None) == INV


def norm(**kw):
    base = dict(n=2, T=5, groups=4, D=32, dtype=B.GDP_BF16, activation=1, centered=1, eps=1e-5, x=0x10000,
                x_n_stride=640, x_t_stride=128, z=0x20000, z_n_stride=640, z_t_stride=128, w=0x30000, b=0x40000,
                y=0x50000)
    base.update(kw)
    return B.GroupNormArgs(**base)


@pytest.mark.parametrize("name,kw,status", [
    ("dtype", dict(dtype=4), INV), ("activation", dict(activation=7), INV), ("groups", dict(groups=0), INV),
    ("D=0", dict(D=0), INV), ("D", dict(D=4097), UNS), ("eps", dict(eps=-1.0), INV), ("eps nan", dict(eps=float("nan")), INV),
    ("C", dict(groups=1 << 20, D=256), UNS), ("n<0", dict(n=-1), INV), ("rows", dict(n=1 << 20, T=1 << 20), UNS), ("x NULL", dict(x=None), INV),
    ("x alignment", dict(x=0x10001), INV), ("z stride", dict(z_t_stride=-1), INV), ("w", dict(w=0x30002), INV)])
def test_group_norm_rejects(name, kw, status):
    L = B.lib()
    a = norm(**kw)
    assert L.gdp_group_norm_fwd(ctypes.byref(a), None) == status
    d = B.GroupNormGrads(dy=0x60000, dy_n_stride=640, dy_t_stride=128, dx=0x70000, dz=0x80000, dw=0x90000, db=0xA0000)
    assert L.gdp_group_norm_bwd(ctypes.byref(a), ctypes.byref(d), 0x1000000, 1 << 40, None) == status
    assert L.gdp_last_error()


def test_group_norm_rejects_outputs_and_workspaces():
    L = B.lib()
    assert L.gdp_group_norm_fwd(ctypes.byref(norm(y=None)), None) == INV
    assert L.gdp_group_norm_fwd(None, None) == INV
    need = L.gdp_group_norm_workspace_bytes(ctypes.byref(norm()))
    assert need > 0 and L.gdp_group_norm_workspace_bytes(ctypes.byref(norm(D=0))) == -1
    good = dict(dy=0x60000, dy_n_stride=640, dy_t_stride=128, dx=0x70000, dz=0x80000, dw=0x90000, db=0xA0000)
    for kw in (dict(dy=None), dict(dx=None), dict(dz=None), dict(dw=0x90001), dict(dy_n_stride=-2)):
        d = B.GroupNormGrads(**{**good, **kw})
        assert L.gdp_group_norm_bwd(ctypes.byref(norm()), ctypes.byref(d), 0x1000000, need, None) == INV, kw
    d = B.GroupNormGrads(**good)
    for ws, n in ((0, need), (0x1000000, need - 1), (0x1000004, need)):
        assert L.gdp_group_norm_bwd(ctypes.byref(norm()), ctypes.byref(d), ws, n, None) == INV
    assert L.gdp_group_norm_bwd(ctypes.byref(norm()), None, 0x1000000, need, None) == INV
    assert L.gdp_group_norm_fwd(ctypes.byref(norm(n=0)), None) == B.GDP_OK


def test_leading_dimensions_fold():
    x = torch.zeros(4, 5, 7, 16)
    assert B._token_rows(x, "x") == (20, 7, 112, 16)
    assert B._token_rows(x[:, :1], "x") == (4, 7, 560, 16)
    assert B._token_rows(x[:1, :2, 1:3], "x") == (2, 2, 112, 16)
    assert B._token_rows(x[0, 0], "x") == (1, 7, 0, 16)
    with pytest.raises(ValueError):
        B._token_rows(x[:, :2], "x")


def test_binding_wants_gpu_tensors():
    x = torch.zeros(1, 4, 2, 64)
    for call in (lambda: B.linattn_fwd(x, x, x), lambda: B.linattn_bwd(x, x, x, x),
                 lambda: B.linattn_decode(x, x, x, torch.zeros(1, 2, 64, 64)), lambda: B.group_norm_fwd(x[0, :, 0], 2),
                 lambda: B.group_norm_bwd(x[0, :, 0], x[0, :, 0], 2)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the tests' own plain form

def test_plain_form_is_the_recurrence():
    gen = torch.Generator().manual_seed(1)
    L, H, HV, K, V = 9, 2, 4, 6, 5
    q, k, v = (torch.randn(L, h, n, generator=gen).double() for h, n in ((H, K), (H, K), (HV, V)))
    g, h0 = -torch.rand(L, HV, generator=gen).double(), torch.randn(HV, V, K, generator=gen).double()
    leaves = [t.requires_grad_() for t in (q, k, v, g, h0)]
    S, o = h0, []
    for t in range(L):
        kt, qt = (x[t].repeat_interleave(2, 0) for x in (k, q))
        S = S * torch.exp(g[t])[:, None, None] + v[t][..., None] * kt[:, None, :]
        o.append((S * qt[:, None, :]).sum(-1) * 0.3)
    o = torch.stack(o)
    do, dht = torch.randn(o.shape, generator=gen).double(), torch.randn(S.shape, generator=gen).double()
    grads = torch.autograd.grad((o * do).sum() + (S * dht).sum(), leaves)
    r = Linear(*(t.detach() for t in (q, k, v, g)), 0.3, h0.detach())
    po, pht = r.forward()
    assert torch.allclose(po, o, atol=1e-12) and torch.allclose(pht, S, atol=1e-12)
    for x, y in zip(r.backward(do, dht), grads):
        assert torch.allclose(x, y, atol=1e-11)
    d = decay_matrix(torch.tensor([[-1.0, float("-inf"), -2.0]]).double())
    assert torch.isfinite(d).all() and d[0, 2, 0] == 0 and d[0, 2, 2] == torch.exp(torch.tensor(-2.0).double())
