"""Refusals and sizes of the gated linear recurrence, the short convolution and
rotary positions on the CPU: every call here fails validation (or has nothing
to launch), so nothing reaches the GPU."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

from gated_delta_product_amd import binding as B
from mixref import Conv, Rec, rotate

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, OK = B.GDP_ERR_INVALID, B.GDP_ERR_UNSUPPORTED, B.GDP_OK
BIG = 1 << 50


@pytest.mark.parametrize("cls,cname", [
    (B.LinrecArgs, "gdp_linrec_args"), (B.LinrecGrads, "gdp_linrec_grads"), (B.LinrecDecodeArgs, "gdp_linrec_decode_args"),
    (B.ConvArgs, "gdp_conv_args"), (B.ConvGrads, "gdp_conv_grads"), (B.ConvDecodeArgs, "gdp_conv_decode_args"),
    (B.RotaryArgs, "gdp_rotary_args")])
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


def rec(**kw):
    base = dict(B=2, T=100, C=64, dtype=B.GDP_BF16, g_dtype=B.GDP_BF16, decay=0, complement=0, cu_seqlens=None, num_seqs=0,
                x=0x10000, x_b_stride=6400, x_t_stride=64, g=0x20000, g_b_stride=6400, g_t_stride=64, h0=0x30000,
                y=0x40000, ht=0x50000)
    base.update(kw)
    return B.LinrecArgs(**base)


SHARED_BAD = [
    ("dtype", dict(dtype=9), INV), ("B<0", dict(B=-1), INV), ("T<0", dict(T=-1), INV), ("C=0", dict(C=0), INV),
    ("C", dict(C=(1 << 20) + 1), UNS), ("cu with B=2", dict(cu_seqlens=0x1000, num_seqs=2), INV),
    ("num_seqs<0", dict(B=1, cu_seqlens=0x1000, num_seqs=-1), INV),
    ("num_seqs", dict(B=1, cu_seqlens=0x1000, num_seqs=1 << 31), UNS),
    ("cu alignment", dict(B=1, cu_seqlens=0x1002, num_seqs=1), INV), ("rows", dict(B=1 << 16, T=1 << 16), UNS),
    ("tokens", dict(B=1, T=1 << 31), UNS), ("x NULL", dict(x=None), INV), ("x alignment", dict(x=0x10001), INV),
    ("x token stride", dict(x_t_stride=-1), INV), ("x batch stride", dict(x_b_stride=-1), INV),
    ("h0 alignment", dict(h0=0x30001), INV),
]


@pytest.mark.parametrize("name,kw,status", SHARED_BAD + [
    ("g dtype", dict(dtype=B.GDP_F32, g_dtype=B.GDP_BF16), INV), ("g dtype 2", dict(g_dtype=5), INV),
    ("decay", dict(decay=2), INV), ("g NULL", dict(g=None), INV), ("g alignment", dict(g=0x20001), INV),
    ("g stride", dict(g_t_stride=-64), INV), ("threads", dict(B=1, T=(1 << 31) - 1, C=65, x_t_stride=65, g_t_stride=65), UNS),
    ], ids=lambda v: v if isinstance(v, str) else "")
def test_linrec_rejects(name, kw, status):
    a = rec(**kw)
    d = B.LinrecGrads(dy=0x60000, dy_b_stride=6400, dy_t_stride=64, dx=0x70000, dg=0x80000)
    L = B.lib()
    assert L.gdp_linrec_bwd(ctypes.byref(a), ctypes.byref(d), 0x1000000, BIG, None) == status
    assert L.gdp_last_error()
    assert L.gdp_linrec_fwd(ctypes.byref(a), 0x1000000, BIG, None) == status
    assert L.gdp_last_error()


def test_linrec_rejects_outputs_and_workspaces():
    L = B.lib()
    ok = rec(T=5000)
    need = L.gdp_linrec_workspace_bytes(ctypes.byref(ok), 0)
    assert need > 0
    for a, ws, n in ((rec(y=None), 0, 0), (rec(y=0x40001), 0, 0), (rec(ht=0x50002), 0, 0), (rec(ht=0x30000), 0, 0), (ok, 0, need),
                     (ok, 0x1000000, need - 1), (ok, 0x1000010, need)):
        assert L.gdp_linrec_fwd(ctypes.byref(a), ws, n, None) == INV
    assert L.gdp_linrec_fwd(None, None, 0, None) == INV
    need = L.gdp_linrec_workspace_bytes(ctypes.byref(ok), 1)
    good = dict(dy=0x60000, dy_b_stride=6400, dy_t_stride=64, dx=0x70000, dg=0x80000)
    for kw in (dict(dy=None), dict(dy=0x60001), dict(dy_t_stride=-1), dict(dx=None), dict(dg=None), dict(dg=0x80001),
               dict(dht=0x90002), dict(dh0=0x90001), dict(dh0=0x30000), dict(dh0=0x90000, dht=0x90000)):
        d = B.LinrecGrads(**{**good, **kw})
        assert L.gdp_linrec_bwd(ctypes.byref(ok), ctypes.byref(d), 0x1000000, need, None) == INV, kw
    d = B.LinrecGrads(**good)
    for ws, n in ((0, need), (0x1000000, need - 1), (0x1000004, need)):
        assert L.gdp_linrec_bwd(ctypes.byref(ok), ctypes.byref(d), ws, n, None) == INV
    assert L.gdp_linrec_bwd(ctypes.byref(ok), None, 0x1000000, need, None) == INV
    assert L.gdp_linrec_workspace_bytes(None, 0) == -1
    assert L.gdp_linrec_workspace_bytes(ctypes.byref(rec(C=0)), 0) == -1


def test_nothing_to_do():
    L = B.lib()
    assert L.gdp_linrec_fwd(ctypes.byref(rec(B=0)), None, 0, None) == OK
    assert L.gdp_linrec_fwd(ctypes.byref(rec(T=0, ht=None)), None, 0, None) == OK
    assert L.gdp_conv_fwd(ctypes.byref(conv(B=0)), None) == OK
    assert L.gdp_conv_fwd(ctypes.byref(conv(T=0, ht=None)), None) == OK
    d = B.ConvGrads(dy=None, dx=None)
    assert L.gdp_conv_bwd(ctypes.byref(conv(T=0)), ctypes.byref(d), None, 0, None) == OK
    assert L.gdp_rotary(ctypes.byref(rot(T=0)), None) == OK
    assert L.gdp_rotary(ctypes.byref(rot(B=1, cu_seqlens=0x1000, num_seqs=0)), None) == OK
    for a, f in ((rdec, L.gdp_linrec_decode), (cdec, L.gdp_conv_decode)):
        assert f(ctypes.byref(a(n=0)), None) == OK and f(ctypes.byref(a(S=0)), None) == OK and f(None, None) == INV


def rdec(**kw):
    base = dict(n=3, S=2, C=64, dtype=B.GDP_BF16, g_dtype=B.GDP_F32, decay=1, complement=1, pool=4, x=0x10000,
                x_n_stride=128, x_t_stride=64, g=0x20000, g_n_stride=128, g_t_stride=64, state=0x30000, slots=0x40000,
                y=0x50000)
    base.update(kw)
    return B.LinrecDecodeArgs(**base)


def cdec(**kw):
    base = dict(n=3, S=2, C=64, W=4, dtype=B.GDP_BF16, activation=1, pool=4, x=0x10000, x_n_stride=128, x_t_stride=64,
                w=0x20000, b=0x28000, state=0x30000, slots=0x40000, y=0x50000)
    base.update(kw)
    return B.ConvDecodeArgs(**base)


DECODE_BAD = [
    ("dtype", dict(dtype=5), INV), ("n<0", dict(n=-1), INV), ("S<0", dict(S=-1), INV), ("S", dict(S=5000), UNS),
    ("C=0", dict(C=0), INV), ("C", dict(C=1 << 21), UNS), ("n", dict(n=1 << 31), UNS), ("pool<0", dict(pool=-1), INV),
    ("pool without slots", dict(pool=2, slots=None), INV), ("slots alignment", dict(slots=0x40002), INV),
    ("x NULL", dict(x=None), INV), ("x alignment", dict(x=0x10001), INV), ("x stride", dict(x_n_stride=-8), INV),
    ("y NULL", dict(y=None), INV), ("y alignment", dict(y=0x50001), INV), ("state NULL", dict(state=None), INV),
    ("state alignment", dict(state=0x30001), INV)]


@pytest.mark.parametrize("name,kw,status", DECODE_BAD + [
    ("g dtype", dict(g_dtype=7), INV), ("g NULL", dict(g=None), INV), ("decay", dict(decay=-1), INV)],
    ids=lambda v: v if isinstance(v, str) else "")
def test_linrec_decode_rejects(name, kw, status):
    assert B.lib().gdp_linrec_decode(ctypes.byref(rdec(**kw)), None) == status
    assert B.lib().gdp_last_error()


@pytest.mark.parametrize("name,kw,status", DECODE_BAD + [
    ("W=1", dict(W=1), UNS), ("W=5", dict(W=5), UNS), ("W=0", dict(W=0), INV), ("activation", dict(activation=9), INV),
    ("w NULL", dict(w=None), INV), ("b alignment", dict(b=0x28002), INV)], ids=lambda v: v if isinstance(v, str) else "")
def test_conv_decode_rejects(name, kw, status):
    assert B.lib().gdp_conv_decode(ctypes.byref(cdec(**kw)), None) == status
    assert B.lib().gdp_last_error()


def conv(**kw):
    base = dict(B=2, T=100, C=64, W=4, dtype=B.GDP_BF16, activation=1, cu_seqlens=None, num_seqs=0, x=0x10000,
                x_b_stride=6400, x_t_stride=64, w=0x20000, b=0x28000, h0=0x30000, y=0x40000, ht=0x50000)
    base.update(kw)
    return B.ConvArgs(**base)


@pytest.mark.parametrize("name,kw,status", SHARED_BAD + [
    ("W=1", dict(W=1), UNS), ("W=5", dict(W=5), UNS), ("W=0", dict(W=0), INV), ("activation", dict(activation=3), INV),
    ("w NULL", dict(w=None), INV), ("w alignment", dict(w=0x20002), INV),
    ("threads", dict(B=1, T=(1 << 31) - 1, C=65, x_t_stride=65), UNS)], ids=lambda v: v if isinstance(v, str) else "")
def test_conv_rejects(name, kw, status):
    L = B.lib()
    a = conv(**kw)
    assert L.gdp_conv_fwd(ctypes.byref(a), None) == status
    assert L.gdp_last_error()
    d = B.ConvGrads(dy=0x60000, dy_b_stride=6400, dy_t_stride=64, dx=0x70000, dw=0x80000, db=0x90000)
    assert L.gdp_conv_bwd(ctypes.byref(a), ctypes.byref(d), 0x1000000, BIG, None) == status
    assert L.gdp_last_error()


def test_conv_rejects_outputs_and_workspaces():
    L = B.lib()
    for kw in (dict(y=None), dict(y=0x40001), dict(y=0x10000), dict(ht=0x50001), dict(ht=0x30000)):
        assert L.gdp_conv_fwd(ctypes.byref(conv(**kw)), None) == INV, kw
    assert L.gdp_conv_fwd(None, None) == INV
    ok = conv()
    need = L.gdp_conv_workspace_bytes(ctypes.byref(ok))
    assert need > 0 and L.gdp_conv_workspace_bytes(ctypes.byref(conv(W=9))) == -1
    good = dict(dy=0x60000, dy_b_stride=6400, dy_t_stride=64, dx=0x70000, dw=0x80000, db=0x90000)
    for kw in (dict(dy=None), dict(dy_t_stride=-1), dict(dx=None), dict(dx=0x10000), dict(dx=0x60000), dict(dw=0x80001),
               dict(db=0x90002), dict(dht=0xA0001), dict(dh0=0xA0001), dict(dh0=0x30000), dict(dh0=0xA0000, dht=0xA0000)):
        d = B.ConvGrads(**{**good, **kw})
        assert L.gdp_conv_bwd(ctypes.byref(ok), ctypes.byref(d), 0x1000000, need, None) == INV, kw
    d = B.ConvGrads(**good)
    for ws, n in ((0, need), (0x1000000, need - 1), (0x1000004, need)):
        assert L.gdp_conv_bwd(ctypes.byref(ok), ctypes.byref(d), ws, n, None) == INV
    assert L.gdp_conv_bwd(ctypes.byref(ok), None, 0x1000000, need, None) == INV


def rot(**kw):
    base = dict(B=2, T=10, H=4, HK=2, D=64, R=32, dtype=B.GDP_BF16, interleaved=0, inverse=0, scale=1.0, cu_seqlens=None,
                num_seqs=0, positions=None, pos_b_stride=10, pos_t_stride=1, offsets=0x8000, freq=0x9000, q=0x10000,
                q_b_stride=2560, q_t_stride=256, k=0x20000, k_b_stride=1280, k_t_stride=128, qo=0x30000, qo_b_stride=2560,
                qo_t_stride=256, ko=0x40000, ko_b_stride=1280, ko_t_stride=128)
    base.update(kw)
    return B.RotaryArgs(**base)


@pytest.mark.parametrize("name,kw,status", [
    ("dtype", dict(dtype=3), INV), ("no heads", dict(H=0, HK=0), INV), ("H<0", dict(H=-1), INV), ("HK<0", dict(HK=-1), INV),
    ("D=0", dict(D=0), INV), ("R=0", dict(R=0), INV), ("R odd", dict(R=31), INV), ("R>D", dict(R=66), INV),
    ("D", dict(D=8192), UNS), ("row", dict(H=1 << 20), UNS), ("scale", dict(scale=float("nan")), INV),
    ("B<0", dict(B=-1), INV), ("cu with B=2", dict(cu_seqlens=0x1000, num_seqs=1), INV),
    ("rows", dict(B=1 << 16, T=1 << 16), UNS), ("two positions", dict(positions=0x7000), INV),
    ("offsets alignment", dict(offsets=0x8002), INV), ("position stride", dict(positions=0x7000, offsets=None, pos_t_stride=-1), INV),
    ("freq NULL", dict(freq=None), INV), ("freq alignment", dict(freq=0x9004), INV), ("q NULL", dict(q=None), INV),
    ("k NULL", dict(k=None), INV), ("qo NULL", dict(qo=None), INV), ("ko alignment", dict(ko=0x40001), INV),
    ("q stride", dict(q_t_stride=-256), INV), ("output tokens overlap", dict(qo_t_stride=255), INV),
    ("output rows overlap", dict(ko_b_stride=64), INV), ("in place, other strides", dict(qo=0x10000, qo_t_stride=512), INV)],
    ids=lambda v: v if isinstance(v, str) else "")
def test_rotary_rejects(name, kw, status):
    assert B.lib().gdp_rotary(ctypes.byref(rot(**kw)), None) == status
    assert B.lib().gdp_last_error()
    assert B.lib().gdp_rotary(None, None) == INV


# ------------------------------------------------------------------ the binding's own checks

@pytest.fixture
def host(monkeypatch):
    """The binding's checks and the library's, without a device."""
    def call(dev, fn, *args):
        B._check(fn(*args, None))

    monkeypatch.setattr(B, "_need_cuda", lambda *ts: torch.device("cpu"))
    monkeypatch.setattr(B, "_call", call)


def test_binding_wants_gpu_tensors():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    for call in (lambda: B.linrec_fwd(x, x), lambda: B.linrec_bwd(x, x, x), lambda: B.linrec_decode(x, x, torch.zeros(1, 8)),
                 lambda: B.conv_fwd(x, w), lambda: B.conv_bwd(x, x, w), lambda: B.conv_decode(x, torch.zeros(1, 3, 8), w),
                 lambda: B.rotary(x[None], None, torch.zeros(4, dtype=torch.float64))):
        with pytest.raises(ValueError):
            call()


X, W8, I32 = torch.zeros(2, 4, 8), torch.zeros(8, 4), torch.int32


@pytest.mark.parametrize("name,call", [
    ("x 2-D", lambda: B.linrec_fwd(X[0], X[0])), ("g shape", lambda: B.linrec_fwd(X, X[:1])),
    ("g dtype", lambda: B.linrec_fwd(X, X.bfloat16())), ("x columns", lambda: B.linrec_fwd(X[..., ::2], X[..., :4])),
    ("decay", lambda: B.linrec_fwd(X, X, decay="exp")), ("h0", lambda: B.linrec_fwd(X, X, initial_state=torch.zeros(1, 8))),
    ("cu dtype", lambda: B.linrec_fwd(X[:1], X[:1], cu_seqlens=torch.zeros(2, dtype=torch.int64))),
    ("y", lambda: B.linrec_fwd(X, X, y=torch.zeros(2, 4, 9))), ("dy", lambda: B.linrec_bwd(X[:1], X, X)),
    ("dht", lambda: B.linrec_bwd(X, X, X, dht=torch.zeros(2, 7))), ("state", lambda: B.linrec_decode(X, X, torch.zeros(2, 9))),
    ("slots", lambda: B.linrec_decode(X, X, torch.zeros(2, 8), slots=torch.zeros(3, dtype=I32))),
    ("weight", lambda: B.conv_fwd(X, W8[:4])), ("weight dtype", lambda: B.conv_fwd(X, W8.bfloat16())),
    ("bias", lambda: B.conv_fwd(X, W8, torch.zeros(7))), ("activation", lambda: B.conv_fwd(X, W8, activation="gelu")),
    ("conv h0", lambda: B.conv_fwd(X, W8, initial_state=torch.zeros(2, 4, 8))), ("conv dy", lambda: B.conv_bwd(X[:, :3], X, W8)),
    ("conv state", lambda: B.conv_decode(X, torch.zeros(2, 8, 3), W8)),
    ("q 3-D", lambda: B.rotary(X, None, torch.zeros(4).double())),
    ("freq dtype", lambda: B.rotary(X[None], None, torch.zeros(4))),
    ("k shape", lambda: B.rotary(X[None], X[None, :1], torch.zeros(4).double())),
    ("positions", lambda: B.rotary(X[None], None, torch.zeros(4).double(), positions=torch.zeros(1, 2))),
    ("offsets", lambda: B.rotary(X[None], None, torch.zeros(4).double(), offsets=torch.zeros(2, dtype=I32))),
    ("out", lambda: B.rotary(X[None], None, torch.zeros(4).double(), out=(X[None], X[None]))),
    ], ids=lambda v: v if isinstance(v, str) else "")
def test_binding_refuses(host, name, call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("name,call,status", [
    ("W=5", lambda: B.conv_fwd(X, torch.zeros(8, 5)), UNS), ("W=1", lambda: B.conv_bwd(X, X, torch.zeros(8, 1)), UNS),
    ("W=9", lambda: B.conv_decode(X, torch.zeros(2, 8, 8), torch.zeros(8, 9)), UNS),
    ("in place", lambda: B.conv_fwd(X, W8, y=X), INV),
    ("R>D", lambda: B.rotary(X[None], None, torch.zeros(5).double()), INV),
    ("no frequency", lambda: B.rotary(X[None], None, torch.zeros(0).double()), INV),
    ("cu with two rows", lambda: B.linrec_fwd(X, X, cu_seqlens=torch.zeros(2, dtype=I32)), INV)],
    ids=lambda v: v if isinstance(v, str) else "")
def test_refusals_keep_the_library_s_status(host, name, call, status):
    with pytest.raises(B.GdpError) as e:
        call()
    assert e.value.status == status, str(e.value)
    assert "workspace" not in str(e.value)


def test_rotary_freq():
    f, s = B.rotary_freq(64)
    assert s == 1.0 and f.dtype == torch.float64 and f.shape == (32,)
    assert torch.allclose(f, torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64), rtol=1e-14)
    lin, s = B.rotary_freq(64, scaling="linear", factor=4.0)
    assert torch.equal(lin, f / 4) and s == 1.0
    base, _ = B.rotary_freq(64, scaling="base", factor=4.0)
    assert base[0] == f[0] and abs(float(base[-1] * 4 / f[-1]) - 1) < 1e-12 and (base <= f).all()
    part, s = B.rotary_freq(128, scaling="parts", factor=8.0, original_length=4096)
    whole, _ = B.rotary_freq(128)
    turns = whole * 4096 / (2 * math.pi)
    assert torch.equal(part[turns > 40], whole[turns > 40]) and torch.allclose(part[turns < 0.8], whole[turns < 0.8] / 8)
    assert (part <= whole).all() and (part >= whole / 8 * (1 - 1e-12)).all() and abs(s - (0.1 * math.log(8) + 1)) < 1e-15
    assert B.rotary_freq(2, scaling="base", factor=2.0)[0].tolist() == [1.0]
    for bad in (dict(rotated=3), dict(rotated=0), dict(rotated=8, base=0.0), dict(rotated=8, factor=0.5),
                dict(rotated=8, scaling="other"), dict(rotated=8, scaling="parts"),
                dict(rotated=8, scaling="parts", original_length=64, fast=1.0, slow=2.0),
                dict(rotated=8, scaling="parts", original_length=64, base=1.0)):
        with pytest.raises(ValueError):
            B.rotary_freq(**bad)


# ------------------------------------------------------------------ the tests' own plain forms

@pytest.mark.parametrize("decay", ["log", "sigmoid"])
@pytest.mark.parametrize("comp", [False, True])
def test_plain_recurrence_and_its_gradients(decay, comp):
    gen = torch.Generator().manual_seed(1)
    T, C, seqs = 17, 3, [(0, 5), (5, 5), (6, 17)]
    x, g, h0, dy, dht = (torch.randn(*s, generator=gen).double() for s in ((T, C), (T, C), (3, C), (T, C), (3, C)))
    g = -g.abs() if decay == "log" else g
    leaves = [t.clone().requires_grad_() for t in (x, g, h0)]
    total, y, ht = 0.0, torch.zeros(T, C).double(), []
    for i, (b, e) in enumerate(seqs):
        h = leaves[2][i]
        for t in range(b, e):
            a = torch.exp(leaves[1][t]) if decay == "log" else torch.sigmoid(leaves[1][t])
            h = a * h + ((1 - a) if comp else 1) * leaves[0][t]
            y[t] = h.detach()
            total = total + (h * dy[t]).sum()
        total = total + (h * dht[i]).sum()
        ht.append(h.detach())
    r = Rec(x, g, seqs, decay, comp, h0)
    assert torch.allclose(r.h, y, atol=1e-12) and torch.allclose(r.ht, torch.stack(ht), atol=1e-12)
    for (p, _), q in zip(r.backward(dy, dht), torch.autograd.grad(total, leaves)):
        assert torch.allclose(p, q, atol=1e-11)


@pytest.mark.parametrize("act", ["silu", "sigmoid", "none"])
def test_plain_convolution_and_its_gradients(act):
    gen = torch.Generator().manual_seed(2)
    T, C, W, seqs = 17, 3, 4, [(0, 2), (2, 2), (3, 17)]
    x, w, b, h0, dy, dht = (torch.randn(*s, generator=gen).double()
                            for s in ((T, C), (C, W), (C,), (3, W - 1, C), (T, C), (3, W - 1, C)))
    leaves = [t.clone().requires_grad_() for t in (x, w, b, h0)]
    total, y = 0.0, torch.zeros(T, C).double()
    for i, (s, e) in enumerate(seqs):
        full = torch.cat([leaves[3][i], leaves[0][s:e]])
        if e > s:
            u = torch.nn.functional.conv1d(full.T[None], leaves[1][:, None], leaves[2], groups=C)[0].T
            v = u if act == "none" else torch.nn.functional.silu(u) if act == "silu" else torch.sigmoid(u)
            y[s:e] = v.detach()
            total = total + (v * dy[s:e]).sum()
        total = total + (full[full.shape[0] - 3:] * dht[i]).sum()
    r = Conv(x, w, b, seqs, act, h0)
    keep = torch.ones(T, dtype=torch.bool)
    keep[2] = False
    assert torch.allclose(r.y[keep], y[keep], atol=1e-12)
    for (p, _), q in zip(r.backward(dy, dht), torch.autograd.grad(total, leaves)):
        assert torch.allclose(p, q, atol=1e-11)


def test_plain_rotation_is_one():
    gen = torch.Generator().manual_seed(3)
    x, pos = torch.randn(9, 2, 12, generator=gen), torch.arange(9) * 1000
    freq, _ = B.rotary_freq(8)
    for inter in (False, True):
        y, _ = rotate(x, pos, freq, inter)
        assert torch.equal(y[..., 8:], x[..., 8:].double())
        pairs = (lambda t: t[..., :8].unflatten(-1, (4, 2))) if inter else (lambda t: t[..., :8].unflatten(-1, (2, 4)).transpose(-1, -2))  # noqa: E731
        z = torch.view_as_complex(pairs(x.double()).contiguous()) * torch.polar(torch.ones(9, 4).double(), pos[:, None] * freq)[:, None]
        assert torch.allclose(pairs(y), torch.view_as_real(z), atol=1e-9)
        assert torch.allclose(rotate(y, pos, freq, inter, inverse=True)[0], x.double(), atol=1e-9)
