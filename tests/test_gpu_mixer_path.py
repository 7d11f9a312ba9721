"""The operators around the mixers as a layer runs them: a projection's slices
through the short convolution, then rotary positions and linear attention, the
gated recurrence, or the prepare step and the gated delta product, then the norm
with its gate; a packed prompt, the steps that continue it, and the gradients."""
import math

import pytest
import torch

from gated_delta_product_amd import binding as G
from mixref import act, half_step
from linref import group_norm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
LENS = [37, 1, 140]


def near(a, b, steps, floor):
    """Equal but for so many roundings to their type, and a floor of the sums' own."""
    a, b = a.double(), b.double()
    bad = (a - b).abs() - 2 * steps * half_step(BF16) * torch.maximum(a.abs(), b.abs()) - floor
    assert torch.isfinite(a).all() and torch.isfinite(b).all()
    assert float(bad.max()) <= 0, float(bad.max())


def prompt_and_steps(C, W=4):
    """Rows of three requests and their last token apart: (rows, cu, prompt rows, cu, last rows)."""
    gen = torch.Generator().manual_seed(C)
    x = torch.randn(1, sum(LENS), C, generator=gen).to(BF16).to(DEV)
    cu = torch.tensor([0] + LENS, device=DEV).cumsum(0).to(torch.int32)
    last = (cu[1:] - 1).long()
    keep = torch.ones(sum(LENS), dtype=torch.bool, device=DEV)
    keep[last] = False
    short = torch.tensor([0] + [n - 1 for n in LENS], device=DEV).cumsum(0).to(torch.int32)
    return x, cu, x[:, keep], short, last, x[0, last][:, None]


def test_recurrence_layer():
    """conv -> gated recurrence -> norm with gate: a prompt at once, or all but its last tokens and then those by a
    step over the pools that the prompt filled."""
    C, heads = 192, 3
    x, cu, px, pcu, last, sx = prompt_and_steps(4 * C)
    gen = torch.Generator().manual_seed(1)
    w, b = 0.5 * torch.randn(C, 4, generator=gen).to(DEV), 0.1 * torch.randn(C, generator=gen).to(DEV)
    nw = torch.rand(C, generator=gen).to(DEV) + 0.5

    def layer(p, cu=None, states=None, slots=None):
        u, r, z = p[..., :C], p[..., C:2 * C], p[..., 2 * C:3 * C]  # slices of the projection
        if states is None:
            c, cs = G.conv_fwd(u, w, b, cu_seqlens=cu, output_final_state=True)
            h, hs = G.linrec_fwd(c, r, decay="sigmoid", complement=True, cu_seqlens=cu, output_final_state=True)
        else:
            cs, hs = states
            c = G.conv_decode(u, cs, w, b, slots=slots)
            h = G.linrec_decode(c, r, hs, decay="sigmoid", complement=True, slots=slots)
        return G.group_norm_fwd(h, heads, nw, gate=z), (cs, hs), h

    y, (cs, hs), h = layer(x, cu)
    py, (pcs, phs), _ = layer(px, pcu)
    pool_c, pool_h = torch.zeros(6, 3, C, dtype=BF16, device=DEV), torch.zeros(6, C, device=DEV)
    slots = torch.tensor([4, 0, 3], dtype=torch.int32, device=DEV)
    pool_c[slots.long()], pool_h[slots.long()] = pcs, phs
    pad = torch.tensor([4, -1, 0, 3], dtype=torch.int32, device=DEV)
    sx = torch.cat([sx[:1], torch.full_like(sx[:1], 5.0), sx[1:]])
    sy, _, sh = layer(sx, states=(pool_c, pool_h), slots=pad)
    assert torch.equal(pool_c[slots.long()], cs), "the convolution's states are copies"
    # states: the same steps in another order of the sums, a few 2^-24 of a thousand
    assert ((pool_h[slots.long()] - hs).abs() <= 2.0 ** -16 * hs.abs().clamp(min=1)).all()
    live = torch.tensor([0, 2, 3], device=DEV)
    near(sh[live][:, 0], h[0, last], 2, 2.0 ** -16)
    # a norm of rows that differ by a rounding: that of each row, and the group's through its variance
    near(sy[live][:, 0], y[0, last], 6, 2.0 ** -7)
    assert not sh[1].any() and not pool_h[[1, 2, 5]].any()


def test_rotary_attention_layer():
    """conv -> rotary positions in place -> linear attention with fixed decays -> norm."""
    H, HV, K, V = 2, 4, 64, 64
    C = 2 * H * K + HV * V
    x, cu, px, pcu, last, sx = prompt_and_steps(C)
    gen = torch.Generator().manual_seed(2)
    w = 0.5 * torch.randn(C, 4, generator=gen).to(DEV)
    g = torch.log1p(-torch.exp2(-2.0 - torch.arange(HV) * 1.0)).to(DEV)
    freq, scale = G.rotary_freq(32, scaling="parts", factor=4.0, original_length=64, device=DEV)

    def split(c):
        q, k, v = c[..., :H * K], c[..., H * K:2 * H * K], c[..., 2 * H * K:]
        return q.unflatten(-1, (H, K)), k.unflatten(-1, (H, K)), v.unflatten(-1, (HV, V))

    def prompt(x, cu):
        c, cs = G.conv_fwd(x, w, cu_seqlens=cu, output_final_state=True)
        q, k, v = split(c)
        G.rotary(q, k, freq, cu_seqlens=cu, scale=scale, out=(q, k))
        o, ht = G.linattn_fwd(q, k, v, g, cu_seqlens=cu, output_final_state=True)
        return o, cs, ht

    o, cs, ht = prompt(x, cu)
    _, pcs, pht = prompt(px, pcu)
    c = G.conv_decode(sx, pcs, w)
    q, k, v = split(c)
    q, k = G.rotary(q, k, freq, positions=(torch.tensor(LENS, device=DEV) - 1).to(torch.int32)[:, None], scale=scale)
    so = G.linattn_decode(q, k, v, pht, g)
    assert torch.equal(pcs, cs)
    size = float(ht.abs().max())
    assert ((pht - ht).abs() <= 2.0 ** -14 * size).all()
    # the attention's rows carry two bf16 parts of their scores: 2^-8 of a row's size in all
    row = o[0, last].double().norm(dim=-1, keepdim=True) / math.sqrt(V)
    assert ((so[:, 0].double() - o[0, last].double()).abs() <= 2.0 ** -6 * (row + o[0, last].double().abs())).all()
    y = G.group_norm_fwd(so.flatten(2), HV, activation="none")
    assert torch.isfinite(y).all()


def test_gated_delta_product_layer():
    """conv -> prepare -> chunked forward, and the steps over the pools: the post-conv activations of both."""
    M, H, Gq, P, N = 2, 2, 1, 64, 64
    C = M * H * P + M * Gq * N + Gq * N
    x, cu, px, pcu, last, sx = prompt_and_steps(C)
    gen = torch.Generator().manual_seed(3)
    w = 0.5 * torch.randn(C, 4, generator=gen).to(DEV)
    A_log, dt = torch.rand(H, generator=gen).to(DEV), torch.randn(H, generator=gen).to(DEV) - 3
    ba = torch.randn(1, sum(LENS), M * H + H, generator=gen).to(BF16).to(DEV)
    keep = torch.ones(sum(LENS), dtype=torch.bool, device=DEV)
    keep[last] = False

    def prompt(x, ba, cu):
        c, cs = G.conv_fwd(x, w, cu_seqlens=cu, output_final_state=True)
        buf = G.chunk_fwd(*G.prefill_prepare(c, ba.contiguous(), A_log, dt, M, H, Gq, P, N), cu_seqlens=cu,
                          output_final_state=True)
        return buf.o, cs, buf.ht

    o, cs, ht = prompt(x, ba, cu)
    _, pcs, pht = prompt(px, ba[:, keep], pcu)
    c = G.conv_decode(sx, pcs, w)
    q, k, v, beta, g = G.decode_prepare(c, ba[0, last][:, None].contiguous(), A_log, dt, M, H, Gq, P, N)
    so = G.decode_update(q, k, v, beta, g, pht, M)
    assert torch.equal(pcs, cs)
    got, want = so[:, M - 1].double(), o[0, last].double()
    # the chunked form's own tolerance against the recurrence (5e-3 of the norm, 2e-2 of a value)
    assert float((got - want).norm() / want.norm()) <= 1e-2 and float((got - want).abs().max()) <= 4e-2


def test_gradients_through_a_layer():
    """norm(recurrence(conv(x))) and every gradient against the same in 64 bits, and against differences."""
    C, heads, cu = 24, 2, [0, 9, 9, 10, 50]
    gen = torch.Generator().manual_seed(4)
    T = cu[-1]
    x, r, z, dy = (torch.randn(1, T, C, generator=gen) for _ in range(4))
    w, b, nw = 0.5 * torch.randn(C, 4, generator=gen), torch.randn(C, generator=gen), torch.rand(C, generator=gen) + 0.5
    d = {n: t.to(DEV) for n, t in dict(x=x, r=r, z=z, dy=dy, w=w, b=b, nw=nw).items()}
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    how = dict(decay="sigmoid", complement=True, cu_seqlens=cud)
    c, _ = G.conv_fwd(d["x"], d["w"], d["b"], cu_seqlens=cud)
    h, _ = G.linrec_fwd(c, d["r"], **how)
    dh, dz, dnw, _ = G.group_norm_bwd(d["dy"], h, heads, d["nw"], gate=d["z"])
    dc, dr, _ = G.linrec_bwd(dh, c, d["r"], **how)
    dx, dw, db, _ = G.conv_bwd(dc, d["x"], d["w"], d["b"], cu_seqlens=cud)
    got = dict(x=dx, r=dr, z=dz, w=dw, b=db, nw=dnw)
    leaf = {n: t.double().requires_grad_() for n, t in dict(x=x, r=r, z=z, w=w, b=b, nw=nw).items()}

    def loss(a):
        rows = []
        for s, e in zip(cu[:-1], cu[1:]):
            full = torch.cat([torch.zeros(3, C, dtype=torch.float64), a["x"][0, s:e]])
            state = torch.zeros(C, dtype=torch.float64)
            for t in range(e - s):
                u = act("silu", (full[t:t + 4] * a["w"].T).sum(0) + a["b"])
                f = torch.sigmoid(a["r"][0, s + t])
                state = f * state + (1 - f) * u
                rows.append(state)
        y = group_norm(torch.stack(rows), heads, a["nw"], None, a["z"][0], "silu", True, 1e-5)
        return (y * dy[0].double()).sum()

    total = loss(leaf)
    want = dict(zip(leaf, torch.autograd.grad(total, list(leaf.values()))))
    for n in got:
        e = (got[n].cpu().double().reshape(want[n].shape) - want[n]).norm() / want[n].norm()
        assert float(e) <= 2e-5, (n, float(e))  # float32 rows between four operators
        v = torch.randn(want[n].shape, generator=gen, dtype=torch.float64)
        base = {k: t.detach() for k, t in leaf.items()}
        diff = (loss({**base, n: base[n] + 1e-5 * v}) - loss({**base, n: base[n] - 1e-5 * v})) / 2e-5
        mine = got[n].cpu().double().reshape(v.shape) * v
        assert abs(float(diff - mine.sum())) <= 1e-4 * float(mine.abs().sum()) + 1e-6, n
