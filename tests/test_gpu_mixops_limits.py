"""Offsets past 2^31 elements, long chains of tiles, the widest rows, and calls
under way together."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from mixref import Rec, worst

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def test_recurrence_of_many_tiles():
    """Odd narrow rows are cut into hundreds of tiles, more groups of them than one look holds."""
    T, C = 20000, 3
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(1, T, C, generator=gen) for _ in range(2))
    g = -torch.rand(1, T, C, generator=gen) * 2e-3
    ref = Rec(x[0], g[0], [(0, T)], "log", False)
    y, ht = G.linrec_fwd(x.to(DEV), g.to(DEV), output_final_state=True)
    assert worst("y", y, ref.h, ref.err) <= 1 and worst("ht", ht, ref.ht, ref.ht_err) <= 1
    dx, dg, _ = G.linrec_bwd(dy.to(DEV), x.to(DEV), g.to(DEV))
    rx, rg, _ = ref.backward(dy[0])
    assert worst("dx", dx, *rx) <= 1 and worst("dg", dg, *rg) <= 1


def test_past_2_31_elements():
    """A tensor of over 2^31 elements: its last columns and rows bit for bit those of a call on the slice alone."""
    T, C = 2100, 1 << 20
    x = torch.empty(1, T, C, dtype=BF16, device=DEV)
    x.normal_()
    cols = slice(C - 128, C)
    part = x[..., cols].contiguous()
    y, ht = G.linrec_fwd(x, x, decay="sigmoid", output_final_state=True)
    wy, wht = G.linrec_fwd(part, part, decay="sigmoid", output_final_state=True)
    assert torch.equal(y[..., cols], wy) and torch.equal(ht[:, cols], wht)
    dx, dg, _ = G.linrec_bwd(x, y, x, decay="sigmoid")
    wx, wg, _ = G.linrec_bwd(part, wy, part, decay="sigmoid")
    assert torch.equal(dx[..., cols], wx) and torch.equal(dg[..., cols], wg)
    del dx, dg
    w = torch.randn(C, 4, device=DEV)
    y, ht = G.conv_fwd(x, w, output_final_state=True, y=y)
    wy, wht = G.conv_fwd(part, w[cols].contiguous(), output_final_state=True)
    assert torch.equal(y[..., cols], wy) and torch.equal(ht[..., cols], wht)
    dx, dw, _, _ = G.conv_bwd(x, y, w)
    wx, ww, _, _ = G.conv_bwd(part, wy, w[cols].contiguous())
    assert torch.equal(dx[..., cols], wx) and torch.equal(dw[cols], ww)
    del dx, y
    q = x.view(1, T, C // 128, 128)
    freq = G.rotary_freq(128, device=DEV)[0]
    a, _ = G.rotary(q, None, freq)
    b, _ = G.rotary(q[:, :, -2:], None, freq)
    assert torch.equal(a[:, :, -2:], b)


def test_far_slots():
    """The last slots of pools of over 2^31 elements."""
    n, C = (1 << 31) // 4096 + 8, 4096
    state = torch.zeros(n, C, device=DEV)
    x, g = torch.randn(2, 1, C, device=DEV).to(BF16), torch.randn(2, 1, C, device=DEV).to(BF16)
    slots = torch.tensor([n - 1, n], dtype=torch.int32, device=DEV)
    y = G.linrec_decode(x, g, state, decay="sigmoid", slots=slots)
    small = torch.zeros(1, C, device=DEV)
    want = G.linrec_decode(x[:1], g[:1], small, decay="sigmoid")
    assert torch.equal(y[:1], want) and torch.equal(state[-1:], small) and not y[1].any()
    assert not state[:-1].any()
    del state
    n = n // 3 + 8
    state = torch.zeros(n, 3, C, dtype=BF16, device=DEV)
    w = torch.randn(C, 4, device=DEV)
    slots = torch.tensor([n - 1, -1], dtype=torch.int32, device=DEV)
    y = G.conv_decode(x, state, w, slots=slots)
    small = torch.zeros(1, 3, C, dtype=BF16, device=DEV)
    assert torch.equal(y[:1], G.conv_decode(x[:1], small, w)) and torch.equal(state[-1:], small) and not y[1].any()
    assert not state[:-1].any()


def test_two_calls_under_way_together():
    """Chains of two streams interleaved many times over: each keeps its own words and results."""
    T, C = 6000, 512
    xs = [torch.randn(1, T, C, device=DEV).to(BF16) for _ in range(2)]
    gs = [torch.randn(1, T, C, device=DEV).to(BF16) + 4 for _ in range(2)]
    want = [(G.linrec_fwd(x, g, decay="sigmoid")[0],) + G.linrec_bwd(x, x, g, decay="sigmoid")[:2] for x, g in zip(xs, gs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, x, g in zip(streams, xs, gs):
            with torch.cuda.stream(s):
                got.append((G.linrec_fwd(x, g, decay="sigmoid")[0],) + G.linrec_bwd(x, x, g, decay="sigmoid")[:2])
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_graphs_share_a_workspace():
    """Graphs replayed one after the other over one workspace, at the C entry: nothing in it outlives a call."""
    import ctypes
    T, C = 3000, 64
    L, out = G.lib(), []
    xs = [torch.randn(1, T, C, device=DEV) for _ in range(2)]
    gs = [-torch.rand(1, T, C, device=DEV) * 0.1 for _ in range(2)]
    ys = [torch.empty_like(x) for x in xs]
    args = [G.LinrecArgs(1, T, C, G.GDP_F32, G.GDP_F32, 0, 0, None, 1, x.data_ptr(), T * C, C, g.data_ptr(), T * C, C, None,
                         y.data_ptr(), None) for x, g, y in zip(xs, gs, ys)]
    need = L.gdp_linrec_workspace_bytes(ctypes.byref(args[0]), 0)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    for a in args:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            G._check(L.gdp_linrec_fwd(ctypes.byref(a), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream))
        out.append(graph)
    for k in range(4):
        for x in xs:
            x.normal_()
        for graph in out:
            graph.replay()
        torch.cuda.synchronize()
        for x, g, y in zip(xs, gs, ys):
            assert torch.equal(G.linrec_fwd(x, g)[0], y), k
