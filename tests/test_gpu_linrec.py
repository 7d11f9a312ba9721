"""Gated linear recurrence on the GPU against its plain 64-bit form
(mixref.Rec), whose bounds the tolerances are."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from helpers import log
from mixref import Rec, spans, worst

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
KINDS = [("log", False), ("log", True), ("sigmoid", False), ("sigmoid", True)]
TYPES = [(BF16, BF16), (BF16, F32), (F32, F32)]


def gpu(t):
    return None if t is None else t.to(DEV)


def draw(B, T, C, dtype, gtype, decay, nseq, seed, h0=True, slow=False):
    gen = torch.Generator().manual_seed(seed)
    x, dy = (torch.randn(B, T, C, generator=gen).to(dtype) for _ in range(2))
    if decay == "log":
        g = -torch.rand(B, T, C, generator=gen) * torch.exp(torch.randn(C, generator=gen) * 2 - (7 if slow else 1))
    else:
        g = torch.randn(B, T, C, generator=gen) + 3 * torch.rand(C, generator=gen) + (6 if slow else 0)
    s, e = (torch.randn(nseq, C, generator=gen) if h0 else None for _ in range(2))
    return x, g.to(gtype), dy, s, e


def check(name, got, want, err):
    w = worst(name, got, want, err)
    log("  %-4s worst error / bound = %.3f" % (name, w))
    assert w <= 1.0, (name, w)


def run(B, T, C, dtype, gtype, decay, comp, seed, cu=None, h0=True, slow=False):
    seqs = spans(B * T, cu, B)
    x, g, dy, s0, dht = draw(B, T, C, dtype, gtype, decay, len(seqs), seed, h0, slow)
    log("linrec B=%d T=%d C=%d %s/%s %s comp=%s cu=%s seed=%d" % (B, T, C, dtype, gtype, decay, comp, cu, seed))
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    how = dict(decay=decay, complement=comp, cu_seqlens=cud, initial_state=gpu(s0))
    mark = torch.full((B, T, C), 77.0, dtype=dtype, device=DEV)
    y, ht = G.linrec_fwd(gpu(x), gpu(g), output_final_state=True, y=mark, **how)
    dx, dg, dh0 = G.linrec_bwd(gpu(dy), gpu(x), gpu(g), dht=gpu(dht), **how)
    torch.cuda.synchronize()
    ref = Rec(x.view(-1, C), g.view(-1, C), seqs, decay, comp, s0)
    out = ~ref.inside
    y = y.cpu().view(-1, C)
    assert (y[out] == 77).all(), "rows outside every request"
    check("y", y[ref.inside], ref.h[ref.inside], ref.err[ref.inside])
    check("ht", ht, ref.ht, ref.ht_err)
    rx, rg, r0 = ref.backward(dy.view(-1, C), dht)
    for t in (dx, dg):
        assert not t.cpu().view(-1, C)[out].any()
    check("dx", dx, *rx)
    check("dg", dg, *rg)
    if h0:
        check("dh0", dh0, *r0)
    else:
        assert dh0 is None


@pytest.mark.parametrize("decay,comp", KINDS)
@pytest.mark.parametrize("dtype,gtype", TYPES, ids=["bf16", "bf16-f32", "f32"])
@pytest.mark.parametrize("B,T,C", [(1, 1, 1), (1, 3, 8), (2, 65, 7), (1, 130, 64), (3, 200, 130), (2, 513, 24), (70, 1, 40)])
def test_rows(B, T, C, dtype, gtype, decay, comp):
    run(B, T, C, dtype, gtype, decay, comp, 13 * T + C, h0=(T + C) % 2 == 0)


@pytest.mark.parametrize("decay,comp", KINDS)
@pytest.mark.parametrize("dtype,gtype", TYPES, ids=["bf16", "bf16-f32", "f32"])
@pytest.mark.parametrize("T,C,cu", [
    (300, 48, [0, 1, 1, 3, 64, 64, 64, 191, 300]),  # empty ones, one row, borders inside and between tiles
    (260, 9, [5, 5, 133, 200, 250]),                # rows before, and behind the last
    (140, 136, [0, 0, 0, 140, 140]),
    (70, 16, [0] + list(range(1, 71))),             # requests of one row
    (40, 32, [7, 7]), (33, 8, [0])])                # none with rows, none at all
def test_packed(T, C, cu, dtype, gtype, decay, comp):
    run(1, T, C, dtype, gtype, decay, comp, 7 * T + C, cu=cu, h0=len(cu) > 1)


@pytest.mark.parametrize("decay,comp", KINDS)
@pytest.mark.parametrize("dtype,gtype,C", [(BF16, BF16, 40), (F32, F32, 20), (BF16, F32, 5)])
def test_many_tiles(dtype, gtype, C, decay, comp):
    """Thousands of rows, channels that remember hundreds of them, several requests among the tiles."""
    run(1, 5000, C, dtype, gtype, decay, comp, 3, slow=True)
    run(1, 4099, C, dtype, gtype, decay, comp, 4, cu=[0, 2900, 2900, 3011, 4090], slow=True)


def test_padded_cu_and_many_requests():
    """More requests than a wave looks through at once; offsets past the end and below zero are clamped."""
    gen = torch.Generator().manual_seed(5)
    cu = [0] + torch.randint(0, 4, (5000,), generator=gen).cumsum(0).tolist()
    run(1, cu[-1] - 40, 24, BF16, BF16, "sigmoid", True, 5, cu=cu)
    run(1, 50, 8, F32, F32, "log", False, 6, cu=[-4, 20, 45, 90])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_strides_and_in_place(dtype):
    """Slices of a wider projection, aligned or not, a broadcast g, and outputs on top of inputs."""
    B, T, C = 2, 150, 64
    x, g, dy, s0, dht = draw(B, T, C, dtype, dtype, "sigmoid", B, 21)
    how = dict(decay="sigmoid", complement=True, initial_state=gpu(s0))
    want, wht = G.linrec_fwd(gpu(x), gpu(g), output_final_state=True, **how)
    wb = G.linrec_bwd(gpu(dy), gpu(x), gpu(g), dht=gpu(dht), **how)
    ref = Rec(x.view(-1, C), g.view(-1, C), spans(B * T, None, B), "sigmoid", True, s0)
    for off in (8, 3):
        wide = torch.zeros(B, T + 4, 3 * C + 16, dtype=dtype, device=DEV)
        xs, gs, ds = (wide[:, 2:T + 2, off + i * C:off + (i + 1) * C] for i in range(3))
        xs.copy_(gpu(x))
        gs.copy_(gpu(g))
        ds.copy_(gpu(dy))
        y, ht = G.linrec_fwd(xs, gs, output_final_state=True, **how)
        b = G.linrec_bwd(ds, xs, gs, dht=gpu(dht), **how)
        if off == 8:
            assert torch.equal(y, want) and torch.equal(ht, wht)
            assert all(torch.equal(p, q) for p, q in zip(b, wb))
        else:
            check("y", y, ref.h, ref.err)
            rx, rg, r0 = ref.backward(dy.view(-1, C), dht)
            check("dx", b[0], *rx)
            check("dg", b[1], *rg)
            check("dh0", b[2], *r0)
    one = gpu(g)[:, :1].expand(B, T, C)  # every token the same decay, by a stride of zero
    y, _ = G.linrec_fwd(gpu(x), one, **how)
    assert torch.equal(y, G.linrec_fwd(gpu(x), one.contiguous(), **how)[0])
    a, b = G.linrec_bwd(gpu(dy), gpu(x), one, **how), G.linrec_bwd(gpu(dy), gpu(x), one.contiguous(), **how)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    for i in range(2):
        pair = [gpu(x).clone(), gpu(g).clone()]
        G.linrec_fwd(*pair, y=pair[i], **how)
        assert torch.equal(pair[i], want)


def test_a_row_cut_in_two():
    """The states of the first part continue in the second: the whole, to its bound."""
    T, C = 700, 72
    x, g, _, s0, _ = draw(1, T, C, BF16, BF16, "log", 1, 8, slow=True)
    ref = Rec(x[0], g[0], [(0, T)], "log", False, s0)
    a, h = G.linrec_fwd(gpu(x)[:, :333], gpu(g)[:, :333], initial_state=gpu(s0), output_final_state=True)
    b, h2 = G.linrec_fwd(gpu(x)[:, 333:], gpu(g)[:, 333:], initial_state=h, output_final_state=True)
    check("y", torch.cat([a, b], 1)[0], ref.h, ref.err)
    check("ht", h2, ref.ht, 2 * ref.ht_err)


def test_rows_far_apart():
    """A narrow slice of very wide rows, rows of one token each, and states off 16 bytes."""
    T, C = 300, 64
    x, g, dy, s0, dht = draw(1, T, C, BF16, BF16, "sigmoid", 1, 22)
    how = dict(decay="sigmoid", initial_state=gpu(s0))
    want = G.linrec_fwd(gpu(x), gpu(g), output_final_state=True, **how) + G.linrec_bwd(gpu(dy), gpu(x), gpu(g), **how)
    wide = torch.zeros(1, T, (1 << 20) + 1000 * C, dtype=BF16, device=DEV)
    xs = wide[..., 64:64 + C]
    xs.copy_(gpu(x))
    got = G.linrec_fwd(xs, gpu(g), output_final_state=True, **how) + G.linrec_bwd(gpu(dy), xs, gpu(g), **how)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    off = torch.zeros(C + 1, device=DEV)[1:].view(1, C)
    off.copy_(gpu(s0))
    got = G.linrec_fwd(gpu(x), gpu(g), decay="sigmoid", initial_state=off, output_final_state=True)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    many = torch.zeros(T, 2, C, dtype=BF16, device=DEV)[:, :1]  # T batch rows of a token, two tokens apart
    many.copy_(gpu(x).view(T, 1, C))
    s = torch.randn(T, C, device=DEV)
    gs = gpu(g).view(T, 1, C)
    a = G.linrec_fwd(many, gs, decay="sigmoid", initial_state=s, output_final_state=True)
    b = G.linrec_fwd(many.contiguous(), gs, decay="sigmoid", initial_state=s, output_final_state=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    d = G.linrec_decode(many, gs, s, decay="sigmoid")
    assert torch.equal(a[0], d) and torch.equal(a[1], s)


def test_nothing_of_other_requests_and_gaps():
    """NaN and infinities in other requests and in rows outside every one change nothing."""
    T, C, cu = 400, 40, [10, 140, 150, 390]
    x, g, dy, s0, dht = draw(1, T, C, F32, F32, "log", 3, 9)
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    how = dict(cu_seqlens=cud, initial_state=gpu(s0))

    def call(x, g, dy):
        y, ht = G.linrec_fwd(gpu(x), gpu(g), output_final_state=True, y=torch.zeros(1, T, C, device=DEV), **how)
        return (y, ht) + G.linrec_bwd(gpu(dy), gpu(x), gpu(g), dht=gpu(dht), **how)

    want = call(x, g, dy)
    bad = [t.clone() for t in (x, g, dy)]
    for t, v in zip(bad, (float("nan"), float("nan"), float("inf"))):
        t[:, :10] = v
        t[:, 390:] = v
        t[:, 140:150] = v  # the second request
    got = call(*bad)
    for i, (p, q) in enumerate(zip(want, got)):
        if i in (1, 4):
            p, q = p[[0, 2]], q[[0, 2]]
        else:
            p, q = (torch.cat([t[:, :140], t[:, 150:]], 1) for t in (p, q))
        assert torch.equal(p, q), i


def test_decays_at_the_ends():
    """A log decay of -inf drops the state, 0 keeps it; gates far out are 0 and 1; their gradients are finite."""
    T, C = 300, 16
    x, _, dy, s0, _ = draw(1, T, C, F32, F32, "log", 1, 10)
    g = torch.zeros(1, T, C)
    g[:, 150] = -float("inf")
    y, _ = G.linrec_fwd(gpu(x), gpu(g), initial_state=gpu(s0))
    ref = Rec(x[0], g[0], [(0, T)], "log", False, s0)
    check("y", y, ref.h, ref.err)
    assert torch.equal(y.cpu()[0, 150], x[0, 150])
    dx, dg, dh0 = G.linrec_bwd(gpu(dy), gpu(x), gpu(g), initial_state=gpu(s0))
    rx, rg, r0 = ref.backward(dy[0])
    check("dx", dx, *rx)
    check("dg", dg, *rg)
    check("dh0", dh0, *r0)
    assert not dg.cpu()[0, 150].any()
    g = torch.where(torch.arange(T)[:, None] % 3 == 0, -200.0, 300.0).expand(1, T, C).contiguous()
    for comp in (False, True):
        y, _ = G.linrec_fwd(gpu(x), gpu(g), decay="sigmoid", complement=comp, initial_state=gpu(s0))
        ref = Rec(x[0], g[0], [(0, T)], "sigmoid", comp, s0)
        check("y", y, ref.h, ref.err)
        assert all(torch.isfinite(t).all() for t in G.linrec_bwd(gpu(dy), gpu(x), gpu(g), decay="sigmoid",
                                                                 complement=comp, initial_state=gpu(s0)))


@pytest.mark.parametrize("decay,comp", KINDS)
def test_gradient_against_differences(decay, comp):
    T, C, cu = 37, 5, [0, 11, 11, 37]
    x, g, dy, s0, dht = draw(1, T, C, F32, F32, decay, 3, 31)
    args = dict(x=x[0].double(), g=g[0].double(), h=s0.double())
    seqs = spans(T, cu)
    grads = G.linrec_bwd(gpu(dy), gpu(x), gpu(g), decay=decay, complement=comp, initial_state=gpu(s0), dht=gpu(dht),
                         cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))

    def loss(a):
        r = Rec(a["x"], a["g"], seqs, decay, comp, a["h"])
        return float((r.h * dy[0].double()).sum() + (r.ht * dht.double()).sum())

    gen = torch.Generator().manual_seed(32)
    for name, grad in zip(("x", "g", "h"), grads):
        u = torch.randn(args[name].shape, generator=gen, dtype=torch.float64)
        want = (loss({**args, name: args[name] + 1e-5 * u}) - loss({**args, name: args[name] - 1e-5 * u})) / 2e-5
        got = grad.cpu().double().reshape(u.shape) * u
        # float32 gradients, and differences of 1e-10 (their third-order term) and 1e-16 / 1e-5
        assert abs(want - float(got.sum())) <= 1e-5 * float(got.abs().sum()) + 1e-7, name


@pytest.mark.parametrize("dtype,gtype", TYPES, ids=["bf16", "bf16-f32", "f32"])
@pytest.mark.parametrize("n,S,C,pad", [(1, 1, 64, 0), (5, 1, 40, 2), (3, 4, 7, 1), (300, 1, 136, 7)])
def test_decode(n, S, C, pad, dtype, gtype):
    for decay, comp in KINDS:
        x, g, _, _, _ = draw(n, S, C, dtype, gtype, decay, n, 17 * n + C)
        gen = torch.Generator().manual_seed(n)
        pool = n + 2
        slots = torch.randperm(pool, generator=gen)[:n].to(torch.int32)
        slots[:pad] = torch.tensor([-1, pool, 2 ** 31 - 1, -2 ** 31, -1, -1, pool + 5])[:pad].to(torch.int32)
        state = torch.randn(pool, C, generator=gen)
        st = gpu(state).clone()
        y = G.linrec_decode(gpu(x), gpu(g), st, decay=decay, complement=comp, slots=gpu(slots)).cpu()
        assert not y[:pad].any()
        seen = state.clone()
        for i in range(pad, n):
            ref = Rec(x[i], g[i], [(0, S)], decay, comp, state[slots[i].item()][None])
            check("y", y[i], ref.h, ref.err)
            check("h", st[slots[i].item()], ref.ht[0], ref.ht_err[0])
            seen[slots[i].item()] = st[slots[i].item()].cpu()
        assert torch.equal(seen, st.cpu()), "slots of no request"
        xs = torch.zeros(n, S, C + 5, dtype=dtype, device=DEV)[..., 3:C + 3]
        xs.copy_(gpu(x))
        st2 = gpu(state).clone()
        y2 = G.linrec_decode(xs, gpu(g), st2, decay=decay, complement=comp, slots=gpu(slots))
        assert torch.equal(y2.cpu(), y) and torch.equal(st2, st)


def test_streams_graph_and_repeats():
    """Bit for bit the same on another stream, from two streams at once, and replayed from a graph."""
    T, C, cu = 3000, 200, [0, 700, 1500, 2990]
    x, g, dy, s0, dht = (gpu(t) for t in draw(1, T, C, BF16, BF16, "sigmoid", 3, 12))
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    how = dict(decay="sigmoid", complement=True, cu_seqlens=cud, initial_state=s0)
    outs = [torch.zeros_like(x) for _ in range(3)]

    def step(i=0):
        y, ht = G.linrec_fwd(x, g, output_final_state=True, y=outs[i], **how)
        return (y, ht) + G.linrec_bwd(dy, x, g, dht=dht, **how)

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            for _ in range(3):
                r = step(i + 1)
            got.append(r)
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(p, q) for p, q in zip(want, r))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(1)
    for k in range(4):
        x.copy_(torch.randn(x.shape, device=DEV))
        dy.copy_(torch.randn(x.shape, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        want = step(2)
        assert all(torch.equal(p, q) for p, q in zip(want, got)), k
