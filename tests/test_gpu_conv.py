"""Short causal convolution on the GPU against its plain 64-bit form
(mixref.Conv), whose bounds the tolerances are."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from helpers import log
from mixref import Conv, spans, worst

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def gpu(t):
    return None if t is None else t.to(DEV)


def draw(B, T, C, W, dtype, nseq, seed, h0=True, bias=True):
    gen = torch.Generator().manual_seed(seed)
    x, dy = (torch.randn(B, T, C, generator=gen).to(dtype) for _ in range(2))
    w, b = 0.6 * torch.randn(C, W, generator=gen), torch.randn(C, generator=gen) if bias else None
    s, e = (torch.randn(nseq, W - 1, C, generator=gen).to(dtype) if h0 else None for _ in range(2))
    return x, dy, w, b, s, e


def check(name, got, want, err):
    r = worst(name, got, want, err)
    log("  %-4s worst error / bound = %.3f" % (name, r))
    assert r <= 1.0, (name, r)


def run(B, T, C, W, dtype, act, seed, cu=None, h0=True, bias=True):
    seqs = spans(B * T, cu, B)
    x, dy, w, b, s0, dht = draw(B, T, C, W, dtype, len(seqs), seed, h0, bias)
    log("conv B=%d T=%d C=%d W=%d %s %s cu=%s seed=%d" % (B, T, C, W, dtype, act, cu, seed))
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    how = dict(activation=act, cu_seqlens=cud, initial_state=gpu(s0))
    mark = torch.full((B, T, C), 77.0, dtype=dtype, device=DEV)
    y, ht = G.conv_fwd(gpu(x), gpu(w), gpu(b), output_final_state=True, y=mark, **how)
    dx, dw, db, dh0 = G.conv_bwd(gpu(dy), gpu(x), gpu(w), gpu(b), dht=gpu(dht), **how)
    torch.cuda.synchronize()
    ref = Conv(x.view(-1, C), w, b, seqs, act, s0)
    out = torch.ones(B * T, dtype=torch.bool)
    for a, e in seqs:
        out[a:e] = False
    y = y.cpu().view(-1, C)
    assert (y[out] == 77).all(), "rows outside every request"
    check("y", y[~out], ref.y[~out], ref.y_err[~out])
    assert torch.equal(ht.cpu().double(), ref.ht), "states are copies"
    rx, rw, rb, r0 = ref.backward(dy.view(-1, C), dht)
    assert not dx.cpu().view(-1, C)[out].any()
    check("dx", dx, *rx)
    check("dw", dw, *rw)
    if bias:
        check("db", db, *rb)
    else:
        assert db is None
    if h0:
        check("dh0", dh0, *r0)
    else:
        assert dh0 is None


@pytest.mark.parametrize("act", ["silu", "sigmoid", "none"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,C", [(1, 1, 1), (1, 2, 8), (2, 3, 7), (1, 130, 64), (3, 67, 130), (70, 1, 40), (2, 400, 24)])
def test_rows(B, T, C, W, dtype, act):
    run(B, T, C, W, dtype, act, 13 * T + C + W, h0=(T + C) % 2 == 0, bias=C % 3 > 0)


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T,C,cu", [
    (300, 48, [0, 1, 1, 3, 64, 64, 64, 66, 300]),   # empty ones, one to three rows, borders inside and between tiles
    (260, 9, [5, 5, 133, 200, 250]),                # rows before, and behind the last
    (140, 520, [0, 0, 0, 140, 140]),
    (70, 16, [0] + list(range(1, 71))),             # requests of one row
    (71, 8, [0] + list(range(2, 71, 2))),           # of two
    (40, 32, [7, 7]), (33, 8, [0])])                # none with rows, none at all
def test_packed(T, C, cu, W, dtype, act):
    run(1, T, C, W, dtype, act, 7 * T + C, cu=cu, h0=len(cu) > 1)


@pytest.mark.parametrize("dtype,C", [(BF16, 24), (F32, 5), (BF16, 1032)])
def test_many_tiles(dtype, C):
    run(1, 5000, C, 4, dtype, "silu", 3)
    gen = torch.Generator().manual_seed(5)
    cu = [0] + torch.randint(0, 5, (1500,), generator=gen).cumsum(0).tolist()
    run(1, cu[-1] - 40, C, 4, dtype, "silu", 4, cu=cu)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_strides(dtype):
    """Slices of a wider projection, aligned or not, and a row that every token shares."""
    B, T, C, W = 2, 150, 64, 4
    x, dy, w, b, s0, dht = draw(B, T, C, W, dtype, B, 21)
    how = dict(initial_state=gpu(s0))
    want = G.conv_fwd(gpu(x), gpu(w), gpu(b), output_final_state=True, **how)
    wb = G.conv_bwd(gpu(dy), gpu(x), gpu(w), gpu(b), dht=gpu(dht), **how)
    ref = Conv(x.view(-1, C), w, b, spans(B * T, None, B), "silu", s0)
    for off in (8, 3):
        wide = torch.zeros(B, T + 4, 2 * C + 16, dtype=dtype, device=DEV)
        xs, ds = (wide[:, 2:T + 2, off + i * C:off + (i + 1) * C] for i in range(2))
        xs.copy_(gpu(x))
        ds.copy_(gpu(dy))
        got = G.conv_fwd(xs, gpu(w), gpu(b), output_final_state=True, **how)
        gb = G.conv_bwd(ds, xs, gpu(w), gpu(b), dht=gpu(dht), **how)
        assert all(torch.equal(p, q) for p, q in zip(want, got))
        if off == 8:
            assert all(torch.equal(p, q) for p, q in zip(wb, gb))
        else:
            for name, g, r in zip(("dx", "dw", "db", "dh0"), gb, ref.backward(dy.view(-1, C), dht)):
                check(name, g, *r)
    one = gpu(x)[:, :1].expand(B, T, C)
    assert torch.equal(G.conv_fwd(one, gpu(w), gpu(b))[0], G.conv_fwd(one.contiguous(), gpu(w), gpu(b))[0])


def test_rows_far_apart_and_taps_off_16_bytes():
    T, C = 1100, 64
    x, dy, w, b, s0, dht = draw(1, T, C, 4, BF16, 1, 23)
    how = dict(initial_state=gpu(s0))
    want = G.conv_fwd(gpu(x), gpu(w), gpu(b), output_final_state=True, **how) + G.conv_bwd(gpu(dy), gpu(x), gpu(w), gpu(b), **how)
    wide = torch.zeros(1, T, 280000, dtype=BF16, device=DEV)
    xs = wide[..., 64:64 + C]
    xs.copy_(gpu(x))
    wo = torch.zeros(4 * C + 1, device=DEV)[1:].view(C, 4)
    bo = torch.zeros(C + 1, device=DEV)[1:]
    wo.copy_(gpu(w))
    bo.copy_(gpu(b))
    got = G.conv_fwd(xs, wo, bo, output_final_state=True, **how) + G.conv_bwd(gpu(dy), xs, wo, bo, **how)
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_nothing_of_other_requests_and_gaps():
    T, C, cu = 400, 40, [10, 140, 150, 390]
    x, dy, w, b, s0, dht = draw(1, T, C, 4, F32, 3, 9)
    how = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), initial_state=gpu(s0))

    def call(x, dy):
        y, ht = G.conv_fwd(gpu(x), gpu(w), gpu(b), output_final_state=True, y=torch.zeros(1, T, C, device=DEV), **how)
        dx, dw, db, dh0 = G.conv_bwd(gpu(dy), gpu(x), gpu(w), gpu(b), dht=gpu(dht), **how)
        return y, ht, dx, dh0, dw, db

    want = call(x, dy)
    bad = [x.clone(), dy.clone()]
    for t, v in zip(bad, (float("nan"), float("inf"))):
        t[:, :10] = v
        t[:, 390:] = v
    got = call(*bad)
    assert all(torch.equal(p, q) for p, q in zip(want, got)), "rows outside every request"
    for t in bad:
        t[:, 140:150] = float("nan")  # the second request
    got = call(*bad)
    for i, (p, q) in enumerate(zip(want[:4], got)):
        if i in (1, 3):
            p, q = p[[0, 2]], q[[0, 2]]
        else:
            p, q = (torch.cat([t[:, :140], t[:, 150:]], 1) for t in (p, q))
        assert torch.equal(p, q), i


def test_activations_far_out():
    """Sums far out on both sides: outputs and slopes at their limits, nothing that is not a number."""
    x = torch.tensor([-3e4, -200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 200.0, 3e4]).repeat_interleave(4)[None, :, None]
    x = x.expand(1, 36, 4).contiguous()
    w = torch.zeros(4, 2)
    w[:, 1] = 1.0
    for act in ("silu", "sigmoid", "none"):
        ref = Conv(x[0], w, None, [(0, 36)], act)
        y, _ = G.conv_fwd(gpu(x), gpu(w), activation=act)
        check("y", y, ref.y, ref.y_err)
        dx, dw, _, _ = G.conv_bwd(gpu(torch.ones_like(x)), gpu(x), gpu(w), activation=act)
        (rx, ex), (rw, ew), _, _ = ref.backward(torch.ones(36, 4))
        check("dx", dx, rx, ex)
        check("dw", dw, rw, ew)


@pytest.mark.parametrize("act", ["silu", "none"])
def test_gradient_against_differences(act):
    T, C, W, cu = 37, 5, 4, [0, 2, 2, 13, 37]
    x, dy, w, b, s0, dht = draw(1, T, C, W, F32, 4, 31)
    args = dict(x=x[0].double(), w=w.double(), b=b.double(), h=s0.double())
    grads = G.conv_bwd(gpu(dy), gpu(x), gpu(w), gpu(b), activation=act, initial_state=gpu(s0), dht=gpu(dht),
                       cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))

    def loss(a):
        r = Conv(a["x"], a["w"], a["b"], spans(T, cu), act, a["h"])
        return float((r.y * dy[0].double()).sum() + (r.ht * dht.double()).sum())

    gen = torch.Generator().manual_seed(32)
    for name, grad in zip(("x", "w", "b", "h"), grads):
        u = torch.randn(args[name].shape, generator=gen, dtype=torch.float64)
        want = (loss({**args, name: args[name] + 1e-5 * u}) - loss({**args, name: args[name] - 1e-5 * u})) / 2e-5
        got = grad.cpu().double().reshape(u.shape) * u
        assert abs(want - float(got.sum())) <= 1e-5 * float(got.abs().sum()) + 1e-7, name


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,S,C,W,pad", [(1, 1, 64, 4, 0), (5, 1, 40, 3, 2), (3, 4, 7, 4, 1), (4, 2, 16, 2, 0),
                                         (300, 1, 136, 4, 7), (2, 2, 8, 4, 0)])
def test_decode(n, S, C, W, pad, dtype):
    x, _, w, b, _, _ = draw(n, S, C, W, dtype, n, 17 * n + C)
    gen = torch.Generator().manual_seed(n)
    pool = n + 2
    slots = torch.randperm(pool, generator=gen)[:n].to(torch.int32)
    slots[:pad] = torch.tensor([-1, pool, 2 ** 31 - 1, -2 ** 31, -1, -1, pool + 5])[:pad].to(torch.int32)
    state = torch.randn(pool, W - 1, C, generator=gen).to(dtype)
    st = gpu(state).clone()
    y = G.conv_decode(gpu(x), st, gpu(w), gpu(b), slots=gpu(slots)).cpu()
    assert not y[:pad].any()
    seen = state.clone()
    for i in range(pad, n):
        ref = Conv(x[i], w, b, [(0, S)], "silu", state[slots[i].item()][None])
        check("y", y[i], ref.y, ref.y_err)
        seen[slots[i].item()] = ref.ht[0].to(dtype)
    assert torch.equal(seen, st.cpu())
    st2, xi = gpu(state).clone(), gpu(x).clone()
    assert G.conv_decode(xi, st2, gpu(w), gpu(b), slots=gpu(slots), y=xi) is xi
    assert torch.equal(xi.cpu(), y) and torch.equal(st2, st)
    xs = torch.zeros(n, S, C + 5, dtype=dtype, device=DEV)[..., 3:C + 3]
    xs.copy_(gpu(x))
    st2 = gpu(state).clone()
    assert torch.equal(G.conv_decode(xs, st2, gpu(w), gpu(b), slots=gpu(slots)).cpu(), y)


def test_streams_graph_and_repeats():
    T, C, cu = 3000, 200, [0, 700, 1500, 2990]
    x, dy, w, b, s0, dht = (gpu(t) for t in draw(1, T, C, 4, BF16, 3, 12))
    how = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), initial_state=s0)
    outs = [torch.zeros_like(x) for _ in range(3)]

    def step(i=0):
        return G.conv_fwd(x, w, b, output_final_state=True, y=outs[i], **how) + G.conv_bwd(dy, x, w, b, dht=dht, **how)

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    got = []
    for i in range(2):
        with torch.cuda.stream(torch.cuda.Stream()):
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
