"""Rotary positions on the GPU against their plain 64-bit form (mixref.rotate),
whose bounds the tolerances are."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from helpers import log
from mixref import rotate, spans, worst

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def gpu(t):
    return None if t is None else t.to(DEV)


def draw(B, T, H, HK, D, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(B, T, H, D, generator=gen).to(dtype)
    return q, torch.randn(B, T, HK, D, generator=gen).to(dtype) if HK else None


def check(name, got, x, pos, freq, inside=None, **kw):
    x = x.reshape(-1, *x.shape[2:])
    y, err = rotate(x, pos, freq, **kw)
    got = got.cpu().reshape(x.shape)
    if inside is not None:
        y, err, got = y[inside], err[inside], got[inside]
    r = worst(name, got, y, err)
    log("  %-3s worst error / bound = %.3f" % (name, r))
    assert r <= 1.0, (name, r)
    R = 2 * freq.numel()
    kept = x if inside is None else x[inside]
    assert torch.equal(got[..., R:], kept[..., R:]), "what is not rotated is copied"


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,HK,D,R", [
    (1, 1, 1, 0, 2, 2), (1, 5, 3, 1, 64, 64), (2, 33, 4, 2, 128, 64), (1, 40, 16, 4, 128, 128), (3, 7, 2, 2, 80, 20),
    (1, 9, 1, 1, 96, 48), (1, 3, 2, 1, 256, 256), (1, 2, 1, 1, 33, 10), (70, 1, 4, 4, 64, 32), (1, 2, 1, 1, 4096, 4096)])
def test_rows(B, T, H, HK, D, R, dtype, interleaved):
    q, k = draw(B, T, H, HK, D, dtype, D + T)
    freq, _ = G.rotary_freq(R)
    gen = torch.Generator().manual_seed(R)
    off = torch.randint(-50, 5000, (B,), generator=gen).to(torch.int32)
    pos = (torch.arange(T) + off[:, None]).reshape(-1)
    for inverse in (False, True):
        kw = dict(interleaved=interleaved, scale=1.25, inverse=inverse)
        qo, ko = G.rotary(gpu(q), gpu(k), gpu(freq), offsets=gpu(off), **kw)
        check("q", qo, q, pos, freq, **kw)
        if HK:
            check("k", ko, k, pos, freq, **kw)
        else:
            assert ko is None
    given = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, T), generator=gen).to(torch.int32)  # any position
    qo, ko = G.rotary(gpu(q), gpu(k), gpu(freq), positions=gpu(given), interleaved=interleaved)
    check("q", qo, q, given.reshape(-1), freq, interleaved=interleaved)
    wide = torch.zeros(B, 2 * T, dtype=torch.int32)
    wide[:, ::2] = given
    q2, _ = G.rotary(gpu(q), gpu(k), gpu(freq), positions=gpu(wide)[:, ::2], interleaved=interleaved)
    assert torch.equal(qo, q2)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,cu", [(300, [0, 1, 1, 3, 64, 64, 64, 191, 300]), (260, [5, 5, 133, 200, 250]), (40, [7, 7]),
                                  (33, [0]), (70, [0] + list(range(1, 71))), (50, [-4, 20, 45, 90])])
def test_packed(T, cu, dtype):
    H, HK, D, R = 4, 2, 64, 64
    q, k = draw(1, T, H, HK, D, dtype, T)
    freq, scale = G.rotary_freq(R, scaling="parts", factor=8.0, original_length=64)
    seqs = spans(T, cu)
    off = torch.arange(len(seqs), dtype=torch.int32) * 1000
    pos, inside = torch.zeros(T, dtype=torch.int64), torch.zeros(T, dtype=torch.bool)
    for i, (a, e) in enumerate(seqs):
        pos[a:e] = torch.arange(e - a) + int(off[i])
        inside[a:e] = True
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out = tuple(torch.full(t.shape, 7.0, dtype=dtype, device=DEV) for t in (q, k))
    qo, ko = G.rotary(gpu(q), gpu(k), gpu(freq), offsets=gpu(off), cu_seqlens=cud, scale=scale, out=out)
    assert qo is out[0] and ko is out[1]
    for x, y in ((q, qo), (k, ko)):
        assert (y.cpu()[0][~inside] == 7).all(), "rows outside every request"
        check("x", y, x, pos, freq, inside, scale=scale)


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("off", [16, 5])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_slices_in_place(dtype, off, interleaved):
    """Queries and keys as slices of one projection, turned where they lie; nothing beside them is touched."""
    B, T, H, HK, D, R = 2, 37, 4, 2, 64, 32
    q, k = draw(B, T, H, HK, D, dtype, 5)
    freq, _ = G.rotary_freq(R)
    want = G.rotary(gpu(q), gpu(k), gpu(freq), interleaved=interleaved)
    width = off + (H + HK) * D + 8
    wide = torch.full((B, T + 3, width), 3.0, dtype=dtype, device=DEV)
    qs = wide[:, 1:T + 1, off:off + H * D].unflatten(2, (H, D))
    ks = wide[:, 1:T + 1, off + H * D:off + (H + HK) * D].unflatten(2, (HK, D))
    qs.copy_(gpu(q))
    ks.copy_(gpu(k))
    G.rotary(qs, ks, gpu(freq), interleaved=interleaved, out=(qs, ks))
    assert torch.equal(qs, want[0]) and torch.equal(ks, want[1])
    rest = wide.clone()
    rest[:, 1:T + 1, off:off + (H + HK) * D] = 3
    assert (rest == 3).all()


def test_back_undoes_and_is_the_gradient():
    B, T, H, D = 1, 50, 3, 64
    q, k = draw(B, T, H, H, D, F32, 6)
    freq, _ = G.rotary_freq(D)
    a, b = G.rotary(gpu(q), gpu(k), gpu(freq))
    c, d = G.rotary(a, b, gpu(freq), inverse=True)
    # two rotations: twice the bound of one, of pairs of their size
    size = lambda x: (x.unflatten(-1, (2, -1)).norm(dim=-2, keepdim=True) * 2).expand(*x.shape[:-1], 2, D // 2).flatten(-2)  # noqa: E731
    for x, y in ((q, c), (k, d)):
        assert ((y.cpu() - x).abs() <= 2 * 34 * 2.0 ** -24 * size(x)).all()
    # <dq, rotate(u)> = <back(dq), u> for the linear map that it is, and differences of the plain form
    gen = torch.Generator().manual_seed(7)
    u = torch.randn(T, H, D, generator=gen, dtype=torch.float64)
    pos = torch.arange(T)
    plain = (rotate(q[0].double() + 1e-3 * u, pos, freq, scale=1.5)[0] - rotate(q[0].double() - 1e-3 * u, pos, freq, scale=1.5)[0]) / 2e-3
    grad, _ = G.rotary(gpu(k), None, gpu(freq), scale=1.5, inverse=True)
    want, got = float((plain * k[0].double()).sum()), (grad.cpu().double()[0] * u)
    assert abs(want - float(got.sum())) <= 1e-5 * float(got.abs().sum())


def test_continues_a_cache():
    """A prompt at once, or its tokens one by one with positions or offsets: the same bits."""
    T, H, D = 24, 2, 64
    q, k = (gpu(t) for t in draw(1, T, H, 1, D, BF16, 8))
    freq = gpu(G.rotary_freq(D, base=500000.0)[0])
    want = G.rotary(q, k, freq, offsets=torch.tensor([100], dtype=torch.int32, device=DEV))
    for t in range(T):
        o = torch.tensor([100 + t], dtype=torch.int32, device=DEV)
        for kw in (dict(offsets=o), dict(positions=o[:, None])):
            a, b = G.rotary(q[:, t:t + 1], k[:, t:t + 1], freq, **kw)
            assert torch.equal(a, want[0][:, t:t + 1]) and torch.equal(b, want[1][:, t:t + 1])


def test_streams_and_graph():
    T, H, D = 500, 8, 128
    q, k = (gpu(t) for t in draw(1, T, H, 2, D, BF16, 9))
    freq = gpu(G.rotary_freq(D)[0])
    off = torch.tensor([3], dtype=torch.int32, device=DEV)
    want = G.rotary(q, k, freq, offsets=off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = G.rotary(q, k, freq, offsets=off)
    s.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = G.rotary(q, k, freq, offsets=off)
    for i in range(3):
        off.fill_(1000 * i)
        q.copy_(torch.randn(q.shape, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, r) for p, r in zip(G.rotary(q, k, freq, offsets=off), got))
