"""Linear attention with a decay for each head on the GPU against its plain
64-bit form (linref): prompts, gradients, decode steps, and a run of them.

Tolerances.  Every rounding is relative to the sum of the absolute values of
what is added (linref.forward_abs and backward_abs, written A below).
float32 results of n terms: each term carries at most 16 roundings (the decay
weight's exponent difference, up to 64 chunks' factors are counted in n, the
power, products, parts) and the sum n, all of 2^-24: (n + 64) 2^-24 A.
bf16 results: the scores, the state as an operand and the result are each
rounded to bf16 once, by 2^-8 at most: 2 * 2^-8 A for the two operands and 2^-8
of the result, itself at most A: 3 * 2^-8 A, and the float32 bound on top."""
import math

import pytest
import torch

from gated_delta_product_amd import binding as G
from helpers import log
from linref import Linear, inv_sqrt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def draws(seed, lens, H, HV, K, V, dtype, decay="token", h0=True, B=None):
    """Inputs of packed sequences (lens) or, with B, of B rows of lens[0] tokens; CPU tensors."""
    gen = torch.Generator().manual_seed(seed)
    T = lens[0] if B else sum(lens)
    n = B or 1
    nseq = B or len(lens)

    def normal(*s):
        return torch.randn(s, generator=gen)

    d = dict(q=normal(n, T, H, K).to(dtype) / 4, k=normal(n, T, H, K).to(dtype) / 4, v=normal(n, T, HV, V).to(dtype),
             do=normal(n, T, HV, V).to(dtype))
    d["g"] = {"token": -torch.exp(1.5 * normal(n, T, HV) - 2.5), "head": -torch.exp(-1.0 - torch.arange(HV) * 0.7),
              "none": None}[decay]
    d["h0"] = normal(nseq, HV, V, K) / 2 if h0 else None
    d["dht"] = normal(nseq, HV, V, K) / 2 if h0 else None
    d["lens"], d["B"] = lens, B
    return d


def cu_of(d):
    if d["B"]:
        return None
    return torch.tensor([0] + d["lens"]).cumsum(0).to(torch.int32).to(DEV)


def sequences(d, scale=None):
    """The plain form of every sequence and where its rows are."""
    K = d["q"].shape[3]
    scale = inv_sqrt(K) if scale is None else scale
    out, t = [], 0
    for i, L in enumerate([d["lens"][0]] * d["B"] if d["B"] else d["lens"]):
        at = (i, slice(0, L)) if d["B"] else (0, slice(t, t + L))
        t += L
        g = d["g"]
        g = g if g is None else (g.expand(L, -1) if g.dim() == 1 else g[at])
        out.append((at, Linear(d["q"][at], d["k"][at], d["v"][at], g, scale, None if d["h0"] is None else d["h0"][i])))
    return out


def gpu(t):
    return None if t is None else t.to(DEV)


def within(name, x, ref, A, n, dtype):
    tol = (n + 64) * 2.0 ** -24 + (3 * 2.0 ** -8 if dtype == BF16 else 0.0)
    err = (x.detach().cpu().double() - ref).abs()
    assert torch.isfinite(x).all(), name
    worst = float((err / (A + 1e-30)).max()) if err.numel() else 0.0
    log("  %-4s n=%-8d worst error / bound = %.3f" % (name, err.numel(), worst / tol))
    assert worst <= tol, (name, worst, tol)


def run_fwd(d, cu, scale=None):
    return G.linattn_fwd(gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), gpu(d["g"]), scale=scale, cu_seqlens=cu,
                         initial_state=gpu(d["h0"]), output_final_state=True)


def check_fwd(d, scale=None):
    o, ht = run_fwd(d, cu_of(d), scale)
    for i, (at, r) in enumerate(sequences(d, scale)):
        (ro, rht), (ao, aht) = r.forward(), r.forward_abs()
        n = r.L + r.K
        within("o", o[at], ro, ao, n, d["q"].dtype)
        within("ht", ht[i], rht, aht, n, F32)


CASES = [  # lens, H, HV, K, V, dtype, decay, B
    ([1], 1, 1, 64, 64, F32, "token", 1),
    ([1], 2, 2, 128, 128, BF16, "token", 2),
    ([63], 1, 2, 64, 128, BF16, "head", 1),
    ([64], 2, 2, 128, 64, BF16, "token", 1),
    ([65], 1, 3, 128, 256, BF16, "none", 2),
    ([200], 2, 4, 128, 128, BF16, "token", 3),
    ([31], 2, 2, 64, 64, F32, "token", 2),
    ([97], 1, 2, 128, 128, F32, "head", 1),
    ([130], 1, 1, 64, 256, F32, "token", 1),
    ([321], 1, 2, 64, 256, BF16, "token", 1),
    ([257, 0, 1, 64, 130, 0], 2, 4, 128, 128, BF16, "token", None),
    ([5, 190, 66], 1, 2, 64, 64, BF16, "head", None),
    ([33, 0, 100, 1], 1, 2, 128, 64, F32, "token", None),
    ([129, 70], 2, 2, 128, 256, F32, "token", None),
]
IDS = ["%s-H%d-%d-K%d-V%d-%s-%s-%s" % ("x".join(map(str, c[0])), c[1], c[2], c[3], c[4],
                                       "bf16" if c[5] == BF16 else "f32", c[6], c[7]) for c in CASES]


@pytest.mark.parametrize("h0", [False, True], ids=["zero", "h0"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case, h0):
    lens, H, HV, K, V, dtype, decay, B = case
    check_fwd(draws(3, lens, H, HV, K, V, dtype, decay, h0, B))


def check_bwd(d, scale=None):
    cu = cu_of(d)
    dq, dk, dv, dg, dh0 = G.linattn_bwd(gpu(d["do"]), gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), gpu(d["g"]), scale=scale,
                                        cu_seqlens=cu, initial_state=gpu(d["h0"]), dht=gpu(d["dht"]))
    dtype = d["q"].dtype
    per_head, bound, n_all = 0.0, 0.0, 0
    for i, (at, r) in enumerate(sequences(d, scale)):
        dht = None if d["dht"] is None else d["dht"][i]
        ref, A = r.backward(d["do"][at], dht), r.backward_abs(d["do"][at], dht)
        n = r.L + r.K + r.V
        for nm, x, y, a in zip(("dq", "dk", "dv"), (dq, dk, dv), ref, A):
            within(nm, x[at], y, a, n, dtype)
        if d["h0"] is not None:
            within("dh0", dh0[i], ref[4], A[4], n, F32)
        # dg is a running sum over rows: each row's share rounds relative to its own absolute sum
        if r.L:
            rows = A[3].max(0).values.expand_as(A[3]) * 2
            if d["g"] is not None and d["g"].dim() == 3:
                within("dg", dg[at], ref[3], rows, 8 * n, F32)
            per_head, bound, n_all = per_head + ref[3].sum(0), bound + rows.sum(0), max(n_all, n)
    if d["g"] is None:
        assert dg is None
    elif d["g"].dim() == 1:
        within("dg", dg, per_head, bound, 8 * n_all, F32)
    assert (dh0 is None) == (d["h0"] is None)


@pytest.mark.parametrize("h0", [False, True], ids=["zero", "h0"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case, h0):
    lens, H, HV, K, V, dtype, decay, B = case
    check_bwd(draws(4, lens, H, HV, K, V, dtype, decay, h0, B))


def test_scale():
    d = draws(5, [150], 1, 2, 64, 64, F32, "token", True, 1)
    check_fwd(d, scale=0.7)
    check_bwd(d, scale=0.7)


def test_gradient_against_differences():
    """<gradient, direction> against central differences of the plain 64-bit loss: the float32 gradients' error
    (their bound above, far under 1e-5 of the abs sums) and the differences' e^2 term stay under 1e-4 of the
    directions' share."""
    d = draws(6, [70, 1, 40], 1, 2, 64, 64, F32, "token", True)
    grads = G.linattn_bwd(gpu(d["do"]), gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), gpu(d["g"]), cu_seqlens=cu_of(d),
                          initial_state=gpu(d["h0"]), dht=gpu(d["dht"]))

    def loss(x):
        total = 0.0
        for i, (at, r) in enumerate(sequences(x)):
            o, ht = r.forward()
            total += float((o * d["do"][at].double()).sum() + (ht * d["dht"][i].double()).sum())
        return total

    gen = torch.Generator().manual_seed(8)
    for name, grad in zip(("q", "k", "v", "g", "h0"), grads):
        u = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
        e = 1e-5
        plus, minus = ({**d, name: d[name].double() + s * e * u} for s in (1, -1))
        want = (loss(plus) - loss(minus)) / (2 * e)
        got = float((grad.cpu().double() * u).sum())
        size = float((grad.cpu().double() * u).norm())
        log("  d%-3s differences %.6f, gradient %.6f" % (name, want, got))
        assert abs(want - got) <= 1e-4 * size + 1e-6, name


# ------------------------------------------------------------------ decays at the edges

@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_resets_and_strong_decays(dtype):
    """-inf and decays past float32's range empty the state; what follows keeps its bits."""
    d = draws(9, [150], 1, 2, 64, 64, dtype, "token", True, 1)
    for t, x in ((0, -1e4), (17, float("-inf")), (18, -300.0), (63, float("-inf")), (64, -104.0), (100, -1e30)):
        d["g"][0, t, 1] = x
    d["g"][0, 120:, 0] = 0.0
    check_fwd(d)
    check_bwd(d)


def test_no_gradient_without_pairs():
    """One row and no state: the decays scale nothing, and dg is exactly zero."""
    d = draws(10, [1], 2, 4, 128, 128, BF16, "token", False, 3)
    dg = G.linattn_bwd(*(gpu(d[x]) for x in ("do", "q", "k", "v", "g")))[3]
    assert torch.equal(dg, torch.zeros_like(dg))


# ------------------------------------------------------------------ layouts

def test_strided_rows_of_one_projection():
    """q, k, v and g as slices of wider rows, and per-head decays as a broadcast g: bit for bit."""
    H, HV, K, V, T, B = 2, 4, 64, 128, 140, 2
    d = draws(11, [T], H, HV, K, V, BF16, "token", True, B)
    wide = torch.zeros(B, T + 3, 2 * H * K + HV * V + 64, dtype=BF16, device=DEV)
    q = wide[:, 1:T + 1, :H * K].view(B, T, H, K)
    k = wide[:, 1:T + 1, H * K:2 * H * K].view(B, T, H, K)
    v = wide[:, 1:T + 1, 2 * H * K:2 * H * K + HV * V].view(B, T, HV, V)
    gw = torch.zeros(B, T, HV + 5, device=DEV)
    g = gw[..., 2:2 + HV]
    for dst, nm in ((q, "q"), (k, "k"), (v, "v"), (g, "g")):
        dst.copy_(gpu(d[nm]))
    o, ht = run_fwd(d, None)
    o2, ht2 = G.linattn_fwd(q, k, v, g, initial_state=gpu(d["h0"]), output_final_state=True)
    assert torch.equal(o, o2) and torch.equal(ht, ht2)
    dow = torch.zeros(B, T, HV * V + 8, dtype=BF16, device=DEV)
    do = dow[..., :HV * V].view(B, T, HV, V)
    do.copy_(gpu(d["do"]))
    a = G.linattn_bwd(gpu(d["do"]), *(gpu(d[x]) for x in ("q", "k", "v", "g")), initial_state=gpu(d["h0"]))
    b = G.linattn_bwd(do, q, k, v, g, initial_state=gpu(d["h0"]))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    head = gpu(torch.tensor([-0.1, -0.5, -0.01, 0.0]))
    x = G.linattn_fwd(q, k, v, head)[0]
    y = G.linattn_fwd(q, k, v, head.expand(B, T, HV))[0]
    assert torch.equal(x, y)


def test_offsets_past_32_bits():
    """Rows 2^20 elements apart: element offsets pass 2^32."""
    T, H, K, V = 4200, 1, 64, 64
    d = draws(12, [T], H, H, K, V, BF16, "head", False, 1)
    big = torch.empty(T * (1 << 20) + 256, dtype=BF16, device=DEV)
    rows = big[: T << 20].view(1, T, 1 << 20)
    q, k, v = (rows[..., 64 * i:64 * i + 64].view(1, T, 1, 64) for i in range(3))
    for dst, nm in ((q, "q"), (k, "k"), (v, "v")):
        dst.copy_(gpu(d[nm]))
    o, ht = G.linattn_fwd(q, k, v, gpu(d["g"]), output_final_state=True)
    o2, ht2 = run_fwd(d, None)
    assert torch.equal(o, o2) and torch.equal(ht, ht2)


def test_rows_outside_the_requests_are_left():
    """Tokens before the first offset and behind the last keep what o held; their gradients are zero."""
    lens, H, HV, K, V = [70, 0, 33], 1, 2, 64, 64
    d = draws(13, [7] + lens + [9], H, HV, K, V, BF16, "token", False)
    cu = torch.tensor([7, 77, 77, 110], dtype=torch.int32, device=DEV)
    o = torch.full((1, 119, HV, V), 5.0, dtype=BF16, device=DEV)
    ins = [gpu(d[x]) for x in ("q", "k", "v", "g")]
    G.linattn_fwd(*ins, cu_seqlens=cu, o=o)
    assert (o[0, :7] == 5).all() and (o[0, 110:] == 5).all()
    inner = [x[:, 7:110].contiguous() for x in ins]
    cu0 = cu - 7
    assert torch.equal(o[:, 7:110], G.linattn_fwd(*inner, cu_seqlens=cu0)[0])
    grads = G.linattn_bwd(gpu(d["do"]), *ins, cu_seqlens=cu)
    want = G.linattn_bwd(gpu(d["do"])[:, 7:110].contiguous(), *inner, cu_seqlens=cu0)
    for x, y in zip(grads[:4], want[:4]):
        assert torch.equal(x[:, 7:110], y)
        assert not x[:, :7].any() and not x[:, 110:].any()


@pytest.mark.parametrize("lens", [[130, 90, 77], [700, 1100, 650], [1, 64, 1]], ids=["one pass", "segments", "rows"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_nan_stays_in_its_request(lens, dtype):
    """NaN in one request (or batch row) and outside every request: the others keep their bits."""
    a, b = 5 + lens[0], 5 + lens[0] + lens[1]
    d = draws(28, [5] + lens + [9], 1, 2, 64, 128, dtype, "token", False)
    cu = torch.tensor([5, a, b, b + lens[2]], dtype=torch.int32, device=DEV)
    clean = [gpu(d[x]) for x in ("do", "q", "k", "v", "g")]
    bad = [x.clone() for x in clean]
    for x in bad:
        x[:, :5] = x[:, a:b] = x[:, b + lens[2]:] = float("nan")
    state = torch.randn(3, 2, 128, 64, device=DEV)

    def run(ins, cu):
        o, ht = G.linattn_fwd(*ins[1:], cu_seqlens=cu, initial_state=state, output_final_state=True)
        return [o, ht] + list(G.linattn_bwd(*ins, cu_seqlens=cu, initial_state=state, dht=state))

    for i, (x, y) in enumerate(zip(run(bad, cu), run(clean, cu))):
        if i in (1, 6):  # by request
            assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2])
        else:
            for t in (slice(5, a), slice(b, b + lens[2])):
                assert torch.equal(x[:, t], y[:, t])
    rows = [torch.cat([x[:, :lens[1]]] * 3) for x in clean]
    nan = [x.clone() for x in rows]
    for x in nan:
        x[1] = float("nan")
    for x, y in zip(run(nan, None), run(rows, None)):
        assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2])


def test_gradients_past_32_bits():
    """Over 2^31 elements of v: the last of two requests against its plain form."""
    T, L, H, HV, K, V = 264000, 150, 32, 64, 128, 128
    d = draws(29, [L], H, HV, K, V, BF16, "token", True)
    ins = []
    for name in ("do", "q", "k", "v", "g"):
        x = torch.zeros(1, T, *d[name].shape[2:], dtype=d[name].dtype, device=DEV)
        x[:, T - L:] = gpu(d[name])
        ins.append(x)
    cu = torch.tensor([0, T - L, T], dtype=torch.int32, device=DEV)
    h0, dht = (torch.cat([torch.zeros(1, HV, V, K), d[x]]).to(DEV) for x in ("h0", "dht"))
    o, ht = G.linattn_fwd(*ins[1:], cu_seqlens=cu, initial_state=h0, output_final_state=True)
    grads = G.linattn_bwd(*ins, cu_seqlens=cu, initial_state=h0, dht=dht)
    (at, r), = sequences(d)
    (ro, rht), (ao, aht) = r.forward(), r.forward_abs()
    within("o", o[0, T - L:], ro, ao, L + K, BF16)
    within("ht", ht[1], rht, aht, L + K, F32)
    ref, A = r.backward(d["do"][at], d["dht"][0]), r.backward_abs(d["do"][at], d["dht"][0])
    for name, x, y, a in zip(("dq", "dk", "dv"), grads, ref, A):
        within(name, x[0, T - L:], y, a, L + K + V, BF16)
        assert not x[0, :T - L].any()
    within("dh0", grads[4][1], ref[4], A[4], L + K + V, F32)
    within("dg", grads[3][0, T - L:], ref[3], A[3].max(0).values.expand_as(A[3]) * 2, 8 * (L + K + V), F32)


def test_unordered_offsets_stay_in_bounds():
    """Offsets that overlap or run backwards give some result and touch nothing outside."""
    d = draws(14, [4096], 1, 2, 64, 64, BF16, "token", False, 1)
    ins = [gpu(d[x]) for x in ("q", "k", "v", "g")]
    for cu in ([0, 4096, 0, 4096, 0, 4096], [-5, 9000, 3], [4096, 0, 0, 0]):
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        o, ht = G.linattn_fwd(*ins, cu_seqlens=cu, output_final_state=True)
        G.linattn_bwd(gpu(d["do"]), *ins, cu_seqlens=cu)
    torch.cuda.synchronize()


def test_empty():
    d = draws(15, [0, 0], 1, 2, 64, 128, BF16, "token", True)
    o, ht = run_fwd(d, cu_of(d))
    assert o.shape == (1, 0, 2, 128) and torch.equal(ht.cpu(), d["h0"])
    grads = G.linattn_bwd(*(gpu(d[x]) for x in ("do", "q", "k", "v", "g")), cu_seqlens=cu_of(d),
                          initial_state=gpu(d["h0"]), dht=gpu(d["dht"]))
    assert torch.equal(grads[4].cpu(), d["dht"])
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    ins = [torch.zeros(1, 5, *s, device=DEV) for s in ((1, 64), (1, 64), (2, 64))]
    o = G.linattn_fwd(*ins, cu_seqlens=none, o=torch.ones(1, 5, 2, 64, device=DEV))[0]
    assert (o == 1).all()
    dg = G.linattn_bwd(ins[2], *ins, g=torch.zeros(2, device=DEV), cu_seqlens=none)[3]
    assert torch.equal(dg, torch.zeros_like(dg))


# ------------------------------------------------------------------ long, in segments

@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_segments_match_short_calls(dtype):
    """A long row, run in segments, against the same row in calls chained by their states (float32 states, so
    only the order of sums differs), and its gradients against the chain's."""
    T, H, HV, K, V = 2500, 1, 2, 128, 128
    d = draws(16, [T], H, HV, K, V, dtype, "token", True, 1)
    ins = [gpu(d[x]) for x in ("q", "k", "v", "g")]
    do, h0, dht = gpu(d["do"]), gpu(d["h0"]), gpu(d["dht"])
    o, ht = G.linattn_fwd(*ins, initial_state=h0, output_final_state=True)
    whole = G.linattn_bwd(do, *ins, initial_state=h0, dht=dht)
    cuts = [0, 64, 700, 701, 1800, T]
    s, states, outs = h0, [], []
    for a, b in zip(cuts, cuts[1:]):
        states.append(s)
        x, s = G.linattn_fwd(*(t[:, a:b] for t in ins), initial_state=s, output_final_state=True)
        outs.append(x)
    parts, r = [], dht
    for a, b, st in reversed(list(zip(cuts, cuts[1:], states))):
        g = G.linattn_bwd(do[:, a:b], *(t[:, a:b] for t in ins), initial_state=st, dht=r)
        parts.append(g)
        r = g[4]
    rel = {BF16: 4 * 2.0 ** -8, F32: 1e-5}[dtype]  # two operands and two results rounded, of like sizes
    pairs = [("o", o, torch.cat(outs, 1), rel), ("ht", ht, s, 1e-5), ("dh0", whole[4], r, 1e-5)]
    pairs += [(nm, whole[i], torch.cat([p[i] for p in reversed(parts)], 1), rel if i < 3 else 1e-5)
              for i, nm in enumerate(("dq", "dk", "dv", "dg"))]
    for nm, x, y, tol in pairs:
        e = float((x.double() - y.double()).norm() / y.double().norm())
        log("  %-4s %.2e" % (nm, e))
        assert e <= tol, nm


def test_deterministic():
    d = draws(17, [900, 3, 400], 2, 8, 128, 128, BF16, "head", True)
    ins = [gpu(d[x]) for x in ("q", "k", "v", "g")]
    kw = dict(cu_seqlens=cu_of(d), initial_state=gpu(d["h0"]))
    a = G.linattn_bwd(gpu(d["do"]), *ins, dht=gpu(d["dht"]), **kw) + G.linattn_fwd(*ins, output_final_state=True, **kw)
    b = G.linattn_bwd(gpu(d["do"]), *ins, dht=gpu(d["dht"]), **kw) + G.linattn_fwd(*ins, output_final_state=True, **kw)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------ decode

@pytest.mark.parametrize("n,S,H,HV,K,V,dtype,decay", [
    (1, 1, 1, 1, 64, 64, F32, "token"), (3, 1, 2, 4, 128, 128, BF16, "token"), (5, 4, 1, 3, 128, 256, BF16, "head"),
    (2, 3, 2, 2, 64, 256, F32, "none"), (130, 1, 4, 16, 128, 128, BF16, "token"), (70, 2, 2, 16, 64, 128, F32, "head"),
    (4, 7, 1, 2, 128, 64, BF16, "none"), (129, 1, 8, 8, 64, 64, BF16, "token")])
def test_decode(n, S, H, HV, K, V, dtype, decay):
    d = draws(20, [S], H, HV, K, V, dtype, decay, False, n)
    gen = torch.Generator().manual_seed(21)
    pool = n + 4
    state = torch.randn(pool, HV, V, K, generator=gen)
    slots = torch.randperm(pool, generator=gen)[:n].to(torch.int32)
    if n > 2:
        slots[1], slots[n - 1] = -1, pool
    st = gpu(state.clone())
    o = G.linattn_decode(*(gpu(d[x]) for x in ("q", "k", "v")), st, gpu(d["g"]), slots=gpu(slots))
    want = state.clone()
    for i in range(n):
        s = int(slots[i])
        if not 0 <= s < pool:
            assert not o[i].any()
            continue
        g = d["g"]
        g = g if g is None else (g.expand(S, -1) if g.dim() == 1 else g[i])
        r = Linear(d["q"][i], d["k"][i], d["v"][i], g, inv_sqrt(K), state[s])
        (ro, rht), (ao, aht) = r.forward(), r.forward_abs()
        # the state stays float32: o rounds once
        tol = (S + K + 64) * 2.0 ** -24
        assert ((o[i].cpu().double() - ro).abs() <= tol * ao + (2.0 ** -8 * ro.abs() if dtype == BF16 else 0)).all()
        assert ((st[s].cpu().double() - rht).abs() <= tol * aht).all()
        want[s] = st[s].cpu()
    assert torch.equal(st.cpu(), want)  # the other slots are left alone


def test_one_token_of_any_stride():
    """Time-major projections, one token: the stride over tokens passes every limit and does not matter."""
    n, H, HV, K, V = 3, 2, 4, 64, 128
    d = draws(27, [1], H, HV, K, V, BF16, "token", False, n)
    far = torch.empty(1 << 24, dtype=BF16, device=DEV)

    def major(x):
        v = torch.as_strided(far, x.shape, (x[0, 0].numel() + 8, (1 << 23) + 3, x.shape[3], 1))
        return v.copy_(gpu(x))

    want = G.linattn_fwd(gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), gpu(d["g"]), output_final_state=True)
    state = torch.zeros(n, HV, V, K, device=DEV)
    step = G.linattn_decode(gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), state.clone(), gpu(d["g"]))
    for name in ("q", "k", "v"):
        ins = [major(d[x]) if x == name else gpu(d[x]) for x in ("q", "k", "v")]
        got = G.linattn_fwd(*ins, gpu(d["g"]), output_final_state=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(G.linattn_decode(*ins, state.clone(), gpu(d["g"])), step)


def test_decode_far_slots():
    """A pool of more than 2^31 state elements."""
    HV, K, V, pool = 4, 128, 128, 33000
    d = draws(22, [1], 1, HV, K, V, BF16, "head", False, 2)
    state = torch.empty(pool, HV, V, K, device=DEV)
    slots = torch.tensor([pool - 1, 3], dtype=torch.int32, device=DEV)
    small = torch.randn(2, HV, V, K, device=DEV)
    state[slots.long()] = small
    ins = [gpu(d[x]) for x in ("q", "k", "v")]
    o = G.linattn_decode(*ins, state, gpu(d["g"]), slots=slots)
    o2 = G.linattn_decode(*ins, small, gpu(d["g"]))
    assert torch.equal(o, o2) and torch.equal(state[slots.long()], small)


# ------------------------------------------------------------------ together

def test_prompt_then_tokens():
    """A packed prompt into a state pool, then tokens one by one and as a draft, then the output norm: the rows of
    the whole sequences."""
    H, HV, K, V, lens, more = 2, 4, 128, 128, [130, 1, 77], 5
    full = draws(23, [L + more for L in lens], H, HV, K, V, BF16, "token", False)
    starts = torch.tensor([0] + [L + more for L in lens]).cumsum(0).tolist()
    prompt = [torch.cat([full[x][0, s:s + L] for s, L in zip(starts, lens)])[None].to(DEV) for x in ("q", "k", "v", "g")]
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    o, ht = G.linattn_fwd(*prompt, cu_seqlens=cu, output_final_state=True)
    pool = torch.zeros(6, HV, V, K, device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    pool[slots.long()] = ht

    def tokens(a, b):
        return [torch.stack([full[x][0, s + L + a:s + L + b] for s, L in zip(starts, lens)]).to(DEV)
                for x in ("q", "k", "v", "g")]

    outs = []
    for a, b in ((0, 1), (1, 2), (2, 5)):
        q, k, v, g = tokens(a, b)
        outs.append(G.linattn_decode(q, k, v, pool, g, slots=slots))
    new = torch.cat(outs, 1)
    w, z = torch.randn(HV * V, device=DEV), torch.randn(3, more, HV * V, dtype=BF16, device=DEV)
    y = G.group_norm_fwd(new.flatten(2), HV, w, gate=z, centered=False)
    for i, ((at, r), L) in enumerate(zip(sequences(full), lens)):
        ro, ao = r.forward()[0], r.forward_abs()[0]
        s = int(cu[i])
        within("o", o[0, s:s + L], ro[:L], ao[:L], r.L + K, BF16)
        within("new", new[i], ro[L:], ao[L:], r.L + K, BF16)
    x = new.double()
    want = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    want = want.flatten(2) * w.double() * (z.double() / (1 + torch.exp(-z.double())))
    assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all()


# ------------------------------------------------------------------ streams and graphs

def _step(d, cu):
    ins = [d[x] for x in ("q", "k", "v", "g")]
    o, ht = G.linattn_fwd(*ins, cu_seqlens=cu, initial_state=d["h0"], output_final_state=True)
    return (o, ht) + G.linattn_bwd(d["do"], *ins, cu_seqlens=cu, initial_state=d["h0"], dht=d["dht"])


def test_other_stream():
    d = {k: gpu(v) if torch.is_tensor(v) else v for k, v in draws(24, [700, 90], 1, 2, 128, 128, BF16).items()}
    cu = cu_of(d)
    want = _step(d, cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = _step(d, cu)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_graph_replays():
    """A captured step, replayed with new inputs and eager work between the replays."""
    d = {k: gpu(v) if torch.is_tensor(v) else v for k, v in draws(25, [800, 64, 5], 1, 4, 64, 128, BF16).items()}
    cu = cu_of(d)
    _step(d, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(d, cu)
    for k in range(4):
        for x in ("q", "v", "do"):
            d[x].copy_(torch.randn(d[x].shape, device=DEV))
        cu.copy_(torch.tensor([0, 800 - 13 * k, 864 - 13 * k, 869], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = _step(d, cu)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got)), k


# ------------------------------------------------------------------ through the C ABI

def _abi(d, cu=None, **kw):
    t = {k: gpu(d[k]) for k in ("q", "k", "v", "g", "h0", "dht", "do")}
    B, T, H, K = t["q"].shape
    HV, V = t["v"].shape[2:]
    a = G.LinattnArgs(B=B, T=T, H=H, HV=HV, K=K, V=V, scale=0.0, dtype=G._dtype_code(t["q"].dtype),
                      cu_seqlens=None if cu is None else cu.data_ptr(), num_seqs=0 if cu is None else cu.numel() - 1,
                      **{x: t[x].data_ptr() for x in ("q", "k", "v", "g", "h0")},
                      **{"%s_%s_stride" % (x, y): t[x].stride(i) for x in ("q", "k", "v", "g")
                         for i, y in enumerate("bt")}, **kw)
    return t, a


def _space(a, backward):
    import ctypes
    need = G.lib().gdp_linattn_workspace_bytes(ctypes.byref(a), backward)
    return torch.full((max(need, 256),), 0xA5, dtype=torch.uint8, device=DEV), need


@pytest.mark.parametrize("T", [100, 2000])
def test_final_state_in_place_of_the_initial_one(T):
    """ht on top of h0, in one pass and in segments, from a workspace full of garbage."""
    import ctypes
    d = draws(30, [T], 1, 2, 64, 128, BF16, "token", True, 1)
    o, ht = run_fwd(d, None)
    t, a = _abi(d)
    out = torch.empty_like(o)
    a.o, a.ht = out.data_ptr(), t["h0"].data_ptr()
    ws, need = _space(a, 0)
    assert (need > 0) == (T > 512)
    G._check(G.lib().gdp_linattn_fwd(ctypes.byref(a), ws.data_ptr(), need, G._stream(torch.device(DEV))))
    torch.cuda.synchronize()
    assert torch.equal(out, o) and torch.equal(t["h0"], ht)


@pytest.mark.parametrize("T", [100, 2000])
def test_gradients_that_are_not_wanted(T):
    """dg without dh0 (the library forms what it needs of it itself), dh0 without dg, and neither."""
    import ctypes
    d = draws(31, [T], 1, 2, 64, 64, F32, "token", True, 1)
    want = G.linattn_bwd(*(gpu(d[x]) for x in ("do", "q", "k", "v", "g")), initial_state=gpu(d["h0"]), dht=gpu(d["dht"]))
    for with_g, with_h in ((True, False), (False, True), (False, False)):
        t, a = _abi(d)
        dq, dk, dv = (torch.empty_like(t[x]) for x in ("q", "k", "v"))
        dg, dh0 = torch.empty_like(t["g"]), torch.empty_like(t["h0"])
        r = G.LinattnGrads(dout=t["do"].data_ptr(), do_b_stride=t["do"].stride(0), do_t_stride=t["do"].stride(1),
                           dht=t["dht"].data_ptr(), dq=dq.data_ptr(), dk=dk.data_ptr(), dv=dv.data_ptr(),
                           dg=dg.data_ptr() if with_g else None, dh0=dh0.data_ptr() if with_h else None)
        ws, need = _space(a, 1)
        G._check(G.lib().gdp_linattn_bwd(ctypes.byref(a), ctypes.byref(r), ws.data_ptr(), need,
                                         G._stream(torch.device(DEV))))
        torch.cuda.synchronize()
        for x, y in ((dq, want[0]), (dk, want[1]), (dv, want[2])):
            assert float((x.double() - y.double()).norm()) <= 1e-5 * float(y.double().norm())
        assert not with_g or torch.equal(dg, want[3])
        assert not with_h or torch.equal(dh0, want[4])


def test_many_short_requests():
    """More requests than a wave has lanes, some empty, none in segments."""
    gen = torch.Generator().manual_seed(32)
    lens = torch.randint(0, 9, (150,), generator=gen).tolist()
    d = draws(33, lens, 1, 1, 64, 64, BF16, "token", True)
    check_fwd(d)
    check_bwd(d)


def test_norm_of_the_gated_delta_product():
    """The output norm behind the other mixer: o [B, T, HV, V] of chunk_fwd, normalised per head and gated."""
    from gated_delta_product_amd import synth
    from helpers import gates
    B, T, H, K, V, M = 1, 150, 2, 64, 128, 2
    c = synth.chunk_draws(B, T, H, H, K, V, M, "bf16", 34)
    beta, g = gates(c)
    buf = G.chunk_fwd(*(x.to(DEV) for x in (c["q"], c["k"], c["v"], beta.reshape(B, T * M, H), g)))
    z, w = torch.randn(B, T, H * V, dtype=BF16, device=DEV), torch.randn(H * V, device=DEV)
    y = G.group_norm_fwd(buf.o.flatten(2), H, w, gate=z, centered=False)
    x = buf.o.double()
    want = (x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)).flatten(2) * w.double()
    want = want * (z.double() / (1 + torch.exp(-z.double())))
    assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all()
