"""Linear attention over rows that are cut into segments and spans, against its
64-bit form in chunks (linref_long), every output of every form.

Bounds.  Rows: those of test_gpu_linattn_precision.  States (ht, dh0): float32
sums, (n + 64) 2^-24 A for each element, and in the norm 2^-20: a state of the
last few hundred rows is the sum of some 50 roundings, each of 2^-24 of it or
less, that are independent (sqrt(50) 2^-24 < 2^-20).  Two bf16 parts in its
updates would leave 2^-17 of each term, or 2^-17 / sqrt(3) and more in the norm.

dg of a token: a running sum of d = rho_q - rho_k over at most all rows of the
sequence, from a border's product.  With an error of 2^-22 in each row's rho
(24-bit parts, a float32 dot product) and in each element's product, it is
2^-22 sqrt(sum d^2 + |S o R|^2) off, of which four times is allowed in the norm
over tokens and heads; and 3e-6 of dg itself, as sums over the 128 to 1280 rows
of a segment leave a few 2^-22 of it.  With states in two parts d alone would be
2^-17 / sqrt(3) off: 1e-5 of dg.

dg of a head: sum over tokens.  A row's d counts at most half a span (256) of
times and a border's product a span (512) of times:
2^-22 sqrt(sum w^2 (rho_q^2 + rho_k^2) + sum w^2 |S o R|^2 + sum (pairs in a chunk by
distance)^2) for each head, of which four times is allowed.  One border to a
segment of 768 rows and more, as it would be without spans, is several times
that off."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from helpers import log
from linref import inv_sqrt
from linref_long import C, Long
from test_gpu_linattn import BF16, DEV, F32, draws, gpu
from test_gpu_linattn_precision import norm_close, parts_of, rows_close

SPAN = 512

CASES = [  # lens, H, HV, K, V, dtype, decay, B, h0, dht
    ([900, 0, 260, 3, 700], 2, 4, 128, 128, BF16, "token", None, True, True),
    ([1300, 150], 1, 2, 64, 64, BF16, "head", None, True, True),
    ([1300, 150], 1, 2, 64, 64, F32, "head", None, True, False),
    ([130, 1000, 64], 1, 3, 64, 256, BF16, "token", None, True, False),
    ([1000], 1, 2, 64, 256, F32, "head", 2, False, True),
    ([777, 500], 2, 2, 128, 64, BF16, "head", None, False, True),
    ([777, 500], 2, 4, 128, 64, F32, "token", None, False, False),
    ([640, 900], 1, 2, 128, 256, BF16, "head", None, True, True),
    ([640, 900], 2, 2, 128, 256, F32, "token", None, True, True),
    ([2050], 2, 4, 128, 128, F32, "token", 1, True, True),
    ([1500, 40, 0, 1100], 1, 4, 128, 128, BF16, "none", None, True, True),
    ([2600], 1, 2, 64, 128, BF16, "head", 2, False, False),
]
IDS = ["%s-H%d-%d-K%d-V%d-%s-%s-%s" % ("x".join(map(str, c[0])), c[1], c[2], c[3], c[4],
                                       "bf16" if c[5] == BF16 else "f32", c[6], c[7]) for c in CASES]


def sequences(d):
    """The 64-bit form of every sequence, on the GPU, and where its rows are."""
    out, t = [], 0
    for i, L in enumerate([d["lens"][0]] * d["B"] if d["B"] else d["lens"]):
        at = (i, slice(0, L)) if d["B"] else (0, slice(t, t + L))
        t += L
        g = d["g"]
        g = g if g is None else (g.expand(L, -1) if g.dim() == 1 else g[at])
        out.append((at, i, Long(gpu(d["q"][at]), gpu(d["k"][at]), gpu(d["v"][at]), gpu(g), inv_sqrt(d["q"].shape[3]),
                                None if d["h0"] is None else gpu(d["h0"][i]), gpu(d["do"][at]),
                                None if d["dht"] is None else gpu(d["dht"][i]))))
    return out


def state_close(name, x, ref, A, n):
    err = (x.double() - ref).abs()
    assert bool((err <= (n + 64) * 2.0 ** -24 * A + 1e-30).all()), name
    e = float(err.norm() / ref.norm()) if float(ref.norm()) else float(err.norm())
    log("  %-4s %.2e off" % (name, e))
    assert e <= 2.0 ** -20, (name, e)


def head_bound(r, dtype):
    """What dg of each head may be off, without the factor 4, squared (one sequence of r.L rows)."""
    pos = torch.arange(C, device=r.dev, dtype=torch.float64)
    M = r.M * (pos[:, None] - pos)  # pairs of a chunk by distance
    if dtype == F32:  # chunks of 32 rows there: the others cross one, and count among the rows' terms
        half = torch.arange(C, device=r.dev) // 32
        same = half[:, None] == half
        cross = r.M * ~same
        q, k = r.rho_q + cross.sum(-1), r.rho_k + cross.sum(-2)
        M = M * same
    else:
        q, k = r.rho_q, r.rho_k
    rows = (q ** 2 + k ** 2).sum((1, 2)) * (SPAN / 2) ** 2
    return rows + SPAN ** 2 * (r.border_norms()[:, :: SPAN // C] ** 2).sum(1) + (M.sum(-1) ** 2).sum((1, 2))


def check(d, cu=None):
    dtype, t = d["q"].dtype, {k: gpu(v) if torch.is_tensor(v) else v for k, v in d.items()}
    ins = [t[x] for x in ("q", "k", "v", "g")]
    if cu is None and not d["B"]:
        cu = torch.tensor([0] + d["lens"]).cumsum(0).to(torch.int32).to(DEV)
    o, ht = G.linattn_fwd(*ins, cu_seqlens=cu, initial_state=t["h0"], output_final_state=True)
    dq, dk, dv, dg, dh0 = G.linattn_bwd(t["do"], *ins, cu_seqlens=cu, initial_state=t["h0"], dht=t["dht"])
    per_head, bound, token, refs, got = 0.0, 0.0, [], {}, {}
    for at, i, r in sequences(d):
        (ro, rht), (ao, aht) = r.forward(), r.absolute().forward()
        ref, A = r.backward(), r.absolute().backward()
        n = r.L + r.K + r.V
        for nm, x, y, a in zip(("o", "dq", "dk", "dv"), (o, dq, dk, dv), (ro,) + ref, (ao,) + A):
            rows_close(nm, x[at], y.cpu(), a.cpu(), n, dtype)
            refs.setdefault(nm, []).append(y.cpu())
            got.setdefault(nm, []).append(x[at].cpu())
        state_close("ht", ht[i], rht, aht, n)
        if d["h0"] is not None:
            state_close("dh0", dh0[i], ref[4], A[4], n)
        if d["g"] is None or not r.L:
            continue
        per_head, bound = per_head + ref[3].sum(0), bound + head_bound(r, dtype)
        terms = ((r.rho_q - r.rho_k) ** 2).sum((1, 2)) + (r.M.sum(-1) ** 2 + r.M.sum(-2) ** 2).sum((1, 2))
        if d["g"].dim() == 3:
            token.append((dg[at].double() - ref[3], r.L * (terms + (r.border_norms() ** 2).amax(1)), ref[3]))
    if dtype == BF16:
        for nm in refs:
            norm_close(nm, torch.cat(got[nm]), torch.cat(refs[nm]), dtype)
    if token:
        err, allowed, size = (float(sum(x.sum() for x in y)) ** 0.5 for y in zip(*((e ** 2, b, x ** 2) for e, b, x in token)))
        log("  dg   %.2e off, %.2e of the bound" % (err / size, err / (4 * 2.0 ** -22 * allowed)))
        assert err <= 4 * 2.0 ** -22 * allowed and err <= 3e-6 * size
    elif d["g"] is not None:
        err, allowed = (dg.double() - per_head).abs(), 4 * 2.0 ** -22 * bound.sqrt() + 2.0 ** -24 * per_head.abs()
        log("  dg   %.2e off in the norm, worst error / bound = %.3f" % (float(err.norm() / per_head.norm()),
                                                                        float((err / allowed).max())))
        assert bool((err <= allowed).all()), (err / allowed).tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_segments(case):
    lens, H, HV, K, V, dtype, decay, B, h0, dht = case
    d = draws(51, lens, H, HV, K, V, dtype, decay, True, B)
    d["h0"], d["dht"] = (d[x] if y else None for x, y in (("h0", h0), ("dht", dht)))
    check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("ends", ["none", "h0", "dht", "both"])
@pytest.mark.parametrize("lens,HV,K,V,dtype,B", [
    ([9000], 32, 64, 64, BF16, 1), ([1300], 32, 64, 64, BF16, 14), ([2500, 700, 4000, 1], 48, 64, 128, BF16, None),
    ([4097], 24, 128, 256, BF16, 1), ([6000], 64, 64, 64, F32, 1)],
    ids=["segments of 768", "no segments", "packed", "V256", "f32"])
def test_decay_per_head_over_spans(lens, HV, K, V, dtype, B, ends):
    """Decays from 2^-2 to 2^-9 a row: memories from part of a chunk to a span; every kind of border."""
    if B and B > 4:
        lens, B = lens * B, None  # rows of their own, packed: more requests than are cut further
    d = draws(52, lens, HV, HV, K, V, dtype, "head", True, B)
    d["g"] = torch.log1p(-torch.exp2(-2.0 - 7.0 * torch.arange(HV) / HV))
    d["h0"] = d["h0"] if ends in ("h0", "both") else None
    d["dht"] = d["dht"] if ends in ("dht", "both") else None
    check(d)


@pytest.mark.gpu
def test_decay_per_head_against_differences():
    """dg of a head against central differences of the 64-bit loss over several spans."""
    d = draws(53, [1800], 1, 2, 64, 64, F32, "head", True, 1)
    t = {k: gpu(v) if torch.is_tensor(v) else v for k, v in d.items()}
    dg = G.linattn_bwd(t["do"], t["q"], t["k"], t["v"], t["g"], initial_state=t["h0"], dht=t["dht"])[3]

    def loss(g):
        (at, i, r), = sequences({**d, "g": g})
        o, ht = r.forward()
        return float((o * r._rows(r.do)).sum() + (ht * r.dht).sum())

    for h in range(2):
        e = torch.zeros(2, dtype=torch.float64)
        e[h] = 1e-6
        want = (loss(d["g"].double() + e) - loss(d["g"].double() - e)) / 2e-6
        # third derivatives: (rows of memory)^2 e^2 of the value; 64-bit sums over 1e-6: 1e-9 of the loss's terms
        assert abs(want - float(dg[h])) <= 1e-4 * abs(want) + 1e-4, h


def test_bounds_need_three_parts():
    """Two bf16 parts in a state's updates, or in the state behind rho, do not pass the bounds above; three do."""
    d = draws(54, [600], 1, 2, 64, 64, BF16, "token", True, 1)
    at = (0, slice(0, 600))
    r = Long(d["q"][at], d["k"][at], d["v"][at], d["g"][at], inv_sqrt(64), d["h0"][0], d["do"][at], d["dht"][0])
    (_, ht), (_, aht) = r.forward(), r.absolute().forward()
    ref = r.backward()[3]

    def state(parts):
        E = parts_of(r.v * r.out[..., None], parts).transpose(2, 3) @ r.k
        S = [r.h0]
        for c in range(r.nc):
            S.append(S[-1] * r.all[:, c, None, None] + E[:, c])
        return S

    def decays(parts):  # d of the rows from states in parts, run from the front of each chunk
        S = torch.stack([parts_of(x, parts) for x in r.states()], 1)[:, :-1]
        R = torch.stack([parts_of(x, parts) for x in r.gradients()], 1)[:, 1:]
        q = (r.scale * (r.do @ S) * r.inn[..., None] * r.q).sum(-1)
        k = ((r.v @ R) * r.out[..., None] * r.k).sum(-1)
        err = (q - r.rho_q) - (k - r.rho_k)
        return float(err.flip(-1).cumsum(-1).norm() / ref.norm())

    state_close("ht", state(3)[-1], ht, aht, 600 + 64)
    with pytest.raises(AssertionError):
        state_close("ht", state(2)[-1], ht, aht, 600 + 64)
    assert decays(3) < 3e-6 < decays(2), (decays(3), decays(2))
