"""The precision that linear attention works in, pinned: every output against
its plain 64-bit form (linref) at bounds that a part less, or an operand
rounded once, does not keep.

A is the sum of absolute values behind each element (forward_abs,
backward_abs), n the number of its terms.

Rows (o, dq, dk, dv).  float32 work is off by (n + 64) 2^-24 A at most (16
roundings a term, the rest in n).  With bf16 rows the scores, the state as an
operand and the decayed rows of its update are sums of two bf16 parts or more:
what two parts leave of a value is 2^-8 2^-8 of it, so 3 * 2^-16 A for the
three.  The result rounds once, by 2^-8 of itself:
    |x - ref| <= 2^-8 |ref| + (3 2^-16 + (n + 64) 2^-24) (1 + 2^-8) A.
Rounded to bf16 once, an operand alone is up to 2^-8 A off, and A is many times
|ref| where terms cancel.

In the 2-norm, x is then off by what rounding ref itself leaves, r, and by the
float32 part, which is uncorrelated with it.  Independent errors of 2^-16 or
less are under a tenth of r (2^-9 and more), so sqrt(1 + 0.01) r <= 1.02 r is
allowed."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from helpers import log
from linref import Linear
from test_gpu_linattn import BF16, DEV, F32, cu_of, draws, gpu, run_fwd, sequences

IDS_DTYPE = {BF16: "bf16", F32: "f32"}


def rows_close(name, x, ref, A, n, dtype):
    x = x.detach().cpu().double()
    tol = (n + 64) * 2.0 ** -24 * A
    if dtype == BF16:
        tol = 2.0 ** -8 * ref.abs() + (tol + 3 * 2.0 ** -16 * A) * (1 + 2.0 ** -8)
    err = (x - ref).abs()
    worst = float((err / (tol + 1e-30)).max()) if err.numel() else 0.0
    log("  %-4s worst error / bound = %.3f" % (name, worst))
    assert worst <= 1.0, (name, worst)


def norm_close(name, x, ref, dtype):
    """bf16 rows against the rounding of the exact ones."""
    ref = ref.double()
    own = float((ref.to(dtype).double() - ref).norm() / ref.norm())
    e = float((x.detach().cpu().double() - ref).norm() / ref.norm())
    log("  %-4s %.3e off, rounded exact rows %.3e" % (name, e, own))
    assert e <= 1.02 * own, (name, e, own)


ROWS = [  # lens, H, HV, K, V, decay, B
    ([200], 2, 4, 128, 128, "token", 2),
    ([5, 1, 2, 3, 64, 33, 4, 1, 128], 1, 2, 64, 64, "head", None),
    ([130], 1, 2, 64, 256, "none", 1),
    ([97, 70], 2, 2, 128, 256, "token", None),
    ([150], 1, 3, 128, 64, "head", 1),
    ([321], 1, 2, 64, 128, "token", 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", ROWS, ids=["x".join(map(str, c[0])) + "-K%d-V%d" % c[3:5] for c in ROWS])
def test_rows_round_once(case, dtype):
    lens, H, HV, K, V, decay, B = case
    d = draws(41, lens, H, HV, K, V, dtype, decay, True, B)
    o = run_fwd(d, cu_of(d))[0]
    o_alone = G.linattn_fwd(gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), gpu(d["g"]), cu_seqlens=cu_of(d),
                            initial_state=gpu(d["h0"]))[0]
    # with dg, and without it (no decay: none is wanted)
    outs = []
    for g in (d["g"], None):
        grads = G.linattn_bwd(gpu(d["do"]), gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), gpu(g), cu_seqlens=cu_of(d),
                              initial_state=gpu(d["h0"]), dht=gpu(d["dht"]))
        outs.append((g, grads[:3]))
    refs, got = {}, {}
    for i, (at, r) in enumerate(sequences(d)):
        ref, A = r.forward()[0], r.forward_abs()[0]
        for nm, x in (("o", o), ("o'", o_alone)):
            rows_close(nm, x[at], ref, A, r.L + r.K, dtype)
            refs.setdefault(nm, []).append(ref)
            got.setdefault(nm, []).append(x[at])
    for which, (g, grads) in enumerate(outs):
        for i, (at, r) in enumerate(sequences({**d, "g": g})):
            ref, A = r.backward(d["do"][at], d["dht"][i]), r.backward_abs(d["do"][at], d["dht"][i])
            for j, nm in enumerate(("dq", "dk", "dv")):
                rows_close(nm, grads[j][at], ref[j], A[j], r.L + r.K + r.V, dtype)
                refs.setdefault(nm + "'" * which, []).append(ref[j])
                got.setdefault(nm + "'" * which, []).append(grads[j][at])
    if dtype == BF16:
        for nm in refs:
            norm_close(nm, torch.cat(got[nm]), torch.cat(refs[nm]), dtype)


def parts_of(x, n):
    """x as the sum of n bf16 parts."""
    out = torch.zeros_like(x)
    for _ in range(n):
        out = out + (x - out).to(BF16).double()
    return out


def test_rows_bound_needs_both_parts():
    """The bound and the norm above tell an operand that is rounded once: the plain form with the scores, or the
    state in front of the queries, in one part fails them, in two passes."""
    d = draws(42, [200], 1, 2, 64, 64, BF16, "token", True, 1)
    (at, r), = sequences(d)
    ref, A = r.forward()[0], r.forward_abs()[0]
    P = (r.q @ r.k.transpose(1, 2)) * r.D

    def rows(scores, state):
        y = parts_of(P, scores) @ r.v + r.D0[..., None] * (r.q @ parts_of(r.h0, state).transpose(1, 2))
        return (r.scale * y).transpose(0, 1).to(BF16)

    rows_close("o", rows(2, 2), ref, A, r.L + r.K, BF16)
    norm_close("o", rows(2, 2), ref, BF16)
    for bad in ((1, 2), (2, 1)):
        with pytest.raises(AssertionError):
            rows_close("o", rows(*bad), ref, A, r.L + r.K, BF16)
    with pytest.raises(AssertionError):
        norm_close("o", rows(1, 2), ref, BF16)
