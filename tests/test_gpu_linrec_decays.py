"""The recurrence's decays over their whole range, in every type of rows."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from helpers import log
from mixref import Rec, worst

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
TYPES = [(BF16, BF16), (BF16, F32), (F32, F32)]
IDS = ["bf16", "bf16-f32", "f32"]


def gpu(t):
    return None if t is None else t.to(DEV)


def check(name, got, want, err):
    w = worst(name, got, want, err)
    log("  %-4s worst error / bound = %.3f" % (name, w))
    assert w <= 1.0, (name, w)


def against(ref, x, g, decay, comp, s0, dy, dht):
    """Every output of one sequence x, g [T, C] in both directions, and of its rows as steps, against ref's bounds."""
    how = dict(decay=decay, complement=comp)
    y, ht = G.linrec_fwd(gpu(x)[None], gpu(g)[None], initial_state=gpu(s0), output_final_state=True, **how)
    grads = G.linrec_bwd(gpu(dy)[None], gpu(x)[None], gpu(g)[None], initial_state=gpu(s0), dht=gpu(dht), **how)
    state = gpu(s0).clone()
    step = G.linrec_decode(gpu(x)[None], gpu(g)[None], state, **how)
    for name, got, want, err in (("y", y, ref.h, ref.err), ("ht", ht, ref.ht, ref.ht_err), ("step", step, ref.h, ref.err),
                                 ("pool", state, ref.ht, ref.ht_err)):
        check(name, got, want, err)
    for name, got, want in zip(("dx", "dg", "dh0"), grads, ref.backward(dy, dht)):
        check(name, got, *want)


@pytest.mark.parametrize("decay", ["log", "sigmoid"])
@pytest.mark.parametrize("comp", [False, True], ids=["plain", "complement"])
@pytest.mark.parametrize("dtype,gtype", TYPES, ids=IDS)
def test_a_decay_of_zero_drops_the_state(dtype, gtype, comp, decay):
    """Whatever the state was: the row's own input is what is left, bit for bit, and nothing goes back past it."""
    T, C, at = 150, 24, 70
    gen = torch.Generator().manual_seed(41)
    x, dy = (torch.randn(1, T, C, generator=gen).to(dtype) for _ in range(2))
    g = torch.rand(1, T, C, generator=gen).to(gtype) * (-0.01 if decay == "log" else 9.0)
    g[:, at] = -float("inf") if decay == "log" else -200.0
    s0 = 1e10 * (1 + torch.rand(1, C, generator=gen))
    how = dict(decay=decay, complement=comp)
    y, _ = G.linrec_fwd(gpu(x), gpu(g), initial_state=gpu(s0), **how)
    y2, ht = G.linrec_fwd(gpu(x[:, at:]), gpu(g[:, at:]), initial_state=gpu(s0), output_final_state=True, **how)
    assert torch.equal(y.cpu()[:, at], x[:, at]) and torch.equal(y2.cpu()[:, 0], x[:, at])
    assert torch.equal(y2, G.linrec_fwd(gpu(x[:, at:]), gpu(g[:, at:]), **how)[0])  # of no state
    state = gpu(s0).clone()
    y1 = G.linrec_decode(gpu(x[:, at:at + 1]), gpu(g[:, at:at + 1]), state, **how)
    assert torch.equal(y1.cpu()[:, 0], x[:, at]) and torch.equal(state.cpu(), x[:, at].float())
    dht = 1e10 * torch.ones(1, C)
    dx, dg, dh0 = G.linrec_bwd(gpu(dy), gpu(x), gpu(g), initial_state=gpu(s0), dht=gpu(dht), **how)
    assert torch.isfinite(dg).all() and not dg[:, at].any()
    part = G.linrec_bwd(gpu(dy[:, :at]), gpu(x[:, :at]), gpu(g[:, :at]), initial_state=gpu(s0), **how)
    for name, p, q in (("dx", dx[:, :at], part[0]), ("dg", dg[:, :at], part[1]), ("dh0", dh0, part[2])):
        assert torch.equal(p, q), name


@pytest.mark.parametrize("comp", [False, True], ids=["plain", "complement"])
@pytest.mark.parametrize("dtype,gtype", TYPES, ids=IDS)
def test_states_that_grow(dtype, gtype, comp):
    """Log decays above zero, from those next to it on, and at it: 1 - a without cancellation there too."""
    T, C = 24, 40
    gen = torch.Generator().manual_seed(42)
    x, dy = (torch.randn(T, C, generator=gen).to(dtype) for _ in range(2))
    g = (10 ** (-7 + 6.5 * torch.rand(T, C, generator=gen))).to(gtype)
    g[5] = 0
    s0, dht = torch.randn(1, C, generator=gen), torch.randn(1, C, generator=gen)
    against(Rec(x, g, [(0, T)], "log", comp, s0), x, g, "log", comp, s0, dy, dht)
