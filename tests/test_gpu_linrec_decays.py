"""The recurrence's decays over their whole range, in every type of rows: a and
1 - a each to a few roundings of itself, however small it is."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from helpers import log
from mixref import U, Rec, TINY, worst

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = [("log", False), ("log", True), ("sigmoid", False), ("sigmoid", True)]
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


class Close(Rec):
    """Rec, where a and 1 - a are each off by roundings of themselves, however small they are: by 2^-24 times

    * 4 for the exponential (of bfloat16 rows |g| more: the power's argument is rounded), 3 for a sum and a reciprocal, 2
      for the last bit, which tells the two kinds of numbers apart, and 1 for the difference from one. Only the smaller
      one of a and 1 - a is kept of a gate;
    * of a log decay away from zero (|g| over 1/4) a is, and up to 4.5 times as large as its distance from one:
      4.5 (4 + 2) + 1 in all. Nearer to zero the distance is kept, a series cut off at 1 and with 3 roundings."""

    def __init__(self, x, g, seqs, decay, complement, h0):
        super().__init__(x.float(), g, seqs, decay, complement, h0)
        s, power = self.s.abs(), 0
        if x.dtype == torch.bfloat16:
            power = (g.double().abs() * self.a).nan_to_num(0.0, 0.0, 0.0) * (self.s if decay == "sigmoid" else 1)
        self.rest_err = U * (28 * s + power)
        self.keep_err = U * (28 * torch.minimum(self.a, 4.5 * s) + power)
        for i, (b, e) in enumerate(seqs):
            er = torch.zeros_like(self.h0[i])
            ha = self.h0[i].abs()
            for t in range(b, e):
                self.prev_err[t] = er
                cx = self.c[t].abs() * self.x[t].abs()
                er = (self.a[t] * er + 8 * U * (self.a[t] * ha + cx) + TINY * ha + self.keep_err[t] * ha
                      + (self.rest_err[t] * self.x[t].abs() if complement else 0))
                ha = self.a[t] * ha + cx
                self.err[t] = er
            self.ht_err[i] = er


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


@pytest.mark.parametrize("decay,comp", KINDS)
@pytest.mark.parametrize("dtype,gtype", TYPES, ids=IDS)
def test_fast_decays(dtype, gtype, decay, comp):
    """What little a fast channel keeps, of large states and where no input hides it."""
    T, C = 40, 48
    gen = torch.Generator().manual_seed(43)
    x, dy = (torch.randn(T, C, generator=gen) for _ in range(2))
    x[:20], dy[20:] = 0, 0  # the state alone, forwards and then backwards
    x, dy = x.to(dtype), dy.to(dtype)
    g = -torch.rand(C, generator=gen) * 3 - torch.rand(T, C, generator=gen) * (16 if decay == "log" else 20)
    g[::5] = g[::5].abs() * (0.01 if decay == "log" else 1)  # and a row that grows, or hardly decays
    g[7] = -50.0
    g[31] = -float("inf") if decay == "log" else -300.0
    g = g.to(gtype)
    s0, dht = 1e3 * torch.randn(1, C, generator=gen), 1e3 * torch.randn(1, C, generator=gen)
    against(Close(x, g, [(0, T)], decay, comp, s0), x, g, decay, comp, s0, dy, dht)


@pytest.mark.parametrize("decay,comp", KINDS)
@pytest.mark.parametrize("dtype,gtype", TYPES, ids=IDS)
def test_one_row_of_every_decay(dtype, gtype, decay, comp):
    """a and 1 - a themselves: a row of nothing but a state, one of nothing but an input, and their gradients."""
    C = 4096
    g = torch.linspace(-40.0, 2.0 if decay == "log" else 40.0, C)
    g[::2] = torch.linspace(-1.0, 1.0, C // 2)
    g = g[None].to(gtype)
    one, zero = torch.ones(1, C), torch.zeros(1, C)
    for x, s0, dy in ((zero, one, zero), (one, zero, one), (one, -one, zero)):
        x, dy = x.to(dtype), dy.to(dtype)
        against(Close(x, g, [(0, 1)], decay, comp, s0), x, g, decay, comp, s0, dy, one)
