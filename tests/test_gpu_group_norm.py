"""Group norm with an activation on the GPU against its plain 64-bit form.

Tolerances.  bf16 outputs round once: 2^-8 of the value; the float32 steps
before that (sums of D squares and D values in a tree, a root, the fast
exponential and reciprocal of the activation, about 2^-21) are relative to the
largest value of the group times the weight: 2^-19 of |w| |gate| (max|xh| + 1),
plus the bias' share.  Gradients of x subtract means of like size: the same
with the terms' sizes.  dweight and dbias sum `rows` float32 terms: 2^-19 plus
rows 2^-24 of the absolute sum."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from helpers import log
from linref import group_norm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32

SHAPES = [  # rows, groups, D
    (1, 1, 1), (5, 3, 7), (3, 2, 40), (17, 3, 64), (256, 16, 128), (9, 4, 80), (33, 2, 96), (4, 1, 160), (7, 2, 256),
    (2, 3, 1000), (3, 1, 4096), (2, 2, 2049), (4099, 2, 8), (515, 1, 513),
]


def draw(rows, groups, D, dtype, seed, gate, affine):
    gen = torch.Generator().manual_seed(seed)
    C = groups * D
    x = (torch.randn(rows, C, generator=gen) * (0.1 + torch.rand(rows, 1, generator=gen)) + 0.3).to(dtype)
    z = (2 * torch.randn(rows, C, generator=gen)).to(dtype) if gate else None
    w = torch.randn(C, generator=gen) if affine else None
    b = torch.randn(C, generator=gen) if affine else None
    return x, z, w, b, torch.randn(rows, C, generator=gen).to(dtype)


def gpu(t):
    return None if t is None else t.to(DEV)


def check(name, x, ref, tol):
    err = (x.cpu().double() - ref).abs()
    assert torch.isfinite(x).all(), name
    worst = float((err / (tol + 1e-30)).max())
    log("  %-3s worst error / bound = %.3f" % (name, worst))
    assert worst <= 1.0, (name, worst)


@pytest.mark.parametrize("gate,affine,act,centered", [
    (True, True, "silu", True), (False, True, "silu", False), (True, False, "sigmoid", False),
    (False, False, "sigmoid", True), (True, True, "none", False), (False, True, "none", True)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,groups,D", SHAPES)
def test_against_plain(rows, groups, D, dtype, gate, affine, act, centered):
    eps = 1e-5
    x, z, w, b, dy = draw(rows, groups, D, dtype, 7 * D + rows, gate, affine)
    kw = dict(weight=gpu(w), bias=gpu(b), gate=gpu(z), activation=act, centered=centered, eps=eps)
    y = G.group_norm_fwd(gpu(x), groups, **kw)
    dx, dz, dw, db = G.group_norm_bwd(gpu(dy), gpu(x), groups, **kw)
    leaves = [t.double().requires_grad_() if t is not None else None for t in (x, z, w, b)]
    ref = group_norm(leaves[0], groups, leaves[2], leaves[3], leaves[1], act, centered, eps)
    named = [t for t in leaves if t is not None]
    grads = iter(torch.autograd.grad(ref, named, dy.double()))
    rx, rz, rw, rb = (next(grads) if t is not None else None for t in leaves)
    step = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    ref = ref.detach()
    u = x.double().reshape(rows, groups, D)
    centre = u - u.mean(-1, keepdim=True) if centered else u
    rstd = 1 / torch.sqrt((centre * centre).mean(-1, keepdim=True) + eps)
    xh = centre * rstd
    # the mean's own rounding, 2^-22 of the row's size, is what is left of a constant row
    amp = (xh.abs().amax(-1, keepdim=True) + 1 + (u.abs().amax(-1, keepdim=True) * rstd if centered else 0))
    amp = amp.expand(rows, groups, D).reshape(rows, -1)
    wa = torch.ones(groups * D, dtype=torch.float64) if w is None else w.double().abs()
    ba = 0.0 if b is None else b.double().abs()
    za = 1.0 if z is None else z.double().abs() + 1
    n = wa * amp + ba
    f32 = 2.0 ** -19
    check("y", y, ref, step * ref.abs() + f32 * n * za * (1 if gate else n + 1))
    du = dy.double().abs() * (za if gate else n + 1)
    dh = (du * wa).reshape(rows, groups, D)
    size = (rstd * (dh + dh.mean(-1, keepdim=True) + xh.abs() * (dh * xh.abs()).mean(-1, keepdim=True)))
    size = size.reshape(rows, -1) * amp
    check("dx", dx, rx, step * rx.abs() + f32 * size * amp)
    if gate:
        check("dz", dz, rz, step * rz.abs() + f32 * dy.double().abs() * n * (za + 1))
    else:
        assert dz is None
    if affine:
        check("dw", dw, rw, (f32 + rows * 2.0 ** -24) * (du * amp * (1 if gate else amp)).sum(0))
        check("db", db, rb, (f32 + rows * 2.0 ** -24) * (du * (1 if gate else amp)).sum(0))
    else:
        assert dw is None and db is None


def test_gradient_against_differences():
    x, z, w, b, dy = draw(6, 2, 24, F32, 3, True, True)
    args = dict(x=x.double(), z=z.double(), w=w.double(), b=b.double())
    grads = G.group_norm_bwd(gpu(dy), gpu(x), 2, gpu(w), gpu(b), gate=gpu(z))

    def loss(a):
        return float((group_norm(a["x"], 2, a["w"], a["b"], a["z"], "silu", True, 1e-5) * dy.double()).sum())

    gen = torch.Generator().manual_seed(4)
    for name, grad in zip(("x", "z", "w", "b"), grads):
        u = torch.randn(args[name].shape, generator=gen, dtype=torch.float64)
        want = (loss({**args, name: args[name] + 1e-5 * u}) - loss({**args, name: args[name] - 1e-5 * u})) / 2e-5
        got = (grad.cpu().double() * u)
        assert abs(want - float(got.sum())) <= 1e-4 * float(got.norm()) + 1e-6, name


def test_strides_and_in_place():
    """Slices of wider rows (aligned or not) and outputs on top of inputs: bit for bit where the units are the
    same, to one rounding step where they are not."""
    rows, groups, D = 50, 4, 64
    C = groups * D
    x, z, w, b, dy = draw(rows, groups, D, BF16, 9, True, True)
    kw = dict(weight=gpu(w), bias=gpu(b))
    want = G.group_norm_fwd(gpu(x), groups, gate=gpu(z), **kw)
    for off in (8, 3):
        wide = torch.zeros(2, 30, 2 * C + 16, dtype=BF16, device=DEV)
        xs, zs = wide[:, :25, off:off + C], wide[:, :25, off + C:off + 2 * C]
        xs.copy_(gpu(x).view(2, 25, C))
        zs.copy_(gpu(z).view(2, 25, C))
        y = G.group_norm_fwd(xs, groups, gate=zs, **kw).view(rows, C)
        if off == 8:
            assert torch.equal(y, want)
        else:
            assert ((y.double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 1e-6).all()
        dys = wide[:, :25, off:off + C].clone()
        a = G.group_norm_bwd(dys, xs, groups, gate=zs, **kw)
        assert all(torch.isfinite(t).all() for t in a)
    for nm in ("x", "z"):
        xi, zi = gpu(x).clone(), gpu(z).clone()
        G.group_norm_fwd(xi, groups, gate=zi, out=xi if nm == "x" else zi, **kw)
        assert torch.equal(xi if nm == "x" else zi, want)


def test_edges():
    """Constant rows, large values, gates far out, and no rows."""
    x = torch.full((3, 64), 4.0, dtype=BF16, device=DEV)
    assert not G.group_norm_fwd(x, 1, activation="none").any()
    big = torch.full((2, 128), 1e18, device=DEV)
    y = G.group_norm_fwd(big, 2, activation="none", centered=False)
    assert ((y - 1).abs() <= 2.0 ** -20).all()
    z = torch.tensor([[-200.0, 200.0, -90.0, 0.0]], device=DEV)
    ones = torch.tensor([[1.0, 1.0, -1.0, -1.0]], device=DEV)
    y = G.group_norm_fwd(ones, 1, gate=z, activation="sigmoid", eps=0.0)
    assert torch.allclose(y.cpu(), torch.tensor([[0.0, 1.0, 0.0, -0.5]]), atol=1e-6)
    y = G.group_norm_fwd(ones, 1, gate=z, activation="silu", eps=0.0)
    assert torch.isfinite(y).all()
    empty = torch.zeros(0, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    assert G.group_norm_fwd(empty, 4, w).shape == (0, 64)
    dx, dz, dw, db = G.group_norm_bwd(empty, empty, 4, w, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_streams_and_graph():
    x, z, w, b, dy = (gpu(t) for t in draw(700, 8, 128, BF16, 11, True, True))

    def step():
        return (G.group_norm_fwd(x, 8, w, b, gate=z),) + G.group_norm_bwd(dy, x, 8, w, b, gate=z)

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        x.copy_(torch.randn(x.shape, device=DEV))
        dy.copy_(torch.randn(x.shape, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(step(), got))
