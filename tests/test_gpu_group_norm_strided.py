"""Gradients of the group norm through slices of wider rows, held against the
same call on contiguous tensors.

Where rows start on 16 bytes the kernel is the same: bit for bit.  Elsewhere
lanes hold single elements, so float32 sums run in another order.  With E the
bound of test_gpu_group_norm on the float32 steps (2^-19 of the sums of absolute
values behind a value), each side is within E of the exact value before its
last rounding and within half a step after it: 2 E plus a step of the value
(2^-7 in bf16, 2^-23 in float32).  dweight and dbias sum `rows` such terms: 2 (2^-19
+ rows 2^-24) of the absolute sum."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from test_gpu_group_norm import BF16, DEV, F32, draw, gpu

pytestmark = pytest.mark.gpu


def sliced(t, off, lead):
    """The rows of t [rows, C] as a [lead, rows / lead, C] slice of wider ones, starting at element off."""
    rows, C = t.shape
    wide = torch.full((lead, rows // lead + 2, C + 24), float("nan"), dtype=t.dtype, device=DEV)
    x = wide[:, 1:1 + rows // lead, off:off + C]
    x.copy_(gpu(t).view(lead, rows // lead, C))
    return x


@pytest.mark.parametrize("which", ["x", "z", "dy", "all"])
@pytest.mark.parametrize("off", [8, 3])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("groups,D,gate", [(4, 64, True), (3, 40, False), (2, 256, True), (1, 7, True)])
def test_gradients_of_slices(groups, D, gate, dtype, off, which):
    if which == "z" and not gate:
        which = "x"
    rows, lead = 50, 2
    x, z, w, b, dy = draw(rows, groups, D, dtype, 13, gate, True)
    kw = dict(weight=gpu(w), bias=gpu(b))
    want = G.group_norm_bwd(gpu(dy), gpu(x), groups, gate=gpu(z), **kw)

    def part(name, t):
        return None if t is None else sliced(t, off, lead) if which in (name, "all") else gpu(t).view(lead, rows // lead, -1)

    got = G.group_norm_bwd(part("dy", dy), part("x", x), groups, gate=part("z", z), **kw)
    if off % (16 // x.element_size()) == 0 and (D * x.element_size()) % 16 == 0:
        for p, q in zip(got, want):
            assert (p is None and q is None) or torch.equal(p.reshape(q.shape), q)
        return
    u = x.double().reshape(rows, groups, D)
    c = u - u.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5)
    xh = (c * rstd).abs()
    amp = xh.amax(-1, keepdim=True) + 1 + u.abs().amax(-1, keepdim=True) * rstd  # as test_gpu_group_norm has it
    n = w.double().abs().view(groups, D) * amp + b.double().abs().view(groups, D)
    g = dy.double().abs().reshape(rows, groups, D)
    za = z.double().abs().reshape(rows, groups, D) + 1 if gate else n + 1
    du = g * za
    dh = du * w.double().abs().view(groups, D)
    size = rstd * (dh + dh.mean(-1, keepdim=True) + xh * (dh * xh).mean(-1, keepdim=True)) * amp * amp
    f32, step = 2.0 ** -19, 2.0 ** -7 if dtype == BF16 else 2.0 ** -23
    many = f32 + rows * 2.0 ** -24
    back = amp if not gate else 1
    bounds = (f32 * size, f32 * g * n * (za + 1) if gate else None, many * (du * amp * back).sum(0), many * (du * back).sum(0))
    for i, (p, q, e) in enumerate(zip(got, want, bounds)):
        if q is None:
            assert p is None
            continue
        p, q = p.reshape(q.shape).double().cpu(), q.double().cpu()
        tol = 2 * e.reshape(q.shape) + (step if i < 2 else 2.0 ** -23) * q.abs()
        assert torch.isfinite(p).all() and bool(((p - q).abs() <= tol).all()), (i, float(((p - q).abs() / tol).max()))
