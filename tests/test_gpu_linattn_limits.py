"""The largest sizes that linear attention accepts in a direction, and what the
documentation allows beside the usual calls, on the GPU."""
import pytest
import torch

from gated_delta_product_amd import binding as G
from linref import Linear, inv_sqrt
from test_gpu_linattn import BF16, DEV, F32, draws, gpu, within

pytestmark = pytest.mark.gpu


def test_most_heads():
    """HV max(K, V) = 2^22: 65536 heads, three of them against their plain form."""
    HV, K = 65536, 64
    d = draws(61, [2], HV, HV, K, K, F32, "head", False, 1)
    d["g"] = -torch.rand(HV, generator=torch.Generator().manual_seed(62))
    t = {k: gpu(v) if torch.is_tensor(v) else v for k, v in d.items()}
    o, ht = G.linattn_fwd(t["q"], t["k"], t["v"], t["g"], output_final_state=True)
    state = torch.zeros(1, HV, K, K, device=DEV)
    step = G.linattn_decode(t["q"], t["k"], t["v"], state, t["g"])
    for h in (0, 32767, HV - 1):
        r = Linear(*(d[x][0, :, h:h + 1] for x in ("q", "k", "v")), d["g"][h:h + 1].expand(2, 1), inv_sqrt(K))
        (ro, rs), (ao, a_s) = r.forward(), r.forward_abs()
        for x, s in ((o, ht), (step, state)):
            within("o", x[0, :, h:h + 1], ro, ao, 2 + K, F32)
            within("S", s[0, h:h + 1], rs, a_s, 2 + K, F32)


def test_two_calls_at_once():
    """Two calls on two streams, each with a workspace of its own, give what they give one after the other."""
    calls = []
    for seed, lens, K, V, decay in ((63, [1900, 300], 128, 128, "head"), (64, [700, 900, 1], 64, 256, "token")):
        d = {k: gpu(v) if torch.is_tensor(v) else v for k, v in draws(seed, lens, 2, 4, K, V, BF16, decay).items()}
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
        calls.append((d, cu))

    def step(d, cu):
        ins = [d[x] for x in ("q", "k", "v", "g")]
        o, ht = G.linattn_fwd(*ins, cu_seqlens=cu, initial_state=d["h0"], output_final_state=True)
        return (o, ht) + G.linattn_bwd(d["do"], *ins, cu_seqlens=cu, initial_state=d["h0"], dht=d["dht"])

    want = [step(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = []
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(step(*c))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for a, b in zip(want, got) for x, y in zip(a, b))


def test_graph_of_a_decay_per_head():
    """Gradients of a decay per head over spans, captured and replayed with eager work between."""
    lens = [1500, 700]
    d = {k: gpu(v) if torch.is_tensor(v) else v for k, v in draws(65, lens, 24, 24, 128, 256, BF16, "head").items()}
    cu = torch.tensor([0, 1500, 2200], dtype=torch.int32, device=DEV)

    def step():
        return G.linattn_bwd(d["do"], d["q"], d["k"], d["v"], d["g"], cu_seqlens=cu, initial_state=d["h0"], dht=d["dht"])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(3):
        d["v"].copy_(torch.randn(d["v"].shape, device=DEV))
        d["g"].copy_(-torch.rand(24, device=DEV))
        cu.copy_(torch.tensor([0, 1500 - 700 * k, 2200], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got)), k
