"""Measured cases of the linear-attention and group-norm operators.

Linear attention with a decay for each head:  S_t = e^{g_t} S_{t-1} + v_t k_t^T  and  o_t = scale S_t q_t, with H key
heads and HV value heads (HV a multiple of H), g a natural-log decay per token [B, T, HV] or per head [HV]:

  fwd      a prompt (equal-length rows, or packed requests with cu_seqlens) -> o and the final states
  bwd      its gradients: dq, dk, dv, dg, and dh0 of the initial states
  decode   S new tokens of each request, the state updated in its slot of a pool

Group norm with an activation, channels last, every token a sample of its own:

  norm     y = (group_norm(x) w + b) act(z), or act(group_norm(x) w + b) without a gate z
  normbwd  its gradients: dx, dz, dw, db

``run`` computes them in plain torch operations, or with ``own`` by the package's entry points.
"""
import math
import random

import torch

own = False

CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def _fwd(name, B, T, H, HV, K, V, dtype="bf16", decay="token", lens="", h0=False):
    return dict(name=name, op="fwd", B=B, T=T, H=H, HV=HV, K=K, V=V, dtype=dtype, decay=decay, lens=lens, h0=h0)


def _bwd(name, B, T, H, HV, K, V, dtype="bf16", decay="token", lens="", h0=False):
    return dict(_fwd(name, B, T, H, HV, K, V, dtype, decay, lens, h0), op="bwd")


def _decode(name, n, S, H, HV, K, V, dtype="bf16", decay="token", pad=0):
    return dict(name=name, op="decode", n=n, S=S, H=H, HV=HV, K=K, V=V, dtype=dtype, decay=decay, pad=pad)


def _norm(name, op, rows, groups, D, dtype="bf16", gate=True, act="silu", centered=True, bias=True):
    return dict(name=name, op=op, rows=rows, groups=groups, D=D, dtype=dtype, gate=gate, act=act, centered=centered,
                bias=bias)


def listed():
    return [
        # a short prompt in float32: the smallest call, where launches count
        _fwd("fwd_short_f32", 1, 128, 2, 2, 64, 64, "f32"),
        # a serving step's packed prompts of ragged lengths, shared key heads, continued from cached states
        _fwd("fwd_packed_gva", 1, 15151, 4, 16, 128, 128, lens="1261,821,2415,1099,1206,2059,3562,2728", h0=True),
        # one long prompt with fixed decays per head
        _fwd("fwd_long_32k", 1, 32768, 16, 16, 128, 128, decay="head"),
        # a training step of a small batch
        _bwd("bwd_batch_1k", 2, 1024, 8, 8, 128, 128),
        # training on packed documents of odd lengths, shared key heads, with initial states
        _bwd("bwd_packed_gva", 1, 15151, 4, 16, 128, 128, lens="1261,821,2415,1099,1206,2059,3562,2728", h0=True),
        # training on long rows with wide value heads and fixed decays
        _bwd("bwd_wide_8k", 1, 8192, 32, 32, 128, 256, decay="head"),
        # one request's next token: latency
        _decode("decode_1", 1, 1, 16, 16, 128, 128),
        # a full serving batch with padding entries and shared key heads
        _decode("decode_256_gva", 256, 1, 4, 16, 128, 128, pad=5),
        # the output norm of a decode step
        _norm("norm_decode_256", "norm", 256, 16, 128),
        # the output norm of a long prompt
        _norm("norm_32k", "norm", 32768, 16, 128),
        # its gradients in a small training step, no gate
        _norm("normbwd_2k", "normbwd", 2048, 8, 128, gate=False),
        # its gradients on a long row, gated
        _norm("normbwd_32k", "normbwd", 32768, 16, 128),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "decode", "decode", "norm", "normbwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm", "normbwd"):
        groups, D = rng.choice([1, 2, 3, 4, 8, 16, 24]), rng.choice([40, 64, 80, 96, 128, 160, 256])
        rows = _logint(rng, 1, 48e6 / (groups * D) if dtype == "bf16" else 24e6 / (groups * D))
        return dict(op=op, rows=rows, groups=groups, D=D, dtype=dtype, gate=rng.random() < 0.7,
                    act=rng.choice(["silu", "silu", "sigmoid", "none"]), centered=rng.random() < 0.6,
                    bias=rng.random() < 0.6)
    K, V, H = rng.choice([64, 128, 128]), rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 3, 4, 8])
    HV, decay = H * rng.choice([1, 1, 2, 4]), rng.choice(["token", "token", "head"])
    if op == "decode":
        n = _logint(rng, 1, min(512, 4096 // HV))
        return dict(op=op, n=n, S=rng.choice([1, 1, 1, 2, 4]), H=H, HV=HV, K=K, V=V, dtype=dtype, decay=decay,
                    pad=min(n - 1, rng.choice([0, 0, 1, 7])))
    most = (65536 if op == "fwd" else 32768) * 128 // max(K, V) // HV
    T, lens, B = _logint(rng, 1, min(16384, most)), "", 1
    if rng.random() < 0.5 and T >= 16:
        part = [rng.uniform(0.5, 1.5) for _ in range(rng.randint(2, 7))]
        cut = [max(1, int(T * p / sum(part))) for p in part]
        lens, T = ",".join(str(c) for c in cut), sum(cut)
    elif rng.random() < 0.5:
        B = rng.randint(1, 4)
        T = max(1, T // B)
    return dict(op=op, B=B, T=T, H=H, HV=HV, K=K, V=V, dtype=dtype, decay=decay, lens=lens, h0=rng.random() < 0.5)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if case["lens"] else [case["T"]] * case["B"]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "normbwd"):
        n = case["rows"] * case["groups"] * case["D"]
        gate = case["gate"]
        if case["op"] == "norm":
            return {"bytes": n * es * (3 if gate else 2), "flops": n * (12 if gate else 8)}
        return {"bytes": n * es * (5 if gate else 3), "flops": n * (30 if gate else 20)}
    H, HV, K, V = case["H"], case["HV"], case["K"], case["V"]
    if case["op"] == "decode":
        n, S = case["n"], case["S"]
        live = n - case["pad"]
        rows = n * S * (2 * H * K + 2 * HV * V) * es + (n * S * HV * 4 if case["decay"] == "token" else HV * 4)
        return {"bytes": rows + live * HV * K * V * 8, "flops": live * S * HV * K * V * 5}
    tok, nseq = case["B"] * case["T"], len(_lens(case))
    g = tok * HV * 4 if case["decay"] == "token" else HV * 4
    state = nseq * HV * K * V * 4
    if case["op"] == "fwd":
        return {"bytes": tok * (2 * H * K + 2 * HV * V) * es + g + state * (2 if case["h0"] else 1),
                "flops": 4 * tok * HV * K * V}
    return {"bytes": tok * (4 * H * K + 3 * HV * V) * es + 2 * g + state * (3 if case["h0"] else 0),
            "flops": 10 * tok * HV * K * V}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    s = dict(case)
    if case["op"] in ("norm", "normbwd"):
        rows, C = case["rows"], case["groups"] * case["D"]
        s["x"] = (normal(rows, C) * (0.25 + uniform(rows, 1)) + 0.5 * normal(1, C)).to(dt)
        s["z"] = normal(rows, C).to(dt) if case["gate"] else None
        s["w"] = 1.0 + 0.2 * normal(C)
        s["b"] = 0.2 * normal(C) if case["bias"] else None
        if case["op"] == "normbwd":
            s["dy"] = normal(rows, C).to(dt)
        return s
    H, HV, K, V = case["H"], case["HV"], case["K"], case["V"]
    n, T = (case["n"], case["S"]) if case["op"] == "decode" else (case["B"], case["T"])

    def directions(*shape):  # queries and keys on the unit sphere, as the package's workloads have them
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    s["q"], s["k"], s["v"] = directions(n, T, H, K), directions(n, T, H, K), normal(n, T, HV, V).to(dt)
    if case["decay"] == "head":  # fixed decays from fast heads to slow ones
        s["g"] = torch.log1p(-torch.exp2(-2.0 - 7.0 * torch.arange(HV, device="cuda") / HV))
    else:  # -A softplus(a + dt_bias): rates 1..16, step sizes around 0.001 to 0.1
        rate, step = 1.0 + 15.0 * uniform(HV), torch.exp(math.log(0.001) + math.log(100.0) * uniform(HV))
        s["g"] = -rate * torch.nn.functional.softplus(normal(n, T, HV) + torch.log(torch.expm1(step)))
    if case["op"] == "decode":
        pool = n + 3
        slots = torch.randperm(pool, generator=gen, device="cuda")[:n].to(torch.int32)
        order = list(range(n))
        random.Random(int(seed)).shuffle(order)
        live = sorted(order[case["pad"]:])
        slots[order[:case["pad"]]] = -1
        s["slots"], s["live"] = slots, torch.tensor(live, device="cuda")
        s["state"] = 0.3 * normal(pool, HV, V, K)
        return s
    lens = _lens(case)
    s["max_len"] = max(lens)
    s["cu"] = None
    if case["lens"]:
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    s["h0"] = 0.3 * normal(len(lens), HV, V, K) if case["h0"] else None
    if case["op"] == "bwd":
        s["do"] = normal(n, T, HV, V).to(dt)
        s["dht"] = 0.1 * normal(len(lens), HV, V, K) if case["h0"] else None
    return s


# ------------------------------------------------------------------ the plain forms

def _rows(s, x):
    """Packed rows [1, T, ...] as padded sequences [nseq, max_len, ...]; padding is zero."""
    if s["cu"] is None:
        return x
    at = s["cu"][:-1, None].long() + torch.arange(s["max_len"], device=x.device)
    inside = at < s["cu"][1:, None]
    x = x[0][at.clamp(max=x.shape[1] - 1)]
    return x * inside.view(*inside.shape, *([1] * (x.dim() - 2)))


def _packed(s, x):
    """The packed rows [1, T, ...] of padded sequences."""
    if s["cu"] is None:
        return x
    inside = torch.arange(s["max_len"], device=x.device) < (s["cu"][1:] - s["cu"][:-1])[:, None]
    at = inside.reshape(-1).to(torch.uint8).argsort(descending=True, stable=True)[: s["T"]]
    return x.reshape(-1, *x.shape[2:])[at][None]


def _heads(x):
    """[n, T, heads, D] -> [n * heads, T, D] float32."""
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3]).float()


def _decayed(a, b, c, g, s0, x=None):
    """y_i = sum_{j<=i} D(i,j) (a_i . b_j) c_j + D(i,start) s0 a_i in chunks, and the state after the last row.

    a, b [N, L, A], c [N, L, C] and s0 of one type; g [N, L] float64 log decays; s0 [N, C, A] or None.  With x [N, L, C] also
    x_i . (y_i without its j = i term): what the decays scale."""
    N, L = g.shape
    nc = -(-L // CHUNK)
    pad = nc * CHUNK - L

    def chunks(x):
        return torch.nn.functional.pad(x, (0, 0, 0, pad)).reshape(N * nc, CHUNK, -1)

    a, b, c = chunks(a), chunks(b), chunks(c)
    G = torch.nn.functional.pad(g, (0, pad)).reshape(N * nc, CHUNK).cumsum(1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=a.device).tril()
    D = (G[:, :, None] - G[:, None, :]).masked_fill(~low, -math.inf).exp().to(a.dtype)
    y = ((a @ b.transpose(1, 2)) * D) @ c
    E = (c * (G[:, -1:] - G).exp().to(a.dtype)[..., None]).transpose(1, 2) @ b  # [N * nc, C, A]
    P = torch.nn.functional.pad(G[:, -1].reshape(N, nc).cumsum(1), (1, 0))  # decay before each boundary
    low = torch.ones(nc + 1, nc, dtype=torch.bool, device=a.device).tril(-1)
    W = (P[:, :, None] - P[:, None, 1:]).masked_fill(~low, -math.inf).exp().to(a.dtype)
    S = (W @ E.reshape(N, nc, -1)).reshape(N, nc + 1, *E.shape[1:])  # the state entering each chunk, and the last
    if s0 is not None:
        S = S + P.exp().to(a.dtype)[:, :, None, None] * s0[:, None]
    before = (a @ S[:, :-1].reshape(N * nc, *E.shape[1:]).transpose(1, 2)) * G.exp().to(a.dtype)[..., None]
    y = (y + before).reshape(N, nc * CHUNK, -1)[:, :L]
    if x is None:
        return y, S[:, -1]
    x = chunks(x)
    inner = ((a @ b.transpose(1, 2)) * D * (x @ c.transpose(1, 2))).tril(-1).sum(-1)
    return y, S[:, -1], (inner.double() + (x * before).sum(-1)).reshape(N, -1)[:, :L]


def _token_decay(s, B, T):
    return s["g"].expand(B, T, -1) if s["g"].dim() == 1 else s["g"]


def _inputs(s):
    r = s["HV"] // s["H"]
    g = _rows(s, _token_decay(s, s["B"], s["T"])).transpose(1, 2)
    q, k, v = (_heads(_rows(s, x)) for x in (s["q"].repeat_interleave(r, 2), s["k"].repeat_interleave(r, 2), s["v"]))
    h0 = None if s["h0"] is None else s["h0"].reshape(-1, s["V"], s["K"])
    return q, k, v, g.reshape(-1, g.shape[-1]).double(), h0


def _plain_fwd(s):
    q, k, v, g, h0 = _inputs(s)
    y, S = _decayed(q * s["K"] ** -0.5, k, v, g, h0)
    o = y.reshape(-1, s["HV"], *y.shape[1:]).transpose(1, 2)
    return _packed(s, o).to(s["v"].dtype), S.reshape(-1, s["HV"], s["V"], s["K"])


def _plain_bwd(s):
    HV, r, dt = s["HV"], s["HV"] // s["H"], s["v"].dtype
    q, k, v, g, h0 = _inputs(s)
    q = q * s["K"] ** -0.5
    do = _heads(_rows(s, s["do"]))
    lens = s["cu"][1:] - s["cu"][:-1] if s["cu"] is not None else torch.full((s["B"],), s["T"], device=q.device)
    dht = None if s["dht"] is None else s["dht"].reshape(-1, s["V"], s["K"])

    def swap(x):
        return None if x is None else x.transpose(1, 2)

    # a per-head decay's gradient is a sum over every row of what nearly cancels: in 64 bits
    q_, k_, v_, do_, h0_, dht_ = ((x.double() if x is not None and s["g"].dim() == 1 else x)
                                  for x in (q, k, v, do, h0, dht))
    dq, _, rows_q = _decayed(do_, v_, k_, g, swap(h0_), q_)
    # backwards in time: padded rows come first there, with zero keys and decays, and leave dht as it is
    back = torch.nn.functional.pad(g[:, 1:], (0, 1)).flip(1)
    dk, _, rows_k = _decayed(v_.flip(1), do_.flip(1), q_.flip(1), back, swap(dht_), k_.flip(1))
    dv, R = _decayed(k.flip(1), q.flip(1), do.flip(1), back, dht)
    dk, dv = dk.flip(1), dv.flip(1)
    # dg_t, the pairs of a row at or after t and one before it: what the rows s >= t take from earlier ones less what
    # they give to later ones, plus the final states' share, in 64 bits (long sums)
    _, ST = _decayed(q_, k_, v_, g, h0_)
    dG = (rows_q - rows_k.flip(1)).flip(1).cumsum(1).flip(1)
    if dht is not None:
        dG = dG + (ST.double() * dht).sum((1, 2))[:, None]
    inside = torch.arange(g.shape[1], device=q.device) < lens[:, None]
    dG = dG.reshape(-1, HV, dG.shape[1]).transpose(1, 2) * inside[..., None]

    def rows(x, heads):
        x = x.reshape(-1, HV, *x.shape[1:]).transpose(1, 2)
        if heads < HV:
            x = x.reshape(*x.shape[:2], heads, r, -1).sum(3)
        return _packed(s, x).to(dt)

    dg = dG.sum((0, 1)).float() if s["g"].dim() == 1 else _packed(s, dG).float()
    dh0 = None if h0 is None else (R * g[:, :1].exp().float()[..., None]).reshape(-1, HV, s["V"], s["K"])
    return rows(dq * s["K"] ** -0.5, s["H"]), rows(dk, s["H"]), rows(dv, HV), dg, dh0


def _plain_decode(s):
    n, S, HV, K, V, r = s["n"], s["S"], s["HV"], s["K"], s["V"], s["HV"] // s["H"]
    live, at = s["live"], s["slots"][s["live"]].long()
    q, k, v = (_heads(x[live]) for x in (s["q"].repeat_interleave(r, 2), s["k"].repeat_interleave(r, 2), s["v"]))
    G = _token_decay(s, n, S)[live].transpose(1, 2).reshape(-1, S).double().cumsum(1)
    old = s["state"][at].reshape(-1, V, K)
    low = torch.ones(S, S, dtype=torch.bool, device=q.device).tril()
    D = (G[:, :, None] - G[:, None, :]).masked_fill(~low, -math.inf).exp().float()
    q = q * K ** -0.5
    y = ((q @ k.transpose(1, 2)) * D) @ v + (q @ old.transpose(1, 2)) * G.exp().float()[..., None]
    new = old * G[:, -1:].exp().float()[..., None] + (v * (G[:, -1:] - G).exp().float()[..., None]).transpose(1, 2) @ k
    s["state"][at] = new.reshape(-1, HV, V, K)
    o = torch.zeros(n, S, HV, V, dtype=s["v"].dtype, device=q.device)
    o[live] = y.reshape(-1, HV, S, V).transpose(1, 2).to(o.dtype)
    return o, s["state"]


def _act(name, x):
    if name == "none":
        return x
    return torch.sigmoid(x) * x if name == "silu" else torch.sigmoid(x)


def _act_slope(name, x):
    if name == "none":
        return torch.ones_like(x)
    y = torch.sigmoid(x)
    return y * (1 + x * (1 - y)) if name == "silu" else y * (1 - y)


EPS = 1e-5


def _normed(s):
    x = s["x"].float().reshape(s["rows"], s["groups"], s["D"])
    if s["centered"]:
        x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * rstd, rstd


def _plain_norm(s):
    xh, _ = _normed(s)
    n = xh.reshape(s["rows"], -1) * s["w"]
    if s["b"] is not None:
        n = n + s["b"]
    y = n * _act(s["act"], s["z"].float()) if s["gate"] else _act(s["act"], n)
    return y.to(s["x"].dtype)


def _plain_normbwd(s):
    xh, rstd = _normed(s)
    flat = xh.reshape(s["rows"], -1)
    n = flat * s["w"]
    if s["b"] is not None:
        n = n + s["b"]
    dy, dz = s["dy"].float(), None
    if s["gate"]:
        z = s["z"].float()
        dz = (dy * n * _act_slope(s["act"], z)).to(s["x"].dtype)
        dn = dy * _act(s["act"], z)
    else:
        dn = dy * _act_slope(s["act"], n)
    dh = (dn * s["w"]).reshape(xh.shape)
    dx = dh - xh * (dh * xh).mean(-1, keepdim=True)
    if s["centered"]:
        dx = dx - dh.mean(-1, keepdim=True)
    dx = (dx * rstd).reshape(s["rows"], -1).to(s["x"].dtype)
    return dx, dz, (dn * flat).double().sum(0).float(), None if s["b"] is None else dn.double().sum(0).float()


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if own:
        from gated_delta_product_amd import binding
        if op == "fwd":
            return binding.linattn_fwd(s["q"], s["k"], s["v"], s["g"], cu_seqlens=s["cu"], initial_state=s["h0"],
                                       output_final_state=True)
        if op == "bwd":
            return binding.linattn_bwd(s["do"], s["q"], s["k"], s["v"], s["g"], cu_seqlens=s["cu"],
                                       initial_state=s["h0"], dht=s["dht"])
        if op == "decode":
            return binding.linattn_decode(s["q"], s["k"], s["v"], s["state"], s["g"], slots=s["slots"]), s["state"]
        if op == "norm":
            return binding.group_norm_fwd(s["x"], s["groups"], s["w"], s["b"], gate=s["z"], activation=s["act"],
                                          centered=s["centered"], eps=EPS)
        return binding.group_norm_bwd(s["dy"], s["x"], s["groups"], s["w"], s["b"], gate=s["z"], activation=s["act"],
                                      centered=s["centered"], eps=EPS)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "decode": _plain_decode, "norm": _plain_norm,
            "normbwd": _plain_normbwd}[op](s)


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _exact_linear(case, s):
    """The recurrence token by token over padded sequences, forwards for S (o, dq) and backwards for its gradient."""
    HV, r = case["HV"], case["HV"] // case["H"]
    lens = _lens(case)
    L, n = max(lens), len(lens)
    dev = s["v"].device

    def rows(x):
        x = x.double()
        if not case["lens"]:
            return x
        out = torch.zeros(n, L, *x.shape[2:], dtype=torch.float64, device=dev)
        start = 0
        for i, m in enumerate(lens):
            out[i, :m] = x[0, start:start + m]
            start += m
        return out

    def packed(x):
        return torch.cat([x[i, :m] for i, m in enumerate(lens)])[None] if case["lens"] else x

    g = s["g"] if s["g"].dim() == 3 else s["g"].view(1, 1, -1).expand(case["B"], case["T"], HV)
    q, k, v, g = rows(s["q"]), rows(s["k"]), rows(s["v"]), rows(g)
    q, k = (x.unsqueeze(3).expand(*x.shape[:3], r, x.shape[3]).flatten(2, 3) * f
            for x, f in ((q, 1.0 / math.sqrt(case["K"])), (k, 1.0)))
    alpha = torch.exp(g)
    S = torch.zeros(n, HV, case["V"], case["K"], dtype=torch.float64, device=dev) if s["h0"] is None else s["h0"].double()
    back = case["op"] == "bwd"
    do = rows(s["do"]) if back else None
    out = []
    taken = []
    for t in range(L):
        S = S * alpha[:, t, :, None, None]
        if back:
            taken.append((do[:, t] * (S @ q[:, t, :, :, None])[..., 0]).sum(2))
        S = S + v[:, t, :, :, None] * k[:, t, :, None, :]
        out.append((do[:, t, :, None, :] @ S)[..., 0, :] if back else (S @ q[:, t, :, :, None])[..., 0])
    out = torch.stack(out, 1)
    if not back:
        return packed(out), S
    R = torch.zeros_like(S) if s["dht"] is None else s["dht"].double()
    end = (S * R).sum((2, 3))  # what every decay of the row scales: the final state's share
    dk, dv, given = [None] * L, [None] * L, [None] * L
    for t in range(L - 1, -1, -1):
        given[t] = (v[:, t] * (R @ k[:, t, :, :, None])[..., 0]).sum(2)
        R = R + do[:, t, :, :, None] * q[:, t, :, None, :]
        dk[t], dv[t] = (v[:, t, :, None, :] @ R)[..., 0, :], (R @ k[:, t, :, :, None])[..., 0]
        R = R * alpha[:, t, :, None, None]
    dk, dv = torch.stack(dk, 1), torch.stack(dv, 1)
    change = torch.stack(taken, 1) - torch.stack(given, 1)
    dg = torch.flip(torch.cumsum(torch.flip(change, [1]), 1), [1]) + end[:, None]
    for i, m in enumerate(lens):
        dg[i, m:] = 0
    per_head = [x.unflatten(2, (case["H"], r)).sum(3) for x in (out / math.sqrt(case["K"]), dk)]
    dg = dg.sum((0, 1)) if s["g"].dim() == 1 else packed(dg)
    return packed(per_head[0]), packed(per_head[1]), packed(dv), dg, None if s["h0"] is None else R


def _exact_decode(case, s):
    r = case["HV"] // case["H"]
    state, o = s["state"].double(), torch.zeros(s["v"].shape, dtype=torch.float64, device=s["v"].device)
    q, k = (x.double().repeat_interleave(r, 2) for x in (s["q"], s["k"]))
    g = s["g"].double().expand(case["n"], case["S"], case["HV"])
    S = state[s["slots"].clamp(min=0).long()]
    for t in range(case["S"]):
        S = torch.exp(g[:, t, :, None, None]) * S + s["v"].double()[:, t, :, :, None] * k[:, t, :, None, :]
        o[:, t] = (S * q[:, t, :, None, :]).sum(-1) / math.sqrt(case["K"])
    o[s["slots"] < 0] = 0
    state[s["slots"][s["live"]].long()] = S[s["live"]]
    return o, state


def _exact_norm(case, s):
    x = s["x"].double().requires_grad_()
    w = s["w"].double().requires_grad_()
    b = s["b"].double().requires_grad_() if s["b"] is not None else None
    z = s["z"].double().requires_grad_() if s["gate"] else None
    u = x.unflatten(1, (case["groups"], case["D"]))
    mean = u.sum(2, keepdim=True) / case["D"] if case["centered"] else 0.0
    var = ((u - mean) ** 2).sum(2, keepdim=True) / case["D"]
    n = ((u - mean) / torch.sqrt(var + EPS)).flatten(1) * w
    n = n if b is None else n + b
    pre = z if z is not None else n
    gate = {"none": lambda a: a, "sigmoid": lambda a: 1 / (1 + torch.exp(-a)),
            "silu": lambda a: a / (1 + torch.exp(-a))}[case["act"]](pre)
    y = n * gate if z is not None else gate
    if case["op"] == "norm":
        return y.detach()
    leaves = [t for t in (x, z, w, b) if t is not None]
    grads = iter(torch.autograd.grad(y, leaves, s["dy"].double()))
    return tuple(next(grads) if t is not None else None for t in (x, z, w, b))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "normbwd"):
        return _exact_norm(case, s)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    return _exact_linear(case, s)
