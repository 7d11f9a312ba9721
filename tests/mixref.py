"""Plain 64-bit forms of the gated linear recurrence, the short causal
convolution and rotary positions, sequence by sequence, and bounds of their
float32 rounding.  Only tests import this.

A bound counts what a float32 evaluation in any order of the same sums may be
off by: U = 2^-24 for each rounding, taken of the sums over absolute values."""
import math

import torch

U = 2.0 ** -24
# e^g of a g below -87.3 lies under float32's normal numbers, where the hardware's power keeps or drops it: a decay is
# then off by at most the smallest of them, however small it is itself
TINY = 2.0 ** -126


def half_step(dtype):
    """Largest rounding of a stored value, relative."""
    return torch.finfo(dtype).eps / 2


def spans(rows, cu=None, B=1):
    """[(first, end)] of the sequences over the rows [B*T]."""
    if cu is None:
        T = rows // B if B else 0
        return [(b * T, (b + 1) * T) for b in range(B)]
    out = []
    for a, b in zip(cu[:-1], cu[1:]):
        a = min(max(a, 0), rows)
        out.append((a, min(max(b, a), rows)))
    return out


def gates(g, decay):
    """a and 1 - a."""
    return (torch.exp(g), -torch.expm1(g)) if decay == "log" else (torch.sigmoid(g), torch.sigmoid(-g))


class Rec:
    """x, g [rows, C], seqs [(first, end)], h0 [nseq, C] or None.

    Of rows in bfloat16 the kernels keep 1 - a (`short`): off by a few U of itself, by the power's (2 + |g|) U of a (of
    a (1 - a) behind a sigmoid), and a state that it decays by a U of the state."""

    def __init__(self, x, g, seqs, decay, complement, h0=None):
        self.x, self.seqs, self.decay, self.comp = x.double(), seqs, decay, complement
        self.a, self.s = gates(g.double(), decay)
        C = x.shape[1]
        self.h0 = torch.zeros(len(seqs), C, dtype=torch.float64) if h0 is None else h0.double()
        self.c = self.s if complement else torch.ones_like(self.s)
        n = x.shape[0]
        # state before each row, after it, the same over absolute values, and the rounding of the state after it
        self.prev, self.h, self.prev_abs, self.h_abs, self.err = (torch.zeros(n, C, dtype=torch.float64) for _ in range(5))
        self.prev_err = torch.zeros(n, C, dtype=torch.float64)
        self.ht, self.ht_err = torch.zeros_like(self.h0), torch.zeros_like(self.h0)
        s_abs = self.s.abs()
        short = x.dtype == torch.bfloat16
        power = ((3 + g.double().abs()) * self.a).nan_to_num(0.0, 0.0, 0.0) * (self.s if decay == "sigmoid" else 1)
        self.rest_err = U * (12 * s_abs + (power if short else 0))
        self.keep_err = self.rest_err + (U if short else 0)
        for i, (b, e) in enumerate(seqs):
            h, ha, er = self.h0[i], self.h0[i].abs(), torch.zeros(C, dtype=torch.float64)
            for t in range(b, e):
                self.prev[t], self.prev_abs[t], self.prev_err[t] = h, ha, er
                # a rounding of the step, of the products that carry a state over many rows, and of 1 - a (12 U:
                # exponential, sum and reciprocal)
                er = (self.a[t] * er + 8 * U * (self.a[t] * ha + self.c[t].abs() * self.x[t].abs()) + TINY * ha
                      + self.keep_err[t] * ha + (self.keep_err[t] * self.x[t].abs() if complement else 0))
                h = self.a[t] * h + self.c[t] * self.x[t]
                ha = self.a[t] * ha + self.c[t].abs() * self.x[t].abs()
                self.h[t], self.h_abs[t], self.err[t] = h, ha, er
            self.ht[i], self.ht_err[i] = h, er
        self.inside = torch.zeros(n, dtype=torch.bool)
        for b, e in seqs:
            self.inside[b:e] = True

    def backward(self, dy, dht=None):
        """((dx, its rounding), (dg, ..), (dh0, ..)), zero outside the sequences."""
        dy = dy.double()
        n, C = self.x.shape
        z = torch.zeros(n, C, dtype=torch.float64)
        dx, dg, dxe, dge = z.clone(), z.clone(), z.clone(), z.clone()
        dh0, dh0e = torch.zeros_like(self.h0), torch.zeros_like(self.h0)
        for i, (b, e) in enumerate(self.seqs):
            m = torch.zeros(C, dtype=torch.float64) if dht is None else dht[i].double()
            ma, me = m.abs(), torch.zeros(C, dtype=torch.float64)
            for t in range(e - 1, b - 1, -1):
                a, s = self.a[t], self.s[t]
                l, la = dy[t] + m, dy[t].abs() + ma
                le = me + U * 2 * la
                dx[t] = self.c[t] * l
                dxe[t] = self.c[t].abs() * (le + 13 * U * la) + (self.rest_err[t] * la if self.comp else 0)
                core = self.prev[t] - (self.x[t] if self.comp else 0)
                core_abs = self.prev_abs[t] + (self.x[t].abs() if self.comp else 0)
                slope = a if self.decay == "log" else a * s
                dg[t] = slope * l * core
                dge[t] = slope * (le * core_abs + la * (self.prev_err[t] + U * core_abs) + 30 * U * la * core_abs) + TINY * la * core_abs
                # a and 1 - a as they are kept
                dge[t] += la * core_abs * (self.keep_err[t] * (s if self.decay == "sigmoid" else 1)
                                           + (self.rest_err[t] * a if self.decay == "sigmoid" else 0))
                m, ma = a * l, a * la
                me = a * le + 6 * U * ma + self.keep_err[t] * la + TINY * la
            dh0[i], dh0e[i] = m, me
        return (dx, dxe), (dg, dge), (dh0, dh0e)


def act(kind, u):
    return u if kind == "none" else u * torch.sigmoid(u) if kind == "silu" else torch.sigmoid(u)


def act_slope(kind, u):
    p = torch.sigmoid(u)
    return torch.ones_like(u) if kind == "none" else p * (1 + u * (1 - p)) if kind == "silu" else p * (1 - p)


class Conv:
    """x [rows, C], w [C, W], b [C] or None, h0 [nseq, W - 1, C] or None."""

    def __init__(self, x, w, b, seqs, kind, h0=None):
        self.w, self.seqs, self.kind, self.W = w.double(), seqs, kind, w.shape[1]
        W, C = self.W, x.shape[1]
        self.x = x.double()
        self.h0 = torch.zeros(len(seqs), W - 1, C, dtype=torch.float64) if h0 is None else h0.double()
        self.b = torch.zeros(C, dtype=torch.float64) if b is None else b.double()
        self.full = [torch.cat([self.h0[i], self.x[s:e]]) for i, (s, e) in enumerate(seqs)]
        self.ht = torch.stack([f[f.shape[0] - (W - 1):] for f in self.full]) if seqs else self.h0
        self.u, self.u_abs = torch.zeros_like(self.x), torch.zeros_like(self.x)
        for f, (s, e) in zip(self.full, seqs):
            for j in range(W):
                self.u[s:e] += f[j:j + e - s] * self.w[:, j]
                self.u_abs[s:e] += f[j:j + e - s].abs() * self.w[:, j].abs()
        self.u += self.b
        self.u_abs += self.b.abs()
        self.u_err = (W + 1) * U * self.u_abs
        self.y = act(kind, self.u)
        # a slope of at most 1.1; the exponential, sum, reciprocal and product of the activation: 12 U
        self.y_err = 1.1 * self.u_err + (0 if kind == "none" else 12 * U * (self.y.abs() + U))

    def backward(self, dy, dht=None, chain=256):
        """((dx, rounding), (dw, ..), (db, ..), (dh0, ..)); chain: terms of a float32 partial sum."""
        W, dy = self.W, dy.double()
        du = dy * act_slope(self.kind, self.u)
        # the slope's own slope is at most 0.5
        due = dy.abs() * (0.5 * self.u_err + (0 if self.kind == "none" else 16 * U * (1 + self.u.abs()))) + U * du.abs()
        dx, dxe = torch.zeros_like(self.x), torch.zeros_like(self.x)
        dw, dwe = torch.zeros_like(self.w), torch.zeros_like(self.w)
        db, dbe = torch.zeros_like(self.b), torch.zeros_like(self.b)
        dh0, dh0e = torch.zeros_like(self.h0), torch.zeros_like(self.h0)
        for i, (f, (s, e)) in enumerate(zip(self.full, self.seqs)):
            d, de = torch.zeros_like(f), torch.zeros_like(f)
            for j in range(W):
                d[j:j + e - s] += du[s:e] * self.w[:, j]
                de[j:j + e - s] += (due[s:e] + (W + 2) * U * du[s:e].abs()) * self.w[:, j].abs()
                dw[:, j] += (du[s:e] * f[j:j + e - s]).sum(0)
                dwe[:, j] += ((due[s:e] + chain * U * du[s:e].abs()) * f[j:j + e - s].abs()).sum(0)
            db += du[s:e].sum(0)
            dbe += (due[s:e] + chain * U * du[s:e].abs()).sum(0)
            if dht is not None:
                d[f.shape[0] - (W - 1):] += dht[i].double()
                de[f.shape[0] - (W - 1):] += U * dht[i].double().abs()
            dh0[i], dh0e[i] = d[:W - 1], de[:W - 1]
            dx[s:e], dxe[s:e] = d[W - 1:], de[W - 1:]
        return (dx, dxe), (dw, dwe), (db, dbe), (dh0, dh0e)


def rotate(x, pos, freq, interleaved=False, scale=1.0, inverse=False):
    """x [rows, heads, D], pos [rows] integers: (x turned, its rounding)."""
    x, R = x.double(), 2 * freq.numel()
    angle = pos.double()[:, None] * freq.double()
    cos, sin = torch.cos(angle)[:, None] * scale, torch.sin(angle)[:, None] * scale
    if inverse:
        sin = -sin
    i, j = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y, err = x.clone(), torch.zeros_like(x)
    u, v = x[..., i], x[..., j]
    y[..., i], y[..., j] = u * cos - v * sin, u * sin + v * cos
    # the angle to 8 U of a radian at 2^31 positions, sine and cosine, and the two products
    err[..., i] = err[..., j] = 16 * U * abs(scale) * (u.abs() + v.abs())
    return y, err


def inv_sqrt(n):
    return 1.0 / math.sqrt(n)


def worst(name, got, want, err, dtype=None):
    """Largest error over its bound; the bound counts the rounding of the stored value too."""
    step = half_step(dtype or got.dtype)
    got = got.detach().cpu().double().reshape(want.shape)
    assert torch.isfinite(got).all(), name
    bound = err * (1 + step) + step * want.abs() + 1e-38
    return float(((got - want).abs() / bound).max()) if want.numel() else 0.0
