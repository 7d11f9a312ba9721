"""Plain 64-bit forms of linear attention with a decay for each head and of
the group norm with an activation, and the sums that bound their rounding.
Only tests import this."""
import math

import torch


def decay_matrix(g):
    """D[t, i, j] over rows of g [..., L] float64, j = 0 the state before the first row and j > 0 row j - 1:
    exp(sum of g over the rows after j - 1 up to i), 0 above the diagonal."""
    L = g.shape[-1]
    out = torch.zeros(*g.shape[:-1], L, L + 1, dtype=torch.float64)
    run = torch.zeros(*g.shape[:-1], L + 1, dtype=torch.float64)  # weight of each column so far
    run[..., 0] = 1.0
    for i in range(L):  # products of the rows' own factors: no differences of long sums
        run[..., : i + 1] *= torch.exp(g[..., i])[..., None]
        run[..., i + 1] = 1.0
        out[..., i, : i + 2] = run[..., : i + 2]
    return out


class Linear:
    """One sequence of L rows: q, k [L, H, K], v [L, HV, V], g [L, HV] or None, h0 [HV, V, K] or None (float64)."""

    def __init__(self, q, k, v, g, scale, h0=None):
        L, H, K = q.shape
        self.HV, self.V, self.r, self.scale = v.shape[1], v.shape[2], v.shape[1] // H, scale
        self.H, self.K, self.L = H, K, L
        self.q, self.k = (x.double().transpose(0, 1).repeat_interleave(self.r, 0) for x in (q, k))  # [HV, L, K]
        self.v = v.double().transpose(0, 1)
        g = torch.zeros(L, self.HV) if g is None else g
        D = decay_matrix(g.double().transpose(0, 1))
        self.D0, self.D = D[..., 0], D[..., 1:]
        self.h0 = torch.zeros(self.HV, self.V, K, dtype=torch.float64) if h0 is None else h0.double()
        if L:
            self.end, self.end0 = self.D[:, -1, :], self.D0[:, -1]
        else:
            self.end, self.end0 = torch.zeros(self.HV, 0, dtype=torch.float64), torch.ones(self.HV, dtype=torch.float64)

    def forward(self):
        """o [L, HV, V], ht [HV, V, K]."""
        s = self.scale
        o = s * ((self.q @ self.k.transpose(1, 2)) * self.D @ self.v + self.D0[..., None] * (self.q @ self.h0.transpose(1, 2)))
        ht = (self.v * self.end[..., None]).transpose(1, 2) @ self.k + self.end0[:, None, None] * self.h0
        return o.transpose(0, 1), ht

    def forward_abs(self):
        """The same sums over absolute values: what every rounding of a term or of a partial sum is relative to."""
        return Linear._with(self, self.q.abs(), self.k.abs(), self.v.abs(), self.h0.abs()).forward()

    def _with(self, q, k, v, h0):
        c = object.__new__(Linear)
        c.__dict__.update(self.__dict__)
        c.q, c.k, c.v, c.h0 = q, k, v, h0
        return c

    def backward(self, do, dht=None):
        """dq, dk [L, H, K], dv [L, HV, V], dg [L, HV], dh0 [HV, V, K], each from its own formula."""
        s, HV = self.scale, self.HV
        do = do.double().transpose(0, 1)
        dht = torch.zeros_like(self.h0) if dht is None else dht.double()
        A = s * (do @ self.v.transpose(1, 2)) * self.D          # [HV, i, j]
        P = s * (self.q @ self.k.transpose(1, 2)) * self.D
        dq = A @ self.k + s * self.D0[..., None] * (do @ self.h0)
        dk = A.transpose(1, 2) @ self.q + self.end[..., None] * (self.v @ dht)
        dv = P.transpose(1, 2) @ do + self.end[..., None] * (self.k @ dht.transpose(1, 2))
        dh0 = s * (do * self.D0[..., None]).transpose(1, 2) @ self.q + self.end0[:, None, None] * dht
        # dg_t: all pairs (i, j) with i >= t > j; the initial state is a column before row 0, dht a row after the last
        M = torch.zeros(HV, self.L + 1, self.L + 1, dtype=torch.float64)
        M[:, : self.L, 1:] = A * (self.q @ self.k.transpose(1, 2))
        M[:, : self.L, 0] = s * self.D0 * (do * (self.q @ self.h0.transpose(1, 2))).sum(-1)
        M[:, self.L, 1:] = self.end * (self.v * (self.k @ dht.transpose(1, 2))).sum(-1)
        M[:, self.L, 0] = self.end0 * (self.h0 * dht).sum((1, 2))
        dg = torch.zeros(HV, self.L, dtype=torch.float64)
        for t in range(self.L):
            dg[:, t] = M[:, t:, : t + 1].sum((1, 2))
        heads = [x.reshape(self.H, self.r, self.L, self.K).sum(1).transpose(0, 1) for x in (dq, dk)]
        return heads[0], heads[1], dv.transpose(0, 1), dg.transpose(0, 1), dh0

    def backward_abs(self, do, dht=None):
        c = self._with(self.q.abs(), self.k.abs(), self.v.abs(), self.h0.abs())
        return c.backward(do.abs(), None if dht is None else dht.abs())


def group_norm(x, groups, w, b, z, act, centered, eps):
    x = x.double()
    u = x.reshape(*x.shape[:-1], groups, -1)
    if centered:
        u = u - u.mean(-1, keepdim=True)
    u = (u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps)).reshape(x.shape)
    n = u * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())

    def f(t):
        return t if act == "none" else t / (1 + torch.exp(-t)) if act == "silu" else 1 / (1 + torch.exp(-t))

    return n * f(z.double()) if z is not None else f(n)


def inv_sqrt(K):
    return 1.0 / math.sqrt(K)
