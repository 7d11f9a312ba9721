"""Linear attention with a decay for each head and its gradients in 64 bits
for long sequences: the recurrence chunk by chunk, rows of C at a time, on any
device.  Only tests import this; linref's sums over all pairs pin it."""
import torch

C = 64


def _abs(x):
    return None if x is None else x.abs()


class Long:
    """One sequence of L rows: q, k [L, H, K], v, do [L, HV, V], g [L, HV] or None, h0, dht [HV, V, K] or None."""

    def __init__(self, q, k, v, g, scale, h0=None, do=None, dht=None):
        L, self.H, self.K = q.shape
        self.HV, self.V, self.r = v.shape[1], v.shape[2], v.shape[1] // q.shape[1]
        self.L, self.nc, self.scale, self.dev = L, -(-L // C), scale, q.device

        def rows(x, rep=1):  # [L, heads, D] -> [heads, nc, C, D]; rows past the end are zero
            x = x.double().transpose(0, 1).repeat_interleave(rep, 0)
            return torch.nn.functional.pad(x, (0, 0, 0, self.nc * C - L)).reshape(x.shape[0], self.nc, C, x.shape[2])

        self.q, self.k, self.v = rows(q, self.r), rows(k, self.r), rows(v)
        self.do = None if do is None else rows(do)
        zero = torch.zeros(self.HV, self.V, self.K, dtype=torch.float64, device=self.dev)
        self.h0 = zero if h0 is None else h0.double()
        self.dht = zero if dht is None else dht.double()
        g = torch.zeros(L, self.HV, dtype=torch.float64, device=self.dev) if g is None else g.double()
        # far below float32's range a decay is a reset; kept finite for the differences of G
        g = g.clamp(min=-200.0).transpose(0, 1)
        g = torch.nn.functional.pad(g, (0, self.nc * C - L)).reshape(self.HV, self.nc, C)
        self.g = g
        G = g.cumsum(-1)
        low = torch.ones(C, C, dtype=torch.bool, device=self.dev).tril()
        self.D = (G[..., :, None] - G[..., None, :]).masked_fill(~low, float("-inf")).exp()
        self.inn, self.out, self.all = G.exp(), (G[..., -1:] - G).exp(), G[..., -1].exp()

    def _like(self, **kw):
        c = object.__new__(Long)
        c.__dict__.update(self.__dict__)
        c.__dict__.update(kw)
        return c

    def absolute(self):
        """The same sums over absolute values."""
        return self._like(**{x: _abs(getattr(self, x)) for x in ("q", "k", "v", "do", "h0", "dht")})

    def _rows(self, x):
        return x.reshape(x.shape[0], -1, x.shape[-1])[:, : self.L].transpose(0, 1)

    def states(self):
        """S before each chunk and after the last, [nc + 1] of [HV, V, K]."""
        E = (self.v * self.out[..., None]).transpose(2, 3) @ self.k
        S = [self.h0]
        for c in range(self.nc):
            S.append(S[-1] * self.all[:, c, None, None] + E[:, c])
        return S

    def gradients(self):
        """R behind each chunk's last row and before the first: [nc + 1], R[c] belongs to the state before chunk c."""
        E = self.scale * (self.do * self.inn[..., None]).transpose(2, 3) @ self.q
        R = [self.dht]
        for c in reversed(range(self.nc)):
            R.append(R[-1] * self.all[:, c, None, None] + E[:, c])
        return R[::-1]

    def forward(self):
        """o [L, HV, V], ht."""
        S = self.states()
        y = ((self.q @ self.k.transpose(2, 3)) * self.D) @ self.v
        y = y + (self.q @ torch.stack(S[:-1], 1).transpose(2, 3)) * self.inn[..., None] if self.nc else y
        return self._rows(self.scale * y), S[-1]

    def backward(self):
        """dq, dk [L, H, K], dv [L, HV, V], dg [L, HV], dh0."""
        if not self.nc:
            z = torch.zeros(0, self.H, self.K, dtype=torch.float64, device=self.dev)
            return z, z, z.new_zeros(0, self.HV, self.V), z.new_zeros(0, self.HV), self.dht
        S, R = torch.stack(self.states(), 1), torch.stack(self.gradients(), 1)
        S0, R1 = S[:, :-1], R[:, 1:]
        A = self.scale * (self.do @ self.v.transpose(2, 3)) * self.D
        P = self.scale * (self.q @ self.k.transpose(2, 3)) * self.D
        xq = self.scale * (self.do @ S0) * self.inn[..., None]
        xk = (self.v @ R1) * self.out[..., None]
        dq, dk = A @ self.k + xq, A.transpose(2, 3) @ self.q + xk
        dv = P.transpose(2, 3) @ self.do + (self.k @ R1.transpose(2, 3)) * self.out[..., None]
        self.rho_q, self.rho_k = (xq * self.q).sum(-1), (xk * self.k).sum(-1)  # across chunks
        self.M = (A * (self.q @ self.k.transpose(2, 3))).tril(-1)  # pairs inside one
        self.through = self.all * (S0 * R1).sum((2, 3))
        # dg_t: pairs (i, j) with i >= t > j: inside the chunk, from before it, to behind it, over it
        inner = self.M.cumsum(-1).roll(1, -1)
        inner[..., 0] = 0  # [i, t] = sum over j < t
        inner = (inner * torch.ones(C, C, dtype=torch.float64, device=self.dev).tril()).sum(-2)
        before = self.rho_q.flip(-1).cumsum(-1).flip(-1)
        behind = self.rho_k.cumsum(-1) - self.rho_k
        dg = inner + before + behind + self.through[..., None]
        heads = [self._rows(x).reshape(self.L, self.H, self.r, self.K).sum(2) for x in (dq, dk)]
        return heads[0], heads[1], self._rows(dv), self._rows(dg[..., None])[..., 0], R[:, 0]

    def border_norms(self):
        """|S o R| at the row before each chunk, [HV, nc]: what the products there round relative to."""
        S, R = torch.stack(self.states(), 1), torch.stack(self.gradients(), 1)
        return (S * R).flatten(2).norm(dim=2)[:, :-1]
