"""Differential attention and paged attention from their definitions in 64 bits, with the error each
output may have.

Bounds (per element, worst case; u = half a step of the inputs' 16-bit type, relative):
  P_t   relative error c: the scores' fp32 sums of d products (an absolute error of x is a relative
        one of exp x), the fp32 sum of the row, the hardware exponential (2^-22)
  O     u of the result; u + c of each p V, because P is rounded to 16 bits for its product
        (paged forms: u^2, the rounded value's remainder goes in as a second factor)
  D_t   sum |dO| (error of O_t, which is read back in 16 bits)
  X1    P1 (G - D1): u + c of the value, P1 times the errors of G and D1;  X2 alike
  dQ, dK, dV  the error of the 16-bit factor times the other factor's size, u of the result
  dlam  c of each P2 G and the error of G, in fp32 throughout; u of the result
A rounded factor is also off by half fp16's smallest step (2^-25) or, in bf16, by what is flushed to
zero (2^-126), and so is P: the hardware exponential returns 0 for results under 2^-126, an absolute
error of that much, whatever the factors G - D or V beside it. Every fp32 sum of n terms adds n 2^-23
(the tensor pipe may truncate) of the sum of magnitudes.
"""
from __future__ import annotations

import math

import torch


FLUSH = 2.0 ** -126


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else FLUSH


def heads_of(t, H):
    return t.repeat_interleave(H // t.shape[1], 1)


def group_sum(t, HK):
    return t.view(t.shape[0], HK, t.shape[1] // HK, *t.shape[2:]).sum(2)


def lam_rows(lam, B, H, NQ):
    lam = lam.double()
    if lam.dim() == 1:
        lam = lam.view(1, H, 1)
    return lam.expand(B, H, NQ).unsqueeze(-1)


class Reference:
    """Everything about one problem, in 64 bits; rows outside the lengths count as zero."""

    def __init__(self, Q1, K1, Q2, K2, V, lam, causal=False, s1=None, s2=None, q_lens=None, k_lens=None,
                 factors=1):
        self.dtype, dev = Q1.dtype, Q1.device
        B, H, NQ, d = Q1.shape
        HK, NK = K1.shape[1:3]
        self.B, self.H, self.HK, self.NQ, self.NK, self.d = B, H, HK, NQ, NK, d
        ql = torch.full((B,), NQ, device=dev) if q_lens is None else q_lens.long().clamp(0, NQ)
        kl = torch.full((B,), NK, device=dev) if k_lens is None else k_lens.long().clamp(0, NK)
        i, j = torch.arange(NQ, device=dev).view(1, 1, NQ, 1), torch.arange(NK, device=dev).view(1, 1, 1, NK)
        q, k = ql.view(B, 1, 1, 1), kl.view(B, 1, 1, 1)
        seen = (i < q) & (j < k)
        if causal:
            seen = seen & (j <= i + k - q)
        self.seen = seen
        self.live = seen.any(-1, keepdim=True)
        rows = (i < q).transpose(2, 3).reshape(B, 1, NQ, 1) & self.live
        keys = (j < k).reshape(B, 1, NK, 1)
        self.Q = [torch.where(rows, t.double(), 0.0) for t in (Q1, Q2)]
        self.K = [heads_of(torch.where(keys, t.double(), 0.0), H) for t in (K1, K2)]
        self.V = heads_of(torch.where(keys, V.double(), 0.0), H)
        self.rows = rows
        self.lam = lam_rows(lam, B, H, NQ)
        self.lam_shape = tuple(lam.shape)
        self.s = [x if x is not None else 1 / math.sqrt(d) for x in (s1, s2)]
        self.P, self.LSE, amp = [], [], 0.0
        for Q, K, s in zip(self.Q, self.K, self.s):
            x = (s * (Q @ K.transpose(2, 3))).masked_fill(~seen, -math.inf)
            lse = torch.logsumexp(x, -1, keepdim=True)
            self.P.append(torch.where(seen, torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)), 0.0))
            self.LSE.append(lse.squeeze(-1))
            if x.numel():
                amp = max(amp, abs(s) * float((Q.abs() @ K.abs().transpose(2, 3)).max()))
        # score error in 32 bits, row sums, exponential
        self.c = 2.0 ** -23 * ((d + 4) * amp + NK + 16)
        self.O_t = [P @ self.V for P in self.P]
        self.O = self.O_t[0] - self.lam * self.O_t[1]
        u, t = half_step(self.dtype), tiny(self.dtype)
        self.u, self.t = u, t
        size = [P @ self.V.abs() for P in self.P]
        low = (t + FLUSH) * (seen.double() @ self.V.abs())
        self.dO_t = [(u ** factors + self.c) * z + low for z in size]   # unrounded outputs
        self.tol_O = (self.dO_t[0] + self.lam.abs() * self.dO_t[1]) * (1 + u) + u * self.O.abs() + t
        self.tol_O2 = self.dO_t[1] * (1 + u) + u * self.O_t[1].abs() + t
        self.tol_LSE = self.c + 2.0 ** -21 * max([1.0] + [float(l[torch.isfinite(l)].abs().max())
                                                         for l in self.LSE if torch.isfinite(l).any()])

    def backward(self, dO):
        """{name: (value, tolerance)} of the six gradients."""
        u, t, c, eps = self.u, self.t, self.c, 2.0 ** -23
        dO = torch.where(self.rows, dO.double(), 0.0)
        G = dO @ self.V.transpose(2, 3)
        eG = self.V.shape[3] * eps * (dO.abs() @ self.V.abs().transpose(2, 3))
        D = [(dO * o).sum(-1, keepdim=True) for o in self.O_t]
        eD2 = (dO.abs() * self.tol_O2).sum(-1, keepdim=True)
        eD1 = (dO.abs() * (self.tol_O + self.lam.abs() * self.tol_O2)).sum(-1, keepdim=True)
        X = [self.P[0] * (G - D[0]), self.lam * self.P[1] * (D[1] - G)]
        eX = [(u + c) * x.abs() + p * (1 + u) * (eG + e) + t + FLUSH * (1 + self.lam.abs()) * ((G - d).abs() + eG + e)
              for x, p, d, e in zip(X, (self.P[0], self.lam.abs() * self.P[1]), D, (eD1, eD2))]
        eX = [torch.where(self.seen, e, 0.0) for e in eX]
        A = self.P[0] - self.lam * self.P[1]
        eA = torch.where(self.seen, u * A.abs() + c * (self.P[0] + self.lam.abs() * self.P[1]) + t
                         + FLUSH * (1 + self.lam.abs()), 0.0)

        def product(x, ex, y, n):
            return x @ y, ex @ y.abs() + n * eps * (x.abs() @ y.abs())

        out = {}
        for k, (Q, K, s, x, ex) in enumerate(zip(self.Q, self.K, self.s, X, eX)):
            v, e = product(x, ex, K, self.NK)
            out[f"dQ{k + 1}"] = (s * v, abs(s) * e)
            v, e = product(x.transpose(2, 3), ex.transpose(2, 3), Q, self.NQ)
            out[f"dK{k + 1}"] = (group_sum(s * v, self.HK), group_sum(abs(s) * e, self.HK))
        v, e = product(A.transpose(2, 3), eA.transpose(2, 3), dO, self.NQ)
        out["dV"] = (group_sum(v, self.HK), group_sum(e, self.HK))
        for n, (v, e) in out.items():
            out[n] = (v, e * (1 + u) + u * v.abs() + t)
        # sums over the keys of the unrounded P2 G; 512: terms one after another of the sums over rows
        size = (self.P[1] * G.abs()).sum(-1)
        dl = -D[1].squeeze(-1)
        el = (self.P[1] * (c * G.abs() + eG)).sum(-1) + (self.NK + 512) * eps * size + FLUSH * G.abs().sum(-1)
        shape = (1, self.lam_shape[0], 1) if len(self.lam_shape) == 1 else self.lam_shape or (1, 1, 1)
        axes = [k for k, n in enumerate(shape) if n == 1 and dl.shape[k] != 1]
        if axes:
            dl, el = dl.sum(axes, keepdim=True), el.sum(axes, keepdim=True)
        out["dlam"] = (dl.reshape(self.lam_shape), (el + u * dl.abs() + t).reshape(self.lam_shape))
        return out


def within(what, got, want, tol):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - tol
    worst = float(over.max()) if over.numel() else -1.0
    assert worst <= 0, (f"{what}: off by {float((got - want).abs().flatten()[over.argmax()]):.3e}, allowed "
                        f"{float(torch.as_tensor(tol).expand_as(want).flatten()[over.argmax()]):.3e}")


def pages_of(cache, table, b, n):
    """The first n rows of sequence b: [HK, n, width]."""
    ps = cache.shape[1]
    at = torch.arange(n, device=cache.device)
    return cache[table[b].long()[at // ps], at % ps].transpose(0, 1)


def paged_reference(Q1, K1, Q2, K2, V, lam, table, lens, s1=None, s2=None):
    """(value, tolerance) of the paged forms; Q2 None: one map."""
    B, H, d = Q1.shape
    dtype, dv = Q1.dtype, V.shape[3]
    out = torch.zeros((B, H, dv), dtype=torch.float64, device=Q1.device)
    tol = torch.zeros_like(out)
    most = table.shape[1] * K1.shape[1]
    for b in range(B):
        n = min(max(int(lens[b]), 0), most)
        if n == 0:
            continue
        two = Q2 is not None
        r = Reference(Q1[b].view(1, H, 1, d), pages_of(K1, table, b, n)[None],
                      (Q2 if two else Q1)[b].view(1, H, 1, d), pages_of(K2 if two else K1, table, b, n)[None],
                      pages_of(V, table, b, n)[None],
                      (lam if lam.dim() < 2 else lam.expand(B, H)[b]) if two else torch.zeros((), device=Q1.device),
                      False, s1, s2, factors=2)
        out[b], tol[b] = r.O[0, :, 0], r.tol_O[0, :, 0]
    return out, tol
