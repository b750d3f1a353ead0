"""Plain 64-bit windowed attention and its gradients, and the inputs their
tests share.  Written from the formulas in include/fa.h; nothing of the
library is used here.

A rounding to bf16 moves a value by at most 2^-8 of it (half a step), one to
fp16 by 2^-11, or by 2^-25 below 2^-14.  The kernels round P to bf16 for its
products with V and dO, 2^15 P to fp16 for dS, dS and the outputs to bf16; sums
are fp32.  `off` bounds what fp32 does to a weight: an exponent's argument is a
sum of d products, scaled and shifted, whose error is below 2^-20 of the sizes
of its terms, and P moves by that factor.
"""
from __future__ import annotations

import torch

HALF_BF16 = 2.0 ** -8


def sees(n, window, sinks):
    i, j = torch.arange(n)[:, None], torch.arange(n)[None]
    return (j <= i) & ((i - j < window) | (j < sinks))


def _weights(q, k, see, scale):
    """Scores (hidden ones -inf) and the sizes of their terms."""
    s = torch.where(see, scale * (q @ k.T), torch.tensor(-float("inf"), dtype=torch.float64))
    size = torch.where(see, scale * (q.abs() @ k.abs().T), torch.zeros((), dtype=torch.float64))
    return s, size


def _product(w, x):
    """w @ x where a weight of zero does not read its row (0 x NaN is 0)."""
    if bool(torch.isfinite(x).all()):
        return w @ x
    out = torch.zeros(w.shape[0], x.shape[1], dtype=torch.float64)
    for i in range(w.shape[0]):
        j = torch.nonzero(w[i] != 0)[:, 0]
        out[i] = w[i, j] @ x[j]
    return out


def forward(q, k, v, window, sinks, scale):
    """One sequence: q [H, n, d], k, v [Hkv, n, d], all float64 -> o, lse and
    the tolerances of both."""
    H, n, d = q.shape
    G, see = H // k.shape[0], sees(n, window, sinks)
    o, lse = torch.empty_like(q), torch.empty(H, n, dtype=torch.float64)
    tol_o, tol_l = torch.empty_like(q), torch.empty_like(lse)
    for h in range(H):
        s, size = _weights(q[h], k[h // G], see, scale)
        lse[h] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[h][:, None])
        off = 2.0 ** -20 * (1 + torch.nan_to_num(size).amax(-1))
        o[h] = _product(p, v[h // G])
        # each weight rounded in the product, not in the sum it is divided by
        tol_o[h] = (HALF_BF16 + 2 * off[:, None]) * (p @ torch.nan_to_num(v[h // G]).abs()) \
            + HALF_BF16 * o[h].abs() + 1e-30
        tol_l[h] = off + 2.0 ** -20 * lse[h].abs()
    return o, lse, tol_o, tol_l


def backward(q, k, v, o, lse, g, window, sinks, scale):
    """One sequence: gradients of sum(o g) with o and lse as they were handed
    over -> (dq, dk, dv) and their tolerances."""
    H, n, d = q.shape
    Hkv = k.shape[0]
    G, see = H // Hkv, sees(n, window, sinks)
    dq, tq = torch.empty_like(q), torch.empty_like(q)
    dk, dv, tk, tv = (torch.zeros_like(k) for _ in range(4))
    for h in range(H):
        kh, vh = k[h // G], v[h // G]
        s, size = _weights(q[h], kh, see, scale)
        p = torch.where(see, torch.exp(s - lse[h][:, None]), torch.zeros((), dtype=torch.float64))
        dlt = (g[h] * o[h]).sum(-1, keepdim=True)
        # (scores without a NaN's own: a weight's error is counted by row)
        off = 2.0 ** -20 * (1 + torch.nan_to_num(size) + torch.nan_to_num(lse[h]).abs()[:, None])
        ds = torch.where(see, p * (g[h] @ vh.T - dlt), torch.zeros((), dtype=torch.float64))
        # dS: P and its product with dP - D rounded; dP and D are fp32 sums
        fine = torch.nan_to_num
        inner = 2.0 ** -20 * (fine(g[h]).abs() @ fine(vh).abs().T
                              + (fine(g[h]) * fine(o[h])).abs().sum(-1, keepdim=True))
        err = fine(ds).abs() * (1.02 * HALF_BF16 + 2.0 ** -11 + 2 * off) + fine(p) * inner
        # (weights below 2^-29: fp16's smallest steps)
        err += torch.where(see, 2.0 ** -40 * fine(g[h] @ vh.T - dlt).abs(),
                           torch.zeros((), dtype=torch.float64))
        dq[h] = scale * _product(ds, kh)
        tq[h] = scale * (err @ fine(kh).abs()) + HALF_BF16 * dq[h].abs() + 1e-30
        gk, gv = scale * _product(ds.T, q[h]), _product(p.T, g[h])
        dk[h // G] += gk
        dv[h // G] += gv
        tk[h // G] += scale * (err.T @ fine(q[h]).abs())
        tv[h // G] += (fine(p) * (HALF_BF16 + 2 * off)).T @ fine(g[h]).abs()
    tk += HALF_BF16 * dk.abs() + 1e-30
    tv += HALF_BF16 * dv.abs() + 1e-30
    return (dq, dk, dv), (tq, tk, tv)


class Batch:
    """bf16 inputs on the host and where each sequence's rows are.  lens: equal
    lengths [B, heads, N, d]; packed: back to back from row `lead` on of
    `lead + sum + tail` rows [heads, total, d], whose other rows hold NaN."""

    def __init__(self, lens, H, Hkv, d, packed, seed, lead=0, tail=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.Hkv, self.d, self.packed = lens, H, Hkv, d, packed
        if packed:
            self.starts = [lead + sum(lens[:b]) for b in range(len(lens))]
            self.total = lead + sum(lens) + tail
            make = lambda h: torch.randn(h, self.total, d, generator=g).bfloat16()
        else:
            make = lambda h: torch.randn(len(lens), h, lens[0], d, generator=g).bfloat16()
        self.q, self.k, self.v, self.g = make(H), make(Hkv), make(Hkv), make(H)
        if packed:
            own = torch.zeros(self.total, dtype=torch.bool)
            own[lead:lead + sum(lens)] = True
            for x in (self.q, self.k, self.v, self.g):
                x[:, ~own] = float("nan")
            self.own = own
            self.cu = torch.tensor([lead] + [lead + sum(lens[:b + 1]) for b in range(len(lens))],
                                   dtype=torch.int32)

    def seq(self, x, b):
        """Rows of sequence b of a tensor (host or device), float64 on the host."""
        x = x.detach().cpu()
        if self.packed:
            x = x[:, self.starts[b]:self.starts[b] + self.lens[b]]
        else:
            x = x[b]
        return x.double()
