"""Plain 64-bit implementations of the Q/K preparation and serving operators,
and the inputs their tests share.  Written from the formulas in
include/fa.h, with numpy on the CPU; nothing of the library is used here.

A rounding to bf16 moves a value by at most 2^-8 of it (half a step),
arithmetic in fp32 by 2^-24 per operation: the tests' tolerances count those.
"""
from __future__ import annotations

import numpy as np
import torch

BF16, E4M3, INT8 = 0, 1, 2
DTYPES = {BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn, INT8: torch.int8}
HALF_BF16 = 2.0 ** -8


def f64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ norm + rotation
def tables(rows, rot, base=10000.0):
    a = np.arange(rows)[:, None] * base ** (-np.arange(0, rot, 2) / rot)[None]
    return torch.from_numpy(np.cos(a)).float(), torch.from_numpy(np.sin(a)).float()


def turn(y, cos, sin, rot, inter):
    """y [..., d] with its first rot elements turned; cos, sin [..., rot / 2]."""
    z = y.copy()
    if inter:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z[..., 0:rot:2], z[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        h = rot // 2
        a, b = y[..., :h], y[..., h:rot]
        z[..., :h], z[..., h:rot] = a * cos - b * sin, b * cos + a * sin
    return z


def norm_rope(x, w, cos, sin, rot, inter, eps):
    """x [B, H, N, d]; cos, sin [B, 1, N, rot / 2]."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return turn(x * r * w, cos, sin, rot, inter)


def norm_rope_backward(g, x, w, cos, sin, rot, inter, eps):
    """(dx, dw) and the sizes of the terms behind them (for tolerances)."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = turn(g, cos, -sin, rot, inter)
    xh, gw = x * r, g * w
    dx = r * (gw - xh * (gw * xh).mean(-1, keepdims=True))
    dw = (g * xh).sum((0, 1, 2))
    dx_size = r * (np.abs(gw) + np.abs(xh) * np.abs(gw * xh).mean(-1, keepdims=True))
    return dx, dw, dx_size, np.abs(g * xh).sum((0, 1, 2))


# ------------------------------------------------------------------ quantised rows
def quantise(x, fmt):
    """What a row x [..., d] reads back as, from the definition."""
    if fmt == BF16:
        return x
    most = 448.0 if fmt == E4M3 else 127.0
    out = np.full_like(x, np.nan)
    ok = np.isfinite(x).all(-1)
    amax = np.abs(np.where(np.isfinite(x), x, 0)).max(-1)
    e = np.full(amax.shape, -100)
    # the smallest exponent that holds the row, as far as the format's largest
    # number times it is finite in bf16
    for k in range(-100, 120 if fmt == E4M3 else 122):
        e = np.where(amax > most * 2.0 ** (k - 1), k, e)
    e = e[..., None]
    z = np.clip(x * 2.0 ** -e.astype(np.float64), -most, most)
    if fmt == E4M3:
        with np.errstate(divide="ignore", invalid="ignore"):
            lead = np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -6)))
        step = 2.0 ** (lead - 3)
    else:
        step = np.ones_like(z)
    with np.errstate(invalid="ignore"):
        y = np.rint(z / step) * step * 2.0 ** e.astype(np.float64)
    out[ok] = y[ok]
    return out


# ------------------------------------------------------------------ attention over a cache
def sees(hist, n, T, mask_row_bits):
    """[T, hist + n] truth values; mask_row_bits: [T, T] truth values or None."""
    s = np.zeros((T, hist + n), bool)
    s[:n, :hist] = True
    if mask_row_bits is None:
        s[:n, hist:] = np.tril(np.ones((n, n), bool))
    else:
        s[:n, hist:] = mask_row_bits[:n, :n]
    return s


def attention(q, k, v, seen, scale):
    """One sequence: q [H, T, d], k, v [Hkv, L, d], seen [T, L] -> o, lse, and
    sum_j p_ij |v_j| and the largest score's size (for tolerances).  A key
    that is not seen takes no part, whatever its numbers are."""
    H, T, d = q.shape
    G = H // k.shape[0]
    o, lse = np.zeros((H, T, d)), np.full((H, T), -np.inf)
    size, score = np.zeros((H, T, d)), np.zeros((H, T))
    plain = bool(np.isfinite(k).all() and np.isfinite(v).all())
    for h in range(H):
        kh, vh = k[h // G], v[h // G]
        if plain:  # all rows at once
            with np.errstate(invalid="ignore", divide="ignore"):
                s = np.where(seen, scale * (q[h] @ kh.T), -np.inf)
                m = s.max(-1, keepdims=True, initial=-np.inf)
                p = np.exp(s - np.where(np.isinf(m), 0, m))
                total = p.sum(-1, keepdims=True)
                lse[h] = (m + np.log(total))[:, 0]
                p = np.where(total > 0, p / total, 0)
            o[h], size[h] = p @ vh, p @ np.abs(vh)
            score[h] = scale * np.where(seen, np.abs(q[h]) @ np.abs(kh).T, 0).max(-1, initial=0)
            continue
        for t in range(T):
            j = np.nonzero(seen[t])[0]
            if not len(j):
                continue
            kk, vv = kh[j], vh[j]
            s = scale * (kk @ q[h, t])
            m = s.max()
            p = np.exp(s - m)
            lse[h, t] = m + np.log(p.sum())
            p /= p.sum()
            o[h, t] = p @ vv
            size[h, t] = p @ np.abs(vv)
            score[h, t] = scale * (np.abs(kk) @ np.abs(q[h, t])).max()
    return o, lse, size, score


def words_of(bits):
    """[..., T, T] truth values -> int32 words [..., T, ceil(T / 32)]."""
    T = bits.shape[-1]
    w = (T + 31) // 32
    pad = np.zeros(bits.shape[:-1] + (w * 32,), np.uint64)
    pad[..., :T] = bits
    words = (pad.reshape(bits.shape[:-1] + (w, 32)) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.from_numpy(words.astype(np.uint32).view(np.int32))


def random_trees(rng, B, T):
    bits = np.zeros((B, T, T), bool)
    for b in range(B):
        for i in range(T):
            bits[b, i, i] = True
            parent = rng.integers(-1, i) if i else -1
            if parent >= 0:
                bits[b, i] |= bits[b, parent]
    return bits


def page_table(rng, need, page, spare=3):
    """(int32 [B, max_pages], num_pages): pages in mixed order, -1 behind each
    sequence's own; `spare` pages belong to nobody."""
    pages = [-(-int(n) // page) for n in need]
    num = sum(pages) + spare
    order = rng.permutation(num)
    table = np.full((len(pages), max(1, max(pages))), -1, np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table), num


def place(cache, table, b, start, rows):
    """Writes rows [Hkv, n, ...] at positions start.. of sequence b of a host
    cache [num_pages, Hkv, page, ...]."""
    page = cache.shape[2]
    for i in range(rows.shape[1]):
        pos = start + i
        cache[int(table[b, pos // page]), :, pos % page] = rows[:, i]
