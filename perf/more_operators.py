"""Attention over a sliding window with a few first tokens that stay visible, and the paged cache behind it.

Five families:
  forward    windowed attention of whole sequences, equal lengths or packed back to back
  backward   its gradients
  cached     windowed attention of new tokens (one token: plain decode) over the paged cache
  plan       page tables, slot maps and positions of a step from its requests' lengths
  append     writing packed tokens to the cache by their slots

Query i sees key j when j <= i and (i - j < window or j < sinks). Where `own` is false, run() computes this with
elementary torch operations in fp32 (whole numbers in 64 bits); where it is true, it makes the library's calls on the
same state.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3, INT8, BF16 = "e4m3", "int8", "bf16"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short batch of ungrouped d = 64 heads at an odd length
        dict(name="window_forward_short", op="forward", packed=False, B=2, H=12, Hkv=12, N=1000, d=64, window=256,
             sinks=4),
        # a long document: the window is a sixteenth of it
        dict(name="window_forward_long", op="forward", packed=False, B=1, H=16, Hkv=4, N=16384, d=128, window=1024,
             sinks=4),
        # training on unequal documents packed back to back
        dict(name="window_train_packed", op="backward", packed=True, B=6, H=12, Hkv=12, N=4096, d=64, window=512,
             sinks=16),
        # training on long sequences with grouped heads
        dict(name="window_train_long", op="backward", packed=False, B=2, H=16, Hkv=4, N=8192, d=128, window=1024,
             sinks=4),
        # one sequence, one token: the smallest decode call
        dict(name="window_token", op="cached", fmt=BF16, B=1, H=16, Hkv=4, T=1, d=128, page=64, far=4096, window=512,
             sinks=4, tree=False),
        # a decode batch far behind whose windows the first pages are kept
        dict(name="window_tokens_e4m3", op="cached", fmt=E4M3, B=64, H=16, Hkv=4, T=1, d=128, page=64, far=32768,
             window=4096, sinks=4, tree=False),
        # drafted trees of an odd size, ungrouped d = 64 heads, small pages
        dict(name="window_drafts", op="cached", fmt=BF16, B=8, H=12, Hkv=12, T=23, d=64, page=16, far=16384,
             window=2048, sinks=64, tree=True),
        # chains of 64 tokens: 256 query rows share each key/value head
        dict(name="window_chains_int8", op="cached", fmt=INT8, B=16, H=16, Hkv=4, T=64, d=128, page=64, far=8192,
             window=1024, sinks=4, tree=False),
        # a decode step of 64 requests with windows: pages behind them go back
        dict(name="plan_step", op="plan", B=64, N=1, page=64, far=8192, window=1024, sinks=4),
        # prompts of unequal lengths admitted at once
        dict(name="plan_prompts", op="plan", B=512, N=2048, page=64, far=1, window=0, sinks=0),
        # one token for each of 64 requests
        dict(name="append_step_e4m3", op="append", fmt=E4M3, B=64, Hkv=4, N=1, d=128, page=64, far=8192),
        # packed prompts straight from a projection
        dict(name="append_prompts", op="append", fmt=BF16, B=32, Hkv=4, N=4096, d=128, page=64, far=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "backward", "cached", "cached", "plan", "append"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice([BF16, E4M3, INT8])
    H, Hkv = rng.choice([(16, 4), (12, 12), (16, 16), (8, 1), (6, 2), (5, 5)])
    sinks = rng.choice([0, 1, 4, 16, 64, 130])
    if op in ("forward", "backward"):
        N = _log_int(rng, 1, 16384)
        window = _log_int(rng, 1, min(N + 100, 4096))
        # rows x keys of no more than 16 heads of 16384 rows with 1024 keys, rows of no more than 16 x 16384
        B = _log_int(rng, 1, max(1, min(16, (16 << 14) // (N * H), (1 << 28) // (N * H * min(N, window + sinks)))))
        if N * H * min(N, window + sinks) > 1 << 28:
            window = max(1, (1 << 28) // (N * H) - sinks)
        return dict(op=op, packed=rng.random() < 0.5, B=B, H=H, Hkv=Hkv, N=N, d=d, window=window, sinks=sinks)
    if op == "cached":
        T = _log_int(rng, 1, 128)
        window = _log_int(rng, 1, 8192)
        tree = rng.random() < 0.5
        if tree:
            window = max(window, T)
        span = window + sinks + T
        keys = min((1 << 20) // Hkv // (2 if fmt == BF16 else 1), (20 << 20) // (H * T))
        far = _log_int(rng, 1, 65536)
        B = _log_int(rng, 1, max(1, min(64, keys // min(span, far + T))))
        return dict(op=op, fmt=fmt, B=B, H=H, Hkv=Hkv, T=T, d=d, page=page, far=far, window=window, sinks=sinks,
                    tree=tree)
    if op == "plan":
        N = _log_int(rng, 1, 2048)
        far = _log_int(rng, 1, 65536)
        B = _log_int(rng, 1, max(1, min(1024, (1 << 20) // N, (1 << 24) // (far + N))))
        return dict(op=op, B=B, N=N, page=page, far=far, window=rng.choice([0, _log_int(rng, 1, 8192)]), sinks=sinks)
    N = _log_int(rng, 1, 4096)
    B = _log_int(rng, 1, max(1, min(256, (1 << (19 if fmt == BF16 else 18)) // (N * Hkv))))
    return dict(op=op, fmt=fmt, B=B, Hkv=Hkv, N=N, d=d, page=page, far=_log_int(rng, 1, 8192))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _lengths(seed, B, far):
    """Unequal lengths on the host, the longest `far`: a server and a data loader both know them there. Every seed
    puts the same ones in another order."""
    n = torch.randint((far + 3) // 4, far + 1, (B,), generator=torch.Generator().manual_seed(B * 1000003 + far))
    n[0] = far
    return n[torch.randperm(B, generator=torch.Generator().manual_seed(int(seed) + 1))].tolist()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    B = case["B"]
    if case["op"] in ("forward", "backward"):
        return _prepare_whole(s, g, seed)
    if case["op"] == "cached":
        return _prepare_cached(s, g, seed)
    page, N = case["page"], case["N"]
    hist = [n - 1 for n in _lengths(seed, B, case["far"])]  # tokens that the cache holds before the step
    counts = _lengths(seed + 7, B, N)
    s["hist"], s["counts"] = _i32(hist), _i32(counts)
    if case["op"] == "plan":
        # the tables that the steps before have left: pages for every token that is still in reach, the window's lower
        # edge one step behind; all other pages in the pool's line
        W, S = case["window"], case["sinks"]
        max_pages = -(-(case["far"] + N) // page)
        i = torch.arange(max_pages, device=DEV)[None]
        have = i < -(-s["hist"].long()[:, None] // page)
        if W:
            edge = torch.div((s["hist"].long()[:, None] - W - page).clamp(min=0), page, rounding_mode="floor")
            have &= (i < -(-S // page)) | (i >= edge)
        used = int(have.sum())
        num = sum(-(-h // page) for h in hist) + sum(-(-n // page) + 1 for n in counts)
        order = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.full((B, max_pages), -1, device=DEV, dtype=torch.int32)
        s["table"][have] = order[:used]
        head = 5 % num  # the line is a ring: it does not begin at its first place
        s["free"] = torch.full((num,), -1, device=DEV, dtype=torch.int32)
        s["free"][(torch.arange(num - used, device=DEV) + head) % num] = order[used:]
        s["state"] = _i32([head, num - used])
        s["num"], s["total"] = num, sum(counts)
        s["slots"] = torch.zeros(s["total"], device=DEV, dtype=torch.int64)
        s["positions"] = torch.zeros(s["total"], device=DEV, dtype=torch.int32)
        s["cu"] = torch.zeros(B + 1, device=DEV, dtype=torch.int32)
        s["granted"] = torch.zeros(B, device=DEV, dtype=torch.int32)
        return s
    Hkv, d, fmt, total = case["Hkv"], case["d"], case["fmt"], sum(counts)
    need = torch.tensor([-(-(h + n) // page) for h, n in zip(hist, counts)], device=DEV)
    max_pages, used = -(-(case["far"] + N) // page), int(need.sum())
    num = sum(-(-h // page) for h in hist) + sum(-(-n // page) + 1 for n in counts)
    s["table"] = torch.full((B, max_pages), -1, device=DEV, dtype=torch.int32)
    s["table"][torch.arange(max_pages, device=DEV)[None] < need[:, None]] = \
        torch.randperm(num, generator=g, device=DEV)[:used].to(torch.int32)
    kv = _randn(g, total, 2 * Hkv, d) * torch.exp(0.5 * _randn(g, 1, 2 * Hkv, d))  # channels of unequal size
    kv = kv.to(torch.bfloat16)
    s["k"], s["v"] = kv[:, :Hkv].transpose(0, 1), kv[:, Hkv:].transpose(0, 1)  # [Hkv, total, d]
    b = torch.repeat_interleave(torch.arange(B, device=DEV), s["counts"].long())
    first = torch.cumsum(s["counts"].long(), 0) - s["counts"].long()
    pos = torch.arange(total, device=DEV) - first[b] + s["hist"].long()[b]
    s["slots"] = s["table"].long()[b, torch.div(pos, page, rounding_mode="floor")] * page + pos % page
    kind = {BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn, INT8: torch.int8}[fmt]
    s["kc"] = torch.zeros(num, Hkv, page, d, device=DEV, dtype=torch.uint8).to(kind)
    s["vc"] = torch.zeros_like(s["kc"])
    s["ks"] = torch.full((num, Hkv, page), 127, device=DEV, dtype=torch.uint8)
    s["vs"] = torch.full_like(s["ks"], 127)
    if fmt != BF16:
        s["k_back"] = torch.zeros(B, Hkv, N, d, device=DEV, dtype=torch.bfloat16)
        s["v_back"] = torch.zeros_like(s["k_back"])
    return s


def _prepare_whole(s, g, seed):
    B, H, Hkv, N, d = s["B"], s["H"], s["Hkv"], s["N"], s["d"]
    if s["packed"]:
        s["lens"] = _lengths(seed, B, N)
        s["cu"] = _i32([sum(s["lens"][:b]) for b in range(B + 1)])
        s["total"] = sum(s["lens"])
        lead, rows = (), s["total"]
    else:
        s["lens"], s["cu"], s["total"] = [N] * B, None, 0
        lead, rows = (B,), N
    s["q"] = (_randn(g, *lead, H, rows, d) * torch.exp(0.3 * _randn(g, H, 1, d))).to(torch.bfloat16)
    s["k"] = _randn(g, *lead, Hkv, rows, d).to(torch.bfloat16)
    s["v"] = _randn(g, *lead, Hkv, rows, d).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(d)
    if s["op"] == "forward":
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(*lead, H, rows, device=DEV)
        return s
    o, s["lse"] = _forward(s)  # what the forward pass has left
    s["o"] = o.to(torch.bfloat16)
    s["do"] = _randn(g, *lead, H, rows, d).to(torch.bfloat16)
    s["dq"], s["dk"], s["dv"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    s["ws"] = None
    return s


def _prepare_cached(s, g, seed):
    B, H, Hkv, T, d, page = s["B"], s["H"], s["Hkv"], s["T"], s["d"], s["page"]
    hist, drafts = _lengths(seed, B, s["far"]), _lengths(seed + 7, B, T)
    s["hist"], s["drafts"] = _i32(hist), _i32(drafts)
    need = torch.tensor([-(-(h + n) // page) for h, n in zip(hist, drafts)], device=DEV)[:, None]
    max_pages = int(need.max())
    i = torch.arange(max_pages, device=DEV)[None]
    edge = torch.div((s["hist"].long()[:, None] + 1 - s["window"]).clamp(min=0), page, rounding_mode="floor")
    have = (i < need) & ((i < -(-s["sinks"] // page)) | (i >= edge))  # pages out of reach have been given back
    num = int(have.sum())
    s["table"] = torch.full((B, max_pages), -1, device=DEV, dtype=torch.int32)
    s["table"][have] = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
    s["q"] = (_randn(g, B, H, T, d) * torch.exp(0.3 * _randn(g, 1, H, 1, d))).to(torch.bfloat16)
    s["kc"], s["ks"] = _stored(_randn(g, num * Hkv * page, d), s["fmt"], (num, Hkv, page, d))
    s["vc"], s["vs"] = _stored(_randn(g, num * Hkv * page, d), s["fmt"], (num, Hkv, page, d))
    s["mask"] = _tree_masks(g, B, T) if s["tree"] else None
    s["scale"] = 1.0 / math.sqrt(d)
    s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, H, T, device=DEV)
    s["ws"] = None
    return s


def _tree_masks(g, B, T):
    """Bits of each draft's ancestors and itself, 32 to a word: int32 [B, T, ceil(T / 32)]."""
    seen = torch.zeros(B, T, T, device=DEV, dtype=torch.bool)
    for i in range(T):
        seen[:, i, i] = True
        if i:  # a parent among the drafts before it, or (-1) the last token of the history
            parent = torch.randint(-1, i, (B,), generator=g, device=DEV)
            seen[:, i] |= seen[torch.arange(B, device=DEV), parent.clamp(min=0)] & (parent >= 0)[:, None]
    words = -(-T // 32)
    seen = torch.nn.functional.pad(seen, (0, words * 32 - T)).reshape(B, T, words, 32).long()
    bits = (seen << torch.arange(32, device=DEV)).sum(-1)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)


# ------------------------------------------------------------------ plain forms
def _pow2(e):
    """2^e in fp32, put together from its bits (a power function may be off in the last one)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantised(x, fmt):
    """(stored numbers, exponents) of fp32 rows: the smallest power of two that brings the row into the type's range."""
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    if fmt == E4M3:  # 448 = 0.875 * 2^9
        e = torch.where(m <= 0.875, e - 9, e - 8)
    else:  # 127 = 0.9921875 * 2^7
        e = torch.where(m <= 0.9921875, e - 7, e - 6)
    e = e.clamp(-100, 119)
    x = x * _pow2(-e)
    return (x.to(torch.float8_e4m3fn) if fmt == E4M3 else x.round().to(torch.int8)), e


def _stored(rows, fmt, shape):
    rows = rows.to(torch.bfloat16)
    if fmt == BF16:
        return rows.reshape(shape), torch.full(shape[:-1], 127, device=DEV, dtype=torch.uint8)
    x, e = _quantised(rows.float(), fmt)
    return x.reshape(shape), (e + 127).to(torch.uint8).reshape(shape[:-1])


def _sequences(s):
    """Index of each sequence's slice of a tensor [B, heads, N, ...] or [heads, total, ...], and its length."""
    at = 0
    for b, n in enumerate(s["lens"]):
        yield ((slice(None), slice(at, at + n)) if s["packed"] else (b,)), n
        at += n


BLOCK = 1024  # query rows whose scores are formed at once


def _blocks(s, n):
    """Query rows [i0, i1), the keys that any of them sees, and who sees which."""
    W, S = s["window"], s["sinks"]
    for i0 in range(0, n, BLOCK):
        i1 = min(n, i0 + BLOCK)
        lo = max(0, i0 - W + 1)
        first = min(S, lo)
        j = torch.cat((torch.arange(first, device=DEV), torch.arange(lo, i1, device=DEV)))
        i = torch.arange(i0, i1, device=DEV)[:, None]
        yield i0, i1, (first, lo), (j <= i) & ((i - j < W) | (j < S))


def _keys(x, i1, span):
    """Rows [0, first) and [lo, i1) of [Hkv, n, d]."""
    first, lo = span
    return torch.cat((x[:, :first], x[:, lo:i1]), 1) if first else x[:, lo:i1]


def _forward(s):
    H, Hkv, d = s["H"], s["Hkv"], s["d"]
    o, lse = torch.empty(s["q"].shape, device=DEV), torch.empty(s["q"].shape[:-1], device=DEV)
    for at, n in _sequences(s):
        q, k, v = s["q"][at].float(), s["k"][at].float(), s["v"][at].float()
        for i0, i1, span, sees in _blocks(s, n):
            kk, vv = _keys(k, i1, span), _keys(v, i1, span)
            x = q[:, i0:i1].reshape(Hkv, H // Hkv * (i1 - i0), d) @ kk.transpose(1, 2)
            x = x.reshape(H, i1 - i0, -1).mul_(s["scale"]).masked_fill_(~sees, -math.inf)
            m = x.amax(-1, keepdim=True)
            x = x.sub_(m).exp_()
            total = x.sum(-1, keepdim=True)
            y = x.reshape(Hkv, H // Hkv * (i1 - i0), -1) @ vv
            o[at][:, i0:i1] = y.reshape(H, i1 - i0, d) / total
            lse[at][:, i0:i1] = (m + total.log())[..., 0]
    return o, lse


def _backward(s):
    H, Hkv, d = s["H"], s["Hkv"], s["d"]
    dq = torch.empty(s["q"].shape, device=DEV)
    dk, dv = torch.zeros(s["k"].shape, device=DEV), torch.zeros(s["k"].shape, device=DEV)
    for at, n in _sequences(s):
        q, k, v, go = s["q"][at].float(), s["k"][at].float(), s["v"][at].float(), s["do"][at].float()
        lse, delta = s["lse"][at], (go * s["o"][at].float()).sum(-1)
        for i0, i1, span, sees in _blocks(s, n):
            kk, vv = _keys(k, i1, span), _keys(v, i1, span)
            rows = (Hkv, H // Hkv * (i1 - i0), d)
            qq, gg = q[:, i0:i1].reshape(rows), go[:, i0:i1].reshape(rows)
            p = (qq @ kk.transpose(1, 2)).reshape(H, i1 - i0, -1).mul_(s["scale"])
            p = p.sub_(lse[:, i0:i1, None]).exp_().masked_fill_(~sees, 0.0)
            dp = (gg @ vv.transpose(1, 2)).reshape(H, i1 - i0, -1)
            ds = dp.sub_(delta[:, i0:i1, None]).mul_(p).mul_(s["scale"]).reshape(Hkv, rows[1], -1)
            p = p.reshape(Hkv, rows[1], -1)
            dq[at][:, i0:i1] = (ds @ kk).reshape(H, i1 - i0, d)
            gk, gv = ds.transpose(1, 2) @ qq, p.transpose(1, 2) @ gg
            first, lo = span
            dk[at][:, :first] += gk[:, :first]
            dv[at][:, :first] += gv[:, :first]
            dk[at][:, lo:i1] += gk[:, first:]
            dv[at][:, lo:i1] += gv[:, first:]
    return dq, dk, dv


def _cached(s):
    B, H, T, d = s["q"].shape
    Hkv, page, W, S = s["kc"].shape[1], s["page"], s["window"], s["sinks"]
    hist, drafts = s["hist"].long()[:, None], s["drafts"].long()[:, None]
    max_pages = s["table"].shape[1]
    # the pages of the first tokens and those from the window's lower edge on
    edge = torch.div((hist + 1 - W).clamp(min=0), page, rounding_mode="floor")
    first = min(-(-S // page), max_pages)
    behind = edge + torch.arange(min(max_pages, (W + T) // page + 2), device=DEV)[None]
    pages = torch.cat((torch.arange(first, device=DEV).expand(B, first),
                       torch.where(behind < first, torch.full_like(behind, max_pages), behind)), 1)
    at = s["table"].long().gather(1, pages.clamp(max=max_pages - 1)).clamp(min=0)
    pos = (pages[:, :, None] * page + torch.arange(page, device=DEV)).flatten(1)[:, None]  # [B, 1, L]

    def rows(cache, scales):
        x = (cache.view(torch.uint8)[at].view(cache.dtype) if s["fmt"] != BF16 else cache[at]).float()
        if s["fmt"] != BF16:
            x *= _pow2(scales[at].int()[..., None] - 127)
        return x.transpose(1, 2).flatten(2, 3)  # [B, Hkv, L, d]

    k, v = rows(s["kc"], s["ks"]), rows(s["vc"], s["vs"])
    t = torch.arange(T, device=DEV)[None, :, None]
    draft = pos - hist[:, :, None]  # which draft a key is
    if s["mask"] is None:
        sees, depth = draft <= t, t
    else:
        b = draft.clamp(0, T - 1).expand(B, T, -1)
        sees = ((s["mask"].gather(2, b // 32) >> (b % 32)) & 1).bool()
        own_bits = sees & (draft >= 0) & (draft < drafts[:, :, None]) & (draft != t)
        depth = own_bits.sum(-1, keepdim=True)  # drafts before it on its path
    sees = (draft < 0) | (sees & (draft < drafts[:, :, None]))
    # a mask's drafts are all within the window (it is no shorter than the tree)
    near = hist[:, :, None] + depth - pos < W
    if s["mask"] is not None:
        near |= draft >= 0
    sees &= (near | (pos < S)) & (t < drafts[:, :, None])
    x = (q_rows(s["q"], Hkv) @ k.transpose(2, 3)).reshape(B, Hkv, H // Hkv, T, -1)
    x = x.mul_(s["scale"]).masked_fill_(~sees[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True).reshape(B, H, T, 1)
    o = (x.reshape(B, Hkv, H // Hkv * T, -1) @ v).reshape(B, H, T, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o, (m.reshape(B, H, T, 1) + total.log())[..., 0]


def q_rows(q, Hkv):
    B, H, T, d = q.shape
    return q.float().reshape(B, Hkv, H // Hkv * T, d)


def _plan(s):
    """Updates table, line of free pages and its state; (slots, positions, cu_seqlens, granted)."""
    table, free, page, num = s["table"], s["free"], s["page"], s["num"]
    B, max_pages = table.shape
    hist, counts = s["hist"].long(), s["counts"].long()
    i = torch.arange(max_pages, device=DEV)[None]
    head, count = s["state"].long()[0], s["state"].long()[1]
    freed = torch.zeros(0, device=DEV, dtype=torch.int32)
    if s["window"]:
        # pages below the first position that the step's first token sees, down to the first that is gone already
        edge = torch.div((hist + 1 - s["window"]).clamp(min=0), page, rounding_mode="floor")[:, None]
        there = ((table >= 0) | (i >= edge)).long()
        run = torch.cumprod(there.flip(1), 1).flip(1).bool()
        out = run & (i < edge) & (i >= -(-s["sinks"] // page))
        freed = table[out]
        table[out] = -1
        free[(head + count + torch.arange(freed.numel(), device=DEV)) % num] = freed
    count = count + freed.numel()
    first = torch.div(hist, page, rounding_mode="floor")[:, None]
    last = torch.div(hist + counts - 1, page, rounding_mode="floor")[:, None]
    need = (table < 0) & (i >= first) & (i <= last)
    where = need.nonzero()
    taken = where.shape[0]  # the pool has enough for the step
    table[where[:, 0], where[:, 1]] = free[(head + torch.arange(taken, device=DEV)) % num]
    s["state"].copy_(torch.stack(((head + taken) % num, count - taken)))
    b = torch.repeat_interleave(torch.arange(B, device=DEV), counts, output_size=s["total"])
    cu = torch.cumsum(counts, 0)
    pos = torch.arange(s["total"], device=DEV) - (cu - counts)[b] + hist[b]
    slots = table.long()[b, torch.div(pos, page, rounding_mode="floor")] * page + pos % page
    cu = torch.cat((torch.zeros_like(cu[:1]), cu))
    return slots, pos.to(torch.int32), cu.to(torch.int32), s["counts"].clone()


def _append(s):
    page = s["page"]
    pg, row = torch.div(s["slots"], page, rounding_mode="floor"), s["slots"] % page
    for x, cache, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x = x.transpose(0, 1)
        if s["fmt"] == BF16:
            cache[pg, :, row] = x
            continue
        x, e = _quantised(x.float(), s["fmt"])
        cache.view(torch.uint8)[pg, :, row] = x.view(torch.uint8)
        scales[pg, :, row] = (e + 127).to(torch.uint8)[..., 0]


def _read(s, cache, scales, back):
    """The step's tokens back from an 8-bit cache: what it holds as the numbers it stands for."""
    B, Hkv, N, d = back.shape
    n = torch.arange(N, device=DEV)[None]
    b, n = (n < s["counts"][:, None]).nonzero(as_tuple=True)
    pos = s["hist"].long()[b] + n
    pg, row = s["table"].long()[b, torch.div(pos, s["page"], rounding_mode="floor")], pos % s["page"]
    x = cache.view(torch.uint8)[pg, :, row].view(cache.dtype).float()
    back.transpose(1, 2)[b, n] = (x * _pow2(scales[pg, :, row].int()[..., None] - 127)).to(torch.bfloat16)
    return back


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    if s["op"] == "forward":
        o, lse = _forward(s)
        return dict(o=o.to(torch.bfloat16), lse=lse)
    if s["op"] == "backward":
        return {name: x.to(torch.bfloat16) for name, x in zip(("dq", "dk", "dv"), _backward(s))}
    if s["op"] == "cached":
        o, lse = _cached(s)
        return dict(o=o.to(torch.bfloat16), lse=lse)
    if s["op"] == "plan":
        slots, positions, cu, granted = _plan(s)
        return dict(table=s["table"], free=s["free"], state=s["state"], slots=slots, positions=positions, cu=cu,
                    granted=granted)
    _append(s)
    if s["fmt"] == BF16:
        return dict(k=s["kc"], v=s["vc"])
    return dict(k=_read(s, s["kc"], s["ks"], s["k_back"]), v=_read(s, s["vc"], s["vs"], s["v_back"]))


def _own(s):
    import io_aware_exact_15_gb300 as fa

    op = s["op"]
    if op in ("forward", "backward"):
        size = (s["B"], s["H"], s["Hkv"], s["N"], s["total"], s["d"])
        reach = (s["window"], s["sinks"])
        if op == "forward":
            status = fa.fa_forward_window(s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu"], *size, s["scale"], *reach)
            out = dict(o=s["o"], lse=s["lse"])
        else:
            if s["ws"] is None:  # kept from call to call
                s["ws"] = torch.empty(fa.fa_backward_window_workspace_size(*size, *reach), device=DEV,
                                      dtype=torch.uint8)
            status = fa.fa_backward_window(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["dq"], s["dk"],
                                           s["dv"], s["cu"], *size, s["scale"], *reach, s["ws"], s["ws"].numel())
            out = dict(dq=s["dq"], dk=s["dk"], dv=s["dv"])
    elif op == "plan":
        B, max_pages = s["table"].shape
        status = fa.fa_cache_plan(s["hist"], s["counts"], s["table"], s["free"], s["state"], s["slots"],
                                  s["positions"], s["cu"], s["granted"], B, s["total"], s["num"], s["page"], max_pages,
                                  s["window"], s["sinks"])
        out = {k: s[k] for k in ("table", "free", "state", "slots", "positions", "cu", "granted")}
    else:
        num, Hkv, page, d = s["kc"].shape
        form = {BF16: fa.FA_CACHE_BF16, E4M3: fa.FA_CACHE_E4M3, INT8: fa.FA_CACHE_INT8}[s["fmt"]]
        max_pages = s["table"].shape[1]
        if op == "cached":
            B, H, T, d = s["q"].shape
            if s["ws"] is None:  # kept as well
                s["ws"] = torch.empty(fa.fa_tree_attention_workspace_size(B, H, Hkv, T, d), device=DEV,
                                      dtype=torch.uint8)
            status = fa.fa_tree_attention_window(
                s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["hist"], s["drafts"], s["mask"], s["o"],
                s["lse"], form, B, H, Hkv, T, d, num, page, max_pages, s["scale"], s["window"], s["sinks"], s["ws"],
                s["ws"].numel())
            out = dict(o=s["o"], lse=s["lse"])
        else:
            status = fa.fa_cache_append_slots(
                s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"], form, Hkv, s["slots"].numel(), d, num,
                page, s["k"].stride()[:2] + s["v"].stride()[:2])
            out = dict(k=s["kc"], v=s["vc"])
            if s["fmt"] != BF16:
                B, _, N, _ = s["k_back"].shape
                status = status or fa.fa_cache_read(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["hist"],
                                                    s["counts"], s["k_back"], s["v_back"], form, B, Hkv, N, d, num,
                                                    page, max_pages)
                out = dict(k=s["k_back"], v=s["v_back"])
    if status != fa.FA_OK:
        raise fa.FaError(status, op)
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def _expected_len(B, far):
    """Mean of _lengths: one sequence of `far`, the others uniform on [far / 4, far]."""
    return (far + (B - 1) * ((far + 3) // 4 + far) / 2) / B


def _pairs(n, W, S):
    """Query and key pairs of a sequence of n tokens: a window each, and the first tokens before it."""
    w = min(n, W)
    pairs = n * w - w * (w - 1) / 2
    m = max(0, n - W)  # rows whose window leaves some tokens out, the r-th of them r (r = 1 .. m)
    f = min(S, m)
    return pairs + f * (f + 1) / 2 + (m - f) * f


def work(case):
    B = case["B"]
    if case["op"] in ("forward", "backward"):
        H, Hkv, d, W, S = case["H"], case["Hkv"], case["d"], case["window"], case["sinks"]
        n = _expected_len(B, case["N"]) if case["packed"] else case["N"]
        pairs = B * H * _pairs(n, W, S)
        rows, kv = B * H * n, B * Hkv * n
        if case["op"] == "forward":
            return {"bytes": rows * (4 * d + 4) + kv * 4 * d, "flops": 4 * d * pairs}
        return {"bytes": rows * (8 * d + 4) + kv * 8 * d, "flops": 10 * d * pairs}
    if case["op"] == "plan":
        hist, n, page = _expected_len(B, case["far"]) - 1, _expected_len(B, case["N"]), case["page"]
        new = (hist + n) // page - hist // page + 1  # pages that the step's tokens touch
        # lengths and counts, the table's entries and the line's; slots, positions, offsets, what was granted
        return {"bytes": B * (8 + 3 * 4 * new + n * 12 + 8) + 16, "flops": B * n * 4}
    Hkv, d, fmt = case["Hkv"], case["d"], case["fmt"]
    elt = 2 if fmt == BF16 else 1
    scale = 0 if fmt == BF16 else 1
    if case["op"] == "append":
        rows = 2 * Hkv * B * _expected_len(B, case["N"])
        # bf16 in, stored out; in 8 bits also read back: stored in, bf16 out
        return {"bytes": rows * (2 * d + elt * d + scale) * (1 if fmt == BF16 else 2) + rows / (2 * Hkv) * 8,
                "flops": rows * d * 4}
    H, T, W, S = case["H"], case["T"], case["window"], case["sinks"]
    hist, n = _expected_len(B, case["far"]), _expected_len(B, T)
    per_row = min(W, hist + n / 2) + min(S, max(0, hist - W))  # keys of a draft
    keys = B * (min(W + n - 1, hist + n) + min(S, max(0, hist + 1 - W)))
    words = -(-T // 32) if case["tree"] else 0
    return {"bytes": keys * Hkv * 2 * (elt * d + scale) + H * B * T * (4 * d + 4) + keys / case["page"] * 4
            + B * (T * words * 4 + 8),
            "flops": 4 * d * H * B * n * per_row}


# ------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "forward":
        return _whole_64(s)
    if case["op"] == "backward":
        return _gradients_64(s)
    if case["op"] == "cached":
        return _cached_64(s)
    if case["op"] == "plan":
        return _plan_64(s)
    return _append_64(s)


def _rows_64(s, n):
    """Stretches of query rows with the list of keys that any of them may see and -inf where one does not."""
    step = 2048
    for r0 in range(0, n, step):
        r1 = min(n, r0 + step)
        j = torch.arange(n, device=DEV)
        j = j[(j < r1) & ((j > r0 - s["window"]) | (j < s["sinks"]))]
        age = torch.arange(r0, r1, device=DEV)[:, None] - j[None]
        hide = torch.zeros(age.shape, device=DEV, dtype=torch.float64)
        hide[(age < 0) | ((age >= s["window"]) & (j >= s["sinks"])[None])] = -math.inf
        yield slice(r0, r1), j, hide


def _whole_64(s):
    o = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
    lse = torch.zeros(s["q"].shape[:-1], device=DEV, dtype=torch.float64)
    for at, n in _sequences(s):
        for rows, j, hide in _rows_64(s, n):
            for h in range(s["H"]):
                hk = h * s["Hkv"] // s["H"]
                x = s["q"][at][h, rows].double() @ s["k"][at][hk, j].double().T * s["scale"] + hide
                lse[at][h, rows] = torch.logsumexp(x, -1)
                o[at][h, rows] = torch.softmax(x, -1) @ s["v"][at][hk, j].double()
    return dict(o=o, lse=lse)


def _gradients_64(s):
    """By the chain rule through the scores, with the softmax's statistics as they were handed over."""
    like = lambda x: torch.zeros(x.shape, device=DEV, dtype=torch.float64)
    dq, dk, dv = like(s["q"]), like(s["k"]), like(s["v"])
    for at, n in _sequences(s):
        for rows, j, hide in _rows_64(s, n):
            for h in range(s["H"]):
                hk = h * s["Hkv"] // s["H"]
                q, g = s["q"][at][h, rows].double(), s["do"][at][h, rows].double()
                k, v = s["k"][at][hk, j].double(), s["v"][at][hk, j].double()
                p = torch.exp(q @ k.T * s["scale"] + hide - s["lse"][at][h, rows].double()[:, None])
                inner = torch.einsum("nd,nd->n", g, s["o"][at][h, rows].double())
                dx = p * (g @ v.T - inner[:, None]) * s["scale"]
                dq[at][h, rows] = dx @ k
                dk[at][hk].index_add_(0, j, dx.T @ q)
                dv[at][hk].index_add_(0, j, p.T @ g)
    return dict(dq=dq, dk=dk, dv=dv)


def _pow2_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _cached_64(s):
    B, H, T, d = s["q"].shape
    Hkv, page = s["kc"].shape[1], s["page"]
    o = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
    lse = torch.full(s["lse"].shape, -math.inf, device=DEV, dtype=torch.float64)
    mask = s["mask"].tolist() if s["mask"] is not None else None
    table = s["table"].tolist()
    for b in range(B):
        hist, n = int(s["hist"][b]), int(s["drafts"][b])
        place = [[(mask[b][i][j // 32] >> (j % 32)) & 1 if mask else int(j <= i) for j in range(n)] for i in range(n)]
        ahead = [sum(row) - row[i] for i, row in enumerate(place)]  # drafts before each on its path
        keys = sorted(set(range(min(s["sinks"], hist))) | set(range(max(0, hist + 1 - s["window"]), hist)))
        sees = torch.zeros(n, len(keys) + n, dtype=torch.bool)
        old = torch.tensor(keys, dtype=torch.int64)
        for i in range(n):
            sees[i, :len(keys)] = (old < s["sinks"]) | (old > hist + ahead[i] - s["window"])
            for j in range(n):
                near = ahead[i] - ahead[j] < s["window"] or hist + j < s["sinks"]
                sees[i, len(keys) + j] = bool(place[i][j]) and near
        where = keys + [hist + j for j in range(n)]
        pg = torch.tensor([table[b][p // page] for p in where], device=DEV)
        row = torch.tensor([p % page for p in where], device=DEV)
        k, v = (_values_64(s, c, e, pg, row) for c, e in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        hide = torch.zeros(sees.shape, dtype=torch.float64).masked_fill(~sees, -math.inf).to(DEV)
        for h in range(H):
            x = s["q"][b, h, :n].double() @ k[:, h * Hkv // H].T * s["scale"] + hide
            lse[b, h, :n] = torch.logsumexp(x, -1)
            o[b, h, :n] = torch.softmax(x, -1) @ v[:, h * Hkv // H]
    return dict(o=o, lse=lse)


def _values_64(s, cache, scales, pg, row):
    """[keys, Hkv, d]"""
    if s["fmt"] == BF16:
        return cache[pg, :, row].double()
    x = cache.view(torch.uint8)[pg, :, row].view(cache.dtype).double()
    return x * _pow2_64(scales[pg, :, row].long() - 127)[..., None]


def _plan_64(s):
    """Request by request and token by token on the host."""
    table, free, (head, count) = s["table"].tolist(), s["free"].tolist(), s["state"].tolist()
    hist, counts, page, num = s["hist"].tolist(), s["counts"].tolist(), s["page"], s["num"]
    if s["window"]:
        for b, h in enumerate(hist):
            gone = []
            i = max(0, h + 1 - s["window"]) // page - 1
            while i >= -(-s["sinks"] // page) and table[b][i] >= 0:
                gone.append(table[b][i])
                table[b][i] = -1
                i -= 1
            for x in reversed(gone):
                free[(head + count) % num] = x
                count += 1
    slots, positions, cu = [], [], [0]
    for b, h in enumerate(hist):
        for p in range(h, h + counts[b]):
            if table[b][p // page] < 0:
                table[b][p // page] = free[head]
                head, count = (head + 1) % num, count - 1
            slots.append(table[b][p // page] * page + p % page)
            positions.append(p)
        cu.append(len(slots))
    whole = lambda x: torch.tensor(x, dtype=torch.int64)
    return dict(table=whole(table), free=whole(free), state=whole([head, count]), slots=whole(slots),
                positions=whole(positions), cu=whole(cu), granted=whole(counts))


def _append_64(s):
    """Each element the nearest multiple of the type's step at its size (ties to even), from the definition."""
    out = {}
    where = s["slots"].tolist()
    counts, hist = s["counts"].tolist(), s["hist"].tolist()
    for name in ("k", "v"):
        x = s[name].double()  # [Hkv, total, d]
        if s["fmt"] == BF16:
            y = s[name + "c"].double().transpose(1, 2).flatten(0, 1)  # [slots, Hkv, d]
            y[torch.tensor(where, device=DEV)] = x.transpose(0, 1)
            out[name] = y.unflatten(0, (-1, s["page"])).transpose(1, 2)
            continue
        most = 448.0 if s["fmt"] == E4M3 else 127.0
        share = x.abs().amax(-1, keepdim=True) / most
        e = torch.ceil(torch.log2(share)).clamp(-100, 119)
        e = torch.where(share <= _pow2_64(e - 1), e - 1, torch.where(share > _pow2_64(e), e + 1, e)).clamp(-100, 119)
        z = x / _pow2_64(e)
        if s["fmt"] == E4M3:  # three bits after the leading one, down to steps of 2^-9
            step = _pow2_64((z.abs().clamp(min=2.0 ** -6).view(torch.int64) >> 52) - 1023 - 3)
        else:
            step = torch.ones_like(z)
        y = torch.round(z / step) * step * _pow2_64(e)
        back = torch.zeros(s["k_back"].shape, device=DEV, dtype=torch.float64)
        at = 0
        for b, n in enumerate(counts):
            back[b, :, :n] = y[:, at:at + n]
            at += n
        out[name] = back
    return out
