"""The serving and Q/K preparation operators, as cases that can be timed and compared.

Three families:
  norm_rope   per-head RMS norm of queries and keys with the position rotation, forward and backward
  cache       quantising new tokens into a paged cache and reading them back
  tree        attention of drafted tokens (one token: plain decode) over the paged cache

Where `own` is false, run() computes them with elementary torch operations in fp32; where it is true, it makes the
library's calls on the same state.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3, INT8, BF16 = "e4m3", "int8", "bf16"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of 8 sequences: one token each, grouped heads
        dict(name="norm_rope_step", op="norm_rope", back=False, B=8, H=16, Hkv=4, N=1, d=128, rot=128, inter=False,
             far=8192),
        # prompts of 4 x 4096 tokens straight from a packed QKV projection
        dict(name="norm_rope_prompt", op="norm_rope", back=False, B=4, H=16, Hkv=4, N=4096, d=128, rot=128,
             inter=False, far=4096),
        # the same batch in training: gradients of Q, K and both norm weights
        dict(name="norm_rope_train", op="norm_rope", back=True, B=4, H=16, Hkv=4, N=4096, d=128, rot=128, inter=False,
             far=4096),
        # ungrouped d = 64 heads, an odd length, half of the dimensions rotated in adjacent pairs
        dict(name="norm_rope_train_d64", op="norm_rope", back=True, B=8, H=12, Hkv=12, N=1023, d=64, rot=32,
             inter=True, far=2000),
        # the cache write of a decode step: one new token for each of 32 sequences
        dict(name="cache_step_e4m3", op="cache", fmt=E4M3, B=32, Hkv=4, N=1, d=128, page=64, far=8192),
        # prompts written at once, unequal lengths
        dict(name="cache_prompt_int8", op="cache", fmt=INT8, B=16, Hkv=4, N=4096, d=128, page=64, far=1),
        # one sequence, one token, a short history: the smallest decode call
        dict(name="tree_first", op="tree", fmt=BF16, B=1, H=16, Hkv=4, T=1, d=128, page=64, far=512, tree=False),
        # a decode batch: one token each over unequal histories
        dict(name="tree_tokens_e4m3", op="tree", fmt=E4M3, B=32, H=16, Hkv=4, T=1, d=128, page=64, far=8192,
             tree=False),
        # drafted trees of an odd size over long histories, unquantised
        dict(name="tree_drafts", op="tree", fmt=BF16, B=8, H=16, Hkv=4, T=23, d=128, page=64, far=16384, tree=True),
        # large trees: 256 query rows share each key/value head
        dict(name="tree_drafts_int8", op="tree", fmt=INT8, B=16, H=16, Hkv=4, T=64, d=128, page=64, far=8192,
             tree=True),
        # two very long sequences
        dict(name="tree_long_e4m3", op="tree", fmt=E4M3, B=2, H=16, Hkv=4, T=16, d=128, page=128, far=131072,
             tree=True),
        # ungrouped d = 64 heads with small pages
        dict(name="tree_d64", op="tree", fmt=BF16, B=8, H=12, Hkv=12, T=33, d=64, page=16, far=4096, tree=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "cache", "tree", "tree"])
    d = rng.choice([64, 128])
    H, Hkv = rng.choice([(16, 4), (12, 12), (16, 16), (8, 1), (6, 2), (32, 8), (5, 5)])
    if op == "norm_rope":
        back = rng.random() < 0.5
        N = _log_int(rng, 1, 8192)
        B = _log_int(rng, 1, max(1, min(64, 327680 // (N * (H + Hkv)))))  # rows as in 16384 tokens of 20 heads
        rot = rng.choice([d, d, d // 2, 16])
        return dict(op=op, back=back, B=B, H=H, Hkv=Hkv, N=N, d=d, rot=rot, inter=rng.random() < 0.5,
                    far=N + _log_int(rng, 1, 100000))
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice([BF16, E4M3, INT8])
    if op == "cache":
        N = _log_int(rng, 1, 8192)
        B = _log_int(rng, 1, max(1, min(128, 262144 // (N * Hkv))))
        return dict(op=op, fmt=fmt, B=B, Hkv=Hkv, N=N, d=d, page=page, far=_log_int(rng, 1, 8192))
    T = _log_int(rng, 1, 128)
    keys = (1 << 20) // (Hkv * (2 if fmt == BF16 else 1))  # of all sequences: the bytes of two times 131072 at e4m3
    keys = min(keys, (80 << 20) // (H * T))  # and the products of 16 times 5120 with 1024 rows of queries each
    far = _log_int(rng, 1, min(131072, keys))
    B = _log_int(rng, 1, max(1, min(64, keys // far)))
    return dict(op=op, fmt=fmt, B=B, H=H, Hkv=Hkv, T=T, d=d, page=page, far=far, tree=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _randint(g, lo, hi, *shape):
    """Whole numbers of [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int64)


def _tables(rows, rot):
    """cos and sin of position x base^(-2 i / rot), formed in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * inv[None]
    return a.cos().float(), a.sin().float()


def _pages(g, B, need, page):
    """A page table that hands out the pages of a pool in mixed order; entries past a sequence's need hold -1."""
    max_pages = max(1, int(-(-int(need.max()) // page)))
    used = torch.arange(max_pages, device=DEV)[None] < (-(-need // page))[:, None]
    num = B * max_pages
    table = torch.randperm(num, generator=g, device=DEV).reshape(B, max_pages)
    return torch.where(used, table, torch.full_like(table, -1)).to(torch.int32), num


def _lengths(g, B, far):
    """Unequal lengths, the longest `far`."""
    n = _randint(g, (far + 3) // 4, far, B)
    n[int(_randint(g, 0, B - 1, 1))] = far
    return n


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    if case["op"] == "norm_rope":
        H, N, rot = case["H"], case["N"], case["rot"]
        qkv = _randn(g, B, N, H + 2 * Hkv, d)
        qkv *= torch.exp(0.5 * _randn(g, 1, 1, H + 2 * Hkv, d))  # channels of unequal size
        qkv = qkv.to(torch.bfloat16)
        s["q"], s["k"] = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hkv].transpose(1, 2)
        s["wq"], s["wk"] = 1 + 0.2 * _randn(g, d), 1 + 0.2 * _randn(g, d)
        rows = max(case["far"], N)
        s["cos"], s["sin"] = _tables(rows, rot)
        first = _randint(g, 0, rows - N, B)  # each sequence goes on from its own position
        s["pos"] = (first[:, None] + torch.arange(N, device=DEV)[None]).to(torch.int32)
        if case["back"]:
            s["gq"] = _randn(g, B, H, N, d).to(torch.bfloat16)
            s["gk"] = _randn(g, B, Hkv, N, d).to(torch.bfloat16)
            dqkv = torch.zeros(B, N, H + 2 * Hkv, d, device=DEV, dtype=torch.bfloat16)
            s["dq"], s["dk"] = dqkv[:, :, :H].transpose(1, 2), dqkv[:, :, H:H + Hkv].transpose(1, 2)
            s["dwq"], s["dwk"] = torch.zeros(d, device=DEV), torch.zeros(d, device=DEV)
            s["ws"] = None
        else:
            s["qo"] = torch.zeros(B, H, N, d, device=DEV, dtype=torch.bfloat16)
            s["ko"] = torch.zeros(B, Hkv, N, d, device=DEV, dtype=torch.bfloat16)
        return s
    page, fmt = case["page"], case["fmt"]
    kind = {BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn, INT8: torch.int8}[fmt]
    if case["op"] == "cache":
        N = case["N"]
        kv = _randn(g, B, N, 2 * Hkv, d) * torch.exp(0.5 * _randn(g, 1, 1, 2 * Hkv, d))
        kv = kv.to(torch.bfloat16)
        s["k"], s["v"] = kv[:, :, :Hkv].transpose(1, 2), kv[:, :, Hkv:].transpose(1, 2)
        s["start"] = (_lengths(g, B, case["far"]) - 1).to(torch.int32)
        s["counts"] = _lengths(g, B, N).to(torch.int32)
        table, num = _pages(g, B, (s["start"] + s["counts"]).long(), page)
        s["table"] = table
        s["kc"] = torch.zeros(num, Hkv, page, d, device=DEV, dtype=torch.uint8).to(kind)
        s["vc"] = torch.zeros_like(s["kc"])
        s["ks"] = torch.full((num, Hkv, page), 127, device=DEV, dtype=torch.uint8)
        s["vs"] = torch.full_like(s["ks"], 127)
        s["k_back"] = torch.zeros(B, Hkv, N, d, device=DEV, dtype=torch.bfloat16)
        s["v_back"] = torch.zeros_like(s["k_back"])
        return s
    H, T = case["H"], case["T"]
    hist = _lengths(g, B, case["far"])
    drafts = _lengths(g, B, T)
    s["hist"], s["drafts"] = hist.to(torch.int32), drafts.to(torch.int32)
    s["table"], num = _pages(g, B, hist + drafts, page)
    s["q"] = (_randn(g, B, H, T, d) * torch.exp(0.3 * _randn(g, 1, H, 1, d))).to(torch.bfloat16)
    rows = _randn(g, num * Hkv * page, d)  # every page holds something, also where no sequence owns it
    s["kc"], s["ks"] = _stored(rows, fmt, (num, Hkv, page, d))
    rows = _randn(g, num * Hkv * page, d)
    s["vc"], s["vs"] = _stored(rows, fmt, (num, Hkv, page, d))
    s["mask"] = _tree_masks(g, B, T) if case["tree"] else None
    s["scale"] = 1.0 / math.sqrt(d)
    s["o"] = torch.zeros(B, H, T, d, device=DEV, dtype=torch.bfloat16)
    s["lse"] = torch.zeros(B, H, T, device=DEV)
    s["ws"] = None
    return s


def _tree_masks(g, B, T):
    """Bits of each draft's ancestors and itself, 32 to a word: int32 [B, T, ceil(T / 32)]."""
    seen = torch.zeros(B, T, T, device=DEV, dtype=torch.bool)
    for i in range(T):
        seen[:, i, i] = True
        if i:  # a parent among the drafts before it, or (-1) the last token of the history
            parent = _randint(g, -1, i - 1, B)
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
    e = e.clamp(-117, 119)
    x = x * _pow2(-e)
    return (x.to(torch.float8_e4m3fn) if fmt == E4M3 else x.round().to(torch.int8)), e


def _stored(rows, fmt, shape):
    rows = rows.to(torch.bfloat16)
    if fmt == BF16:
        return rows.reshape(shape), torch.full(shape[:-1], 127, device=DEV, dtype=torch.uint8)
    x, e = _quantised(rows.float(), fmt)
    return x.reshape(shape), (e + 127).to(torch.uint8).reshape(shape[:-1])


def _rotate(y, cos, sin, rot, inter, back):
    """The first `rot` elements of y turned by each row's angles (against them where `back`)."""
    sin = -sin if back else sin
    z = y[..., :rot]
    if inter:
        a, b = z[..., 0::2], z[..., 1::2]
        z = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = z[..., :rot // 2], z[..., rot // 2:]
        z = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((z, y[..., rot:]), -1)


def _norm_rope(s, x, w, real):
    at = s["pos"].long()
    cos, sin = s["cos"].to(real)[at][:, None], s["sin"].to(real)[at][:, None]
    x = x.to(real)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return _rotate(x * r * w.to(real), cos, sin, s["rot"], s["inter"], False)


def _norm_rope_back(s, g, x, w, real):
    at = s["pos"].long()
    cos, sin = s["cos"].to(real)[at][:, None], s["sin"].to(real)[at][:, None]
    g = _rotate(g.to(real), cos, sin, s["rot"], s["inter"], True)
    x = x.to(real)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    x = x * r
    dw = (g * x).sum((0, 1, 2))
    g = g * w.to(real)
    return r * (g - x * (g * x).mean(-1, keepdim=True)), dw


def _slots(s, at):
    """Page and row of positions at [B, n]."""
    page = s["page"]
    where = torch.div(at, page, rounding_mode="floor").clamp(max=s["table"].shape[1] - 1)
    return s["table"].long().gather(1, where), at % page


def _write(s, x, cache, scales):
    B, Hkv, N, d = x.shape
    n = torch.arange(N, device=x.device)[None]
    b, n = (n < s["counts"][:, None]).nonzero(as_tuple=True)  # the tokens that exist
    pg, row = _slots(s, s["start"].long()[:, None] + torch.arange(N, device=x.device)[None])
    pg, row = pg[b, n], row[b, n]
    x = x.transpose(1, 2)[b, n].float()
    if s["fmt"] == BF16:
        cache[pg, :, row] = x.to(torch.bfloat16)
        return
    x, e = _quantised(x, s["fmt"])
    cache.view(torch.uint8)[pg, :, row] = x.view(torch.uint8)
    scales[pg, :, row] = (e + 127).to(torch.uint8)[..., 0]


def _read(s, cache, scales, back):
    B, Hkv, N, d = back.shape
    n = torch.arange(N, device=back.device)[None]
    b, n = (n < s["counts"][:, None]).nonzero(as_tuple=True)
    pg, row = _slots(s, s["start"].long()[:, None] + torch.arange(N, device=back.device)[None])
    pg, row = pg[b, n], row[b, n]
    x = cache.view(torch.uint8)[pg, :, row].view(cache.dtype) if s["fmt"] != BF16 else cache[pg, :, row]
    x = x.float()
    if s["fmt"] != BF16:
        x = x * _pow2(scales[pg, :, row].int()[..., None] - 127)
    back.transpose(1, 2)[b, n] = x.to(torch.bfloat16)
    return back


def _all_keys(s, cache, scales, b, real):
    """Keys or values of the sequences of slice b in order: [sequences, Hkv, max_pages * page, d]."""
    table = s["table"][b].long().clamp(min=0)
    n, pages = table.shape
    x = cache.view(torch.uint8)[table].view(cache.dtype) if s["fmt"] != BF16 else cache[table]
    x = x.to(real)
    if s["fmt"] != BF16:
        x *= _pow2(scales[table].int()[..., None] - 127)
    return x.transpose(1, 2).reshape(n, x.shape[2], pages * s["page"], s["d"])


def _tree(s, b, real):
    q = s["q"][b].to(real)
    n, H, T, d = q.shape
    Hkv = s["kc"].shape[1]
    k, v = _all_keys(s, s["kc"], s["ks"], b, real), _all_keys(s, s["vc"], s["vs"], b, real)
    L = k.shape[2]
    hist, drafts = s["hist"][b].long()[:, None, None], s["drafts"][b].long()[:, None, None]
    j, i = torch.arange(L, device=q.device)[None, None], torch.arange(T, device=q.device)[None, :, None]
    draft = j - hist  # which draft a key is
    if s["mask"] is None:
        sees = draft <= i
    else:
        at = draft.clamp(0, T - 1).expand(n, T, L)
        sees = ((s["mask"][b].gather(2, at // 32) >> (at % 32)) & 1).bool()
    sees = ((draft < 0) | (sees & (draft < drafts))) & (i < drafts)  # [n, T, L]
    x = (q.reshape(n, Hkv, H // Hkv * T, d) @ k.transpose(2, 3)).reshape(n, Hkv, H // Hkv, T, L)
    del k
    x = x.mul_(s["scale"]).masked_fill_(~sees[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.reshape(n, Hkv, H // Hkv * T, L) @ v).reshape(n, H, T, d)
    total, m = total.reshape(n, H, T, 1), m.reshape(n, H, T, 1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o, (m + total.log())[..., 0]


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    if s["op"] == "norm_rope":
        real = torch.float32
        if s["back"]:
            dq, dwq = _norm_rope_back(s, s["gq"], s["q"], s["wq"], real)
            dk, dwk = _norm_rope_back(s, s["gk"], s["k"], s["wk"], real)
            return dict(dq=dq.to(torch.bfloat16), dk=dk.to(torch.bfloat16), dwq=dwq, dwk=dwk)
        return dict(q=_norm_rope(s, s["q"], s["wq"], real).to(torch.bfloat16),
                    k=_norm_rope(s, s["k"], s["wk"], real).to(torch.bfloat16))
    if s["op"] == "cache":
        _write(s, s["k"], s["kc"], s["ks"])
        _write(s, s["v"], s["vc"], s["vs"])
        return dict(k=_read(s, s["kc"], s["ks"], s["k_back"]), v=_read(s, s["vc"], s["vs"], s["v_back"]))
    o, lse = _tree(s, slice(None), torch.float32)
    return dict(o=o.to(torch.bfloat16), lse=lse)


def _own(s):
    import io_aware_exact_15_gb300 as fa

    if s["op"] == "norm_rope":
        B, H, N, d = s["q"].shape
        size = (B, H, s["Hkv"], N, d, s["rot"], s["cos"].shape[0], s["inter"], 1e-6)
        if s["back"]:
            if s["ws"] is None:  # kept from call to call
                s["ws"] = torch.empty(fa.fa_qk_norm_rope_workspace_size(d), device=DEV, dtype=torch.uint8)
            status = fa.fa_qk_norm_rope_backward(
                s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], s["dq"], s["dk"],
                s["dwq"], s["dwk"], *size, s["q"].stride()[:3] + s["k"].stride()[:3],
                s["dq"].stride()[:3] + s["dk"].stride()[:3], s["ws"], s["ws"].numel())
            out = dict(dq=s["dq"], dk=s["dk"], dwq=s["dwq"], dwk=s["dwk"])
        else:
            status = fa.fa_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], s["qo"],
                                        s["ko"], *size, s["q"].stride()[:3] + s["k"].stride()[:3])
            out = dict(q=s["qo"], k=s["ko"])
    elif s["op"] == "cache":
        B, Hkv, N, d = s["k"].shape
        num, _, page, _ = s["kc"].shape
        form = {BF16: fa.FA_CACHE_BF16, E4M3: fa.FA_CACHE_E4M3, INT8: fa.FA_CACHE_INT8}[s["fmt"]]
        size = (form, B, Hkv, N, d, num, page, s["table"].shape[1])
        status = fa.fa_cache_append(s["k"], s["v"], s["table"], s["start"], s["counts"], s["kc"], s["vc"], s["ks"],
                                    s["vs"], *size, s["k"].stride()[:3] + s["v"].stride()[:3])
        status = status or fa.fa_cache_read(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["start"], s["counts"],
                                            s["k_back"], s["v_back"], *size)
        out = dict(k=s["k_back"], v=s["v_back"])
    else:
        B, H, T, d = s["q"].shape
        num, Hkv, page, _ = s["kc"].shape
        form = {BF16: fa.FA_CACHE_BF16, E4M3: fa.FA_CACHE_E4M3, INT8: fa.FA_CACHE_INT8}[s["fmt"]]
        if s["ws"] is None:  # kept as well
            s["ws"] = torch.empty(fa.fa_tree_attention_workspace_size(B, H, Hkv, T, d), device=DEV, dtype=torch.uint8)
        status = fa.fa_tree_attention(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["hist"], s["drafts"],
                                      s["mask"], s["o"], s["lse"], form, B, H, Hkv, T, d, num, page,
                                      s["table"].shape[1], s["scale"], s["ws"], s["ws"].numel())
        out = dict(o=s["o"], lse=s["lse"])
    if status != fa.FA_OK:
        raise fa.FaError(status, s["op"])
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def _expected_len(B, far):
    """Mean of _lengths: one sequence of `far`, the others uniform on [far / 4, far]."""
    return (far + (B - 1) * ((far + 3) // 4 + far) / 2) / B


def work(case):
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    if case["op"] == "norm_rope":
        heads = B * case["N"] * (case["H"] + Hkv)
        table = B * case["N"] * (4 * case["rot"] + 4)  # the rows of cos and sin that the positions name, positions
        per = 6 if case["back"] else 4
        return {"bytes": heads * d * per + table + 8 * d * (2 if case["back"] else 1),
                "flops": heads * d * (16 if case["back"] else 8)}
    elt = 2 if case["fmt"] == BF16 else 1
    scale = 0 if case["fmt"] == BF16 else 1
    if case["op"] == "cache":
        rows = 2 * Hkv * B * _expected_len(B, case["N"])  # key and value rows that exist
        # written: bf16 in, stored out; read back: stored in, bf16 out
        return {"bytes": rows * 2 * (2 * d + elt * d + scale) + B * 8, "flops": rows * d * 4}
    H, T = case["H"], case["T"]
    keys = B * (_expected_len(B, case["far"]) + _expected_len(B, T))
    rows = H * B * T
    words = -(-T // 32) if case["tree"] else 0
    return {"bytes": keys * Hkv * 2 * (elt * d + scale) + rows * (4 * d + 4) + keys / case["page"] * 4
            + B * (T * words * 4 + 8),
            "flops": 4 * d * H * _expected_len(B, T) * keys}


# ------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    real = torch.float64
    if case["op"] == "norm_rope":
        return _norm_rope_64(s)
    if case["op"] == "cache":
        return dict(k=_cache_64(s, s["k"]), v=_cache_64(s, s["v"]))
    o = torch.zeros(s["o"].shape, device=DEV, dtype=real)
    lse = torch.full(s["lse"].shape, -math.inf, device=DEV, dtype=real)
    mask = s["mask"].tolist() if s["mask"] is not None else None
    G = case["H"] // case["Hkv"]
    for b in range(case["B"]):
        hist, n, page = int(s["hist"][b]), int(s["drafts"][b]), case["page"]
        at = s["table"][b, :-(-(hist + n) // page)].long()
        k, v = (_values_64(c[at], e[at], case["fmt"]).transpose(0, 1).flatten(1, 2)[:, :hist + n]
                for c, e in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        if mask is None:
            sees = torch.ones(n, n, dtype=torch.bool).tril()
        else:
            sees = torch.tensor([[(mask[b][i][j // 32] >> (j % 32)) & 1 for j in range(n)] for i in range(n)]).bool()
        hide = torch.zeros(n, hist + n, device=DEV, dtype=real)
        hide[:, hist:] = torch.zeros(n, n, dtype=real).masked_fill(~sees, -math.inf).to(DEV)
        for h in range(case["H"]):
            x = s["q"][b, h, :n].to(real) @ k[h // G].T * s["scale"] + hide
            lse[b, h, :n] = torch.logsumexp(x, -1)
            o[b, h, :n] = torch.softmax(x, -1) @ v[h // G]
    return dict(o=o, lse=lse)


def _values_64(x, e, fmt):
    x = x.to(torch.float64)
    return x if fmt == BF16 else x * _pow2_64(e.long() - 127)[..., None]


def _pow2_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _cache_64(s, x):
    """What reads back: each element the nearest multiple of the type's step at its size (ties to even), from the definition."""
    x = x.to(torch.float64)
    y = x
    if s["fmt"] != BF16:
        most = 448.0 if s["fmt"] == E4M3 else 127.0
        share = x.abs().amax(-1, keepdim=True) / most
        e = torch.ceil(torch.log2(share)).clamp(-117, 119)
        e = torch.where(share <= _pow2_64(e - 1), e - 1, torch.where(share > _pow2_64(e), e + 1, e)).clamp(-117, 119)
        scale = _pow2_64(e)
        z = x / scale
        if s["fmt"] == E4M3:  # three bits after the leading one, down to steps of 2^-9
            step = _pow2_64((z.abs().clamp(min=2.0 ** -6).view(torch.int64) >> 52) - 1023 - 3)  # the leading bit's place
        else:
            step = torch.ones_like(z)
        y = torch.round(z / step) * step * scale
    n = torch.arange(x.shape[2], device=DEV)[None, None, :, None]
    return torch.where(n < s["counts"].long()[:, None, None, None], y, torch.zeros_like(y))


def _norm_rope_64(s):
    """Norm and rotation as products of complex numbers; the gradient from the norm's Jacobian, row by row."""
    out = {}
    real = torch.float64
    at = s["pos"].long()
    turn = torch.complex(s["cos"].to(real), s["sin"].to(real))[at][:, None]  # [B, 1, N, rot / 2]
    half = s["rot"] // 2

    def turned(y, z):
        pairs = y[..., :2 * half]
        pairs = pairs.unflatten(-1, (half, 2)) if s["inter"] else pairs.unflatten(-1, (2, half)).transpose(-1, -2)
        c = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        c = c.flatten(-2) if s["inter"] else c.transpose(-1, -2).flatten(-2)
        return torch.cat((c, y[..., 2 * half:]), -1)

    for name in ("q", "k"):
        x, w = s[name].to(real), s["w" + name].to(real)
        size = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / s["d"] + 1e-6)
        if not s["back"]:
            out[name] = turned(x / size * w, turn)
            continue
        g = turned(s["g" + name].to(real), turn.conj())
        out["dw" + name] = (g * x / size).sum((0, 1, 2))
        g = g * w
        out["d" + name] = g / size - x * (g * x).sum(-1, keepdim=True) / (s["d"] * size.pow(3))
    return out
