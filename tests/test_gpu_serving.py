"""The operators together, as a model uses them: a verification step of
drafted tokens (projection -> norm and rotation -> cache -> tree attention ->
accepted tokens moved -> next token), and a training step through the
attention kernels with the gradient back to the projection."""
import numpy as np
import pytest

from gpu_common import device, status_ok, torch
import serving_ref as R

import io_aware_exact_15_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.INT8])
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (3, 3, 64)])
def test_verification_step(H, Hkv, d, fmt):
    dev = device()
    B, T, page, eps = 2, 11, 32, 1e-5
    hist = [150, 37]
    rng = np.random.default_rng(d + fmt)
    g = torch.Generator().manual_seed(d + fmt)
    bits = R.random_trees(rng, B, T)
    depth = bits.sum(-1) - 1
    qkv = lambda n: torch.randn(B, n, H + 2 * Hkv, d, generator=g).bfloat16().to(dev)
    split = lambda x: (x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2),
                       x[:, :, H + Hkv:].transpose(1, 2))
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g)).to(dev), torch.ones(d, device=dev)
    cos, sin = (t.to(dev) for t in R.tables(512, d))
    table, num = R.page_table(rng, [h + T + 1 for h in hist], page)
    table = table.to(dev)
    kc, vc = (torch.zeros(num, Hkv, page, d, device=dev).to(R.DTYPES[fmt]) for _ in range(2))
    ks, vs = (torch.zeros(num, Hkv, page, dtype=torch.uint8, device=dev) for _ in range(2))
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)
    cache = dict(k_scale=ks, v_scale=vs)

    # 64-bit: the same step from the projections
    def ref_rows(x, w, pos):
        at = np.asarray(pos)
        c, s = R.f64(cos)[at][:, None], R.f64(sin)[at][:, None]
        return R.norm_rope(R.f64(x), R.f64(w), c, s, d, False, eps)

    stored = lambda x: R.quantise(torch.from_numpy(x).bfloat16().double().numpy(), fmt)

    past = qkv(max(hist))
    q0, k0, v0 = split(past)
    pos0 = np.broadcast_to(np.arange(max(hist)), (B, max(hist)))
    _, k0r = fa.qk_norm_rope(q0, k0, wq, wk, cos, sin, i32(pos0), eps)
    fa.cache_append(k0r, v0, kc, vc, table, i32([0, 0]), i32(hist), **cache)
    new = qkv(T)
    q1, k1, v1 = split(new)
    pos1 = np.array(hist)[:, None] + depth
    q1r, k1r = fa.qk_norm_rope(q1, k1, wq, wk, cos, sin, i32(pos1), eps)
    fa.cache_append(k1r, v1, kc, vc, table, i32(hist), None, **cache)
    o, lse = fa.tree_attention(q1r, kc, vc, table, i32(hist), None, R.words_of(bits).to(dev),
                               **cache)
    status_ok()
    qr = R.f64(q1r)
    kh, kd = ref_rows(k0, wk, pos0), ref_rows(k1, wk, pos1)
    # queries and keys: one bf16 rounding each
    for got, want in ((q1r, ref_rows(q1, wq, pos1)), (k1r, kd)):
        assert (np.abs(R.f64(got) - want) <= R.HALF_BF16 * np.abs(want) + 1e-4).all()
    back_k, back_v = fa.cache_read(kc, vc, table, i32([0, 0]), max(hist) + T, i32(hist) + T, **cache)
    for b in range(B):
        # the cache holds the definition's value of what the norm wrote
        want = R.quantise(np.concatenate([R.f64(k0r)[b, :, :hist[b]], R.f64(k1r)[b]], 1), fmt)
        assert np.array_equal(R.f64(back_k)[b, :, :hist[b] + T], want)
        kk, vv = R.f64(back_k)[b, :, :hist[b] + T], R.f64(back_v)[b, :, :hist[b] + T]
        ref, ref_l, size, score = R.attention(qr[b], kk, vv, R.sees(hist[b], T, T, bits[b]),
                                              d ** -0.5)
        off = 2.0 ** -20 * (1 + score)
        tol = (R.HALF_BF16 + 2 * off[..., None]) * size + R.HALF_BF16 * np.abs(ref)
        assert (np.abs(R.f64(o)[b] - ref) <= tol).all()
        assert (np.abs(R.f64(lse)[b] - ref_l) <= off + 2.0 ** -20 * np.abs(ref_l)).all()

    # the deepest branch is accepted: its tokens move up behind the history
    path = [np.nonzero(bits[b, int(depth[b].argmax())])[0] for b in range(B)]
    n = [len(p) for p in path]
    moved_k, moved_v = (torch.zeros(B, Hkv, max(n), d, dtype=torch.bfloat16, device=dev)
                        for _ in range(2))
    dk, dv = fa.cache_read(kc, vc, table, i32(hist), T, None, **cache)
    for b in range(B):
        at = torch.from_numpy(path[b]).to(dev)
        moved_k[b, :, :n[b]], moved_v[b, :, :n[b]] = dk[b][:, at], dv[b][:, at]
    fa.cache_append(moved_k, moved_v, kc, vc, table, i32(hist), i32(n), **cache)
    hist2 = [h + m for h, m in zip(hist, n)]
    q2, k2, v2 = split(qkv(1))
    q2r, k2r = fa.qk_norm_rope(q2, k2, wq, wk, cos, sin, i32(np.array(hist2)[:, None]), eps)
    fa.cache_append(k2r, v2, kc, vc, table, i32(hist2), None, **cache)
    o, lse = fa.tree_attention(q2r, kc, vc, table, i32(hist2), **cache)
    status_ok()
    for b in range(B):
        kk = np.concatenate([R.f64(back_k)[b, :, :hist[b]], R.f64(back_k)[b][:, hist[b] + path[b]],
                             stored(R.f64(k2r)[b])], 1)
        vv = np.concatenate([R.f64(back_v)[b, :, :hist[b]], R.f64(back_v)[b][:, hist[b] + path[b]],
                             stored(R.f64(v2)[b])], 1)
        ref, ref_l, size, score = R.attention(R.f64(q2r)[b], kk, vv, R.sees(hist2[b], 1, 1, None),
                                              d ** -0.5)
        off = 2.0 ** -20 * (1 + score)
        tol = (R.HALF_BF16 + 2 * off[..., None]) * size + R.HALF_BF16 * np.abs(ref)
        assert (np.abs(R.f64(o)[b] - ref) <= tol).all()


def test_prompt_then_decode_agrees_with_the_prompt_kernel():
    """Causal attention over a prompt by fa_forward, and the same rows as a
    chain of drafts over the cache: both round P and O to bf16 once, so they
    differ by at most twice those roundings."""
    dev = device()
    B, H, Hkv, N, d, page = 1, 4, 2, 200, 64, 16
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(B, h, N, d, generator=g).bfloat16().to(dev) for h in (H, Hkv, Hkv))
    want, want_l = fa.attention_forward(q, k, v, causal=True)
    T = 60
    table = torch.arange(13, dtype=torch.int32, device=dev).flip(0)[None].contiguous()
    kc, vc = (torch.empty(13, Hkv, page, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    fa.cache_append(k, v, kc, vc, table, zero)
    o, lse = fa.tree_attention(q[:, :, N - T:].contiguous(), kc, vc, table, zero + N - T)
    status_ok()
    most = v.float().abs().max().item()
    assert (o.float() - want[:, :, N - T:].float()).abs().max() <= 4 * R.HALF_BF16 * most
    assert (lse - want_l[:, :, N - T:]).abs().max() <= 2e-2  # fa_forward's bound on lse, twice


def test_training_step():
    """d loss / d projection through norm + rotation and the attention
    kernels, against 64-bit autograd of the same step."""
    dev = device()
    B, H, Hkv, N, d, eps = 1, 4, 2, 150, 64, 1e-6
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(B, N, H + 2 * Hkv, d, generator=g).bfloat16()
    do = torch.randn(B, H, N, d, generator=g).bfloat16()
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g) for _ in range(2))
    cos, sin = R.tables(N, d)
    x = qkv.to(dev)
    q, k, v = (x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2),
               x[:, :, H + Hkv:].transpose(1, 2).contiguous())
    c, s = cos.to(dev), sin.to(dev)
    qr, kr = fa.qk_norm_rope(q, k, wq.to(dev), wk.to(dev), c, s, eps=eps)
    o, lse = fa.attention_forward(qr, kr, v, causal=True)
    dqr, dkr, dv = fa.attention_backward(qr, kr, v, o, do.to(dev), lse, causal=True)
    dx = torch.zeros_like(x)
    _, _, dwq, dwk = fa.qk_norm_rope_backward(
        dqr, dkr, q, k, wq.to(dev), wk.to(dev), c, s, eps=eps, dq=dx[:, :, :H].transpose(1, 2),
        dk=dx[:, :, H:H + Hkv].transpose(1, 2))
    dx[:, :, H + Hkv:] = dv.transpose(1, 2)
    status_ok()

    y = qkv.double().requires_grad_()
    a, b = wq.double().requires_grad_(), wk.double().requires_grad_()

    def rope(t, w):
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + eps) * w
        t1, t2 = t[..., :d // 2], t[..., d // 2:]
        return torch.cat((t1 * cos.double() - t2 * sin.double(),
                          t2 * cos.double() + t1 * sin.double()), -1)

    qq, kk = rope(y[:, :, :H].transpose(1, 2), a), rope(y[:, :, H:H + Hkv].transpose(1, 2), b)
    vv = y[:, :, H + Hkv:].transpose(1, 2)
    kk, vv = kk.repeat_interleave(H // Hkv, 1), vv.repeat_interleave(H // Hkv, 1)
    sc = (qq @ kk.transpose(2, 3)) / d ** 0.5
    sc = sc.masked_fill(~torch.ones(N, N).tril().bool(), -float("inf"))
    out = sc.softmax(-1) @ vv
    (out * do.double()).sum().backward()
    # the attention gradients' bound (parity.py: 5e-2 of the largest)
    for got, want in ((dx, y.grad), (dwq, a.grad), (dwk, b.grad)):
        assert (got.cpu().double() - want).abs().max() <= 5e-2 * want.abs().max()
