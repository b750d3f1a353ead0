"""Calls that follow each other directly on one stream may share memory: a
kernel that starts early must not write what the kernel before it reads."""
import pytest

from gpu_common import device, status_ok, torch
import serving_ref as R

import io_aware_exact_15_gb300 as fa

pytestmark = pytest.mark.gpu


class Backward:
    """An attention backward with few rows, so that its dQ accumulator begins
    a few kilobytes into its workspace."""

    def __init__(self, B, H, N, d, dev):
        g = torch.Generator().manual_seed(N)
        self.size = (B, H, N, d)
        self.q, self.k, self.v, self.do = (torch.randn(B, H, N, d, generator=g).bfloat16().to(dev)
                                           for _ in range(4))
        self.o, self.lse = fa.attention_forward(self.q, self.k, self.v)
        self.need = fa.fa_backward_workspace_size(B, H, N, d)
        self.grads = [torch.empty_like(self.q) for _ in range(3)]

    def run(self, ws):
        assert fa.fa_backward(self.q, self.k, self.v, self.o, self.do, self.lse, *self.grads,
                              *self.size, self.size[3] ** -0.5, False, ws, ws.numel()) == fa.FA_OK
        return self.grads


def close(a, b):
    """dQ is summed with fp32 atomics before its one rounding to bf16 (half a
    step on each side); the sums' order moves it far less."""
    a, b = a.double(), b.double()
    return ((a - b).abs() <= 2 * R.HALF_BF16 * b.abs() + 2.0 ** -12 * b.abs().max()).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_backward_then_attention_backward_on_one_workspace(d, inter):
    dev = device()
    att = Backward(4, 16, 128, d, dev)
    B, H, Hkv, N = 2, 6, 2, 1500
    g = torch.Generator().manual_seed(1)
    q, k, gq, gk = (torch.randn(B, h, N, d, generator=g).bfloat16().to(dev)
                    for h in (H, Hkv, H, Hkv))
    wq, wk = (torch.randn(d, generator=g).to(dev) for _ in range(2))
    cos, sin = (t.to(dev) for t in R.tables(N, d))
    ws = torch.empty(max(att.need, fa.fa_qk_norm_rope_workspace_size(d)), dtype=torch.uint8,
                     device=dev)
    want = [t.clone() for t in att.run(ws)]
    args = (gq, gk, q, k, wq, wk, cos, sin, None, 1e-6, inter)
    torch.cuda.synchronize()
    alone = fa.qk_norm_rope_backward(*args)
    torch.cuda.synchronize()
    for _ in range(60):
        out = fa.qk_norm_rope_backward(*args, workspace=ws)
        att.run(ws)
        assert all(torch.equal(a, b) for a, b in zip(out, alone))
        assert all(close(a, b) for a, b in zip(att.grads, want))
    status_ok()


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3])
@pytest.mark.parametrize("T", [2, 40, 130])
def test_tree_attention_then_attention_backward_on_one_workspace(T, fmt):
    dev = device()
    att = Backward(1, 64, 128, 128, dev)
    B, H, Hkv, d, page, hist = 3, 4, 2, 128, 64, 9000
    g = torch.Generator().manual_seed(T)
    pages = -(-(hist + T) // page)
    table = torch.randperm(B * pages, generator=g).int().view(B, pages).to(dev)
    kc, vc = (torch.empty(B * pages, Hkv, page, d, dtype=R.DTYPES[fmt], device=dev)
              for _ in range(2))
    ks, vs = (torch.empty(B * pages, Hkv, page, dtype=torch.uint8, device=dev) for _ in range(2))
    k, v = (torch.randn(B, Hkv, hist + T, d, generator=g).bfloat16().to(dev) for _ in range(2))
    zero = torch.zeros(B, dtype=torch.int32, device=dev)
    fa.cache_append(k, v, kc, vc, table, zero, None, ks, vs)
    q = torch.randn(B, H, T, d, generator=g).bfloat16().to(dev)
    ws = torch.empty(max(att.need, fa.fa_tree_attention_workspace_size(B, H, Hkv, T, d)),
                     dtype=torch.uint8, device=dev)
    want = [t.clone() for t in att.run(ws)]
    args = dict(q=q, k_cache=kc, v_cache=vc, page_table=table, hist_lens=zero + hist, k_scale=ks,
                v_scale=vs)
    torch.cuda.synchronize()
    alone = fa.tree_attention(**args)
    torch.cuda.synchronize()
    for _ in range(60):
        out = fa.tree_attention(**args, workspace=ws)
        att.run(ws)
        assert all(torch.equal(a, b) for a, b in zip(out, alone))
        assert all(close(a, b) for a, b in zip(att.grads, want))
    status_ok()


def test_freed_inputs_handed_to_the_next_call():
    """Tensors freed right after the call that reads them: the next call's
    workspace takes their place, and the first call's result stays right."""
    dev = device()
    B, H, N, d = 2, 16, 512, 128
    g = torch.Generator().manual_seed(2)
    host = [torch.randn(B, H, N, d, generator=g).bfloat16() for _ in range(4)]
    q, k, v, do = (t.to(dev) for t in host)
    w = torch.ones(d, device=dev)
    cos, sin = (t.to(dev) for t in R.tables(N, d))
    want = fa.qk_norm_rope(q, k, w, w, cos, sin)
    want_o, want_l = fa.attention_forward(q, k, v)
    torch.cuda.synchronize()
    for _ in range(40):
        q2, k2 = q.clone(), k.clone()
        out = fa.qk_norm_rope(q2, k2, w, w, cos, sin)
        del q2, k2
        fa.attention_backward(q, k, v, want_o, do, want_l)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        o, lse = fa.attention_forward(q2, k2, v2)
        del q2, k2, v2
        fa.attention_backward(q, k, v, want_o, do, want_l)
        assert torch.equal(o, want_o) and torch.equal(lse, want_l)
    status_ok()


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.INT8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", [(3, 100), (1, 257), (5, 120)])
def test_last_groups_of_at_most_128_rows(G, T, d, fmt):
    """300, 257 and 600 rows: the last group of a head occupies one of the two
    softmax warpgroups, the other goes on to the next head's.  Many problems
    of a tile or two, the same bits every time, no wait runs out."""
    dev = device()
    B, Hkv, page = 24, 3, 32
    g = torch.Generator().manual_seed(G + T + d)
    hist = torch.randint(0, 260, (B,), generator=g).int()
    hist[::5] = 0
    pages = -(-(260 + T) // page)
    table = torch.randperm(B * pages, generator=g).int().view(B, pages).to(dev)
    kc, vc = (torch.empty(B * pages, Hkv, page, d, dtype=R.DTYPES[fmt], device=dev)
              for _ in range(2))
    ks, vs = (torch.empty(B * pages, Hkv, page, dtype=torch.uint8, device=dev) for _ in range(2))
    k, v = (torch.randn(B, Hkv, 260 + T, d, generator=g).bfloat16() for _ in range(2))
    zero = torch.zeros(B, dtype=torch.int32, device=dev)
    fa.cache_append(k.to(dev), v.to(dev), kc, vc, table, zero, None, ks, vs)
    q = torch.randn(B, Hkv * G, T, d, generator=g).bfloat16()
    run = lambda: fa.tree_attention(q.to(dev), kc, vc, table, hist.to(dev), k_scale=ks, v_scale=vs)
    o, lse = run()
    status_ok()
    for b in (0, 1, B - 1):  # the values, where every draft sees those before it
        h = int(hist[b])
        kk, vv = (R.quantise(R.f64(x[b, :, :h + T]), fmt) for x in (k, v))
        ref, ref_l, size, score = R.attention(R.f64(q[b]), kk, vv, R.sees(h, T, T, None), d ** -0.5)
        # one rounding of each weight and of the result to bf16, scores in fp32
        off = 2.0 ** -20 * (1 + score)
        tol = (R.HALF_BF16 + 2 * off[..., None]) * size + R.HALF_BF16 * abs(ref) + 1e-30
        assert (abs(R.f64(o[b]) - ref) <= tol).all()
        assert (abs(R.f64(lse[b]) - ref_l) <= off + 2.0 ** -20 * abs(ref_l)).all()
    for _ in range(30):
        again = run()
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    status_ok()
