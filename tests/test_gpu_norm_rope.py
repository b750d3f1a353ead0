"""Per-head norm of Q and K with the rotation, forward and backward, against
the 64-bit formulas; strided views, both pairings, partial rotation,
positions in any order and out of range, one token to odd lengths."""
import numpy as np
import pytest

from gpu_common import device, status_ok, torch
import serving_ref as R

import fa_workloads as W
import io_aware_exact_15_gb300 as fa

pytestmark = pytest.mark.gpu

EPS = 1e-6


def packed(B, H, Hkv, N, d, seed, dev):
    """q, k as views of one projection [B, N, H + 2 Hkv, d]."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, N, H + 2 * Hkv, d, generator=g)
    x = (x * torch.exp(torch.randn(1, 1, H + 2 * Hkv, d, generator=g))).bfloat16().to(dev)
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g) for _ in range(2))
    return x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2), wq.to(dev), wk.to(dev)


def angles(cos, sin, positions, B, N):
    at = np.broadcast_to(np.arange(N), (B, N)) if positions is None else positions.cpu().numpy()
    at = np.clip(at, 0, cos.shape[0] - 1)
    return R.f64(cos)[at][:, None], R.f64(sin)[at][:, None]


CASES = [  # B, H, Hkv, N, d, rot, interleaved, positions, table rows
    (1, 1, 1, 1, 64, 64, False, None, 1),
    (2, 4, 4, 1, 128, 128, True, "mixed", 300),
    (3, 6, 2, 37, 64, 16, False, "mixed", 5000),
    (2, 5, 3, 129, 128, 64, True, None, 129),
    (1, 9, 1, 65, 128, 128, False, "outside", 50),
    (2, 3, 7, 33, 64, 48, True, "mixed", 100),
    (2, 16, 4, 1030, 128, 128, False, "mixed", 131072),
    (1, 12, 12, 1500, 64, 32, True, None, 1500),
    # more tokens than warps: a warp's next token is in another sequence
    (5, 2, 1, 1031, 64, 64, False, None, 1031),
    (2501, 1, 3, 3, 128, 96, True, "mixed", 77),
]


def make(case, dev, seed):
    B, H, Hkv, N, d, rot, inter, pos, rows = case
    q, k, wq, wk = packed(B, H, Hkv, N, d, seed, dev)
    cos, sin = (t.to(dev) for t in R.tables(rows, rot))
    if pos is not None:
        lo, hi = (-20, rows + 20) if pos == "outside" else (0, rows - 1)
        g = torch.Generator().manual_seed(seed + 1)
        pos = torch.randint(lo, hi + 1, (B, N), generator=g, dtype=torch.int32).to(dev)
    return q, k, wq, wk, cos, sin, pos


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward(case):
    dev = device()
    B, H, Hkv, N, d, rot, inter, _, _ = case
    q, k, wq, wk, cos, sin, pos = make(case, dev, sum(case[:6]))
    out = fa.qk_norm_rope(q, k, wq, wk, cos, sin, pos, EPS, inter)
    status_ok()
    c, s = angles(cos, sin, pos, B, N)
    for got, x, w in zip(out, (q, k), (wq, wk)):
        want = R.norm_rope(R.f64(x), R.f64(w), c, s, rot, inter, EPS)
        plain = np.abs(R.norm_rope(R.f64(x), R.f64(w), 1 + 0 * c, 0 * s, rot, inter, EPS))
        # one rounding to bf16; fp32 sums of 128 squares (relative to the
        # row's size) and products before it: far below 2^-18 of the row
        tol = R.HALF_BF16 * np.abs(want) + 2.0 ** -18 * plain.max(-1, keepdims=True)
        assert (np.abs(R.f64(got) - want) <= tol).all()
        assert got.is_contiguous()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("into_packed", [False, True])
def test_backward(case, into_packed):
    dev = device()
    B, H, Hkv, N, d, rot, inter, _, _ = case
    q, k, wq, wk, cos, sin, pos = make(case, dev, 7 + sum(case[:6]))
    g = torch.Generator().manual_seed(3)
    gq = W.randn_bf16((B, H, N, d), g).to(dev)
    gk = W.randn_bf16((B, Hkv, N, d), g).to(dev)
    dq = dk = None
    if into_packed:
        whole = torch.full((B, N, H + 2 * Hkv, d), 5.0, dtype=torch.bfloat16, device=dev)
        dq, dk = whole[:, :, :H].transpose(1, 2), whole[:, :, H:H + Hkv].transpose(1, 2)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, pos, EPS, inter,
                                                dq, dk)
    status_ok()
    if into_packed:
        assert (whole[:, :, H + Hkv:] == 5.0).all()  # the values' place is not touched
    c, s = angles(cos, sin, pos, B, N)
    for dx, dw, gg, x, w in ((dq, dwq, gq, q, wq), (dk, dwk, gk, k, wk)):
        want, want_w, size, size_w = R.norm_rope_backward(R.f64(gg), R.f64(x), R.f64(w), c, s, rot,
                                                          inter, EPS)
        # fp32 steps are relative to the size of the terms, the largest of a
        # pair where the rotation mixes two
        row = size.max(-1, keepdims=True)
        assert (np.abs(R.f64(dx) - want) <= R.HALF_BF16 * np.abs(want) + 2.0 ** -18 * row).all()
        # a lane adds at most rows / 8 of the terms one after another here,
        # then trees: at most 2^8 roundings of 2^-24, plus those of the terms
        assert (np.abs(R.f64(dw) - want_w) <= 2.0 ** -15 * size_w + 1e-30).all()


def test_backward_is_reproducible():
    dev = device()
    case = (2, 16, 4, 1030, 128, 128, False, "mixed", 4096)
    q, k, wq, wk, cos, sin, pos = make(case, dev, 5)
    gq, gk = torch.randn_like(q).contiguous(), torch.randn_like(k).contiguous()
    a = fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, pos)
    b = fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, pos)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_broadcast_heads_and_nothing_past_the_end():
    """Stride 0 (one head read by all) and outputs between guard bands."""
    dev = device()
    B, H, N, d = 2, 5, 19, 64
    g = torch.Generator().manual_seed(0)
    one = W.randn_bf16((B, 1, N, d), g).to(dev)
    q = one.expand(B, H, N, d)
    wq = torch.ones(d, device=dev)
    cos, sin = (t.to(dev) for t in R.tables(N, d))
    n = B * H * N * d
    band = torch.full((n + 2048,), 3.0, dtype=torch.bfloat16, device=dev)
    q_out = band[1024:1024 + n].view(B, H, N, d)
    k_out = torch.empty_like(one)
    assert fa.fa_qk_norm_rope(q, one, wq, wq, cos, sin, None, q_out, k_out, B, H, 1, N, d, d, N,
                              False, EPS, q.stride()[:3] + one.stride()[:3]) == fa.FA_OK
    status_ok()
    assert (band[:1024] == 3.0).all() and (band[1024 + n:] == 3.0).all()
    assert torch.equal(q_out, k_out.expand(B, H, N, d))


def test_values_past_the_rotation_keep_infinities_apart():
    """An infinite row gives NaN in itself only; rows of zeros give zeros."""
    dev = device()
    x = torch.ones(1, 2, 4, 64, dtype=torch.bfloat16, device=dev)
    x[0, 0, 1, 5] = float("inf")
    x[0, 1, 2] = 0
    w = torch.ones(64, device=dev)
    cos, sin = (t.to(dev) for t in R.tables(4, 16))
    y, _ = fa.qk_norm_rope(x, x, w, w, cos, sin)
    status_ok()
    bad = torch.isnan(y)
    assert bad[0, 0, 1].any() and bad.sum() == bad[0, 0, 1].sum()
    assert (y[0, 1, 2] == 0).all()


def test_two_streams_and_graph():
    """The same call on a side stream and replayed from a graph."""
    dev = device()
    case = (2, 6, 2, 37, 64, 64, False, "mixed", 500)
    q, k, wq, wk, cos, sin, pos = make(case, dev, 9)
    want = fa.qk_norm_rope(q, k, wq, wk, cos, sin, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.qk_norm_rope(q, k, wq, wk, cos, sin, pos, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    gq, gk = torch.randn_like(want[0]), torch.randn_like(want[1])
    want = fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, pos)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def places(n):
    """Where a test puts its infinities: in the rotated part, on both sides
    of its end, in the same pair of elements, in the last ones."""
    return [n - 1, n, n + 1, n + 2, n + 9]


@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (128, 32), (128, 64), (128, 112)])
@pytest.mark.parametrize("inter", [False, True])
def test_infinities_beside_elements_that_are_not_rotated(d, rot, inter):
    """Elements from `rot` on are only normed: an infinite neighbour leaves
    them as the formula has them (forward: zeros beside a NaN; gradients and
    the sums of their columns: finite)."""
    dev = device()
    B, H, N = 1, len(places(rot)), 5
    g = torch.Generator().manual_seed(rot)
    x = torch.randn(B, H, N, d, generator=g).bfloat16()
    gq = torch.randn(B, H, N, d, generator=g).bfloat16()
    w = (1 + 0.3 * torch.randn(d, generator=g))
    cos, sin = R.tables(N, rot)
    bad, gbad = x.clone(), gq.clone()
    for h, at in enumerate(places(rot)):
        bad[0, h, 2, at] = float("inf") * (-1) ** h
        gbad[0, h, 3, at] = float("inf") * (-1) ** h
    c, s = angles(cos, sin, None, B, N)
    y, _ = fa.qk_norm_rope(bad.to(dev), x.to(dev), w.to(dev), w.to(dev), cos.to(dev), sin.to(dev),
                           eps=EPS, interleaved=inter)
    status_ok()
    with np.errstate(invalid="ignore"):
        want = R.norm_rope(R.f64(bad), R.f64(w), c, s, rot, inter, EPS)
    got = R.f64(y)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    # as test_forward; a pair's turn keeps its length
    tol = R.HALF_BF16 * np.abs(want) + 2.0 ** -18 * 2 * np.nanmax(np.abs(want), -1, keepdims=True)
    assert (np.abs(got - want) <= tol)[fine].all()
    dq, _, dwq, _ = fa.qk_norm_rope_backward(gbad.to(dev), gq.to(dev), x.to(dev), x.to(dev),
                                             w.to(dev), w.to(dev), cos.to(dev), sin.to(dev),
                                             eps=EPS, interleaved=inter)
    status_ok()
    with np.errstate(invalid="ignore"):
        want, want_w, _, size_w = R.norm_rope_backward(R.f64(gbad), R.f64(x), R.f64(w), c, s, rot,
                                                       inter, EPS)
    # a row with an infinite gradient has a NaN or infinite mean and is no
    # number anywhere; the columns of dw that no infinity reaches are
    got_w = R.f64(dwq)
    assert np.array_equal(np.isnan(got_w), np.isnan(want_w))
    fine = np.isfinite(want_w)
    assert fine.sum() >= d - 2 * H
    assert np.array_equal(got_w[np.isinf(want_w)], want_w[np.isinf(want_w)])
    assert (np.abs(got_w[fine] - want_w[fine]) <= 2.0 ** -15 * size_w[fine] + 1e-30).all()
    rows = [n for n in range(N) if n != 3]
    assert np.isfinite(R.f64(dq)[:, :, rows]).all() and not np.isfinite(R.f64(dq)[:, :, 3]).any()


def test_infinite_weights_stay_in_their_columns():
    """An infinite or NaN weight of an element that is not rotated reaches
    that column alone."""
    dev = device()
    for inter in (False, True):
        x = torch.ones(1, 1, 3, 64, dtype=torch.bfloat16, device=dev)
        w = torch.ones(64, device=dev)
        w[40], w[51] = float("inf"), float("nan")
        cos, sin = (t.to(dev) for t in R.tables(3, 32))
        y, _ = fa.qk_norm_rope(x, x, w, w, cos, sin, interleaved=inter)
        status_ok()
        assert torch.isposinf(y[..., 40]).all() and torch.isnan(y[..., 51]).all()
        assert torch.isfinite(y).sum() == 3 * 62
