"""Sliding windows with first tokens that stay visible: both passes against a
plain 64-bit evaluation over lengths, windows, head groups and packed batches;
numbers that belong to other rows; streams, graphs and repeats."""
import pytest

from gpu_common import device, status_ok, torch
import window_ref as R

import io_aware_exact_15_gb300 as fa

pytestmark = pytest.mark.gpu


def run(x, window, sinks, dev, scale=None, o=None, lse=None):
    """(o, lse, dq, dk, dv) of a Batch, the backward with the given o, lse."""
    q, k, v, g = (t.to(dev) for t in (x.q, x.k, x.v, x.g))
    kw = dict(scale=scale, causal=True, window=window, sinks=sinks)
    if x.packed:
        kw.update(cu_seqlens=x.cu.to(dev), max_seqlen=max(max(x.lens), 1))
    fo, fl = fa.attention_forward(q, k, v, **kw)
    o = fo if o is None else o
    lse = fl if lse is None else lse
    grads = fa.attention_backward(q, k, v, o, g, lse, **kw)
    status_ok()
    return (fo, fl) + grads


def check(x, out, window, sinks, scale=None):
    scale = 1.0 / x.d ** 0.5 if scale is None else scale
    o, lse, *grads = out
    for b, n in enumerate(x.lens):
        if n == 0:
            continue
        q, k, v, g = (x.seq(t, b) for t in (x.q, x.k, x.v, x.g))
        ro, rl, to, tl = R.forward(q, k, v, window, sinks, scale)
        close("o", b, x.seq(o, b), ro, to)
        close("lse", b, (x.seq(lse[..., None], b))[..., 0], rl, tl)
        ref, tol = R.backward(q, k, v, x.seq(o, b), x.seq(lse[..., None], b)[..., 0], g, window,
                              sinks, scale)
        for name, got, r, t in zip(("dq", "dk", "dv"), grads, ref, tol):
            close(name, b, x.seq(got, b), r, t)


def close(name, b, got, ref, tol):
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fine), (name, b, "finite where the formula is not, or not")
    err = torch.where(fine, (got - ref).abs(), torch.zeros((), dtype=torch.float64))
    tol = torch.nan_to_num(tol)
    assert bool((err <= tol)[fine].all()), \
        (name, b, float((err / tol)[fine].max()), torch.nonzero(fine & ~(err <= tol))[:3].tolist())


DENSE = [
    # B, H, Hkv, N, d, window, sinks
    (1, 1, 1, 1, 64, 1, 0),
    (2, 2, 1, 5, 128, 2, 1),
    (1, 2, 2, 128, 64, 128, 0),
    (1, 2, 2, 129, 128, 128, 0),
    (2, 3, 1, 130, 64, 1, 0),
    (1, 4, 2, 300, 128, 50, 4),
    (1, 2, 2, 300, 64, 300, 7),      # the window is the sequence
    (1, 2, 1, 300, 128, 100000, 0),  # and more than it
    (1, 2, 2, 515, 64, 129, 130),    # first tokens in two tiles
    (1, 2, 1, 640, 128, 127, 128),
    (1, 1, 1, 700, 64, 3, 1000),     # every token is a first one
    (2, 5, 5, 777, 64, 256, 16),
    (1, 6, 2, 1281, 128, 200, 4),    # the first tile's walk in parts
    (1, 4, 4, 2050, 64, 65, 1),
    (1, 8, 1, 1537, 64, 384, 300),
]


@pytest.mark.parametrize("case", DENSE)
def test_equal_lengths(case):
    B, H, Hkv, N, d, window, sinks = case
    x = R.Batch([N] * B, H, Hkv, d, False, 11 + N)
    check(x, run(x, window, sinks, device()), window, sinks)


PACKED = [
    # lengths, H, Hkv, d, window, sinks, rows before and behind
    ([1], 1, 1, 64, 1, 0, 0, 0),
    ([3, 1, 0, 200], 2, 1, 128, 64, 4, 0, 0),
    ([129, 0, 127, 128, 1], 4, 2, 64, 100, 2, 0, 57),
    ([0, 640, 31], 2, 2, 64, 200, 130, 5, 300),
    ([1300, 77, 1100], 4, 1, 128, 150, 4, 0, 1),  # parts in some sequences, none in others
    ([0, 0, 9], 3, 3, 128, 1, 0, 130, 2),
]


@pytest.mark.parametrize("case", PACKED)
def test_packed(case):
    lens, H, Hkv, d, window, sinks, lead, tail = case
    x = R.Batch(lens, H, Hkv, d, True, 7 + sum(lens), lead, tail)
    check(x, run(x, window, sinks, device()), window, sinks)


def test_two_tile_form():
    """More than four waves of two-tile CTAs: the other instantiation."""
    dev = device()
    for d in (64, 128):
        x = R.Batch([300] * 160, 10, 5, d, False, 5)
        out = run(x, 140, 4, dev)
        for b in (0, 77, 159):
            y = R.Batch([300], 10, 5, d, False, 5)
            y.q, y.k, y.v, y.g = (t[b:b + 1] for t in (x.q, x.k, x.v, x.g))
            check(y, [t[b:b + 1] for t in out], 140, 4)


@pytest.mark.parametrize("count,longest,lead,window", [(33, 300, 0, 40), (1100, 3, 7, 2),
                                                       (160, 700, 130, 100000)])
def test_many_packed_sequences(count, longest, lead, window):
    """More sequences than a warp looks at together, empty ones among them; the
    last case in both of the forward's forms."""
    gen = torch.Generator().manual_seed(count)
    lens = torch.randint(0, longest + 1, (count,), generator=gen).tolist()
    for H, Hkv, d in ((1, 1, 64), (6, 2, 128)) if count == 160 else ((2, 1, 64),):
        x = R.Batch(lens, H, Hkv, d, True, 3, lead, 5)
        out = run(x, window, 2, device())
        some = range(count) if count != 160 else (0, 1, 31, 32, 33, 100, 158, 159)
        y = R.Batch(lens, H, Hkv, d, True, 3, lead, 5)
        y.lens = [n if b in some else 0 for b, n in enumerate(lens)]
        check(y, out, window, 2)


@pytest.mark.parametrize("d,sinks,lead", [(64, 3, 0), (128, 200, 77)])
def test_long_sequences_among_short_ones(d, sinks, lead):
    """First tiles' walks in parts, at offsets all over the batch: a sequence
    with parts beside ones without, and two on end."""
    lens = [5, 0, 1400, 130] + [3] * 90 + [1025, 1300, 0, 1, 2100] + [7, 0, 60] * 9 + [1024, 1100]
    x = R.Batch(lens, 2, 1, d, True, 21, lead, 300)
    check(x, run(x, 60, sinks, device()), 60, sinks)


def test_numbers_beyond_the_batch():
    """A longest length and a window that are more than there is, past 32 bits
    too; a longest length below zero."""
    dev = device()
    x = R.Batch([70, 0, 200], 2, 1, 64, True, 31, 0, 9)
    q, k, v, g, cu = (t.to(dev) for t in (x.q, x.k, x.v, x.g, x.cu))
    kw = dict(causal=True, sinks=2, cu_seqlens=cu)
    for N, window in ((4096, 30), (2**40, 2**32 + 1)):
        o, lse = fa.attention_forward(q, k, v, max_seqlen=N, window=window, **kw)
        grads = fa.attention_backward(q, k, v, o, g, lse, max_seqlen=N, window=window, **kw)
        status_ok()
        check(x, (o, lse) + grads, min(window, 1000), 2)
    with pytest.raises(ValueError):
        fa.attention_forward(q, k, v, max_seqlen=-1, window=30, **kw)


def test_rows_of_no_sequence_are_left():
    """Rows in front of the first sequence and behind the last."""
    dev = device()
    x = R.Batch([130, 0, 60], 2, 1, 64, True, 3, 40, 200)
    q, k, v, g = (t.to(dev) for t in (x.q, x.k, x.v, x.g))
    cu, T = x.cu.to(dev), x.total
    mark = lambda *s, dtype=torch.bfloat16: torch.full(s, 123.0, dtype=dtype, device=dev)
    o, lse = mark(2, T, 64), mark(2, T, dtype=torch.float32)
    dq, dk, dv = mark(2, T, 64), mark(1, T, 64), mark(1, T, 64)
    size = (3, 2, 1, 130, T, 64)
    assert fa.fa_forward_window(q, k, v, o, lse, cu, *size, 0.125, 33, 2) == fa.FA_OK
    n = fa.fa_backward_window_workspace_size(*size, 33, 2)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=dev)  # NaN in every type
    assert fa.fa_backward_window(q, k, v, o, g, lse, dq, dk, dv, cu, *size, 0.125, 33, 2, ws,
                                 n) == fa.FA_OK
    status_ok()
    out = ~x.own.to(dev)
    for t in (o, lse, dq, dk, dv):
        assert bool((t[:, out] == 123.0).all())
        assert bool(torch.isfinite(t).all())
    check(x, (o, lse, dq, dk, dv), 33, 2, 0.125)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["k", "v", "q", "g"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_numbers_reach_only_their_rows(which, bad, d):
    """One element of one row: rows of the same tiles that do not see it (or
    that it does not see) come out as if it were not there."""
    x = R.Batch([420, 260], 2, 1, d, True, 99)
    window, sinks = 60, 3
    row = x.starts[0] + 200
    getattr(x, which)[0, row, 5] = bad
    # (an infinite score's own row is a matter of inf - inf: look at the others)
    out = run(x, window, sinks, device())
    scale = 1.0 / d ** 0.5
    clean = R.Batch([420, 260], 2, 1, d, True, 99)
    ref = run(clean, window, sinks, device())
    touched = torch.zeros(x.total, dtype=torch.bool)
    i = torch.arange(420)
    if which in ("k", "v"):
        rows = (i >= 200) & (i - 200 < window)   # queries that see key 200
    else:
        rows = i == 200                          # the query itself
    fwd = torch.zeros(420, dtype=torch.bool) if which == "g" else rows
    see = R.sees(420, window, sinks)
    keys = (see & rows[:, None]).any(0)          # keys that those queries see
    for name, a, r, hit in zip(("o", "lse", "dq", "dk", "dv"), out, ref,
                               (fwd, fwd, rows, keys, keys)):
        touched[:] = False
        touched[x.starts[0]:x.starts[0] + 420] = hit
        a, r = a.cpu(), r.cpu()
        assert bool(torch.isfinite(a[:, ~touched]).all()), name
        # sums in another order: twice a rounding of the result, and of its
        # terms where a row was formed again (2^-8 of P, dS)
        size = r[:, ~touched].abs().float().amax()
        assert float((a[:, ~touched].float() - r[:, ~touched].float()).abs().max()) <= \
            4 * R.HALF_BF16 * float(size), name
    assert not bool(torch.isfinite(out[0 if which != "g" else 2]).all())


def test_all_rows_bad():
    """Every row NaN: nothing to save, and it ends soon."""
    dev = device()
    x = R.Batch([1500], 4, 2, 64, False, 1)
    x.v[:] = float("nan")
    o, lse, dq, dk, dv = run(x, 700, 4, dev)
    assert bool(torch.isnan(o).all()) and bool(torch.isfinite(lse).all())
    for t in (dq, dk):
        assert bool(torch.isnan(t).all())


def test_window_of_the_sequence_is_causal():
    """fa_forward_gqa rounds the weights of its sums too, and its backward P,
    dP - D and their product (2^-8 of a term each): within that of each other."""
    dev = device()
    x = R.Batch([900, 900], 4, 2, 128, False, 21)
    q, k, v, g = (t.to(dev) for t in (x.q, x.k, x.v, x.g))
    o, lse = fa.attention_forward(q, k, v, causal=True)
    w, wl = fa.attention_forward(q, k, v, causal=True, window=900)
    a = fa.attention_backward(q, k, v, o, g, lse, causal=True)
    b = fa.attention_backward(q, k, v, o, g, lse, causal=True, window=900)
    status_ok()
    for i in range(2):
        f = [x.seq(t, i) for t in (x.q, x.k, x.v)]
        _, _, to, tl = R.forward(*f, 900, 0, 128 ** -0.5)
        assert bool(((x.seq(o, i) - x.seq(w, i)).abs() <= 3 * to).all())
        assert bool(((lse[i] - wl[i]).cpu().double().abs() <= 2 * tl + R.HALF_BF16).all())
        _, tols = R.backward(*f, x.seq(o, i), lse[i].cpu().double(), x.seq(g, i), 900, 0, 128 ** -0.5)
        for y, z, t in zip(a, b, tols):
            assert bool(((x.seq(y, i) - x.seq(z, i)).abs() <= 4 * t).all())


def test_gradients_against_differences():
    """sum(dq u) and so on against central differences of the 64-bit forward."""
    x = R.Batch([333], 2, 1, 64, False, 8)
    window, sinks, scale = 70, 5, 0.125
    _, _, *grads = run(x, window, sinks, device(), scale)
    f = [x.seq(t, 0) for t in (x.q, x.k, x.v)]
    g = x.seq(x.g, 0)
    gen = torch.Generator().manual_seed(1)
    loss = lambda y: float((R.forward(*y, window, sinks, scale)[0] * g).sum())
    tols = R.backward(*f, *R.forward(*f, window, sinks, scale)[:2], g, window, sinks, scale)[1]
    for i in range(3):
        u = torch.randn(f[i].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        up, down = (f[:i] + [f[i] + e * u] + f[i + 1:] for e in (h, -h))
        want = (loss(up) - loss(down)) / (2 * h)
        got = float((x.seq(grads[i], 0) * u).sum())
        # o and lse reach the backward rounded (o by 2^-8, through D): counted
        # as one more rounding of every dS term, as the tolerances count three
        assert abs(got - want) <= 2 * float((tols[i] * u.abs()).sum()) + 1e-6, i


def test_two_streams_and_a_graph():
    dev = device()
    x = R.Batch([700, 0, 333], 4, 2, 64, True, 31, 0, 10)
    q, k, v, g = (t.to(dev) for t in (x.q, x.k, x.v, x.g))
    cu, size = x.cu.to(dev), (3, 4, 2, 700, x.total, 64)
    n = fa.fa_backward_window_workspace_size(*size, 90, 4)

    def buffers():
        e = torch.zeros_like
        return dict(o=e(q), lse=torch.zeros(4, x.total, device=dev), dq=e(q), dk=e(k), dv=e(v),
                    ws=torch.empty(n, dtype=torch.uint8, device=dev))

    def call(t, stream=None):
        assert fa.fa_forward_window(q, k, v, t["o"], t["lse"], cu, *size, 0.125, 90, 4, stream) == 0
        assert fa.fa_backward_window(q, k, v, t["o"], g, t["lse"], t["dq"], t["dk"], t["dv"], cu,
                                     *size, 0.125, 90, 4, t["ws"], n, stream) == 0

    one = buffers()
    call(one)
    torch.cuda.synchronize()
    check(x, [one[m] for m in ("o", "lse", "dq", "dk", "dv")], 90, 4, 0.125)
    sides = [buffers() for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s, t in zip(streams, sides):
            call(t, s)
    torch.cuda.synchronize()
    graph, t = torch.cuda.CUDAGraph(), buffers()
    sides.append(t)
    with torch.cuda.graph(graph):
        call(t)
    for _ in range(3):
        graph.replay()
    status_ok()
    for t in sides:
        for m in ("o", "lse", "dk", "dv"):
            assert torch.equal(t[m], one[m]), m
        assert bool(((t["dq"] - one["dq"]).abs().float()
                     <= 2 * R.HALF_BF16 * one["dq"].abs().float() + 1e-4).all())


@pytest.mark.parametrize("case", [
    # few key tiles: walks cut by the group's heads too
    (1, 8, 1, 140, 64, 20, 0), (1, 12, 2, 700, 128, 150, 4), (2, 6, 1, 1100, 64, 260, 129),
    (1, 16, 4, 1025, 128, 1025, 2), (3, 16, 1, 257, 128, 64, 1),
])
def test_few_key_tiles(case):
    B, H, Hkv, N, d, window, sinks = case
    x = R.Batch([N] * B, H, Hkv, d, False, 17 + N)
    check(x, run(x, window, sinks, device()), window, sinks)
    if B == 1:
        x = R.Batch([N // 3, 0, N - N // 3], H, Hkv, d, True, 19 + N, 3, 9)
        check(x, run(x, window, sinks, device()), window, sinks)


def test_an_infinity_that_everyone_sees():
    """In a first token's value: one column of every later row, formed again
    only until it is met; the other columns as without it."""
    dev = device()
    x = R.Batch([2500], 4, 2, 64, False, 41)
    clean = run(x, 300, 4, dev)
    x.v[0, :, 2, 7] = float("inf")
    o, lse, dq, dk, dv = run(x, 300, 4, dev)
    assert bool(torch.isinf(o[0, :, 2:, 7]).all()) and torch.equal(lse, clean[1])
    keep = [c for c in range(64) if c != 7]
    assert torch.equal(o[..., keep], clean[0][..., keep])
    # rows 0 and 1 do not see it: formed again, both within the formula's tolerance
    _, _, tol, _ = R.forward(*(x.seq(t, 0)[:, :2] for t in (x.q, x.k, x.v)), 300, 4, 0.125)
    assert bool(((o[0, :, :2] - clean[0][0, :, :2]).cpu().double().abs() <= 2 * tol).all())
    assert bool(torch.isfinite(dv).all()) and not bool(torch.isfinite(dq[0, :, 2:]).any())
