"""Windowed attention where a row sees a NaN or an infinity: which of its
outputs, and of the gradients that it has a part in, are NaN.  On a GPU."""
import pytest
import torch

import io_aware_exact_15_gb300 as fa
import window_ref as R
from gpu_common import device, status_ok

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def run(x, window, sinks, dev):
    q, k, v, g = (t.to(dev) for t in (x.q, x.k, x.v, x.g))
    kw = dict(causal=True, window=window, sinks=sinks)
    if x.packed:
        kw |= dict(cu_seqlens=x.cu.to(dev), max_seqlen=max(x.lens))
    o, lse = fa.attention_forward(q, k, v, **kw)
    grads = fa.attention_backward(q, k, v, o, g, lse, **kw)
    status_ok()
    return (o, lse) + tuple(grads)


CASES = [
    # lengths, H, Hkv, d, window, sinks, packed, the bad row (of the first sequence)
    ([420, 260], 2, 1, 64, 60, 3, True, 200),
    ([420, 260], 2, 1, 128, 60, 3, True, 419),
    ([300], 4, 2, 128, 300, 0, False, 129),
    ([1281], 2, 2, 64, 200, 4, False, 2),    # a first token: its walk is cut
    ([1300, 77, 1100], 4, 1, 128, 150, 4, True, 700),
    ([1], 1, 1, 64, 1, 0, False, 0),
]


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("case", CASES)
def test_a_nan_score(which, case):
    """lse and o of the rows with such a score are NaN whole, dv and dk of all
    keys that they see, and their dq; everything else has its number."""
    lens, H, Hkv, d, window, sinks, packed, row = case
    x = R.Batch(lens, H, Hkv, d, packed, 51)
    getattr(x, which)[..., 0 if packed else slice(None), row, :][..., 9] = NAN
    out = run(x, window, sinks, device())
    scale = d ** -0.5
    for b, n in enumerate(lens):
        q, k, v, g = (x.seq(t, b) for t in (x.q, x.k, x.v, x.g))
        o, lse, tol_o, tol_l = R.forward(q, k, v, window, sinks, scale)
        got_o, got_l = x.seq(out[0], b), x.seq(out[1][..., None], b)[..., 0]
        nan = torch.isnan(lse)
        assert bool(nan.any()) == (b == 0)
        assert torch.equal(torch.isnan(got_l), nan) and bool(torch.isfinite(got_l[~nan]).all())
        assert bool(torch.isnan(got_o[nan]).all())
        assert bool(((got_l - lse).abs() <= tol_l)[~nan].all())
        assert bool(((got_o - o).abs() <= tol_o)[~nan].all())
        ref, tol = R.backward(q, k, v, got_o, got_l, g, window, sinks, scale)
        for name, a, r, t in zip(("dq", "dk", "dv"), out[2:], ref, tol):
            a = x.seq(a, b)
            assert torch.equal(torch.isnan(a), torch.isnan(r)), (name, b)
            err = torch.where(torch.isnan(r), torch.zeros((), dtype=torch.float64), (a - r).abs())
            assert bool((err <= torch.nan_to_num(t)).all()), (name, b)


def test_a_nan_score_in_the_two_tile_form():
    """More than four waves of two-tile CTAs: the other instantiation."""
    for d in (64, 128):
        x = R.Batch([300] * 160, 10, 5, d, False, 5)
        x.k[77, 3, 140, 1] = NAN
        o, lse, *_ = run(x, 140, 4, device())
        want = torch.zeros(160, 10, 300, dtype=torch.bool)
        want[77, 6:8, 140:280] = True
        assert torch.equal(torch.isnan(lse).cpu(), want)
        assert torch.equal(torch.isnan(o).all(-1).cpu(), want)
        assert torch.equal(torch.isnan(o).any(-1).cpu(), want)


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("d", [64, 128])
def test_an_infinite_score(which, d):
    """A score of +infinity (with any others): lse and o are NaN.  One of
    -infinity is a weight of zero."""
    x = R.Batch([420, 260], 2, 1, d, True, 52)
    window, sinks, row = 60, 3, 200
    getattr(x, which)[0, row, 9] = INF
    o, lse, *_ = run(x, window, sinks, device())
    clean = R.Batch([420, 260], 2, 1, d, True, 52)
    for b in range(2):
        ref, want, _, _ = R.forward(*(x.seq(t, b) for t in (x.q, x.k, x.v)), window, sinks, d ** -0.5)
        # of the scores that are numbers, whose terms the clean batch has too
        tol = R.forward(*(clean.seq(t, b) for t in (clean.q, clean.k, clean.v)), window, sinks,
                        d ** -0.5)[3]
        got_o, got_l = x.seq(o, b), x.seq(lse[..., None], b)[..., 0]
        up = torch.isposinf(want) | torch.isnan(want)
        assert bool(up.any()) == (b == 0)
        assert bool(torch.isnan(got_l[up]).all()) and bool(torch.isnan(got_o[up]).all())
        assert bool(torch.isfinite(got_o[~up]).all())
        assert bool(((got_l - want).abs() <= tol + 2.0 ** -20 * want.abs())[~up].all())


@pytest.mark.parametrize("case", [
    # lengths, H, Hkv, d, window, sinks, packed, the row
    ([420, 260], 2, 1, 64, 60, 3, True, 400),
    ([420, 260], 4, 2, 128, 500, 0, True, 419),
    ([300], 4, 1, 128, 300, 0, False, 17),
    ([300], 4, 1, 64, 1, 0, False, 299),
    ([1281], 2, 2, 64, 200, 4, False, 1100),
])
def test_a_row_whose_scores_are_all_minus_infinity(case):
    """It sees nothing: o 0, lse -infinity, dq 0, and no share in dk, dv.  The
    next sequence (all NaN) shares its last tile and shows nowhere."""
    lens, H, Hkv, d, window, sinks, packed, row = case
    x = R.Batch(lens, H, Hkv, d, packed, 53)
    at = (slice(None), row) if packed else (slice(None), slice(None), row)
    x.k[..., 5] = 1.0
    x.g[at] = 0.0  # for the formula: a row without a gradient has no share either
    n = lens[0]
    q, k, v, g = (x.seq(t, 0) for t in (x.q, x.k, x.v, x.g))
    ro, rl, to, tl = R.forward(q, k, v, window, sinks, d ** -0.5)
    x.q[at + (5,)] = -INF
    x.g[at] = 1.0
    for t in (x.q, x.k, x.v, x.g):
        if packed:
            t[:, n:] = NAN
    out = run(x, window, sinks, device())
    o, lse = x.seq(out[0], 0), x.seq(out[1][..., None], 0)[..., 0]
    assert bool(torch.isneginf(lse[:, row]).all()) and bool((o[:, row] == 0).all())
    rest = torch.arange(n) != row
    assert bool(((o - ro).abs() <= to)[:, rest].all())
    assert bool(((lse - rl).abs() <= tl)[:, rest].all())
    o[:, row], lse[:, row] = ro[:, row], rl[:, row]
    ref, tol = R.backward(q, k, v, o, lse, g, window, sinks, d ** -0.5)
    for name, a, r, t in zip(("dq", "dk", "dv"), out[2:], ref, tol):
        a = x.seq(a, 0)
        assert bool(torch.isfinite(a).all()), name
        if name == "dq":
            assert bool((a[:, row] == 0).all())
            a, r, t = a[:, rest], r[:, rest], t[:, rest]
        assert bool(((a - r).abs() <= t).all()), name
