"""Attention of drafted tokens over the paged cache with a sliding window and
first tokens that stay visible, against a plain 64-bit evaluation: formats,
head groups, chains and trees, pages that are gone, and garbage wherever
nothing may be read from."""
import numpy as np
import pytest

from gpu_common import device, status_ok, torch
import serving_ref as R
import window_ref
from test_gpu_tree import Problem

import io_aware_exact_15_gb300 as fa

pytestmark = pytest.mark.gpu


def sees(hist, n, T, bits, window, sinks):
    """[T, hist + n]: who sees what, from the definition."""
    s = R.sees(hist, n, T, bits)
    for i in range(n):
        other = int(bits[i, :n].sum()) - int(bits[i, i]) if bits is not None else i
        j = np.arange(hist + n)
        near = (j > hist + other - window) | (j < sinks)
        if bits is not None:
            near[hist:] = True
        s[i] &= near
    return s


class Windowed(Problem):
    """What no draft sees is poisoned: rows in pages that stay, and pages that
    go (their table entries become -1 or some number)."""

    def __init__(self, fmt, case, seed, dev, **kw):
        B, H, Hkv, T, d, page, hist, drafts, mask, self.window, self.sinks = case
        super().__init__(fmt, B, H, Hkv, T, d, page, hist, drafts, mask, seed, dev, **kw)
        rng = np.random.default_rng(seed + 1)
        table = self.table.numpy().copy()
        for b in range(B):
            n = self.drafts[b]
            seen = self.seen(b)[:max(n, 1)].any(0) if n else np.zeros(hist[b], bool)
            for p in range(-(-(hist[b] + n) // page)):
                rows = seen[p * page:(p + 1) * page]
                where = int(table[b, p])
                if not rows.any():
                    table[b, p] = rng.choice([-1, -7, 1 << 30, where])
                    rows = np.zeros(page, bool)
                dead = torch.from_numpy(np.nonzero(~rows)[0]).to(dev)
                for c, s in ((self.kc, self.ks), (self.vc, self.vs)):
                    if fmt == R.BF16:
                        c[where, :, dead] = float("nan")
                    else:
                        c.view(torch.uint8)[where, :, dead] = 0x7F
                        s[where, :, dead] = 255
        self.table_d = torch.from_numpy(table).to(dev)

    def seen(self, b):
        return sees(self.hist[b], self.drafts[b], self.T,
                    None if self.bits is None else self.bits[b], self.window, self.sinks)

    def run(self, scale=None, **kw):
        return super().run(scale, window=self.window, sinks=self.sinks, **kw)

    def check(self, o, lse, scale=None):
        scale = 1.0 / self.d ** 0.5 if scale is None else scale
        o, lse = R.f64(o), R.f64(lse)
        for b in range(self.B):
            kk, vv = (R.quantise(R.f64(x[b]), self.fmt) for x in (self.k, self.v))
            ref, ref_l, size, score = R.attention(R.f64(self.q[b]), kk, vv, self.seen(b), scale)
            # as in Problem.check
            off = 2.0 ** -20 * (1 + score)
            tol = (R.HALF_BF16 + 2 * off[..., None]) * size + R.HALF_BF16 * np.abs(ref) + 1e-30
            if self.fmt != R.BF16 and vv.size:
                tol = tol + vv.shape[1] * 2.0 ** -31 * np.abs(vv[np.isfinite(vv)]).max(initial=0)
            fine = np.isfinite(ref)
            assert np.array_equal(np.isfinite(o[b]), fine), (b, "finite where the formula is not, or not")
            err = np.abs(np.where(fine, o[b] - ref, 0))
            assert (err <= tol)[fine].all(), \
                (b, np.argwhere(fine & ~(err <= tol))[:4], float(np.nanmax(err / tol)))
            none = np.isneginf(ref_l)
            assert np.array_equal(np.isneginf(lse[b]), none)
            ok = np.isfinite(ref_l)
            with np.errstate(invalid="ignore"):
                far = np.abs(lse[b] - ref_l)
            assert (far[ok] <= (off + 2.0 ** -20 * np.abs(ref_l))[ok]).all()


CASES = [
    # B, H, Hkv, T, d, page, hist, drafts, mask, window, sinks
    (1, 1, 1, 1, 64, 16, [0], None, None, 1, 0),
    (3, 4, 2, 1, 128, 64, [1, 300, 900], None, None, 100, 4),
    (3, 4, 1, 1, 64, 16, [127, 128, 129], None, None, 128, 16),
    (4, 8, 2, 1, 128, 128, [512, 513, 640, 2000], None, None, 1, 1),
    (2, 2, 2, 1, 128, 32, [700, 5], None, None, 129, 130),
    (3, 2, 2, 5, 64, 32, [0, 127, 500], [5, 1, 0], "tree", 7, 3),
    (2, 8, 1, 33, 128, 128, [129, 1065], None, "tree", 40, 4),
    (4, 6, 3, 17, 64, 16, [40, 0, 255, 600], [17, 3, 9, 0], "any", 64, 0),
    (1, 16, 2, 40, 128, 64, [1700], [39], "any", 333, 64),
    (2, 3, 1, 65, 64, 128, [3, 860], [65, 64], None, 20, 2),     # chains longer than the window
    (1, 12, 1, 100, 64, 32, [900], None, None, 128, 200),
    (2, 1, 1, 130, 128, 16, [426, 2], [130, 77], None, 1, 0),
    (2, 2, 1, 130, 128, 64, [1426, 700], [130, 77], "tree", 256, 4),
    (1, 8, 8, 7, 128, 32, [3001], None, "tree", 1024, 4),
    (5, 4, 4, 2, 64, 64, [1023, 5, 0, 512, 77], [2, 2, 2, 1, 0], None, 100000, 4),
    (2, 4, 2, 300, 64, 64, [1000, 0], [300, 150], None, 90, 7),  # a prompt in chunks
    (33, 4, 2, 1, 64, 16, [37 * i for i in range(33)], None, None, 200, 20),
    (1, 2, 1, 6, 128, 64, [500], None, None, 4, 1024),           # all of it first tokens
    # long windows and few problems: several CTAs on each, also on those of a tile or none
    (1, 4, 1, 1, 128, 64, [2900], None, None, 2500, 4),
    (5, 4, 2, 1, 64, 32, [1500, 0, 129, 640, 2600], [1, 0, 1, 1, 1], None, 1400, 70),
    (9, 8, 4, 1, 128, 16, [1000, 3, 999, 0, 300, 128, 127, 1300, 700], None, None, 1024, 0),
    (18, 4, 4, 1, 64, 64, [97 * i for i in range(18)], None, None, 600, 16),
    (2, 4, 1, 4, 128, 128, [1900, 60], None, "tree", 1100, 200),
    (3, 2, 2, 12, 64, 32, [0, 1111, 800], [12, 1, 7], "any", 500, 3),
]


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.INT8])
@pytest.mark.parametrize("case", CASES)
def test_against_the_formula(case, fmt):
    p = Windowed(fmt, case, 3 + len(case[6]), device())
    o, lse = p.run()
    status_ok()
    p.check(o, lse)


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.INT8])
@pytest.mark.parametrize("heads", [(2, 2), (12, 2), (40, 1), (160, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_numbers_of_some_drafts(heads, fmt, d):
    """A NaN or an infinity in a value at the window's edge or in a draft
    reaches the drafts that see it and no other."""
    H, Hkv = heads
    case = (2, H, Hkv, 5, d, 32, [400, 130], None, None, 50, 3)
    p = Windowed(fmt, case, 77, device())
    bad = [float("nan"), float("inf")]
    for b in range(2):
        for i, at in enumerate((p.hist[b] - 50 + 3, p.hist[b] + 2)):  # seen by drafts 0-2; by 2-4
            p.v[b][0, at, 9] = bad[i]
    # write those rows again as the cache holds them
    for b in range(2):
        for at in (p.hist[b] - 50 + 3, p.hist[b] + 2):
            row = torch.tensor([at], dtype=torch.int32, device=p.dev)
            fa.cache_append(p.k[b][None, :, at:at + 1].contiguous().to(p.dev),
                            p.v[b][None, :, at:at + 1].contiguous().to(p.dev), p.kc, p.vc,
                            p.table_d[b:b + 1].contiguous(), row, None, p.ks, p.vs)
    o, lse = p.run()
    status_ok()
    with np.errstate(invalid="ignore"):
        p.check(o, lse)
    o = R.f64(o)
    assert not np.isfinite(o[:, 0]).all()
    if Hkv > 1:  # other key/value heads
        assert np.isfinite(o[:, H - 1]).all()
    if fmt == R.BF16:  # other columns (an 8-bit row is bad as a whole)
        assert np.isfinite(o[..., :9]).all()


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3])
def test_same_as_whole_sequence(fmt):
    """A chain of tokens over the cache is the last rows of the windowed
    forward pass, both within their tolerances of the same numbers."""
    dev = device()
    case = (1, 4, 2, 20, 64, 64, [333], None, None, 70, 4)
    p = Windowed(fmt, case, 5, dev)
    o, lse = p.run()
    n = 353
    k, v = (torch.from_numpy(R.quantise(R.f64(x[0]), fmt)).bfloat16().to(dev)[None] for x in (p.k, p.v))
    q = torch.zeros(1, 4, n, 64, dtype=torch.bfloat16, device=dev)
    q[:, :, 333:] = p.q_d
    fo, fl = fa.attention_forward(q, k, v, causal=True, window=70, sinks=4)
    status_ok()
    ro, rl, to, tl = window_ref.forward(q[0].cpu().double(), k[0].cpu().double(), v[0].cpu().double(),
                                        70, 4, 0.125)
    # both sides are within `to` of the formula (the cache's: one rounding less)
    assert bool(((o[0] - fo[0, :, 333:]).cpu().double().abs() <= 2 * to[:, 333:]).all())
    assert bool(((lse[0] - fl[0, :, 333:]).cpu().double().abs() <= 2 * tl[:, 333:]).all())


def test_window_beyond_everything_is_tree_attention():
    """The same sums, cut in other places: both within the same tolerances."""
    dev = device()
    for T, mask in ((1, None), (9, "tree"), (70, "tree"), (140, None)):
        p = Problem(R.BF16, 2, 4, 2, T, 128, 32, [500, 77], None, mask, 9, dev)
        a, b = p.run(), p.run(window=1 << 30, sinks=4)
        status_ok()
        p.check(*a)
        p.check(*b)


def test_streams_and_a_graph():
    dev = device()
    case = (3, 8, 2, 3, 128, 64, [900, 20, 450], [3, 1, 2], "tree", 200, 4)
    p = Windowed(R.INT8, case, 15, dev)
    o, lse = p.run()
    outs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            outs.append(p.run(stream=s))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs.append(p.run())
    for _ in range(3):
        graph.replay()
    status_ok()
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)
    p.check(o, lse)
