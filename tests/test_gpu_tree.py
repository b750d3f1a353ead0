"""Attention of drafted tokens over the paged cache against a plain 64-bit
evaluation: formats, head groups, lengths from none to several thousand,
trees, chains, rows that see nothing, and garbage wherever nothing may be
read from."""
import numpy as np
import pytest

from gpu_common import device, status_ok, torch
import serving_ref as R

import io_aware_exact_15_gb300 as fa

pytestmark = pytest.mark.gpu


class Problem:
    """A cache on the device whose rows are known on the host.  Every byte
    that no sequence owns is garbage: NaN, infinities, any scale byte."""

    def __init__(self, fmt, B, H, Hkv, T, d, page, hist, drafts, mask, seed, dev, size=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.B, self.H, self.Hkv, self.T, self.d = fmt, B, H, Hkv, T, d
        self.hist, self.drafts = hist, [T] * B if drafts is None else drafts
        total = [a + b for a, b in zip(hist, self.drafts)]
        self.table, num = R.page_table(rng, total, page)
        self.k = [(size * torch.randn(Hkv, n, d, generator=g)).bfloat16() for n in total]
        self.v = [torch.randn(Hkv, n, d, generator=g).bfloat16() for n in total]
        self.q = torch.randn(B, H, T, d, generator=g).bfloat16()
        if mask == "tree":
            self.bits = R.random_trees(rng, B, T)
        elif mask == "any":
            self.bits = rng.random((B, T, T)) < 0.3
            self.bits[:, T // 2] = False  # sees no draft, not even itself
        else:
            self.bits = None
        kind = R.DTYPES[fmt]
        if fmt == R.BF16:
            junk = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38]).bfloat16()
            cache = [junk.repeat(num * Hkv * page * d // 4).view(num, Hkv, page, d).clone()
                     for _ in range(2)]
        else:
            cache = [torch.from_numpy(rng.integers(0, 256, (num, Hkv, page, d), dtype=np.uint8))
                     for _ in range(2)]
        scale = [torch.from_numpy(rng.integers(0, 256, (num, Hkv, page), dtype=np.uint8))
                 for _ in range(2)]
        self.kc, self.vc = (c.view(kind).to(dev) for c in cache)
        self.ks, self.vs = (s.to(dev) for s in scale)
        self.table_d = self.table.to(dev)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        self.hist_d = i32(hist)
        self.drafts_d = None if drafts is None else i32(drafts)
        self.mask_d = None if self.bits is None else R.words_of(self.bits).to(dev)
        self.q_d = self.q.to(dev)
        self.dev = dev
        self.fill()

    def fill(self):
        """Appends every sequence's rows."""
        most = max(1, max(k.shape[1] for k in self.k))
        pad = lambda xs: torch.stack([torch.nn.functional.pad(x, (0, 0, 0, most - x.shape[1]))
                                      for x in xs]).to(self.dev)
        zero = torch.zeros(self.B, dtype=torch.int32, device=self.dev)
        count = torch.tensor([k.shape[1] for k in self.k], dtype=torch.int32, device=self.dev)
        fa.cache_append(pad(self.k), pad(self.v), self.kc, self.vc, self.table_d, zero, count,
                        self.ks, self.vs)

    def run(self, scale=None, **kw):
        return fa.tree_attention(self.q_d, self.kc, self.vc, self.table_d, self.hist_d,
                                 self.drafts_d, self.mask_d, scale, self.ks, self.vs, **kw)

    def check(self, o, lse, scale=None, rows=None):
        """rows: (sequence, draft) pairs to look at, or all of them."""
        scale = 1.0 / self.d ** 0.5 if scale is None else scale
        o, lse = R.f64(o), R.f64(lse)
        for b in range(self.B):
            kk, vv = (R.quantise(R.f64(x[b]), self.fmt) for x in (self.k, self.v))
            seen = R.sees(self.hist[b], self.drafts[b], self.T,
                          None if self.bits is None else self.bits[b])
            ref, ref_l, size, score = R.attention(R.f64(self.q[b]), kk, vv, seen, scale)
            # P and O are rounded to bf16 once each; scores are fp32 sums of d
            # products and the exponential's argument is fp32: an error of
            # 2^-20 of the largest score's terms moves P by that factor, twice
            # (its own weight and the sum's)
            off = 2.0 ** -20 * (1 + score)
            tol = (R.HALF_BF16 + 2 * off[..., None]) * size + R.HALF_BF16 * np.abs(ref) + 1e-30
            # 8-bit caches: weights times the values' scales are f16
            # numbers of up to 2^15, the largest at least 2^7: below 2^-14 they
            # are off by up to 2^-25, which is 2^-32 of the largest.  A value's
            # number is at most 448 times its scale (127) and a row's largest
            # at least half of that (or the scale is 2^-100), so a key adds at
            # most 2^-32 x 2 x the largest weighted value
            if self.fmt != R.BF16 and vv.size:
                tol = tol + vv.shape[1] * 2.0 ** -31 * np.abs(vv[np.isfinite(vv)]).max(initial=0)
            keep = np.ones(self.T, bool) if rows is None else \
                np.array([(b, t) in rows for t in range(self.T)])
            err = np.abs(o[b] - ref)
            assert (err <= tol)[:, keep].all(), \
                (b, np.argwhere(~(err <= tol))[:4], float(np.nanmax(err / tol)))
            none = np.isinf(ref_l)
            assert np.array_equal(np.isneginf(lse[b])[:, keep], none[:, keep])
            with np.errstate(invalid="ignore"):
                far = np.abs(lse[b] - ref_l) > off + 2.0 ** -20 * np.abs(ref_l)
            assert not far[~none & keep[None]].any()


CASES = [
    # B, H, Hkv, T, d, page, hist, drafts, mask
    (1, 1, 1, 1, 64, 16, [0], None, None),
    (2, 4, 2, 1, 128, 64, [1, 300], None, None),
    (3, 2, 2, 5, 64, 32, [0, 127, 128], [5, 1, 0], "tree"),
    (2, 8, 1, 33, 128, 128, [129, 65], None, "tree"),
    (4, 6, 3, 17, 64, 16, [40, 0, 255, 1], [17, 3, 9, 0], "any"),
    (1, 16, 2, 40, 128, 64, [700], [39], "any"),
    (2, 3, 1, 65, 64, 128, [3, 60], [65, 64], "tree"),
    (1, 12, 1, 100, 64, 32, [200], None, None),
    (2, 1, 1, 130, 128, 16, [126, 2], [130, 77], "tree"),
    (1, 8, 8, 7, 128, 32, [3001], None, "tree"),
    (5, 4, 4, 2, 64, 64, [1023, 5, 0, 512, 77], [2, 2, 2, 1, 0], None),
]
FORMATS = [R.BF16, R.E4M3, R.INT8]


def name(c):
    return "-".join(map(str, c[:6]))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", CASES, ids=name)
def test_against_plain(case, fmt):
    p = Problem(fmt, *case, seed=sum(case[:6]) + fmt, dev=device())
    o, lse = p.run()
    status_ok()
    p.check(o, lse)


def many(B, lo, hi, seed):
    return [int(x) for x in np.random.default_rng(seed).integers(lo, hi, B)]


MANY = [
    # as CASES, with several problems and several tiles for each SM: runs that
    # begin and end inside problems, problems of one tile, all three of
    # up to 128 rows, up to 256, and groups of 256 with a short last one
    (40, 8, 8, 2, 64, 32, many(40, 0, 700, 1), many(40, 0, 3, 2), None),
    (60, 4, 4, 3, 128, 16, many(60, 0, 260, 3), None, "tree"),
    (30, 3, 1, 50, 64, 64, many(30, 0, 900, 4), many(30, 0, 51, 5), "any"),
    (24, 3, 1, 100, 128, 128, many(24, 0, 800, 6), many(24, 1, 101, 7), "tree"),
    (20, 5, 1, 120, 64, 16, many(20, 100, 600, 8), None, "any"),
    # long runs
    (4, 8, 2, 23, 128, 64, [9000, 8192, 5001, 12345], [23, 9, 22, 1], "tree"),
    (3, 2, 1, 29, 64, 128, [30000, 16384, 777], None, "any"),
    (2, 8, 2, 64, 128, 32, [8192, 6003], [64, 63], "tree"),
    # few rows (up to 16, up to 32), long and short
    (6, 8, 2, 4, 128, 16, many(6, 3000, 9000, 9), [4, 1, 0, 3, 4, 2], "tree"),
    (5, 8, 1, 4, 64, 32, many(5, 100, 9000, 10), None, None),
    (3, 6, 2, 10, 128, 64, [8191, 8193, 4000], [10, 9, 10], "any"),
    (70, 16, 4, 1, 64, 128, many(70, 0, 500, 11), None, None),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", MANY, ids=name)
def test_runs_over_many_problems(case, fmt):
    p = Problem(fmt, *case, seed=sum(case[:6]) + fmt, dev=device())
    o, lse = p.run()
    status_ok()
    p.check(o, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_growing_scores(fmt):
    """Keys that grow along the sequence: the running max moves far, by more
    than fp32 exponents hold."""
    p = Problem(fmt, 2, 4, 2, 6, 64, 16, [500, 260], None, "tree", seed=3, dev=device())
    for k in p.k:
        k *= torch.exp2(torch.linspace(-8, 6, k.shape[1]))[None, :, None].bfloat16()
    p.fill()
    o, lse = p.run(scale=1.0)
    status_ok()
    p.check(o, lse, scale=1.0)


@pytest.mark.parametrize("T", [1, 9, 40])
def test_eight_bit_result_is_that_of_the_values_read_back(T):
    """An 8-bit cache gives what a bf16 cache of its values gives: the same
    products, with sums in another order (lse: 2^-20), each weight rounded
    once on either side and O once (O: 2^-8 of the sums' size, twice, and
    2^-8 of the value, twice)."""
    dev = device()
    for fmt in (R.E4M3, R.INT8):
        p = Problem(fmt, 2, 8, 2, T, 128, 64, [333, 70], [T, (T + 1) // 2], "tree", seed=21,
                    dev=dev)
        o, lse = p.run()
        most = max(k.shape[1] for k in p.k)
        zero = torch.zeros(2, dtype=torch.int32, device=dev)
        count = p.hist_d + p.drafts_d
        k, v = fa.cache_read(p.kc, p.vc, p.table_d, zero, most, count, p.ks, p.vs)
        kc, vc = (torch.empty(p.kc.shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
        fa.cache_append(k, v, kc, vc, p.table_d, zero, count)
        o2, lse2 = fa.tree_attention(p.q_d, kc, vc, p.table_d, p.hist_d, p.drafts_d, p.mask_d)
        status_ok()
        seen = torch.isfinite(lse2)
        assert torch.equal(torch.isfinite(lse), seen)
        assert ((lse - lse2)[seen].abs() <= 2.0 ** -20 * (1 + lse2[seen].abs())).all()
        size = v.float().abs().max()  # at most this is sum p |v|
        tol = 2 * R.HALF_BF16 * (size + o2.float().abs())
        assert ((o.float() - o2.float()).abs() <= tol).all()
        p.check(o, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_numbers_in_other_branches(fmt):
    """NaN and infinities in the keys and values of drafts reach the rows
    that see them and no others."""
    dev = device()
    p = Problem(fmt, 2, 4, 2, 12, 64, 32, [100, 0], None, "tree", seed=8, dev=dev)
    for what in ("k", "v"):
        p = Problem(fmt, 2, 4, 2, 12, 64, 32, [100, 0], None, "tree", seed=8, dev=dev)
        bad = {0: 4, 1: 7}  # a draft of each sequence
        for b, i in bad.items():
            rows = (p.k if what == "k" else p.v)[b]
            rows[:, p.hist[b] + i, 3] = float("nan")
            rows[:, p.hist[b] + i, 40] = float("inf")
        p.fill()
        o, lse = p.run()
        status_ok()
        clean = {(b, t) for b in range(2) for t in range(12) if not p.bits[b, t, bad[b]]}
        assert len(clean) > 4 and len(clean) < 24
        p.check(o, lse, rows=clean)
        for b in range(2):
            for t in range(12):
                if (b, t) not in clean:
                    assert torch.isnan(o[b, :, t, 3]).all()
                    if what == "v":
                        assert not torch.isfinite(o[b, :, t, 40]).any()
                        assert torch.isfinite(lse[b, :, t]).all()


def test_nothing_outside_is_written():
    """Outputs and workspace between guard bands; workspace contents on
    entry do not matter."""
    dev = device()
    p = Problem(R.BF16, 2, 4, 2, 5, 64, 16, [900, 30], [5, 2], "tree", seed=2, dev=dev)
    want = p.run()
    B, H, T, d = 2, 4, 5, 64
    n, need = B * H * T * d, fa.fa_tree_attention_workspace_size(B, H, 2, T, d)
    for fill in (0x00, 0xFF):
        band = torch.full((n + 512,), 7.0, dtype=torch.bfloat16, device=dev)
        lband = torch.full((B * H * T + 64,), 7.0, device=dev)
        ws = torch.full((need + 512,), fill, dtype=torch.uint8, device=dev)
        o, lse = band[256:256 + n].view(B, H, T, d), lband[32:32 + B * H * T].view(B, H, T)
        assert fa.fa_tree_attention(p.q_d, p.kc, p.vc, p.ks, p.vs, p.table_d, p.hist_d, p.drafts_d,
                                    p.mask_d, o, lse, fa.FA_CACHE_BF16, B, H, 2, T, d,
                                    p.kc.shape[0], 16, p.table.shape[1], 0.125, ws[256:],
                                    need) == fa.FA_OK
        status_ok()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert (band[:256] == 7).all() and (band[256 + n:] == 7).all()
        assert (lband[:32] == 7).all() and (lband[32 + B * H * T:] == 7).all()
        assert (ws[:256] == fill).all() and (ws[256 + need:] == fill).all()


def test_bad_lengths_and_tables_stay_inside():
    """Lengths past the table and page ids outside the pool give some result
    and no access outside; a negative length is an empty history."""
    dev = device()
    for fmt in FORMATS:
        p = Problem(fmt, 3, 2, 1, 4, 64, 16, [50, 20, 10], None, None, seed=4, dev=dev)
        p.table_d[1] = torch.tensor([-5, 10 ** 6, 2 ** 31 - 1, -1][:p.table.shape[1]],
                                    dtype=torch.int32)
        p.hist_d.copy_(torch.tensor([10 ** 9, 20, -7], dtype=torch.int32))
        p.drafts_d = torch.tensor([2 ** 31 - 1, 3, -1], dtype=torch.int32, device=dev)
        o, lse = p.run()
        status_ok()
        assert (o[2] == 0).all() and torch.isneginf(lse[2]).all()


def test_streams_graphs_and_a_shared_workspace():
    """A side stream; two graphs over one workspace, replayed in turn while
    the lengths change between replays."""
    dev = device()
    p = Problem(R.E4M3, 2, 8, 2, 6, 128, 64, [1500, 400], None, "tree", seed=6, dev=dev)
    want = p.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = p.run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.empty(fa.fa_tree_attention_workspace_size(2, 8, 2, 6, 128), dtype=torch.uint8,
                     device=dev)
    outs, graphs = [], []
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(p.run(workspace=ws))
        graphs.append(graph)
    for k in range(4):
        graphs[k % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[k % 2], want))
    p.hist_d.copy_(torch.tensor([700, 0], dtype=torch.int32))
    want = p.run()
    graphs[0].replay()
    status_ok()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want))


EDGES = [  # G, T: query rows per key/value head on both sides of every change of form
    (1, 8), (3, 3), (1, 16), (1, 17), (2, 12), (5, 5), (4, 8), (3, 11), (2, 64), (3, 43), (4, 64),
    (1, 257), (1, 513), (2, 1024),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", EDGES)
def test_numbers_of_rows(G, T, d):
    for fmt in FORMATS:
        p = Problem(fmt, 2, 2 * G, 2, T, d, 32, [190, 31], [T, (T + 1) // 2], "tree",
                    seed=G + T + fmt, dev=device())
        o, lse = p.run()
        status_ok()
        p.check(o, lse)


@pytest.mark.parametrize("T", [1, 4, 12, 80])
def test_bad_queries(T):
    """NaN and infinities in one draft's queries are that draft's alone."""
    for fmt in FORMATS:
        p = Problem(fmt, 2, 4, 2, T, 128, 64, [300, 20], None, None, seed=T, dev=device())
        p.q[0, :, T // 2, 5] = float("nan")
        p.q[1, :, 0, 9] = float("inf")
        p.q[1, :, T - 1] = 0  # every key the same weight
        if T > 1:
            p.q[0, :, 0] *= 2.0 ** -100
        p.q_d.copy_(p.q)
        o, lse = p.run()
        status_ok()
        bad = {(0, T // 2)} | ({(1, 0)} if T > 1 else set())
        p.check(o, lse, rows={(b, t) for b in range(2) for t in range(T)} - bad)
        assert torch.isnan(o[0, :, T // 2]).all() and torch.isnan(lse[0, :, T // 2]).all()


@pytest.mark.parametrize("T", [2, 40])
def test_offsets_past_32_bits(T):
    """Pages more than 2^32 elements into the pool give what pages at its
    front give (16384 + 8 pages of 2^18 elements)."""
    dev = device()
    Hkv, page, d, num = 16, 128, 128, 16384 + 8
    for fmt in (R.BF16, R.E4M3):
        p = Problem(fmt, 2, Hkv, Hkv, T, d, page, [200, 310], None, "tree", seed=T, dev=dev)
        want = p.run()
        kc, vc = (torch.empty(num, Hkv, page, d, dtype=p.kc.dtype, device=dev) for _ in range(2))
        ks, vs = (torch.empty(num, Hkv, page, dtype=torch.uint8, device=dev) for _ in range(2))
        p.kc, p.vc, p.ks, p.vs = kc, vc, ks, vs
        p.table_d = num - 1 - p.table_d
        p.fill()
        got = p.run()
        status_ok()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        zero = torch.zeros(2, dtype=torch.int32, device=dev)
        k, v = fa.cache_read(kc, vc, p.table_d, zero, 200, None, ks, vs)
        for b in range(2):
            n = min(200, p.k[b].shape[1])
            assert np.array_equal(R.f64(k)[b, :, :n], R.quantise(R.f64(p.k[b]), fmt)[:, :n])
        del kc, vc, p
        torch.cuda.empty_cache()


def test_two_streams_at_once():
    """Different problems on two streams, their workspaces the wrapper's."""
    dev = device()
    ps = [Problem(f, 8, 8, 2, T, 128, 64, many(8, 1000, 5000, T), None, "tree", seed=T, dev=dev)
          for f, T in ((R.E4M3, 2), (R.BF16, 30))]
    want = [p.run() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = [[p.run(stream=s) for p, s in zip(ps, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    status_ok()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T,H", [(16, 8), (70, 8), (9, 2), (23, 6)])
def test_same_bits_every_time(T, H):
    """Long runs whose loads, conversions and products race each other: one
    result, over many calls with other work in between."""
    dev = device()
    noise = torch.empty(1 << 26, device=dev)
    for fmt in FORMATS:
        p = Problem(fmt, 2, H, 2, T, 128, 128, [40001, 23456], None, "tree", seed=T, dev=dev)
        want = p.run()
        p.check(*want)
        for k in range(60):
            if k % 3 == 0:
                noise.fill_(k)
            got = p.run()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (fmt, k)
        status_ok()
