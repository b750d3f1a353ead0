"""The paged cache: what is written reads back as the formats' definition
says, bit by bit; skipped tokens, bad tables and neighbours stay untouched."""
import numpy as np
import pytest

from gpu_common import device, status_ok, torch
import serving_ref as R

import io_aware_exact_15_gb300 as fa

pytestmark = pytest.mark.gpu

FORMATS = [R.BF16, R.E4M3, R.INT8]


def empty_cache(num, Hkv, page, d, fmt, dev, fill=0xA5):
    kind = R.DTYPES[fmt]
    size = 2 if fmt == R.BF16 else 1
    c = [torch.full((num, Hkv, page, d * size), fill, dtype=torch.uint8, device=dev).view(kind)
         for _ in range(2)]
    s = [torch.full((num, Hkv, page), fill, dtype=torch.uint8, device=dev) for _ in range(2)]
    return c[0], c[1], s[0], s[1]


def rows(B, Hkv, N, d, seed):
    """Rows over the whole range of sizes: from 2^-100 to 2^100, one row of
    zeros, one of equal values, one just at a format's limit."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, Hkv, N, d, generator=g)
    x = x * torch.exp2(torch.randint(-100, 100, (B, Hkv, N, 1), generator=g).float())
    x = x.bfloat16()
    x[0, 0, 0] = 0
    if N > 5:
        x[0, 0, 1] = 448.0  # e4m3's and int8's largest: the exponent steps here
        x[0, 0, 2] = 127.0
        x[0, 0, 3] = torch.tensor(127.5)
        x[0, 0, 4] = 2.0 ** -130  # below the smallest scale
        x[0, 0, 5, 0] = 3.38e38  # close to bf16's largest
    return x


def host_bytes(t):
    return t.contiguous().view(torch.uint8).cpu()


CASES = [  # B, Hkv, N, d, page, starts, counts
    (1, 1, 1, 64, 16, [0], None),
    (3, 2, 1, 128, 64, [5, 63, 64], [1, 0, 1]),
    (2, 3, 7, 64, 32, [30, 0], [7, 3]),
    (3, 4, 70, 128, 16, [0, 13, 127], [70, 33, 1]),
    (2, 5, 300, 64, 128, [100, 1], None),
    (4, 1, 129, 128, 128, [0, 127, 128, 5], [129, 128, 0, 2]),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])))
def test_written_and_read_back(case, fmt):
    dev = device()
    B, Hkv, N, d, page, starts, counts = case
    rng = np.random.default_rng(sum(case[:5]))
    n = counts or [N] * B
    table, num = R.page_table(rng, [s + c for s, c in zip(starts, n)], page)
    kc, vc, ks, vs = empty_cache(num, Hkv, page, d, fmt, dev)
    before = [host_bytes(t) for t in (kc, vc, ks, vs)]
    k, v = rows(B, Hkv, N, d, 1).to(dev), rows(B, Hkv, N, d, 2).to(dev)
    start = torch.tensor(starts, dtype=torch.int32, device=dev)
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=dev)
    table_d = table.to(dev)
    fa.cache_append(k, v, kc, vc, table_d, start, cnt, ks, vs)
    back = fa.cache_read(kc, vc, table_d, start, N, cnt, ks, vs)
    status_ok()
    for x, y in zip((k, v), back):
        want = R.quantise(R.f64(x), fmt)
        got = R.f64(y)
        for b in range(B):
            assert np.array_equal(got[b, :, :n[b]], want[b, :, :n[b]])  # exact, no tolerance
            assert (got[b, :, n[b]:] == 0).all()
    # bytes that belong to no written token are as they were
    own = torch.zeros(num, Hkv, page, dtype=torch.bool)
    for b in range(B):
        R.place(own, table, b, starts[b], torch.ones(Hkv, n[b], dtype=torch.bool))
    for t, was in zip((kc, vc), before[:2]):
        now = host_bytes(t).reshape(num, Hkv, page, -1)
        assert torch.equal(now[~own], was.reshape(now.shape)[~own])
    for t, was in zip((ks, vs), before[2:]):
        keep = ~own if fmt != R.BF16 else torch.ones_like(own)
        assert torch.equal(host_bytes(t)[keep], was[keep])
    # appending what was read back changes no value
    again = empty_cache(num, Hkv, page, d, fmt, dev, fill=0)
    fa.cache_append(*back, again[0], again[1], table_d, start, cnt, again[2], again[3])
    twice = fa.cache_read(again[0], again[1], table_d, start, N, cnt, again[2], again[3])
    assert all(torch.equal(a, b) for a, b in zip(back, twice))


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_every_stored_number_reads_back(fmt):
    """All 256 codes but e4m3's NaN, under every scale byte that is written
    and the NaN scale."""
    dev = device()
    codes = np.arange(256, dtype=np.uint8)
    if fmt == R.E4M3:
        codes[[0x7F, 0xFF]] = 0
    d, page = 64, 16
    num = 64  # 64 pages x 16 rows = 256 scale bytes x 4 rows of codes
    kc, vc, ks, vs = empty_cache(num, 1, page, d, fmt, dev)
    kc.view(torch.uint8).copy_(torch.from_numpy(np.tile(codes, num * page * d // 256)).view(
        num, 1, page, d))
    ks.copy_(torch.arange(256, dtype=torch.uint8).repeat_interleave(4).view(num, 1, page))
    vc.copy_(kc)
    vs.copy_(ks)
    table = torch.arange(num, dtype=torch.int32, device=dev)[None]
    k, v = fa.cache_read(kc, vc, table, torch.zeros(1, dtype=torch.int32, device=dev), num * page,
                         None, ks, vs)
    status_ok()
    if fmt == R.INT8:
        value = codes.view(np.int8).astype(np.float64)
    else:
        value = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    value = np.tile(value, num * page * d // 256).reshape(num * page, d)
    byte = np.arange(256).repeat(4)
    want = value * 2.0 ** (byte.astype(np.float64) - 127)[:, None]
    got = R.f64(k)[0, 0]
    fine = (byte >= 27) & (byte <= 246)
    assert np.array_equal(got[fine], want[fine])
    assert np.isnan(got[byte == 255]).all()
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_rows_with_nan_or_infinity(fmt):
    dev = device()
    x = torch.ones(1, 1, 8, 64, dtype=torch.bfloat16)
    x[0, 0, 2, 63] = float("nan")
    x[0, 0, 3, 0] = float("inf")
    x[0, 0, 4, 9] = -float("inf")
    x = x.to(dev)
    kc, vc, ks, vs = empty_cache(1, 1, 16, 64, fmt, dev)
    table = torch.zeros(1, 1, dtype=torch.int32, device=dev)
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    fa.cache_append(x, x, kc, vc, table, zero, None, ks, vs)
    k, v = fa.cache_read(kc, vc, table, zero, 8, None, ks, vs)
    status_ok()
    for y in (k, v):
        bad = torch.isnan(y[0, 0]).cpu()
        assert bad[2:5].all() and not bad[:2].any() and not bad[5:].any()
        assert (y[0, 0, [0, 1, 5, 6, 7]] == 1).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_positions_and_pages_are_skipped(fmt):
    """Positions in front of 0 or behind the table, page ids outside the
    pool: nothing is written, zeros are read."""
    dev = device()
    Hkv, page, d, num = 2, 16, 64, 4
    kc, vc, ks, vs = empty_cache(num, Hkv, page, d, fmt, dev)
    before = [host_bytes(t) for t in (kc, vc, ks, vs)]
    table = torch.tensor([[0, 9], [-1, -7], [1, 2]], dtype=torch.int32, device=dev)
    start = torch.tensor([16, 0, 30], dtype=torch.int32, device=dev)
    x = torch.ones(3, Hkv, 6, d, dtype=torch.bfloat16, device=dev)
    fa.cache_append(x, x, kc, vc, table, start, None, ks, vs)
    k, v = fa.cache_read(kc, vc, table, start, 6, None, ks, vs)
    status_ok()
    assert (k[:2] == 0).all() and (k[2, :, :2] == 1).all() and (k[2, :, 2:] == 0).all()
    own = torch.zeros(num, Hkv, page, dtype=torch.bool)
    own[2, :, 14:] = True
    for t, was in zip((kc, vc), before[:2]):
        now = host_bytes(t).reshape(num, Hkv, page, -1)
        assert torch.equal(now[~own], was.reshape(now.shape)[~own])
    for bad_start in ([-3, 0, 0], [2 ** 31 - 1, 0, 0]):
        start = torch.tensor(bad_start, dtype=torch.int32, device=dev)
        count = torch.tensor([6, 0, -5], dtype=torch.int32, device=dev)
        now = [host_bytes(t) for t in (kc, vc, ks, vs)]
        fa.cache_append(2 * x, x, kc, vc, table, start, count, ks, vs)
        status_ok()
        assert all(torch.equal(a, host_bytes(b)) for a, b in zip(now, (kc, vc, ks, vs)))


def test_strided_rows():
    dev = device()
    B, Hkv, N, d, page = 2, 3, 21, 128, 32
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn(B, N, 4 + 2 * Hkv, d, generator=g).bfloat16().to(dev)
    k, v = qkv[:, :, 4:4 + Hkv].transpose(1, 2), qkv[:, :, 4 + Hkv:].transpose(1, 2)
    table = torch.arange(2 * B, dtype=torch.int32, device=dev).view(B, 2)
    start = torch.zeros(B, dtype=torch.int32, device=dev)
    out = []
    for a, b in ((k, v), (k.contiguous(), v.contiguous())):
        kc, vc, ks, vs = empty_cache(2 * B, Hkv, page, d, R.E4M3, dev)
        fa.cache_append(a, b, kc, vc, table, start, None, ks, vs)
        out.append([host_bytes(t) for t in (kc, vc, ks, vs)])
    status_ok()
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_largest_numbers_saturate(fmt):
    """bf16's largest number, of either sign, among others: the largest
    stored number at the largest scale, and finite."""
    dev = device()
    big = 2.0 ** 128 - 2.0 ** 120
    x = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    x[..., 0], x[..., 1], x[..., 2], x[..., 3] = big, -big, big / 2, 2.0 ** 121
    x = x.to(dev)
    kc, vc, ks, vs = empty_cache(1, 1, 16, 64, fmt, dev)
    table = torch.zeros(1, 1, dtype=torch.int32, device=dev)
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    for n in (1, 16):
        fa.cache_append(x[:, :, :n], x[:, :, :n], kc, vc, table, zero, None, ks, vs)
    y, _ = fa.cache_read(kc, vc, table, zero, 16, None, ks, vs)
    status_ok()
    most = 127 * 2.0 ** 121 if fmt == R.INT8 else 448 * 2.0 ** 119
    # half of it: 63.75 steps of 2^121, or 255 of 2^119 in steps of 16
    half = 64 * 2.0 ** 121 if fmt == R.INT8 else 256 * 2.0 ** 119
    want = torch.tensor([most, -most, half, 2.0 ** 121] + [0.0] * 60, dtype=torch.float64)
    assert torch.equal(y[0, 0].double().cpu(), want.expand(16, 64))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", FORMATS)
def test_row_counts_next_to_the_largest(fmt, d):
    """N = 2^31 - 2 for one head (the largest that is accepted), its rows one
    row of memory: the tokens that exist are written, up to the table's end,
    and nothing else."""
    dev = device()
    N, page, num = 2 ** 31 - 2, 16, 6
    g = torch.Generator().manual_seed(d)
    k, v = (torch.randn(1, 1, 1, d, generator=g).bfloat16() for _ in range(2))
    kd, vd = (t.to(dev).expand(1, 1, N, d) for t in (k, v))
    table = torch.tensor([[4, 2, 0, 5]], dtype=torch.int32, device=dev)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    for start, count, most in ((5, 41, 46), (3, None, 64), (0, 0, 0), (50, N, 64)):
        kc, vc, ks, vs = empty_cache(num, 1, page, d, fmt, dev)
        before = [host_bytes(t) for t in (kc, vc, ks, vs)]
        fa.cache_append(kd, vd, kc, vc, table, i32(start), None if count is None else i32(count),
                        ks, vs)
        back = fa.cache_read(kc, vc, table, i32(start), 70, i32(max(most - start, 0)), ks, vs)
        status_ok()
        for x, y in zip((k, v), back):
            want = R.quantise(R.f64(x), fmt)[0, 0, 0]
            n = max(most - start, 0)
            assert np.array_equal(R.f64(y)[0, 0, :n], np.tile(want, (n, 1)))
        own = torch.zeros(num, 1, page, dtype=torch.bool)
        R.place(own, table.cpu(), 0, start, torch.ones(1, max(most - start, 0), dtype=torch.bool))
        for t, was in zip((kc, vc), before[:2]):
            now = host_bytes(t).reshape(num, 1, page, -1)
            assert torch.equal(now[~own], was.reshape(now.shape)[~own])
