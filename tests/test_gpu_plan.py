"""Page tables, slots and positions of serving steps against a plain
implementation, entry by entry; packed writes by slot; and all of a windowed
serving loop together."""
import numpy as np
import pytest

from gpu_common import device, status_ok, torch
import serving_ref as R
import window_ref

import io_aware_exact_15_gb300 as fa

pytestmark = pytest.mark.gpu


def plan(lens, counts, table, line, state, page, max_tokens, window, sinks):
    """The definition in include/fa.h, request by request; table, line and
    state are changed in place."""
    B, max_pages = table.shape
    num, cap = len(line), max_pages * page
    ok = lambda x: 0 <= x < num
    head, count = int(state[0]), int(state[1])
    lens = [min(max(int(n), 0), cap) for n in lens]
    for b in range(B):
        back = []
        if counts[b] < 0:
            back = [i for i in range(max_pages) if ok(table[b, i])]
        elif window:
            i = max(lens[b] - window + 1, 0) // page - 1
            while i >= -(-sinks // page) and ok(table[b, i]):
                back.insert(0, i)
                i -= 1
        for i in back:
            if count < num:
                line[(head + count) % num] = table[b, i]
                count += 1
        for i in range(max_pages) if counts[b] < 0 else back:
            table[b, i] = -1
    slots, positions = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int32)
    cu, granted, at = [], [], 0
    for b in range(B):
        n, dry = max(int(counts[b]), 0), None
        for i in range(lens[b] // page, max_pages):
            if n == 0 or i * page >= lens[b] + min(n, cap - lens[b]):
                break
            if ok(table[b, i]):
                continue
            if count == 0 or dry is not None:
                dry = i if dry is None else dry
                continue
            table[b, i] = line[head]
            head, count = (head + 1) % num, count - 1
        fit = min(n, cap - lens[b])
        if dry is not None:
            fit = min(fit, max(dry * page - lens[b], 0))
        fit = min(fit, max(max_tokens - at, 0))
        for t in range(min(n, max(max_tokens - at, 0))):
            pos = lens[b] + t
            positions[at + t] = pos
            if t < fit:
                slots[at + t] = int(table[b, pos // page]) * page + pos % page
        cu.append(min(at, max_tokens))
        granted.append(fit)
        at += n
    cu.append(min(at, max_tokens))
    state[:] = head, count
    return slots, positions, np.array(cu, np.int32), np.array(granted, np.int32)


class Pool:
    def __init__(self, B, max_pages, num, head, dev):
        self.table = np.full((B, max_pages), -1, np.int32)
        self.line = np.roll(np.arange(num, dtype=np.int32), head)
        self.state = np.array([head, num], np.int32)
        up = lambda x: torch.from_numpy(x).to(dev)
        self.dev, self.d = dev, [up(x.copy()) for x in (self.table, self.line, self.state)]

    def step(self, lens, counts, page, max_tokens, window, sinks):
        up = lambda x: torch.tensor([int(y) for y in x], dtype=torch.int32, device=self.dev)
        got = fa.cache_plan(up(lens), up(counts), *self.d, page, max_tokens, window or None, sinks)
        want = plan(lens, counts, self.table, self.line, self.state, page, max_tokens, window, sinks)
        status_ok()
        for name, a, b in zip(("slots", "positions", "cu_seqlens", "granted"), got, want):
            assert np.array_equal(a.cpu().numpy(), b), (name, np.argwhere(a.cpu().numpy() != b)[:3])
        for name, a, b in zip(("table", "line", "state"), self.d, (self.table, self.line, self.state)):
            assert np.array_equal(a.cpu().numpy(), b), (name, np.argwhere(a.cpu().numpy() != b)[:3])
        return got, want


CASES = [
    # B, page, max_pages, pages, window, sinks, largest prompt
    (1, 16, 4, 3, 0, 0, 40),
    (3, 16, 40, 60, 20, 4, 200),
    (5, 64, 10, 30, 64, 0, 300),
    (32, 32, 64, 200, 100, 33, 400),   # runs out of pages
    (33, 16, 300, 4000, 1, 1, 2000),   # long runs of pages go back
    (70, 128, 8, 300, 0, 0, 500),
    (300, 16, 30, 5000, 50, 16, 200),
    (1100, 64, 6, 3000, 128, 4, 100),
    (8192, 16, 3, 20000, 17, 0, 20),
]


@pytest.mark.parametrize("case", CASES)
def test_steps_of_a_server(case):
    """Prompts, single tokens, drafts of which some are taken back, pauses and
    ends, step after step on the same tables."""
    B, page, max_pages, num, window, sinks, prompt = case
    rng = np.random.default_rng(B)
    pool = Pool(B, max_pages, num, 5 % num, device())
    lens = np.zeros(B, np.int64)
    for step in range(8):
        kind = rng.random(B)
        counts = np.where(kind < 0.5, 1, np.where(kind < 0.75, rng.integers(1, 9, B),
                                                  rng.integers(0, prompt + 1, B)))
        if step == 0:
            counts = rng.integers(0, prompt + 1, B)
        counts = np.where(rng.random(B) < 0.1, 0, counts)
        if step > 1:
            counts = np.where(rng.random(B) < 0.1, -1 - rng.integers(0, 5, B), counts)
        listed = int(np.maximum(counts, 0).sum())
        _, want = pool.step(lens, counts, page, listed + int(rng.integers(0, 40)), window, sinks)
        lens = np.where(counts < 0, 0, lens + want[3])
        lens = np.maximum(lens - (rng.random(B) < 0.2) * rng.integers(0, 5, B), 0)  # rejected drafts
    held = pool.table[pool.table >= 0]
    assert len(set(held.tolist())) == len(held)  # no page twice
    head, count = pool.state
    free = [int(pool.line[(head + i) % num]) for i in range(count)]
    assert sorted(free + held.tolist()) == list(range(num))  # and none lost


def test_long_lists():
    """More tokens than the first kernel lists itself, some requests empty."""
    rng = np.random.default_rng(4)
    counts = rng.integers(0, 900, 200)
    counts[rng.random(200) < 0.3] = 0
    counts[:3] = 0
    lens = rng.integers(0, 300, 200)
    lens[7] = 1200 - 5  # its table ends
    pool = Pool(200, 75, 20000, 19990, device())
    pool.step(np.zeros(200), lens, 16, int(lens.sum()), 0, 0)
    pool.step(lens, counts, 16, int(counts.sum()) + 777, 0, 0)


@pytest.mark.parametrize("spare", [-1000, -1, 0, 8000, 20000])
def test_lists_that_are_too_short(spare):
    counts = [100, 0, 7000, 3, -1, 5000, 1]
    pool = Pool(7, 1000, 3000, 0, device())
    pool.step([0] * 7, counts, 16, max(0, 12104 + spare), 0, 0)


def test_no_tokens():
    pool = Pool(4, 8, 40, 3, device())
    pool.step([0] * 4, [100, 20, 0, 1], 16, 121, 0, 0)
    pool.step([100, 20, 0, 1], [-1, 0, 0, -1], 16, 0, 30, 0)


def test_entries_that_are_no_pages():
    """Numbers outside the pool in a row count as missing, lengths are clamped."""
    pool = Pool(5, 12, 100, 0, device())
    pool.step([0] * 5, [150] * 5, 16, 750, 0, 0)
    pool.table[0, 9], pool.table[1, 3], pool.table[2, 10] = 100, -5, 2 ** 31 - 1
    pool.d[0].copy_(torch.from_numpy(pool.table))
    pool.step([150, 150, 150, -7, 10 ** 9], [20, 20, 20, 3, 3], 16, 80, 40, 16)


def test_pages_that_went_back_are_taken_in_the_same_step():
    pool = Pool(2, 64, 20, 0, device())
    pool.step([0, 0], [300, 0], 16, 300, 0, 0)
    assert pool.state[1] == 1
    _, want = pool.step([300, 0], [1, 250], 16, 251, 32, 16)
    assert want[3].tolist() == [1, 250]


def test_a_ring_that_would_overflow():
    """A page that two rows hold breaks the rules: the line keeps its size."""
    pool = Pool(2, 4, 6, 0, device())
    pool.table[:] = [[0, 1, 2, 3], [0, 1, 2, 3]]
    pool.d[0].copy_(torch.from_numpy(pool.table))
    pool.step([64, 64], [-1, -1], 16, 0, 0, 0)
    assert pool.state[1] == 6


def test_streams_and_a_graph():
    """Two pools on two streams, and a captured step replayed."""
    dev = device()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    lens, counts = i32(100, 31, 0), i32(1, 2, 40)
    def pool():
        return (torch.full((3, 20), -1, dtype=torch.int32, device=dev),
                torch.arange(50, dtype=torch.int32, device=dev), i32(0, 50))
    ref = pool()
    want = fa.cache_plan(lens, counts, *ref, 16, 60, 64, 4)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        pools = [pool() for _ in streams]
        torch.cuda.synchronize()
        outs = [fa.cache_plan(lens, counts, *p, 16, 60, 64, 4, stream=s)
                for p, s in zip(pools, streams)]
        torch.cuda.synchronize()
        for p, o in zip(pools, outs):
            assert all(torch.equal(a, b) for a, b in zip(o + p, want + ref))
    p = pool()
    keep = [t.clone() for t in p]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = fa.cache_plan(lens, counts, *p, 16, 60, 64, 4)
    for _ in range(2):
        for t, k in zip(p, keep):
            t.copy_(k)
        graph.replay()
        status_ok()
        assert all(torch.equal(a, b) for a, b in zip(out + p, want + ref))


# ------------------------------------------------------------------ writes by slot
@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.INT8])
@pytest.mark.parametrize("N,Hkv,d,page", [(1, 1, 64, 16), (5, 4, 128, 64), (8, 2, 64, 32), (33, 3, 128, 16),
                                          (300, 2, 64, 128), (1001, 1, 128, 32),
                                          (9001, 4, 64, 64), (5003, 4, 128, 16)])
def test_slots(N, Hkv, d, page, fmt):
    """As if each token had been appended by table and position; skipped tokens
    and all other rows left as they were."""
    dev = device()
    rng = np.random.default_rng(N)
    g = torch.Generator().manual_seed(N)
    num = -(-N // page) + 3
    kv = (torch.randn(N, 2 * Hkv, d, generator=g) * 3).bfloat16().to(dev)
    k, v = kv[:, :Hkv].transpose(0, 1), kv[:, Hkv:].transpose(0, 1)
    slots = rng.permutation(num * page)[:N].astype(np.int64)
    skip = rng.random(N) < 0.2
    slots[skip] = rng.choice([-1, -page, num * page, 2 ** 40, -2 ** 63], skip.sum())
    kind = R.DTYPES[fmt]
    new = lambda: torch.full((num, Hkv, page, d), 7, dtype=torch.uint8, device=dev).to(kind)
    sc = lambda: torch.full((num, Hkv, page), 9, dtype=torch.uint8, device=dev)
    a, b = [new(), new(), sc(), sc()], [new(), new(), sc(), sc()]
    fa.cache_append_slots(k, v, a[0], a[1], torch.from_numpy(slots).to(dev), a[2], a[3])
    # one token to a "sequence" whose table is the page itself
    good = np.nonzero(~skip)[0]
    if len(good):
        pick = torch.from_numpy(good).to(dev)
        i32 = lambda x: torch.from_numpy(x.astype(np.int32)).to(dev)
        fa.cache_append(kv[pick][:, :Hkv, None].contiguous(), kv[pick][:, Hkv:, None].contiguous(),
                        b[0], b[1], i32(slots[good] // page)[:, None].contiguous(),
                        i32(slots[good] % page), None, b[2], b[3])
    status_ok()
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_slots_far_into_a_large_pool():
    """Rows whose offsets pass 32 bits."""
    dev = device()
    Hkv, d, page = 2, 128, 128
    num = (1 << 32) // (Hkv * d * page) + 10  # elements pass 2^32
    kc = torch.zeros(num, Hkv, page, d, dtype=torch.bfloat16, device=dev)
    vc = torch.zeros_like(kc)
    k = torch.randn(Hkv, 3, d, device=dev).bfloat16()
    slots = torch.tensor([num * page - 1, 0, (num - 5) * page + 3], device=dev)
    fa.cache_append_slots(k, k, kc, vc, slots)
    status_ok()
    for n, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // page, :, s % page], k[:, n])
        assert torch.equal(vc[s // page, :, s % page], k[:, n])
    assert int((kc != 0).any(-1).sum()) == 3 * Hkv


def test_no_slots():
    dev = device()
    kc = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device=dev)
    k = torch.zeros(1, 0, 64, dtype=torch.bfloat16, device=dev)
    fa.cache_append_slots(k, k, kc, kc.clone(), torch.zeros(0, dtype=torch.int64, device=dev))


# ------------------------------------------------------------------ all of it together
@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3])
def test_a_windowed_server(fmt):
    """Prompts by the packed windowed forward, then tokens over the cache, with
    a pool far too small for the histories: every token's output is that of
    the whole sequence's windowed attention."""
    dev = device()
    B, H, Hkv, d, page, window, sinks = 3, 4, 2, 64, 16, 40, 4
    scale = d ** -0.5
    prompts, steps = [70, 1, 33], 60
    g = torch.Generator().manual_seed(6)
    n = [p + steps for p in prompts]
    qkv = [torch.randn(m, H + 2 * Hkv, d, generator=g).bfloat16() for m in n]
    table = torch.full((B, -(-max(n) // page)), -1, dtype=torch.int32, device=dev)
    num = 24  # the windows' pages, the first tokens' and a prompt's
    line, state = torch.arange(num, dtype=torch.int32, device=dev), \
        torch.tensor([0, num], dtype=torch.int32, device=dev)
    kind = R.DTYPES[fmt]
    cache = [torch.zeros(num, Hkv, page, d, dtype=torch.uint8, device=dev).to(kind) for _ in range(2)]
    scales = [torch.full((num, Hkv, page), 127, dtype=torch.uint8, device=dev) for _ in range(2)]
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    outs = [[] for _ in range(B)]
    for step in range(1 + steps):
        at = [0 if step == 0 else p + step - 1 for p in prompts]
        new = prompts if step == 0 else [1] * B
        counts = torch.tensor(new, dtype=torch.int32, device=dev)
        slots, pos, cu, granted = fa.cache_plan(lens, counts, table, line, state, page, sum(new) + 2,
                                                window, sinks)
        x = torch.cat([t[a:a + m] for t, a, m in zip(qkv, at, new)] +
                      [torch.full((2, H + 2 * Hkv, d), float("nan")).bfloat16()]).to(dev)
        q, k, v = (y.transpose(0, 1) for y in x.split([H, Hkv, Hkv], 1))
        fa.cache_append_slots(k, v, *cache, slots, *scales)
        if step == 0:
            # the prompt sees what the cache will hold: it is read back
            m = max(prompts)
            kb, vb = fa.cache_read(*cache, table, lens, m, counts, *scales)
            pack = lambda y: torch.cat([y[b, :, :prompts[b]] for b in range(B)] +
                                       [torch.full_like(y[0, :, :2], float("nan"))], 1)
            o, _ = fa.attention_forward(q.contiguous(), pack(kb), pack(vb), causal=True,
                                        cu_seqlens=cu, max_seqlen=m, window=window, sinks=sinks)
            for b in range(B):
                outs[b].append(o[:, int(cu[b]):int(cu[b + 1])].cpu().double())
        else:
            o, _ = fa.tree_attention(q[:, :B].transpose(0, 1)[:, :, None].contiguous(), *cache, table,
                                     lens, None, None, None, *scales, window=window, sinks=sinks)
            for b in range(B):
                outs[b].append(o[b].cpu().double())
        assert torch.equal(granted, counts)
        assert pos[:sum(new)].tolist() == [a + i for a, m in zip(at, new) for i in range(m)]
        lens += granted
    status_ok()
    assert int((table[0] >= 0).sum()) < table.shape[1]  # pages did go back
    for b in range(B):
        q, k, v = (y.double().transpose(0, 1) for y in qkv[b].split([H, Hkv, Hkv], 1))
        k, v = (torch.from_numpy(R.quantise(y.numpy(), fmt)) for y in (k, v))
        ro, _, to, _ = window_ref.forward(q, k, v, window, sinks, scale)
        got = torch.cat(outs[b], 1)
        # 8 bits: f16 weights add at most 2^-31 of the largest value per key
        more = 0 if fmt == R.BF16 else n[b] * 2.0 ** -31 * float(v.abs().max())
        assert bool(((got - ro).abs() <= to + more).all())


def test_long_lists_of_single_tokens():
    """Many requests to a warp's stretch of the list, runs of empty ones."""
    rng = np.random.default_rng(8)
    counts = (rng.random(8192) < 0.9).astype(np.int64) * rng.integers(1, 4, 8192)
    counts[1000:1700] = 0
    lens = rng.integers(0, 40, 8192)
    pool = Pool(8192, 4, 33000, 0, device())
    pool.step(np.zeros(8192), lens, 16, int(lens.sum()), 0, 0)
    pool.step(lens, counts, 16, int(counts.sum()), 0, 0)
