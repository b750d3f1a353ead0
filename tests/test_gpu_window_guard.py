"""Windowed attention, its cached form, plans and slot writes between
sentinel margins: nothing outside their outputs and workspaces is written, and
inputs stay as they are."""
import pytest

from gpu_common import device, torch
from test_gpu_guard_bands import Guarded, _inputs, _unchanged

import fa_workloads as W
import io_aware_exact_15_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,window,sinks", [(1, 1, 0), (7, 3, 1), (129, 20, 4), (255, 300, 130),
                                            (1281, 100, 4)])
def test_window(N, window, sinks, d):
    dev = device()
    B, H, Hkv = 2, 4, 2
    scale = 1.0 / d ** 0.5
    q, k, v, do = _inputs((B, H, N, d), dev, 60 + N + d)
    k, v = k[:, :Hkv].contiguous(), v[:, :Hkv].contiguous()
    copies = [t.clone() for t in (q, k, v, do)]
    g = Guarded(dev)
    o, lse = g.tensor((B, H, N, d), torch.bfloat16, "O"), g.tensor((B, H, N), torch.float32, "lse")
    dq = g.tensor((B, H, N, d), torch.bfloat16, "dQ")
    dk, dv = (g.tensor((B, Hkv, N, d), torch.bfloat16, n) for n in ("dK", "dV"))
    size = (B, H, Hkv, N, 0, d)
    nb = fa.fa_backward_window_workspace_size(*size, window, sinks)
    ws = g.workspace(nb)
    assert fa.fa_forward_window(q, k, v, o, lse, None, *size, scale, window, sinks) == fa.FA_OK
    g.check("forward")
    assert fa.fa_backward_window(q, k, v, o, do, lse, dq, dk, dv, None, *size, scale, window, sinks,
                                 ws, nb) == fa.FA_OK
    g.check("backward")
    _unchanged((q, k, v, do), copies, "window")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [(1, 0, 7), (129, 255, 3), (255,), (1300, 0, 131)])
def test_packed_window(lengths, d):
    dev = device()
    H, Hkv, window, sinks = 4, 2, 60, 4
    scale = 1.0 / d ** 0.5
    cu = W.cu_seqlens(lengths)
    T, B, L = int(cu[-1]), len(lengths), max(lengths)
    g0 = torch.Generator().manual_seed(8 + T + d)
    q, do = (W.randn_bf16((H, T, d), g0).to(dev) for _ in range(2))
    k, v = (W.randn_bf16((Hkv, T, d), g0).to(dev) for _ in range(2))
    copies = [t.clone() for t in (q, k, v, do)]
    g = Guarded(dev)
    cud = g.tensor((B + 1,), torch.int32, "cu_seqlens")
    cud.copy_(torch.from_numpy(cu))
    o, lse = g.tensor((H, T, d), torch.bfloat16, "O"), g.tensor((H, T), torch.float32, "lse")
    dq = g.tensor((H, T, d), torch.bfloat16, "dQ")
    dk, dv = (g.tensor((Hkv, T, d), torch.bfloat16, n) for n in ("dK", "dV"))
    size = (B, H, Hkv, L, T, d)
    nb = fa.fa_backward_window_workspace_size(*size, window, sinks)
    ws = g.workspace(nb)
    assert fa.fa_forward_window(q, k, v, o, lse, cud, *size, scale, window, sinks) == fa.FA_OK
    g.check("forward")
    assert fa.fa_backward_window(q, k, v, o, do, lse, dq, dk, dv, cud, *size, scale, window, sinks,
                                 ws, nb) == fa.FA_OK
    g.check("backward")
    # offsets that break the rules: unspecified values, nothing outside
    for bad in ([5, 2, T + 900, -3], [T, T, 0, T], [0, T, T, 2 ** 31 - 1]):
        cud.copy_(torch.tensor((bad * B)[:B + 1], dtype=torch.int32))
        assert fa.fa_forward_window(q, k, v, o, lse, cud, *size, scale, window, sinks) == fa.FA_OK
        assert fa.fa_backward_window(q, k, v, o, do, lse, dq, dk, dv, cud, *size, scale, window,
                                     sinks, ws, nb) == fa.FA_OK
        g.check(f"offsets {bad}")
    _unchanged((q, k, v, do), copies, "packed window")


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("T,d,H,Hkv", [(1, 128, 4, 2), (5, 64, 6, 1), (40, 128, 4, 1), (70, 64, 8, 2)])
def test_cached_window(T, d, H, Hkv, fmt):
    """Also with lengths and page ids that break the rules."""
    dev = device()
    B, page, most, num = 3, 32, 20, 40
    kind = (torch.bfloat16, torch.float8_e4m3fn, torch.int8)[fmt]
    q = W.randn_bf16((B, H, T, d), torch.Generator().manual_seed(T)).to(dev)
    kc, vc = (torch.zeros(num, Hkv, page, d, dtype=torch.uint8, device=dev).to(kind) for _ in range(2))
    ks, vs = (torch.full((num, Hkv, page), 127, dtype=torch.uint8, device=dev) for _ in range(2))
    g = Guarded(dev)
    o, lse = g.tensor((B, H, T, d), torch.bfloat16, "O"), g.tensor((B, H, T), torch.float32, "lse")
    nb = fa.fa_tree_attention_workspace_size(B, H, Hkv, T, d)
    ws = g.workspace(nb)
    table = torch.randint(0, num, (B, most), dtype=torch.int32, device=dev)
    table[1, 3], table[2, 5] = 2 ** 31 - 1, -2 ** 31
    for hist in ([500, 0, 77], [640, 639, 10 ** 9], [-5, -2 ** 31, 600]):
        for window, sinks in ((1, 0), (64, 40), (2 ** 31 - 1, 1024)):
            h = torch.tensor(hist, dtype=torch.int32, device=dev)
            assert fa.fa_tree_attention_window(q, kc, vc, ks, vs, table, h, None, None, o, lse, fmt, B,
                                               H, Hkv, T, d, num, page, most, 0.1, window, sinks, ws,
                                               nb) == fa.FA_OK
            g.check(f"hist {hist} window {window}")


def test_plan_and_slots():
    dev = device()
    B, page, most, num, tokens = 37, 16, 9, 150, 300
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    gen = torch.Generator().manual_seed(3)
    for state in ([0, num], [149, 60], [-7, 10 ** 9], [2 ** 31 - 1, -4]):
        g = Guarded(dev)
        table = g.tensor((B, most), torch.int32, "table")
        line, st = g.tensor((num,), torch.int32, "line"), g.tensor((2,), torch.int32, "state")
        slots, pos = g.tensor((tokens,), torch.int64, "slots"), g.tensor((tokens,), torch.int32, "pos")
        cu, granted = g.tensor((B + 1,), torch.int32, "cu"), g.tensor((B,), torch.int32, "granted")
        table.copy_(torch.randint(-3, num + 3, (B, most), generator=gen).int())
        line.copy_(torch.randint(-9, num + 9, (num,), generator=gen).int())
        st.copy_(i32(state))
        lens = torch.randint(-5, most * page + 5, (B,), generator=gen).int().to(dev)
        counts = torch.randint(-2, 40, (B,), generator=gen).int().to(dev)
        counts[5] = 2 ** 31 - 1
        for window in (0, 1, 50):
            assert fa.fa_cache_plan(lens, counts, table, line, st, slots, pos, cu, granted, B, tokens,
                                    num, page, most, window, 20) == fa.FA_OK
            g.check(f"plan {state} {window}")
        kc, vc = (g.tensor((num, 2, page, 64), torch.int8, n) for n in ("K", "V"))
        ks, vs = (g.tensor((num, 2, page), torch.uint8, n) for n in ("ks", "vs"))
        k = W.randn_bf16((2, tokens, 64), gen).to(dev)
        assert fa.fa_cache_append_slots(k, k, slots, kc, vc, ks, vs, 2, 2, tokens, 64, num,
                                        page) == fa.FA_OK
        g.check("slots")
