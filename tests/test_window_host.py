"""Refusals of the window, plan and slot entry points (no GPU: every case
returns before the first CUDA call), and the 64-bit formulas that the GPU
tests use against differences."""
import pytest
import torch

import io_aware_exact_15_gb300 as fa
import window_ref as R

A = 1 << 20      # fake device pointers, never dereferenced
MIS = A + 8
BAD, UNSUP, ALIGN, WS = (fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_MISALIGNED,
                         fa.FA_ERR_WORKSPACE)


def forward(B=2, H=4, Hkv=2, N=300, total=0, d=64, scale=0.1, window=50, sinks=4, cu=None,
            ptrs=(A,) * 5):
    return fa.fa_forward_window(*ptrs, cu, B, H, Hkv, N, total, d, scale, window, sinks, 0)


def backward(B=2, H=4, Hkv=2, N=300, total=0, d=64, scale=0.1, window=50, sinks=4, cu=None,
             ptrs=(A,) * 9, ws=A, size=None):
    if size is None:
        size = 1 << 40
    return fa.fa_backward_window(*ptrs, cu, B, H, Hkv, N, total, d, scale, window, sinks, ws, size, 0)


SIZES = [
    (dict(B=0), BAD), (dict(H=0), BAD), (dict(N=0), BAD), (dict(Hkv=0), BAD), (dict(Hkv=3), BAD),
    (dict(Hkv=8), BAD), (dict(scale=0.0), BAD), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD), (dict(window=0), BAD), (dict(window=-1), BAD),
    (dict(sinks=-1), BAD), (dict(sinks=1025), UNSUP), (dict(d=32), UNSUP), (dict(total=-1), BAD),
    (dict(total=300), BAD),  # a total without offsets
    (dict(N=1 << 30), UNSUP), (dict(B=1 << 20, H=1 << 20, Hkv=1 << 20), UNSUP),
    (dict(B=1 << 30, H=1 << 30, Hkv=1, N=1 << 30), UNSUP),
    (dict(B=1 << 21, H=4, N=1), UNSUP),  # tiles
    (dict(cu=A, total=100), BAD),    # the longest is longer than all rows
    (dict(cu=A, total=300, N=0), BAD), (dict(cu=A + 2, total=300), ALIGN),
    (dict(cu=A, total=1 << 24, H=64), UNSUP),
]


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("kw,want", SIZES)
def test_window_refuses_sizes(call, kw, want):
    assert call(**kw) == want
    if want in (BAD, UNSUP):
        args = dict(B=2, H=4, Hkv=2, N=300, total=0, d=64, window=50, sinks=4)
        args.update({k: v for k, v in kw.items() if k in args})
        if not set(kw) & {"scale", "cu"} and kw != dict(total=300):
            assert fa.fa_backward_window_workspace_size(*args.values()) == 0


@pytest.mark.parametrize("call,n", [(forward, 5), (backward, 9)])
def test_window_refuses_pointers(call, n):
    lse = 4 if call is forward else 5
    for i in range(n):
        assert call(ptrs=tuple(None if j == i else A for j in range(n))) == BAD
        off = A + 2 if i == lse else MIS
        assert call(ptrs=tuple(off if j == i else A for j in range(n))) == ALIGN


def test_window_refuses_workspaces():
    n = fa.fa_backward_window_workspace_size(2, 4, 2, 300, 0, 64, 50, 4)
    assert backward(size=n - 1) == WS and backward(ws=None) == BAD and backward(ws=A + 16) == ALIGN
    # packed and with parts of the first tiles' walks
    n = fa.fa_backward_window_workspace_size(3, 4, 2, 4000, 9000, 128, 50, 4)
    parts = 3 * 2 * 1 * 4 * 2 * 128 * 128 * 4  # (sequences, heads, tiles, parts) x dV, dK
    assert n >= 4 * 9000 * (4 + 4 * 128) + parts
    assert backward(B=3, N=4000, total=9000, d=128, cu=A, size=n - 1) == WS


def test_a_packed_batch_takes_what_its_rows_take():
    """1023 short sequences and one of 32768 rows: D and the accumulator (516
    bytes a row), and not a slot for every part that a sequence might have."""
    total = 1023 * 20 + 32768
    n = fa.fa_backward_window_workspace_size(1024, 8, 8, 32768, total, 128, 512, 4)
    assert 516 * 8 * total <= n < 2 * 516 * 8 * total
    assert backward(B=1024, H=8, Hkv=8, N=32768, total=total, d=128, window=512, cu=A, size=n - 1) == WS


def test_empty_packed_batch():
    """Nothing to do and nothing to point to."""
    assert forward(cu=A, total=0, N=0, ptrs=(None,) * 5) == fa.FA_OK
    assert backward(cu=A, total=0, N=0, ptrs=(None,) * 9, ws=None, size=0) == fa.FA_OK


def test_python_refusals():
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    for kw in (dict(causal=False), dict(causal=True, dropout_p=0.1),
               dict(causal=True, block_mask=torch.ones(1, 1, 1, dtype=torch.uint8)),
               dict(causal=True)):  # the last: tensors on the CPU
        with pytest.raises(ValueError):
            fa.attention_forward(q, q, q, window=4, **kw)
        with pytest.raises(ValueError):
            fa.attention_backward(q, q, q, q, q, torch.zeros(1, 2, 8), window=4, **kw)
    with pytest.raises(ValueError):
        fa.attention_forward(q, q, q, causal=True, sinks=4)


def test_numbers_past_32_bits():
    """A C int would take 2^32 + 1 for 1, another window."""
    assert fa._int32(2**32 + 1) == fa._int32(2**31) == fa._int32(2**31 - 1) == 2**31 - 1
    assert fa._int32(-2**32 + 1) == fa._int32(-1) == -1 and fa._int32(0) == 0
    # the longest window there is, and more first tokens than there may be
    assert fa.fa_backward_window_workspace_size(2, 4, 2, 300, 0, 64, fa._int32(2**40), 4) > 0
    assert forward(sinks=fa._int32(2**32 + 1)) == UNSUP and forward(window=fa._int32(-2**40)) == BAD


def test_gradient_formula_against_differences():
    x = R.Batch([40], 4, 2, 64, False, 2)
    q, k, v, g = (x.seq(t, 0) for t in (x.q, x.k, x.v, x.g))
    o, lse, _, _ = R.forward(q, k, v, 9, 3, 0.125)
    grads, _ = R.backward(q, k, v, o, lse, g, 9, 3, 0.125)
    gen = torch.Generator().manual_seed(3)
    args = [q, k, v]
    for i in range(3):
        u = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        f = lambda e: float((R.forward(*(args[:i] + [args[i] + e * u] + args[i + 1:]), 9, 3,
                                       0.125)[0] * g).sum())
        h = 1e-5
        # central differences of a smooth function: h^2, and rounding over h
        assert abs((f(h) - f(-h)) / (2 * h) - float((grads[i] * u).sum())) < 1e-6


def cached(B=2, H=4, Hkv=2, T=3, d=64, fmt=0, num=8, page=16, most=4, scale=0.1, window=50, sinks=4,
           mask=A, ptrs=(A,) * 10, ws=A, size=1 << 40):
    """q, the caches, their scales, table, lengths, drafts, o, lse."""
    return fa.fa_tree_attention_window(*ptrs[:8], mask, *ptrs[8:], fmt, B, H, Hkv, T, d, num, page,
                                       most, scale, window, sinks, ws, size, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(window=0), BAD), (dict(window=-5), BAD), (dict(sinks=-1), BAD), (dict(sinks=1025), UNSUP),
    (dict(T=51), UNSUP), (dict(window=2), UNSUP),  # a tree longer than the window
    (dict(B=0), BAD), (dict(Hkv=3), BAD), (dict(scale=0.0), BAD), (dict(d=32), UNSUP),
    (dict(page=8), UNSUP), (dict(T=1025, mask=None), UNSUP), (dict(size=100), WS), (dict(ws=None), BAD),
    (dict(ws=A + 16), ALIGN), (dict(mask=A + 2), ALIGN),
    (dict(B=1 << 20, H=256, Hkv=256, T=1, d=64, most=1 << 20, mask=None), UNSUP),
])
def test_cached_window_refuses(kw, want):
    assert cached(**kw) == want


def test_cached_window_refuses_pointers():
    for i in range(10):
        if i not in (3, 4, 7):  # bf16 has no scales; drafts may be null
            assert cached(ptrs=tuple(None if j == i else A for j in range(10))) == BAD, i
        if i not in (3, 4):
            assert cached(ptrs=tuple(A + 2 if j == i else A for j in range(10))) == ALIGN, i


def test_sinks_without_a_window():
    with pytest.raises(ValueError):
        fa.tree_attention(None, None, None, None, None, sinks=4)


def plan(B=2, tokens=5, num=8, page=16, most=4, window=0, sinks=0, ptrs=(A,) * 9):
    return fa.fa_cache_plan(*ptrs, B, tokens, num, page, most, window, sinks, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), BAD), (dict(B=8193), UNSUP), (dict(tokens=-1), BAD), (dict(num=0), BAD),
    (dict(page=8), UNSUP), (dict(page=48), UNSUP), (dict(most=0), BAD),
    (dict(most=(1 << 26) + 1), UNSUP), (dict(window=-1), BAD), (dict(sinks=-1), BAD),
    (dict(tokens=(1 << 30) + 1), UNSUP),
])
def test_plan_refuses_sizes(kw, want):
    assert plan(**kw) == want


def test_plan_refuses_pointers():
    for i in range(9):
        assert plan(ptrs=tuple(None if j == i else A for j in range(9))) == BAD, i
        off = A + 4 if i == 5 else A + 2  # slots are 64-bit
        assert plan(ptrs=tuple(off if j == i else A for j in range(9))) == ALIGN, i


def slots(fmt=1, Hkv=2, N=4, d=64, num=8, page=16, strides=None, ptrs=(A,) * 7):
    return fa.fa_cache_append_slots(*ptrs, fmt, Hkv, N, d, num, page, strides, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), BAD), (dict(Hkv=0), BAD), (dict(num=0), BAD), (dict(fmt=-1), BAD), (dict(fmt=3), BAD),
    (dict(d=32), UNSUP), (dict(page=8), UNSUP), (dict(num=1 << 30), UNSUP),
    (dict(Hkv=1 << 10, N=1 << 22), UNSUP), (dict(strides=(256, 60, 256, 64)), ALIGN),
    (dict(strides=(256, 64, -8, 64)), BAD), (dict(strides=(1 << 62, 64, 256, 64)), BAD),
])
def test_slots_refuse_sizes(kw, want):
    assert slots(**kw) == want


def test_slots_refuse_pointers():
    for i in range(7):
        assert slots(ptrs=tuple(None if j == i else A for j in range(7))) == BAD, i
        off = A + 4 if i == 2 else A + 2
        assert slots(ptrs=tuple(off if j == i else A for j in range(7))) == ALIGN, i
    with pytest.raises(ValueError):
        slots(strides=(256, 64, 256))
    assert slots(N=0, ptrs=(None, None, None) + (A,) * 4) == fa.FA_OK


def test_plan_and_slots_python_refusals():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    args = (i32(2), i32(2), i32(2, 4), i32(8), i32(2), 16, 4)
    for kw in (dict(), dict(sinks=3), dict(window=0)):  # (the first: tensors on the CPU)
        with pytest.raises(ValueError):
            fa.cache_plan(*args, **kw)
    for tokens in (-1, 2**30 + 1, 2**32 + 4):
        with pytest.raises(ValueError, match="max_tokens"):
            fa.cache_plan(*args[:6], tokens)
    k = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    c = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.cache_append_slots(k, k, c, c, torch.zeros(4, dtype=torch.int64))
