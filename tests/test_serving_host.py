"""Refusals of the Q/K preparation and serving entry points (no GPU: every
case returns before the first CUDA call), and checks of the 64-bit formulas
the GPU tests use."""
import numpy as np
import pytest
import torch

import io_aware_exact_15_gb300 as fa
import serving_ref as R

A = 1 << 20      # fake device pointers, never dereferenced
MIS = A + 8
BAD, UNSUP, ALIGN, WS = (fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_MISALIGNED,
                         fa.FA_ERR_WORKSPACE)


def rope(B=2, H=4, Hkv=2, N=8, d=64, rot=64, rows=16, eps=1e-6, strides=None, ptrs=(A,) * 9):
    return fa.fa_qk_norm_rope(*ptrs, B, H, Hkv, N, d, rot, rows, 0, eps, strides, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), BAD), (dict(H=0), BAD), (dict(Hkv=0), BAD), (dict(N=0), BAD), (dict(rows=0), BAD),
    (dict(eps=0.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(d=96), UNSUP), (dict(rot=8), UNSUP), (dict(rot=24), UNSUP), (dict(rot=80), UNSUP),
    (dict(rot=0), UNSUP), (dict(B=1 << 20, N=1 << 20), UNSUP),
    (dict(ptrs=(None,) + (A,) * 8), BAD), (dict(ptrs=(MIS,) + (A,) * 8), ALIGN),
    (dict(ptrs=(A,) * 2 + (None,) + (A,) * 6), BAD), (dict(ptrs=(A,) * 3 + (A + 4,) + (A,) * 5), ALIGN),
    (dict(ptrs=(A,) * 4 + (MIS,) + (A,) * 4), ALIGN), (dict(ptrs=(A,) * 6 + (A + 2,) + (A,) * 2), ALIGN),
    (dict(ptrs=(A,) * 7 + (None, A)), BAD), (dict(ptrs=(A,) * 8 + (MIS,)), ALIGN),
    (dict(strides=(2048, 512, 68, 1024, 512, 64)), ALIGN),
    (dict(strides=(2048, 512, 64, 1024, -512, 64)), BAD),
    (dict(strides=(1 << 62, 512, 64, 1024, 512, 64)), BAD),
])
def test_norm_rope_refuses(kw, want):
    assert rope(**kw) == want


def rope_back(B=2, H=4, Hkv=2, N=8, d=64, rot=64, rows=16, eps=1e-6, strides=None, grads=None,
              ptrs=(A,) * 13, ws=A, size=None):
    size = fa.fa_qk_norm_rope_workspace_size(d) if size is None else size
    return fa.fa_qk_norm_rope_backward(*ptrs, B, H, Hkv, N, d, rot, rows, 1, eps, strides, grads,
                                       ws, size, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), BAD), (dict(d=32), UNSUP), (dict(ptrs=(None,) + (A,) * 12), BAD),
    (dict(ptrs=(A,) * 9 + (MIS,) + (A,) * 3), ALIGN), (dict(ptrs=(A,) * 11 + (None, A)), BAD),
    (dict(ptrs=(A,) * 12 + (A + 2,)), ALIGN),
    (dict(ws=None), BAD), (dict(ws=A + 16), ALIGN), (dict(size=100), WS),
    # gradients whose rows overlap: equal strides, a head inside a row, stride 0
    (dict(grads=(2048, 64, 64, 1024, 512, 64)), BAD),
    (dict(grads=(2048, 512, 32, 1024, 512, 64)), BAD),
    (dict(grads=(2048, 0, 64, 1024, 512, 64)), BAD),
    (dict(grads=(2048, 512, 64, 512, 512, 64)), BAD),
])
def test_norm_rope_backward_refuses(kw, want):
    assert rope_back(**kw) == want


def test_packed_gradient_strides_are_disjoint():
    """[B, N, H + 2 Hkv, d] slices pass the overlap check: the next check (the
    workspace) answers."""
    H, Hkv, N, d = 4, 2, 8, 64
    row = (H + 2 * Hkv) * d
    assert rope_back(grads=(N * row, d, row) * 2, size=0) == WS
    # axes of length 1 may have any stride
    assert rope_back(B=1, grads=(3, d, row) * 2, size=0) == WS


def cache(write, fmt=1, B=2, Hkv=2, N=4, d=64, num=8, page=16, most=4, strides=None,
          ptrs=(A,) * 9):
    if write:
        return fa.fa_cache_append(*ptrs, fmt, B, Hkv, N, d, num, page, most, strides, 0)
    return fa.fa_cache_read(*ptrs, fmt, B, Hkv, N, d, num, page, most, 0)


SIZES = [
    (dict(B=0), BAD), (dict(N=0), BAD), (dict(Hkv=0), BAD), (dict(num=0), BAD), (dict(most=0), BAD),
    (dict(fmt=-1), BAD), (dict(fmt=3), BAD), (dict(d=32), UNSUP), (dict(page=8), UNSUP),
    (dict(page=48), UNSUP), (dict(page=256), UNSUP), (dict(most=1 << 27), UNSUP),
    (dict(most=(1 << 26) + 1), UNSUP),
    (dict(num=1 << 30), UNSUP), (dict(B=1 << 20, N=1 << 20), UNSUP), (dict(B=1 << 28), UNSUP),
]


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("kw,want", SIZES)
def test_cache_refuses_sizes(write, kw, want):
    assert cache(write, **kw) == want


@pytest.mark.parametrize("write", [True, False])
def test_cache_refuses_pointers(write):
    for i in range(9):
        null = tuple(None if j == i else A for j in range(9))
        counts = i == (4 if write else 6)
        if not counts:  # counts alone may be null
            assert cache(write, ptrs=null) == BAD, i
        off = tuple(A + 2 if j == i else A for j in range(9))
        assert cache(write, ptrs=off) == ALIGN, i
    if write:
        assert cache(write, strides=(512, 256, 60, 512, 256, 64)) == ALIGN
        assert cache(write, strides=(512, 256, 64, 512, -8, 64)) == BAD


def test_strides_need_six_numbers():
    with pytest.raises(ValueError):
        cache(True, strides=(512, 256, 64))


def tree(fmt=0, B=2, H=4, Hkv=2, T=4, d=64, num=8, page=16, most=4, scale=0.1, ptrs=(A,) * 11,
         ws=A, size=None):
    size = fa.fa_tree_attention_workspace_size(B, H, Hkv, T, d) if size is None else size
    return fa.fa_tree_attention(*ptrs, fmt, B, H, Hkv, T, d, num, page, most, scale, ws, size, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), BAD), (dict(H=0), BAD), (dict(T=0), BAD), (dict(Hkv=0), BAD), (dict(Hkv=3), BAD),
    (dict(Hkv=8), BAD), (dict(num=0), BAD), (dict(most=0), BAD), (dict(fmt=7), BAD),
    (dict(scale=0.0), BAD), (dict(scale=float("nan")), BAD), (dict(scale=-1.0), BAD),
    (dict(d=80), UNSUP), (dict(page=24), UNSUP), (dict(T=1025), UNSUP),
    (dict(B=1 << 16, H=64, T=64, d=64), UNSUP), (dict(most=1 << 27), UNSUP),
    (dict(most=(1 << 26) + 1), UNSUP),
    # 2^23 tiles in a table, 256 (sequence, head) pairs: 2^31 units; with 512
    # rows per key/value head twice as many again
    (dict(B=128, Hkv=2, most=1 << 26), UNSUP), (dict(B=64, H=256, Hkv=2, most=1 << 26), UNSUP),
    (dict(ws=None), BAD), (dict(ws=A + 128), ALIGN), (dict(size=0), WS),
])
def test_tree_refuses(kw, want):
    assert tree(**kw) == want


def test_tree_refuses_pointers():
    for fmt in (0, 1, 2):
        for i in range(11):
            optional = i in (7, 8) or (fmt == 0 and i in (3, 4))
            if not optional:
                null = tuple(None if j == i else A for j in range(11))
                assert tree(fmt=fmt, ptrs=null) == BAD, i
            if not (fmt == 0 and i in (3, 4)):
                off = tuple(A + 2 if j == i else A for j in range(11))
                assert tree(fmt=fmt, ptrs=off) == ALIGN, i


def test_workspace_sizes():
    assert fa.fa_qk_norm_rope_workspace_size(128) == 1024 * 2 * 128 * 4
    assert fa.fa_qk_norm_rope_workspace_size(0) == 0
    assert fa.fa_tree_attention_workspace_size(0, 1, 1, 1, 64) == 0
    assert fa.fa_tree_attention_workspace_size(1, 4, 2, 1, 64) > 0


def test_wrappers_refuse_host_tensors_and_wrong_types():
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    cos = torch.zeros(4, 32)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q, q, w, w, cos, cos)  # not on a GPU
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q.float(), q, w, w, cos, cos)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q[0], q, w, w, cos, cos)
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    t = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.cache_append(q, q, kc, kc, t, t[0])
    with pytest.raises(ValueError):
        fa.tree_attention(q, kc.bfloat16(), kc.bfloat16(), t, t[0])


# ------------------------------------------------------------------ the formulas themselves
@pytest.mark.parametrize("inter", [False, True])
def test_backward_formula_against_differences(inter):
    rng = np.random.default_rng(0)
    B, H, N, d, rot, eps = 1, 2, 3, 8, 4, 1e-3
    x, g, w = rng.normal(size=(B, H, N, d)), rng.normal(size=(B, H, N, d)), rng.normal(size=d)
    a = rng.normal(size=(B, 1, N, rot // 2))
    c, s = np.cos(a), np.sin(a)
    f = lambda x, w: (g * R.norm_rope(x, w, c, s, rot, inter, eps)).sum()
    dx, dw, _, _ = R.norm_rope_backward(g, x, w, c, s, rot, inter, eps)
    h = 1e-6
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        # central differences: h^2 / 6 of the third derivative, 1e-16 f / h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for i in range(d):
        e = np.zeros(d)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_rotation_keeps_lengths_and_relative_positions():
    """The product of two turned rows depends on the distance of their
    positions alone; a planted sign flip does not have that property."""
    rng = np.random.default_rng(1)
    cos, sin = (R.f64(t) for t in R.tables(50, 16))
    a, b = rng.normal(size=16), rng.normal(size=16)
    for inter in (False, True):
        dot = lambda i, j, sg=1: (R.turn(a, cos[i], sin[i], 16, inter) *
                                  R.turn(b, cos[j], sg * sin[j], 16, inter)).sum()
        assert abs(dot(3, 10) - dot(33, 40)) < 1e-5
        assert abs(dot(3, 10, -1) - dot(33, 40, -1)) > 1e-2


def test_quantise_definition():
    """Values on the formats' grids stay; ties go to even; a row's largest
    number decides the step."""
    x = np.array([[448.0, 1.0, 0.0, -3.25], [449.0, 1.0, 0.0, 0.0], [0.0] * 4,
                  [1.0, np.nan, 0.0, 0.0]])
    y = R.quantise(x, R.E4M3)
    assert np.array_equal(y[0], x[0]) and y[1, 0] == 448.0 and np.array_equal(y[2], x[2])
    assert np.isnan(y[3]).all()
    z = R.quantise(np.array([[127.0, 0.5, 1.5, -2.5], [127.5, 1.0, 3.0, 0.0]]), R.INT8)
    assert np.array_equal(z[0], [127.0, 0.0, 2.0, -2.0])
    assert np.array_equal(z[1], [128.0, 0.0, 4.0, 0.0])  # steps of 2 now, ties to even
    rng = np.random.default_rng(2)
    x = rng.normal(size=(200, 64)) * 2.0 ** rng.integers(-60, 60, (200, 1))
    for fmt, half in ((R.E4M3, 2.0 ** -4), (R.INT8, None)):
        y = R.quantise(x, fmt)
        assert np.array_equal(R.quantise(y, fmt), y)
        amax = np.abs(x).max(-1, keepdims=True)
        # e4m3: half a step of 2^-3 of the value, or of its smallest numbers
        bound = half * np.abs(x) + 2.0 ** -10 / 224 * amax if half else amax / 126
        assert (np.abs(x - y) <= bound).all()


def test_trees():
    rng = np.random.default_rng(3)
    bits = R.random_trees(rng, 3, 40)
    assert bits[:, np.arange(40), np.arange(40)].all() and not np.triu(bits, 1).any()
    w = R.words_of(bits).numpy().view(np.uint32)
    for b, i, j in ((0, 5, 3), (1, 39, 0), (2, 39, 39), (2, 35, 33)):
        assert bool(w[b, i, j // 32] >> (j % 32) & 1) == bits[b, i, j]
