"""The windowed backward at d = 64 beside kernels that take its place on an SM
at once.  On a GPU."""
import pytest
import torch

import io_aware_exact_15_gb300 as fa
import window_ref as R
from gpu_common import device, status_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[130], [1], [700, 0, 90, 128]])
def test_short_units_in_a_row(lens):
    """Few and short units, so that a CTA ends right behind its last products
    and the next kernel's barriers stand where its own stood: every run gives
    the same dk, dv, whatever runs next."""
    dev = device()
    x = R.Batch(lens, 2, 2, 64, True, 77, 0, 3)
    q, k, v, g, cu = (t.to(dev) for t in (x.q, x.k, x.v, x.g, x.cu))
    kw = dict(causal=True, cu_seqlens=cu, max_seqlen=max(lens), window=40, sinks=2)
    o, lse = fa.attention_forward(q, k, v, **kw)
    first = fa.attention_backward(q, k, v, o, g, lse, **kw)
    status_ok()
    for _ in range(50):
        again = fa.attention_backward(q, k, v, o, g, lse, **kw)
        o2, lse2 = fa.attention_forward(q, k, v, **kw)
        rows = x.own.to(dev)
        assert torch.equal(o2[:, rows], o[:, rows]) and torch.equal(lse2[:, rows], lse[:, rows])
        for a, b in zip(again[1:], first[1:]):
            assert torch.equal(a[:, rows], b[:, rows])
    status_ok()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        f = [x.seq(t, b) for t in (x.q, x.k, x.v)]
        ref, tol = R.backward(*f, x.seq(o, b), x.seq(lse[..., None], b)[..., 0], x.seq(x.g, b),
                              40, 2, 0.125)
        for a, r, t in zip(first, ref, tol):
            assert bool(((x.seq(a, b) - r).abs() <= t).all())
