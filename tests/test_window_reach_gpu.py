"""A value that is not finite in a sequence's own row: results further than 254
positions from the windows that hold the row have the bits that they had without
it, and so have those of other sequences and heads."""
import pytest
import torch

import sparse_attention_backward_gb300 as sab

from .test_window_gpu import BF, HF, Case, Pages

pytestmark = pytest.mark.gpu

REACH = 254


@pytest.mark.parametrize("d,dtype,n1,n2", [(128, BF, 4, 4), (64, HF, 4, 2), (128, HF, 16, 1)])
@pytest.mark.parametrize("left,right", [(1, 0), (100, 30), (-1, 0)])
@pytest.mark.parametrize("what", ["q", "k", "v", "dy", "o"])
def test_reach(d, dtype, n1, n2, left, right, what):
    c = Case([1300, 200], [1300, 200], n1, n2, d, dtype, left, right, seed=90)
    lost = torch.arange(1500, device="cuda")
    at = 700
    clean = sab.window_forward(c.q, c.k, c.v, **c.args())
    if what in ("q", "k", "v"):
        getattr(c, what)[at, 0, 7] = float("nan")
        o, lse = sab.window_forward(c.q, c.k, c.v, check=True, **c.args())
        if what != "q":
            seen_by = (lost >= at - right - REACH) & (lost <= (at + left + REACH if left >= 0 else 1299))
        else:
            seen_by = lost == at
        for x, y in zip((o, lse), clean):
            assert torch.equal(x[~seen_by], y[~seen_by])
            if n2 > 1:
                assert torch.equal(x[:, n1 // n2:], y[:, n1 // n2:])
        if what in ("q", "k", "v"):
            getattr(c, what)[at, 0, 7] = 0.5
    # the gradient, from an attention_out that is finite
    o, lse = sab.window_forward(c.q, c.k, c.v, **c.args())
    x = {"q": c.q, "k": c.k, "v": c.v, "dy": c.dy, "o": o}
    want = sab.window_backward(x["q"], x["k"], x["v"], x["o"], x["dy"], lse, **c.args())
    x[what][at, 0, 7] = float("nan")
    got = sab.window_backward(x["q"], x["k"], x["v"], x["o"], x["dy"], lse, check=True, **c.args())
    rows = (lost >= at - right - REACH) & (lost <= (at + left + REACH if left >= 0 else 1299))     # that may see key `at`
    keys = (lost <= at + right + REACH) & (lost >= (at - left - REACH if left >= 0 else 0))        # that row `at` may see
    for a, b, touched in zip(got, want, (rows if what in ("k", "v") else lost == at, keys, keys)):
        if what in ("k", "v") and a is not got[0]:
            touched = lost == at
        assert torch.equal(a[~touched], b[~touched])
    if n2 > 1:
        assert torch.equal(got[0][:, n1 // n2:], want[0][:, n1 // n2:])
        assert torch.equal(got[1][:, 1:], want[1][:, 1:]) and torch.equal(got[2][:, 1:], want[2][:, 1:])


@pytest.mark.parametrize("d,dtype", [(128, BF), (64, HF)])
def test_reach_over_pages(d, dtype):
    c = Case([900], [1300], 4, 4, d, dtype, 60, 0, seed=91)
    p = Pages(c, 32)
    clean = p.forward(c)
    at = 800                                                     # a key; query 400 stands there
    c.v[at, 0, 7] = float("nan")
    o, lse = Pages(c, 32).forward(c)
    rows = torch.arange(900, device="cuda")
    touched = (rows >= 400 - 127) & (rows <= 400 + 60 + 127)
    assert torch.equal(o[~touched], clean[0][~touched]) and torch.equal(lse, clean[1])
    assert torch.equal(o[:, 1:], clean[0][:, 1:]) and bool(torch.isnan(o[400:461, 0, 7]).all())
