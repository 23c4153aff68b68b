"""fp16 gradients of windowed attention where rows of very different size lie out
of each other's reach.

dS is rounded to fp16 under a power of two.  A row that a key (or a query) does
not see must not take part in the choice of that power: the bounds, those of
test_window_gpu.py, hold for every element whatever lies outside its window.

A power of two for everything that a sum joins keeps 2^e |dS| <= 2^15, so what a
subnormal half loses is at most 2^-25 2^-e <= 2^-39 of the largest |dS| that the
bound allows: far below the 2^-13 of fp32 arithmetic that the bounds count.
"""
import pytest
import torch

import sparse_attention_backward_gb300 as sab

from .test_window_gpu import BF, HF, Case, _within

pytestmark = pytest.mark.gpu

R = 20          # the large rows are 2^R times the others


def _uneven(c, side, first):
    """The first `first` tokens of each sequence: dY (or V) 2^R times the others', all of it numbers that fp16 holds."""
    base = 2.0 ** -11
    for name, lens in (("dy", c.l1), ("v", c.l2)):
        if side not in (name, "both"):
            continue
        x = getattr(c, name)
        x *= base
        for b, n in enumerate(lens):
            n = min(n, first)
            at = (b, slice(0, n)) if c.padded else slice((c.cu1 if name == "dy" else c.cu2)[b], (c.cu1 if name == "dy" else c.cu2)[b] + n)
            x[at] *= 2.0 ** R
    return c


def _check(c, side):
    o, lse = sab.window_forward(c.q, c.k, c.v, check=True, **c.args())
    grads = sab.window_backward(c.q, c.k, c.v, o, c.dy, lse, check=True, **c.args())
    want, tol = c.backward(o, lse)
    most = torch.finfo(c.dtype).max
    for name, x, w, t in zip(("dq", "dk", "dv"), grads, want, tol):
        # large dY and V together give sums beyond the type: infinities of their sign there
        x, lim = x.reshape(w.shape), 1.01 * (w.abs() * torch.finfo(c.dtype).eps / 2 + t)
        beyond = w.abs() + lim >= most
        sure = w.abs() - lim >= most * (1 + torch.finfo(c.dtype).eps)
        assert bool((x[sure] == w[sure].sign() * float("inf")).all()), name
        assert not beyond.any() or side == "both"
        _within(name, x.masked_fill(beyond, 0.0), w.masked_fill(beyond, 0.0), t, c.dtype)


@pytest.mark.parametrize("side", ["dy", "v", "both"])
@pytest.mark.parametrize("d,n1,n2", [(128, 4, 2), (64, 3, 3), (128, 16, 1), (64, 20, 2)])
@pytest.mark.parametrize("left,right", [(-1, 0), (300, 0), (127, 0), (128, 0), (7, 0), (0, 0), (3, 5), (40, -1), (90, 200)])
def test_rows_out_of_reach(side, d, n1, n2, left, right):
    # the border of the large rows inside a tile
    _check(_uneven(Case([900], [900], n1, n2, d, HF, left, right, seed=n1 + 50), side, 70), side)


@pytest.mark.parametrize("side", ["dy", "v"])
@pytest.mark.parametrize("l1,l2", [([500, 700], [900, 400]), ([0, 300, 41], [60, 300, 0])])
@pytest.mark.parametrize("left,right", [(-1, 0), (100, 30)])
@pytest.mark.parametrize("padded", [False, True])
def test_masks_padding_and_lengths_that_differ(side, l1, l2, left, right, padded):
    _check(_uneven(Case(l1, l2, 6, 2, 128, HF, left, right, padded=padded, mask=0.3, seed=51), side, 64), side)


# units whole, in pieces and shared by clusters, of either kernel
@pytest.mark.parametrize("side", ["dy", "v"])
@pytest.mark.parametrize("l1,l2,n1,n2,d,left,right", [
    ([8192], [8192], 1, 1, 64, -1, 0), ([1195], [1195], 32, 8, 128, 600, 0), ([5327, 2511], [5327, 1255], 1, 1, 128, -1, 0),
    ([705], [1410], 1, 1, 128, 300, 0), ([3000], [3000], 2, 1, 128, -1, 0), ([4100], [4100], 4, 4, 64, 2600, 0)])
def test_units_shared_by_ctas(side, l1, l2, n1, n2, d, left, right):
    _check(_uneven(Case(l1, l2, n1, n2, d, HF, left, right, seed=52), side, 64), side)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_rows_that_are_not_finite_do_not_scale_others(bad):
    """A row of dY that is not finite spoils the sums it is joined to, and no key that is out of its query tile's reach."""
    c = Case([900], [900], 4, 2, 128, HF, 30, 0, seed=53)
    o, lse = sab.window_forward(c.q, c.k, c.v, **c.args())
    clean = sab.window_backward(c.q, c.k, c.v, o, c.dy, lse, **c.args())
    c.dy[3, 1, 5] = bad
    spoilt = sab.window_backward(c.q, c.k, c.v, o, c.dy, lse, check=True, **c.args())
    for x, y in zip(clean, spoilt):
        assert torch.equal(x[300:], y[300:])
    assert not bool(torch.isfinite(spoilt[2][3]).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("l,n1,n2,left", [([700, 300], 8, 2, 100), ([3000], 2, 1, -1), ([120] * 40, 32, 8, 60)])
def test_calls_of_other_inputs_in_one_workspace(dtype, l, n1, n2, left):
    """Nothing of a call is left for the next: a captured forward and gradient, replayed with one input after the other."""
    cases = [Case(l, l, n1, n2, 128, dtype, left, 0, seed=54 + i, dy_scale=4.0 ** -i) for i in range(3)]
    want = []
    for c in cases:
        o, lse = sab.window_forward(c.q, c.k, c.v, **c.args())
        want.append((o, lse) + sab.window_backward(c.q, c.k, c.v, o, c.dy, lse, **c.args()))
    a = cases[0]
    desc = sab.make_window_desc(a.cu1, a.cu2, n1, n2, 128, a.scale, left, 0, sab.SAG_FP16 if dtype is HF else sab.SAG_BF16)
    ws = torch.empty(max(sab.window_fwd_workspace_size(desc), sab.window_grad_workspace_size(desc)), dtype=torch.uint8, device="cuda")
    held = [torch.empty_like(x) for x in (a.q, a.k, a.v, a.dy)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = sab.window_forward(*held[:3], desc=desc, workspace=ws)
        outs = (o, lse) + sab.window_backward(*held[:3], o, held[3], lse, desc=desc, workspace=ws)
    for turn in range(30):
        c = cases[turn * 2 % 3]
        for x, y in zip(held, (c.q, c.k, c.v, c.dy)):
            x.copy_(y)
        g.replay()
        for x, y in zip(outs, want[turn * 2 % 3]):
            assert torch.equal(x, y)
