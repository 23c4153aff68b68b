"""Forwards of windowed and paged attention whose CTAs take unit after unit, and
those whose long loops are shared by CTAs, element by element against the
definition in 64 bits with the bounds of test_window_gpu.py.

Two CTAs of 128-wide heads run on each of 152 SMs, so a launch of more than 304
units, each a tile of 128 query rows of a key/value head, has CTAs that take
another unit when one is done: state of one unit must not show in the next.
"""
import pytest
import torch

import sparse_attention_backward_gb300 as sab

from .test_window_gpu import BF, HF, Case, Pages, check_forward

pytestmark = pytest.mark.gpu

AT_ONCE = 304


def _units(c):
    tokens = 128 // (c.n1 // c.n2)
    return sum(-(-(c.s1 if c.padded else n) // tokens) for n in c.l1) * c.n2


def _ragged(count, most, seed, context=0):
    """Lengths of `count` sequences up to `most`: some without queries, some without keys, some of a token, and contexts before
    the queries or keys that are fewer than them."""
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    l1, l2 = [], []
    for b in range(count):
        a = r(1, most)
        n = max(a + r(-40, context), 0)
        if b % 7 == 2:
            a = 0
        if b % 9 == 4:
            n = 0
        if b % 11 == 6:
            a = 1
        l1.append(a)
        l2.append(n)
    return l1, l2


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("masked", [None, 0.3])
@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("n1,n2,left,right", [(32, 8, 100, 0), (12, 4, -1, 0), (6, 6, 40, 70)])
def test_windows_unit_after_unit(dtype, masked, padded, n1, n2, left, right):
    l1, l2 = _ragged(40 if n1 > n2 else 60, 300, n1)
    c = Case(l1, l2, n1, n2, 128, dtype, left, right, padded=padded, mask=masked, seed=60 + n1)
    assert _units(c) > AT_ONCE + 200
    check_forward(c, *sab.window_forward(c.q, c.k, c.v, check=True, **c.args()))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("page", [16, 48, 64])
@pytest.mark.parametrize("n1,n2,left,padded", [(32, 8, 100, False), (12, 4, -1, True)])
def test_pages_unit_after_unit(dtype, page, n1, n2, left, padded):
    l1, l2 = _ragged(40, 300, n1, context=500)
    c = Case(l1, l2, n1, n2, 128, dtype, left, 0, padded=padded, seed=70 + n1)
    assert _units(c) > AT_ONCE + 200
    check_forward(c, *Pages(c, page, strided=padded).forward(c))


@pytest.mark.parametrize("page", [None, 64])
def test_unit_after_unit_is_the_same_unit_alone(page):
    """Each sequence's rows have the bits of a call of its own wherever that has loops in one piece too."""
    l1, l2 = _ragged(30, 120, 5)
    c = Case(l1, l2, 32, 8, 128, BF, 50, 0, seed=80)
    assert _units(c) > AT_ONCE and max(l2) < 8 * 64          # loops of fewer than 8 tiles are never shared
    p = Pages(c, page) if page else None
    o, lse = p.forward(c) if p else sab.window_forward(c.q, c.k, c.v, check=True, **c.args())
    for b, (a, n) in enumerate(zip(l1, l2)):
        rows, keys = slice(c.cu1[b], c.cu1[b + 1]), slice(c.cu2[b], c.cu2[b + 1])
        if p:
            x, y = sab.paged_forward(c.q[rows], p.k, p.v, p.table[b:b + 1], p.lens[b:b + 1], [0, a], c.scale, 50, 0)
        else:
            x, y = sab.window_forward(c.q[rows], c.k[keys], c.v[keys], [0, a], [0, n], c.scale, 50, 0)
        assert torch.equal(o[rows], x) and torch.equal(lse[rows], y)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("masked", [None, 0.2])
def test_long_windows_in_pieces(dtype, masked):
    # 18 units of full query tiles in 16 pieces each, of more than 2048 keys: tiles of 128 keys, and a second kernel that joins
    c = Case([200], [33000], 9, 9, 128, dtype, -1, 0, mask=masked, seed=81)
    d = sab.make_window_desc(c.cu1, c.cu2, 9, 9, 128, c.scale)
    assert _units(c) == 18 and sab.window_fwd_workspace_size(d) > 18 * 16 * 128 * 130 * 4
    check_forward(c, *sab.window_forward(c.q, c.k, c.v, check=True, **c.args()))


@pytest.mark.parametrize("dtype,page", [(BF, 64), (HF, 48), (BF, 128)])
def test_long_pages_in_pieces(dtype, page):
    c = Case([200], [33000], 9, 9, 128, dtype, -1, 0, seed=82)
    p = Pages(c, page)
    d = sab.make_paged_desc(c.cu1, 9, 9, 128, c.scale, p.k.shape[0], page, p.width)
    assert _units(c) == 18 and sab.paged_fwd_workspace_size(d) > 18 * 16 * 128 * 130 * 4
    check_forward(c, *p.forward(c))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("page", [None, 64])
def test_long_loops_shared_by_clusters(dtype, page):
    # 128 units: clusters of two, with more than 2048 keys a CTA: tiles of 128 keys
    c = Case([700, 300], [4400, 2500], 16, 8, 128, dtype, -1, 0, seed=83)
    assert 97 < _units(c) <= 152 and max(c.l2) >= 2 * 2048
    check_forward(c, *(Pages(c, page).forward(c) if page else sab.window_forward(c.q, c.k, c.v, check=True, **c.args())))
