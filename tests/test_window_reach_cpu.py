"""How far a value that is not finite reaches beyond the windows that hold its row:
the tiles that the kernels load (their arithmetic restated), against the number
that the header states."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def stated():
    txt = open(os.path.join(ROOT, "include", "selattn.h")).read()
    part = txt[txt.index("A sequence's own rows have to be finite"):]
    return int(re.search(r"up to (\d+) (?:positions|rows)", part).group(1))


def beyond(at, lo, hi):
    """Positions from `at` to the nearest of lo .. hi, 0 inside."""
    return max(lo - at, at - hi, 0)


def reach_over_keys(tokens, n, left, right, keys):
    """Forward (V) and dQ (K): rows of a query tile take all keys of the tiles that their windows together touch."""
    far = 0
    for t0 in range(0, n, tokens):
        t1 = min(t0 + tokens, n) - 1
        lo, hi = max(0, t0 - left), min(n, t1 + right + 1)
        last = min(lo + -(-(hi - lo) // keys) * keys, n) - 1           # (rows that are not the sequence's are zeroed)
        for p in (t0, t1):
            far = max(far, *(beyond(j, p - left, p + right) for j in (lo, last)))
    return far


def reach_over_queries(tokens, n, left, right, keys=128):
    """dK and dV: the keys of a key tile take all rows of the query tiles that see any of them."""
    far = 0
    for k0 in range(0, n, keys):
        k1 = min(k0 + keys, n) - 1
        first, to = max(0, k0 - right), min(n, k1 + left + 1)
        first, last = first // tokens * tokens, min(-(-to // tokens) * tokens, n) - 1
        for j in (k0, k1):
            far = max(far, *(beyond(i, j - right, j + left) for i in (first, last)))
    return far


@pytest.mark.parametrize("group", [1, 2, 3, 4, 8, 16, 32])
def test_no_value_reaches_further_than_stated(group):
    tokens, most = 128 // group, 0
    for left in list(range(0, 140)) + [200, 255, 256, 300, 511]:
        for right in (0, 1, 5, 64, 127, 128):
            for n in (1024, 1000):
                most = max([most] + [reach_over_keys(tokens, n, left, right, keys) for keys in (64, 128)] +
                           [reach_over_queries(tokens, n, left, right)])
    assert most <= stated()
    if group == 1:
        assert most == stated()


def test_pages_reach_less():
    """Over pages V's rows outside a tile's windows are zeroed: a row's neighbours in its query tile only."""
    for tokens in (128, 64, 42, 8, 4):
        for left in (0, 1, 63, 200):
            for t0 in range(0, 1024, tokens):
                t1 = min(t0 + tokens, 1024) - 1
                assert beyond(t1, t0 - left, t0) <= 127 and beyond(t0 - left, t1 - left, t1) <= 127
