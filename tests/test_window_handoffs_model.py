"""A host-side model of the hand-offs of the windowed forward whose CTAs take
unit after unit (csrc/xfwd.cuh, x_walks), in the manner of the cross attention's
(tests/test_cross_handoffs_model.py): over many random interleavings no wait
blocks forever, and every operation finds the tiles it is meant to read.

Two score tiles are in flight, and the MMA warp goes on to the next unit's
scores as soon as their tiles have landed, without waiting for the softmax.  So
the end of a unit has a barrier of its own, and what the last but one product
commits to a score barrier is looked for before the last probabilities are
handed over.  The planted mistake commits the last product to a score barrier
too: the next unit's scores may then complete on it before a softmax warp has
looked, which waits for a phase that is two behind.
"""
import pytest

from tests.test_cross_handoffs_model import WARPS, _halves, _Model, _mma_tile, _Ring

NB = 2          # score tiles in flight


def _walk(seed, units, st, planted):
    m = _Model(seed, {"p": WARPS})
    ring = _Ring(m, "r", st)

    def order(n):
        """Loads of a unit: (kind, tile)."""
        for i in range(-NB, n):
            if i >= 0:
                yield "v", i
            if i + NB < n:
                yield "k", i + NB

    def place(n, i):
        """Number of V i among the unit's loads; K i + NB follows it."""
        return i + (i + NB if i + NB < n else n)

    def producer():
        loads = q = 0
        for u, n in enumerate(units):
            if n == 0:
                continue
            if q:
                yield ((("qe", 0), (q - 1) & 1),)
            m.load(("q", 0), ("q", 0), u)
            q += 1
            for kind, i in order(n):
                yield ring.free(loads)
                ring.load(loads, (kind, u, i))
                loads += 1

    def mma():
        base = q = 0
        written = [0, 0]                # phases of the P barriers before this unit
        for u, n in enumerate(units):
            def issue_s(i, j):
                _mma_tile(m, {("q", 0): u, ("r", (base + j) % st): ("k", u, i)}, ("s", i % NB), ("s", u, i))
                m.commit(("s", i % NB))
                ring.release(base + j)
                if i + 1 == n:
                    m.commit(("qe", 0))

            for i in range(min(NB, n)):
                yield ((("q", 0), q & 1), ring.landed(base + i))
                issue_s(i, i)
            for i in range(n):
                more, jv = i + NB < n, place(n, i)
                p = (("p", i % NB), (written[i % NB] + i // NB) & 1)
                yield (p, ring.landed(base + jv), ring.landed(base + jv + 1)) if more else (p, ring.landed(base + jv))
                _mma_tile(m, _halves(m, ("s", i % NB), ("p", u, i)) | {("r", (base + jv) % st): ("v", u, i)}, "o", ("o", u, i))
                ring.release(base + jv)
                if more:
                    issue_s(i + NB, jv + 1)
                elif i + 1 < n or planted:
                    m.commit(("s", i % NB))
                else:
                    m.commit(("end", 0))
            base += 2 * n
            q += n > 0
            for b in range(NB):
                written[b] += len(range(b, n, NB))

    def softmax(w):
        base = ends = 0
        formed_by = [0, 0]
        for u, n in enumerate(units):
            def formed(i):
                return (("s", i % NB), (formed_by[i % NB] + i // NB) & 1)

            for i in range(n):
                yield (formed(i),)
                m.check((("s", i % NB), w), ("s", u, i))
                if m.rnd.random() < 0.3:                # a tile that lacks keys: V's rows are cleared
                    yield (ring.landed(base + place(n, i)),)
                    m.check(("r", (base + place(n, i)) % st), ("v", u, i))
                if i > 0 and m.rnd.random() < 0.3:      # the maximum grows: O is rescaled
                    yield (formed(i - 1 + NB),)
                    m.check(("o", w), ("o", u, i - 1))
                m.mem[(("s", i % NB), w)] = ("p", u, i)
                if not planted and n > 1 and i + 1 == n:
                    yield (formed(n),)
                m.arrive(("p", i % NB))
            if n:
                if planted:
                    yield (formed(n - 1 + NB),)
                    if n > 1:
                        yield (formed(n - 2 + NB),)
                else:
                    yield ((("end", 0), ends & 1),)
                m.check(("o", w), ("o", u, n - 1))
                ends += 1
            base += 2 * n
            for b in range(NB):
                formed_by[b] += len(range(b, n, NB))
            if planted:
                formed_by[0] += n > 0
                formed_by[1] += n > 1
            elif n > 1:
                formed_by[n % NB] += 1

    roles = {"producer": producer(), "mma": mma()}
    roles.update({f"softmax {w}": softmax(w) for w in range(WARPS)})
    return m.run(roles)


def _outcome(seed, units, st, planted):
    try:
        return _walk(seed, units, st, planted)
    except AssertionError as e:
        return str(e)


@pytest.mark.parametrize("units", [[1, 1, 1, 1], [2, 2, 2], [3, 1, 2, 5], [0, 4, 0, 0, 3], [9, 9, 8], [1, 2, 1, 2, 1], [7]])
@pytest.mark.parametrize("st", [5, 3])
def test_units_one_after_the_other(units, st):
    for seed in range(300):
        assert _outcome(seed, units, st, False) == "ok", (seed, units)


def test_an_end_on_a_score_barrier_is_caught():
    bad = [_outcome(seed, units, 5, True) for units in ([1, 1, 1, 1], [3, 1, 2, 5], [2, 2, 2]) for seed in range(300)]
    assert any(x != "ok" for x in bad)
