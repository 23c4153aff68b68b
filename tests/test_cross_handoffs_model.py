"""A host-side model of the hand-offs of the cross-attention kernels
(csrc/cross_fwd.cu, csrc/cross_bwd.cu): producer, MMA and softmax roles.

Each role is a generator that waits on mbarrier phases by parity, as the
kernels do; a combined wait passes when all of its phases are complete at one
look.  Loads land and tensor-core operations complete (in the order of their
issue) at random times, and any role may pause for long (a miss in the
instruction cache).  Over many random interleavings:
- no wait blocks forever (one that finds its barrier two phases on would);
- every operation finds the tiles it is meant to read, in shared memory and in
  tensor memory.

One barrier for the dS tiles of k_xdq is the planted mistake: both score tiles
and the next dP are issued by then, so the softmax may finish two tiles while
the MMA warp has yet to look for the first, and arrivals of two tiles may mix.
"""
import random

import pytest

WARPS = 3       # softmax warps of the model


class _Model:
    def __init__(self, seed, counts):
        self.rnd = random.Random(seed)
        self.left = {}
        self.phase = {}
        self.count = counts
        self.pipe, self.loads, self.mem = [], [], {}

    def arrive(self, bar):
        n = self.count.get(bar[0], 1)
        self.left[bar] = self.left.get(bar, n) - 1
        if self.left[bar] == 0:
            self.left[bar] = n
            self.phase[bar] = self.phase.get(bar, 0) + 1

    def done(self, wait):
        return all((self.phase.get(bar, 0) & 1) != parity for bar, parity in wait)

    # a load, an operation that reads {place: tag} and writes `out`, a commit
    def load(self, bar, place, tag):
        self.loads.append((bar, place, tag))

    def mma(self, reads, place, tag):
        self.pipe.append((reads, place, tag))

    def commit(self, bar):
        self.pipe.append(bar)

    def check(self, place, tag):
        assert self.mem.get(place) == tag, f"{place} holds {self.mem.get(place)}, not {tag}"

    def run(self, roles):
        asleep = {k: 0 for k in roles}
        wait = {k: () for k in roles}
        while roles:
            ready = [k for k in roles if not asleep[k] and self.done(wait[k])]
            choices = ready + ["pipe"] * bool(self.pipe) + ["load"] * bool(self.loads)
            resting = [k for k in roles if asleep[k]]
            for k in resting:
                asleep[k] -= 1
            if not choices:
                if resting:
                    continue
                return f"blocked: {wait}"
            c = self.rnd.choice(choices)
            if c == "pipe":
                item = self.pipe.pop(0)
                if len(item) == 3:
                    for place, tag in item[0].items():
                        self.check(place, tag)
                    self.mem[item[1]] = item[2]
                else:
                    self.arrive(item)
            elif c == "load":
                bar, place, tag = self.loads.pop(self.rnd.randrange(len(self.loads)))
                self.mem[place] = tag
                self.arrive(bar)
            else:
                try:
                    wait[c] = next(roles[c])
                    if self.rnd.random() < 0.1:
                        asleep[c] = self.rnd.randint(1, 60)
                except StopIteration:
                    del roles[c]
        return "ok"


class _Ring:
    def __init__(self, m, name, n):
        self.m, self.name, self.n = m, name, n

    def landed(self, i):
        return ((self.name + "_full", i % self.n), (i // self.n) & 1)

    def free(self, i):
        return (((self.name + "_empty", i % self.n), (i // self.n - 1) & 1),) if i >= self.n else ()

    def load(self, i, tag):
        self.m.load((self.name + "_full", i % self.n), (self.name, i % self.n), tag)

    def release(self, i):
        self.m.commit((self.name + "_empty", i % self.n))


def _halves(m, place, tags):
    """The softmax warps' parts of a tile, as what an operation reads."""
    return {(place, w): tags for w in range(WARPS)}


def _write_tile(m, place, tag):
    """What an operation leaves behind for every softmax warp."""
    return [((place, w), tag) for w in range(WARPS)]


def _mma_tile(m, reads, place, tag):
    first = True
    for where, t in _write_tile(m, place, tag):
        m.mma(reads if first else {}, where, t)
        first = False


def _gradient_q(seed, units, ra_n, rb_n, rx_n, ds_bars):
    """`units`: tiles of each, 0 without work."""
    m = _Model(seed, {"pf": WARPS, "ds": WARPS, "unit_empty": WARPS + 1})
    ra, rb, rx, ru = _Ring(m, "k", ra_n), _Ring(m, "v", rb_n), _Ring(m, "x", rx_n), _Ring(m, "unit", 2)
    units = units + [-1]

    def ds(g):
        return (("ds", g % ds_bars), (g // ds_bars) & 1)

    def producer():
        la = lb = u = 0
        for k, n in enumerate(units):
            yield ru.free(k)
            m.arrive(("unit_full", k % 2))
            if n <= 0:
                continue
            yield rx.free(u)
            rx.load(u, u)
            u += 1
            yield ra.free(la)
            ra.load(la, la)
            la += 1
            for i in range(n):
                yield rb.free(lb)
                rb.load(lb, lb)
                lb += 1
                if i + 1 < n:
                    yield ra.free(la)
                    ra.load(la, la)
                    la += 1

    def mma():
        def issue_s(g, u):
            _mma_tile(m, {("x", u % rx_n): u, ("k", g % ra_n): g}, ("s", g & 1), ("s", g))
            m.commit(("s", g & 1))

        def issue_dp(g, u):
            _mma_tile(m, {("x", u % rx_n): u, ("v", g % rb_n): g}, "dp", ("dp", g))
            m.commit(("dp", 0))
            rb.release(g)

        g = u = 0
        for k, n in enumerate(units):
            yield (ru.landed(k),)
            m.arrive(("unit_empty", k % 2))
            if n <= 0:
                continue
            yield (rx.landed(u), ra.landed(g))
            issue_s(g, u)
            yield (rb.landed(g),)
            issue_dp(g, u)
            if n > 1:
                yield (ra.landed(g + 1),)
                issue_s(g + 1, u)
            else:
                rx.release(u)
            for i in range(n):
                if i + 1 < n:
                    yield ((("pf", 0), g & 1), rb.landed(g + 1))
                    issue_dp(g + 1, u)
                    if i + 2 == n:
                        rx.release(u)
                yield (ds(g), ra.landed(g + 2)) if i + 2 < n else (ds(g),)
                m.mma(_halves(m, ("s", g & 1), ("ds", g)) | {("k", g % ra_n): g}, "dq", u)
                ra.release(g)
                if i + 2 < n:
                    issue_s(g + 2, u)
                g += 1
            m.commit(("acc", 0))
            u += 1

    def softmax(w):
        g = u = 0

        def begin(k):
            yield (ru.landed(k),)
            m.arrive(("unit_empty", k % 2))

        yield from begin(0)
        for k, n in enumerate(units[:-1]):
            for _ in range(n):
                yield ((("s", g & 1), (g >> 1) & 1),)
                m.check((("s", g & 1), w), ("s", g))
                yield ((("dp", 0), g & 1),)
                m.check(("dp", w), ("dp", g))
                m.arrive(("pf", 0))
                yield ()
                m.mem[(("s", g & 1), w)] = ("ds", g)
                m.arrive(ds(g)[0])
                g += 1
            yield from begin(k + 1)
            if n:
                yield ((("acc", 0), u & 1),)
                yield ()                        # stores
                m.check("dq", u)
                u += 1

    return m.run(dict({w: softmax(w) for w in range(WARPS)}, producer=producer(), mma=mma()))


def _gradient_kv(seed, units, ra_n, rb_n, rx_n):
    m = _Model(seed, {"pf": WARPS, "ds": WARPS, "st_empty": WARPS})
    ra, rb, rs, rx = _Ring(m, "q", ra_n), _Ring(m, "dy", rb_n), _Ring(m, "st", 2), _Ring(m, "x", rx_n)

    def producer():
        g = 0
        for u, n in enumerate(units):
            yield rx.free(u)
            rx.load(u, u)
            for _ in range(n):
                yield ra.free(g)
                ra.load(g, g)
                yield rs.free(g)
                rs.load(g, g)
                yield rb.free(g)
                rb.load(g, g)
                g += 1

    def mma():
        def issue_s(g, u):
            _mma_tile(m, {("x", u % rx_n): u, ("q", g % ra_n): g}, "s", ("s", g))
            m.commit(("s", 0))

        def issue_dp(g, u, last):
            _mma_tile(m, {("x", u % rx_n): u, ("dy", g % rb_n): g}, "dp", ("dp", g))
            m.commit(("dp", 0))
            if last:
                rx.release(u)

        g = 0
        for u, n in enumerate(units):
            yield (rx.landed(u), ra.landed(g))
            issue_s(g, u)
            yield (rb.landed(g),)
            issue_dp(g, u, n == 1)
            for i in range(n):
                more = i + 1 < n
                yield ((("pf", 0), g & 1), ra.landed(g + 1)) if more else ((("pf", 0), g & 1),)
                m.mma(_halves(m, "s", ("p", g)) | {("dy", g % rb_n): g}, "dv", u)
                rb.release(g)
                if more:
                    issue_s(g + 1, u)
                yield ((("ds", 0), g & 1), rb.landed(g + 1)) if more else ((("ds", 0), g & 1),)
                m.mma(_halves(m, "dp", ("ds", g)) | {("q", g % ra_n): g}, "dk", u)
                ra.release(g)
                if more:
                    issue_dp(g + 1, u, i + 2 == n)
                g += 1
            m.commit(("acc", 0))

    def softmax(w):
        g = 0
        for u, n in enumerate(units):
            for _ in range(n):
                yield (rs.landed(g), (("s", 0), g & 1))
                m.check(("st", g % 2), g)
                m.check(("s", w), ("s", g))
                m.mem[("s", w)] = ("p", g)
                m.arrive(("pf", 0))
                yield ((("dp", 0), g & 1),)
                m.check(("dp", w), ("dp", g))
                m.check(("st", g % 2), g)
                m.mem[("dp", w)] = ("ds", g)
                m.arrive(("ds", 0))
                m.arrive(("st_empty", g % 2))
                g += 1
            yield ((("acc", 0), u & 1),)
            yield ()
            m.check("dv", u)
            m.check("dk", u)

    return m.run(dict({w: softmax(w) for w in range(WARPS)}, producer=producer(), mma=mma()))


def _forward(seed, n, stages, bufs, halves):
    m = _Model(seed, {"p": WARPS})
    ring = _Ring(m, "kv", stages)

    def place_v(i):
        return i + (i + bufs if i + bufs < n else n)

    def place_k(i):
        return i if i < bufs else place_v(i - bufs) + 1

    def written(i, h):
        return (("p", h), i & 1) if halves == 2 else (("p", i % bufs), (i // bufs) & 1)

    def formed(i):
        return (("s", i % bufs), (i // bufs) & 1)

    def producer():
        m.load(("q", 0), "q", 0)
        at = 0
        for i in range(-bufs, n):
            for tag in ([("v", i)] if i >= 0 else []) + ([("k", i + bufs)] if i + bufs < n else []):
                yield ring.free(at)
                ring.load(at, tag)
                at += 1

    def mma():
        def issue_s(i):
            j = place_k(i)
            for h in range(halves):
                _mma_tile(m, {"q": 0, ("kv", j % stages): ("k", i)}, ("s", i % bufs, h), ("s", i))
            m.commit(("s", i % bufs))
            ring.release(j)

        for i in range(min(bufs, n)):
            yield ((("q", 0), 0), ring.landed(i))
            issue_s(i)
        for i in range(n):
            more = i + bufs < n
            jv = place_v(i)
            follows = (ring.landed(jv + 1),) if more else ()
            for h in range(halves):
                yield (written(i, h),) + ((ring.landed(jv),) if h == 0 else ()) + (follows if h + 1 == halves else ())
                m.mma(_halves(m, ("s", i % bufs, h), ("p", i)) | {("kv", jv % stages): ("v", i)}, "o", i)
            ring.release(jv)
            if more:
                issue_s(i + bufs)
            else:
                m.commit(("s", i % bufs))

    def softmax(w):
        rnd = random.Random(seed * 7 + w)
        for i in range(n):
            yield (formed(i),)
            for h in range(halves):
                m.check((("s", i % bufs, h), w), ("s", i))
            if rnd.random() < 0.3:          # dead keys: the rows of V are cleared, so it has to be there
                yield (ring.landed(place_v(i)),)
                m.check(("kv", place_v(i) % stages), ("v", i))
            if i > 0 and rnd.random() < 0.3:    # the maximum grows: O is rescaled behind the product before
                yield (formed(i - 1 + bufs),)
                m.check("o", i - 1)
            for h in range(halves):
                yield ()
                m.mem[(("s", i % bufs, h), w)] = ("p", i)
                m.arrive(written(i, h)[0])
        yield (formed(n - 1 + bufs),)
        m.check("o", n - 1)

    return m.run(dict({w: softmax(w) for w in range(WARPS)}, producer=producer(), mma=mma()))


@pytest.mark.parametrize("ra,rb,rx", [(3, 2, 1), (4, 4, 2)])
@pytest.mark.parametrize("units", [[1], [2], [5], [1, 2, 3, 1, 4], [2, 2, 1, 7], [1] * 9])
def test_gradient_hand_offs(ra, rb, rx, units):
    for seed in range(60):
        assert _gradient_q(seed, units, ra, rb, rx, 2) == "ok"
        assert _gradient_kv(seed, units, ra, rb, rx) == "ok"


EMPTY = [[0], [0, 0, 0], [1, 0, 0, 0, 0, 1], [0, 3, 0, 0, 0, 2, 1, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0, 1, 1, 0, 1]]


@pytest.mark.parametrize("ra,rb,rx", [(3, 2, 1), (4, 4, 2)])
@pytest.mark.parametrize("units", EMPTY)
def test_units_without_work(ra, rb, rx, units):
    for seed in range(60):
        assert _gradient_q(seed, units, ra, rb, rx, 2) == "ok"


def test_one_barrier_for_two_ds_tiles_fails():
    ends = set()
    for seed in range(300):
        try:
            ends.add(_gradient_q(seed, [5], 3, 2, 1, 1).split(":")[0])
        except AssertionError:
            ends.add("wrong tile")      # warps arrive for the next tile in place of slower ones
    assert ends == {"ok", "blocked", "wrong tile"}


@pytest.mark.parametrize("stages,bufs,halves", [(5, 2, 1), (2, 1, 2), (4, 1, 1)])
@pytest.mark.parametrize("n", [1, 2, 3, 8])
def test_forward_hand_offs(stages, bufs, halves, n):
    for seed in range(100):
        assert _forward(seed, n, stages, bufs, halves) == "ok"
