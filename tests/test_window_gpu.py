"""Windowed attention, over rows and over pages, on the GPU against the definition
in 64 bits, with a bound for every element.

The bounds are those of the cross attention, with u = eps / 2 of the 16-bit type
and s = 2^-13 for everything fp32 (a score is a sum of d <= 128 products, off by
at most d 2^-24 sum |c q k|, and the inputs keep sum |c q k| <= 16):

    |O err|  <= u |O|  + (u + s) P |V|
    |dV err| <= u |dV| + (u + s) P^T |dY|
    |dQ err| <= u |dQ| + c ((u + s) |dS| |K| + s A |K|)    A = P (|dY| |V|^T + |dY| . |O|)
    |dK err| <= u |dK| + c ((u + s) |dS|^T |Q| + s A^T |Q|)

and products of two small terms are covered by a factor of 1.01.
"""
import math

import pytest
import torch

import sparse_attention_backward_gb300 as sab

pytestmark = pytest.mark.gpu

S32 = 2.0 ** -13
BF, HF = torch.bfloat16, torch.float16
NAN = float("nan")


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


class Case:
    """Inputs of a batch of sequences and the definition in 64 bits."""

    def __init__(self, l1, l2, n1, n2, d, dtype, left, right, padded=False, mask=None, seed=0, grow=1.0, dy_scale=1.0):
        g = torch.Generator().manual_seed(2000 + seed)
        self.l1, self.l2, self.n1, self.n2, self.d, self.dtype, self.padded = l1, l2, n1, n2, d, dtype, padded
        self.left, self.right, self.scale = left, right, d ** -0.5
        self.s1, self.s2, self.cu1, self.cu2 = max(l1), max(l2), _cu(l1), _cu(l2)
        lead1 = (len(l1), self.s1) if padded else (sum(l1),)
        lead2 = (len(l2), self.s2) if padded else (sum(l2),)
        rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.q, self.dy = (rnd(*lead1, n1, d) * grow).to(dtype), (rnd(*lead1, n1, d) * dy_scale).to(dtype)
        self.k, self.v = rnd(*lead2, n2, d).to(dtype), rnd(*lead2, n2, d).to(dtype)
        self.mask = None
        if mask is not None:
            self.mask = torch.rand(lead2, generator=g) >= mask
            self.k[~self.mask], self.v[~self.mask] = NAN, float("inf")
        if padded:      # nothing of the padding may count
            for b in range(len(l1)):
                self.q[b, l1[b]:], self.dy[b, l1[b]:], self.k[b, l2[b]:], self.v[b, l2[b]:] = NAN, NAN, NAN, NAN
                if self.mask is not None:
                    self.mask[b, l2[b]:] = True
        self.q, self.k, self.v, self.dy = (x.cuda() for x in (self.q, self.k, self.v, self.dy))
        if self.mask is not None:
            self.mask = self.mask.cuda()

    def flat(self, x):
        return x.reshape((-1,) + tuple(x.shape[2:])) if self.padded else x

    def parts(self):
        """(rows of q, rows of k, which pairs count, head) of every sequence and query head."""
        for b, (a, n) in enumerate(zip(self.l1, self.l2)):
            i = torch.arange(a, device="cuda") + (b * self.s1 if self.padded else self.cu1[b])
            j = torch.arange(n, device="cuda") + (b * self.s2 if self.padded else self.cu2[b])
            p, c = torch.arange(a, device="cuda")[:, None] + (n - a), torch.arange(n, device="cuda")
            seen = torch.ones(a, n, dtype=torch.bool, device="cuda")
            if self.left >= 0:
                seen &= c >= p - self.left
            if self.right >= 0:
                seen &= c <= p + self.right
            if self.mask is not None:
                seen &= self.mask.reshape(-1)[j]
            for h in range(self.n1):
                yield i, j, seen, h

    def kv(self, j, h):
        n = h // (self.n1 // self.n2)
        k, v = self.flat(self.k)[j, n].double(), self.flat(self.v)[j, n].double()
        if self.mask is not None:
            there = self.mask.reshape(-1)[j][:, None]
            k, v = torch.where(there, k, 0.0), torch.where(there, v, 0.0)
        return n, k, v

    def forward(self):
        q = self.flat(self.q)
        o, mag = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
        for i, j, seen, h in self.parts():
            if not len(i):
                continue
            _, k, v = self.kv(j, h)
            s = (q[i, h].double() @ k.T * self.scale).masked_fill(~seen, -math.inf)
            lse[i, h] = s.logsumexp(1) if len(j) else -math.inf
            p = (s - lse[i, h][:, None]).exp().nan_to_num(0.0)
            o[i, h], mag[i, h] = p @ v, p @ v.abs()
        return o, lse, mag

    def backward(self, o, lse):
        q, dy, o, lse = (self.flat(x) for x in (self.q, self.dy, o, lse))
        z = lambda x: torch.zeros(x.shape, dtype=torch.float64, device="cuda")  # noqa: E731
        dq, dk, dv, tq, tk, tv = z(q), z(self.flat(self.k)), z(self.flat(self.v)), z(q), z(self.flat(self.k)), z(self.flat(self.v))
        u, c = torch.finfo(self.dtype).eps / 2, self.scale
        for i, j, seen, h in self.parts():
            if not len(j) or not len(i):
                continue
            n, kk, vv = self.kv(j, h)
            x, y, w = q[i, h].double(), dy[i, h].double(), o[i, h].double()
            p = torch.where(seen, (x @ kk.T * c - lse[i, h].double()[:, None]).exp(), 0.0)
            ds = p * (y @ vv.T - (y * w).sum(1, keepdim=True))
            a = p * (y.abs() @ vv.abs().T + (y * w).abs().sum(1, keepdim=True))
            dq[i, h] = c * ds @ kk
            dk[j, n] += c * ds.T @ x
            dv[j, n] += p.T @ y
            tq[i, h] = c * ((u + S32) * ds.abs() + S32 * a) @ kk.abs()
            tk[j, n] += c * ((u + S32) * ds.abs() + S32 * a).T @ x.abs()
            tv[j, n] += (u + S32) * p.T @ y.abs()
        return (dq, dk, dv), (tq, tk, tv)

    def args(self):
        return dict(cu_seqlens_q=self.cu1, cu_seqlens_kv=self.cu2, scale=self.scale, left=self.left, right=self.right, key_mask=self.mask)


def _within(name, got, want, tol, dtype):
    u = torch.finfo(dtype).eps / 2
    got = got.double().reshape(want.shape)
    assert bool(torch.isfinite(got).all()), f"{name}: not finite"
    # + half a step of the smallest numbers the type has
    lim = 1.01 * (u * want.abs() + tol) + torch.finfo(dtype).smallest_normal * u
    over = (got - want).abs() - lim
    assert bool((over <= 0).all()), f"{name}: {float(over.max()):.3e} over its bound, at {float(want.abs().max()):.3e}"


def check_forward(c, o, lse):
    wo, wl, mag = c.forward()
    _within("o", o, wo, (torch.finfo(c.dtype).eps / 2 + S32) * mag, c.dtype)
    l = lse.double().reshape(wl.shape)
    empty = wl == -math.inf
    assert torch.equal(l == -math.inf, empty)
    assert bool(((l - wl)[~empty].abs() <= S32 + 2.0 ** -20 * wl[~empty].abs()).all())
    assert bool((o.reshape(wo.shape)[empty] == 0).all())


def run(c):
    o, lse = sab.window_forward(c.q, c.k, c.v, check=True, **c.args())
    check_forward(c, o, lse)
    grads = sab.window_backward(c.q, c.k, c.v, o, c.dy, lse, check=True, **c.args())
    want, tol = c.backward(o, lse)
    for name, x, w, t in zip(("dq", "dk", "dv"), grads, want, tol):
        _within(name, x, w, t, c.dtype)
    return (o, lse) + tuple(grads)


BANDS = [(-1, 0), (63, 0), (0, 0), (127, 0), (128, 0), (5, 9), (-1, 20), (40, -1), (-1, -1), (200, 130), (0, 64)]


@pytest.mark.parametrize("d,dtype", [(64, BF), (64, HF), (128, BF), (128, HF)])
@pytest.mark.parametrize("left,right", BANDS)
def test_windows(d, dtype, left, right):
    run(Case([300, 1, 65, 128], [300, 1, 65, 128], 4, 2, d, dtype, left, right, seed=left + 7))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n1,n2", [(1, 1), (3, 1), (8, 1), (10, 2), (16, 1), (32, 1), (12, 4)])
@pytest.mark.parametrize("left,right", [(-1, 0), (70, 3)])
def test_groups(d, n1, n2, left, right):
    run(Case([211, 77], [211, 77], n1, n2, d, BF, left, right, seed=n1))


@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF)])
@pytest.mark.parametrize("left,right", [(-1, 0), (33, 0), (100, 70)])
@pytest.mark.parametrize("l1,l2", [([1, 1, 1], [1, 200, 700]), ([50, 3], [700, 3]), ([200, 40], [90, 0]), ([0, 130], [5, 131]),
                                   ([257], [256]), ([129, 5], [1000, 129])])
@pytest.mark.parametrize("padded", [False, True])
def test_lengths_that_differ(d, dtype, left, right, l1, l2, padded):
    # new queries behind a context, more queries than keys (whose first rows see nothing), empty sequences
    run(Case(l1, l2, 4, 2, d, dtype, left, right, padded=padded, seed=len(l1)))


@pytest.mark.parametrize("d,dtype", [(64, BF), (128, HF)])
@pytest.mark.parametrize("left,right", [(-1, 0), (50, 0), (90, 31)])
@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("drop", [0.2, 0.97])
def test_masked_keys(d, dtype, left, right, padded, drop):
    c = run(Case([310, 200, 1], [310, 200, 1], 6, 2, d, dtype, left, right, padded=padded, mask=drop, seed=3))
    assert c[0].shape[-1] == d


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("l1,l2,left", [([2500], [2500], -1), ([1500], [4000], 2300), ([300, 280], [4500, 2100], -1)])
def test_long_loops_of_wide_heads(dtype, l1, l2, left):
    run(Case(l1, l2, 16, 8, 128, dtype, left, 0, seed=21))


@pytest.mark.parametrize("d,dtype,n1,n2", [(64, BF, 4, 1), (64, HF, 2, 2), (128, BF, 16, 2), (128, HF, 5, 1)])
@pytest.mark.parametrize("l1,l2,left", [([1], [8000], -1), ([1, 1], [9000, 70], -1), ([3], [6001], 5000), ([40], [12000], -1),
                                        ([2, 0, 5], [7000, 10, 4], -1)])
def test_few_queries_of_long_contexts(d, dtype, n1, n2, l1, l2, left):
    # loops in clusters and in pieces that a second kernel joins
    run(Case(l1, l2, n1, n2, d, dtype, left, 0, seed=5))


# units of few heads and long loops are cut into pieces, some of which have nothing to do, or shared by clusters: the first, of
# the units of dK and dV; the next two of both kernels', or with a cluster for the others; then a cluster for dQ alone
@pytest.mark.parametrize("dtype,drop", [(BF, None), (HF, 0.3)])
@pytest.mark.parametrize("l1,l2,n1,n2,d,left,right", [
    ([1195], [1195], 32, 8, 128, 2000, 0), ([697, 5290], [348, 10580], 1, 1, 64, 1000, -1), ([5327, 2511], [5327, 1255], 1, 1, 128, -1, 0),
    ([705], [1410], 1, 1, 128, -1, 0), ([3000], [3000], 2, 1, 128, -1, 0), ([2500, 300, 0], [2500, 700, 60], 8, 2, 64, -1, 0), ([4100], [4100], 4, 4, 64, 2600, 0),
    ([2000], [2900], 6, 2, 128, -1, 300), ([3500], [1700], 2, 2, 64, -1, 0), ([1800], [1800], 16, 1, 128, 1700, -1)])
def test_gradient_in_pieces(l1, l2, n1, n2, d, dtype, drop, left, right):
    run(Case(l1, l2, n1, n2, d, dtype, left, right, mask=drop, seed=l1[0]))


def test_pieces_are_added_up_in_their_order():
    c = Case([3000], [3000], 8, 2, 128, BF, -1, 0, seed=23)
    o, lse = sab.window_forward(c.q, c.k, c.v, **c.args())
    want = sab.window_backward(c.q, c.k, c.v, o, c.dy, lse, check=True, **c.args())
    for _ in range(20):
        for x, y in zip(want, sab.window_backward(c.q, c.k, c.v, o, c.dy, lse, **c.args())):
            assert torch.equal(x, y)


def test_pieces_of_padded_batches():
    run(Case([1, 3], [6000, 5000], 2, 1, 128, BF, -1, 0, padded=True, mask=0.2, seed=6))


@pytest.mark.parametrize("l1,l2", [([0], [200]), ([200], [0]), ([0, 0], [0, 0]), ([0, 7], [300, 0])])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_sides_without_rows(l1, l2, dtype):
    c = Case(l1, l2, 4, 2, 64, dtype, 30, 0, seed=17)
    o, lse, dq, dk, dv = run(c)
    assert dq.shape == c.q.shape and bool((dk == 0).all()) and bool((dv == 0).all())
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


def test_many_sequences():
    l = [(b * 7) % 40 + 1 for b in range(300)]
    run(Case(l, l, 2, 1, 64, BF, 11, 0, seed=9))


@pytest.mark.parametrize("dtype,scale", [(HF, 2.0 ** 13), (HF, 2.0 ** -13), (BF, 2.0 ** 40)])
def test_loss_scales(dtype, scale):
    run(Case([400], [400], 4, 2, 128, dtype, 90, 0, dy_scale=scale, seed=12))


def test_growing_scores():
    run(Case([500], [500], 4, 2, 128, BF, 200, 0, grow=6.0, seed=13))


def test_no_window_is_the_cross_attention():
    c = Case([300, 70], [500, 70], 4, 2, 128, BF, -1, -1, seed=14)
    o, lse = sab.window_forward(c.q, c.k, c.v, **c.args())
    # (not bit for bit: the two split loops over CTAs by rules of their own, so sums are taken in another order)
    check_forward(c, o, lse)
    check_forward(c, *sab.cross_forward(c.q, c.k, c.v, c.cu1, c.cu2, c.scale))


def test_rows_behind_the_last_sequence_and_strides():
    l = [150, 90]
    c = Case(l, l, 4, 2, 64, BF, 40, 0, seed=15)
    fused = torch.full((300, 8, 64), NAN, dtype=BF, device="cuda")
    fused[:240, :4], fused[:240, 4:6], fused[:240, 6:] = c.q, c.k, c.v
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    o, lse = torch.full((300, 4, 64), 7.0, dtype=BF, device="cuda"), torch.full((300, 4), 7.0, device="cuda")
    sab.window_forward(q, k, v, out=(o, lse), check=True, **c.args())
    assert bool((o[240:] == 7).all()) and bool((lse[240:] == 7).all())
    check_forward(c, o[:240], lse[:240])
    dy = torch.full((300, 4, 64), NAN, dtype=BF, device="cuda")
    dy[:240] = c.dy
    out = tuple(torch.full((300, n, 64), 7.0, dtype=BF, device="cuda") for n in (4, 2, 2))
    sab.window_backward(q, k, v, o, dy, lse, out=out, check=True, **c.args())
    want, tol = c.backward(o[:240], lse[:240])
    for name, x, w, t in zip(("dq", "dk", "dv"), out, want, tol):
        assert bool((x[240:] == 7).all())
        _within(name, x[:240], w, t, BF)


def test_bitwise_and_captured_on_another_stream():
    l = [700, 300]
    c = Case(l, l, 8, 2, 128, HF, 100, 0, mask=0.1, seed=16)
    want = run(c)
    kw = dict(left=100, right=0, dtype=sab.SAG_FP16)
    desc = sab.make_window_desc(c.cu1, c.cu2, 8, 2, 128, c.scale, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.full((max(sab.window_fwd_workspace_size(desc), sab.window_grad_workspace_size(desc)),), 255, dtype=torch.uint8, device="cuda")
    o, lse = sab.window_forward(c.q, c.k, c.v, key_mask=c.mask, desc=desc, workspace=ws, stream=s)
    grads = sab.window_backward(c.q, c.k, c.v, o, c.dy, lse, key_mask=c.mask, desc=desc, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for x, y in zip(want, (o, lse) + grads):
        assert torch.equal(x, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = sab.window_forward(c.q, c.k, c.v, key_mask=c.mask, desc=desc, workspace=ws)
        grads = sab.window_backward(c.q, c.k, c.v, o, c.dy, lse, key_mask=c.mask, desc=desc, workspace=ws)
    for _ in range(3):
        ws.fill_(255)
        g.replay()
        for x, y in zip(want, (o, lse) + grads):
            assert torch.equal(x, y)


@pytest.mark.parametrize("d,dtype", [(64, HF), (128, HF)])
@pytest.mark.parametrize("left,right", [(-1, 0), (7, 4)])
def test_gradient_against_differences(d, dtype, left, right):
    """Central differences, in 64 bits, of sum O dY along the gradient itself; the kernel's bound plus that of its own o and
    lse (o is off by e = u |O| + (u + s) P |V|, which moves dS by P |dY| . e; lse by r = s + 2^-20 |lse|) is what it may be off by."""
    c = Case([30, 9], [30, 40], 4, 2, d, dtype, left, right, seed=36)
    o, lse = sab.window_forward(c.q, c.k, c.v, **c.args())
    got = [x.double() for x in sab.window_backward(c.q, c.k, c.v, o, c.dy, lse, check=True, **c.args())]
    base = [x.double() for x in (c.q, c.k, c.v)]
    g, u = c.n1 // c.n2, torch.finfo(dtype).eps / 2

    def value(x):
        total = 0.0
        for i, j, seen, h in c.parts():
            s = (x[0][i, h] @ x[1][j, h // g].T * c.scale).masked_fill(~seen, -math.inf)
            total = total + ((s.softmax(1).nan_to_num(0.0) @ x[2][j, h // g]) * c.dy[i, h].double()).sum()
        return total

    leaves = [x.clone().requires_grad_() for x in base]
    want = torch.autograd.grad(value(leaves), leaves)
    lim = [torch.zeros_like(x) for x in base]
    for i, j, seen, h in c.parts():
        n, kk, vv = c.kv(j, h)
        x, y = base[0][i, h], c.dy[i, h].double()
        sc = (x @ kk.T * c.scale).masked_fill(~seen, -math.inf)
        p, r = sc.softmax(1), S32 + 2.0 ** -20 * sc.logsumexp(1, keepdim=True).abs()
        w = p @ vv
        ds = p * (y @ vv.T - (y * w).sum(1, keepdim=True))
        a = p * (y.abs() @ vv.abs().T + (y * w).abs().sum(1, keepdim=True))
        moved = p * (y.abs() * (u * w.abs() + (u + S32) * (p @ vv.abs()))).sum(1, keepdim=True)
        ds = (u + S32 + r) * ds.abs() + S32 * a + moved
        lim[0][i, h] = c.scale * ds @ kk.abs()
        lim[1][j, n] += c.scale * ds.T @ x.abs()
        lim[2][j, n] += ((u + S32 + r) * p).T @ y.abs()
    for at, name in enumerate(("dq", "dk", "dv")):
        bound = 1.01 * (u * want[at].abs() + lim[at]) + 2.0 ** -25
        assert float(bound.norm()) < 0.1 * float(want[at].norm())       # zeros would fail
        assert bool(((got[at] - want[at]).abs() <= bound).all()), name
        e, h = want[at] / want[at].norm(), 1e-3
        up, down = list(base), list(base)
        up[at], down[at] = base[at] + h * e, base[at] - h * e
        diff = float(value(up) - value(down)) / (2 * h)
        allowed = float((bound * e.abs()).sum())
        assert allowed < 0.1 * abs(diff)
        assert abs(float((got[at] * e).sum()) - diff) <= allowed + 1e-4 * abs(diff), name


def test_offsets_beyond_32_bits():
    """A sequence behind one of so many tokens that elements and bytes before it pass 32 bits."""
    c, rows = Case([300], [300], 16, 16, 128, BF, 63, 0, seed=40), 2 ** 20 + 70000
    assert rows * 16 * 128 > 2 ** 31
    cu = [0, rows - 300, rows]

    def behind(x):
        big = torch.zeros(rows, 16, 128, dtype=BF, device="cuda")
        big[-300:] = x
        return big

    q, k, v, dy = (behind(x) for x in (c.q, c.k, c.v, c.dy))
    o, lse = sab.window_forward(q, k, v, cu, cu, c.scale, left=63, check=True)
    check_forward(c, o[-300:], lse[-300:])
    assert bool((o[:-300:4099] == 0).all())
    grads = sab.window_backward(q, k, v, o, dy, lse, cu, cu, c.scale, left=63, check=True)
    want, tol = c.backward(o[-300:], lse[-300:])
    for name, x, w, t in zip(("dq", "dk", "dv"), grads, want, tol):
        _within(name, x[-300:], w, t, BF)
        assert bool((x[:-300:4099] == 0).all())


# ------------------------------------------------------------------- pages
class Pages:
    """A case's keys and values in shuffled pages of a cache that holds NaN elsewhere, and a table with junk where nothing
    has to look."""

    def __init__(self, c, page, extra=3, strided=False, seed=0):
        g = torch.Generator().manual_seed(300 + seed)
        counts = [-(-n // page) for n in c.l2]
        self.width = max(counts) + 2
        pages = sum(counts) + extra
        shape = (pages, 2, page, c.n2, c.d) if strided else (2, pages, page, c.n2, c.d)
        both = torch.full(shape, NAN, dtype=c.dtype, device="cuda")
        self.k, self.v = (both[:, 0], both[:, 1]) if strided else (both[0], both[1])
        order = torch.randperm(pages, generator=g).tolist()
        self.table = torch.randint(-2 ** 31, 2 ** 31 - 1, (len(c.l2), self.width), generator=g, dtype=torch.int64).to(torch.int32)
        for b, n in enumerate(c.l2):
            off = c.l2[b] - c.l1[b]
            first = max(0, off - c.left) if c.left >= 0 else 0       # keys before the first window need no page
            for p in range(counts[b]):
                if (p + 1) * page <= first:
                    continue
                at = order.pop()
                self.table[b, p] = at
                lo, hi = p * page, min(n, (p + 1) * page)
                src = (b, slice(lo, hi)) if c.padded else slice(c.cu2[b] + lo, c.cu2[b] + hi)
                self.k[at, :hi - lo], self.v[at, :hi - lo] = c.k[src], c.v[src]
                if lo < first:                                       # part of a page that no window holds
                    self.k[at, :first - lo] = self.v[at, :first - lo] = NAN
        self.table, self.lens = self.table.cuda(), torch.tensor(c.l2, dtype=torch.int32, device="cuda")

    def forward(self, c, **kw):
        return sab.paged_forward(c.q, self.k, self.v, self.table, self.lens, c.cu1, c.scale, c.left, c.right, check=True, **kw)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("d,dtype", [(64, BF), (64, HF), (128, BF), (128, HF)])
@pytest.mark.parametrize("left", [-1, 70])
def test_paged(page, d, dtype, left):
    c = Case([1, 65, 200, 3, 0], [300, 65, 513, 1024, 40], 4, 2, d, dtype, left, 0, seed=page)
    check_forward(c, *Pages(c, page).forward(c))


@pytest.mark.parametrize("page", [16, 80, 64])
@pytest.mark.parametrize("n1,n2", [(1, 1), (6, 2), (16, 1), (32, 1)])
@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("left,right", [(-1, 0), (0, 0), (150, -1), (-1, 5)])
def test_paged_groups(page, n1, n2, padded, left, right):
    c = Case([1, 40, 130], [129, 40, 400], n1, n2, 128, BF, left, right, padded=padded, seed=n1)
    check_forward(c, *Pages(c, page, strided=padded).forward(c))


@pytest.mark.parametrize("d,dtype,n1,n2", [(64, HF, 4, 1), (128, BF, 16, 2), (128, HF, 3, 3)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("l1,l2,left", [([1], [9000], -1), ([1, 1], [7000, 0], -1), ([1, 2], [33, 9001], 4000), ([5], [2], -1)])
def test_paged_tokens_of_long_contexts(d, dtype, n1, n2, page, l1, l2, left):
    c = Case(l1, l2, n1, n2, d, dtype, left, 0, seed=3)
    check_forward(c, *Pages(c, page).forward(c))


@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_paged_long_loops(page, dtype):
    c = Case([700, 300], [4000, 2500], 16, 8, 128, dtype, -1, 0, seed=22)
    check_forward(c, *Pages(c, page).forward(c))


def test_paged_is_the_windowed_attention():
    c = Case([100, 64], [500, 640], 8, 2, 128, BF, -1, 0, seed=4)
    check_forward(c, *Pages(c, 64).forward(c))
    check_forward(c, *sab.window_forward(c.q, c.k, c.v, **c.args()))


def test_no_new_tokens():
    c = Case([0, 0], [30, 40], 4, 2, 64, BF, -1, 0, seed=18)
    p = Pages(c, 16)
    before = p.k.clone()
    o, lse = p.forward(c)
    assert o.shape == c.q.shape
    sab.paged_append(c.q[:, :2], c.q[:, :2], p.k, p.v, p.table, p.lens, c.cu1, check=True)
    assert torch.equal(p.k.nan_to_num(0.0), before.nan_to_num(0.0))


def test_expected_length_only_splits_the_work():
    c = Case([1, 3], [6000, 4000], 4, 2, 128, BF, -1, 0, seed=19)
    p = Pages(c, 64)
    for expected in (0, 64, 1000, 6000, 2 ** 31 - 1):
        desc = sab.make_paged_desc(c.cu1, 4, 2, 128, c.scale, p.k.shape[0], 64, p.width, kv_expected=expected)
        check_forward(c, *sab.paged_forward(c.q, p.k, p.v, p.table, p.lens, desc=desc, check=True))


def test_many_paged_sequences():
    c = Case([1] * 200, [(b * 13) % 90 for b in range(200)], 4, 2, 64, BF, -1, 0, seed=8)
    check_forward(c, *Pages(c, 16).forward(c))


def test_captured_step_follows_growing_sequences():
    c = Case([1, 1], [700, 130], 4, 2, 128, BF, -1, 0, seed=5)
    p = Pages(c, 32)
    desc = sab.make_paged_desc(c.cu1, 4, 2, 128, c.scale, p.k.shape[0], 32, p.width)
    ws = torch.zeros(sab.paged_fwd_workspace_size(desc), dtype=torch.uint8, device="cuda")
    full, table = p.lens.clone(), p.table.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = sab.paged_forward(c.q, p.k, p.v, p.table, p.lens, workspace=ws, desc=desc)
    for cut in (300, 129, 0):
        for b in range(2):
            c.l2[b] = max(int(full[b]) - cut, 0)
        p.lens.copy_(torch.tensor(c.l2, dtype=torch.int32))
        p.table.copy_(table)
        ws.fill_(255)
        g.replay()
        check_forward(c, o, lse)


@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length"])
def test_pages_and_lengths_out_of_range_are_reported(what):
    c = Case([3, 1], [200, 100], 4, 2, 128, BF, -1, 0, seed=6)
    p = Pages(c, 32)
    if what == "length":
        p.table[1] = 0
        p.lens[1] = p.width * 32 + 1
    elif what == "negative length":
        p.lens[1] = -5
    else:
        p.table[0, 2] = p.k.shape[0] if what == "page" else -1
    with pytest.raises(sab.SagError) as e:
        p.forward(c)
    assert e.value.status == sab.SAG_ERR_INDEX
    torch.cuda.synchronize()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("page,n2,d", [(16, 1, 64), (32, 2, 128), (48, 3, 64), (128, 8, 192), (16, 5, 8)])
@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("strided", [False, True])
def test_append(dtype, page, n2, d, padded, strided):
    l1, l2 = [1, 70, 0, 33, 9], [200, 70, 30, 60, 4]       # the last: five positions before 0
    g = torch.Generator().manual_seed(page + d)
    lead = (5, 70) if padded else (sum(l1) + 2,)
    k, v = (torch.randn(*lead, n2, d, generator=g).to(dtype).cuda() for _ in range(2))
    if strided:
        wide = torch.stack((k, v), -3)
        k, v = wide[..., 0, :, :], wide[..., 1, :, :]
    width = 14
    pages = 40
    both = torch.randn(pages, 2, page, n2, d, generator=g).to(dtype).cuda()
    kc, vc = (both[:, 0], both[:, 1]) if strided else (both[:, 0].contiguous(), both[:, 1].contiguous())
    table = torch.full((5, width), -9, dtype=torch.int32)
    order = torch.randperm(pages, generator=g).tolist()
    for b in range(5):
        for p in range(-(-l2[b] // page)):
            table[b, p] = order.pop()
    wk, wv = kc.clone(), vc.clone()
    cu = _cu(l1)
    for b in range(5):
        for i in range(l1[b]):
            at = l2[b] - l1[b] + i
            if at >= 0:
                row = (b, i) if padded else cu[b] + i
                wk[table[b, at // page], at % page], wv[table[b, at // page], at % page] = k[row], v[row]
    lens = torch.tensor(l2, dtype=torch.int32, device="cuda")
    got = sab.paged_append(k, v, kc, vc, table.cuda(), lens, cu, check=True)
    assert got[0] is kc and got[1] is vc
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    before = kc.clone()
    bad = table.clone()
    bad[1, 0] = pages
    with pytest.raises(sab.SagError) as e:      # its tokens are not written
        sab.paged_append(k, v, kc, vc, bad.cuda(), lens, cu, check=True)
    assert e.value.status == sab.SAG_ERR_INDEX and torch.equal(kc, before)


def test_pages_beyond_32_bits():
    """Pages whose elements and bytes pass 32 bits, written by the append and read by the attention."""
    c, pages = Case([5, 130], [400, 900], 8, 2, 128, HF, -1, 0, seed=41), 600000
    p = Pages(c, 16)
    big = [torch.empty(pages, 16, 2, 128, dtype=HF, device="cuda") for _ in range(2)]
    assert big[0].numel() > 2 ** 31
    table = torch.where(p.table >= 0, p.table, 0)           # (entries that nothing looks at hold any number)
    for b, n in enumerate(c.l2):
        used = p.table[b, :-(-n // 16)].long()
        far = pages - 1 - used * 1000                       # over all of the cache
        big[0][far], big[1][far] = p.k[used], p.v[used]
        table[b, :len(far)] = far.int()
        for at in range(n - c.l1[b], n):
            big[0][far[at // 16], at % 16] = big[1][far[at // 16], at % 16] = NAN
    new = torch.cat([torch.arange(c.cu2[b + 1] - c.l1[b], c.cu2[b + 1]) for b in range(2)]).cuda()
    sab.paged_append(c.k[new], c.v[new], *big, table, p.lens, c.cu1, check=True)
    check_forward(c, *sab.paged_forward(c.q, *big, table, p.lens, c.cu1, c.scale, check=True))


def test_append_of_many_sequences_then_attention():
    """The step as a server takes it: append, then attend, against the attention over rows."""
    b, page = 90, 16
    c = Case([1 + i % 3 for i in range(b)], [5 + (i * 37) % 200 for i in range(b)], 4, 2, 128, BF, -1, 0, seed=7)
    p = Pages(c, page)
    new_k, new_v = torch.empty(sum(c.l1), 2, 128, dtype=BF, device="cuda"), torch.empty(sum(c.l1), 2, 128, dtype=BF, device="cuda")
    for i in range(b):
        src = slice(c.cu2[i + 1] - c.l1[i], c.cu2[i + 1])
        new_k[c.cu1[i]:c.cu1[i + 1]], new_v[c.cu1[i]:c.cu1[i + 1]] = c.k[src], c.v[src]
        for at in range(c.l2[i] - c.l1[i], c.l2[i]):
            p.k[p.table[i, at // page], at % page] = NAN
            p.v[p.table[i, at // page], at % page] = NAN
    desc = sab.make_paged_desc(c.cu1, 4, 2, 128, c.scale, p.k.shape[0], page, p.width)
    sab.paged_append(new_k, new_v, p.k, p.v, p.table, p.lens, desc=desc, check=True)
    o, lse = sab.paged_forward(c.q, p.k, p.v, p.table, p.lens, desc=desc, check=True)
    check_forward(c, o, lse)
