"""Cross attention on the GPU against the definition in 64 bits, with a bound
for every element.

With u = eps / 2 of the 16-bit type (half a step) and s = 2^-13 for everything
fp32 (a score is a sum of d <= 128 products, off by at most d 2^-24 sum |c q k|,
and the inputs keep sum |c q k| <= 16; exp turns that into a relative error):

    |O err|  <= u |O|  + (u + s) P |V|                   P rounded, O rounded
    |dV err| <= u |dV| + (u + s) P^T |dY|
    |dQ err| <= u |dQ| + c ((u + s) |dS| |K| + s A |K|)    A = P (|dY| |V|^T + |dY| . |O|): what dS is a difference of
    |dK err| <= u |dK| + c ((u + s) |dS|^T |Q| + s A^T |Q|)

Products of two small terms are covered by a factor of 1.01.
"""
import math

import pytest
import torch

import sparse_attention_backward_gb300 as sab

pytestmark = pytest.mark.gpu

S32 = 2.0 ** -13


class Case:
    """Inputs of a batch of sequences (CPU tensors) and the definition in 64 bits."""

    def __init__(self, l1, l2, n1, n2, d, dtype, padded=False, mask=None, seed=0, scale=None, grow=1.0, dy_scale=1.0):
        g = torch.Generator().manual_seed(1000 + seed)
        self.l1, self.l2, self.n1, self.n2, self.d, self.dtype, self.padded = l1, l2, n1, n2, d, dtype, padded
        self.scale = d ** -0.5 if scale is None else scale
        self.s1, self.s2 = max(l1), max(l2)
        self.cu1, self.cu2 = self._cu(l1), self._cu(l2)
        lead1 = (len(l1), self.s1) if padded else (sum(l1),)
        lead2 = (len(l2), self.s2) if padded else (sum(l2),)
        rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.q, self.dy = (rnd(*lead1, n1, d) * grow).to(dtype), (rnd(*lead1, n1, d) * dy_scale).to(dtype)
        self.k, self.v = rnd(*lead2, n2, d).to(dtype), rnd(*lead2, n2, d).to(dtype)
        self.mask = None
        if mask is not None:
            self.mask = torch.rand(lead2, generator=g) >= mask
            self.k[~self.mask], self.v[~self.mask] = float("nan"), float("inf")
        if padded:      # nothing of the padding may count
            for b in range(len(l1)):
                self.q[b, l1[b]:], self.dy[b, l1[b]:] = float("nan"), float("nan")
                self.k[b, l2[b]:], self.v[b, l2[b]:] = float("nan"), float("nan")
                if self.mask is not None:
                    self.mask[b, l2[b]:] = True

    @staticmethod
    def _cu(lens):
        out = [0]
        for n in lens:
            out.append(out[-1] + n)
        return out

    def parts(self):
        """(rows of q, rows of k that are there, head) of every sequence and query head."""
        for b in range(len(self.l1)):
            i = torch.arange(self.l1[b]) + (b * self.s1 if self.padded else self.cu1[b])
            j = torch.arange(self.l2[b]) + (b * self.s2 if self.padded else self.cu2[b])
            if self.mask is not None:
                j = j[self.mask.reshape(-1)[j]]
            for h in range(self.n1):
                yield i, j, h

    def flat(self, x):
        return x.reshape((-1,) + tuple(x.shape[2:])) if self.padded else x

    def forward(self):
        q, k, v = (self.flat(x) for x in (self.q, self.k, self.v))
        o, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
        lse = torch.zeros(q.shape[:2], dtype=torch.float64)
        for i, j, h in self.parts():
            n = h // (self.n1 // self.n2)
            s = q[i, h].double() @ k[j, n].double().T * self.scale
            lse[i, h] = s.logsumexp(1)
            p = s.softmax(1)
            o[i, h], mag[i, h] = p @ v[j, n].double(), p @ v[j, n].double().abs()
        return o, lse, mag

    def backward(self, o, lse):
        q, k, v, dy = (self.flat(x) for x in (self.q, self.k, self.v, self.dy))
        o, lse = self.flat(o), self.flat(lse)
        z = lambda x: torch.zeros(x.shape, dtype=torch.float64)  # noqa: E731
        dq, dk, dv, tq, tk, tv = z(q), z(k), z(v), z(q), z(k), z(v)
        u = torch.finfo(self.dtype).eps / 2
        c = self.scale
        for i, j, h in self.parts():
            if not len(j) or not len(i):
                continue
            n = h // (self.n1 // self.n2)
            x, y, w, kk, vv = q[i, h].double(), dy[i, h].double(), o[i, h].double(), k[j, n].double(), v[j, n].double()
            p = (x @ kk.T * c - lse[i, h].double()[:, None]).exp()
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
        return dict(key_mask=None if self.mask is None else self.mask.cuda())


def _within(name, got, want, tol, dtype):
    u = torch.finfo(dtype).eps / 2
    got = got.cpu().double().reshape(want.shape)
    assert bool(torch.isfinite(got).all()), f"{name}: not finite"
    # + half a step of the smallest numbers the type has
    lim = 1.01 * (u * want.abs() + tol) + torch.finfo(dtype).smallest_normal * u
    over = (got - want).abs() - lim
    assert bool((over <= 0).all()), f"{name}: {float(over.max()):.3e} over its bound, at {float(want.abs().max()):.3e}"


def run(c, check=True):
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    o, lse = sab.cross_forward(q, k, v, c.cu1, c.cu2, c.scale, check=check, **c.args())
    wo, wl, mag = c.forward()
    u = torch.finfo(c.dtype).eps / 2
    _within("o", o, wo, (u + S32) * mag, c.dtype)
    l = lse.cpu().double().reshape(wl.shape)
    empty = wl == -math.inf
    assert torch.equal(l == -math.inf, empty)
    assert bool(((l - wl)[~empty].abs() <= S32 + 2.0 ** -20 * wl[~empty].abs()).all())
    dq, dk, dv = sab.cross_backward(q, k, v, o, c.dy.cuda(), lse, c.cu1, c.cu2, c.scale, check=check, **c.args())
    want, tol = c.backward(o.cpu(), lse.cpu())
    for name, x, w, t in zip(("dq", "dk", "dv"), (dq, dk, dv), want, tol):
        _within(name, x, w, t, c.dtype)
    return o, lse, dq, dk, dv


BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("l1,l2", [
    ([1], [1]), ([1], [577]), ([128], [128]), ([129], [127]), ([300], [129]), ([257], [1000]), ([2], [4097]),
])
def test_one_sequence(dtype, d, l1, l2):
    run(Case(l1, l2, 4, 4, d, dtype))


@pytest.mark.parametrize("n1,n2", [(1, 1), (8, 2), (6, 2), (5, 1), (32, 1), (24, 8), (7, 1), (31, 1), (16, 16)])
@pytest.mark.parametrize("padded", [False, True])
def test_groups_and_layouts(n1, n2, padded):
    run(Case([33, 0, 140, 1], [70, 129, 0, 300], n1, n2, 64 if n1 % 2 else 128, BF if n2 > 1 else HF, padded=padded, seed=n1))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("drop", [0.1, 0.9, 1.0])
def test_masked_states(dtype, padded, drop):
    # nine of ten: whole key tiles away; all: every row empty
    run(Case([20, 150], [400, 137], 6, 2, 128, dtype, padded=padded, mask=drop))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("l1,l2", [([200], [3000]), ([40], [20000]), ([6000], [77]), ([3000, 1000], [130, 20])])
def test_loops_split_over_a_cluster(d, l1, l2):
    # few tiles on one side: the CTAs of a cluster share the loop over the other
    run(Case(l1, l2, 2, 1, d, BF))


def test_long_fp16_probabilities_and_loss_scales():
    # P around 1 / 30000 lies under fp16's normal range, dY around 3000 makes dP overflow it
    run(Case([64], [30000], 2, 1, 64, HF, dy_scale=1.0))
    run(Case([64], [600], 2, 1, 64, HF, dy_scale=3000.0))
    run(Case([64], [600], 2, 1, 64, HF, dy_scale=2.0 ** -12))


def test_growing_maximum():
    # scores of a wide range, ordered so that the maximum grows from tile to tile
    c = Case([130], [1024], 2, 2, 64, BF, grow=1.0)
    ramp = torch.linspace(0.05, 3.0, 1024)[:, None, None]
    c.k = (torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(3)) * ramp).to(BF).contiguous()
    c.q = (c.q * 0.3).to(BF)
    run(c)


def test_gradient_against_differences():
    # fp16 inputs, central differences of <dY, O> in 64 bits along random directions of q, k and v
    c = Case([9, 20], [33, 60], 4, 2, 64, HF, seed=5)
    o, lse, dq, dk, dv = run(c)
    g = torch.Generator().manual_seed(9)
    base = [c.q.double(), c.k.double(), c.v.double()]

    def value(x):
        save = c.q, c.k, c.v
        c.q, c.k, c.v = x
        w = (c.forward()[0] * c.dy.double()).sum()
        c.q, c.k, c.v = save
        return float(w)

    # the bound adds up the elements' bounds; differences of step h are off by O(h^2), far below
    want, tol = c.backward(o.cpu(), lse.cpu())
    u, h = 2.0 ** -11, 1e-4
    for at, (grad, t, w) in enumerate(zip((dq, dk, dv), tol, want)):
        e = torch.randn(base[at].shape, generator=g, dtype=torch.float64)
        up, down = list(base), list(base)
        up[at], down[at] = base[at] + h * e, base[at] - h * e
        diff = (value(up) - value(down)) / (2 * h)
        got = float((grad.cpu().double() * e).sum())
        # Delta comes from the rounded o: off by u |dY||O|, which moves dS by P times that
        lim = float(((1.01 * (u * w.abs() + t) + u * 16 * w.abs().mean()) * e.abs()).sum())
        assert abs(got - diff) <= lim + 1e-5 * abs(diff)


def test_bitwise_repeatable():
    c = Case([500, 70], [900, 2000], 8, 2, 128, BF, seed=2)
    a = run(c)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, run(c, check=False)))


def test_strided_rows_of_fused_projections():
    c = Case([150, 33], [220, 64], 8, 2, 64, BF, seed=6)
    want = run(c)
    qx = torch.full((183, 12, 64), float("nan"), dtype=BF)
    qx[:, 2:10] = c.q
    kv = torch.full((284, 2, 2, 64), float("nan"), dtype=BF)
    kv[:, 0], kv[:, 1] = c.k, c.v
    q, kv = qx.cuda()[:, 2:10], kv.cuda()
    k, v = kv[:, 0], kv[:, 1]
    o, lse = sab.cross_forward(q, k, v, c.cu1, c.cu2, c.scale)
    grads = sab.cross_backward(q, k, v, o, c.dy.cuda(), lse, c.cu1, c.cu2, c.scale)
    assert all(torch.equal(x, y) for x, y in zip((o, lse) + grads, want))


def test_rows_behind_the_last_sequence_are_left_alone():
    c = Case([60, 10], [50, 200], 4, 2, 64, BF, seed=7)
    want = run(c)
    more = lambda x, n: torch.cat([x, torch.full((n,) + tuple(x.shape[1:]), float("nan"), dtype=x.dtype)]).cuda()  # noqa: E731
    q, k, v, dy = more(c.q, 5), more(c.k, 3), more(c.v, 3), more(c.dy, 5)
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    sab.cross_forward(q, k, v, c.cu1, c.cu2, c.scale, out=(o, lse))
    outs = tuple(torch.full_like(x, 7.0) for x in (q, k, v))
    sab.cross_backward(q, k, v, o, dy, lse, c.cu1, c.cu2, c.scale, out=outs)
    for x, w in zip((o, lse) + outs, want):
        assert torch.equal(x[:len(w)], w) and bool((x[len(w):] == 7.0).all())


@pytest.mark.parametrize("batch", [64, 65, 1100])
def test_many_sequences(batch):
    l1 = [(b * 3) % 5 for b in range(batch)]
    l2 = [(b * 5) % 9 for b in range(batch)]
    run(Case(l1, l2, 2, 1, 64, BF, seed=batch))


@pytest.mark.parametrize("l1,l2", [([0, 0], [5, 7]), ([3, 4], [0, 0]), ([0], [0])])
def test_a_side_without_rows(l1, l2):
    c = Case(l1, l2, 2, 1, 64, BF)
    o, lse, dq, dk, dv = run(c)
    assert not any(x.any() for x in (o, dq, dk, dv))


def test_streams_workspaces_and_graphs():
    a, b = Case([200], [900], 4, 2, 128, BF, seed=8), Case([90, 5], [300, 40], 4, 4, 64, HF, seed=9)
    wants = [run(a), run(b)]
    # two calls at once on streams and workspaces of their own
    streams = [torch.cuda.Stream() for _ in range(2)]
    tensors = [tuple(x.cuda() for x in (c.q, c.k, c.v, c.dy)) for c in (a, b)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = []
        for c, st, (q, k, v, dy) in zip((a, b), streams, tensors):
            o, lse = sab.cross_forward(q, k, v, c.cu1, c.cu2, c.scale, stream=st)
            got.append((o, lse) + sab.cross_backward(q, k, v, o, dy, lse, c.cu1, c.cu2, c.scale, stream=st))
    torch.cuda.synchronize()
    for w, g in zip(wants, got):
        assert all(torch.equal(x, y) for x, y in zip(w, g))
    # both captured into graphs that share one workspace and are replayed one after the other, on changed inputs
    descs = [sab.make_cross_desc(c.cu1, c.cu2, c.n1, c.n2, c.d, c.scale, sab.SAG_FP16 if c.dtype == HF else sab.SAG_BF16)
             for c in (a, b)]
    ws = torch.empty(max(sab.cross_grad_workspace_size(x) for x in descs), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for c, desc, (q, k, v, dy) in zip((a, b), descs, tensors):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = sab.cross_forward(q, k, v, workspace=ws, desc=desc)
            outs.append((o, lse) + sab.cross_backward(q, k, v, o, dy, lse, workspace=ws, desc=desc))
        graphs.append(g)
    for q, _, _, _ in tensors:
        q.neg_()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for c, (q, k, v, dy), o in zip((a, b), tensors, outs):
        c.q = q.cpu()
        assert all(torch.equal(x, y) for x, y in zip(run(c), o))


def test_large_batch_captured():
    # a table too large for the kernel parameters is part of the captured call as well
    l1, l2 = [1] * 300, [(b % 7) + 1 for b in range(300)]
    c = Case(l1, l2, 2, 1, 64, BF, seed=11)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    want = run(c)
    desc = sab.make_cross_desc(c.cu1, c.cu2, 2, 1, 64, c.scale)
    ws = torch.zeros(sab.cross_fwd_workspace_size(desc), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = sab.cross_forward(q, k, v, workspace=ws, desc=desc)
    ws.fill_(255)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("drop", [None, 0.2])
@pytest.mark.parametrize("l1,l2", [([300], [2100]), ([200, 64], [5000, 2300]), ([260], [9000])])
def test_long_loops_of_wide_heads(dtype, drop, l1, l2):
    # full query tiles and at least 2048 keys: the forward's tiles of 128 keys
    run(Case(l1, l2, 16, 8, 128, dtype, mask=drop, seed=21))


def test_growing_maximum_in_long_loops():
    # every few tiles the maximum grows beyond the lazy reference, in either half of a tile
    c = Case([256], [4096], 16, 8, 128, BF, seed=22)
    ramp = torch.linspace(0.02, 2.5, 4096)[:, None, None]
    ramp = ramp.reshape(64, 64, 1, 1)[torch.arange(64) ^ 1].reshape(4096, 1, 1)      # the larger half first
    c.k = (torch.randn(1, 8, 128, generator=torch.Generator().manual_seed(4)) * ramp).to(BF).contiguous()
    c.q = (c.q * 0.4).to(BF)
    run(c)


# units beyond full rounds of 152 SMs, with loops long enough that they are cut: (key tiles, query tiles, both kernels'
# last round, no full round before it)
@pytest.mark.parametrize("dtype,drop", [(BF, None), (HF, 0.3)])
@pytest.mark.parametrize("l1,l2,n1,n2,d", [
    ([2000], [1280], 16, 16, 128), ([640], [2000], 32, 16, 128), ([1050, 1100], [2100, 2050], 32, 8, 64),
    ([8192], [1300], 8, 8, 64)])
def test_last_units_in_pieces(dtype, drop, l1, l2, n1, n2, d):
    run(Case(l1, l2, n1, n2, d, dtype, mask=drop, seed=l1[0]))


def test_pieces_are_added_up_in_their_order():
    c = Case([2048], [1280], 16, 16, 128, BF, seed=5)
    q, k, v, dy = (x.cuda() for x in (c.q, c.k, c.v, c.dy))
    o, lse = sab.cross_forward(q, k, v, c.cu1, c.cu2, c.scale)
    want = sab.cross_backward(q, k, v, o, dy, lse, c.cu1, c.cu2, c.scale, check=True)
    for _ in range(20):
        for x, y in zip(want, sab.cross_backward(q, k, v, o, dy, lse, c.cu1, c.cu2, c.scale)):
            assert torch.equal(x, y)


def test_pieces_without_work():
    # all states of one sequence masked, and a piece's whole share of the other's
    c = Case([2048, 2040], [640, 640], 16, 16, 64, BF, mask=0.0, seed=6)
    c.mask[:640] = False
    c.k[:640], c.v[:640] = float("nan"), float("inf")
    run(c)
    c = Case([640], [2048], 32, 16, 64, HF, mask=0.0, seed=7)
    c.mask[1024:] = False
    c.k[1024:], c.v[1024:] = float("nan"), float("inf")
    run(c)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (HF, 64), (BF, 128), (HF, 128)])
@pytest.mark.parametrize("what", ["states", "far", "value"])
@pytest.mark.parametrize("l1,l2,first,last", [
    ([3], [64], 16, 37), ([3], [577], 144, 336), ([3], [577], 128, 192), ([130], [577], 128, 192), ([256], [4097], 1024, 2048)])
def test_nan_in_states_that_are_there(dtype, d, what, l1, l2, first, last):
    # loops split over a cluster, where in the last three cases some CTAs see these states and no others: every score is NaN
    # ("states"), or one is and the others lie so far below the maximum that their share underflows ("far"), or a column of V
    # is NaN there ("value")
    c = Case(l1, l2, 4, 2, d, dtype, seed=31)
    there = slice(first, last)
    c.q, c.k = torch.ones_like(c.q), torch.zeros_like(c.k)
    if what != "states":
        c.k[there] = -20.0          # scores of -20 sqrt(d): 2^-230 of the others and less
    if what == "value":
        c.v[there, :, 5] = float("nan")
    else:
        c.k[there if what == "states" else first, 0] = float("nan")
    o, lse = sab.cross_forward(c.q.cuda(), c.k.cuda(), c.v.cuda(), c.cu1, c.cu2, c.scale, check=True)
    wo, wl, mag = c.forward()
    o, lse = o.cpu(), lse.cpu()
    assert torch.equal(lse.isnan(), wl.isnan()) and torch.equal(o.isnan(), wo.isnan())
    assert bool(wo.isnan().any()) and not bool(wo.isnan().all())
    u = torch.finfo(dtype).eps / 2
    _within("o", o.nan_to_num(0.0), wo.nan_to_num(0.0), (u + S32) * mag.nan_to_num(0.0), dtype)
    assert bool(((lse - wl).nan_to_num(0.0).abs() <= S32 + 2.0 ** -20 * wl.nan_to_num(0.0).abs()).all())


# a cluster's unit, whole units, pieces
@pytest.mark.parametrize("l1,l2,n1,n2,d", [([64], [30000], 2, 1, 64), ([640], [1500], 16, 16, 128), ([640], [3001], 32, 16, 128)])
def test_rows_of_small_output_gradients_in_fp16(l1, l2, n1, n2, d):
    """dY rows that differ by 2^18 in one sequence: each row of dQ keeps its bits.

    Rounding dS (u of each, independent) gives a row an error of at most u c sqrt(sum_j dS_j^2 |K_j|^2) in the root mean
    square, the fp32 part s c sqrt(sum_j A_j^2 |K_j|^2); four times that, plus the rounding of dQ itself."""
    c = Case(l1, l2, n1, n2, d, HF, seed=33)
    spread = 2.0 ** (13 - 18 * torch.arange(l1[0]) / (l1[0] - 1))
    spread = spread[torch.randperm(l1[0], generator=torch.Generator().manual_seed(34))]
    c.dy = (torch.randn(c.dy.shape, generator=torch.Generator().manual_seed(35)) * spread[:, None, None]).to(HF)
    q, k, v, dy = (x.cuda() for x in (c.q, c.k, c.v, c.dy))
    o, lse = sab.cross_forward(q, k, v, c.cu1, c.cu2, c.scale)
    got = sab.cross_backward(q, k, v, o, dy, lse, c.cu1, c.cu2, c.scale, check=True)
    o, lse = o.cpu(), lse.cpu()
    want, tol = c.backward(o, lse)
    for name, x, w, t in zip(("dq", "dk", "dv"), got, want, tol):
        _within(name, x, w, t, HF)
    u = 2.0 ** -11
    for h in range(n1):
        n = h // (n1 // n2)
        x, y, w, kk, vv = c.q[:, h].double(), c.dy[:, h].double(), o[:, h].double(), c.k[:, n].double(), c.v[:, n].double()
        p = (x @ kk.T * c.scale - lse[:, h].double()[:, None]).exp()
        ds = p * (y @ vv.T - (y * w).sum(1, keepdim=True))
        a = p * (y.abs() @ vv.abs().T + (y * w).abs().sum(1, keepdim=True))
        kn = kk.norm(dim=1)
        lim = 4 * c.scale * (u * (ds * kn).norm(dim=1) + S32 * (a * kn).norm(dim=1)) + u * want[0][:, h].norm(dim=1)
        err = (got[0][:, h].cpu().double() - want[0][:, h]).norm(dim=1)
        over = err - lim - d ** 0.5 * 2.0 ** -25
        assert bool((over <= 0).all()), (h, float((err / want[0][:, h].norm(dim=1)).max()))


# whole units, a cluster's, and pieces
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("l1,l2,n1,n2,d", [([20, 30], [400, 90], 4, 2, 128), ([900], [400], 4, 2, 64), ([2048], [1280], 16, 16, 64)])
@pytest.mark.parametrize("padded", [False, True])
def test_absent_states_get_zeros_whatever_the_queries_hold(dtype, l1, l2, n1, n2, d, padded):
    c = Case(l1, l2, n1, n2, d, dtype, padded=padded, mask=0.3, seed=32)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    o, lse = sab.cross_forward(q, k, v, c.cu1, c.cu2, c.scale, **c.args())
    first = (0, 7) if padded else (7,)
    c.dy[first] = float("inf")      # an overflowed loss scale
    dq, dk, dv = sab.cross_backward(q, k, v, o, c.dy.cuda(), lse, c.cu1, c.cu2, c.scale, check=True, **c.args())
    there = c.mask.clone()
    if padded:
        for b, n in enumerate(l2):
            there[b, n:] = False
    for x in (dk.cpu(), dv.cpu()):
        assert bool((x[~there] == 0).all())
        seen = x[0][there[0]] if padded else x[:l2[0]][there[:l2[0]]]
        assert not bool(seen.isfinite().all())      # the others of that sequence show it
    rest = dq.cpu().reshape(-1, n1, d).clone()
    assert not bool(rest[7].isfinite().any())
    rest[7] = 0
    assert bool(rest.isfinite().all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("drop", [None, 0.3])
def test_gradient_of_the_forward_definition(d, drop):
    """Against 64-bit autograd of the definition of O, element by element, and against its central differences.

    The kernel gets its own o and lse: o is off by e = u |O| + (u + s) P |V|, which moves Delta by |dY| . e and dS by P times
    that; lse is off by r = s + 2^-20 |lse|, which moves P, and so dS and dV, by a factor of 1 + r."""
    c = Case([9, 20], [33, 60], 4, 2, d, HF, mask=drop, seed=36)
    q, k, v, dy = (x.cuda() for x in (c.q, c.k, c.v, c.dy))
    o, lse = sab.cross_forward(q, k, v, c.cu1, c.cu2, c.scale, **c.args())
    got = [x.cpu().double() for x in sab.cross_backward(q, k, v, o, dy, lse, c.cu1, c.cu2, c.scale, check=True, **c.args())]
    u, s, g = 2.0 ** -11, c.scale, c.n1 // c.n2

    def value(x):
        total = 0.0
        for i, j, h in c.parts():
            total = total + (((x[0][i, h] @ x[1][j, h // g].T * s).softmax(1) @ x[2][j, h // g]) * c.dy[i, h].double()).sum()
        return total

    base = [x.double() for x in (c.q, c.k, c.v)]
    if c.mask is not None:      # absent rows are not read: any finite value
        base[1][~c.mask], base[2][~c.mask] = 0.0, 0.0
    leaves = [x.clone().requires_grad_() for x in base]
    want = torch.autograd.grad(value(leaves), leaves)
    lim = [torch.zeros_like(x) for x in base]
    for i, j, h in c.parts():
        n = h // g
        x, y, kk, vv = base[0][i, h], c.dy[i, h].double(), base[1][j, n], base[2][j, n]
        sc = x @ kk.T * s
        p, r = sc.softmax(1), S32 + 2.0 ** -20 * sc.logsumexp(1, keepdim=True).abs()
        w = p @ vv
        ds = p * (y @ vv.T - (y * w).sum(1, keepdim=True))
        a = p * (y.abs() @ vv.abs().T + (y * w).abs().sum(1, keepdim=True))
        moved = p * (y.abs() * (u * w.abs() + (u + S32) * (p @ vv.abs()))).sum(1, keepdim=True)
        ds = (u + S32 + r) * ds.abs() + S32 * a + moved
        lim[0][i, h] = s * ds @ kk.abs()
        lim[1][j, n] += s * ds.T @ x.abs()
        lim[2][j, n] += ((u + S32 + r) * p).T @ y.abs()
    for at, name in enumerate(("dq", "dk", "dv")):
        bound = 1.01 * (u * want[at].abs() + lim[at]) + 2.0 ** -25
        assert float(bound.norm()) < 0.1 * float(want[at].norm())       # zeros would fail
        assert bool(((got[at] - want[at]).abs() <= bound).all()), name
        # along the gradient itself, where the difference is its norm
        e, h = want[at] / want[at].norm(), 1e-3
        up, down = list(base), list(base)
        up[at], down[at] = base[at] + h * e, base[at] - h * e
        diff = float(value(up) - value(down)) / (2 * h)
        allowed = float((bound * e.abs()).sum())
        assert allowed < 0.1 * abs(diff)
        assert abs(float((got[at] * e).sum()) - diff) <= allowed + 1e-4 * abs(diff), name


@pytest.mark.parametrize("d,grad,heads", [
    (128, True, {15: 8, 16: 6, 23: 6, 24: 5, 29: 4, 37: 3, 47: 2, 77: 1}), (128, False, {36: 8, 37: 7, 39: 6, 47: 5, 59: 4, 75: 3, 98: 2}),
    (64, True, {15: 8, 16: 6, 76: 2, 77: 1}), (64, False, {66: 8, 72: 7, 78: 6, 95: 5, 115: 4})])
def test_clusters_of_a_launch_run_at_once(d, grad, heads):
    """One query tile a head and long loops: as many CTAs a head as fit the GPU beside the other heads', by the number of
    status words that a call leaves (the first word of its workspace; k_xdkv, with 16 tiles a head, has more units than SMs)."""
    for n, split in heads.items():
        q, k = (torch.zeros(rows, n, d, dtype=BF, device="cuda") for rows in (128, 2048))
        desc = sab.make_cross_desc([0, 128], [0, 2048], n, n, d, 0.1)
        ws = torch.zeros((sab.cross_grad_workspace_size if grad else sab.cross_fwd_workspace_size)(desc), dtype=torch.uint8, device="cuda")
        o, lse = sab.cross_forward(q, k, k, desc=desc, workspace=None if grad else ws)
        if grad:
            sab.cross_backward(q, k, k, o, q, lse, desc=desc, workspace=ws, check=True)
        ctas = int(ws[:4].view(torch.int32)) - (152 if grad else 0)
        assert ctas == n * split, (n, ctas)
