"""Norms of queries and keys with the rotation in the same pass, on the GPU
against the definition in 64 bits, element by element.

u = eps / 2 of the 16-bit type: one rounding of each output.  Everything before
it is fp32: a sum of d <= 512 products is off by at most d 2^-24 of the sum of
their sizes, the square root, the sines and the products by a few 2^-24 more, so
s = (d + 64) 2^-24 covers each chain:

    |y err|  <= u |y|  + s (|xa wa r| + |xb wb r|)              over the columns that turn together
    |dx err| <= u |dx| + 2 s r (G + |x| r^2 mean(G |x|))        G = (|dya| + |dyb|) |w|
    |dw err| <= (N 2^-24 + 2 s) sum of (|dya| + |dyb|) |x| r    N heads in all (a sum in some order)
"""
import pytest
import torch

import sparse_attention_backward_gb300 as sab

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
NAN = float("nan")


def _turn(x, rot, pos, sign):
    """x [rows, heads, d] turned, in 64 bits, and |a| + |b| of the columns that turn together."""
    f = torch.tensor(rot.inv_freq, dtype=torch.float64)
    r, h = rot.d_rot, rot.d_rot // 2
    cols = torch.arange(r) + rot.offset
    first, second = (cols[:h], cols[h:]) if rot.style == sab.SRT_HALF else (cols[0::2], cols[1::2])
    ang = sign * pos.double()[:, None, None] * f
    y, mag = x.clone(), x.abs()
    a, b = x[..., first], x[..., second]
    y[..., first] = rot.magnitude * (a * ang.cos() - b * ang.sin())
    y[..., second] = rot.magnitude * (a * ang.sin() + b * ang.cos())
    mag[..., first] = mag[..., second] = abs(rot.magnitude) * (a.abs() + b.abs())
    return y, mag


def _within(name, got, want, lim, dtype):
    got = got.cpu().double()
    assert bool(torch.isfinite(got).all()), name
    if dtype is not None:
        lim = lim + torch.finfo(dtype).eps / 2 * (want.abs() + lim) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    over = (got - want).abs() - 1.01 * lim
    assert bool((over <= 0).all()), f"{name}: {float(over.max()):.3e} over its bound, at {float(want.abs().max()):.3e}"


class Case:
    def __init__(self, lens, n1, n2, d, rot, dtype, padded=False, positions=False, weight="own", plus=0.0, eps=1e-6, seed=0, grow=1.0):
        g = torch.Generator().manual_seed(500 + seed)
        self.lens, self.n, self.d, self.rot, self.dtype, self.padded, self.plus, self.eps = lens, (n1, n2), d, rot, dtype, padded, plus, eps
        self.cu = [0]
        for n in lens:
            self.cu.append(self.cu[-1] + n)
        s = max(lens)
        lead = (len(lens), s) if padded else (sum(lens),)
        self.x = [(torch.randn(*lead, n, d, generator=g) * grow).to(dtype) for n in (n1, n2)]
        self.dy = [torch.randn(*lead, n, d, generator=g).to(dtype) for n in (n1, n2)]
        self.w = None if weight is None else [(1 - plus + 0.2 * torch.randn(d, generator=g)).to(dtype if weight == "own" else torch.float32)
                                              for _ in range(2)]
        self.rows = torch.cat([torch.arange(n) + (b * s if padded else self.cu[b]) for b, n in enumerate(lens)])
        pos = torch.randint(-2 ** 31, 2 ** 31 - 1, lead, generator=g).to(torch.int32)
        self.positions = pos.cuda() if positions else None
        self.pos = pos.reshape(-1)[self.rows] if positions else torch.cat([torch.arange(n) for n in lens])
        if padded:
            for b, n in enumerate(lens):
                for t in self.x + self.dy:
                    t[b, n:] = NAN

    def flat(self, t):
        return t.reshape(-1, *t.shape[-2:])[self.rows].double()

    def spread(self, y, like):
        out = torch.zeros(like.reshape(-1, *like.shape[-2:]).shape, dtype=torch.float64)
        out[self.rows] = y
        return out.reshape(like.shape)

    def kw(self):
        return dict(eps=self.eps, weight_offset=self.plus, cu_seqlens=self.cu, positions=self.positions)

    def gpu(self, out=None, back=None):
        q, k = (t.cuda() for t in self.x)
        w = (None, None) if self.w is None else tuple(t.cuda() for t in self.w)
        got = sab.norm_rotary_forward(q, k, self.rot, *w, out=out, **self.kw())
        grads = sab.norm_rotary_backward(q, k, *(t.cuda() for t in self.dy), self.rot, *w, out=back, **self.kw())
        return got, grads

    def check(self, got, grads):
        s = (self.d + 64) * 2.0 ** -24
        for side, name in ((0, "q"), (1, "k")):
            x, dy = self.flat(self.x[side]), self.flat(self.dy[side])
            w = torch.ones(self.d, dtype=torch.float64) if self.w is None else self.w[side].double() + self.plus
            r = 1 / (x.square().mean(-1, keepdim=True) + self.eps).sqrt()
            y, mag = _turn(x * r * w, self.rot, self.pos, 1.0)
            _within(name, got[side], self.spread(y, self.x[side]), self.spread(s * mag, self.x[side]), self.dtype)
            dn, gm = _turn(dy, self.rot, self.pos, -1.0)
            g, big = dn * w, gm * w.abs()
            dx = r * (g - x * r ** 2 * (g * x).mean(-1, keepdim=True))
            lim = 2 * s * r * (big + x.abs() * r ** 2 * (big * x.abs()).mean(-1, keepdim=True))
            _within("d" + name, grads[side], self.spread(dx, self.x[side]), self.spread(lim, self.x[side]), self.dtype)
            if self.w is None:
                assert grads[2 + side] is None
            else:
                size = x.shape[0] * x.shape[1]
                _within("dw" + name, grads[2 + side], (dn * x * r).sum((0, 1)),
                        (size * 2.0 ** -24 + 2 * s) * (gm * x.abs() * r).sum((0, 1)) + 2.0 ** -126, None)


def run(c):
    c.check(*c.gpu())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("d,r,offset", [
    (128, 128, 0), (64, 64, 0), (192, 64, 128), (192, 192, 0), (256, 256, 0), (80, 16, 64), (96, 96, 0), (512, 64, 448), (512, 256, 8),
    (8, 8, 0), (24, 16, 8), (16, 2, 5), (13, 6, 3), (511, 254, 257), (130, 128, 2), (2, 2, 0), (300, 4, 100)])
def test_heads(dtype, style, d, r, offset):
    run(Case([5, 1, 30], 3, 2, d, sab.Rotary(r, offset=offset, style=style), dtype, seed=d))


@pytest.mark.parametrize("n1,n2", [(1, 1), (64, 4), (5, 5), (128, 1), (40, 8)])
@pytest.mark.parametrize("lens", [[1], [16], [700], [3, 0, 90, 1]])
@pytest.mark.parametrize("padded", [False, True])
def test_rows(n1, n2, lens, padded):
    run(Case(lens, n1, n2, 128, sab.Rotary(128, base=5e5), BF, padded=padded, seed=n1))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("weight", ["own", "f32", None])
@pytest.mark.parametrize("plus", [0.0, 1.0])
def test_weights_and_far_positions(dtype, weight, plus):
    rot = sab.Rotary(64, offset=64, scaling="ramp", factor=4.0, original_length=4096)
    run(Case([40, 9], 6, 2, 192, rot, dtype, positions=True, weight=weight, plus=plus, padded=True, seed=7))


@pytest.mark.parametrize("grow,eps", [(2.0 ** -12, 1e-6), (2.0 ** 10, 1e-6), (2.0 ** -20, 1e-12), (1.0, 0.1)])
def test_sizes_of_values(grow, eps):
    run(Case([50], 4, 2, 128, sab.Rotary(128), BF, eps=eps, grow=grow, seed=8))


def test_heads_of_zeros():
    c = Case([9], 4, 2, 128, sab.Rotary(128), BF, seed=9)
    for x in c.x:
        x[3], x[5, 1] = 0, 0
    run(c)


def test_many_sequences():
    run(Case([(b * 5) % 9 for b in range(300)], 4, 2, 64, sab.Rotary(64), HF, seed=10))
    run(Case([(b * 5) % 9 for b in range(300)], 4, 2, 64, sab.Rotary(64), HF, padded=True, seed=10))


def test_no_rows():
    q = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    rot = sab.Rotary(64)
    assert sab.norm_rotary_forward(q, None, rot, w, cu_seqlens=[0, 0]).shape == q.shape
    dq, dw = sab.norm_rotary_backward(q, None, q, None, rot, w, cu_seqlens=[0, 0])
    assert bool((dw == 0).all())


def test_no_key_and_weight_gradients_left_out():
    c = Case([70], 6, 1, 128, sab.Rotary(128), BF, seed=11)
    want, grads = c.gpu()
    q, dq, w = c.x[0].cuda(), c.dy[0].cuda(), c.w[0].cuda()
    assert torch.equal(sab.norm_rotary_forward(q, None, c.rot, w, cu_seqlens=c.cu), want[0])
    dx, dw = sab.norm_rotary_backward(q, None, dq, None, c.rot, w, cu_seqlens=c.cu)
    assert torch.equal(dx, grads[0])
    size = 70 * 6       # the blocks are shared otherwise, so the order of the sum differs
    assert bool(((dw - grads[2]).abs() <= size * 2.0 ** -23 * grads[2].abs().max()).all())
    out = torch.empty_like(q)
    got = sab.norm_rotary_backward(q, None, dq, None, c.rot, w, cu_seqlens=c.cu, out=(out, None))
    assert got[0] is out and got[1] is None and torch.equal(out, dx)


@pytest.mark.parametrize("d,r,offset", [(128, 128, 0), (80, 32, 48), (30, 8, 3)])
def test_in_place_strided_and_rows_behind(d, r, offset):
    c = Case([33, 20], 4, 2, d, sab.Rotary(r, offset=offset), BF, seed=12)
    want, grads = c.gpu()
    wide = torch.full((60, 8, d), 5.0, dtype=BF, device="cuda")
    q, k = wide[:, :4], wide[:, 4:6]
    q[:53], k[:53] = c.x[0].cuda(), c.x[1].cuda()
    before = wide.clone()
    w = [t.cuda() for t in c.w]
    dy = torch.full((60, 8, d), 5.0, dtype=BF, device="cuda")
    dq, dk = dy[:, :4], dy[:, 4:6]
    dq[:53], dk[:53] = c.dy[0].cuda(), c.dy[1].cuda()
    got = sab.norm_rotary_backward(q, k, dq, dk, c.rot, *w, out=(dq, dk, torch.empty(d, device="cuda"), torch.empty(d, device="cuda")), **c.kw())
    for x, y in zip(got[:2], grads[:2]):
        assert torch.equal(x[:53], y)
    assert bool((dy[53:] == 5).all()) and bool((dy[:, 6:] == 5).all()) and torch.equal(wide, before)
    sab.norm_rotary_forward(q, k, c.rot, *w, out=(q, k), **c.kw())
    assert torch.equal(q[:53], want[0]) and torch.equal(k[:53], want[1])
    assert bool((wide[53:] == 5).all()) and bool((wide[:, 6:] == 5).all())
    # the gradient over its input
    wide.copy_(before)
    dq[:53], dk[:53] = c.dy[0].cuda(), c.dy[1].cuda()
    got = sab.norm_rotary_backward(q, k, dq, dk, c.rot, *w, out=(q, k), **c.kw())
    assert torch.equal(q[:53], grads[0]) and torch.equal(k[:53], grads[1]) and got[2] is None


def test_bitwise_and_captured_on_another_stream():
    c = Case([900, 300], 16, 4, 128, sab.Rotary(128), BF, seed=13)
    want, grads = c.gpu()
    q, k, dq, dk = (t.cuda() for t in c.x + c.dy)
    w = [t.cuda() for t in c.w]
    desc = sab.make_norm_rotary_desc(c.rot, c.cu, 16, 4, 128)
    ws = torch.full((sab.norm_rotary_grad_workspace_size(desc),), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = sab.norm_rotary_backward(q, k, dq, dk, None, *w, desc=desc, workspace=ws, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        for x, y in zip(got, grads):
            assert torch.equal(x, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = sab.norm_rotary_forward(q, k, None, *w, desc=desc)
        got = sab.norm_rotary_backward(q, k, dq, dk, None, *w, desc=desc, workspace=ws)
    for _ in range(2):
        ws.fill_(255)
        g.replay()
        for a, b in zip(want + grads, y + got):
            assert torch.equal(a, b)


def test_offsets_beyond_32_bits():
    """A sequence behind one of so many tokens that elements and bytes before it pass 32 bits; those are zeros, which give
    zeros and add nothing to the weights' gradients."""
    c, rows = Case([300], 16, 16, 128, sab.Rotary(128), BF, seed=60), 2 ** 20 + 70000
    assert rows * 16 * 128 > 2 ** 31
    c.cu = [0, rows - 300, rows]

    def behind(x):
        big = torch.zeros(rows, 16, 128, dtype=BF, device="cuda")
        big[-300:] = x.cuda()
        return big

    x, dy, w = [behind(t) for t in c.x], [behind(t) for t in c.dy], [t.cuda() for t in c.w]
    got = sab.norm_rotary_forward(*x, c.rot, *w, **c.kw())
    grads = sab.norm_rotary_backward(*x, *dy, c.rot, *w, **c.kw())
    for t in got + grads[:2]:
        assert bool((t[:-300:4099] == 0).all())
    c.check([t[-300:] for t in got], [t[-300:] for t in grads[:2]] + list(grads[2:]))


def test_rotation_alone_agrees():
    # a head of unit mean square and no weight is rotated as rotary_forward does, but for roundings of the norm
    rot = sab.Rotary(64, offset=32)
    x = torch.where(torch.rand(40, 3, 128, generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0).to(BF).cuda()
    a = sab.norm_rotary_forward(x, None, rot, eps=1e-12, cu_seqlens=[0, 40])
    b = sab.rotary_forward(x, None, rot, cu_seqlens=[0, 40])
    assert bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 2.0 ** -14).all())


def test_gradient_against_differences():
    """Central differences in 64 bits of sum y dy along the gradient of each input; the kernel's bound is that of the 64-bit
    comparison above, so here the formula itself is checked."""
    c = Case([7, 5], 2, 1, 32, sab.Rotary(16, offset=8), HF, seed=14)
    _, grads = c.gpu()

    def value(x, w):
        total = 0.0
        for side in (0, 1):
            n = x[side] / (x[side].square().mean(-1, keepdim=True) + c.eps).sqrt() * w[side]
            total = total + (_turn(n, c.rot, c.pos, 1.0)[0] * c.flat(c.dy[side])).sum()
        return float(total)

    x, w = [c.flat(t) for t in c.x], [t.double() for t in c.w]
    for side in (0, 1):
        for which, at in ((x, grads[side].cpu().double()), (w, grads[2 + side].cpu().double())):
            e, h, keep = at / at.norm(), 1e-4, which[side]
            which[side] = keep + h * e
            up = value(x, w)
            which[side] = keep - h * e
            down = value(x, w)
            which[side] = keep
            # each element is within u of the gradient; cancelling parts of 1.5 times its size more
            assert abs((up - down) / (2 * h) - float(at.norm())) <= 2.0 ** -10 * float(at.norm())
