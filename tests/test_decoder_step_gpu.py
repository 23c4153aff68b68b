"""The operators of a decoder layer together, as a layer uses them: in training,
normed and rotated queries and keys for a selected and a local branch whose
gradients come back through the norms; in serving, the same layer token by
token over a paged cache."""
import math

import pytest
import torch

import sparse_attention_backward_gb300 as sab
from tests import _support as S

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _norm64(x, w, rot, pos, eps):
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
    f = torch.tensor(rot.inv_freq, dtype=torch.float64)
    ang = pos.double()[:, None, None] * f
    h, r = rot.d_rot // 2, rot.d_rot
    a, b = n[..., :h], n[..., h:r]
    return torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos(), n[..., r:]], -1)


def _attend64(q, k, v, cu, scale, left=None):
    """Causal within `left` (None: every key of the sequence)."""
    g = q.shape[1] // k.shape[1]
    out = []
    for a, b in zip(cu[:-1], cu[1:]):
        kk, vv = k[a:b].repeat_interleave(g, 1), v[a:b].repeat_interleave(g, 1)
        s = torch.einsum("qhd,khd->hqk", q[a:b], kk) * scale
        if left is not None:
            i = torch.arange(b - a)
            s = s.masked_fill((i > i[:, None]) | (i < i[:, None] - left), -math.inf)
        out.append(torch.einsum("hqk,khd->qhd", s.softmax(-1), vv))
    return torch.cat(out)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_training_step(dtype):
    n1, n2, d, bs, count, left, eps = 8, 2, 128, 16, 5, 20, 1e-6
    cu = [0, 80, 160]
    g = torch.Generator().manual_seed(41)
    r = lambda n: torch.randn(160, n, d, generator=g).to(dtype)  # noqa: E731
    q, k, v, dy = r(n1), r(n2), r(n2), r(n1)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(dtype) for _ in range(2))
    rot, c = sab.Rotary(96, base=500000.0), d ** -0.5
    topk = torch.arange(count, dtype=torch.int32).expand(160, n2, count).contiguous().cuda()
    qg, kg, vg, dyg, wqg, wkg = (x.cuda() for x in (q, k, v, dy, wq, wk))

    qn, kn = sab.norm_rotary_forward(qg, kg, rot, wqg, wkg, eps=eps, cu_seqlens=cu)
    o1, m, l = sab.forward(qn, kn, vg, topk, cu, cu, c, bs, count, check=True)
    o2, lse = sab.window_forward(qn, kn, vg, cu, cu, c, left=left, check=True)
    a = sab.backward(qn, kn, vg, o1, dyg, m, l, topk, cu, cu, c, bs, count, deterministic=True, check=True)
    b = sab.window_backward(qn, kn, vg, o2, dyg, lse, cu, cu, c, left=left, check=True)
    dq, dk, dwq, dwk = sab.norm_rotary_backward(qg, kg, a[0] + b[0], a[1] + b[1], rot, wqg, wkg, eps=eps, cu_seqlens=cu)

    x = [t.double().requires_grad_() for t in (q, k, v, wq, wk)]
    pos = torch.arange(80).repeat(2)
    nq, nk = _norm64(x[0], x[3], rot, pos, eps), _norm64(x[1], x[4], rot, pos, eps)
    # every block is selected, so the selected branch is the dense one
    y1, y2 = _attend64(nq, nk, x[2], cu, c), _attend64(nq, nk, x[2], cu, c, left)
    grads = torch.autograd.grad(((y1 + y2) * dy.double()).sum(), x)
    # each of the chain's up to six steps may be off by the repository's 5e-3 of a tensor's norm
    pairs = [("o1", o1, y1), ("o2", o2, y2), ("dq", dq, grads[0]), ("dk", dk, grads[1]), ("dv", a[2].float() + b[2].float(), grads[2]),
             ("dwq", dwq, grads[3]), ("dwk", dwk, grads[4])]
    for name, got, want in pairs:
        want = want.detach()
        rel = float((got.cpu().double() - want).norm() / want.norm())
        assert rel <= 6 * S.REL_FRO, (name, rel)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (HF, 64)])
@pytest.mark.parametrize("left", [-1, 24])
def test_serving_follows_training(dtype, d, left):
    """Three sequences: a chunk of their first tokens at once, then one by one, in a captured step that is replayed while the
    lengths and positions move on.  The outputs are those of the whole sequences."""
    n1, n2, page, first, steps = 8, 2, 16, [37, 5, 64], 21
    full = [f + steps for f in first]
    cu = [0, full[0], full[0] + full[1], sum(full)]
    g = torch.Generator().manual_seed(43)
    q, k, v = (torch.randn(sum(full), n, d, generator=g).to(dtype).cuda() for n in (n1, n2, n2))
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2))
    rot, c = sab.Rotary(64), d ** -0.5
    want_q, want_k = sab.norm_rotary_forward(q, k, rot, wq, wk, cu_seqlens=cu)
    want, want_lse = sab.window_forward(want_q, want_k, v, cu, cu, c, left=left, check=True)

    width, pages = 8, 30
    kc, vc = (torch.full((pages, page, n2, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    table = torch.randperm(pages, generator=g)[:3 * width].reshape(3, width).to(torch.int32).cuda()
    lens = torch.tensor(first, dtype=torch.int32, device="cuda")
    kind = sab.SAG_FP16 if dtype is HF else sab.SAG_BF16
    got, got_lse = torch.empty_like(want), torch.empty_like(want_lse)

    # the prompts
    rows = torch.cat([torch.arange(f) + a for f, a in zip(first, cu)]).cuda()
    cu1 = [0, first[0], first[0] + first[1], sum(first)]
    desc = sab.make_paged_desc(cu1, n1, n2, d, c, pages, page, width, left=left, dtype=kind)
    qn, kn = sab.norm_rotary_forward(q[rows], k[rows], rot, wq, wk, cu_seqlens=cu1)
    sab.paged_append(kn, v[rows], kc, vc, table, lens, desc=desc, check=True)
    got[rows], got_lse[rows] = sab.paged_forward(qn, kc, vc, table, lens, desc=desc, check=True)

    # the steps
    desc = sab.make_paged_desc([0, 1, 2, 3], n1, n2, d, c, pages, page, width, left=left, dtype=kind)
    nd = sab.make_norm_rotary_desc(rot, [0, 1, 2, 3], n1, n2, d, dtype=kind)
    work = torch.empty(max(sab.paged_fwd_workspace_size(desc), sab.paged_append_workspace_size(desc)), dtype=torch.uint8, device="cuda")
    row = torch.tensor([a + f for f, a in zip(first, cu)], device="cuda")
    position = lens.clone()

    def step():
        lens.add_(1)
        qs, ks = sab.norm_rotary_forward(q[row], k[row], None, wq, wk, positions=position, desc=nd)
        sab.paged_append(ks, v[row], kc, vc, table, lens, workspace=work, desc=desc)
        out = sab.paged_forward(qs, kc, vc, table, lens, workspace=work, desc=desc)
        got[row], got_lse[row] = out
        row.add_(1)
        position.add_(1)

    step()
    graph = torch.cuda.CUDAGraph()
    state = [t.clone() for t in (lens, row, position)]
    with torch.cuda.graph(graph):
        step()
    for t, was in zip((lens, row, position), state):
        t.copy_(was)
    for _ in range(steps - 1):
        graph.replay()
    torch.cuda.synchronize()
    # the same normed keys, and queries; O differs by the order of its sums, both within u |O| + (u + s) P |V| of the definition
    u, s = torch.finfo(dtype).eps / 2, 2.0 ** -13
    bound = 2 * (u * want.double().abs() + (u + s) * v.double().abs().max())
    assert bool(((got.double() - want.double()).abs() <= bound).all())
    rel = float((got.double() - want.double()).norm() / want.double().norm())
    assert rel <= 2 * S.REL_FRO, rel
    assert bool(((got_lse - want_lse).abs() <= 2 * s + 2.0 ** -19 * want_lse.abs()).all())


def test_refusals_of_tensors():
    q = torch.zeros(8, 4, 64, dtype=BF, device="cuda")
    k = torch.zeros(8, 2, 64, dtype=BF, device="cuda")
    cu, rot = [0, 8], sab.Rotary(64)
    w = torch.ones(64, dtype=BF, device="cuda")
    lse = torch.zeros(8, 4, device="cuda")
    either = (ValueError, sab.SagError)
    for bad in (q.float(), q.transpose(0, 1), q[..., ::2], q[:, :, :32], q[:4], q[:1].expand(8, 4, 64)):
        with pytest.raises(either):
            sab.window_forward(bad, k, k, cu, cu, 0.1)
        with pytest.raises(either):
            sab.window_forward(q, bad[:, :2], k, cu, cu, 0.1)
        with pytest.raises(either):
            sab.window_backward(q, k, k, bad, q, lse, cu, cu, 0.1)
        with pytest.raises(either):
            sab.norm_rotary_forward(q, bad[:, :3], rot, w, w, cu_seqlens=[0, 8])
        with pytest.raises(either):
            sab.norm_rotary_backward(q, k, bad, k, rot, w, w, cu_seqlens=cu)
    for bad in (w[:32], w.float()[:63], w.half(), w.cpu(), torch.ones(128, dtype=BF, device="cuda")[::2]):
        with pytest.raises(either):
            sab.norm_rotary_forward(q, k, rot, bad, bad, cu_seqlens=cu)
    with pytest.raises(either):
        sab.norm_rotary_forward(q, k, rot, w, w.float(), cu_seqlens=cu)
    with pytest.raises(either):
        sab.norm_rotary_forward(q, k, rot, w, w, cu_seqlens=cu, positions=torch.zeros(8, dtype=torch.int64, device="cuda"))
    cache = torch.zeros(5, 16, 2, 64, dtype=BF, device="cuda")
    table, lens = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.full((1,), 8, dtype=torch.int32, device="cuda")
    sab.paged_forward(q, cache, cache, table, lens, cu, 0.1, check=True)
    for args in ((q.float(), cache, cache, table, lens), (q, cache.half(), cache, table, lens), (q, cache, cache[:4], table, lens),
                 (q, cache, cache.transpose(1, 2), table, lens), (q, cache, cache, table.long(), lens), (q, cache, cache, table[:, :1].T, lens[:0]),
                 (q, cache, cache, table, lens.cpu()), (q, cache, cache, table, lens.float()), (q[:7], cache, cache, table, lens),
                 (q, cache[..., :32], cache[..., :32], table, lens), (q, cache, cache.cpu(), table, lens)):
        with pytest.raises(either):
            sab.paged_forward(*args, cu, 0.1)
        with pytest.raises(either):
            sab.paged_append(args[0][:, :2], args[0][:, :2], *args[1:], cu)
    # host memory in the place of the workspace is an error, not a fault
    d = sab.make_window_desc(cu, cu, 4, 2, 64, 0.1)
    p = sab.make_paged_desc(cu, 4, 2, 64, 0.1, 5, 16, 2)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    if ws.data_ptr() % 16 == 0:
        for call in (lambda: sab.window_forward(q, k, k, desc=d, workspace=ws), lambda: sab.paged_append(k, k, cache, cache, table, lens, desc=p, workspace=ws),
                     lambda: sab.paged_forward(q, cache, cache, table, lens, desc=p, workspace=ws),
                     lambda: sab.norm_rotary_backward(q, k, q, k, rot, w, w, cu_seqlens=cu, workspace=ws)):
            with pytest.raises(sab.SagError) as e:
                call()
            assert e.value.status == sab.SAG_ERR_CUDA


def test_descriptors_that_were_changed():
    q = torch.randn(8, 4, 64, device="cuda").to(BF)
    k = torch.randn(8, 2, 64, device="cuda").to(BF)
    cu, rot = [0, 8], sab.Rotary(64)
    w = torch.rand(64, device="cuda").to(BF)
    d = sab.make_window_desc(cu, cu, 4, 2, 64, 0.1, left=3)
    d.q_stride, d.k_stride = 4096, 8192        # strides: the tensors' own
    for x, y in zip(sab.window_forward(q, k, k, desc=d), sab.window_forward(q, k, k, cu, cu, 0.1, left=3)):
        assert torch.equal(x, y)
    d.left, d.right = 1, 2
    for x, y in zip(sab.window_forward(q, k, k, desc=d), sab.window_forward(q, k, k, cu, cu, 0.1, left=1, right=2)):
        assert torch.equal(x, y)
    d.n1 = 8
    with pytest.raises(ValueError):
        sab.window_forward(q, k, k, desc=d)
    d = sab.make_norm_rotary_desc(rot, cu, 4, 2, 64)
    d.q_stride, d.weight_fp32, d.q_out_stride = 512, 1, 4096
    for weights in ((w, w), (w.float(), w.float())):
        for x, y in zip(sab.norm_rotary_forward(q, k, None, *weights, desc=d), sab.norm_rotary_forward(q, k, rot, w, w, cu_seqlens=cu)):
            assert torch.equal(x, y)
    d.eps = 1.0
    for x, y in zip(sab.norm_rotary_forward(q, k, None, w, w, desc=d), sab.norm_rotary_forward(q, k, rot, w, w, eps=1.0, cu_seqlens=cu)):
        assert torch.equal(x, y)
    cache = torch.randn(5, 16, 2, 64, device="cuda").to(BF)
    table, lens = torch.tensor([[3, 1]], dtype=torch.int32, device="cuda"), torch.full((1,), 20, dtype=torch.int32, device="cuda")
    p = sab.make_paged_desc(cu, 4, 2, 64, 0.1, 5, 16, 2)
    p.k_row, p.k_page, p.left = 4096, 65536, 7
    for x, y in zip(sab.paged_forward(q, cache, cache, table, lens, desc=p), sab.paged_forward(q, cache, cache, table, lens, cu, 0.1, left=7)):
        assert torch.equal(x, y)
