"""Rotary positions and cross attention together with the selected attention,
as a decoder layer uses them: rotated queries and keys, selected self-attention,
its output as the queries of a cross attention to an encoder's states, and the
gradients back through all three."""
import math

import pytest
import torch

import sparse_attention_backward_gb300 as sab
from tests import _support as S

pytestmark = pytest.mark.gpu


def _inputs(lead1, lead2, n1, n2, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda lead, n: torch.randn(lead + (n, d), generator=g).to(dtype)  # noqa: E731
    return r(lead1, n1), r(lead1, n2), r(lead1, n2), r(lead2, n2), r(lead2, n2), r(lead1, n1)


def _blocks(rows, n2, count):
    return torch.arange(count, dtype=torch.int32).expand(rows, n2, count).contiguous()


def _rotate64(x, rot, cu):
    """Half style over the first d_rot columns, in 64 bits, differentiable."""
    f = torch.tensor(rot.inv_freq, dtype=torch.float64)
    pos = torch.cat([torch.arange(b - a) for a, b in zip(cu[:-1], cu[1:])])
    ang = pos.double()[:, None, None] * f
    h, r = rot.d_rot // 2, rot.d_rot
    a, b = x[..., :h], x[..., h:r]
    return torch.cat([rot.magnitude * (a * ang.cos() - b * ang.sin()), rot.magnitude * (a * ang.sin() + b * ang.cos()), x[..., r:]], -1)


def _attend64(q, k, v, cu1, cu2, scale):
    g = q.shape[1] // k.shape[1]
    out = []
    for a, b, c, d in zip(cu1[:-1], cu1[1:], cu2[:-1], cu2[1:]):
        kk, vv = k[c:d].repeat_interleave(g, 1), v[c:d].repeat_interleave(g, 1)
        out.append(torch.einsum("hqk,khd->qhd", (torch.einsum("qhd,khd->hqk", q[a:b], kk) * scale).softmax(-1), vv))
    return torch.cat(out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_layer_forward_and_gradients(dtype):
    n1, n2, d, bs, count = 8, 2, 128, 16, 5
    cu1, cu2 = [0, 80, 160], [0, 33, 200]
    q, k, v, ek, ev, dy = _inputs((160,), (200,), n1, n2, d, dtype, 31)
    rot = sab.Rotary(96, scaling="ramp", factor=4.0, original_length=64)
    c = d ** -0.5
    topk = _blocks(160, n2, count).cuda()
    qg, kg, vg, ekg, evg, dyg = (x.cuda() for x in (q, k, v, ek, ev, dy))

    o1, m, l = sab.forward(qg, kg, vg, topk, cu1, cu1, c, bs, count, rotary=rot, check=True)
    o2, lse = sab.cross_forward(o1, ekg, evg, cu1, cu2, c, check=True)
    do1, dek, dev = sab.cross_backward(o1, ekg, evg, o2, dyg, lse, cu1, cu2, c, check=True)
    dq, dk, dv = sab.backward(qg, kg, vg, o1, do1, m, l, topk, cu1, cu1, c, bs, count, deterministic=True, rotary=rot, check=True)

    x = [t.double().requires_grad_() for t in (q, k, v, ek, ev)]
    # every block is selected, so the self-attention is the dense one
    y1 = _attend64(_rotate64(x[0], rot, cu1), _rotate64(x[1], rot, cu1), x[2], cu1, cu1, c)
    y2 = _attend64(y1, x[3], x[4], cu1, cu2, c)
    grads = torch.autograd.grad((y2 * dy.double()).sum(), x)
    # each of the chain's up to six steps may be off by the repository's 5e-3 of a tensor's norm
    for name, got, want in [("o1", o1, y1), ("o2", o2, y2)] + list(zip(("dq", "dk", "dv", "dek", "dev"), (dq, dk, dv, dek, dev), grads)):
        want = want.detach()
        rel = float((got.cpu().double() - want).norm() / want.norm())
        assert rel <= 6 * S.REL_FRO, (name, rel)


@pytest.mark.parametrize("padded", [False, True])
def test_rotary_of_forward_and_backward_is_the_operator(padded):
    n1, n2, d, bs, count = 4, 2, 192, 16, 3
    cu = [0, 48, 96]
    lead = (2, 64) if padded else (96,)
    cu2 = cu
    q, k, v, _, _, dy = _inputs(lead, (1,), n1, n2, d, torch.bfloat16, 5)
    v, dy = v[..., :128].contiguous(), dy[..., :128].contiguous()
    topk = _blocks(lead[0] * (lead[1] if padded else 1), n2, count).reshape(lead + (n2, count)).cuda()
    rot = sab.Rotary(64, offset=128, style="interleaved")
    q, k, v, dy = (x.cuda() for x in (q, k, v, dy))
    c = d ** -0.5
    qr, kr = sab.rotary_forward(q, None, rot, cu), sab.rotary_forward(k, None, rot, cu2)
    want = sab.forward(qr, kr, v, topk, cu, cu2, c, bs, count)
    got = sab.forward(q, k, v, topk, cu, cu2, c, bs, count, rotary=rot)
    assert torch.equal(got[1], want[1])                     # the maxima are exact in any order
    gr = sab.backward(qr, kr, v, want[0], dy, want[1], want[2], topk, cu, cu2, c, bs, count, deterministic=True)
    got = sab.backward(q, k, v, want[0], dy, want[1], want[2], topk, cu, cu2, c, bs, count, deterministic=True, rotary=rot)
    assert torch.equal(got[0], sab.rotary_backward(gr[0], None, rot, cu))
    assert torch.equal(got[1], sab.rotary_backward(gr[1], None, rot, cu2))
    assert torch.equal(got[2], gr[2])


def test_rotary_with_split_heads_and_positions():
    n1, n2, bs, count = 4, 1, 16, 4
    cu = [0, 64]
    g = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    q, k, v, dy, qr, kr = r(64, n1, 128), r(64, n2, 128), r(64, n2, 128), r(64, n1, 128), r(64, n1, 64), r(64, n2, 64)
    pos = torch.randint(0, 100000, (64,), generator=g, dtype=torch.int32).cuda()
    topk = _blocks(64, n2, count).cuda()
    rot, c = sab.Rotary(64), 192 ** -0.5
    tq, tk = sab.rotary_forward(qr, kr, rot, cu, positions=pos)
    want = sab.forward(q, k, v, topk, cu, cu, c, bs, count, q_rope=tq, k_rope=tk)
    got = sab.forward(q, k, v, topk, cu, cu, c, bs, count, q_rope=qr, k_rope=kr, rotary=rot, q_positions=pos, k_positions=pos)
    assert torch.equal(got[1], want[1])
    args = (want[0], dy, want[1], want[2], topk, cu, cu, c, bs, count)
    gw = sab.backward(q, k, v, *args, deterministic=True, q_rope=tq, k_rope=tk)
    gg = sab.backward(q, k, v, *args, deterministic=True, q_rope=qr, k_rope=kr, rotary=rot, q_positions=pos, k_positions=pos)
    bq, bk = sab.rotary_backward(gw[3], gw[4], rot, cu, positions=pos)
    assert all(torch.equal(a, b) for a, b in zip(gg, (gw[0], gw[1], gw[2], bq, bk)))


def test_refusals_of_tensors():
    q = torch.zeros(8, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu, rot = [0, 8], sab.Rotary(64)
    for bad in (q.float(), q.transpose(0, 1), q[..., ::2], q[:, :, :32], q[:4], q[:1].expand(8, 4, 64)):
        with pytest.raises((ValueError, sab.SagError)):
            sab.cross_forward(bad, k, k, cu, cu, 0.1)
        with pytest.raises((ValueError, sab.SagError)):
            sab.cross_forward(q, bad[:, :2], k, cu, cu, 0.1)
    with pytest.raises(ValueError):
        sab.cross_forward(q, k, k, cu, cu, 0.1, key_mask=torch.ones(8, device="cuda"))
    with pytest.raises(ValueError):
        sab.cross_forward(q, k, k, cu, cu, 0.1, key_mask=torch.ones(7, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        sab.cross_forward(q, k, k.cpu(), cu, cu, 0.1)
    with pytest.raises(sab.SagError):
        sab.cross_forward(q, k, k.half(), cu, cu, 0.1)
    with pytest.raises(ValueError):
        sab.cross_forward(q, k, k, [0, 9], cu, 0.1)
    with pytest.raises(sab.SagError):
        sab.rotary_forward(q, k, rot, cu, positions=torch.zeros(8, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        sab.rotary_forward(q, k[:7], rot, cu)
    with pytest.raises((ValueError, sab.SagError)):
        sab.rotary_forward(q.float(), None, rot, cu)
    desc = sab.make_rotary_desc(rot, cu, 4, 2, 64)
    with pytest.raises(ValueError):
        sab.rotary_forward(q, None, rot, desc=desc)
    # host memory in the place of the workspace is an error, not a fault
    d = sab.make_cross_desc(cu, cu, 4, 2, 64, 0.1)
    ws = torch.empty(sab.cross_fwd_workspace_size(d), dtype=torch.uint8)
    if ws.data_ptr() % 16 == 0:
        with pytest.raises(sab.SagError) as e:
            sab.cross_forward(q, k, k, desc=d, workspace=ws)
        assert e.value.status == sab.SAG_ERR_CUDA


def test_descriptors_that_were_changed():
    q = torch.randn(8, 4, 64, device="cuda").to(torch.bfloat16)
    k = torch.randn(8, 2, 64, device="cuda").to(torch.bfloat16)
    cu, rot = [0, 8], sab.Rotary(64)
    # strides: the tensors' own
    d = sab.make_rotary_desc(rot, cu, 4, 2, 64)
    d.q_stride, d.q_out_stride, d.k_stride = 4096, 512, 256
    for x, y in zip(sab.rotary_forward(q, k, rot, desc=d), sab.rotary_forward(q, k, rot, cu)):
        assert torch.equal(x, y)
    d = sab.make_cross_desc(cu, cu, 4, 2, 64, 0.1)
    d.q_stride, d.k_stride, d.v_stride = 4096, 4096, 8192
    for x, y in zip(sab.cross_forward(q, k, k, desc=d), sab.cross_forward(q, k, k, cu, cu, 0.1)):
        assert torch.equal(x, y)
    # another scale is taken, another size refused
    d.scale = 0.2
    for x, y in zip(sab.cross_forward(q, k, k, desc=d), sab.cross_forward(q, k, k, cu, cu, 0.2)):
        assert torch.equal(x, y)
    d.n1 = 8
    with pytest.raises(ValueError):
        sab.cross_forward(q, k, k, desc=d)
    d = sab.make_rotary_desc(rot, cu, 4, 2, 64)
    d.d = 128
    with pytest.raises(ValueError):
        sab.rotary_forward(q, k, rot, desc=d)
