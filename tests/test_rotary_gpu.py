"""Rotary positions on the GPU against the definition in 64 bits.

Tolerance: one rounding to the 16-bit type (u = eps / 2 relative), fp32
arithmetic before it.  Each output is a sum of two products of a value and a
sine; sine and cosine are off by less than 2^-20 (the angle's last kept bit is
2^-24 turns of pi, sincospif is accurate to a few 2^-24), so
|error| <= u |y| + 2^-20 m (|a| + |b|).
"""
import math

import pytest
import torch

import sparse_attention_backward_gb300 as sab

pytestmark = pytest.mark.gpu


def _exact(x, rot, pos, sign):
    """x [rows, heads, d] and positions [rows], in 64 bits; also the bound's |a| + |b|."""
    f = torch.tensor(rot.inv_freq, dtype=torch.float64)
    r, h = rot.d_rot, rot.d_rot // 2
    cols = torch.arange(r) + rot.offset
    first, second = (cols[:h], cols[h:]) if rot.style == sab.SRT_HALF else (cols[0::2], cols[1::2])
    ang = sign * pos.double()[:, None, None] * f
    y, mag = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first] = rot.magnitude * (a * ang.cos() - b * ang.sin())
    y[..., second] = rot.magnitude * (a * ang.sin() + b * ang.cos())
    mag[..., first] = mag[..., second] = rot.magnitude * (a.abs() + b.abs())
    return y, mag


def _close(got, want, mag):
    u = torch.finfo(got.dtype).eps / 2
    err = (got.cpu().double() - want).abs()
    tol = u * want.abs() + 2.0 ** -20 * mag + torch.finfo(got.dtype).smallest_normal * u
    assert bool((err <= tol).all()), float((err - tol).max())


def _x(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


CASES = [
    # d, d_rot, offset: whole heads, leading and trailing parts, every vector width (8, 4, 2, 1 elements)
    (128, 128, 0), (192, 64, 128), (192, 96, 0), (64, 64, 0), (64, 8, 20), (36, 20, 4), (22, 14, 6), (17, 2, 9), (512, 256, 256),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("d,r,off", CASES)
@pytest.mark.parametrize("backward", [False, True])
def test_columns_styles_types(dtype, style, d, r, off, backward):
    rot = sab.Rotary(r, style=style, offset=off)
    lens = [5, 0, 37, 1]
    cu = [0, 5, 5, 42, 43]
    q, k = _x((43, 6, d), dtype, 1).cuda(), _x((43, 2, d), dtype, 2).cuda()
    call = sab.rotary_backward if backward else sab.rotary_forward
    if style == "interleaved" and d % 2:
        with pytest.raises(sab.SagError) as e:     # pairs at odd addresses
            call(q, k, rot, cu)
        assert e.value.status == sab.SAG_ERR_UNSUPPORTED
        return
    got = call(q, k, rot, cu)
    pos = torch.cat([torch.arange(n) for n in lens])
    for x, y in zip((q, k), got):
        want, mag = _exact(x.cpu(), rot, pos, -1 if backward else 1)
        _close(y, want, mag)
        rest = [c for c in range(d) if not off <= c < off + r]
        assert torch.equal(y[..., rest], x[..., rest])


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "ramp", "bands"])
def test_scalings_at_far_and_negative_positions(scaling):
    rot = sab.Rotary(64, style="half", scaling=scaling, factor=8.0, original_length=4096, base=500000.0)
    pos = torch.tensor([0, 1, -1, 131071, 2 ** 21, 2 ** 31 - 1, -2 ** 31, 77777], dtype=torch.int32)
    q = _x((8, 3, 64), torch.float16, 3).cuda()
    got = sab.rotary_forward(q, None, rot, [0, 8], positions=pos.cuda())
    # the definition itself keeps 53 bits of p f: 2^31 positions leave 2^-22 of a radian
    want, mag = _exact(q.cpu(), rot, pos, 1)
    _close(got, want, 2 * mag)


def test_padded_batch_zeroes_padding_and_reads_none_of_it():
    rot = sab.Rotary(128)
    lens, s = [7, 0, 12], 12
    q = _x((3, s, 4, 128), torch.bfloat16, 4)
    for b, n in enumerate(lens):
        q[b, n:] = float("nan")
    cu = [0, 7, 7, 19]
    got = sab.rotary_forward(q.cuda(), None, rot, cu)
    inplace = q.cuda()
    sab.rotary_forward(inplace, None, rot, cu, out=inplace)
    assert torch.equal(got, inplace)
    for b, n in enumerate(lens):
        assert not got[b, n:].any()
        want, mag = _exact(q[b, :n], rot, torch.arange(n), 1)
        _close(got[b, :n], want, mag)


def test_in_place_on_slices_of_a_fused_projection_and_rows_behind():
    rot = sab.Rotary(64, offset=64, style="interleaved")
    n1, n2, d, rows = 6, 2, 128, 50
    qkv = _x((rows + 3, n1 + 2 * n2, d), torch.bfloat16, 5).cuda()
    before = qkv.clone()
    q, k = qkv[:, :n1], qkv[:, n1:n1 + n2]
    dense = sab.rotary_forward(q[:rows].contiguous(), k[:rows].contiguous(), rot, [0, 20, rows])
    sab.rotary_forward(q, k, rot, [0, 20, rows], out=(q, k))
    assert torch.equal(q[:rows], dense[0]) and torch.equal(k[:rows], dense[1])
    assert torch.equal(qkv[rows:], before[rows:])                  # behind the last sequence
    assert torch.equal(qkv[:, n1 + n2:], before[:, n1 + n2:])      # the values beside


@pytest.mark.parametrize("batch", [64, 65, 1024, 1500])
def test_many_sequences(batch):
    rot = sab.Rotary(64)
    lens = [(b * 7) % 4 for b in range(batch)]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    q = _x((cu[-1], 2, 64), torch.bfloat16, 6)
    got = sab.rotary_forward(q.cuda(), None, rot, cu)
    want, mag = _exact(q, rot, torch.cat([torch.arange(n) for n in lens]), 1)
    _close(got, want, mag)


def test_gradient_is_the_transposed_map():
    # <R x, y> = <x, R^T y>, and differences of the linear map are the map itself
    rot = sab.Rotary(96, offset=16, style="half", scaling="ramp", factor=4.0, original_length=2048)
    x, y = _x((33, 3, 128), torch.float16, 7), _x((33, 3, 128), torch.float16, 8)
    fx = sab.rotary_forward(x.cuda(), None, rot, [0, 33]).cpu().double()
    gy = sab.rotary_backward(y.cuda(), None, rot, [0, 33]).cpu().double()
    u = 2.0 ** -11
    a, b = (fx * y.double()).sum(), (x.double() * gy).sum()
    tol = 1.01 * u * ((fx * y.double()).abs().sum() + (x.double() * gy).abs().sum())
    assert abs(float(a - b)) <= float(tol)


def test_streams_and_graph_replay():
    rot = sab.Rotary(64)
    q = _x((300, 4, 64), torch.bfloat16, 9).cuda()
    want = sab.rotary_forward(q, None, rot, [0, 300])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = sab.rotary_forward(q, None, rot, [0, 300], stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sab.rotary_forward(q, None, rot, [0, 300], out=out)
    q.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, sab.rotary_forward(q, None, rot, [0, 300]))


def test_no_rows():
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert sab.rotary_forward(q, None, sab.Rotary(64), [0, 0, 0]).shape == (0, 4, 64)


def test_workspace_in_host_memory_is_refused():
    # 65 sequences: the table of them goes through the workspace
    cu = list(range(66))
    q = _x((65, 2, 64), torch.bfloat16, 10).cuda()
    rot = sab.Rotary(64)
    desc = sab.make_rotary_desc(rot, cu, 2, 0, 64)
    need = sab.rotary_workspace_size(desc)
    host = torch.empty(need + 16, dtype=torch.uint8)
    host = host[-host.data_ptr() % 16:][:need]
    for call in (sab.rotary_forward, sab.rotary_backward):
        with pytest.raises(sab.SagError) as e:
            call(q, None, rot, desc=desc, workspace=host)
        assert e.value.status == sab.SAG_ERR_CUDA
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(sab.rotary_forward(q, None, rot, desc=desc, workspace=ws), sab.rotary_forward(q, None, rot, cu))
