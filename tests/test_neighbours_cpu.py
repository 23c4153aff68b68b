"""Rotary positions and cross attention without a GPU: the entry points are
exported, phase 1 and the host-side checks of phase 2 refuse what the header
refuses before anything is enqueued, and the frequencies follow their formulas."""
import ctypes
import math
import os
import re

import pytest
import torch

import sparse_attention_backward_gb300 as sab
from sparse_attention_backward_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPE, NULL, ALIGN = sab.SAG_ERR_SHAPE, sab.SAG_ERR_NULL, sab.SAG_ERR_ALIGN
UNSUP, DTYPE, WORK, OK = sab.SAG_ERR_UNSUPPORTED, sab.SAG_ERR_DTYPE, sab.SAG_ERR_WORKSPACE, sab.SAG_OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return sab._lib_neighbours()


def test_declared_and_exported(lib):
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "selattn.h")).read(), flags=re.S)
    names = set(re.findall(r"\b((?:rotary|cross_attn)_\w*)\s*\(", txt))
    assert names == set(sab.EXPORTED_NEIGHBOURS)
    for n in names:
        assert hasattr(lib, n)


# ------------------------------------------------------------------- rotary
@pytest.mark.parametrize("r", [2, 4, 64, 96, 256])
def test_frequencies(r):
    base, factor, length = 10000.0, 8.0, 4096
    plain = [base ** (-2 * i / r) for i in range(r // 2)]
    assert sab.Rotary(r).inv_freq == pytest.approx(plain, rel=1e-14)
    assert sab.Rotary(r, scaling="linear", factor=factor).inv_freq == pytest.approx([f / factor for f in plain], rel=1e-14)
    if r >= 4:
        b = base * factor ** (r / (r - 2))
        got = sab.Rotary(r, scaling="base", factor=factor)
        assert got.inv_freq == pytest.approx([b ** (-2 * i / r) for i in range(r // 2)], rel=1e-13)
        # the slowest pair turns as under linear scaling, the fastest as without any
        assert got.inv_freq[-1] == pytest.approx(plain[-1] / factor, rel=1e-12) and got.inv_freq[0] == 1.0
    bands = sab.Rotary(r, scaling="bands", factor=factor, original_length=length, low=1.0, high=4.0)
    for f, g in zip(plain, bands.inv_freq):
        turns = length * f / (2 * math.pi)
        if turns >= 4:
            assert g == pytest.approx(f, rel=1e-14)
        elif turns <= 1:
            assert g == pytest.approx(f / factor, rel=1e-14)
        else:
            assert f / factor < g < f
    ramp = sab.Rotary(r, scaling="ramp", factor=factor, original_length=length)
    assert ramp.magnitude == pytest.approx(0.1 * math.log(factor) + 1)
    assert all(f / factor * (1 - 1e-14) <= g <= f * (1 + 1e-14) for f, g in zip(plain, ramp.inv_freq))


@pytest.mark.parametrize("kw", [
    dict(d_rot=3), dict(d_rot=0), dict(d_rot=258), dict(d_rot=64, base=1.0), dict(d_rot=64, base=float("nan")),
    dict(d_rot=64, scaling="linear", factor=0.5), dict(d_rot=64, scaling="linear", factor=float("inf")),
    dict(d_rot=2, scaling="base", factor=2.0), dict(d_rot=64, scaling="ramp", factor=2.0, original_length=0),
    dict(d_rot=64, scaling="ramp", factor=2.0, original_length=4096, beta_fast=1.0, beta_slow=1.0),
    dict(d_rot=64, scaling="bands", factor=2.0, original_length=4096, low=4.0, high=4.0),
])
def test_frequency_refusals(kw):
    with pytest.raises(sab.SagError) as e:
        sab.Rotary(**kw)
    assert e.value.status == SHAPE


def test_rotary_arguments():
    with pytest.raises(ValueError):
        sab.Rotary(64, style="other")
    with pytest.raises(ValueError):
        sab.Rotary(64, scaling="other")
    with pytest.raises(ValueError):
        sab.Rotary(64, inv_freq=[1.0] * 31)
    with pytest.raises(ValueError):
        sab.rotary_forward(torch.zeros(4, 2, 64, dtype=torch.bfloat16), None, sab.Rotary(64), [0, 4])


def _rot(**kw):
    a = dict(cu=[0, 3, 3, 10], n1=4, n2=2, d=128, d_rot=64, offset=0, dtype=sab.SAG_BF16, layout=0, s_max=0)
    a.update(kw)
    r = sab.Rotary(a["d_rot"], offset=a["offset"])
    return sab.make_rotary_desc(r, a["cu"], a["n1"], a["n2"], a["d"], a["dtype"], a["layout"], a["s_max"])


def _phase1(lib, name, desc):
    n = ctypes.c_size_t(12345)
    return getattr(lib, name)(ctypes.byref(desc), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(n2=0), OK), (dict(offset=64), OK), (dict(offset=65), SHAPE), (dict(offset=-2), SHAPE),
    (dict(d_rot=130), SHAPE), (dict(n1=0), SHAPE), (dict(n1=129), SHAPE), (dict(n2=129), SHAPE), (dict(d=513), SHAPE),
    (dict(dtype=2), DTYPE), (dict(layout=2), SHAPE), (dict(s_max=5), SHAPE), (dict(cu=[0, 5, 4]), SHAPE), (dict(cu=[1, 5]), SHAPE),
    (dict(layout=1, s_max=7), OK), (dict(layout=1, s_max=6), SHAPE), (dict(layout=1, s_max=-1), SHAPE), (dict(cu=[0, 0]), OK),
    (dict(cu=[0, 2 * 1024 * 1024]), OK), (dict(cu=[0, 2 * 1024 * 1024 + 1]), SHAPE), (dict(cu=[0] * 65538), UNSUP),
])
def test_rotary_phase1(lib, kw, want):
    d = _rot(**kw)
    st, n = _phase1(lib, "rotary_workspace_size", d)
    assert st == want
    assert n == (0 if want == OK else 12345)


def test_rotary_large_batch_workspace(lib):
    sizes = [_phase1(lib, "rotary_workspace_size", _rot(cu=list(range(b + 1))))[1] for b in (64, 65, 65536)]
    assert sizes[0] == 0 and 0 < sizes[1] < sizes[2]


def test_rotary_fields(lib):
    for field, value in (("style", 2), ("magnitude", float("nan")), ("q_stride", 511), ("k_out_stride", 255), ("q_stride", -1)):
        d = _rot()
        setattr(d, field, value)
        assert _phase1(lib, "rotary_workspace_size", d)[0] == SHAPE
    d = _rot()
    d.inv_freq[3] = float("inf")
    assert _phase1(lib, "rotary_workspace_size", d)[0] == SHAPE
    assert lib.rotary_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == NULL
    assert lib.rotary_workspace_size(ctypes.byref(_rot()), None) == NULL


def test_rotary_phase2_host_checks(lib):
    call = lambda d, io, ws=None, n=0: lib.rotary_fwd(ctypes.byref(d), io if io is None else ctypes.byref(io), ws, n, None)  # noqa: E731
    good = dict(query=4096, key=8192, query_out=4096, key_out=8192)
    assert call(_rot(), None) == NULL
    for missing in good:
        assert call(_rot(), sab.SrtIo(**{k: v for k, v in good.items() if k != missing})) == NULL
    assert call(_rot(), sab.SrtIo(**dict(good, key=8200))) == ALIGN
    assert call(_rot(), sab.SrtIo(positions=6, **good)) == ALIGN
    big = _rot(cu=list(range(66)))
    assert call(big, sab.SrtIo(**good)) == WORK
    assert call(big, sab.SrtIo(**good), 4096, 16) == WORK
    assert call(_rot(cu=[0, 0]), sab.SrtIo()) == OK        # no rows: nothing to do


def test_rotary_in_place_with_another_stride(lib):
    # the device is asked for only after the argument checks, and there is none here; with one, the strides are refused
    d = _rot()
    d.q_out_stride = 1024
    io = sab.SrtIo(query=4096, key=8192, query_out=4096, key_out=16384)
    assert lib.rotary_fwd(ctypes.byref(d), ctypes.byref(io), None, 0, None) in (SHAPE, sab.SAG_ERR_CUDA)


# --------------------------------------------------------- cross attention
def _cross(**kw):
    a = dict(cu_seqlens_q=[0, 3, 10], cu_seqlens_kv=[0, 7, 7], n1=8, n2=2, d=128, scale=0.1)
    a.update(kw)
    return sab.make_cross_desc(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(d=64), OK), (dict(d=96), UNSUP), (dict(d=192), UNSUP), (dict(d=0), SHAPE),
    (dict(n1=6), OK), (dict(n1=7), SHAPE), (dict(n1=66), SHAPE), (dict(n1=64), OK), (dict(n1=256, n2=128), SHAPE),
    (dict(n1=0, n2=0), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(dtype=5), DTYPE), (dict(layout=3), SHAPE), (dict(cu_seqlens_kv=[0, 9, 7]), SHAPE),
    (dict(cu_seqlens_q=[0, 0, 0]), OK), (dict(cu_seqlens_kv=[0, 0, 0]), OK), (dict(s1_max=4), SHAPE),
    (dict(layout=1, s1_max=7, s2_max=7), OK), (dict(layout=1, s1_max=6, s2_max=7), SHAPE), (dict(layout=1, s1_max=7, s2_max=6), SHAPE),
    (dict(cu_seqlens_q=[0, 2 ** 21 + 1], cu_seqlens_kv=[0, 1]), SHAPE), (dict(cu_seqlens_q=[0] * 65538, cu_seqlens_kv=[0] * 65538), UNSUP),
])
def test_cross_phase1(lib, kw, want):
    d = _cross(**kw)
    for name in ("cross_attn_fwd_workspace_size", "cross_attn_grad_workspace_size"):
        st, n = _phase1(lib, name, d)
        assert st == want and (n > 0 if want == OK else n == 12345)


def test_cross_fields(lib):
    for field, value in (("q_stride", 1020), ("q_stride", 1028), ("k_stride", 248), ("v_stride", -8)):
        d = _cross()
        setattr(d, field, value)
        assert _phase1(lib, "cross_attn_fwd_workspace_size", d)[0] == SHAPE
    for field in ("cu_seqlens_q", "cu_seqlens_kv"):
        d = _cross()
        setattr(d, field, None)
        assert _phase1(lib, "cross_attn_grad_workspace_size", d)[0] == NULL
    assert lib.cross_attn_fwd_workspace_size(ctypes.byref(_cross()), None) == NULL
    with pytest.raises(ValueError):
        _cross(cu_seqlens_q=[0, 1])


@pytest.mark.parametrize("entry", ["cross_attn_fwd", "cross_attn_grad"])
def test_cross_phase2_host_checks(lib, entry):
    size = _phase1(lib, entry + "_workspace_size", _cross())[1]
    call = lambda io, ws=1 << 20, n=size, d=None: getattr(lib, entry)(  # noqa: E731
        ctypes.byref(d or _cross()), io if io is None else ctypes.byref(io), ws, n, None)
    good = dict(query=4096, key=8192, value=12288, attention_out=16384, softmax_lse=20480)
    if entry == "cross_attn_grad":
        good.update(attention_out_grad=24576, dq=28672, dk=32768, dv=36864)
    assert call(None) == NULL
    for missing in good:
        assert call(sab.ScaIo(**{k: v for k, v in good.items() if k != missing})) == NULL
        assert call(sab.ScaIo(**dict(good, **{missing: good[missing] + 8}))) == ALIGN
    assert call(sab.ScaIo(**good), None) == WORK
    assert call(sab.ScaIo(**good), n=size - 1) == WORK
    assert call(sab.ScaIo(**good), ws=(1 << 20) + 8) == ALIGN
    assert lib.cross_attn_query_error(None, None) == NULL


def test_cross_arguments():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sab.cross_forward(x, x, x, [0, 4], [0, 4], 0.1)
    with pytest.raises(ValueError):
        sab.cross_backward(x, x, x, x, x, torch.zeros(4, 2), [0, 4], [0, 4], 0.1)


def test_workspace_of_partial_sums():
    """Only gradients with long, alike loops hold the sums of pieces (304 x 128 KB at most)."""
    def size(cu1, cu2, **kw):
        return sab.cross_grad_workspace_size(sab.make_cross_desc(cu1, cu2, 16, 16, 128, 0.1, **kw))

    assert size([0, 1600], [0, 1600]) < 4 << 20
    assert 304 * (128 << 10) <= size([0, 4096], [0, 4096]) < 304 * (128 << 10) + (8 << 20)
    assert size([0, 4096, 5000], [0, 4096, 5000]) < 8 << 20
    assert size([0, 4096, 4096], [0, 4096, 4100], layout=sab.SAG_LAYOUT_BSND, s1_max=4096, s2_max=4096) < 16 << 20


@pytest.mark.parametrize("entry", ["rotary_fwd", "rotary_grad"])
@pytest.mark.parametrize("which", ["q", "k"])
def test_rows_of_an_output_over_its_input_lie_where_the_inputs_do(lib, entry, which):
    """Refused before the device is looked for (these addresses belong to none), and nothing else is."""
    width = dict(q=512, k=256)[which]
    io = sab.SrtIo(query=4096, key=8192, query_out=4096 if which == "q" else 12288, key_out=8192 if which == "k" else 16384)

    def call(**strides):
        d = _rot()
        for name, value in strides.items():
            setattr(d, f"{which}_{name}", value)
        return getattr(lib, entry)(ctypes.byref(d), ctypes.byref(io), None, 0, None)

    assert call(out_stride=width + 8) == call(stride=width + 8) == call(stride=width + 8, out_stride=width + 16) == SHAPE
    for legal in (dict(), dict(out_stride=width), dict(stride=width + 8, out_stride=width + 8)):
        assert call(**legal) == sab.SAG_ERR_CUDA


def test_descriptors_that_were_changed_are_brought_up_to_date():
    """What the tensor calls check tensors against follows fields that were set after a descriptor was made."""
    for field, value in (("n1", 4), ("d", 64), ("dtype", sab.SAG_FP16), ("batch", 1), ("scale", 0.5), ("q_stride", 1024), ("v_stride", 512)):
        kept, made = _cross(), _cross(**({field: value} if field in ("n1", "d", "dtype", "scale") else {}))
        size = sab.cross_fwd_workspace_size
        kept.__dict__[size] = 1 << 40
        assert sab._given(kept) is kept and size in kept.__dict__ and kept._dense
        setattr(kept, field, value)
        assert sab._given(kept) is kept and not kept._dense and size not in kept.__dict__
        want = (((3, 8, 128), (7, 2, 128)) if field == "batch" else made._shapes)
        assert kept._shapes == want and kept._dtype == made._dtype
    kept = _rot(layout=1, s_max=7)
    assert kept._shapes == ((3, 7, 4, 128), (3, 7, 2, 128))
    kept.s_max, kept.n2 = 9, 1
    assert sab._given(kept)._shapes == ((3, 9, 4, 128), (3, 9, 1, 128))
    kept.layout = kept.s_max = 0
    assert sab._given(kept)._shapes == ((10, 4, 128), (10, 1, 128))
    kept.batch = -1
    assert sab._given(kept)._shapes[0][0] == 0
