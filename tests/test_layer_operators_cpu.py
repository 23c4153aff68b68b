"""Windowed attention, the paged cache and the norms with rotation without a GPU:
the entry points are exported, and phase 1 and the host-side checks of phase 2
refuse what the header refuses before anything is enqueued."""
import ctypes
import os
import re

import pytest
import torch

import sparse_attention_backward_gb300 as sab
from sparse_attention_backward_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPE, NULL, ALIGN = sab.SAG_ERR_SHAPE, sab.SAG_ERR_NULL, sab.SAG_ERR_ALIGN
UNSUP, DTYPE, WORK, OK = sab.SAG_ERR_UNSUPPORTED, sab.SAG_ERR_DTYPE, sab.SAG_ERR_WORKSPACE, sab.SAG_OK
MIB = 1024 * 1024


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return sab._lib_neighbours()


def test_declared_and_exported(lib):
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "selattn.h")).read(), flags=re.S)
    names = set(re.findall(r"\b((?:norm_rotary|window_attn|paged)_\w*)\s*\(", txt))
    assert names == set(sab.EXPORTED_LAYER)
    for n in names:
        assert hasattr(lib, n)


def _phase1(lib, name, desc):
    n = ctypes.c_size_t(12345)
    return getattr(lib, name)(ctypes.byref(desc), ctypes.byref(n)), n.value


def _set(desc, fields):
    for k, v in fields.items():
        setattr(desc, k, v)
    return desc


def _window(**kw):
    a = dict(cu=[0, 3, 3, 10], ck=[0, 5, 6, 10], n1=4, n2=2, d=128, scale=0.1, left=3, right=0, dtype=sab.SAG_BF16, layout=0, s1=0, s2=0)
    a.update({k: v for k, v in kw.items() if k in a})
    d = sab.make_window_desc(a["cu"], a["ck"], a["n1"], a["n2"], a["d"], a["scale"], a["left"], a["right"], a["dtype"], a["layout"],
                             a["s1"], a["s2"])
    return _set(d, {k: v for k, v in kw.items() if k not in a})


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(d=64), OK), (dict(left=-1, right=-1), OK), (dict(left=-2 ** 31, right=2 ** 31 - 1), OK), (dict(left=0, right=0), OK),
    (dict(d=96), UNSUP), (dict(d=192), UNSUP), (dict(d=0), SHAPE), (dict(n1=3), SHAPE), (dict(n1=66, n2=2), SHAPE), (dict(n2=0), SHAPE),
    (dict(n1=129, n2=129), SHAPE), (dict(dtype=2), DTYPE), (dict(layout=2), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(s1=7), SHAPE), (dict(layout=1, s1=7, s2=5), OK),
    (dict(layout=1, s1=6, s2=5), SHAPE), (dict(layout=1, s1=7, s2=3), SHAPE), (dict(cu=[0, 3, 2, 10]), SHAPE), (dict(cu=[1, 3, 3, 10]), SHAPE),
    (dict(q_stride=513), SHAPE), (dict(q_stride=504), SHAPE), (dict(q_stride=520), OK), (dict(v_stride=248), SHAPE), (dict(v_stride=-8), SHAPE),
    (dict(cu=[0] * 4, ck=[0] * 4), OK), (dict(cu=[0, 2 * MIB], ck=[0, 2 * MIB]), OK), (dict(cu=[0, 2 * MIB + 1], ck=[0, 1]), SHAPE),
    (dict(cu=[0] * 65538, ck=[0] * 65538), UNSUP),
])
def test_window_phase1(lib, kw, want):
    for name in ("window_attn_fwd_workspace_size", "window_attn_grad_workspace_size"):
        st, n = _phase1(lib, name, _window(**kw))
        assert st == want and (n > 0 if want == OK else n == 12345)


def test_window_phase2(lib):
    d = _window()
    need = sab.window_fwd_workspace_size(d)
    io = sab.ScaIo(*[4096] * 6)
    io.key_mask = None
    call = lambda x, ws=4096, n=need: lib.window_attn_fwd(ctypes.byref(d), x and ctypes.byref(x), ws, n, None)  # noqa: E731
    assert call(None) == NULL
    assert call(io, None) == WORK and call(io, 4096, need - 1) == WORK and call(io, 4100) == ALIGN
    for name in ("query", "key", "value", "attention_out", "softmax_lse"):
        for bad, want in ((None, NULL), (4104, ALIGN)):
            keep = getattr(io, name)
            setattr(io, name, bad)
            assert call(io) == want, name
            setattr(io, name, keep)
    need = sab.window_grad_workspace_size(d)
    io = sab.ScaIo(*[4096] * 10)
    io.key_mask = None
    grad = lambda x, ws=4096, n=need: lib.window_attn_grad(ctypes.byref(d), ctypes.byref(x), ws, n, None)  # noqa: E731
    assert grad(io, None) == WORK and grad(io, 4096, need - 1) == WORK
    for name in ("query", "key", "value", "attention_out", "attention_out_grad", "softmax_lse", "dq", "dk", "dv"):
        for bad, want in ((None, NULL), (4104, ALIGN)):
            keep = getattr(io, name)
            setattr(io, name, bad)
            assert grad(io) == want, name
            setattr(io, name, keep)
    assert lib.window_attn_fwd(None, ctypes.byref(io), 4096, need, None) == NULL
    assert lib.window_attn_fwd_workspace_size(ctypes.byref(d), None) == NULL
    assert lib.window_attn_query_error(None, None) == NULL


@pytest.mark.parametrize("given,held", [(0, 0), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1),
                                        (2 ** 63, 2 ** 31 - 1), (-1, -1), (-2 ** 32, -1), (-2 ** 31 - 5, -1)])
def test_sides_beyond_32_bits(given, held):
    w = sab.make_window_desc([0, 3], [0, 5], 2, 2, 64, 0.1, left=given, right=given)
    p = sab.make_paged_desc([0, 3], 2, 2, 64, 0.1, 8, 16, 4, left=given, right=given)
    assert (w.left, w.right, p.left, p.right) == (held,) * 4


@pytest.mark.parametrize("step,ok", [((64, 0), False), ((0, 128), False), ((128 * 15, 128), False), ((128 * 16, 64), False),
                                     ((128 * 16, 127), False), ((256, 128), False), ((128 * 17, 128), True), ((256 * 16, 256), True)])
def test_caches_whose_rows_overlap_are_refused(step, ok):
    """Strides of 0 mean dense ones to the library, which would look beyond an expanded tensor."""
    t = torch.empty(64 * 1024, dtype=torch.bfloat16).as_strided((4, 16, 2, 64), step + (64, 1))
    if ok:
        assert sab._cache_strides("k_cache", t, t.shape, t.dtype, t.get_device()) == (step[1], step[0])
        return
    with pytest.raises(ValueError, match="overlap"):
        sab._cache_strides("k_cache", t, t.shape, t.dtype, t.get_device())


def test_window_arguments():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):
        sab.window_forward(z(4, 2, 64), z(4, 2, 64), z(4, 2, 64), [0, 4], [0, 4], 0.1)
    with pytest.raises(ValueError):
        sab.make_window_desc([0, 4], [0, 4, 5], 2, 2, 64, 0.1)


def test_a_kept_descriptor_follows_fields_set_later():
    d = _window()
    sab._size_of(d, sab.window_fwd_workspace_size)
    d.n1 = 8
    d = sab._given(d)
    assert d._shapes[0] == (10, 8, 128) and sab.window_fwd_workspace_size not in d.__dict__


def _paged(**kw):
    a = dict(cu=[0, 3, 3, 10], n1=4, n2=2, d=128, scale=0.1, pages=9, page=16, width=4, left=-1, right=0, dtype=sab.SAG_BF16, layout=0, s1=0)
    a.update({k: v for k, v in kw.items() if k in a})
    d = sab.make_paged_desc(a["cu"], a["n1"], a["n2"], a["d"], a["scale"], a["pages"], a["page"], a["width"], a["left"], a["right"],
                            a["dtype"], a["layout"], a["s1"])
    return _set(d, {k: v for k, v in kw.items() if k not in a})


@pytest.mark.parametrize("kw,want,append", [
    (dict(), OK, OK), (dict(d=64), OK, OK), (dict(d=192), UNSUP, OK), (dict(d=512), UNSUP, OK), (dict(d=520), SHAPE, SHAPE),
    (dict(d=60), UNSUP, UNSUP), (dict(page=8), UNSUP, UNSUP), (dict(page=24), UNSUP, UNSUP), (dict(page=48), OK, OK), (dict(page=0), SHAPE, SHAPE),
    (dict(page=65536), OK, OK), (dict(page=65552), SHAPE, SHAPE), (dict(pages=0), SHAPE, SHAPE), (dict(width=0), SHAPE, SHAPE),
    (dict(page=65536, width=4096), OK, OK), (dict(page=65536, width=4097), SHAPE, SHAPE), (dict(n1=3), SHAPE, SHAPE), (dict(n1=68), SHAPE, SHAPE),
    (dict(dtype=3), DTYPE, DTYPE), (dict(layout=1, s1=7), OK, OK), (dict(layout=1, s1=6), SHAPE, SHAPE), (dict(s1=7), SHAPE, SHAPE),
    (dict(scale=0.0), SHAPE, SHAPE), (dict(kv_expected=-1), SHAPE, SHAPE), (dict(kv_expected=64), OK, OK), (dict(reserved_=1), SHAPE, SHAPE),
    (dict(k_row=248), SHAPE, SHAPE), (dict(k_row=257), SHAPE, SHAPE), (dict(k_row=512), OK, OK), (dict(v_page=4096), OK, OK),
    (dict(v_page=4088), SHAPE, SHAPE), (dict(v_row=512, v_page=4096), SHAPE, SHAPE), (dict(v_row=512, v_page=7936), OK, OK),
    (dict(q_stride=504), SHAPE, SHAPE), (dict(k_stride=248), SHAPE, SHAPE), (dict(v_stride=260), SHAPE, SHAPE), (dict(cu=[0, 0]), OK, OK),
    (dict(cu=[0, 2 * MIB + 1]), SHAPE, SHAPE), (dict(cu=[0] * 65538), UNSUP, UNSUP),
])
def test_paged_phase1(lib, kw, want, append):
    for name, w in (("paged_attn_fwd_workspace_size", want), ("paged_append_workspace_size", append)):
        st, n = _phase1(lib, name, _paged(**kw))
        assert st == w and (n > 0 if w == OK else n == 12345), name


def test_paged_phase2(lib):
    d = _paged()
    for entry, size, names in ((lib.paged_attn_fwd, sab.paged_fwd_workspace_size,
                                ("query", "key_cache", "value_cache", "attention_out", "softmax_lse")),
                               (lib.paged_append, sab.paged_append_workspace_size, ("key", "value", "key_cache", "value_cache"))):
        need = size(d)
        io = sab.SpaIo(*[4096] * 9)
        call = lambda x, ws=4096, n=need: entry(ctypes.byref(d), x and ctypes.byref(x), ws, n, None)  # noqa: E731
        assert call(None) == NULL and entry(None, ctypes.byref(io), 4096, need, None) == NULL
        assert call(io, None) == WORK and call(io, 4096, need - 1) == WORK and call(io, 4100) == ALIGN
        for name in names + ("page_table", "kv_lens"):
            for bad, want in ((None, NULL), (4098, ALIGN)):
                setattr(io, name, bad)
                assert call(io) == want, name
                setattr(io, name, 4096)
    assert lib.paged_query_error(None, None) == NULL


def test_pieces_have_room_in_the_workspace(lib):
    """One token over a long cache: pieces of 128 rows of O, maximum and sum for each."""
    n = [_phase1(lib, "paged_attn_fwd_workspace_size", _paged(cu=[0, 1], page=64, width=w))[1] for w in (16, 2048)]
    assert n[0] < 64 * 1024 < 16 * 128 * 130 * 4 < n[1] < 64 * MIB
    kept = _phase1(lib, "paged_attn_fwd_workspace_size", _paged(cu=[0, 1], page=64, width=2048, kv_expected=1024))[1]
    assert kept == n[0]


def _norm(**kw):
    a = dict(cu=[0, 3, 3, 10], n1=4, n2=2, d=128, d_rot=64, offset=0, dtype=sab.SAG_BF16, layout=0, s_max=0, eps=1e-6, plus=0.0)
    a.update({k: v for k, v in kw.items() if k in a})
    r = sab.Rotary(a["d_rot"], offset=a["offset"])
    d = sab.make_norm_rotary_desc(r, a["cu"], a["n1"], a["n2"], a["d"], a["eps"], a["plus"], a["dtype"], a["layout"], a["s_max"])
    return _set(d, {k: v for k, v in kw.items() if k not in a})


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(n2=0), OK), (dict(offset=64), OK), (dict(offset=65), SHAPE), (dict(d=513), SHAPE), (dict(n1=129), SHAPE),
    (dict(dtype=2), DTYPE), (dict(layout=2), SHAPE), (dict(s_max=5), SHAPE), (dict(layout=1, s_max=7), OK), (dict(layout=1, s_max=6), SHAPE),
    (dict(cu=[0, 5, 4]), SHAPE), (dict(cu=[0, 0]), OK), (dict(cu=[0] * 65538), UNSUP), (dict(eps=0.0), SHAPE), (dict(eps=-1e-6), SHAPE),
    (dict(eps=float("inf")), SHAPE), (dict(eps=1e-60), SHAPE), (dict(eps=1e60), SHAPE), (dict(plus=float("nan")), SHAPE), (dict(plus=1.0), OK),
    (dict(weight_fp32=2), SHAPE), (dict(reserved_=1), SHAPE), (dict(q_stride=511), SHAPE), (dict(q_grad_stride=511), SHAPE),
    (dict(k_grad_stride=-1), SHAPE), (dict(q_grad_stride=513), OK), (dict(style=2), SHAPE), (dict(magnitude=float("nan")), SHAPE),
])
def test_norm_phase1(lib, kw, want):
    for name in ("norm_rotary_fwd_workspace_size", "norm_rotary_grad_workspace_size"):
        st, n = _phase1(lib, name, _norm(**kw))
        assert st == want and (n == 12345) == (want != OK), name
    if want == OK:
        assert n > 0 and _phase1(lib, "norm_rotary_fwd_workspace_size", _norm(**kw))[1] == 0


def test_norm_phase2(lib):
    d = _norm()
    io = sab.SnrIo(*[4096 * (1 + i) for i in range(13)])
    call = lambda x, e=lib.norm_rotary_fwd, ws=None, n=0: e(ctypes.byref(d), x and ctypes.byref(x), ws, n, None)  # noqa: E731
    assert call(None) == NULL and lib.norm_rotary_fwd(None, ctypes.byref(io), None, 0, None) == NULL
    need = sab.norm_rotary_grad_workspace_size(d)
    grad = lambda x, ws=65536, n=need: call(x, lib.norm_rotary_grad, ws, n)  # noqa: E731
    assert grad(io, None) == WORK and grad(io, 65536, need - 1) == WORK and grad(io, 65544) == ALIGN
    for names, e in ((("query", "key", "query_out", "key_out"), call),
                     (("query", "key", "query_out_grad", "key_out_grad", "query_grad", "key_grad"), grad)):
        for name in names:
            keep = getattr(io, name)
            for bad, want in ((None, NULL), (4104, ALIGN)):
                setattr(io, name, bad)
                assert e(io) == want, name
            setattr(io, name, keep)
    for name in ("query_weight", "key_weight", "positions"):
        keep = getattr(io, name)
        setattr(io, name, 4099)
        assert call(io) == ALIGN, name
        setattr(io, name, keep)
    io.query_weight_grad = 4098
    assert grad(io) == ALIGN
    # an output over its input with another stride
    io.query_out = io.query
    d.q_out_stride = 1024
    assert call(io) == SHAPE
    io.query_weight_grad, io.query_grad = 4096, io.query_out_grad
    assert grad(io) == SHAPE


def test_norm_arguments():
    z = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sab.norm_rotary_forward(z, None, sab.Rotary(64), cu_seqlens=[0, 4])
    with pytest.raises(ValueError):
        sab.norm_rotary_backward(z, z, z, None, sab.Rotary(64), cu_seqlens=[0, 4])
    with pytest.raises(ValueError):
        sab.paged_forward(z, z, z, z, z, [0, 4], 0.1)
    with pytest.raises(ValueError):
        sab.paged_append(z, z, z, z, z, z, [0, 4])
