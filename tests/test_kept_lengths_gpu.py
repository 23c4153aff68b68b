"""Calls with kept descriptors whose lengths were edited in place: tensors of the
old lengths are refused before anything is launched, and other sequences of the
same rows give what a new descriptor gives."""
import pytest
import torch

import sparse_attention_backward_gb300 as sab

pytestmark = pytest.mark.gpu

ROT = dict(n1=4, n2=2, d=64)


def _calls():
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn(10, n, 64, generator=g).cuda().bfloat16() for n in (4, 2))
    kc = torch.randn(9, 16, 2, 64, generator=g).cuda().bfloat16()
    w = torch.randn(64, generator=g).cuda().bfloat16()
    table = torch.arange(8, dtype=torch.int32, device="cuda").reshape(2, 4)
    lens = torch.tensor([40, 30], dtype=torch.int32, device="cuda")
    rot = sab.Rotary(64)
    o, lse = torch.randn_like(q), torch.randn(10, 4, device="cuda")
    caches = lambda: (torch.zeros_like(kc), torch.zeros_like(kc))  # noqa: E731
    pair = ("cu_seqlens_q", "cu_seqlens_kv")
    return {
        "rotary": (lambda cu: sab.make_rotary_desc(rot, cu, **ROT), ("cu_seqlens",), lambda d: sab.rotary_forward(q, k, None, desc=d)),
        "norm": (lambda cu: sab.make_norm_rotary_desc(rot, cu, **ROT), ("cu_seqlens",),
                 lambda d: sab.norm_rotary_forward(q, k, None, w, w, desc=d)),
        "norm gradient": (lambda cu: sab.make_norm_rotary_desc(rot, cu, **ROT), ("cu_seqlens",),
                          lambda d: sab.norm_rotary_backward(q, k, q, k, None, w, w, desc=d)),
        "cross": (lambda cu: sab.make_cross_desc(cu, cu, scale=0.1, **ROT), pair, lambda d: sab.cross_forward(q, k, k, desc=d)),
        "cross gradient": (lambda cu: sab.make_cross_desc(cu, cu, scale=0.1, **ROT), pair,
                           lambda d: sab.cross_backward(q, k, k, o, q, lse, desc=d)),
        "window": (lambda cu: sab.make_window_desc(cu, cu, scale=0.1, **ROT), pair, lambda d: sab.window_forward(q, k, k, desc=d)),
        "window gradient": (lambda cu: sab.make_window_desc(cu, cu, scale=0.1, **ROT), pair,
                            lambda d: sab.window_backward(q, k, k, o, q, lse, desc=d)),
        "paged": (lambda cu: sab.make_paged_desc(cu, scale=0.1, pages=9, page_size=16, width=4, **ROT), ("cu_seqlens_q",),
                  lambda d: sab.paged_forward(q, kc, kc, table, lens, desc=d)),
        "append": (lambda cu: sab.make_paged_desc(cu, scale=0.1, pages=9, page_size=16, width=4, **ROT), ("cu_seqlens_q",),
                   lambda d: sab.paged_append(k, k, *caches(), table, lens, desc=d)),
    }


@pytest.mark.parametrize("which", ["rotary", "norm", "norm gradient", "cross", "cross gradient", "window", "window gradient", "paged",
                                   "append"])
def test_lengths_edited_in_place(which):
    make, prefixes, call = _calls()[which]
    d = make([0, 6, 10])
    call(d)
    for p in prefixes:
        getattr(d, p)[1] = 3
    for x, y in zip(call(d), call(make([0, 3, 10]))):
        assert torch.equal(x, y)
    for p in prefixes:
        getattr(d, p)[2] = 5000
    with pytest.raises(ValueError):
        call(d)
    torch.cuda.synchronize()
