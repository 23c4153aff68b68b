"""Kept descriptors whose lengths are edited in place (and workspaces): the arrays behind
cu_seqlens are the caller's to reach (desc.cu_seqlens_q[1] = n), the library
reads them anew at every call, and so must what the tensors are checked against
and the workspace size kept with the descriptor: tensors of the old lengths under
a plan for new ones would be written past their ends."""
import pytest
import torch

import sparse_attention_backward_gb300 as sab
from sparse_attention_backward_gb300 import build as libbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()


ROT = dict(n1=4, n2=2, d=64)
MAKE = {
    "rotary": (lambda cu: sab.make_rotary_desc(sab.Rotary(64), cu, **ROT), ("cu_seqlens",), ()),         # (its workspace size is not kept)
    "norm": (lambda cu: sab.make_norm_rotary_desc(sab.Rotary(64), cu, **ROT), ("cu_seqlens",),
             (sab.norm_rotary_fwd_workspace_size, sab.norm_rotary_grad_workspace_size)),
    "cross": (lambda cu: sab.make_cross_desc(cu, cu, scale=0.1, **ROT), ("cu_seqlens_q", "cu_seqlens_kv"),
              (sab.cross_fwd_workspace_size, sab.cross_grad_workspace_size)),
    "window": (lambda cu: sab.make_window_desc(cu, cu, scale=0.1, **ROT), ("cu_seqlens_q", "cu_seqlens_kv"),
               (sab.window_fwd_workspace_size, sab.window_grad_workspace_size)),
    "paged": (lambda cu: sab.make_paged_desc(cu, scale=0.1, pages=9, page_size=16, width=400, **ROT), ("cu_seqlens_q",),
              (sab.paged_fwd_workspace_size, sab.paged_append_workspace_size)),
}


@pytest.mark.parametrize("which", MAKE)
@pytest.mark.parametrize("side", [0, 1])
def test_lengths_edited_in_place_are_followed(which, side):
    make, prefixes, sizes = MAKE[which]
    prefix = prefixes[min(side, len(prefixes) - 1)]
    d = make([0, 6, 10])
    for size in sizes:
        sab._size_of(d, size)
    assert sab._unchanged(d) and sab._given(d) is d and d._dense
    getattr(d, prefix)[2] = 5000
    assert not sab._unchanged(d)
    d = sab._given(d)
    at = 1 if prefix == "cu_seqlens_kv" else 0
    assert d._shapes[at][0] == 5000 and sab._unchanged(d)
    fresh = make([0, 6, 10])
    getattr(fresh, prefix)[2] = 5000
    for size in sizes:
        assert sab._size_of(d, size) == size(fresh)
    # the same number of rows, other sequences
    getattr(d, prefix)[1] = 4000
    assert not sab._unchanged(d)
    d = sab._given(d)
    for size in sizes:
        assert size not in d.__dict__
    assert d._shapes[at][0] == 5000


@pytest.mark.parametrize("which", MAKE)
def test_a_descriptor_that_was_left_alone_keeps_its_sizes(which):
    make, _, sizes = MAKE[which]
    d = make([0] * 70)
    for size in sizes:
        d.__dict__[size] = 1 << 40
    assert sab._given(d) is d and all(sab._size_of(d, size) == 1 << 40 for size in sizes) and d._dense
    d.batch = -1
    assert sab._given(d)._shapes[0][0] == 0


def test_workspaces_with_less_memory_than_elements_are_refused(lib):
    sab._lib_neighbours()
    small, large = torch.empty(16, dtype=torch.uint8), torch.empty(1000, dtype=torch.uint8)
    assert sab._scratch(large, 1000, "cpu") is large and sab._scratch(large[100:], 900, "cpu").data_ptr() == large.data_ptr() + 100
    assert sab._scratch(small, 17, "cpu").numel() == 17 and sab._scratch(None, 5, "cpu").numel() == 5
    for bad in (small[:1].expand(1000), large[::2]):
        with pytest.raises(ValueError, match="workspace"):
            sab._scratch(bad, 500, "cpu")
