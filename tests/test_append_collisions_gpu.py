"""New tokens that a page table sends to the same place of the cache: parts of 16
bytes of either, and nothing else touched; and sequences that share the pages of
a common prefix, which are read only."""
import pytest
import torch

import sparse_attention_backward_gb300 as sab

from .test_window_gpu import BF, HF, Case, Pages, check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n2,d", [(1, 64), (8, 128), (5, 8)])
def test_tokens_of_the_same_place(n2, d):
    batch, page = 40, 16
    g = torch.Generator().manual_seed(n2)
    k, v = (torch.randn(batch, n2, d, generator=g).cuda().to(BF) for _ in range(2))
    kc, vc = (torch.randn(3, page, n2, d, generator=g).cuda().to(BF) for _ in range(2))
    before = kc.clone(), vc.clone()
    table = torch.full((batch, 2), 1, dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), 21, dtype=torch.int32, device="cuda")         # all of them to row 4 of page 1
    sab.paged_append(k, v, kc, vc, table, lens, list(range(batch + 1)), check=True)
    for new, cache, old in zip((k, v), (kc, vc), before):
        parts = cache[1, 4].reshape(-1, 8)
        of = (new.reshape(batch, -1, 8) == parts).all(-1).any(0)
        assert bool(of.all())
        cache[1, 4] = old[1, 4]
        assert torch.equal(cache, old)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_sequences_that_share_pages(dtype):
    c = Case([1, 1, 9], [300, 300, 300], 8, 2, 128, dtype, -1, 0, seed=95)
    for x in (c.k, c.v):
        x[300:556], x[600:856] = x[:256].clone(), x[:256].clone()
    p = Pages(c, 32)
    p.table[1:, :8] = p.table[0, :8]
    check_forward(c, *p.forward(c))
