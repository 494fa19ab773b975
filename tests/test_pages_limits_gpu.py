"""Pages of the cache at the edges of what their operators take."""
from __future__ import annotations

import pytest
import torch

from memory_bound_normalization_fwd_gb300 import binding as B
from test_pages_gpu import DEV, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [11_520_000, 11_600_001, 12_000_000, 12_580_000, 12_700_000])
def test_compact_of_millions_of_pages(pages):
    """Around the sizes from which a block's counts need more shared memory than a kernel has by default."""
    c = B.Cache(pages, 1, 1, 2, "e2m1")
    p = torch.arange(pages, device=DEV)
    for k, t in enumerate((c.k_codes, c.k_scales, c.v_codes, c.v_scales)):
        t.view(-1).copy_((p * (2 * k + 3) >> 3).to(torch.uint8))
    before = [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    refs = ((p * 2654435761 >> 7) % 5 < 2).int()
    L = int(refs.sum())
    live, rf, _ = B.cache_compact(c, refs, _i32([[-1]]))
    used = refs > 0
    src, dst = p[used & (p >= L)], p[~used & (p < L)]
    for t, got in zip(before, (c.k_codes, c.k_scales, c.v_codes, c.v_scales)):
        t[dst] = t[src]
        assert torch.equal(t, got)
    assert live.tolist() == [L] and bool((rf[:L] == 1).all()) and not bool(rf[L:].any())
