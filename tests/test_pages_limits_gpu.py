"""Pages of the cache at the edges of what their operators take."""
from __future__ import annotations

import random

import pytest
import torch

import serve_util as S
from graph_nodes import captured_grids
from memory_bound_normalization_fwd_gb300 import binding as B
from test_pages_gpu import DEV, _cache, _i32, _same, _status

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


@pytest.mark.parametrize("most", [1, 2, 7, 100])
@pytest.mark.parametrize("shape", [(16, 8, 128), (1, 1, 7)])
def test_compact_in_few_ctas(most, shape):
    rng = random.Random(most)
    pages = 3000 if shape[0] == 1 else 700
    refs = [rng.randint(0, 2) for _ in range(pages)]
    live = [p for p in range(pages) if refs[p]]
    rng.shuffle(live)
    table = [live[:50], live[20:70]]
    c = _cache(pages, *shape)
    want = S.compact(c, refs, table)
    first = [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    rf, t = _i32(refs), _i32(table)
    got = B.cache_compact(c, rf, t, max_ctas=most)
    assert [g.tolist() for g in got] == [[want[0]], want[1], want[2]]
    _same(c, want[3])
    for a, b in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), first):
        a.copy_(b)
    got = B.cache_compact(c, rf, t, refs_out=rf, table_out=t, max_ctas=most)  # in place
    assert [g.tolist() for g in got] == [[want[0]], want[1], want[2]]
    _same(c, want[3])
    assert _status() == 0
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    grids = captured_grids(lambda: B.cache_compact(c, rf, t, refs_out=rf, table_out=t, workspace=ws, max_ctas=most))
    assert len(grids) == 2 and max(grids) <= most, grids


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_fork_of_a_last_page_that_is_not_there(first, fmt):
    """An entry of a parent's tokens that names no page is copied as it is, the last one's too: the child
    gets no page of other tokens for it."""
    page, pages = 4, 9
    c = _cache(pages, page, 2, 32, fmt, first)
    table = [[0, -1, -1], [1, pages, -1], [2, 3, -1], [-5, -1, -1]] + [[-1] * 3 for _ in range(5)]
    lengths = [6, 7, 5, 2, 0, 0, 0, 0, 0]
    refs = [1, 1, 1, 1, 0, 0, 0, 0, 1]
    t, ln, rf = _i32(table), _i32(lengths), _i32(refs)
    before = S.arrays(c)
    B.cache_fork(c, rf, t, ln, _i32([0, 1, 3]), _i32([4, 5, 6]))
    assert _status() == -12
    assert t.tolist()[4:7] == [[0, -1, -1], [1, pages, -1], [-5, -1, -1]] and ln.tolist()[4:7] == [6, 7, 2]
    assert rf.tolist() == [2, 2, 1, 1, 0, 0, 0, 0, 1]
    _same(c, before)
    # those beside it are forked as ever
    B.cache_fork(c, rf, t, ln, _i32([0, 2]), _i32([7, 8]))
    assert _status() == -12
    assert t.tolist()[7] == [0, -1, -1] and t.tolist()[8][0] == 2 and t.tolist()[8][2] == -1
    new = t.tolist()[8][1]
    assert 4 <= new < 8 and rf.tolist() == [3, 2, 2, 1] + [int(p == new) for p in range(4, 8)] + [1]
    for got, old in zip(S.arrays(c), before):
        if first:
            assert torch.equal(got[new, :, :1], old[3, :, :1])
        else:
            assert torch.equal(got[new, :1], old[3, :1])
        got[new] = old[new]
        assert torch.equal(got, old)
