"""Pages of the cache copied, forked, freed and compacted, against plain lists. Every byte and
every count has to be equal."""
from __future__ import annotations

import random

import pytest
import torch

import serve_util as S
from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cache(pages, page, heads, D, fmt="e2m1", first=False, values=True, seed=0):
    c = B.Cache(pages, page, heads, D, fmt, heads_first=first, values=values)
    g = torch.Generator().manual_seed(seed)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        if t is not None:
            t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    return c


def _same(cache, want):
    for got, w in zip(S.arrays(cache), want):
        assert torch.equal(got, w)


def _status():
    return B.lib().rmsnorm_check_device_status(0)


# page size, heads, head size: whole vectors, and sizes that are none
SHAPES = [(16, 8, 128), (1, 8, 128), (1, 1, 7), (5, 3, 33), (24, 5, 96), (64, 8, 256), (3, 1, 64), (2, 3, 6)]


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES)
def test_copy(fmt, shape):
    for values in (True, False):
        c = _cache(23, *shape, fmt=fmt, values=values, first=values)
        want = S.arrays(c)
        src, dst = [3, -1, 22, 0, 7, 7, 5], [4, 9, 1, 21, -1, 13, -5]
        for t in want:
            old = t.clone()
            for a, b in zip(src, dst):
                if a >= 0 and b >= 0:
                    t[b] = old[a]
        B.cache_copy_pages(c, _i32(src), _i32(dst))
        _same(c, want)
        assert _status() == 0
        B.cache_copy_pages(c, _i32([]), _i32([]))
        B.cache_copy_pages(c, _i32([23, 2, 1 << 30]), _i32([5, 23, 8]))  # past the cache
        _same(c, want)
        assert _status() == -12


def _shared(rng, S_, width, pages, page, most):
    """A table with sequences that share pages: their lengths, counts and rows."""
    order = list(range(pages))
    rng.shuffle(order)
    table, lengths, refs = [[-1] * width for _ in range(S_)], [0] * S_, [0] * pages
    for b in range(most):
        n = rng.randint(0, width * page)
        need = -(-n // page)
        if need > len(order):
            break
        lengths[b] = n
        for j in range(need):
            table[b][j] = order.pop()
            refs[table[b][j]] += 1
    for b in range(most, min(S_, most + 3)):  # full pages shared with the row before
        other = b - most
        lengths[b] = lengths[other] // page * page
        for j in range(lengths[b] // page):
            table[b][j] = table[other][j]
            refs[table[b][j]] += 1
    return table, lengths, refs


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("first", [False, True])
def test_fork_and_free(fmt, shape, first):
    rng = random.Random(str((fmt, shape)))
    page, pages, width = shape[0], 61, 5
    c = _cache(pages, *shape, fmt=fmt, first=first)
    table, lengths, refs = _shared(rng, 20, width, pages, page, 6)
    empty = [b for b in range(20) if lengths[b] == 0 and b > 8]
    t, ln, rf = _i32(table), _i32(lengths), _i32(refs)
    parents = [0, 0, 1, 2, -1, 6, 7, 3]
    children = empty[:4] + [empty[4], empty[5], -3, empty[6]]
    out, reported = S.fork(c, refs, table, lengths, parents, children)
    B.cache_fork(c, rf, t, ln, _i32(parents), _i32(children))
    _same(c, out)
    assert (rf.tolist(), t.tolist(), ln.tolist()) == (refs, table, lengths)
    assert not reported and _status() == 0
    # freed: parents first, a child twice, padding
    rows = [0, children[0], children[0], -1, 2]
    for r in (0, children[0], 2):
        for p in table[r]:
            if p >= 0:
                refs[p] -= 1
        table[r], lengths[r] = [-1] * width, 0
    B.cache_free(rf, t, ln, _i32(rows))
    assert (rf.tolist(), t.tolist(), ln.tolist()) == (refs, table, lengths)
    assert _status() == 0
    B.cache_free(rf, t, ln, _i32([]))
    # everything freed: no page is in use
    B.cache_free(rf, t, ln, torch.arange(20, dtype=torch.int32, device=DEV))
    assert not bool(rf.any()) and not bool(ln.any()) and bool((t == -1).all())


def test_fork_that_cannot_be():
    page, width = 4, 3
    c = _cache(6, page, 1, 32)
    table = [[0, 1, -1], [2, 3, 4], [-1] * 3, [-1] * 3, [-1] * 3, [-1] * 3, [9, -1, -1], [-1] * 3, [-1] * 3]
    lengths = [6, 12, 0, 0, 0, 0, 4, 13, 0]
    refs = [1, 1, 1, 1, 1, 0]
    t, ln, rf = _i32(table), _i32(lengths), _i32(refs)
    cases = [([0, 0, 0], [2, 2, 3]),      # named twice; then no free page is left
             ([1, 0], [0, 99]),           # a child that is not empty, a row past the table
             ([99, 4], [4, 4]),           # a parent past the table, its own parent
             ([7], [4]),                  # more tokens than the row holds
             ([6], [4])]                  # a parent's page past the cache
    for parents, children in cases:
        out, reported = S.fork(c, refs, table, lengths, parents, children)
        B.cache_fork(c, rf, t, ln, _i32(parents), _i32(children))
        _same(c, out)
        assert (rf.tolist(), t.tolist(), ln.tolist()) == (refs, table, lengths), (parents, children)
        assert reported and _status() == -12
    B.cache_free(rf, t, ln, _i32([9, 1 << 30]))  # rows past the table
    assert rf.tolist() == refs and _status() == -12
    B.cache_free(rf, t, ln, _i32([6]))           # an entry past the cache
    assert _status() == -12
    rf.zero_()
    B.cache_free(rf, t, ln, _i32([1]))           # pages without references
    assert not bool(rf.any()) and _status() == -12


def test_fork_of_many():
    rng = random.Random(1)
    page, pages, width, P, C = 8, 9000, 6, 40, 3000
    c = _cache(pages, page, 1, 32)
    table, lengths, refs = _shared(rng, P + 3 + C, width, pages, page, P)
    for p in range(pages - 2500, pages):  # nearly all else in use: the free pages lie far back
        refs[p] = max(refs[p], 0)
    for p in range(200, 5000):
        refs[p] = max(refs[p], 1)
    parents = [rng.randrange(P) for _ in range(C)]
    children = list(range(P + 3, P + 3 + C))
    t, ln, rf = _i32(table), _i32(lengths), _i32(refs)
    out, reported = S.fork(c, refs, table, lengths, parents, children)
    B.cache_fork(c, rf, t, ln, _i32(parents), _i32(children))
    _same(c, out)
    assert (rf.tolist(), t.tolist(), ln.tolist()) == (refs, table, lengths)
    assert not reported and _status() == 0


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("pages", [1, 2, 33, 1024, 1025, 5000])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 0.97, 1.0])
def test_compact(shape, pages, share):
    if pages > 100 and shape[0] * shape[1] * shape[2] > 4096:
        shape = (2, 1, 64)
    rng = random.Random(pages * 10 + int(share * 100))
    refs = [(rng.randint(1, 3) if rng.random() < share else 0) for _ in range(pages)]
    live = [p for p in range(pages) if refs[p]]
    rng.shuffle(live)
    table = [(live[b::4] + [-1] * 5)[:max(1, pages // 3)] for b in range(4)]
    width = max(len(r) for r in table)
    table = [r + [-1] * (width - len(r)) for r in table]
    for fmt, place in (("e2m1", False), ("e4m3", True)):
        c = _cache(pages, *shape, fmt=fmt, first=place)
        n, new, rows, out, reported = S.compact(c, refs, table)
        rf, t = _i32(refs), _i32(table)
        got = B.cache_compact(c, rf, t, refs_out=rf if place else None, table_out=t if place else None)
        assert got[0].tolist() == [n] and got[1].tolist() == new and got[2].tolist() == rows
        if not place:
            assert rf.tolist() == refs and t.tolist() == table
        _same(c, out)
        assert _status() == 0
        again = B.cache_compact(c, got[1], got[2])  # nothing is left to move
        assert again[0].tolist() == [n] and again[1].tolist() == new and again[2].tolist() == rows
        _same(c, out)


def test_compact_keeps_entries_that_name_nothing():
    c = _cache(40, 2, 1, 32)
    refs = [0] * 40
    refs[39] = 1
    table = [[39, 7, -1, 40, -9]]
    live, rf, t = B.cache_compact(c, _i32(refs), _i32(table))
    assert t.tolist() == [[0, 7, -1, 40, -9]] and live.tolist() == [1] and rf.tolist() == [1] + [0] * 39
    assert _status() == -12
    live, rf, t = B.cache_compact(c, _i32(refs), _i32([]).view(0, 5))  # a table of no rows
    assert live.tolist() == [1] and t.shape == (0, 5)


def test_compact_of_many_pages():
    pages = 1_300_001
    c = _cache(pages, 1, 1, 2, "e2m1")
    g = torch.Generator().manual_seed(4)
    refs = (torch.rand(pages, generator=g) < 0.4).int()
    before = S.arrays(c)
    live, rf, _ = B.cache_compact(c, refs.to(DEV), _i32([[-1]]))
    L = int(refs.sum())
    used, p = refs > 0, torch.arange(pages)
    src, dst = p[used & (p >= L)], p[~used & (p < L)]
    for t in before:
        t[dst] = t[src]
    _same(c, before)
    assert live.tolist() == [L] and bool((rf[:L] == 1).all()) and not bool(rf[L:].any())


def test_pages_past_32_bits():
    pages = (1 << 31) // (64 * 8 * 256) + 40
    c = B.Cache(pages, 64, 8, 256, "e4m3")
    c.k_codes[pages - 2].fill_(7)
    c.v_scales[pages - 2].fill_(9)
    B.cache_copy_pages(c, _i32([pages - 2]), _i32([pages - 1]))
    assert bool((c.k_codes[pages - 1] == 7).all()) and bool((c.v_scales[pages - 1] == 9).all())
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[pages - 1] = 2
    live, refs, table = B.cache_compact(c, refs, _i32([[pages - 1]]))
    assert bool((c.k_codes[0] == 7).all()) and table.tolist() == [[0]] and refs[0] == 2


def test_streams_and_graphs():
    rng = random.Random(3)
    page, pages, width = 16, 61, 5
    c = _cache(pages, page, 4, 64)
    table, lengths, refs = _shared(rng, 20, width, pages, page, 6)
    children = [b for b in range(20) if lengths[b] == 0 and b > 8][:5]
    t, ln, rf = _i32(table), _i32(lengths), _i32(refs)
    parents, kids = _i32([0, 1, 0, 2, 3]), _i32(children)
    out, _ = S.fork(c, refs, table, lengths, [0, 1, 0, 2, 3], children)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.cache_fork(c, rf, t, ln, parents, kids, stream=side)
    B.cache_free(rf, t, ln, kids, stream=side)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):  # freed and forked again, every replay the same
        B.cache_free(rf, t, ln, kids)
        B.cache_fork(c, rf, t, ln, parents, kids)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    _same(c, out)
    assert (rf.tolist(), t.tolist(), ln.tolist()) == (refs, table, lengths)
    assert _status() == 0
