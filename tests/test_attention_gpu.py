"""Attention over the quantised cache against the plain 64-bit implementation."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

import ops_util as U
import serve_util as S
from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
VARIANTS = ("generic", "auto")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _cu(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _filled(lens, page, heads, D, fmt, seed, first=False, dtype=torch.bfloat16, width=None):
    """A cache that holds `lens` tokens of each sequence on pages in any order, garbage in every
    other slot, and its table."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    cache = B.Cache(pages, page, heads, D, fmt, heads_first=first)
    for t in (cache.k_codes, cache.v_codes):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(255)
    order = torch.randperm(pages, generator=g).tolist()
    width = max(need + [1]) + 1 if width is None else width
    table = [[order.pop() for _ in range(n)] + [-1] * (width - n) for n in need]
    slots = [table[b][t // page] * page + t % page for b, n in enumerate(lens) for t in range(n)]
    kv = torch.randn(len(slots), 2 * heads, D, generator=g)
    kv[:, :heads, ::32] *= 6
    kv = kv.to(dtype).to(DEV)
    B.cache_write(cache, kv[:, :heads], kv[:, heads:], torch.tensor(slots, dtype=torch.int64, device=DEV))
    return cache, table


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _q(rows, H, D, dtype, seed):
    g = torch.Generator().manual_seed(seed + 77)
    return torch.randn(rows, H + 2, D, generator=g).to(dtype).to(DEV)[:, 1:H + 1]


def _run(cache, table, lens, counts, H, dtype, seed=0, scale=None, causal=True, window=0, status=0,
         variants=VARIANTS, q=None):
    cu = _cu(counts)
    q = _q(cu[-1], H, cache.head_dim, dtype, seed) if q is None else q
    sc = cache.head_dim ** -0.5 if scale is None else scale
    want = S.attention(cache, q, table, lens, cu, sc, causal, window)
    for variant in variants:
        out, lse = B.cache_attention(cache, q, _i32(table), _i32(lens), cu_q=_i32(cu), scale=scale,
                                     causal=causal, window=window, lse=True, variant=variant)
        assert B.lib().rmsnorm_check_device_status(0) == status, variant
        S.check_attention(out, lse, want, dtype, (variant, cache.fmt, cache.head_dim, H, counts))
    return out, lse


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("D", [32, 64, 80, 96, 128, 192, 256, 1, 7, 33, 40, 512])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_one_token_each(fmt, D, dtype):
    lens = [1, 0, 37, 130, 16, 64]
    cache, table = _filled(lens, 16, 2, D, fmt, D)
    _run(cache, table, lens, [1] * 6, 6, U.DT[dtype], D)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("page", [1, 5, 24, 64])
@pytest.mark.parametrize("heads,G", [(1, 16), (5, 1), (3, 7), (8, 8), (1, 33), (12, 2)])
def test_heads_and_pages(fmt, page, heads, G):
    lens = [70, 3, 201]
    for first in (False, True):
        cache, table = _filled(lens, page, heads, 64, fmt, page + G, first)
        _run(cache, table, lens, [1, 1, 1], heads * G, torch.bfloat16, page)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 20), (True, 100)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_several_queries(dtype, fmt, causal, window, D):
    # more queries than tokens (rows that see nothing), none, one, many
    lens, counts = [9, 50, 0, 130, 77, 33], [12, 0, 3, 65, 1, 33]
    cache, table = _filled(lens, 24, 2, D, fmt, D + window)
    _run(cache, table, lens, counts, 8, U.DT[dtype], window, causal=causal, window=window)


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_long_sequences_are_split_and_joined(D, fmt):
    lens = [5000, 1, 2777]
    cache, table = _filled(lens, 16, 1, D, fmt, D)
    for G in (1, 8, 16):
        _run(cache, table, lens, [1, 1, 1], G, torch.float16, G)


@pytest.mark.parametrize("D", [72, 80, 96, 176, 192, 224])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("page,heads,first", [(1, 1, False), (3, 1, True), (3, 3, False), (8, 2, True)])
def test_scale_bytes_anywhere_in_a_word(D, fmt, page, heads, first):
    # a head's 3, 5, 6 or 7 bytes begin at every place of a word; arrays that are not whole words
    lens = [67, 2, 41]
    cache, table = _filled(lens, page, heads, D, fmt, D + page, first)
    for dtype in (torch.bfloat16, torch.float32):
        _run(cache, table, lens, [1, 2, 1], 4 * heads, dtype, 1)


@pytest.mark.parametrize("D", [64, 96, 128, 192])
@pytest.mark.parametrize("window", [0, 30])
def test_rows_around_a_block(D, window):
    # rows of a key head around the 8, 16 and 32 of a block, long sequences and a short table
    for lens in ([900, 400], [130, 33]):
        cache, table = _filled(lens, 16, 2, D, "e2m1", D)
        for G, n in ((8, 1), (3, 3), (4, 4), (17, 1), (8, 3), (8, 4), (3, 11), (8, 5), (16, 3)):
            _run(cache, table, lens, [n, n], 2 * G, torch.bfloat16, n, window=window, variants=("auto",))


def test_many_sequences():
    lens = [(7 * i) % 61 for i in range(700)]
    cache, table = _filled(lens, 8, 2, 64, "e2m1", 1)
    _run(cache, table, lens, [1] * 700, 4, torch.bfloat16, 3, variants=("auto",))
    # more sequences than the plan of a call looks ahead at
    lens = [(5 * i) % 23 for i in range(5000)]
    cache, table = _filled(lens, 8, 1, 32, "e4m3", 2)
    _run(cache, table, lens, [1] * 5000, 2, torch.bfloat16, 4, variants=("auto",))


@pytest.mark.parametrize("G", [4, 5])
def test_a_prompt(G):
    lens, counts = [300, 190], [190, 190]
    for fmt in ("e2m1", "e4m3"):
        cache, table = _filled(lens, 16, 2, 128, fmt, 5)
        for dtype in (torch.bfloat16, torch.float16, torch.float32):
            _run(cache, table, lens, counts, 2 * G, dtype, 9, variants=("auto",))


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 150)])
def test_long_prompts(fmt, D, dtype, causal, window):
    """Enough rows for the tensor cores: blocks of 256 rows that end inside, sequences that hold more
    than their queries, and fewer, a group that is not a power of two."""
    heads, G = 6, 5
    lens, counts = [700, 300, 129, 40, 513], [300, 300, 129, 260, 1]
    cache, table = _filled(lens, 24, heads, D, fmt, D + window, first=bool(window))
    _run(cache, table, lens, counts, heads * G, U.DT[dtype], window, causal=causal, window=window, variants=("auto",))


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_long_prompts_with_what_is_not_finite_or_not_there(fmt):
    heads, G = 8, 8
    lens, counts = [500, 260, 300], [200, 250, 260]
    cache, table = _filled(lens, 16, heads, 128, fmt, 2)
    g = torch.Generator().manual_seed(3)
    # scales far apart, from token to token and from tile to tile
    cache.v_scales[torch.tensor(table[0][:31]).long()] += torch.randint(
        -9, 20, cache.v_scales[torch.tensor(table[0][:31]).long()].shape, generator=g).to(torch.uint8).to(DEV)
    cache.v_scales[table[0][28]] += 12
    for page, head, grp, which in ((table[0][20], 3, 2, "k"), (table[1][8], 0, 0, "v"), (table[1][15], 7, 3, "v")):
        getattr(cache, which + "_scales")[page, 5, head, grp] = 255
    table[2][3], table[2][9] = -1, cache.pages
    for dtype in (torch.bfloat16, torch.float16):
        _run(cache, table, lens, counts, heads * G, dtype, 1, status=-12, variants=("auto",))


def test_long_prompts_on_odd_strides_and_twice():
    heads, G, D = 8, 4, 128
    lens, counts = [600, 500], [600, 500]
    cache, table = _filled(lens, 16, heads, D, "e2m1", 2)
    cu, q = [0, 600, 1100], _q(1100, heads * G, D, torch.bfloat16, 3)
    want = S.attention(cache, q, table, lens, cu, D ** -0.5, True, 0)
    ref, lse = B.cache_attention(cache, q, _i32(table), _i32(lens), cu_q=_i32(cu), lse=True)
    S.check_attention(ref, lse, want, torch.bfloat16, "prompt")
    odd = torch.zeros(1100, heads * G + 1, D + 3, dtype=torch.bfloat16, device=DEV)
    for _ in range(3):  # rows of the output on no vector's border; the same bits
        B.cache_attention(cache, q, _i32(table), _i32(lens), cu_q=_i32(cu), out=odd[:, 1:, 1:D + 1])
        assert torch.equal(odd[:, 1:, 1:D + 1], ref)
    assert bool((odd[:, 0] == 0).all()) and bool((odd[..., 0] == 0).all()) and bool((odd[..., D + 1:] == 0).all())
    # rows behind the last sequence stay
    out = torch.full((1130, heads * G, D), 3.0, dtype=torch.bfloat16, device=DEV)
    more = torch.cat([q, q[:30]])
    B.cache_attention(cache, more, _i32(table), _i32(lens), cu_q=_i32(cu), out=out)
    assert torch.equal(out[:1100], ref) and bool((out[1100:] == 3).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t, ln, c = _i32(table), _i32(lens), _i32(cu)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got, _ = B.cache_attention(cache, q, t, ln, cu_q=c)
    graph.replay()
    assert torch.equal(ref, got)
    both = [B.cache_attention(cache, q, _i32(table), _i32(lens), cu_q=_i32(cu), stream=s)[0] for s in (side, None, side)]
    torch.cuda.synchronize()
    assert all(torch.equal(ref, b) for b in both)


def test_no_cu_is_one_row_each_and_out_and_strides():
    lens = [20, 33]
    cache, table = _filled(lens, 16, 2, 64, "e2m1", 8)
    q = _q(2, 4, 64, torch.bfloat16, 5)
    want = S.attention(cache, q, table, lens, [0, 1, 2], 0.3, True, 0)
    wide = torch.full((2, 6, 80), 7.0, dtype=torch.bfloat16, device=DEV)
    out, lse = B.cache_attention(cache, q, _i32(table), _i32(lens), scale=0.3, out=wide[:, 1:5, 8:72])
    assert lse is None
    S.check_attention(out, None, want, torch.bfloat16, "strides")
    wide[:, 1:5, 8:72] = 7.0
    assert bool((wide == 7).all())
    # rows that start on no vector's border
    q1 = torch.randn(2, 4, 65, device=DEV).to(torch.bfloat16)[..., 1:]
    want = S.attention(cache, q1, table, lens, [0, 1, 2], 0.3, True, 0)
    odd = torch.zeros(2, 4, 67, dtype=torch.bfloat16, device=DEV)
    B.cache_attention(cache, q1, _i32(table), _i32(lens), scale=0.3, out=odd[..., 1:65])
    S.check_attention(odd[..., 1:65], None, want, torch.bfloat16, "odd strides")


def test_cache_memory_on_no_vectors_border():
    lens = [20, 133]
    cache, table = _filled(lens, 16, 2, 64, "e4m3", 8)
    shifted = []
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        raw = torch.zeros(t.numel() + 16, dtype=torch.uint8, device=DEV)
        raw[3:3 + t.numel()] = t.flatten()
        shifted.append(raw[3:3 + t.numel()].view(t.shape))
    moved = B.Cache(cache.pages, 16, 2, 64, "e4m3", tensors=shifted)
    _run(moved, table, lens, [1, 1], 4, torch.bfloat16)


def test_rows_behind_the_last_sequence_stay():
    lens = [40]
    cache, table = _filled(lens, 16, 1, 64, "e2m1", 8)
    q = _q(9, 2, 64, torch.bfloat16, 5)
    for variant in VARIANTS:
        out = torch.full((9, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
        B.cache_attention(cache, q, _i32(table), _i32(lens), cu_q=_i32([0, 3]), out=out, variant=variant)
        assert bool((out[3:] == 5).all()) and not bool((out[:3] == 5).any())
        full = torch.empty_like(out)
        B.cache_attention(cache, q[:3], _i32(table), _i32(lens), cu_q=_i32([0, 3]), out=full[:3], variant=variant)
        assert torch.equal(out[:3], full[:3])


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_groups_that_are_not_finite(fmt):
    """k's NaN reaches the rows that see it, v's the group's values of those rows."""
    lens, counts = [50, 60, 45], [20, 20, 3]
    cache, table = _filled(lens, 16, 2, 128, fmt, 21)
    # sequence 0: token 40 of k's head 0; sequence 1: token 47 of v's head 1, values 32..63;
    # sequence 2: a first token of v outside of a window
    def at(b, t):
        return table[b][t // 16], t % 16
    p, i = at(0, 40)
    cache.k_scales[p, i, 0, 1] = 255
    p, i = at(1, 47)
    cache.v_scales[p, i, 1, 1] = 255
    p, i = at(2, 0)
    cache.v_scales[p, i, :, :] = 255
    cache.k_scales[p, i, :, :] = 255
    out, _ = _run(cache, table, lens, counts, 4, torch.bfloat16, 2, window=40)
    assert bool(torch.isnan(out).any()) and not bool(torch.isnan(out[40:]).any())


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_scales_of_any_size(fmt):
    """Tokens whose values lie many powers of two apart, and rows of q likewise."""
    lens = [100, 37]
    cache, table = _filled(lens, 16, 2, 64, fmt, 31)
    g = torch.Generator().manual_seed(3)
    cache.v_scales.copy_(torch.randint(100, 150, cache.v_scales.shape, generator=g, dtype=torch.uint8))
    cache.k_scales.copy_(torch.randint(112, 128, cache.k_scales.shape, generator=g, dtype=torch.uint8))
    q = _q(2, 8, 64, torch.float32, 4)
    q = q * torch.pow(2.0, torch.randint(-9, 3, (2, 8, 1), generator=g).float()).to(DEV)
    for dtype in (torch.float32, torch.bfloat16):
        _run(cache, table, lens, [1, 1], 8, dtype, q=q.to(dtype))
    # far apart: tiny and huge groups next to each other
    cache.v_scales.copy_(torch.randint(1, 240, cache.v_scales.shape, generator=g, dtype=torch.uint8))
    _run(cache, table, lens, [1, 1], 8, torch.float32, q=q)


def test_large_and_zero_queries():
    lens = [100, 37]
    cache, table = _filled(lens, 16, 2, 64, "e2m1", 31)
    for dtype, size in ((torch.float16, 60000.0), (torch.bfloat16, 2.0 ** 100), (torch.float32, 2.0 ** -120),
                        (torch.float16, 6e-8), (torch.float32, 0.0)):
        q = _q(2, 4, 64, torch.float32, 4)
        q = (q / q.abs().max() * size).to(dtype)
        # a scale that keeps the scores within what a softmax tells apart
        _run(cache, table, lens, [1, 1], 4, dtype, q=q, scale=0.1 / size if 1e-30 < size < 2.0 ** 90 else 2.0 ** -103
             if size > 1 else 0.1)


def test_pages_that_are_not_there():
    lens = [64, 64, 500]
    cache, table = _filled([64, 64, 64], 16, 2, 64, "e2m1", 13)
    table[0][1], table[1][0] = -1, cache.pages
    _run(cache, table, [64, 64, 64], [1, 2, 1], 4, torch.bfloat16, status=-12)
    # lengths of nothing, and below
    out, _ = B.cache_attention(cache, _q(3, 4, 64, torch.bfloat16, 0), _i32(table), _i32([0, 0, -5]))
    assert bool((out == 0).all())
    assert B.rmsnorm_check_device_status(0) == 0


@pytest.mark.parametrize("D,heads,G,counts", [(64, 2, 2, [3, 1]), (512, 2, 2, [3, 1]), (128, 8, 8, [310, 200])])
def test_tokens_past_the_row_of_the_table(D, heads, G, counts):
    """A length that the row has no room for: the positions are the true ones, the tokens past the
    row are left out and reported."""
    held = [400, 200]
    cache, table = _filled(held, 16, heads, D, "e2m1", 5, width=25)
    _run(cache, table, [440, 200], counts, heads * G, torch.bfloat16, 1, status=-12, variants=("auto",))
    _run(cache, table, [440, 200], counts, heads * G, torch.bfloat16, 1, status=-12, variants=("auto",), window=60)
    _run(cache, table, [400, 200], counts, heads * G, torch.bfloat16, 1, variants=("auto",))


def test_a_wait_that_runs_out():
    """Waits of the tensor cores' roles on one another, with no time to wait: the status says so, and the
    next call is whole."""
    heads, G, lens = 8, 8, [600, 500]
    cache, table = _filled(lens, 16, heads, 128, "e4m3", 2)
    q = _q(1100, heads * G, 128, torch.bfloat16, 3)
    args = (cache, q, _i32(table), _i32(lens))
    cu = _i32([0, 600, 1100])
    ref, _ = B.cache_attention(*args, cu_q=cu)
    B.cache_attention(*args, cu_q=cu, wait_limit_ns=1)
    assert B.lib().rmsnorm_check_device_status(0) == -7
    assert B.lib().rmsnorm_check_device_status(0) == 0
    again, _ = B.cache_attention(*args, cu_q=cu)
    assert torch.equal(ref, again) and B.lib().rmsnorm_check_device_status(0) == 0


def test_the_first_call_of_a_process_may_be_captured():
    code = """
import sys, torch
sys.path.insert(0, %r)
from memory_bound_normalization_fwd_gb300 import binding as B
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
for rows, heads in ((2, 4), (2400, 32)):
    c = B.Cache(200, 16, 4, 64, "e2m1")
    c.k_scales.fill_(127), c.v_scales.fill_(127), c.v_codes.fill_(0x22)
    n = rows // 2
    q = torch.randn(rows, heads, 64, device="cuda").to(torch.bfloat16)
    t, ln, cu = i32([list(range(100)), list(range(100, 200))]), i32([1500, 1400]), i32([0, n, rows])
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        B.cache_attention(c, q, t, ln, cu_q=cu, out=out, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert bool((out == 1).all()), out
""" % ROOT
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr[-2000:]


def test_slots_past_32_bits():
    """A cache of more than 2^31 code bytes: the last pages are read where they are."""
    pages = (1 << 31) // (64 * 8 * 256) + 40
    cache = B.Cache(pages, 64, 8, 256, "e4m3")
    g = torch.Generator().manual_seed(1)
    table = [[pages - 1, 0, pages - 7], [pages // 2, pages - 2, 5]]
    lens = [190, 131]
    slots = [table[b][t // 64] * 64 + t % 64 for b, n in enumerate(lens) for t in range(n)]
    kv = torch.randn(len(slots), 16, 256, generator=g).to(torch.bfloat16).to(DEV)
    B.cache_write(cache, kv[:, :8], kv[:, 8:], torch.tensor(slots, dtype=torch.int64, device=DEV))
    q = _q(2, 16, 256, torch.bfloat16, 0)
    outs = [B.cache_attention(cache, q, _i32(table), _i32(lens), variant=v)[0] for v in VARIANTS]
    small = B.Cache(6, 64, 8, 256, "e4m3", tensors=[
        torch.stack([t[p] for r in table for p in r]).contiguous()
        for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)])
    ref = [B.cache_attention(small, q, _i32([[0, 1, 2], [3, 4, 5]]), _i32(lens), variant=v)[0] for v in VARIANTS]
    assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_other_streams_captured_and_at_once():
    lens = [3000, 500, 7]
    cache, table = _filled(lens, 16, 2, 128, "e2m1", 3)
    q = _q(3, 8, 128, torch.bfloat16, 1)
    t, ln = _i32(table), _i32(lens)
    ref = B.cache_attention(cache, q, t, ln)[0]
    for _ in range(3):  # the same bits every time
        assert torch.equal(ref, B.cache_attention(cache, q, t, ln)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [B.cache_attention(cache, q, t, ln, stream=side)[0] for _ in range(4)]
    here = [B.cache_attention(cache, q, t, ln)[0] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(ref, o) for o in outs + here)
    # two graphs that share a workspace, replayed one after the other, over changed inputs
    ws = torch.empty(B.rmsnorm_cache_attention_workspace_size(2, 8, 128, 3, 3), dtype=torch.uint8, device=DEV)
    graphs, res = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res.append(B.cache_attention(cache, q, t, ln, workspace=ws)[0])
        graphs.append(graph)
    ln.copy_(_i32([100, 2999, 64]))
    ln[1] = 480
    want = B.cache_attention(cache, q, t, ln)[0]
    for graph in graphs * 2:
        graph.replay()
    torch.cuda.synchronize()
    # (bits: sequence 2 now reaches slots that were never written, whose scales say NaN, and
    # tokens past its pages, which are reported)
    assert all(torch.equal(want.view(torch.int16), r.view(torch.int16)) for r in res)
    assert B.lib().rmsnorm_check_device_status(0) == -12


def test_joined_with_attention_over_other_tokens():
    """lse is what two parts of a context are joined by."""
    lens = [96]
    cache, table = _filled(lens, 16, 2, 64, "e4m3", 3)
    q = _q(1, 4, 64, torch.float32, 1)
    whole, wl = B.cache_attention(cache, q, _i32(table), _i32([96]), lse=True)
    a, la = B.cache_attention(cache, q, _i32(table), _i32([48]), lse=True)
    b, lb = B.cache_attention(cache, q, _i32([table[0][3:6]]), _i32([48]), lse=True)
    top = torch.logaddexp(la, lb)
    both = a * torch.exp(la - top)[..., None] + b * torch.exp(lb - top)[..., None]
    assert torch.allclose(top, wl, atol=1e-5) and torch.allclose(both, whole, atol=1e-5)


def test_no_rows_and_no_sequences():
    cache, table = _filled([5], 16, 2, 64, "e4m3", 3)
    out, lse = B.cache_attention(cache, _q(0, 4, 64, torch.bfloat16, 0), _i32(table)[:0], _i32([]), lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, _ = B.cache_attention(cache, _q(0, 4, 64, torch.bfloat16, 0), _i32(table), _i32([5]), cu_q=_i32([0, 0]))
    assert out.shape == (0, 4, 64)
