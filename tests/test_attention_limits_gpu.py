"""Attention over the quantised cache at the edges of its number formats and its launches."""
from __future__ import annotations

import pytest
import torch

import serve_util as S
from memory_bound_normalization_fwd_gb300 import binding as B
from test_attention_gpu import DEV, _filled, _i32, _q, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [72, 80, 160, 224])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("heads", [1, 3, 8])
def test_short_slots_of_heads_that_are_not_whole_groups(D, fmt, heads):
    """What lies behind a token's codes in shared memory is zero before the first copy, whatever
    a call before left there (codes that are NaN, on the same SMs)."""
    lens = [(37 * i) % 120 for i in range(40)]
    cache, table = _filled(lens, 16, heads, D, fmt, D + heads)
    left = B.Cache(40, 64, heads, 256, "e4m3")
    for t in (left.k_codes, left.v_codes):
        t.fill_(0x7f)
    for t in (left.k_scales, left.v_scales):
        t.fill_(127)
    wide, one = _i32([[i] for i in range(40)]), _i32([64] * 40)
    q, ql = _q(40, 2 * heads, D, torch.bfloat16, 1), _q(40, 2 * heads, 256, torch.bfloat16, 2)
    want = S.attention(cache, q, table, lens, list(range(41)), D ** -0.5, True, 0)
    t, ln = _i32(table), _i32(lens)
    outs = []
    for _ in range(5):
        B.cache_attention(left, ql, wide, one)
        outs.append(B.cache_attention(cache, q, t, ln, lse=True))
    for out, lse in outs:
        S.check_attention(out, lse, want, torch.bfloat16, (D, fmt, heads))
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
    assert B.lib().rmsnorm_check_device_status(0) == 0


# ---- prompts on the tensor cores ---------------------------------------------------

HEADS, G, NEW = 4, 8, 256  # one sequence's rows are a wave of the tensor cores' blocks


def _prompt(lens, D, fmt, seed, first=False):
    """A cache whose sequences' v has the scale byte 127 and codes that are numbers."""
    cache, table = _filled(lens, 16, HEADS, D, fmt, seed, first)
    g = torch.Generator().manual_seed(seed + 1)
    cache.v_codes.copy_(torch.randint(0, 256, cache.v_codes.shape, generator=g, dtype=torch.uint8) & 0xf7)
    cache.v_scales.fill_(127)
    return cache, table


def _tokens(cache, table_row, from_, to):
    """(pages, places in them) of a sequence's tokens."""
    t = torch.arange(from_, to)
    pages = torch.tensor(table_row)[t // cache.page_size]
    return (pages.to(DEV), (t % cache.page_size).to(DEV))


def _put(cache, name, row, from_, to, value, group=None):
    """Sets what a sequence's tokens hold (of one group of scales) to a value, or adds to it."""
    t = getattr(cache, name)
    t = t.transpose(1, 2) if cache.heads_first else t
    at = _tokens(cache, row, from_, to)
    if group is not None:
        t[at[0], at[1], :, group] = value
    else:
        t[at] = value


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("byte", [8, 121, 127, 128, 129, 200])
@pytest.mark.parametrize("tiles", [(1,), (0,), (2, 3), (4,)])
def test_prompts_over_tiles_of_zero_v(fmt, byte, tiles):
    """Tokens whose v is zero (scale byte 0, as cache_write stores zeros) keep their weight: whole
    tiles of 128, in any place, and a short last one."""
    D, lens = 64, [528]
    cache, table = _prompt(lens, D, fmt, byte)
    cache.v_scales.fill_(byte)
    for t in tiles:
        _put(cache, "v_codes", table[0], t * 128, min(528, t * 128 + 128), 0)
        _put(cache, "v_scales", table[0], t * 128, min(528, t * 128 + 128), 0)
    for causal in (True, False):
        _run(cache, table, lens, [NEW], HEADS * G, torch.bfloat16, byte, causal=causal, variants=("auto", "generic"))


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("D", [96, 128])
def test_prompts_over_tiles_of_written_zeros(fmt, D):
    """The same by cache_write, heads and sequences of their own: padding behind a prompt."""
    lens = [300, 401]
    cache, table = _filled(lens, 24, HEADS, D, fmt, D, first=True)
    slots = torch.tensor([table[b][t // 24] * 24 + t % 24 for b, n in enumerate(lens) for t in range(n // 2, n)],
                         device=DEV)
    kv = _q(len(slots), 2 * HEADS, D, torch.bfloat16, 4).contiguous()
    kv[:, HEADS:] = 0
    kv[:, HEADS + 1] = 1.0  # one head has values
    B.cache_write(cache, kv[:, :HEADS], kv[:, HEADS:], slots)
    for dtype in (torch.bfloat16, torch.float16):
        _run(cache, table, lens, [200, 260], HEADS * G, dtype, 3, variants=("auto", "generic"))


@pytest.mark.parametrize("byte", [121, 127, 129])
def test_prompts_over_a_tile_whose_pages_are_not_there(byte):
    lens = [528]
    cache, table = _prompt(lens, 128, "e2m1", byte)
    cache.v_scales.fill_(byte)
    for j in range(8, 16):
        table[0][j] = -1
    _run(cache, table, lens, [NEW], HEADS * G, torch.bfloat16, byte, status=-12)
