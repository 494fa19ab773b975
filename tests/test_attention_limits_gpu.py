"""Attention over the quantised cache at the edges of its number formats and its launches."""
from __future__ import annotations

import pytest
import torch

import ops_util as U
import serve_util as S
from memory_bound_normalization_fwd_gb300 import binding as B
from graph_nodes import captured_grids
from test_attention_gpu import DEV, _cu, _filled, _i32, _q, _run

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
@pytest.mark.parametrize("tiles", [(1,), (0,), (2, 3), (4,), (0, 1, 2, 3)])
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


def _apart(cache, q, row, from_, to, gap):
    """Puts tokens' scores `gap` (natural) above the others' (below, where it is negative): value 0 of
    k and q is theirs."""
    D = cache.head_dim
    q[..., 0] = 8.0
    code = cache.k_codes  # value 0 of everyone: 0
    if cache.fmt == "e2m1":
        code[..., 0] &= 0xf0
    else:
        code[..., 0] = 0
    # the code 1.0, times the group's scale: a power of two next to the gap
    _put(cache, "k_scales", row, from_, to, 0, 0)
    at = _tokens(cache, row, from_, to)
    one = (2 if gap > 0 else 10) if cache.fmt == "e2m1" else (0x38 if gap > 0 else 0xb8)
    t = code.transpose(1, 2) if cache.heads_first else code
    t[at[0], at[1], :, :cache.k_codes.shape[-1] // (D // 32)] = 0
    t[at[0], at[1], :, 0] = one
    e = int(torch.log2(torch.tensor(abs(gap) * D ** 0.5 / 8.0)).round())
    _put(cache, "k_scales", row, from_, to, 127 + e, 0)


def _check_prompt(cache, table, lens, counts, q, dtype, rounded=0.0):
    """As check_attention, plus `rounded`: what each value of v may be off by."""
    cu = _cu(counts)
    out, lse, mag, s, floor = S.attention(cache, q, table, lens, cu, cache.head_dim ** -0.5, True, 0)
    want = (out, lse, mag, s, floor + rounded)
    got, got_lse = B.cache_attention(cache, q, _i32(table), _i32(lens), cu_q=_i32(cu), lse=True)
    assert B.lib().rmsnorm_check_device_status(0) == 0
    S.check_attention(got, got_lse, want, dtype, (cache.fmt, cache.head_dim))


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gap", [11.0, 15.0])
def test_prompts_with_a_sink_token(fmt, D, gap):
    """A token that takes nearly all of the weight and whose v is zero: what the others' small
    probabilities add up to has the bits that the interface states."""
    lens = [400]
    cache, table = _prompt(lens, D, fmt, D)
    q = _q(NEW, HEADS * G, D, torch.bfloat16, 5).contiguous()
    _apart(cache, q, table[0], 0, 1, gap)
    _put(cache, "v_codes", table[0], 0, 1, 0)
    _put(cache, "v_scales", table[0], 0, 1, 0)
    _check_prompt(cache, table, lens, [NEW], q, torch.bfloat16)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("apart", [12, 20, 25, 33])
@pytest.mark.parametrize("where", [0, 1, 2])
def test_prompts_with_tiles_of_v_far_apart(fmt, apart, where):
    """A tile whose v lies powers of two above the others', and which hardly anything weighs."""
    lens = [400]
    cache, table = _prompt(lens, 64, fmt, apart)
    q = _q(NEW, HEADS * G, 64, torch.bfloat16, 5).contiguous()
    _apart(cache, q, table[0], where * 128, where * 128 + 128, -60.0)
    _put(cache, "v_scales", table[0], where * 128, where * 128 + 128, 127 + apart)
    _check_prompt(cache, table, lens, [NEW], q, torch.bfloat16)


@pytest.mark.parametrize("fmt,apart", [("e4m3", 21), ("e4m3", 25), ("e4m3", 33), ("e2m1", 35), ("e2m1", 40)])
def test_prompts_with_groups_of_v_far_apart_in_a_tile(fmt, apart):
    """In a tile of 128 tokens v is exact within 2^21 of the largest scale (8 bits; 4 bits: 2^35), and off
    by at most 2^-22 (2^-34) of it below."""
    lens = [300]
    cache, table = _prompt(lens, 64, fmt, apart)
    _put(cache, "v_scales", table[0], 37, 38, 127 + apart, 0)
    q = _q(NEW, HEADS * G, 64, torch.bfloat16, 5).contiguous()
    _apart(cache, q, table[0], 37, 38, -60.0)
    exact = 21 if fmt == "e4m3" else 35
    _check_prompt(cache, table, lens, [NEW], q, torch.bfloat16,
                  0.0 if apart <= exact else 2.0 ** (apart - (22 if fmt == "e4m3" else 34)))


@pytest.mark.parametrize("fmt,apart", [("e4m3", 10), ("e4m3", 21), ("e2m1", 21), ("e2m1", 35)])
def test_prompts_with_groups_of_k_far_apart_in_a_tile(fmt, apart):
    """k is exact there too: a group that lies above the others, where q is zero, takes nothing from them."""
    lens = [300]
    cache, table = _prompt(lens, 64, fmt, apart)
    _put(cache, "k_scales", table[0], 37, 38, 127 + apart, 1)
    cache.k_scales.clamp_(min=127, max=127 + apart)
    q = _q(NEW, HEADS * G, 64, torch.bfloat16, 5).contiguous()
    q[..., 32:] = 0
    q *= 0.1
    _check_prompt(cache, table, lens, [NEW], q, torch.bfloat16)


# ---- k of scale byte 0 ---------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_k_of_the_lowest_scale(fmt, dtype, D):
    """A scale byte 0 is 2^-127, beside q near the type's largest values: scores of ordinary size."""
    lens = [90, 33, 400]
    cache, table = _filled(lens, 16, 2, D, fmt, D)
    cache.k_codes &= 0x77
    cache.k_scales.fill_(0)
    g = torch.Generator().manual_seed(2)
    more = torch.randint(0, 2, cache.k_scales.shape, generator=g, dtype=torch.uint8).to(DEV)
    q = (_q(3, 8, D, torch.float32, 3).clamp(-3, 3) * 2.0 ** (118 if fmt == "e4m3" else 122)).to(U.DT[dtype])
    for add in (0, 1):
        cache.k_scales += add * more  # bytes 0 and 1
        _run(cache, table, lens, [1, 1, 1], 8, U.DT[dtype], q=q, scale=0.5)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("byte", [0, 3, 9])
def test_prompts_over_k_of_the_lowest_scales(fmt, byte):
    lens = [300]
    cache, table = _prompt(lens, 64, fmt, 3)
    cache.k_codes &= 0x77
    cache.k_scales.fill_(byte)
    size = 2.0 ** ((118 if fmt == "e4m3" else 122) - byte)
    q = (_q(NEW, HEADS * G, 64, torch.float32, 3).clamp(-3, 3) * size).to(torch.bfloat16)
    _run(cache, table, lens, [NEW], HEADS * G, torch.bfloat16, q=q, scale=0.5)


# ---- a cap on the CTAs ------------------------------------------------------------------

@pytest.mark.parametrize("most", [1, 3, 8, 40])
@pytest.mark.parametrize("D,heads", [(64, 2), (96, 5), (128, 8), (192, 8)])
def test_whole_slots_in_few_ctas(most, D, heads):
    """A short table: CTAs take slots whole, no more of them than the call allows (one a block of key heads
    at least)."""
    lens = [(29 * i) % 150 for i in range(60)]
    cache, table = _filled(lens, 16, heads, D, "e2m1", D)
    _run(cache, table, lens, [1] * 60, 4 * heads, torch.bfloat16, variants=("auto",))
    q, t, ln = _q(60, 4 * heads, D, torch.bfloat16, 0), _i32(table), _i32(lens)
    out, lse = B.cache_attention(cache, q, t, ln, lse=True, max_ctas=most)
    S.check_attention(out, lse, S.attention(cache, q, table, lens, list(range(61)), D ** -0.5, True, 0),
                      torch.bfloat16, (most, D))
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    res = torch.empty_like(q)
    grids = captured_grids(lambda: B.cache_attention(cache, q, t, ln, out=res, workspace=ws, max_ctas=most))
    assert len(grids) == 1 and grids[0] <= max(most, -(-heads // 8)), grids
    grids = captured_grids(lambda: B.cache_attention(cache, q, t, ln, out=res, workspace=ws))
    assert grids[0] > 40
