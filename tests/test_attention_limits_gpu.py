"""Attention over the quantised cache at the edges of its number formats and its launches."""
from __future__ import annotations

import pytest
import torch

import serve_util as S
from memory_bound_normalization_fwd_gb300 import binding as B
from test_attention_gpu import _filled, _i32, _q

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
