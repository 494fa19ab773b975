"""A workspace passed to the backward calls is taken for all of its bytes and no others:
a view whose elements do not lie one after another is refused before any launch (an
expanded one would be written past its storage, a strided one between its elements).
"""
from __future__ import annotations

import pytest
import torch

from memory_bound_normalization_fwd_gb300 import binding as B

CPU = -1  # what Tensor.get_device() says of the host


def test_the_bytes_of_a_contiguous_workspace():
    for t in (torch.empty(1000, dtype=torch.uint8), torch.empty(7, 11), torch.empty(64)[8:24]):
        assert B._given(t, CPU) == (t.data_ptr(), t.numel() * t.element_size())


@pytest.mark.parametrize("make", [lambda: torch.empty(1).expand(1 << 30), lambda: torch.empty(4, 1).expand(4, 1 << 20),
                                  lambda: torch.empty(4096)[::2], lambda: torch.empty(64, 64)[:, :32],
                                  lambda: torch.empty(64, 32).t()])
def test_views_with_holes_or_repeats_are_refused(make):
    with pytest.raises(ValueError, match="contiguous"):
        B._given(make(), CPU)


def test_a_workspace_on_another_device_is_refused():
    with pytest.raises(ValueError, match="must be on cuda:0"):
        B._given(torch.empty(16), 0)


@pytest.mark.gpu
def test_the_backward_calls_refuse_them():
    M, N, D = 40, 512, 64
    h, dy = torch.randn(2, M, N, device="cuda").bfloat16()
    w = torch.randn(N, device="cuda").bfloat16()
    s, _, a, b = B.block_fwd(h, dy, w, w)
    q, dq = torch.randn(2, 8, 2, D, device="cuda").bfloat16()
    steps, _ = B.rope_steps(D)
    out, _, rstd, _ = B.rope_fwd(q, None, steps, w_q=w[:D])
    one = torch.zeros(1, dtype=torch.uint8, device="cuda")
    big = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    for ws in (one.expand(1 << 26), big[::2], big.cpu()):
        with pytest.raises(ValueError):
            B.block_bwd(h, s, a, b, dy, None, w, w, workspace=ws)
        with pytest.raises(ValueError):
            B.rope_bwd(dq, None, steps, q=q, rstd_q=rstd, w_q=w[:D], workspace=ws)
    assert B.rmsnorm_check_device_status(0) == 0
    assert int(big.count_nonzero()) == 0 and int(one) == 0
    want = B.block_bwd(h, s, a, b, dy, None, w, w)
    for x, y in zip(B.block_bwd(h, s, a, b, dy, None, w, w, workspace=big), want):
        assert x is y is None or torch.equal(x, y)
