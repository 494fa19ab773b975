"""The block operator of a batch without rows: every gradient that exists is zero,
a gate's among them, whatever was in the memory before.
"""
from __future__ import annotations

import pytest
import torch

from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV, N = "cuda", 512


def _dirty():
    """Leaves a freed block of NaN of the gate's size for the next allocations."""
    for rows in (1, 3):
        torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    torch.full((N,), float("nan"), dtype=torch.float32, device=DEV)


@pytest.mark.parametrize("shape", [(0, N), (2, 0, N), (0, 5, N)])
@pytest.mark.parametrize("gate_shape,gate_rows", [((N,), None), ((N,), 7), ((1, N), None), ((3, N), 4), ((0, N), 1), ((3, N), None)])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_gradients_of_no_rows_are_zero(shape, gate_shape, gate_rows, post, pre):
    h = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(N, dtype=torch.bfloat16, device=DEV)
    w_post, w_pre = w if post else None, w if pre else None
    gate = torch.ones(gate_shape, dtype=torch.bfloat16, device=DEV)
    s, y, a, b = B.block_fwd(h, h.clone(), w_post, w_pre, gate, gate_rows)
    assert s.shape == shape
    _dirty()
    dh, dr, dgate, dw_post, dw_pre = B.block_bwd(h, s, a, b, h.clone() if pre else None, h.clone(), w_post, w_pre,
                                                 gate, gate_rows)
    assert dh.shape == dr.shape == shape and dgate.shape == gate_shape and dgate.dtype == gate.dtype
    for got, given in ((dgate, True), (dw_post, post), (dw_pre, pre)):
        assert (got is not None) == given
        if given:
            assert bool((got == 0).all())


@pytest.mark.parametrize("shape", [(0, N), (2, 0, N), (0, 5, N)])
def test_a_gate_per_element_of_no_rows(shape):
    # the gate in h's shape, without gate_rows and with them
    h = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(N, dtype=torch.bfloat16, device=DEV)
    for gate_rows in (None, 1, 5):
        gate = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        s, y, a, b = B.block_fwd(h, h.clone(), w, w, gate, gate_rows)
        assert s.shape == y.shape == shape and a.shape == b.shape == shape[:-1]
        dgate = B.block_bwd(h, s, a, b, h.clone(), h.clone(), w, w, gate, gate_rows)[2]
        assert dgate.shape == shape and dgate.dtype == gate.dtype
