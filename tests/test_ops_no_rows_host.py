"""A gate without rows has no address: the block entry points take it in a batch without
rows, and refuse rows per gate row without a gate where there are rows.
"""
from __future__ import annotations

import pytest

from memory_bound_normalization_fwd_gb300 import binding as B
from memory_bound_normalization_fwd_gb300 import build as BUILD

W = 0x100000000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    BUILD.build()
    return B.lib()


@pytest.mark.parametrize("M,gate_rows,code", [(0, 0, 0), (0, 1, 0), (0, 100, 0), (0, -1, -2), (1, 1, -2), (4, 100, -2)])
def test_gate_rows_without_a_gate(M, gate_rows, code):
    args = B.BlockArgs(struct_size=160, dtype=0, M=M, N=8, gate_rows=gate_rows, w_post=W, w_pre=W, ldh=8, ldr=8,
                       ldg=8, lds=8, ldy=8, alpha=1.0, beta=1.0)
    assert B.rmsnorm_block_fwd(args, None, 0) == code
