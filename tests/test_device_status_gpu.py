"""rmsnorm_check_device_status reports what happened since the last check, each kind once:
where a wait ran out and an index was out of range, the wait first, the index by the
check after it.
"""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_an_index_is_not_lost_behind_a_wait():
    cache = B.Cache(4, 16, 2, 64)
    k = torch.randn(3, 2, 64, device=DEV).bfloat16()
    bad = torch.tensor([1, 64, 2], device=DEV)  # the cache has 64 slots
    h, r = torch.randn(2, 6000, 2048, device=DEV)
    w = torch.ones(2048, device=DEV)
    assert B.rmsnorm_check_device_status(0) == 0
    both = 0
    for _ in range(50):
        B.block_fwd(h, r, w, w, wait_limit_ns=1)
        B.cache_write(cache, k, None, bad)
        status = B.rmsnorm_check_device_status(0)
        if status == -7:  # whether a wait of a few cycles runs out is a matter of timing
            both += 1
            status = B.rmsnorm_check_device_status(0)
        assert status == -12
        assert B.rmsnorm_check_device_status(0) == 0
    assert both > 0


FIRST = """
import torch
from memory_bound_normalization_fwd_gb300 import binding as B
assert B.rmsnorm_check_device_status(0) == 0
cache = B.Cache(4, 16, 2, 64)
k = torch.randn(1, 2, 64, device="cuda").bfloat16()
slot = torch.tensor([3], device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    B.cache_write(cache, k, None, slot)
assert B.rmsnorm_check_device_status(0) == 0
slot.fill_(64)
graph.replay()
assert B.rmsnorm_check_device_status(0) == -12
graph.replay()
slot.fill_(2)
graph.replay()
assert B.rmsnorm_check_device_status(0) == -12
assert B.rmsnorm_check_device_status(0) == 0
"""


def test_an_index_met_by_the_only_launch_of_a_process_a_replayed_graph():
    p = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, cwd=ROOT)
    assert p.returncode == 0, p.stderr
