"""Block kernels whose bounded waits run out: with limits from a few cycles to a few
microseconds some rows land in time and some do not, and whichever it is, the call
ends, says so, writes nothing outside its outputs, and the next call is right.
Each form has one reduction per row (one norm, the backward) or two (both norms), the
backward of long rows an exchange between CTAs besides.
"""
from __future__ import annotations

import pytest
import torch

import ops_util as U
from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMITS = (1, 1, 50, 400, 1000, 2500, 1)
CASES = [(30000, 512, "bf16", 0), (30000, 1000, "fp16", 1), (6000, 4096, "bf16", 100), (6000, 8192, "bf16", 0),
         (3000, 16384, "bf16", 7), (6000, 2048, "fp32", 0)]


def _calls(M, N, dtype, gate_rows, post, pre):
    """The forward and the backward of a case, as functions of the options."""
    g = torch.Generator(device=DEV).manual_seed(M + N)
    dt = U.DT[dtype]

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device=DEV).to(dt)

    h, r, ds = rnd(M, N), rnd(M, N), rnd(M, N)
    dy = rnd(M, N) if pre else None
    w_post, w_pre = rnd(N) if post else None, rnd(N) if pre else None
    gate = rnd(-(-M // gate_rows), N) if gate_rows else None
    args = (w_post, w_pre, gate, gate_rows or None)
    s, y, a, b = B.block_fwd(h, r, *args)
    return (lambda **kw: B.block_fwd(h, r, *args, **kw),
            lambda **kw: B.block_bwd(h, s, a, b, dy, ds, *args, **kw))


def _reported(call):
    """How many of the limits were reported; the others' results are right."""
    want = call()
    assert B.rmsnorm_check_device_status(0) == 0
    out = 0
    for limit in LIMITS:
        got = call(wait_limit_ns=limit)
        status = B.rmsnorm_check_device_status(0)
        assert status in (0, -7)
        out += status == -7
        if status == 0:
            assert all(p is None if q is None else torch.equal(p, q) for p, q in zip(got, want))
    assert all(p is None if q is None else torch.equal(p, q) for p, q in zip(call(), want))
    assert B.rmsnorm_check_device_status(0) == 0
    return out


def test_waits_that_run_out_end_the_call():
    out = [0, 0]
    for post, pre in ((True, False), (False, True), (True, True)):
        for case in CASES:
            for i, call in enumerate(_calls(*case, post, pre)):
                out[i] += _reported(call)
    assert min(out) > 0, f"no wait of the forward or the backward ran out: {out}"
