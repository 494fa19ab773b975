"""Backward passes of rows and heads whose rstd is large (RMS of 1e-14 with eps 0, which
the calls take): the gradients are representable, and their factors of rstd^3 must not
pass fp32's range on the way. Parity by the bounds of ops_util, which are relative to
the terms' magnitudes.
"""
from __future__ import annotations

import pytest
import torch

import ops_util as U
from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _check(out, want, mag, dt, where):
    for name, got in zip(("dh", "dr", "dgate", "dw_post", "dw_pre"), out):
        if name not in want:
            assert got is None, name
            continue
        assert bool(torch.isfinite(got).all()), f"{where} {name}"
        U.check(got, want[name], mag[name], torch.float32 if name.startswith("dw") else dt, f"{where} {name}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 512, 777, 3001, 4096, 8192, 8200, 20001])
@pytest.mark.parametrize("post,gate_rows", [(False, 0), (False, 5), (True, 0), (True, 1)])
@pytest.mark.parametrize("size", [1e-14, 1e-16])
def test_block_rows(dtype, N, post, gate_rows, size):
    M, dt = 19, U.DT[dtype]
    g = torch.Generator().manual_seed(N)

    def rnd(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(dt).to(DEV)

    h, r, dy, ds = rnd(M, N, scale=size), rnd(M, N, scale=size), rnd(M, N), rnd(M, N)
    w_post, w_pre = rnd(N) if post else None, rnd(N)
    gate = rnd(-(-M // gate_rows), N) if gate_rows else None
    alpha = size if post else 1.0  # both rstd are large then
    for variant in ("auto", "generic"):
        s, _, a, b = B.block_fwd(h, r, w_post, w_pre, gate, gate_rows or None, eps=0.0, alpha=alpha, variant=variant)
        assert float(b.min()) > 0.1 / size
        want, mag = U.block_bwd(h, s, a, b, dy, ds, w_post, w_pre, gate, gate_rows, 0.0, alpha, 1.0)
        out = B.block_bwd(h, s, a, b, dy, ds, w_post, w_pre, gate, gate_rows or None, alpha=alpha, variant=variant)
        _check(out, want, mag, dt, f"{N} {dtype} {variant}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (80, 20), (256, 256), (66, 32), (7, 6)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size", [1e-14, 1e-16])
def test_rope_heads(dtype, D, R, interleaved, size):
    T, hq, hk, dt = 11, 5, 2, U.DT[dtype]
    g = torch.Generator().manual_seed(D + R)

    def rnd(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(dt).to(DEV)

    q, k, dq, dk = rnd(T, hq, D, scale=size), rnd(T, hk, D, scale=size), rnd(T, hq, D), rnd(T, hk, D)
    w_q, w_k = rnd(D), rnd(D)
    steps, _ = B.rope_steps(R)
    angle = U.rope_angles(steps, torch.arange(T, device=DEV))
    for variant in ("auto", "generic"):
        _, _, a, b = B.rope_fwd(q, k, steps, None, w_q, w_k, interleaved, eps=0.0, variant=variant)
        out = B.rope_bwd(dq, dk, steps, None, q, k, a, b, w_q, w_k, interleaved, variant=variant)
        for x, d, r, w, dx, dw in ((q, dq, a, w_q, out[0], out[2]), (k, dk, b, w_k, out[1], out[3])):
            want, wdw, m, mdw = U.rope_bwd(d, x, r, angle, w, R, interleaved, 0.0, 1.0)
            assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())
            U.check(dx, want, m, dt, f"{variant} dx")
            U.check(dw, wdw, mdw, torch.float32, f"{variant} dw")
