"""The block backward of short rows, where a team is a warp and there are more teams
than CTAs: the vector kernels take them at any number of rows, with the workspace that
rmsnorm_block_bwd_workspace_size() asks for, and are right there, as the others are.
"""
from __future__ import annotations

import pytest
import torch

import ops_util as U
from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(M, N, dtype, gate_rows, post=True, pre=True):
    g = torch.Generator(device=DEV).manual_seed(M + N + gate_rows)
    dt = U.DT[dtype]

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device=DEV).to(dt)

    h, r, dy, ds = rnd(M, N), rnd(M, N), rnd(M, N) if pre else None, rnd(M, N)
    w_post, w_pre = rnd(N) if post else None, rnd(N) if pre else None
    gate = rnd(-(-M // gate_rows), N) if gate_rows else None
    s, _, a, b = B.block_fwd(h, r, w_post, w_pre, gate, gate_rows or None)
    return h, s, a, b, dy, ds, w_post, w_pre, gate, gate_rows or None


def _check(args, out, where):
    h, s, a, b, dy, ds, w_post, w_pre, gate, gate_rows = args
    want, mag = U.block_bwd(h, s, a, b, dy, ds, w_post, w_pre, gate, gate_rows, 0.0, 1.0, 1.0)
    for name, got in zip(("dh", "dr", "dgate", "dw_post", "dw_pre"), out):
        if name not in want:
            assert got is None, name
            continue
        dt = torch.float32 if name.startswith("dw") else h.dtype
        U.check(got, want[name], mag[name], dt, f"{where} {name}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N", [(1217, 8), (1300, 64), (3700, 128), (8231, 64), (20000, 64), (20000, 256), (40001, 248)])
@pytest.mark.parametrize("gate_rows", [0, 1, 3, 100, 1000000])
def test_the_vector_kernels_take_short_rows(M, N, dtype, gate_rows):
    args = _case(M, N, dtype, gate_rows)
    need = B.rmsnorm_block_bwd_workspace_size(M, N, B._code(U.DT[dtype]))
    full = torch.full((need + 4096,), 255, dtype=torch.uint8, device=DEV)
    for variant in ("cta", "auto", "generic"):
        out = B.block_bwd(*args, workspace=full[:need], variant=variant)
        _check(args, out, f"{M}x{N} {dtype} gate_rows={gate_rows} {variant}")
        assert bool((full[need:] == 255).all())
        again = B.block_bwd(*args, variant=variant)
        assert all(p is q is None or torch.equal(p, q) for p, q in zip(out, again))


@pytest.mark.parametrize("post,pre", [(True, False), (False, True)])
@pytest.mark.parametrize("N", [64, 256])
@pytest.mark.parametrize("gate_rows", [0, 1, 100, 1000000])
def test_with_one_norm(N, post, pre, gate_rows):
    args = _case(9000, N, "bf16", gate_rows, post, pre)
    for kw in (dict(variant="cta"), dict(variant="cta", max_ctas=5), dict()):
        _check(args, B.block_bwd(*args, **kw), f"{N} {post} {pre} {gate_rows} {kw}")


def test_the_workspace_never_shrinks_with_more_rows():
    for N in (8, 256, 257, 1000, 16384):
        sizes = [B.rmsnorm_block_bwd_workspace_size(M, N, B.BF16) for M in (0, 1, 100, 1216, 1217, 5000, 10 ** 6)]
        assert sizes == sorted(sizes)
