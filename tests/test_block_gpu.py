"""GPU parity of the block operator (norm after a block, gate, scaled residual,
norm before the next block; forward and backward) with the plain 64-bit
implementation, by the bounds of ops_util.
"""
from __future__ import annotations

import itertools

import pytest
import torch

import ops_util as U
from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _make(M, N, dtype, seed, post=True, pre=True, gate_rows=0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    dt = U.DT[dtype]

    def rnd(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(dt).to(DEV)

    size = torch.exp(torch.randn(M, 1, generator=g))
    d = dict(h=(torch.randn(M, N, generator=g) * size).to(dt).to(DEV), r=rnd(M, N, scale=3.0),
             w_post=rnd(N) if post else None, w_pre=rnd(N) if pre else None, gate=None)
    if gate_rows:
        d["gate"] = rnd(-(-M // gate_rows), N)
    d["dy"] = rnd(M, N) if pre else None
    d["ds"] = rnd(M, N)
    return d


def _variants(**kw):
    return [dict(variant="auto", **kw), dict(variant="generic", **kw)]


def _check_fwd(d, out, gate_rows, eps, offset, alpha, beta, where):
    s, y, a, b, ms, my = U.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], gate_rows, eps,
                                     offset, alpha, beta)
    dt = d["h"].dtype
    gs, gy, ga, gb = out
    U.check(gs, s, ms, dt, f"{where} s")
    if y is None:
        assert gy is None and gb is None
    else:
        U.check(gy, y, my, dt, f"{where} y")
        U.check(gb, b, b, torch.float32, f"{where} rstd_pre")
    if a is None:
        assert ga is None
    else:
        U.check(ga, a, a, torch.float32, f"{where} rstd_post")


def _check_bwd(d, kept, out, gate_rows, offset, alpha, beta, where):
    s, a, b = kept
    want, mag = U.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], d["w_post"], d["w_pre"], d["gate"], gate_rows,
                            offset, alpha, beta)
    dt = d["h"].dtype
    for name, got in zip(("dh", "dr", "dgate", "dw_post", "dw_pre"), out):
        if name not in want:
            assert got is None, name
            continue
        U.check(got, want[name], mag[name], torch.float32 if name.startswith("dw") else dt, f"{where} {name}")


def _both(M, N, dtype, seed, post, pre, gate_rows, offset, alpha, beta, opts, ds=True):
    d = _make(M, N, dtype, seed, post, pre, gate_rows)
    if not ds:
        d["ds"] = None
    out = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], gate_rows, eps=1e-6, offset=offset,
                      alpha=alpha, beta=beta, **opts)
    where = f"{M}x{N} {dtype} post={post} pre={pre} gate_rows={gate_rows} {opts}"
    _check_fwd(d, out, gate_rows, 1e-6, offset, alpha, beta, where)
    s, _, a, b = out
    grads = B.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], d["w_post"], d["w_pre"], d["gate"], gate_rows,
                        offset=offset, alpha=alpha, beta=beta, **opts)
    _check_bwd(d, (s, a, b), grads, gate_rows, offset, alpha, beta, where)


SHAPES = [(1, 8), (1, 1), (5, 3), (37, 512), (130, 520), (3, 777), (70, 1000), (33, 4096), (9, 8192), (4, 8200),
          (5, 16384), (2, 20000), (300, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("variant", ["auto", "generic"])
def test_parity_over_shapes(M, N, dtype, variant):
    _both(M, N, dtype, M + N, True, True, 0, 0.0, 1.0, 1.0, dict(variant=variant))
    _both(M, N, dtype, M + N, True, True, max(1, M // 3), 1.0, 0.5, 0.9, dict(variant=variant))


@pytest.mark.parametrize("N", [512, 520, 999])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("gate_rows", [0, 1, 2, 5, 64, 1000])
def test_parity_over_parts(N, post, pre, gate_rows):
    for opts in _variants():
        _both(67, N, "bf16", gate_rows + N, post, pre, gate_rows, 1.0, -0.75, 1.25, opts)


@pytest.mark.parametrize("N", [264, 777, 8208 + 3])
@pytest.mark.parametrize("M", [1, 67])
def test_gate_rows_far_past_the_last_row(M, N):
    d = _make(M, N, "bf16", 3, gate_rows=1000)
    for opts in _variants():
        want = None
        for gate_rows in (1000, 1 << 40, 1 << 62, (1 << 63) - 1):
            s, y, a, b = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], gate_rows, **opts)
            got = (s, y, *B.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], d["w_post"], d["w_pre"], d["gate"],
                                      gate_rows, **opts))
            want = want or got
            assert all(torch.equal(g, w) for g, w in zip(got, want)), (gate_rows, opts)


def test_no_columns():
    x, w = torch.empty(2, 0, device=DEV), torch.empty(0, device=DEV)
    with pytest.raises(B.RMSNormError):
        B.block_fwd(x, x, w, w, gate=w)
    with pytest.raises(B.RMSNormError):
        B.block_fwd(x, x, w, w)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("max_ctas", [1, 3, 7, 50])
@pytest.mark.parametrize("gate_rows", [1, 2, 3, 16, 25, 100])
def test_gate_rows_that_cross_the_ranges_of_ctas(dtype, max_ctas, gate_rows):
    for opts in _variants(max_ctas=max_ctas):
        _both(100, 264, dtype, 5, True, True, gate_rows, 0.0, 1.0, 1.0, opts)


@pytest.mark.parametrize("dtype,N", [("bf16", 4104), ("bf16", 5000), ("bf16", 8192), ("fp16", 16384), ("bf16", 32768),
                                     ("fp32", 4100), ("fp32", 8192), ("fp32", 16384)])
@pytest.mark.parametrize("gate_rows", [0, 1, 5, 1000])
def test_wide_rows(dtype, N, gate_rows):
    for kw in (dict(), dict(max_ctas=3), dict(max_ctas=40)):
        _both(41, N, dtype, gate_rows + N, True, True, gate_rows, 1.0, 0.5, 1.5, kw)
    _both(300, N, dtype, gate_rows + N, True, False, gate_rows, 1.0, 0.5, 1.5, {})
    _both(7, N, dtype, gate_rows + N, False, True, gate_rows, 1.0, 0.5, 1.5, {})


def test_backward_without_the_residuals_gradient():
    for opts in _variants():
        _both(40, 512, "bf16", 3, True, True, 8, 0.0, 1.0, 1.0, opts, ds=False)
        _both(40, 512, "bf16", 3, False, True, 0, 0.0, 1.0, 1.0, opts, ds=False)


@pytest.mark.parametrize("M,N,dtype", [(16384, 512, "bf16"), (4099, 4096, "fp16"), (2048, 1000, "fp32")])
def test_many_rows(M, N, dtype):
    _both(M, N, dtype, 1, True, True, 1000, 0.0, 1.0, 1.0, dict(variant="auto"))


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 0), (8, 1), (40, 8)])
def test_strided_and_shifted_rows(pad, shift):
    # h, r, s, y (and the backward's arrays) as column slices of wider tensors:
    # the padding stays as it was.
    M, N, dt = 50, 512, torch.bfloat16
    d = _make(M, N, "bf16", 9, gate_rows=10)
    w = N + pad + shift

    def wide(t=None):
        full = torch.full((M, w), 7.0, dtype=dt, device=DEV)
        view = full[:, shift:shift + N]
        if t is not None:
            view.copy_(t)
        return full, view

    (_, h), (_, r), (_, ds), (_, dy) = (wide(d[k]) for k in ("h", "r", "ds", "dy"))
    (fs, s), (fy, y), (fh, dh), (fr, dr) = wide(), wide(), wide(), wide()
    fg = torch.full((5, 6 * N), 7.0, dtype=dt, device=DEV)
    gate = fg[:, 2 * N:3 * N]
    gate.copy_(d["gate"])
    out = B.block_fwd(h, r, d["w_post"], d["w_pre"], gate, 10, s=s, y=y)
    _check_fwd(d, out, 10, 1e-6, 0.0, 1.0, 1.0, "strided")
    res = B.block_bwd(h, s, out[2], out[3], dy, ds, d["w_post"], d["w_pre"], gate, 10, dh=dh, dr=dr)
    _check_bwd(d, (s, out[2], out[3]), res, 10, 0.0, 1.0, 1.0, "strided")
    for full in (fs, fy, fh, fr):
        rest = torch.cat([full[:, :shift], full[:, shift + N:]], 1)
        assert bool((rest == 7.0).all())


@pytest.mark.parametrize("N", [512, 1000, 777, 20001])
@pytest.mark.parametrize("s_on,y_on", [("r", "h"), ("h", "r"), ("r", None), (None, "h")])
def test_in_place_gives_the_same_bits(N, s_on, y_on):
    d = _make(33, N, "bf16", 4, gate_rows=11)
    want = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], 11)
    h, r = d["h"].clone(), d["r"].clone()
    on = {"h": h, "r": r, None: None}
    got = B.block_fwd(h, r, d["w_post"], d["w_pre"], d["gate"], 11, s=on[s_on], y=on[y_on])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("N", [512, 777, 8192, 20001])
@pytest.mark.parametrize("dh_on,dr_on", [("dy", "ds"), ("h", "s"), ("ds", "dy"), (None, "ds")])
def test_backward_in_place_gives_the_same_bits(N, dh_on, dr_on):
    d = _make(33, N, "fp16", 4, gate_rows=11)
    s, _, a, b = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], 11)
    args = (d["w_post"], d["w_pre"], d["gate"], 11)
    want = B.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], *args)
    c = {k: v.clone() for k, v in dict(h=d["h"], s=s, dy=d["dy"], ds=d["ds"]).items()}
    c[None] = None
    got = B.block_bwd(c["h"], c["s"], a, b, c["dy"], c["ds"], *args, dh=c[dh_on], dr=c[dr_on])
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_y_equals_the_plain_norm_of_the_unrounded_residual_in_fp32():
    # With fp32 tensors s is not rounded, so y is the framework's own forward of s.
    d = _make(40, 1000, "fp32", 2)
    s, y, _, b = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"])
    y2, b2 = B.fwd(s, d["w_pre"])
    assert torch.allclose(y, y2, rtol=1e-6, atol=1e-7) and torch.allclose(b, b2, rtol=1e-6)


def test_the_backward_of_the_plain_norm_is_the_frameworks():
    # Without w_post, gate and scales the backward of y is rmsnorm_bwd's.
    d = _make(60, 1000, "fp32", 6, post=False)
    s, y, _, b = B.block_fwd(d["h"], d["r"], None, d["w_pre"])
    dh, dr, _, _, dw = B.block_bwd(d["h"], s, None, b, d["dy"], None, None, d["w_pre"])
    dx, dwf = B.bwd(s, d["w_pre"], b, d["dy"])
    assert torch.equal(dh, dr)
    assert torch.allclose(dr, dx, rtol=1e-5, atol=1e-6) and torch.allclose(dw, dwf, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("variant", ["auto", "generic"])
def test_rows_of_zeros_infinities_and_nan_stay_by_themselves(variant):
    d = _make(12, 512, "bf16", 8)
    bad = {k: d[k].clone() for k in ("h", "r")}
    bad["h"][2] = 0
    bad["r"][2] = 0
    bad["h"][5, 7] = float("inf")
    bad["r"][8, 100] = float("nan")
    good = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], variant=variant)
    got = B.block_fwd(bad["h"], bad["r"], d["w_post"], d["w_pre"], variant=variant)
    keep = [i for i in range(12) if i not in (2, 5, 8)]
    for a, b in zip(got, good):
        assert torch.equal(a[keep], b[keep])
    assert bool((got[0][2] == 0).all()) and bool((got[1][2] == 0).all())
    assert torch.allclose(got[2][2], torch.tensor(1e3, device=DEV), rtol=1e-6)
    assert bool(got[1][8].isnan().all())


def test_no_rows():
    for shape in ((0, 64), (2, 0, 64)):
        h = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
        s, y, a, b = B.block_fwd(h, h.clone(), w, w)
        assert s.shape == y.shape == shape and a.shape == shape[:-1]
        dh, dr, _, dwa, dwb = B.block_bwd(h, s, a, b, h.clone(), h.clone(), w, w)
        assert dh.shape == shape and bool((dwa == 0).all()) and bool((dwb == 0).all())


def test_batched_shapes_and_gates():
    Bt, S, N = 3, 17, 512
    d = _make(Bt * S, N, "bf16", 12, gate_rows=S)
    h, r, ds, dy = (d[k].view(Bt, S, N) for k in ("h", "r", "ds", "dy"))
    want = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], S)
    for gate in (d["gate"], d["gate"].view(Bt, 1, N)):
        got = B.block_fwd(h, r, d["w_post"], d["w_pre"], gate)
        for a, b in zip(got, want):
            assert torch.equal(a.reshape(b.shape), b)
        res = B.block_bwd(h, got[0], got[2], got[3], dy, ds, d["w_post"], d["w_pre"], gate)
        _check_bwd(d, want[0:1] + want[2:], [t.reshape(-1, N) if t.dim() > 1 else t for t in res], S, 0.0, 1.0,
                   1.0, "batched")
        assert res[2].shape == gate.shape
    one = B.block_fwd(h, r, d["w_post"], d["w_pre"], d["gate"][0])     # a gate per channel
    two = B.block_fwd(h, r, d["w_post"], d["w_pre"], d["gate"][0].expand(Bt, S, N).contiguous())
    for a, b in zip(one, two):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        B.block_fwd(h, r, d["w_post"], d["w_pre"], d["gate"][:2])


@pytest.mark.parametrize("N", [512, 4096, 8192, 777])
def test_results_do_not_depend_on_the_run(N):
    d = _make(700, N, "bf16", 21, gate_rows=90)
    runs = []
    for _ in range(3):
        s, y, a, b = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], 90)
        runs.append((s, y, a, b) + B.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], d["w_post"], d["w_pre"],
                                               d["gate"], 90))
    for other in runs[1:]:
        for x, y in zip(runs[0], other):
            assert torch.equal(x, y)


@pytest.mark.parametrize("pdl", [True, False])
@pytest.mark.parametrize("N", [512, 4096, 5000])
def test_a_chain_of_layers_keeps_stream_order(N, pdl):
    # Each layer's r is the layer's before s, its h that layer's y; then all the
    # backward calls in turn through one workspace. The same calls with the
    # device synchronised between them give the same bits.
    d = _make(3000, N, "bf16", 31)
    ws = torch.empty(B.rmsnorm_block_bwd_workspace_size(3000, N, B.BF16), dtype=torch.uint8, device=DEV)

    def layers(sync):
        outs, h, r = [], d["h"], d["r"]
        for _ in range(4):
            o = B.block_fwd(h, r, d["w_post"], d["w_pre"], pdl=pdl)
            if sync:
                torch.cuda.synchronize()
            outs.append((h, o))
            r, h = o[0], o[1]
        dh, dr, res = d["dy"], d["ds"], []
        for h, (s, _, a, b) in reversed(outs):
            dh, dr, _, dwa, dwb = B.block_bwd(h, s, a, b, dh, dr, d["w_post"], d["w_pre"], workspace=ws, pdl=pdl)
            if sync:
                torch.cuda.synchronize()
            res += [dh, dr, dwa, dwb]
        torch.cuda.synchronize()
        return [t for _, o in outs for t in o] + res

    for a, b in zip(layers(False), layers(True)):
        assert torch.equal(a, b)


def test_captured_and_replayed_on_new_inputs():
    d = _make(200, 1000, "bf16", 41, gate_rows=50)
    e = _make(200, 1000, "bf16", 42, gate_rows=50)
    stream = torch.cuda.Stream()
    ws = torch.empty(B.rmsnorm_block_bwd_workspace_size(200, 1000, B.BF16), dtype=torch.uint8, device=DEV)

    def step(x):
        s, y, a, b = B.block_fwd(x["h"], x["r"], x["w_post"], x["w_pre"], x["gate"], 50)
        return (s, y, a, b) + B.block_bwd(x["h"], s, a, b, x["dy"], x["ds"], x["w_post"], x["w_pre"], x["gate"],
                                          50, workspace=ws)

    static = {k: v.clone() for k, v in d.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = step(static)
    for x in (e, d):
        for k, v in x.items():
            static[k].copy_(v)
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step(x)):
            assert torch.equal(a, b)


def test_on_another_stream_than_the_current_one():
    d = _make(500, 4096, "bf16", 51)
    want = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], stream=side)
    s, _, a, b = got
    res = B.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], d["w_post"], d["w_pre"], stream=side)
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    _check_bwd(d, (s, a, b), res, 0, 0.0, 1.0, 1.0, "side stream")


@pytest.mark.parametrize("M,N", [(1, 64), (100, 1000), (3000, 512)])
def test_the_workspace_is_as_large_as_it_says(M, N):
    d = _make(M, N, "bf16", 61, gate_rows=7)
    s, _, a, b = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], d["gate"], 7)
    need = B.rmsnorm_block_bwd_workspace_size(M, N, B.BF16)
    full = torch.full((need + 4096,), 255, dtype=torch.uint8, device=DEV)
    for opts in _variants():
        res = B.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], d["w_post"], d["w_pre"], d["gate"], 7,
                          workspace=full[:need], **opts)
        _check_bwd(d, (s, a, b), res, 7, 0.0, 1.0, 1.0, "workspace")
        assert bool((full[need:] == 255).all())
    with pytest.raises(B.RMSNormError) as e:
        B.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], d["w_post"], d["w_pre"], d["gate"], 7,
                    workspace=full[:need - 16])
    assert e.value.status == -11
    with pytest.raises(B.RMSNormError) as e:
        B.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], d["w_post"], d["w_pre"], d["gate"], 7, workspace=s)
    assert e.value.status in (-5, -11)


def test_the_vector_kernels_can_be_asked_for():
    d = _make(20, 512, "bf16", 81)
    for N in (512, 8192):
        d = _make(20, N, "bf16", 81)
        want = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"])
        got = B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], variant="cta")
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    d = _make(20, 511, "bf16", 81)
    with pytest.raises(B.RMSNormError) as e:
        B.block_fwd(d["h"], d["r"], d["w_post"], d["w_pre"], variant="cta")
    assert e.value.status == -8


@pytest.mark.parametrize("M,N,dtype", [(500, 512, "bf16"), (500, 4096, "bf16"), (500, 8192, "bf16"),
                                       (20000, 512, "bf16"), (8192, 4096, "bf16"), (4096, 8192, "bf16"),
                                       (4096, 8192, "fp32")])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(M, N, dtype):
    # With a limit of a few cycles a wait for a staged row that has not landed ends
    # at once: the kernel gives up, in bounds, and says so. Where every row happens to
    # land before it is waited for, the call is right instead. Which of the two is a
    # matter of timing; that it is one of them is not.
    d = _make(M, N, dtype, 91, gate_rows=100)
    args = (d["w_post"], d["w_pre"], d["gate"], 100)
    s, y, a, b = B.block_fwd(d["h"], d["r"], *args)
    want = B.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], *args)
    assert B.rmsnorm_check_device_status(0) == 0

    def short(call, right):
        got = call()
        status = B.rmsnorm_check_device_status(0)
        assert status in (0, -7)
        if status == 0:
            for p, q in zip(got, right):
                assert torch.equal(p, q)
        assert B.rmsnorm_check_device_status(0) == 0

    short(lambda: B.block_fwd(d["h"], d["r"], *args, wait_limit_ns=1), (s, y, a, b))
    short(lambda: B.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], *args, wait_limit_ns=1), want)
    for p, q in zip((s, y, a, b), B.block_fwd(d["h"], d["r"], *args)):
        assert torch.equal(p, q)
    for p, q in zip(want, B.block_bwd(d["h"], s, a, b, d["dy"], d["ds"], *args)):
        assert torch.equal(p, q)
    assert B.rmsnorm_check_device_status(0) == 0


@pytest.mark.slow
@pytest.mark.parametrize("M,N", [(530000, 4096), (2800000, 777)])
def test_offsets_past_32_bits(M, N):
    # Tensors of more than 2^31 elements made of 1000 rows again and again: every
    # thousand rows of the outputs are alike, and the sums over rows are theirs.
    base = _make(1000, N, "bf16", 101)
    want = B.block_fwd(base["h"], base["r"], base["w_post"], base["w_pre"])

    def tall(t):
        return t.expand(M // 1000, *t.shape).reshape(M, N)

    h, r = tall(base["h"]), tall(base["r"])
    s, y, a, b = B.block_fwd(h, r, base["w_post"], base["w_pre"], s=r, y=None)
    for got, w in ((s, want[0]), (y, want[1]), (a, want[2]), (b, want[3])):
        got = got.view(M // 1000, *w.shape)
        assert torch.equal(got[0], w) and torch.equal(got[-1], w) and torch.equal(got[M // 2000], w)
    dy, ds = tall(base["dy"]), tall(base["ds"])
    one = B.block_bwd(base["h"], want[0], want[2], want[3], base["dy"], base["ds"], base["w_post"], base["w_pre"])
    dh, dr, _, dwa, dwb = B.block_bwd(h, s, a, b, dy, ds, base["w_post"], base["w_pre"], dh=dy, dr=ds)
    for got, w in ((dh, one[0]), (dr, one[1])):
        got = got.view(M // 1000, *w.shape)
        assert torch.equal(got[0], w) and torch.equal(got[-1], w) and torch.equal(got[M // 2000], w)
    # The sums: the thousand rows' times M / 1000, each within TAU of its magnitudes
    # (the magnitudes of the sum over rows are M / 1000 times the thousand rows').
    _, mag = U.block_bwd(base["h"], want[0], want[2], want[3], base["dy"], base["ds"], base["w_post"],
                         base["w_pre"], None, 0, 0.0, 1.0, 1.0)
    for got, w, name in ((dwa, one[3], "dw_post"), (dwb, one[4], "dw_pre")):
        err = (got.double() / (M // 1000) - w.double()).abs()
        # a chain of M / 152 additions in fp32 per CTA: at most that many half steps of the sum
        assert bool((err <= (2 * U.TAU + M / 152 * 2.0 ** -24) * mag[name]).all())


def test_refused_tensors():
    d = _make(4, 64, "bf16", 71)
    ok = dict(h=d["h"], r=d["r"], w_post=d["w_post"], w_pre=d["w_pre"])
    for change in (dict(r=d["r"].float()), dict(w_pre=d["w_pre"].half()), dict(r=d["r"][:3]),
                   dict(w_post=d["w_post"][:32]), dict(h=d["h"].cpu()), dict(w_post=d["w_post"].cpu()),
                   dict(gate=d["h"][:, :32]), dict(gate_rows=2), dict(y=d["h"], w_pre=None),
                   dict(h=d["h"].t().contiguous().t())):
        with pytest.raises(ValueError):
            B.block_fwd(**{**ok, **change})
    with pytest.raises(TypeError):
        B.block_fwd(d["h"].double(), d["r"].double(), d["w_post"].double())
    with pytest.raises(B.RMSNormError):
        B.block_fwd(d["h"], d["r"])
