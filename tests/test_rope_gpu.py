"""GPU parity of rotary positions with head norms (forward and backward) with
the plain 64-bit implementation, by the bounds of ops_util. Beside those, the
angle itself is off by its fp32 value (2^-25 half turns) and sincospi's own
rounding: within 3e-7 of the pair's magnitude, inside TAU.
"""
from __future__ import annotations

import pytest
import torch

import ops_util as U
from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _make(shape, hq, hk, D, R, dtype, seed, norm=True, far=5000):
    g = torch.Generator().manual_seed(seed)
    dt = U.DT[dtype]

    def rnd(*s):
        return torch.randn(*s, generator=g).to(dt).to(DEV)

    d = dict(q=rnd(*shape, hq, D), k=rnd(*shape, hk, D) if hk else None, dq=rnd(*shape, hq, D),
             dk=rnd(*shape, hk, D) if hk else None, w_q=rnd(D) if norm else None,
             w_k=rnd(D) if norm and hk else None)
    d["positions"] = torch.randint(0, far, shape, generator=g).to(DEV)
    d["steps"], _ = B.rope_steps(R, 10000.0, device=DEV)
    return d


def _angle(d, shape):
    pos = d["positions"]
    if pos is None:
        pos = torch.arange(shape[-1], device=DEV)
    return U.rope_angles(d["steps"], pos)


def _check_fwd(d, out, R, inter, offset, mag, eps=1e-6, where=""):
    dt, angle = d["q"].dtype, _angle(d, d["q"].shape[:-2])
    for x, w, got, rstd in ((d["q"], d["w_q"], out[0], out[2]), (d["k"], d["w_k"], out[1], out[3])):
        if x is None:
            assert got is None
            continue
        want, r, m = U.rope_fwd(x, angle, w, R, inter, eps, offset, mag)
        U.check(got, want, m, dt, f"{where} out")
        if w is None:
            assert rstd is None
        else:
            U.check(rstd, r, r, torch.float32, f"{where} rstd")


def _check_bwd(d, rstds, out, R, inter, offset, mag, where=""):
    dt, angle = d["q"].dtype, _angle(d, d["q"].shape[:-2])
    for x, w, g, rstd, got, dw in ((d["q"], d["w_q"], d["dq"], rstds[0], out[0], out[2]),
                                   (d["k"], d["w_k"], d["dk"], rstds[1], out[1], out[3])):
        if x is None:
            assert got is None and dw is None
            continue
        want, wdw, m, mdw = U.rope_bwd(g, x, rstd, angle, w, R, inter, offset, mag)
        U.check(got, want, m, dt, f"{where} dx")
        if w is None:
            assert dw is None
        else:
            U.check(dw, wdw, mdw, torch.float32, f"{where} dw")


def _both(d, R, inter, offset=0.0, mag=1.0, where="", **opts):
    out = B.rope_fwd(d["q"], d["k"], d["steps"], d["positions"], d["w_q"], d["w_k"], inter, offset=offset,
                     magnitude=mag, **opts)
    _check_fwd(d, out, R, inter, offset, mag, where=where)
    res = B.rope_bwd(d["dq"], d["dk"], d["steps"], d["positions"], d["q"], d["k"], out[2], out[3], d["w_q"],
                     d["w_k"], inter, offset, mag, **opts)
    _check_bwd(d, out[2:], res, R, inter, offset, mag, where=where)


HEADS = [(64, 64), (128, 128), (128, 64), (128, 32), (80, 80), (80, 20), (96, 48), (112, 112), (192, 64),
         (256, 256), (512, 512), (576, 64), (8, 2), (16, 16), (7, 6), (2, 2), (66, 32), (1000, 10)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,R", HEADS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [True, False])
def test_parity_over_heads(D, R, dtype, inter, norm):
    d = _make((37,), 5, 2, D, R, dtype, D + R, norm)
    for variant in ("auto", "generic"):
        _both(d, R, inter, 1.0, 1.25, f"D={D} R={R} {dtype} {inter} {norm} {variant}", variant=variant)


@pytest.mark.parametrize("T,hq,hk", [(1, 1, 0), (1, 32, 8), (2, 7, 1), (3, 64, 8), (64, 32, 8), (1021, 4, 4),
                                     (5000, 3, 1), (700, 41, 3)])
@pytest.mark.parametrize("norm", [True, False])
def test_parity_over_tokens(T, hq, hk, norm):
    d = _make((T,), hq, hk, 128, 128, "bf16", T, norm)
    for opts in (dict(), dict(max_ctas=2), dict(variant="generic")):
        _both(d, 128, False, where=f"T={T} {hq}/{hk} {opts}", **opts)


@pytest.mark.parametrize("which", ["q", "k"])
def test_norm_of_one_tensor_alone(which):
    d = _make((50,), 4, 2, 128, 128, "bf16", 3)
    d["w_" + which] = None
    for variant in ("auto", "generic"):
        _both(d, 128, False, where=which, variant=variant)


@pytest.mark.parametrize("position", [0, 1, 4097, 131071, (1 << 20) - 1, (1 << 31) + 7, (1 << 40) + 12345, -1,
                                      -100000, (1 << 63) - 1, -(1 << 63)])
def test_angles_of_any_position(position):
    d = _make((9,), 3, 1, 128, 128, "fp32", 11, norm=False)
    d["positions"] = torch.full((9,), position, dtype=torch.int64, device=DEV)
    _both(d, 128, False, where=f"position {position}")


def test_angles_agree_with_the_frequencies_they_stand_for():
    # Against cos and sin of position * frequency in 64 bits: the step's own
    # rounding (2^-65 turns) times the position is far below fp32's.
    d = _make((64,), 2, 1, 128, 128, "fp32", 12, norm=False, far=1 << 20)
    inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device=DEV) / 64)
    angle = d["positions"].double()[:, None] * inv
    out = B.rope_fwd(d["q"], d["k"], d["steps"], d["positions"])
    want, _, m = U.rope_fwd(d["q"], angle, None, 128, False, 0.0, 0.0, 1.0)
    U.check(out[0], want, m, torch.float32, "frequencies")


def test_default_positions_and_batches():
    shape = (3, 21)
    d = _make(shape, 4, 2, 64, 64, "bf16", 13)
    base = {k: v for k, v in d.items()}
    rows = torch.arange(100, 121, device=DEV)
    for pos, full in ((None, torch.arange(21, device=DEV).expand(3, 21)), (rows, rows.expand(3, 21)),
                      (d["positions"], d["positions"])):
        d["positions"] = full.contiguous()
        out = B.rope_fwd(d["q"], d["k"], d["steps"], pos, d["w_q"], d["w_k"])
        _check_fwd(d, out, 64, False, 0.0, 1.0, where="batched")
        res = B.rope_bwd(d["dq"], d["dk"], d["steps"], pos, d["q"], d["k"], out[2], out[3], d["w_q"], d["w_k"])
        _check_bwd(d, out[2:], res, 64, False, 0.0, 1.0, where="batched")
    wide = torch.randint(0, 1000, (3, 40), device=DEV)      # positions as a slice of a longer row
    d["positions"] = wide[:, 5:26]
    _both(d, 64, False, where="sliced positions")
    assert base["q"] is d["q"]


@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (128, 64, True), (80, 80, False), (72, 20, False)])
@pytest.mark.parametrize("in_place", [False, True])
def test_slices_of_a_projection(D, R, inter, in_place):
    T, hq, hk = 45, 6, 2
    d = _make((T,), hq, hk, D, R, "bf16", 14)
    qkv = torch.full((T, hq + 2 * hk, D), 3.0, dtype=torch.bfloat16, device=DEV)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    q.copy_(d["q"])
    k.copy_(d["k"])
    want = B.rope_fwd(d["q"], d["k"], d["steps"], d["positions"], d["w_q"], d["w_k"], inter)
    kept = qkv.clone()
    got = B.rope_fwd(q, k, d["steps"], d["positions"], d["w_q"], d["w_k"], inter,
                     q_out=q if in_place else None, k_out=k if in_place else None)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(qkv[:, hq + hk:], kept[:, hq + hk:])
    if not in_place:
        assert torch.equal(qkv, kept)
    # the backward writes its gradients into slices, and takes expanded ones
    g = torch.full_like(qkv, 5.0)
    dq, dk = g[:, :hq], g[:, hq:hq + hk]
    dq.copy_(d["dq"])
    dk.copy_(d["dk"])
    res = B.rope_bwd(dq, dk, d["steps"], d["positions"], d["q"], d["k"], want[2], want[3], d["w_q"], d["w_k"],
                     inter, dq=dq if in_place else None, dk=dk if in_place else None)
    _check_bwd(d, want[2:], res, R, inter, 0.0, 1.0, where="slices")
    assert bool((g[:, hq + hk:] == 5.0).all())
    e = dict(d)
    e["dq"] = d["dq"][:1, :1].expand(T, hq, D)
    e["dk"] = d["dk"][:1].expand(T, hk, D)
    res = B.rope_bwd(e["dq"], e["dk"], d["steps"], d["positions"], d["q"], d["k"], want[2], want[3], d["w_q"],
                     d["w_k"], inter)
    _check_bwd(e, want[2:], res, R, inter, 0.0, 1.0, where="expanded")


def test_heads_before_tokens_and_shifted_addresses():
    Bt, S, hq, hk, D = 2, 19, 4, 2, 128
    d = _make((Bt, S), hq, hk, D, D, "bf16", 15)
    want = B.rope_fwd(d["q"], d["k"], d["steps"], d["positions"], d["w_q"], d["w_k"])
    for shift in (0, 1):
        def heads_first(t):
            H = t.shape[2]
            m = torch.empty(Bt * H * S * D + 8, dtype=t.dtype, device=DEV)[shift:shift + Bt * H * S * D]
            v = m.view(Bt, H, S, D).transpose(1, 2)
            v.copy_(t)
            return v
        q, k = heads_first(d["q"]), heads_first(d["k"])
        oq, ok = heads_first(torch.zeros_like(d["q"])), heads_first(torch.zeros_like(d["k"]))
        got = B.rope_fwd(q, k, d["steps"], d["positions"], d["w_q"], d["w_k"], q_out=oq, k_out=ok)
        _check_fwd(d, got, D, False, 0.0, 1.0, where=f"heads first {shift}")
        for a, b in zip(got, want):
            # the element-wise kernel sums a head in another order
            assert torch.equal(a, b) if shift == 0 else torch.allclose(a.float(), b.float(), rtol=2e-2, atol=1e-2)
        res = B.rope_bwd(heads_first(d["dq"]), heads_first(d["dk"]), d["steps"], d["positions"], q, k, got[2],
                         got[3], d["w_q"], d["w_k"])
        _check_bwd(d, got[2:], res, D, False, 0.0, 1.0, where=f"heads first {shift}")


@pytest.mark.parametrize("D,R,inter", [(128, 64, False), (80, 20, True), (80, 20, False), (64, 6, True), (33, 2, True)])
def test_values_behind_the_rotated_part_stay_whatever_they_are(D, R, inter):
    d = _make((11,), 3, 1, D, R, "bf16", 22, norm=False)
    d["q"][..., R::2] = float("inf")
    d["q"][..., R + 1::4] = float("nan")
    for variant in ("auto", "generic"):
        out = B.rope_fwd(d["q"], d["k"], d["steps"], d["positions"], interleaved=inter, variant=variant)
        assert torch.equal(torch.nan_to_num(out[0][..., R:], nan=7.0), torch.nan_to_num(d["q"][..., R:], nan=7.0))
        assert bool(torch.isfinite(out[0][..., :R].float()).all())
        back = B.rope_bwd(d["q"], d["k"], d["steps"], d["positions"], interleaved=inter, variant=variant)
        assert torch.equal(torch.nan_to_num(back[0][..., R:], nan=7.0), torch.nan_to_num(d["q"][..., R:], nan=7.0))


def test_turning_back_undoes_the_turn():
    d = _make((33,), 4, 4, 64, 64, "fp32", 16, norm=False)
    out = B.rope_fwd(d["q"], d["k"], d["steps"], d["positions"])
    q, k, _, _ = B.rope_bwd(out[0], out[1], d["steps"], d["positions"])
    assert torch.allclose(q, d["q"], rtol=1e-5, atol=1e-5) and torch.allclose(k, d["k"], rtol=1e-5, atol=1e-5)


def test_zero_rows_and_no_tokens():
    d = _make((4,), 2, 1, 64, 64, "bf16", 17)
    d["q"][1] = 0
    out = B.rope_fwd(d["q"], d["k"], d["steps"], d["positions"], d["w_q"], d["w_k"])
    assert bool((out[0][1] == 0).all()) and bool(torch.isfinite(out[0].float()).all())
    e = {k: (v[:0] if k in ("q", "k", "dq", "dk", "positions") else v) for k, v in d.items()}
    out = B.rope_fwd(e["q"], e["k"], e["steps"], e["positions"], e["w_q"], e["w_k"])
    assert out[0].shape == (0, 2, 64)
    res = B.rope_bwd(e["dq"], e["dk"], e["steps"], e["positions"], e["q"], e["k"], out[2], out[3], e["w_q"], e["w_k"])
    assert res[0].shape == (0, 2, 64) and bool((res[2] == 0).all()) and bool((res[3] == 0).all())


def test_results_do_not_depend_on_the_run_and_streams():
    d = _make((3000,), 8, 2, 128, 128, "bf16", 18)
    runs, side = [], torch.cuda.Stream()
    for i in range(3):
        torch.cuda.synchronize()
        s = side if i == 2 else None
        out = B.rope_fwd(d["q"], d["k"], d["steps"], d["positions"], d["w_q"], d["w_k"], stream=s)
        runs.append(out + B.rope_bwd(d["dq"], d["dk"], d["steps"], d["positions"], d["q"], d["k"], out[2], out[3],
                                     d["w_q"], d["w_k"], stream=s))
        torch.cuda.synchronize()
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


def test_captured_decoding_steps_move_on_with_the_positions():
    d = _make((8,), 4, 2, 128, 128, "bf16", 19)
    pos = d["positions"].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = B.rope_fwd(d["q"], d["k"], d["steps"], pos, d["w_q"], d["w_k"])
        pos += 1
    for _ in range(3):
        d["positions"] = pos.clone()
        graph.replay()
        torch.cuda.synchronize()
        _check_fwd(d, out, 128, False, 0.0, 1.0, where="replay")


def test_workspace_of_the_backward():
    d = _make((2000,), 4, 2, 128, 128, "bf16", 20)
    out = B.rope_fwd(d["q"], d["k"], d["steps"], d["positions"], d["w_q"], d["w_k"])
    need = B.rmsnorm_rope_bwd_workspace_size(128)
    full = torch.full((need + 4096,), 255, dtype=torch.uint8, device=DEV)
    args = (d["dq"], d["dk"], d["steps"], d["positions"], d["q"], d["k"], out[2], out[3], d["w_q"], d["w_k"])
    for variant in ("auto", "generic"):
        res = B.rope_bwd(*args, workspace=full[:need], variant=variant)
        _check_bwd(d, out[2:], res, 128, False, 0.0, 1.0, where="workspace")
        assert bool((full[need:] == 255).all())
    with pytest.raises(B.RMSNormError) as e:
        B.rope_bwd(*args, workspace=full[:need - 4])
    assert e.value.status == -11


@pytest.mark.slow
def test_offsets_past_32_bits():
    T, hq, D = 530000, 32, 128
    d = _make((1000,), hq, 0, D, D, "bf16", 31)
    want = B.rope_fwd(d["q"], None, d["steps"], d["positions"], d["w_q"])
    n = T // 1000
    q = d["q"].expand(n, *d["q"].shape).reshape(T, hq, D)
    pos = d["positions"].expand(n, 1000).reshape(T)
    keep = q.clone()
    out, _, rstd, _ = B.rope_fwd(q, None, d["steps"], pos, d["w_q"], q_out=q)
    for got, w in ((out, want[0]), (rstd, want[2])):
        got = got.view(n, *w.shape)
        assert torch.equal(got[0], w) and torch.equal(got[-1], w) and torch.equal(got[n // 2], w)
    one = B.rope_bwd(d["dq"], None, d["steps"], d["positions"], d["q"], None, want[2], None, d["w_q"])
    dq = d["dq"].expand(n, *d["dq"].shape).reshape(T, hq, D)
    got, _, _, _ = B.rope_bwd(dq, None, d["steps"], pos, keep, None, rstd, None, d["w_q"], dq=dq)
    got = got.view(n, *one[0].shape)
    assert torch.equal(got[0], one[0]) and torch.equal(got[-1], one[0]) and torch.equal(got[n // 2], one[0])


def test_refused_tensors():
    d = _make((4,), 2, 1, 64, 64, "bf16", 21)
    ok = dict(q=d["q"], k=d["k"], steps=d["steps"], positions=d["positions"], w_q=d["w_q"], w_k=d["w_k"])
    for change in (dict(q=d["q"][0]), dict(k=d["k"][:3]), dict(k=d["k"].half()), dict(steps=d["steps"].cpu()),
                   dict(steps=d["steps"].float()), dict(positions=d["positions"].int()),
                   dict(positions=d["positions"][:3]), dict(w_q=d["w_q"][:32]), dict(q=d["q"].cpu()),
                   dict(q_out=d["q"][:, :1]), dict(q=d["q"].transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            B.rope_fwd(**{**ok, **change})
    with pytest.raises(B.RMSNormError) as e:            # more pairs than the head has
        B.rope_fwd(**{**ok, "steps": torch.zeros(40, dtype=torch.int64, device=DEV)})
    assert e.value.status == -2
    with pytest.raises(ValueError):
        B.rope_bwd(d["dq"], d["dk"], d["steps"], d["positions"], q=d["q"][:2], w_q=d["w_q"])
