"""The plain implementations that the operators' GPU tests compare with, tested
themselves: backward formulas against differentiation of the forward ones, the
rotation against complex numbers, the 8- and 4-bit codes against torch's own
conversion, and the frequencies of rmsnorm_rope_steps.
"""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import ops_util as U
from memory_bound_normalization_fwd_gb300 import binding as B
from memory_bound_normalization_fwd_gb300 import build as BUILD


@pytest.fixture(scope="module", autouse=True)
def _built():
    BUILD.build()


def _rand(*shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("post,pre,gate_rows", [(True, True, 0), (True, True, 7), (True, True, 2),
                                               (True, True, 1), (True, False, 3), (False, True, 2),
                                               (False, True, 0), (True, False, 0)])
def test_block_gradients_are_the_derivatives_of_the_forward(post, pre, gate_rows):
    M, N, off, al, be = 7, 6, 1.0, 0.7, 0.9
    h, r = _rand(M, N).requires_grad_(), _rand(M, N, seed=1).requires_grad_()
    wa = _rand(N, seed=2).requires_grad_() if post else None
    wb = _rand(N, seed=3).requires_grad_() if pre else None
    gate = _rand(-(-M // gate_rows), N, seed=4).requires_grad_() if gate_rows else None
    s, y, a, b, _, _ = U.block_fwd(h, r, wa, wb, gate, gate_rows, 1e-6, off, al, be)
    ds, dy = _rand(M, N, seed=5), _rand(M, N, seed=6)
    loss = (s * ds).sum() + ((y * dy).sum() if pre else 0)
    ins = {"dh": h, "dr": r, "dgate": gate, "dw_post": wa, "dw_pre": wb}
    ins = {k: v for k, v in ins.items() if v is not None}
    want = dict(zip(ins, torch.autograd.grad(loss, list(ins.values()))))
    with torch.no_grad():
        got, _ = U.block_bwd(h, s, a, b, dy if pre else None, ds, wa, wb, gate, gate_rows, off, al, be)
    assert set(got) == set(want)
    for k in want:
        assert torch.allclose(got[k], want[k], rtol=1e-10, atol=1e-10), k
    # and against differences of the forward itself
    def f(hh):
        s1, y1, *_ = U.block_fwd(hh, r, wa, wb, gate, gate_rows, 1e-6, off, al, be)
        return (s1 * ds).sum() + ((y1 * dy).sum() if pre else 0)
    d = _rand(M, N, seed=7)
    with torch.no_grad():
        diff = (f(h + 1e-6 * d) - f(h - 1e-6 * d)) / 2e-6
    assert abs(float(diff - (want["dh"] * d).sum())) < 1e-6


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R,norm", [(8, 8, True), (8, 4, True), (10, 6, False), (7, 2, True)])
def test_rope_gradients_are_the_derivatives_of_the_forward(D, R, norm, interleaved):
    T, H = 3, 2
    x = _rand(T, H, D).requires_grad_()
    w = _rand(D, seed=1).requires_grad_() if norm else None
    angle = _rand(T, R // 2, seed=2) * 10
    y, rstd, _ = U.rope_fwd(x, angle, w, R, interleaved, 1e-6, 1.0, 1.3)
    d = _rand(T, H, D, seed=3)
    want = torch.autograd.grad((y * d).sum(), [x, w] if norm else [x])
    with torch.no_grad():
        dx, dw, _, _ = U.rope_bwd(d, x, rstd, angle, w, R, interleaved, 1.0, 1.3)
    assert torch.allclose(dx, want[0], rtol=1e-10, atol=1e-10)
    if norm:
        assert torch.allclose(dw, want[1], rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("interleaved", [False, True])
def test_turning_is_multiplication_by_a_complex_unit(interleaved):
    R = 6
    x, angle = _rand(4, 1, 8), _rand(4, 3, seed=1) * 100
    y = U.turn(x, angle, R, interleaved, 1.0, 1.0)
    pick = (lambda t: torch.complex(t[..., 0:R:2], t[..., 1:R:2])) if interleaved else \
        (lambda t: torch.complex(t[..., :R // 2].contiguous(), t[..., R // 2:R].contiguous()))
    want = pick(x) * torch.polar(torch.ones_like(angle), angle)[:, None]
    assert torch.allclose(pick(y), want, rtol=1e-12, atol=1e-12)
    assert torch.equal(y[..., R:], x[..., R:])


def test_e4m3_codes_are_torchs_own():
    x = torch.cat([_rand(4000) * 100, torch.tensor(U._e4m3_values()[:127], dtype=torch.float64),
                   torch.tensor([448.0] * 32, dtype=torch.float64)]).float()
    x = x[: x.numel() // 32 * 32].clamp(-448, 448).view(-1, 32)
    x[:, 0] = 448.0  # scale 1 for every group
    codes, scales = U.encode(x, "e4m3")
    assert bool((scales == 127).all())
    assert torch.equal(codes.flatten(-2) if codes.dim() > 2 else codes, x.to(torch.float8_e4m3fn).view(torch.uint8))
    v = U.code_values("e4m3")[codes.long()]
    assert torch.equal(v.float(), x.to(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("x,fmt,byte,code", [
    (448.0, "e4m3", 127, 126), (449.0, "e4m3", 128, 118), (224.0, "e4m3", 126, 126),
    (0.0, "e4m3", 0, 0), (2.0 ** -140, "e4m3", 0, 0), (6.0, "e2m1", 127, 7), (6.01, "e2m1", 128, 5),
    (3.0, "e2m1", 126, 7), (-3.0, "e2m1", 126, 15), (float("inf"), "e4m3", 255, 0),
])
def test_scale_byte_is_the_smallest_power_of_two(x, fmt, byte, code):
    codes, scales = U.encode(torch.tensor([x, 0.0], dtype=torch.float64), fmt)
    assert int(scales[0]) == byte and int(codes[0]) == code


def test_encode_rounds_ties_to_the_even_code():
    x = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0], dtype=torch.float64)
    codes, scales = U.encode(x, "e2m1")
    assert int(scales[0]) == 127
    assert codes.tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 14]


# ---- rmsnorm_rope_steps (host only) -----------------------------------------------

def _freq(steps):
    return [int(v) % (1 << 64) / 2.0 ** 64 * 2 * math.pi for v in steps.tolist()]


@pytest.mark.parametrize("R,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (80, 1.5)])
def test_plain_steps(R, base):
    steps, mag = B.rope_steps(R, base, device="cpu")
    assert mag == 1.0 and steps.shape == (R // 2,)
    for i, f in enumerate(_freq(steps)):
        assert f == pytest.approx(base ** (-2.0 * i / R), rel=1e-13)


def test_scaled_steps():
    R, base = 64, 10000.0
    plain = [base ** (-2.0 * i / R) for i in range(R // 2)]
    lin, mag = B.rope_steps(R, base, dict(kind="linear", factor=4.0), device="cpu")
    assert mag == 1.0 and _freq(lin) == pytest.approx([f / 4 for f in plain], rel=1e-13)
    ntk, _ = B.rope_steps(R, base, dict(kind="ntk", factor=8.0), device="cpu")
    assert _freq(ntk)[0] == pytest.approx(1.0) and _freq(ntk)[-1] == pytest.approx(plain[-1] / 8, rel=1e-12)
    yarn, mag = B.rope_steps(R, base, dict(kind="yarn", factor=16.0, length=4096), device="cpu")
    assert mag == pytest.approx(0.1 * math.log(16.0) + 1.0, rel=1e-6)
    got = _freq(yarn)
    assert got[0] == pytest.approx(plain[0], rel=1e-13)              # turns often: stays
    assert got[-1] == pytest.approx(plain[-1] / 16, rel=1e-12)       # under one turn: divided
    ratio = [g / p for g, p in zip(got, plain)]
    assert all(a >= b - 1e-12 for a, b in zip(ratio, ratio[1:]))      # a falling ramp between
    bands, mag = B.rope_steps(R, base, dict(kind="bands", factor=8.0, length=8192), device="cpu")
    assert mag == 1.0
    for f, p in zip(_freq(bands), plain):
        turns = 8192 * p / (2 * math.pi)
        want = p if turns > 4 else p / 8 if turns < 1 else \
            p / 8 * (1 - (turns - 1) / 3) + p * (turns - 1) / 3
        assert f == pytest.approx(want, rel=1e-12)


@pytest.mark.parametrize("R,base,length,divided", [
    (64, 1e4, 1.0, True), (64, 1e4, 6.0, True), (128, 1e4, 0.01, True),   # under one turn, all
    (64, 100.0, 1e9, False), (128, 2.0, 1e5, False), (2, 1e4, 1e9, False),  # above 32 turns, all
])
def test_yarn_where_all_pairs_are_on_one_side_of_the_ramp(R, base, length, divided):
    steps, _ = B.rope_steps(R, base, dict(kind="yarn", factor=4.0, length=length), device="cpu")
    for i, f in enumerate(_freq(steps)):
        turns = length * base ** (-2.0 * i / R) / (2 * math.pi)
        assert turns <= 1 if divided else turns >= 32
        assert f == pytest.approx(base ** (-2.0 * i / R) / (4 if divided else 1), rel=1e-13)


@pytest.mark.parametrize("R,base,scaling,code", [
    (0, 1e4, None, -2), (3, 1e4, None, -2), (-2, 1e4, None, -2), (1 << 17, 1e4, None, -2),
    (64, 1.0, None, -4), (64, float("nan"), None, -4), (64, float("inf"), None, -4),
    (64, 1e4, dict(kind="linear", factor=0.5), -4), (64, 1e4, dict(kind="ntk", factor=float("inf")), -4),
    (2, 1e4, dict(kind="ntk", factor=2.0), -2), (64, 1e4, dict(kind="yarn", factor=2.0), -4),
    (64, 1e4, dict(kind="yarn", factor=2.0, length=10, beta_fast=1.0, beta_slow=2.0), -4),
    (64, 1e4, dict(kind="bands", factor=2.0, length=10, beta_slow=0.0), -4),
])
def test_steps_refusals(R, base, scaling, code):
    with pytest.raises(B.RMSNormError) as e:
        B.rope_steps(R, base, scaling, device="cpu")
    assert e.value.status == code


def test_steps_refuse_unknown_scalings():
    with pytest.raises(ValueError):
        B.rope_steps(64, scaling=dict(kind="other"), device="cpu")
    with pytest.raises(ValueError):
        B.rope_steps(64, scaling=dict(kind="linear", factr=2.0), device="cpu")
    sc = B.RopeScaling(ctypes.sizeof(B.RopeScaling), 9, 1.0, 0.0, 0.0, 0.0)
    out = (ctypes.c_uint64 * 32)()
    assert B.rmsnorm_rope_steps(64, 1e4, sc, ctypes.addressof(out)) == -9
    assert B.rmsnorm_rope_steps(64, 1e4, None, 0) == -1
