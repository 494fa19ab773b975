"""Plain 64-bit implementations of the block, rope and cache operators, written
from the formulas of include/rmsnorm.h, and the error bounds of their tests.

Bounds. A value computed in fp32 and rounded once to its dtype is off by half a
step of the dtype (finfo.eps / 2 relative, half the smallest subnormal near
zero) plus the fp32 error of its terms. Each term is a product of a few fp32
values and, for the norms, of a row sum; the kernels' sums run over at most
about 150 terms per thread, then over at most 64 partial sums, so each
sum is within (150 + 64) * 2^-24 = 1.3e-5 of the sum of its terms' magnitudes in
the worst case, which random rounding keeps far below: TAU = 1e-5 relative to the
magnitudes (the bound of the forward's and backward's own tests).
"""
from __future__ import annotations

import torch

TAU = 1e-5
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(v, dtype):
    """Half a step of dtype at |v| (64-bit tensors)."""
    fi = torch.finfo(dtype)
    tiny = fi.smallest_normal * fi.eps
    return torch.clamp(v.abs() * (fi.eps / 2) * (1 + 1e-9), min=tiny / 2)


def check(got, want, magnitude, dtype, what):
    """|got - want| <= half a step of dtype + TAU * magnitude, elementwise."""
    if dtype is not None:
        assert got.dtype == dtype, (what, got.dtype)
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bound = TAU * magnitude.expand(want.shape) + half_step(want, got.dtype if dtype is None else dtype)
    err = (got - want).abs()
    ok = err <= bound
    if not bool(ok.all()):
        i = int(torch.nan_to_num(err / bound, nan=float("inf")).argmax())
        raise AssertionError(f"{what}: off by {float((err / bound).flatten()[i]):.3g} of the bound at "
                             f"{i}: {float(got.flatten()[i])!r} for {float(want.flatten()[i])!r}")


# ---- block ----------------------------------------------------------------------

def gate_index(M, gate_rows, device):
    return torch.arange(M, device=device) // gate_rows


def block_fwd(h, r, w_post, w_pre, gate, gate_rows, eps, offset, alpha, beta):
    """s, y, rstd_post, rstd_pre in 64 bits and the magnitudes behind s and y."""
    h, r = h.double(), r.double()
    a = b = y = my = None
    n = h
    if w_post is not None:
        a = 1 / torch.sqrt((h * h).mean(-1) + eps)
        n = h * a[:, None] * (offset + w_post.double())
    if gate is not None:
        n = n * gate.double()[gate_index(h.shape[0], gate_rows, h.device)]
    s = beta * r + alpha * n
    ms = abs(beta) * r.abs() + abs(alpha) * n.abs()
    if w_pre is not None:
        w = offset + w_pre.double()
        b = 1 / torch.sqrt((s * s).mean(-1) + eps)
        y = s * b[:, None] * w
        my = (ms + s.abs()) * b[:, None] * w.abs()
    return s, y, a, b, ms, my


def block_bwd(h, s, a, b, dy, ds, w_post, w_pre, gate, gate_rows, offset, alpha, beta):
    """Gradients in 64 bits by the header's formulas, and their magnitudes:
    dicts with dh, dr, dgate, dw_post, dw_pre."""
    M, N = h.shape
    h = h.double()
    t = torch.zeros_like(h) if ds is None else ds.double()
    mt = t.abs()
    out, mag = {}, {}
    if w_pre is not None:
        s, b, w, dy = s.double(), b.double()[:, None], offset + w_pre.double(), dy.double()
        u = dy * w
        t = t + b * (u - s * b * b * (u * s).sum(-1, keepdim=True) / N)
        mt = mt + b * (u.abs() + s.abs() * b * b * (u * s).abs().sum(-1, keepdim=True) / N)
        out["dw_pre"], mag["dw_pre"] = (dy * s * b).sum(0), (dy * s * b).abs().sum(0)
    out["dr"], mag["dr"] = beta * t, abs(beta) * mt
    g = torch.ones(M, N, dtype=torch.float64, device=h.device)
    if gate is not None:
        which = gate_index(M, gate_rows, h.device)
        g = gate.double()[which]
    if w_post is None:
        n, k, w = h, None, None
    else:
        k, w = a.double()[:, None], offset + w_post.double()
        n = h * k * w
    if gate is not None:
        z = torch.zeros(gate.shape, dtype=torch.float64, device=h.device)
        out["dgate"] = z.index_add(0, which, alpha * t * n)
        mag["dgate"] = z.index_add(0, which, abs(alpha) * mt * n.abs())
    if w_post is None:
        out["dh"], mag["dh"] = alpha * g * t, (alpha * g).abs() * mt
        return out, mag
    out["dw_post"] = (alpha * g * t * h * k).sum(0)
    mag["dw_post"] = ((alpha * g * h * k).abs() * mt).sum(0)
    v, mv = alpha * g * t * w, (alpha * g * w).abs() * mt
    out["dh"] = k * (v - h * k * k * (v * h).sum(-1, keepdim=True) / N)
    mag["dh"] = k * (mv + h.abs() * k * k * (mv * h.abs()).sum(-1, keepdim=True) / N)
    return out, mag


# ---- rope -----------------------------------------------------------------------

def rope_angles(steps, positions):
    """Angles in 64 bits from the integer phases: positions [..., T], steps as
    the call takes them, modulo one turn in exact integer arithmetic."""
    pos = [int(v) for v in positions.flatten().tolist()]
    st = [int(v) % (1 << 64) for v in steps.tolist()]
    turns = [[((p * f) % (1 << 64)) / 2.0 ** 64 for f in st] for p in pos]
    a = torch.tensor(turns, dtype=torch.float64).view(*positions.shape, len(st))
    return 2 * torch.pi * a.to(positions.device)


def _pairs(D, R, interleaved):
    half = R // 2
    i = torch.arange(half)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + half)


def turn(x, angle, R, interleaved, magnitude, sign):
    """x [..., T, H, D] turned by sign * angle [..., T, R/2]."""
    a, b = _pairs(x.shape[-1], R, interleaved)
    c, s = magnitude * torch.cos(angle)[..., None, :], sign * magnitude * torch.sin(angle)[..., None, :]
    out = x.clone()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def turn_magnitude(m, R, interleaved, magnitude):
    a, b = _pairs(m.shape[-1], R, interleaved)
    out = m.clone()
    both = abs(magnitude) * (m[..., a] + m[..., b])
    out[..., a] = both
    out[..., b] = both
    return out


def rope_fwd(x, angle, w, R, interleaved, eps, offset, magnitude):
    x = x.double()
    rstd = None
    if w is not None:
        rstd = 1 / torch.sqrt((x * x).mean(-1) + eps)
        x = x * rstd[..., None] * (offset + w.double())
    return (turn(x, angle, R, interleaved, magnitude, 1.0), rstd,
            turn_magnitude(x.abs(), R, interleaved, magnitude))


def rope_bwd(d, x, rstd, angle, w, R, interleaved, offset, magnitude):
    """dx, dw in 64 bits and their magnitudes."""
    d = d.double()
    t = turn(d, angle, R, interleaved, magnitude, -1.0)
    mt = turn_magnitude(d.abs(), R, interleaved, magnitude)
    if w is None:
        return t, None, mt, None
    x, r, w = x.double(), rstd.double()[..., None], offset + w.double()
    D = x.shape[-1]
    over = tuple(range(x.dim() - 1))
    dw, mdw = (t * x * r).sum(over), (mt * (x * r).abs()).sum(over)
    dx = r * (t * w - x * r * r * (t * w * x).sum(-1, keepdim=True) / D)
    mw = mt * w.abs()
    mdx = r * (mw + x.abs() * r * r * (mw * x.abs()).sum(-1, keepdim=True) / D)
    return dx, dw, mdx, mdw


# ---- cache ----------------------------------------------------------------------

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3_values():
    out = []
    for c in range(128):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    out[127] = float("nan")
    return out


def code_values(fmt):
    """The value of every code, in 64 bits (a code's sign is its top bit)."""
    v = _e4m3_values() if fmt == "e4m3" else E2M1
    return torch.tensor(v + [-x for x in v], dtype=torch.float64)


def encode(x, fmt):
    """Codes (one per value) and scale bytes of x [..., D], by search: the scale is the
    first power of two that brings the group's largest value within the format,
    a code the nearest value, of two equally near the one with an even code."""
    x = x.double().cpu()
    D = x.shape[-1]
    groups = -(-D // 32)
    pad = torch.zeros(*x.shape[:-1], groups * 32, dtype=torch.float64)
    pad[..., :D] = x
    f = pad.unflatten(-1, (groups, 32))
    mags = torch.tensor((_e4m3_values()[:127] if fmt == "e4m3" else E2M1), dtype=torch.float64)
    peak = f.abs().amax(-1)
    bad = ~torch.isfinite(f).all(-1)
    peak = torch.where(bad, torch.ones_like(peak), peak)
    powers = torch.pow(torch.tensor(2.0, dtype=torch.float64), torch.arange(-127, 128, dtype=torch.float64))
    byte = torch.searchsorted(mags[-1] * powers, peak.contiguous())  # first with limit >= peak
    f = torch.where(bad[..., None], torch.zeros_like(f), f) / powers[byte][..., None]
    m = f.abs()
    hi = torch.searchsorted(mags, m.contiguous()).clamp(max=len(mags) - 1)
    lo = (hi - 1).clamp(min=0)
    down, up = m - mags[lo], mags[hi] - m
    code = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = code + torch.signbit(f) * (128 if fmt == "e4m3" else 8)
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    return code.flatten(-2)[..., :D].to(torch.uint8), byte.to(torch.uint8)


def pack(code, fmt):
    if fmt == "e4m3":
        return code
    if code.shape[-1] % 2:
        code = torch.cat([code, torch.zeros_like(code[..., :1])], -1)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def unpack(codes, fmt, D):
    if fmt == "e4m3":
        return codes
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :D]


def decode(codes, scales, fmt, D, dtype):
    """Values of packed codes and scale bytes, rounded once to dtype (on the CPU)."""
    v = code_values(fmt)[unpack(codes.cpu(), fmt, D).long()]
    e = scales.cpu().long()
    p = torch.pow(torch.tensor(2.0, dtype=torch.float64), (e - 127).double())
    p = torch.where(e == 255, torch.full_like(p, float("nan")), p)
    v = v * p.repeat_interleave(32, -1)[..., :D]
    if dtype is torch.float32:
        return v.to(dtype)
    # via fp32 the values are exact, so this rounds once
    return v.float().to(dtype)
