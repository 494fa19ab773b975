"""The angles of rotary positions, one output at a time: where one value of a pair is
zero, each output is a value times a cos or a sin, and must have all its bits however
small that is, for every type, layout and kernel.

Bound, in u = 2^-24, relative to the output: the angle's fp32 value is off by at most
2 u of itself (a conversion and a sum), which moves a sin by at most 2 u of it and a cos
by 1.6 u (angles are within an eighth of a turn of a quarter turn's multiple); their own
sums by 1.5 u, the magnitude by u, the product by u: 5.5 u. 6 u are allowed, and half a
step of the output's type.
"""
from __future__ import annotations

import math

import pytest
import torch

import ops_util as U
from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
U32 = 2.0 ** -24
POSITIONS = [0, 1, 2, 3, 17, 1000, 131071, 10 ** 7 + 1, (1 << 40) + 5, (1 << 62) + 12345, -1, -4096, -(1 << 63)]


def _cos_sin(phase):
    """cos and sin of phase / 2^64 turns in 64 bits, to a relative 2^-52: the multiple of
    a quarter turn is taken off in integers."""
    phase %= 1 << 64
    quarter = ((phase + (1 << 61)) >> 62) % 4
    rest = phase - (((phase + (1 << 61)) >> 62) << 62)
    t = 2 * math.pi * math.ldexp(rest, -64)
    c, s = math.cos(t), math.sin(t)
    return ((c, s), (-s, c), (-c, -s), (s, -c))[quarter]


def _steps(kind, half):
    if kind == "frequencies":
        return B.rope_steps(2 * half, 10000.0, device="cpu")[0].tolist()
    # tiny turns, and steps a little off the quarters and eighths of a turn
    odd = [1, 3, 1 << 10, (1 << 30) + 7, (1 << 40) - 1, (1 << 50) + 3]
    for k in range(1, 8):
        odd += [(k << 61) - 1, (k << 61) + 1, (k << 61) + (1 << 33), (k << 61) - (1 << 41)]
    odd = [v - (1 << 64) if v >= 1 << 63 else v for v in odd]
    return (odd * 8)[:half]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (80, 20), (66, 66), (512, 512)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["frequencies", "odd"])
@pytest.mark.parametrize("magnitude", [1.0, 1.2079])
def test_outputs_of_one_value_keep_their_bits(dtype, D, R, interleaved, kind, magnitude):
    dt, half, T = U.DT[dtype], R // 2, len(POSITIONS)
    steps = _steps(kind, half)
    table = [[_cos_sin(p * f) for f in steps] for p in POSITIONS]
    cs = torch.tensor(table, dtype=torch.float64, device=DEV)[:, None]  # [T, 1, half, 2]
    c, s = cs[..., 0], cs[..., 1]
    g = torch.Generator().manual_seed(D + R)
    v = (1 + torch.rand(T, 3, half, generator=g)).to(dt).to(DEV)
    a, b = U._pairs(D, R, interleaved)
    st = torch.tensor(steps, dtype=torch.int64, device=DEV)
    pos = torch.tensor(POSITIONS, dtype=torch.int64, device=DEV)
    m = float(torch.tensor(magnitude, dtype=torch.float32))
    for variant in ("auto", "generic"):
        for first in (True, False):
            x = torch.zeros(T, 3, D, dtype=dt, device=DEV)
            x[..., a if first else b] = v
            kw = dict(interleaved=interleaved, magnitude=magnitude, variant=variant)
            out = B.rope_fwd(x, None, st, pos, **kw)[0].double()
            back = B.rope_bwd(x, None, st, pos, **kw)[0].double()
            vd = m * v.double()
            want = (vd * c, vd * s) if first else (-vd * s, vd * c)
            turned_back = (vd * c, -vd * s) if first else (vd * s, vd * c)
            for got, (wa, wb), where in ((out, want, "out"), (back, turned_back, "back")):
                for w, at in ((wa, a), (wb, b)):
                    bound = U.half_step(w, dt) + 6 * U32 * w.abs()
                    err = (got[..., at] - w).abs()
                    worst = float((err / bound).max())
                    assert worst <= 1, f"{where} {variant} first={first}: {worst:.3g} of the bound"
                assert bool((got[..., R:] == 0).all())
