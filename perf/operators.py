"""The operators of a transformer block that run between its matrix products:
what is measured of them.

Three operators, each with the calls that belong to it:

block   the norm after a block, its gate, the scaled residual and the norm
        before the next block, forward and backward
rope    rotary positions on the heads of q and k, with the RMSNorm of each
        head in front where a model has one, forward and backward
cache   a paged cache of k and v in 8 or 4 bits per value with one power-of-two
        scale for 32 values: written token by token, read back by page table

`run` computes a case in elementary torch operations (in 32 bits, angles in
64), or, where `own` is true, by the calls of this package. `exact` computes
the same from the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EB = {"bf16": 2, "fp16": 2, "fp32": 4}
DEV = "cuda"


# ---- the cases -------------------------------------------------------------

def listed():
    return [
        # One decoding step of 16 sequences at the hidden size of the 131072x4096
        # workload: the smallest call, all latency.
        dict(name="block_fwd_decode", op="block_fwd", M=16, N=4096, dtype="bf16", gate="none",
             post=True, pre=True, offset=0.0, alpha=1.0, beta=1.0),
        # Eight packed training sequences of 2048 tokens, each with its own gate row.
        dict(name="block_fwd_train", op="block_fwd", M=16384, N=4096, dtype="bf16", gate="group",
             group=2048, post=True, pre=True, offset=0.0, alpha=1.0, beta=1.0),
        # The same batch's backward pass: the largest training call.
        dict(name="block_bwd_train", op="block_bwd", M=16384, N=4096, dtype="bf16", gate="group",
             group=2048, post=True, pre=True, offset=0.0, alpha=1.0, beta=1.0),
        # An odd batch at the non-power-of-two hidden size, 32-bit, a gate for
        # every element, weights about zero (offset 1), a scaled residual.
        dict(name="block_bwd_odd_fp32", op="block_bwd", M=4091, N=1000, dtype="fp32",
             gate="element", post=True, pre=True, offset=1.0, alpha=0.5, beta=0.9),
        # One decoding step of 64 sequences far into long contexts: head norms and
        # rotation of 32 query heads over 8 key heads.
        dict(name="rope_fwd_decode", op="rope_fwd", T=64, hq=32, hk=8, D=128, R=128,
             interleaved=False, dtype="bf16", norm=True, offset=0.0, scaling="none", far=131072),
        # A prompt of 16384 tokens with half of each head rotated in the interleaved
        # layout, frequencies scaled to a longer context, no head norms.
        dict(name="rope_fwd_prompt_fp16", op="rope_fwd", T=16384, hq=32, hk=8, D=128, R=64,
             interleaved=True, dtype="fp16", norm=False, offset=0.0, scaling="yarn", far=131072),
        # Training: the backward pass through rotation and head norms.
        dict(name="rope_bwd_train", op="rope_bwd", T=16384, hq=32, hk=8, D=128, R=128,
             interleaved=False, dtype="bf16", norm=True, offset=0.0, scaling="none", far=4096),
        # An odd token count, few heads of an odd width, 32-bit.
        dict(name="rope_bwd_odd_fp32", op="rope_bwd", T=1021, hq=7, hk=1, D=80, R=80,
             interleaved=False, dtype="fp32", norm=True, offset=1.0, scaling="linear", far=8192),
        # One decoding step of 64 sequences appended to an 8-bit cache.
        dict(name="cache_write_decode", op="cache_write", T=64, heads=8, D=128, fmt="e4m3",
             dtype="bf16", page=16, pages=512),
        # A long prompt written into the cache, some of its tokens padding.
        dict(name="cache_write_prompt", op="cache_write", T=32768, heads=8, D=128, fmt="e4m3",
             dtype="bf16", page=16, pages=2560),
        # Chunked prompts of 32 sequences read back for attention: the largest read.
        dict(name="cache_read_long", op="cache_read", B=32, longest=8192, heads=8, D=128,
             fmt="e4m3", dtype="bf16", page=16),
        # A ragged batch through the 4-bit cache and back, as a 4-bit cache is used.
        dict(name="cache_trip_e2m1", op="cache_trip", B=9, longest=397, heads=5, D=96, fmt="e2m1",
             dtype="fp16", page=24),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["block_fwd", "block_bwd", "rope_fwd", "rope_bwd", "cache_write", "cache_read",
                     "cache_trip"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op.startswith("block"):
        N = _log(rng, 64, 8192)
        if rng.random() < 0.8:  # hidden sizes are whole 16-byte vectors nearly always
            N = max(8, N // 8 * 8)
        M = min(_log(rng, 1, 32768), 16384 * 4096 * 2 * 3 // 4 // (N * EB[dtype]))
        gate = rng.choice(["none", "channel", "group", "element"])
        post = rng.random() < 0.8
        return dict(op=op, M=M, N=N, dtype=dtype, gate=gate, group=_log(rng, 2, 4096), post=post,
                    pre=not post or rng.random() < 0.8, offset=float(rng.randrange(2)),
                    alpha=rng.choice([1.0, 0.25]), beta=rng.choice([1.0, 0.75]))
    if op.startswith("rope"):
        D = rng.choice([64, 80, 96, 112, 128, 128, 192, 256])
        hk = rng.choice([1, 2, 4, 5, 8])
        hq = hk * rng.choice([1, 2, 4, 7])
        R = rng.choice([D, D, D // 2, D // 4 // 2 * 2])
        T = min(_log(rng, 1, 32768), 16384 * 40 * 128 * 2 // ((hq + hk) * D * EB[dtype]))
        return dict(op=op, T=T, hq=hq, hk=hk, D=D, R=R, interleaved=rng.random() < 0.5, dtype=dtype,
                    norm=rng.random() < 0.6, offset=float(rng.randrange(2)),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                    far=_log(rng, 64, 1 << 20))
    heads, D = rng.choice([1, 2, 5, 8]), rng.choice([64, 96, 128, 256])
    page = rng.choice([1, 8, 16, 24, 64])
    fmt = rng.choice(["e4m3", "e2m1"]) if op != "cache_write" else "e4m3"
    if op == "cache_write":
        T = min(_log(rng, 1, 32768), 32768 * 1024 * 2 // (heads * D * EB[dtype]))
        return dict(op=op, T=T, heads=heads, D=D, fmt=fmt, dtype=dtype, page=page,
                    pages=-(-T * 5 // 4 // page) + 1)
    B = _log(rng, 1, 64)
    longest = _log(rng, 1, 8192)
    cap = (16 if op == "cache_read" else 4) * 8192 * 1024 * 2 // (heads * D * EB[dtype])
    return dict(op=op, B=B, longest=max(1, min(longest, cap // B)), heads=heads, D=D, fmt=fmt,
                dtype=dtype, page=page)


# ---- inputs ----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return _PREPARE[case["op"].split("_")[0]](case, g)


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _weight(g, n, offset, dtype):
    w = 0.5 + torch.rand(n, generator=g, device=DEV) if offset == 0.0 else \
        0.3 * torch.randn(n, generator=g, device=DEV)
    return w.to(dtype)


def _gate_rows(case):
    return {"none": 0, "channel": case["M"], "group": case.get("group", 0), "element": 1}[case["gate"]]


def _prepare_block(case, g):
    M, N, dt, off = case["M"], case["N"], DT[case["dtype"]], case["offset"]
    st = dict(case=case, w_post=_weight(g, N, off, dt) if case["post"] else None,
              w_pre=_weight(g, N, off, dt) if case["pre"] else None, gate=None, eps=1e-6)
    # A block's output varies in size from token to token, and so does the
    # residual stream, which has grown over the layers before.
    size = torch.exp(torch.randn(M, 1, generator=g, device=DEV))
    st["h"] = (torch.randn(M, N, generator=g, device=DEV) * size).to(dt)
    st["r"] = _randn(g, M, N, dtype=dt, scale=4.0)
    rows = _gate_rows(case)
    if rows:
        st["gate"] = _randn(g, -(-M // rows), N, dtype=dt, scale=0.5) + 0.5
    if case["op"] == "block_bwd":
        # What the forward pass kept: the new residual and both rows' rstd.
        s, y, a, b = _plain_block_fwd(st)
        st.update(s=s, rstd_post=a, rstd_pre=b, dy=None, ds=_randn(g, M, N, dtype=dt))
        if case["pre"]:
            st["dy"] = _randn(g, M, N, dtype=dt)
        del st["r"]
    if own:
        from memory_bound_normalization_fwd_gb300 import binding
        st["B"] = binding
    return st


def _scaling(case):
    kind = case["scaling"]
    return {"none": None, "linear": dict(kind="linear", factor=4.0),
            "ntk": dict(kind="ntk", factor=8.0),
            "yarn": dict(kind="yarn", factor=32.0, length=4096),
            "bands": dict(kind="bands", factor=8.0, length=8192)}[kind]


def _frequencies(R, base, sc):
    """Radians per position of each pair (64-bit, Python floats), and the factor
    on cos and sin, for a rotation scaled to longer contexts."""
    kind = sc["kind"] if sc else "none"
    if kind == "ntk" and R > 2:
        base = base * sc["factor"] ** (R / (R - 2))
    inv = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if kind == "linear":
        inv = [f / sc["factor"] for f in inv]
    elif kind == "yarn":
        def at(turns):
            return R * math.log(sc["length"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), R - 1)
        hi = hi + 0.001 if hi == lo else hi
        out = []
        for i, f in enumerate(inv):
            t = min(max((i - lo) / (hi - lo), 0.0), 1.0)
            out.append(f / sc["factor"] * t + f * (1.0 - t))
        return out, 0.1 * math.log(sc["factor"]) + 1.0
    elif kind == "bands":
        out = []
        for f in inv:
            waves = sc["length"] * f / (2 * math.pi)
            t = min(max((waves - 1.0) / (4.0 - 1.0), 0.0), 1.0)
            out.append(f / sc["factor"] * (1.0 - t) + f * t)
        inv = out
    return inv, 1.0


def _prepare_rope(case, g):
    T, hq, hk, D, R = case["T"], case["hq"], case["hk"], case["D"], case["R"]
    dt, off = DT[case["dtype"]], case["offset"]
    st = dict(case=case, eps=1e-6)
    # q and k are slices of one projection's rows, with v behind them.
    qkv = _randn(g, T, hq + 2 * hk, D, dtype=dt)
    st["q"], st["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
    start = int(torch.randint(0, max(1, case["far"] - T + 1), (1,), generator=g, device=DEV))
    st["positions"] = start + torch.arange(T, device=DEV) if T > 256 else \
        torch.randint(0, case["far"], (T,), generator=g, device=DEV)
    st["w_q"] = _weight(g, D, off, dt) if case["norm"] else None
    st["w_k"] = _weight(g, D, off, dt) if case["norm"] else None
    inv, mag = _frequencies(R, 10000.0, _scaling(case))
    st["inv"], st["mag"] = torch.tensor(inv, dtype=torch.float64, device=DEV), mag
    if case["op"] == "rope_bwd":
        st["dq"] = _randn(g, T, hq, D, dtype=dt)
        st["dk"] = _randn(g, T, hk, D, dtype=dt)
        if case["norm"]:
            st["rstd_q"] = torch.rsqrt(st["q"].float().square().mean(-1) + 1e-6)
            st["rstd_k"] = torch.rsqrt(st["k"].float().square().mean(-1) + 1e-6)
    if own:
        from memory_bound_normalization_fwd_gb300 import binding
        st["B"] = binding
        st["steps"], st["mag"] = binding.rope_steps(R, base=10000.0, scaling=_scaling(case),
                                                    device=DEV)
    return st


def _code_bytes(case):
    return case["D"] if case["fmt"] == "e4m3" else case["D"] // 2


def _lengths(case):
    """The rows of each sequence: the same for every seed, one of them the longest."""
    rng = random.Random(case["B"] * 65537 + case["longest"])
    lens = [rng.randint(0, case["longest"]) for _ in range(case["B"])]
    lens[case["B"] // 2] = case["longest"]
    return lens


def _prepare_cache(case, g):
    heads, D, page, dt = case["heads"], case["D"], case["page"], DT[case["dtype"]]
    st = dict(case=case)
    if case["op"] == "cache_write":
        T, pages = case["T"], case["pages"]
        kv = _randn(g, T, 2 * heads, D, dtype=dt)
        # Keys have a few channels far above the rest.
        kv[:, :heads, :: 32] *= 8
        st["k"], st["v"] = kv[:, :heads], kv[:, heads:]
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:T]
        pad = torch.rand(T, generator=g, device=DEV) < 0.05
        st["slots"] = torch.where(pad, torch.full_like(slots, -1), slots)
    else:
        B, longest = case["B"], case["longest"]
        lens = torch.tensor(_lengths(case), device=DEV)
        width = -(-longest // page) + 1
        pages = B * width
        st["table"] = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).view(B, width)
        cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
        cu[1:] = lens.cumsum(0)
        st["cu"] = cu
        rows = int(cu[-1])
        st["rows"] = rows
        # Which slot each row of the batch lives in.
        row = torch.arange(rows, device=DEV)
        seq = torch.searchsorted(cu[1:].contiguous(), row.to(torch.int32), right=True)
        at = row - cu[seq].long()
        st["slots"] = st["table"][seq, at // page].long() * page + at % page
        if case["op"] == "cache_trip":
            kv = _randn(g, rows, 2 * heads, D, dtype=dt)
            st["k"], st["v"] = kv[:, :heads], kv[:, heads:]
    shape = (pages, page, heads)
    st["k_codes"], st["v_codes"] = (torch.zeros(*shape, _code_bytes(case), dtype=torch.uint8,
                                                device=DEV) for _ in range(2))
    st["k_scales"], st["v_scales"] = (torch.zeros(*shape, D // 32, dtype=torch.uint8, device=DEV)
                                      for _ in range(2))
    if case["op"] == "cache_read":
        for c in (st["k_codes"], st["v_codes"]):
            c.random_(0, 256, generator=g)
            if case["fmt"] == "e4m3":
                c[(c & 127) == 127] = 0  # the format's two NaN codes
        for c in (st["k_scales"], st["v_scales"]):
            c.random_(115, 131, generator=g)
    if own:
        from memory_bound_normalization_fwd_gb300 import binding
        st["B"] = binding
        st["cache"] = binding.Cache(pages, page, heads, D, fmt=case["fmt"], tensors=(
            st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"]))
    return st


_PREPARE = {"block": _prepare_block, "rope": _prepare_rope, "cache": _prepare_cache}


# ---- one pass --------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return _own(op, state) if own else _PLAIN[op](state)


def _own(op, st):
    B, c = st["B"], st["case"]
    if op == "block_fwd":
        return [t for t in B.block_fwd(st["h"], st["r"], w_post=st["w_post"], w_pre=st["w_pre"],
                                       gate=st["gate"], gate_rows=_gate_rows(c), eps=st["eps"],
                                       offset=c["offset"], alpha=c["alpha"], beta=c["beta"])
                if t is not None]
    if op == "block_bwd":
        return [t for t in B.block_bwd(st["h"], st["s"], st["rstd_post"], st["rstd_pre"],
                                       dy=st["dy"], ds=st["ds"], w_post=st["w_post"],
                                       w_pre=st["w_pre"], gate=st["gate"],
                                       gate_rows=_gate_rows(c), offset=c["offset"],
                                       alpha=c["alpha"], beta=c["beta"]) if t is not None]
    if op == "rope_fwd":
        return [t for t in B.rope_fwd(st["q"], st["k"], st["steps"], positions=st["positions"],
                                      w_q=st["w_q"], w_k=st["w_k"], interleaved=c["interleaved"],
                                      eps=st["eps"], offset=c["offset"], magnitude=st["mag"])
                if t is not None]
    if op == "rope_bwd":
        norm = c["norm"]
        return [t for t in B.rope_bwd(st["dq"], st["dk"], st["steps"], positions=st["positions"],
                                      q=st["q"] if norm else None, k=st["k"] if norm else None,
                                      rstd_q=st["rstd_q"] if norm else None,
                                      rstd_k=st["rstd_k"] if norm else None,
                                      w_q=st["w_q"], w_k=st["w_k"], interleaved=c["interleaved"],
                                      offset=c["offset"], magnitude=st["mag"]) if t is not None]
    if op == "cache_write":
        B.cache_write(st["cache"], st["k"], st["v"], st["slots"])
        return _cache_values(st)
    if op == "cache_trip":
        B.cache_write(st["cache"], st["k"], st["v"], st["slots"])
    return B.cache_read(st["cache"], st["table"], st["cu"], st["rows"], dtype=DT[c["dtype"]])


def _cache_values(st):
    f8 = torch.float8_e4m3fn
    return [st["k_codes"].view(f8), st["k_scales"], st["v_codes"].view(f8), st["v_scales"]]


def _gate_of(st, M, to):
    rows = _gate_rows(st["case"])
    if not rows:
        return None
    gate = st["gate"].to(to)
    return gate if rows == 1 else gate[:1] if rows >= M else \
        gate.repeat_interleave(rows, 0)[:M]


def _plain_block_fwd(st):
    c = st["case"]
    h, r, off, eps = st["h"].float(), st["r"].float(), c["offset"], st["eps"]
    dt = st["h"].dtype
    a = b = y = None
    if c["post"]:
        a = torch.rsqrt((h * h).mean(-1) + eps)
        h = h * a[:, None] * (off + st["w_post"].float())
    gate = _gate_of(st, c["M"], torch.float32)
    if gate is not None:
        h = h * gate
    s = c["beta"] * r + c["alpha"] * h
    if c["pre"]:
        b = torch.rsqrt((s * s).mean(-1) + eps)
        y = (s * b[:, None] * (off + st["w_pre"].float())).to(dt)
    return s.to(dt), y, a, b


def _group_sum(t, rows, M, N):
    """Sums of the rows of t that share a gate row."""
    G = -(-M // rows)
    if G * rows != M:
        t = torch.cat([t, t.new_zeros(G * rows - M, N)])
    return t.view(G, rows, N).sum(1)


def _plain_block_bwd(st):
    c, dt = st["case"], st["h"].dtype
    M, N, off = c["M"], c["N"], c["offset"]
    ds, h = st["ds"].float(), st["h"].float()
    out = {}
    if c["pre"]:
        s, b, dy = st["s"].float(), st["rstd_pre"][:, None], st["dy"].float()
        sb = s * b
        u = dy * (off + st["w_pre"].float())
        ds = ds + b * (u - sb * (u * sb).mean(-1, keepdim=True))
        out["dw_pre"] = (dy * sb).sum(0)
    m = c["alpha"] * ds
    n = h
    if c["post"]:
        a, w = st["rstd_post"][:, None], off + st["w_post"].float()
        xhat = h * a
        n = xhat * w
    gate = _gate_of(st, M, torch.float32)
    if gate is not None:
        out["dgate"] = _group_sum(m * n, _gate_rows(c), M, N).to(dt)
        m = m * gate
    if c["post"]:
        out["dw_post"] = (m * xhat).sum(0)
        u = m * w
        m = a * (u - xhat * (u * xhat).mean(-1, keepdim=True))
    out["dh"], out["dr"] = m.to(dt), (c["beta"] * ds).to(dt)
    return [out[k] for k in ("dh", "dr", "dgate", "dw_post", "dw_pre") if k in out]


def _cos_sin(st):
    angle = st["positions"].double()[:, None] * st["inv"]
    return (angle.cos() * st["mag"]).float()[:, None], (angle.sin() * st["mag"]).float()[:, None]


def _turn(x, cos, sin, R, interleaved):
    """The rotation of the first R values of each head (32-bit)."""
    if interleaved:
        x1, x2 = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    else:
        x1, x2 = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    return torch.cat([turned, x[..., R:]], -1) if R < x.shape[-1] else turned


def _plain_rope_fwd(st):
    c = st["case"]
    cos, sin = _cos_sin(st)
    out, kept = [], []
    for x, w in ((st["q"], st["w_q"]), (st["k"], st["w_k"])):
        f = x.float()
        if w is not None:
            a = torch.rsqrt((f * f).mean(-1) + st["eps"])
            kept.append(a)
            f = f * a[..., None] * (c["offset"] + w.float())
        out.append(_turn(f, cos, sin, c["R"], c["interleaved"]).to(x.dtype))
    return out + kept


def _plain_rope_bwd(st):
    c = st["case"]
    cos, sin = _cos_sin(st)
    out, dws = [], []
    for n in "qk":
        d = _turn(st["d" + n].float(), cos, -sin, c["R"], c["interleaved"])
        if c["norm"]:
            a, w = st["rstd_" + n][..., None], c["offset"] + st["w_" + n].float()
            xhat = st[n].float() * a
            dws.append((d * xhat).sum((0, 1)))
            u = d * w
            d = a * (u - xhat * (u * xhat).mean(-1, keepdim=True))
        out.append(d.to(st["d" + n].dtype))
    return out + dws


# The values of the 4-bit format's eight magnitudes, and the borders between
# them: a value on a border goes to the neighbour whose last bit is zero.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _plain_encode(x, fmt):
    """Codes and scale bytes of x[..., D]: groups of 32 values share the smallest
    power of two that brings the largest of them within the format."""
    f = x.float().unflatten(-1, (-1, 32))
    bits = f.abs().amax(-1).view(torch.int32)
    top, whole = (0x600000, 8) if fmt == "e4m3" else (0x400000, 2)
    e = ((bits >> 23) - whole + ((bits & 0x7FFFFF) > top).int()).clamp(0, 254)
    f = (f * ((254 - e) << 23).view(torch.float32)[..., None]).flatten(-2)
    if fmt == "e4m3":
        return f.to(torch.float8_e4m3fn).view(torch.uint8), e.to(torch.uint8)
    m, code = f.abs(), torch.zeros_like(f, dtype=torch.uint8)
    for i, border in enumerate(BORDERS):
        code += (m > border) if i % 2 == 0 else (m >= border)
    code += torch.signbit(f).to(torch.uint8) * 8
    return code[..., 0::2] | (code[..., 1::2] << 4), e.to(torch.uint8)


def _plain_decode(codes, scales, fmt, dt):
    if fmt == "e4m3":
        f = codes.view(torch.float8_e4m3fn).float()
    else:
        c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        f = torch.tensor(E2M1, device=codes.device)[(c & 7).long()]
        f = torch.where(c > 7, -f, f)
    e = scales.int()
    p = torch.where(e > 0, e << 23, 1 << 22).view(torch.float32)  # 2^(e - 127)
    return (f.unflatten(-1, (-1, 32)) * p[..., None]).flatten(-2).to(dt)


def _plain_cache_write(st):
    used = st["slots"] >= 0
    slots = st["slots"][used]
    for n in "kv":
        codes, scales = _plain_encode(st[n], st["case"]["fmt"])
        st[n + "_codes"].flatten(0, 1)[slots] = codes[used]
        st[n + "_scales"].flatten(0, 1)[slots] = scales[used]
    return _cache_values(st) if st["case"]["op"] == "cache_write" else None


def _plain_cache_read(st):
    c, rows, page = st["case"], st["rows"], st["case"]["page"]
    row = torch.arange(rows, device=st["cu"].device, dtype=torch.int32)
    seq = torch.searchsorted(st["cu"][1:].contiguous(), row, right=True)
    at = row - st["cu"][seq]
    slots = st["table"][seq, at // page].long() * page + at % page
    return [_plain_decode(st[n + "_codes"].flatten(0, 1)[slots],
                          st[n + "_scales"].flatten(0, 1)[slots], c["fmt"], DT[c["dtype"]])
            for n in "kv"]


def _plain_cache_trip(st):
    _plain_cache_write(st)
    return _plain_cache_read(st)


_PLAIN = {"block_fwd": lambda st: [t for t in _plain_block_fwd(st) if t is not None],
          "block_bwd": _plain_block_bwd, "rope_fwd": _plain_rope_fwd, "rope_bwd": _plain_rope_bwd,
          "cache_write": _plain_cache_write, "cache_read": _plain_cache_read,
          "cache_trip": _plain_cache_trip}


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    e = EB[case["dtype"]]
    op = case["op"]
    if op.startswith("block"):
        M, N = case["M"], case["N"]
        rows = _gate_rows(case)
        gate = e * N * -(-M // rows) if rows else 0
        norms = int(case["post"]) + int(case["pre"])
        if op == "block_fwd":
            arrays = 3 + int(case["pre"])
            return {"bytes": e * M * N * arrays + gate + norms * (e * N + 4 * M),
                    "flops": M * N * (3 + 5 * norms + bool(rows))}
        arrays = 3 + (2 if case["pre"] else 0) + int(case["post"] or bool(rows))
        return {"bytes": e * M * N * arrays + 2 * gate + norms * (e * N + 4 * N + 4 * M),
                "flops": M * N * (2 + 10 * norms + 3 * bool(rows))}
    if op.startswith("rope"):
        heads, D, T = case["hq"] + case["hk"], case["D"], case["T"]
        norm = int(case["norm"])
        arrays = 3 if norm and op == "rope_bwd" else 2
        n = T * heads
        return {"bytes": e * n * D * arrays + 8 * T + 4 * case["R"]
                + norm * (4 * n + 2 * e * D + (8 * D if op == "rope_bwd" else 0)),
                "flops": n * (3 * case["R"] + norm * (5 if op == "rope_fwd" else 10) * D)}
    heads, D = case["heads"], case["D"]
    held = _code_bytes(case) + D // 32
    if op == "cache_write":
        # about 5% of the tokens are padding, which nothing is read for
        n = case["T"] * heads * 2 * 95 // 100
        return {"bytes": n * (e * D + held) + 8 * case["T"], "flops": 3 * n * D}
    n = sum(_lengths(case)) * heads * 2
    if op == "cache_read":
        return {"bytes": n * (e * D + held), "flops": n * D}
    return {"bytes": 2 * n * (e * D + held), "flops": 4 * n * D}


# ---- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return _EXACT[case["op"]](case, st)


def _rms(x, eps):
    return torch.sqrt(torch.linalg.vector_norm(x, dim=-1).pow(2) / x.shape[-1] + eps)


def _exact_gate(case, st):
    rows = _gate_rows(case)
    if not rows:
        return None
    which = torch.arange(case["M"], device=st["h"].device) // rows
    return which, st["gate"].double()


def _exact_block_fwd(case, st):
    n, a, b, y = st["h"].double(), None, None, None
    if case["post"]:
        d = _rms(n, st["eps"])
        a, n = 1 / d, n / d[:, None] * (case["offset"] + st["w_post"].double())
    gate = _exact_gate(case, st)
    if gate is not None:
        n = n * gate[1][gate[0]]
    s = case["beta"] * st["r"].double() + case["alpha"] * n
    if case["pre"]:
        d = _rms(s, st["eps"])
        b, y = 1 / d, s / d[:, None] * (case["offset"] + st["w_pre"].double())
    return [t for t in (s, y, a, b) if t is not None]


def _norm_vjp(x, rstd, w, d):
    """Gradients of x * rstd * w for x (rstd depending on it) and w, given d."""
    r = rstd.double()[..., None]
    dx = r * w * d - x * r.pow(3) * (w * d * x).sum(-1, keepdim=True) / x.shape[-1]
    return dx, (d * x * r).flatten(0, -2).sum(0)


def _exact_block_bwd(case, st):
    ds, h = st["ds"].double(), st["h"].double()
    dgate = dw_post = dw_pre = None
    if case["pre"]:
        dx, dw_pre = _norm_vjp(st["s"].double(), st["rstd_pre"],
                               case["offset"] + st["w_pre"].double(), st["dy"].double())
        ds = ds + dx
    dn = case["alpha"] * ds
    w = case["offset"] + st["w_post"].double() if case["post"] else None
    gate = _exact_gate(case, st)
    if gate is not None:
        n = h * st["rstd_post"].double()[:, None] * w if case["post"] else h
        dgate = torch.zeros_like(gate[1]).index_add_(0, gate[0], dn * n)
        dn = dn * gate[1][gate[0]]
    if case["post"]:
        dn, dw_post = _norm_vjp(h, st["rstd_post"], w, dn)
    return [t for t in (dn, case["beta"] * ds, dgate, dw_post, dw_pre) if t is not None]


def _exact_turn(x, case, st, sign):
    """Pairs as complex numbers, turned by the angle of their position."""
    R = case["R"]
    angle = sign * st["positions"].double()[:, None, None] * st["inv"]
    mag = torch.full_like(angle, float(st["mag"]))
    head = x[..., :R]
    pairs = head.unflatten(-1, (R // 2, 2)) if case["interleaved"] else \
        head.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(mag, angle)
    pairs = torch.view_as_real(z)
    turned = pairs.flatten(-2) if case["interleaved"] else pairs.transpose(-1, -2).flatten(-2)
    return torch.cat([turned, x[..., R:]], -1)


def _exact_rope_fwd(case, st):
    outs, kept = [], []
    for n in "qk":
        x = st[n].double()
        if case["norm"]:
            d = _rms(x, st["eps"])
            kept.append(1 / d)
            x = x / d[..., None] * (case["offset"] + st["w_" + n].double())
        outs.append(_exact_turn(x, case, st, 1.0))
    return outs + kept


def _exact_rope_bwd(case, st):
    outs, dws = [], []
    for n in "qk":
        d = _exact_turn(st["d" + n].double(), case, st, -1.0)
        if case["norm"]:
            d, dw = _norm_vjp(st[n].double(), st["rstd_" + n],
                              case["offset"] + st["w_" + n].double(), d)
            dws.append(dw)
        outs.append(d)
    return outs + dws


def _by_two(x, e):
    """x * 2^e, the power made from its bits."""
    return x * ((e.long() + 1023) << 52).view(torch.float64)


def _exact_encode(x, fmt):
    """(values of the codes, scale bytes) by exponents and remainders in 64 bits."""
    f = x.double().unflatten(-1, (-1, 32))
    largest, low, bits = (448.0, -6, 3) if fmt == "e4m3" else (6.0, 0, 1)
    peak = f.abs().amax(-1)
    # the smallest power of two p with peak <= largest * p
    m, e = torch.frexp(peak / largest)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(peak == 0, torch.full_like(e, -127), e).clamp(min=-127)
    f = _by_two(f, -e[..., None])
    at = (torch.frexp(f)[1] - 1).clamp(min=low) - bits
    values = _by_two(torch.round(_by_two(f, -at)), at)
    return values, e


def _exact_cache_write(case, st):
    used = st["slots"] >= 0
    out = []
    for n in "kv":
        values, e = _exact_encode(st[n], case["fmt"])
        shape = st[n + "_codes"].shape[:3]
        full = torch.zeros(*shape, case["D"], dtype=torch.float64, device=DEV)
        full.flatten(0, 1)[st["slots"][used]] = values.flatten(-2)[used]
        scale = torch.zeros(*shape, case["D"] // 32, dtype=torch.uint8, device=DEV)
        scale.flatten(0, 1)[st["slots"][used]] = (e + 127).to(torch.uint8)[used]
        out += [full, scale]
    return out


def _exact_cache_read(case, st):
    if case["fmt"] == "e4m3":
        c = torch.arange(256, device=DEV)
        ex, m = (c >> 3) & 15, (c & 7).double()
        value = torch.where(ex == 0, m / 512, _by_two(1 + m / 8, ex - 7))
        value = torch.where(c >= 128, -value, value)
    else:
        value = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=DEV)
    out = []
    for n in "kv":
        codes = st[n + "_codes"].flatten(0, 1)[st["slots"]].long()
        if case["fmt"] == "e2m1":
            codes = torch.stack([codes % 16, codes // 16], -1).flatten(-2)
        e = st[n + "_scales"].flatten(0, 1)[st["slots"]].long() - 127
        out.append(_by_two(value[codes].unflatten(-1, (-1, 32)), e[..., None]).flatten(-2))
    return out


def _exact_cache_trip(case, st):
    out = []
    for n in "kv":
        values, e = _exact_encode(st[n], case["fmt"])
        out.append(_by_two(values, e[..., None]).flatten(-2))
    return out


_EXACT = {"block_fwd": _exact_block_fwd, "block_bwd": _exact_block_bwd,
          "rope_fwd": _exact_rope_fwd, "rope_bwd": _exact_rope_bwd,
          "cache_write": _exact_cache_write, "cache_read": _exact_cache_read,
          "cache_trip": _exact_cache_trip}
