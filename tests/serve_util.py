"""Plain 64-bit implementations of the operators that serve from the cache, written from the
formulas of include/rmsnorm.h, and the error bounds of their tests.

Bounds of attention. With S = scale * max over t of sum |q k| (the magnitude behind a
score), a score is off by at most about 32 roundings of fp32 sums, 32 * 2^-23 * S < 4e-6 * S; a
probability by that, the exponential's 2^-22 and its own rounding: half a step of fp16, which is
finfo.eps / 2 = 2^-11 (a step is 2^-10 in [1, 2)), for 16-bit outputs; for fp32 the rest of that, at most
2^-11, is rounded to fp16 again, so 2^-11 * 2^-11 = 2^-22. Sums by TAU, as for the other
operators. Numerator and denominator both carry the score's error, so an output is
within (r + 2 * (4e-6 * S + TAU)) * sum p |v| and half a step of its dtype.

Floor. A probability goes into the product in fp16 as p * 2^(b - B + 8), b the token's largest
scale byte (of a head) and B the largest so far; below 2^-14 its rounding is no
longer relative but half of fp16's smallest value, 2^-25. In v's units that is 2^-25 *
2^(B - 127 - 8) * |code| for a token, and the sum of p, which divides it, is at least 1 (the
maximum's own p). B is at most the largest byte of the sequence's tokens, so an output may be off by
2^-33 * 2^(largest byte - 127) * sum |code| over the tokens seen. It shows where the tokens of
large p have the code 0: (p 2^-23 beside a token of p 1 and code 0 keeps 10 bits).
v goes into it as code * 2^(group's byte - b + C), C = 6 for 8-bit codes (whose last bit is at least
2^-9) and 12 for 4-bit ones (2^-1): exact while the last bit is at least 2^-24, that is for groups within
2^21 (2^35) of the token's largest; below it is off by 2^-25, and groups beyond 2^-(C + 24) are
left out, which is at most 448 * 2^-31 < 2^-22 (6 * 2^-37 < 2^-34) of 2^(b - 127) for a token.
"""
from __future__ import annotations

import torch

import ops_util as U


def tokens_of(cache, which, pages, have):
    """The first `have` tokens behind a row of page numbers: [have, heads, D] in 64 bits on
    the CPU, and whether each token's page is there."""
    codes = getattr(cache, which + "_codes").cpu()
    scales = getattr(cache, which + "_scales").cpu()
    if cache.heads_first:
        codes, scales = codes.transpose(1, 2), scales.transpose(1, 2)
    t = torch.arange(have)
    col = t // cache.page_size
    there = col < len(pages)
    page = torch.where(there, torch.as_tensor(pages).long()[col.clamp(max=max(0, len(pages) - 1))], -1) \
        if len(pages) else torch.full_like(t, -1)
    there = (page >= 0) & (page < cache.pages)
    page = page.clamp(0, cache.pages - 1)
    c, s = codes[page, t % cache.page_size], scales[page, t % cache.page_size]
    code = U.unpack(c, cache.fmt, cache.head_dim).long()
    v = U.code_values(cache.fmt)[code]
    e = s.long()
    p = torch.pow(torch.tensor(2.0, dtype=torch.float64), (e - 127).double())
    p = torch.where(e == 255, torch.full_like(p, float("nan")), p)
    return v * p.repeat_interleave(32, -1)[..., :cache.head_dim], there


def codes_of(cache, pages, have):
    """|code| and scale of v's tokens behind a row of page numbers (NaN as 0), as tokens_of."""
    fake = B_like(cache)
    fake.v_scales = torch.full_like(cache.v_scales, 127)
    code, _ = tokens_of(fake, "v", pages, have)
    code = code.abs().nan_to_num(0.0)
    fake.v_codes = torch.full_like(cache.v_codes, 0x22 if cache.fmt == "e2m1" else 0x38)  # every code 1
    fake.v_scales = torch.where(cache.v_scales == 255, 0, cache.v_scales)
    scale, _ = tokens_of(fake, "v", pages, have)
    return code, scale


class B_like:
    """The fields of a cache that tokens_of reads."""

    def __init__(self, cache):
        self.__dict__.update({n: getattr(cache, n) for n in (
            "k_codes", "k_scales", "v_codes", "v_scales", "heads_first", "page_size", "pages", "fmt", "head_dim")})


def attention(cache, q, table, lengths, cu, scale, causal, window):
    """out, lse, the magnitudes (sum p |v|, S) and the floor in 64 bits on the CPU."""
    q = q.double().cpu()
    rows, H, D = q.shape
    G = H // cache.heads
    out, mag = torch.zeros(rows, H, D, dtype=torch.float64), torch.zeros(rows, H, D, dtype=torch.float64)
    lse = torch.full((rows, H), -float("inf"), dtype=torch.float64)
    S, floor = torch.zeros(rows, H, dtype=torch.float64), torch.zeros(rows, H, D, dtype=torch.float64)
    for b, have in enumerate(lengths):
        n = cu[b + 1] - cu[b]
        if n == 0 or have <= 0:
            continue
        k, there = tokens_of(cache, "k", table[b], have)
        v, _ = tokens_of(cache, "v", table[b], have)
        code, scale_v = codes_of(cache, table[b], have)
        largest = (scale_v * there[:, None, None]).amax(0)
        t, rows_b = torch.arange(have), slice(cu[b], cu[b + 1])
        pos = have - n + torch.arange(n)
        see = there[None].expand(n, have).clone()
        if causal:
            see &= t[None] <= pos[:, None]
        if window:
            see &= t[None] > pos[:, None] - window
        some = see.any(-1)
        seen = see.double()
        for h in range(H):
            kk, vv, cc, qq = k[:, h // G], v[:, h // G], code[:, h // G], q[rows_b, h]
            # a score that is not a number where it is seen makes the row so
            s = torch.where(see, scale * (qq @ kk.nan_to_num(0.0).T), -torch.inf)
            lost = (see & torch.isnan(kk).any(-1)[None]).any(-1)
            z = torch.logsumexp(s, -1)
            p = torch.where(see, torch.exp(s - z[:, None].nan_to_num(neginf=0.0)), 0.0)
            o = p @ vv.nan_to_num(0.0)
            o[(seen @ torch.isnan(vv).double()) > 0] = torch.nan
            o[lost], z[lost] = torch.nan, torch.nan
            out[rows_b, h], lse[rows_b, h] = torch.where(some[:, None], o, 0.0), z
            mag[rows_b, h] = p @ vv.nan_to_num(0.0).abs()
            top = scale_v[:, h // G].amax(-1, keepdim=True)
            far = top * (scale_v[:, h // G] * 2.0 ** (21 if cache.fmt == "e4m3" else 35) < top)
            floor[rows_b, h] = 2.0 ** -33 * largest[h // G].amax() * (seen @ cc) + \
                2.0 ** (-22 if cache.fmt == "e4m3" else -34) * (p @ far)
            big = (scale * (qq.abs() @ kk.nan_to_num(0.0).abs().T)).abs()
            S[rows_b, h] = torch.where(see, big, 0.0).amax(-1)
    return out, lse, mag, S, floor


def check_attention(got, lse, want, dtype, what):
    out, ref_lse, mag, S, floor = want
    got = got.double().cpu()
    assert got.shape == out.shape, what
    r = 2.0 ** -22 if dtype is torch.float32 else torch.finfo(torch.float16).eps / 2
    bad = torch.isnan(out)
    assert torch.equal(torch.isnan(got), bad), (what, "NaN elsewhere", int(torch.isnan(got).sum()), int(bad.sum()))
    delta = 4e-6 * S + U.TAU
    bound = (r + 2 * delta)[..., None] * mag + U.half_step(out, dtype) + floor
    err = torch.where(bad, 0.0, (got - out).abs())
    # past the type's largest value by half a step (65520 in fp16) a result is rounded to infinity
    top = torch.finfo(dtype).max
    past = torch.isinf(got) & (got.sign() == out.sign()) & (out.abs() + bound >= top * (1 + torch.finfo(dtype).eps / 4))
    ok = bad | past | (err <= bound)
    assert bool(ok.all()), (what, float((err / bound).nan_to_num(0).max()), int((~ok).sum()))
    if lse is not None:
        got = lse.double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref_lse)), (what, "lse NaN")
        assert torch.equal(got == -float("inf"), ref_lse == -float("inf")), (what, "lse of empty rows")
        fine = torch.isfinite(ref_lse)
        err = (got - ref_lse)[fine].abs()
        assert bool((err <= (delta + 2.0 ** -22 * ref_lse.abs())[fine]).all()), (what, float(err.max()))


# ---- pages ------------------------------------------------------------------------

def arrays(cache):
    return [t.cpu().clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)
            if t is not None]


def fork(cache, refs, table, lengths, parents, children):
    """The state after a fork (lists, in place), the cache's arrays, and whether anything was
    reported."""
    page, S, W = cache.page_size, len(table), len(table[0]) if table else 0
    old, out = arrays(cache), arrays(cache)
    before = list(lengths)
    free = [p for p in range(len(refs)) if refs[p] <= 0]
    named, reported = set(), False
    rows0 = [list(r) for r in table]
    for a, c in zip(parents, children):
        if a < 0 or c < 0:
            continue
        if a >= S or c >= S or a == c or before[c] != 0 or c in named or before[a] < 0 or \
                -(-before[a] // page) > W:
            reported = True
            if c < S:
                named.add(c)
            continue
        named.add(c)
        full, rest = divmod(before[a], page)
        row = rows0[a][:full]
        if rest:
            if not free:
                reported = True
                continue
            new, src = free.pop(0), rows0[a][full]
            row = row + [new]
            if not 0 <= src < cache.pages:
                reported = True
            else:
                for o, t in zip(out, old):
                    if cache.heads_first:
                        o[new, :, :rest] = t[src, :, :rest]
                    else:
                        o[new, :rest] = t[src, :rest]
        for p in row:
            if 0 <= p < cache.pages:
                refs[p] += 1
            else:
                reported = True
        table[c] = row + [-1] * (W - len(row))
        lengths[c] = before[a]
    return out, reported


def compact(cache, refs, table):
    """live, refs, table after compaction, the cache's arrays, whether anything was reported."""
    P = len(refs)
    live = sum(r > 0 for r in refs)
    src = [p for p in range(live, P) if refs[p] > 0]
    dst = [p for p in range(live) if refs[p] <= 0]
    out, old = arrays(cache), arrays(cache)
    new, to = list(refs), {}
    for s, d in zip(src, dst):
        to[s] = d
        new[d], new[s] = refs[s], 0
        for o, t in zip(out, old):
            o[d] = t[s]
    return live, new, [[to.get(p, p) for p in r] for r in table], out, any(p >= P for r in table for p in r)
