"""The operators that serve a model from the quantised cache: what is measured of them.

Three operators, each with the calls that belong to it:

attn    attention of ragged queries over the paged cache of k and v in 4 or 8 bits,
        by page table: a token a sequence, a few, or a prompt's chunk
pages   pages of the cache copied, forked with copy on write, freed and compacted
axes    rotary positions with several axes (time, height, width), behind the heads'
        RMSNorm, forward and backward

`run` computes a case in elementary torch operations (in 32 bits, angles in 64), or,
where `own` is true, by the calls of this package. `exact` computes the same from the
definitions in 64 bits.
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
        # A chat server with few users: one decoding step of four short sequences.
        dict(name="attn_decode_few", op="attn", B=4, q=1, longest=509, hk=8, group=4, D=128,
             fmt="e2m1", dtype="bf16", page=16, window=0, causal=True, heads_first=False, lse=False),
        # One decoding step of a full server: 32 sequences of up to 8192 tokens, 4 bits.
        dict(name="attn_decode_long", op="attn", B=32, q=1, longest=8192, hk=8, group=4, D=128,
             fmt="e2m1", dtype="bf16", page=16, window=0, causal=True, heads_first=False, lse=False),
        # Two very long contexts of a model with one key head for 16 query heads, in 8 bits.
        dict(name="attn_decode_one_head", op="attn", B=2, q=1, longest=131072, hk=1, group=16, D=256,
             fmt="e4m3", dtype="bf16", page=64, window=0, causal=True, heads_first=False, lse=True),
        # Drafted tokens checked: five queries a sequence, odd pages, heads first, a window.
        dict(name="attn_verify_window", op="attn", B=17, q=5, longest=4099, hk=5, group=4, D=96,
             fmt="e2m1", dtype="fp16", page=24, window=1000, causal=True, heads_first=True, lse=False),
        # Chunks of three prompts behind what the cache holds already: the most arithmetic.
        dict(name="attn_prompt_chunk", op="attn", B=3, q=2048, longest=8192, hk=8, group=4, D=128,
             fmt="e2m1", dtype="bf16", page=16, window=0, causal=True, heads_first=False, lse=False),
        # Sampling several answers to a prompt: every finished answer's row is freed and
        # forked again from its prompt, whose last page is half full.
        dict(name="pages_fork", op="fork", parents=8, children=56, longest=2000, heads=8, D=128,
             fmt="e2m1", page=16, heads_first=False),
        # Prefixes copied page by page, 4 bits, to where another batch owns them.
        dict(name="pages_copy", op="copy", pages=16384, n=6000, heads=8, D=128, fmt="e2m1", page=16,
             heads_first=False),
        # A worn cache brought together before its tail is given back: a third is in use.
        dict(name="pages_compact", op="compact", pages=16384, rows=96, used=5500, shared=16, heads=8,
             D=128, fmt="e4m3", page=16, heads_first=False),
        # A small cache of odd pages, heads first: latency.
        dict(name="pages_compact_small", op="compact", pages=301, rows=9, used=97, shared=3, heads=5,
             D=96, fmt="e2m1", page=24, heads_first=True),
        # One decoding step of 64 sequences behind images: three axes, head norms.
        dict(name="axes_fwd_decode", op="axes_fwd", T=64, hq=32, hk=8, D=128, R=128, axes=3,
             first=16, in_turn=False, separate=False, interleaved=False, dtype="bf16", norm=True,
             offset=0.0, far=131072),
        # A video's tokens: the axes take the pairs in turn, no head norms.
        dict(name="axes_fwd_video", op="axes_fwd", T=16384, hq=32, hk=8, D=128, R=128, axes=3,
             first=24, in_turn=True, separate=False, interleaved=False, dtype="bf16", norm=False,
             offset=0.0, far=32768),
        # Training on video: three axes with frequencies of their own, pairs side by side, head
        # norms of q and k, the backward pass.
        dict(name="axes_bwd_train", op="axes_bwd", T=16381, hq=24, hk=24, D=128, R=128, axes=3,
             first=22, in_turn=False, separate=True, interleaved=True, dtype="bf16", norm=True,
             offset=0.0, far=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn", "fork", "copy", "compact", "axes_fwd", "axes_bwd"])
    D = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    if op == "attn":
        hk, group = rng.choice([1, 2, 4, 5, 8, 8]), rng.choice([1, 2, 4, 4, 7, 8, 16])
        q = rng.choice([1, 1, 1, _log(rng, 2, 8), _log(rng, 9, 2048)])
        # No more products of queries and keys than the prompts' chunks have, and no more
        # of keys and values than the full server.
        most = min(18_000_000 * 4096 // (q * hk * group * D), 32 * 8192 * 8 * 128 // (hk * D))
        longest = min(_log(rng, max(q, 2), 32768), most)
        B = min(_log(rng, 1, 128), most // longest)
        causal = rng.random() < 0.85
        return dict(op=op, B=B, q=q, longest=longest, hk=hk, group=group, D=D,
                    fmt=rng.choice(["e2m1", "e2m1", "e4m3"]), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    page=rng.choice([1, 8, 16, 16, 24, 32, 64]),
                    window=_log(rng, 16, 4096) if causal and rng.random() < 0.25 else 0, causal=causal,
                    heads_first=rng.random() < 0.3, lse=rng.random() < 0.3)
    if op.startswith("axes"):
        hk = rng.choice([1, 2, 4, 5, 8])
        hq = hk * rng.choice([1, 2, 4, 7])
        R = rng.choice([D, D, D // 2])
        axes = rng.choice([2, 3, 3, 4])
        in_turn = rng.random() < 0.4
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        T = min(_log(rng, 1, 32768), 16381 * 48 * 128 * 2 // ((hq + hk) * D * EB[dtype]))
        rest = R // 2 // axes
        return dict(op=op, T=T, hq=hq, hk=hk, D=D, R=R, axes=axes,
                    first=R // 2 - (axes - 1) * (rest - rng.randrange(rest // 2)), in_turn=in_turn,
                    separate=not in_turn and rng.random() < 0.5, interleaved=rng.random() < 0.5,
                    dtype=dtype, norm=rng.random() < 0.6, offset=float(rng.randrange(2)),
                    far=_log(rng, 512, 1 << 20))
    case = dict(op=op, heads=rng.choice([1, 2, 4, 5, 8]), D=D, fmt=rng.choice(["e2m1", "e4m3"]),
                page=rng.choice([1, 8, 16, 16, 24, 64]), heads_first=rng.random() < 0.3)
    token = case["heads"] * D * (2 if case["fmt"] == "e4m3" else 1)
    if op == "fork":
        case["parents"] = _log(rng, 1, 32)
        case["longest"] = _log(rng, 1, 8192)
        case["children"] = _log(rng, 1, 512)
        return case
    pages = max(4, min(_log(rng, 16, 65536), 16384 * 16 * 2048 // (case["page"] * token)))
    case["pages"] = pages
    if op == "copy":
        case["n"] = rng.randint(1, pages // 2)
    else:
        case["used"] = rng.randint(1, pages - 1)
        case["rows"] = _log(rng, 1, 200)
        case["shared"] = rng.randint(0, case["rows"])
    return case


# ---- inputs ----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = _PREPARE[case["op"]](case, g)
    st["case"] = case
    if own:
        from memory_bound_normalization_fwd_gb300 import binding
        st["B"] = binding
        if "k_codes" in st:
            pages, heads, D = st["k_codes"].shape[0], case.get("hk", case.get("heads")), case["D"]
            st["cache"] = binding.Cache(pages, case["page"], heads, D, fmt=case["fmt"],
                                        heads_first=case["heads_first"], tensors=_arrays(st))
        else:
            st["layout"] = binding.RopeAxes(_pairs(case), in_turn=case["in_turn"])
            st["steps"], st["mag"] = binding.rope_steps(
                case["R"], base=10000.0, device=DEV, axes=st["layout"] if case["separate"] else None)
    return st


def _arrays(st):
    return st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"]


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


# The values of the 4-bit format's eight magnitudes, and the borders between them.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _groups(D):
    return -(-D // 32)


def _code_bytes(case):
    return case["D"] if case["fmt"] == "e4m3" else case["D"] // 2


def _encoded(x, fmt):
    """Codes and scale bytes of x[..., D], as the cache holds them."""
    D = x.shape[-1]
    f = torch.nn.functional.pad(x, (0, _groups(D) * 32 - D)).unflatten(-1, (-1, 32))
    peak = f.abs().amax(-1).clamp(min=1e-30)
    e = torch.ceil(torch.log2(peak / (448.0 if fmt == "e4m3" else 6.0)))
    f = (f * torch.exp2(-e)[..., None]).flatten(-2)[..., :D]
    e = (e + 127).to(torch.uint8)
    if fmt == "e4m3":
        return f.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), e
    code = torch.bucketize(f.abs(), torch.tensor(BORDERS, device=DEV)).to(torch.uint8)
    code += torch.signbit(f).to(torch.uint8) * 8
    return code[..., 0::2] | (code[..., 1::2] << 4), e


def _cache_of(case, g, pages, heads, held=None):
    """The four arrays of a cache of `pages` pages. Slots beside `held` keep what
    a freed sequence left behind: any codes, scales of groups that were NaN."""
    D, page, st = case["D"], case["page"], {}
    for n in "kv":
        x = _randn(g, pages * page, heads, D)
        if n == "k":
            x[..., ::32] *= 8  # keys have a few channels far above the rest
        codes, scales = _encoded(x, case["fmt"])
        if held is not None:
            free = torch.ones(pages * page, dtype=torch.bool, device=DEV)
            free[held] = False
            scales[free] = 255
        for name, t in (("_codes", codes), ("_scales", scales)):
            t = t.unflatten(0, (pages, page))
            st[n + name] = (t.transpose(1, 2) if case["heads_first"] else t).contiguous()
    return st


def _lengths(case):
    """(tokens held, queries) of each sequence: the same for every seed, one of them the
    longest; one sequence in twelve is empty."""
    rng = random.Random(case["B"] * 65537 + case["longest"])
    held = [0 if rng.random() < 1 / 12 else rng.randint(case["longest"] // 8, case["longest"])
            for _ in range(case["B"])]
    held[case["B"] // 2] = case["longest"]
    queries = [case["q"] if case["q"] <= 8 else rng.randint(case["q"] // 2, case["q"]) for _ in held]
    return held, queries


def _prepare_attn(case, g):
    held, queries = _lengths(case)
    B, page, hq, dt = case["B"], case["page"], case["hk"] * case["group"], DT[case["dtype"]]
    lens = torch.tensor(held, device=DEV)
    width = -(-case["longest"] // page) + 1
    need = -(-lens // page)
    used = int(need.sum())
    pages = used + 3
    # Pages in any order; entries behind a sequence's last page name none.
    col = torch.arange(width, device=DEV)
    has = col < need[:, None]
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[has] = torch.randperm(pages, generator=g, device=DEV)[:used].to(torch.int32)
    at = torch.arange(width * page, device=DEV)
    slots = table.long().repeat_interleave(page, 1) * page + at % page
    st = _cache_of(case, g, pages, case["hk"], slots[at < lens[:, None]])
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.tensor(queries, device=DEV).cumsum(0)
    rows = sum(queries)
    # q is a slice of one projection's rows, with k and v behind it.
    qkv = _randn(g, rows, hq + 2 * case["hk"], case["D"], dtype=dt)
    st.update(q=qkv[:, :hq], table=table, lengths=lens.to(torch.int32), cu=cu)
    return st


def _table_of(case, g, rows, width, per_row, pages):
    """Rows of a table with `per_row` pages each, drawn from a permutation of all pages."""
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    has = torch.arange(width, device=DEV) < per_row[:, None]
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table[has] = order[:int(per_row.sum())]
    return table


def _counts(table, pages):
    named = table[table >= 0].long()
    return torch.bincount(named, minlength=pages).to(torch.int32)


def _prepare_fork(case, g):
    P, C, page = case["parents"], case["children"], case["page"]
    rng = random.Random(P * 65537 + case["longest"])
    held = torch.tensor([case["longest"]] + [rng.randint(0, case["longest"]) for _ in range(P - 1)],
                        device=DEV)
    need = -(-held // page)
    width = -(-case["longest"] // page) + 2
    pages = int(need.sum()) + C + 5
    table = torch.full((P + C, width), -1, dtype=torch.int32, device=DEV)
    table[:P] = _table_of(case, g, P, width, need, pages)
    st = _cache_of(case, g, pages, case["heads"])
    lengths = torch.zeros(P + C, dtype=torch.int32, device=DEV)
    lengths[:P] = held
    st.update(table=table, lengths=lengths, refs=_counts(table, pages),
              children=(P + torch.randperm(C, generator=g, device=DEV)).to(torch.int32),
              parents=torch.randint(0, P, (C,), generator=g, device=DEV, dtype=torch.int32))
    return st


def _prepare_copy(case, g):
    st = _cache_of(case, g, case["pages"], case["heads"])
    order = torch.randperm(case["pages"], generator=g, device=DEV).to(torch.int32)
    src, dst = order[:case["n"]].clone(), order[case["n"]:2 * case["n"]].clone()
    src[torch.rand(case["n"], generator=g, device=DEV) < 0.03] = -1  # nothing to copy
    st.update(src=src, dst=dst)
    return st


def _prepare_compact(case, g):
    rows, used, pages = case["rows"], case["used"], case["pages"]
    cuts = sorted(random.Random(pages * 257 + rows).choices(range(used + 1), k=rows - 1))
    per_row = torch.diff(torch.tensor([0] + cuts + [used], device=DEV))
    width = int(per_row.max()) + 1
    table = _table_of(case, g, rows, width, per_row, pages)
    table = torch.cat([table, table[:case["shared"]]])  # sequences that share pages
    st = _cache_of(case, g, pages, case["heads"])
    st.update(table=table, refs=_counts(table, pages))
    return st


def _pairs(case):
    """Pairs of each axis: the first has its own number, the others share the rest."""
    rest = case["R"] // 2 - case["first"]
    others = case["axes"] - 1
    return (case["first"],) + tuple(rest // others + (i < rest % others) for i in range(others))


def _axis_of(case):
    """The axis of each pair: consecutive pairs, or pair i on axis i modulo the axes
    while that one has pairs left, and on the first otherwise."""
    pairs, n = _pairs(case), case["axes"]
    if case["in_turn"]:
        return [i % n if i // n < pairs[i % n] else 0 for i in range(case["R"] // 2)]
    return [a for a in range(n) for _ in range(pairs[a])]


def _frequencies(case):
    """Radians per position of each pair (64-bit, Python floats)."""
    if case["separate"]:
        return [10000.0 ** (-i / n) for n in _pairs(case) for i in range(n)]
    return [10000.0 ** (-2.0 * i / case["R"]) for i in range(case["R"] // 2)]


def _weight(g, n, offset, dtype):
    w = 0.5 + torch.rand(n, generator=g, device=DEV) if offset == 0.0 else \
        0.3 * torch.randn(n, generator=g, device=DEV)
    return w.to(dtype)


def _prepare_axes(case, g):
    T, hq, hk, D, dt = case["T"], case["hq"], case["hk"], case["D"], DT[case["dtype"]]
    qkv = _randn(g, T, hq + 2 * hk, D, dtype=dt)
    st = dict(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], eps=1e-6, mag=1.0)
    if T <= 256:  # decoding: every sequence somewhere behind its images
        pos = torch.randint(0, case["far"], (case["axes"], T), generator=g, device=DEV)
    else:  # frames of 24 x 40 patches behind some text
        start = torch.randint(0, case["far"] // 4, (1,), generator=g, device=DEV)
        i = torch.arange(T, device=DEV)
        pos = start + torch.stack([i // 960, i % 960 // 40, i % 40, i % 7][:case["axes"]])
    st["positions"] = pos
    st["w_q"] = _weight(g, D, case["offset"], dt) if case["norm"] else None
    st["w_k"] = _weight(g, D, case["offset"], dt) if case["norm"] else None
    st["inv"] = torch.tensor(_frequencies(case), dtype=torch.float64, device=DEV)
    st["axis"] = torch.tensor(_axis_of(case), device=DEV)
    if case["op"] == "axes_bwd":
        st["dq"] = _randn(g, T, hq, D, dtype=dt)
        st["dk"] = _randn(g, T, hk, D, dtype=dt)
        if case["norm"]:
            st["rstd_q"] = torch.rsqrt(st["q"].float().square().mean(-1) + 1e-6)
            st["rstd_k"] = torch.rsqrt(st["k"].float().square().mean(-1) + 1e-6)
    return st


_PREPARE = {"attn": _prepare_attn, "fork": _prepare_fork, "copy": _prepare_copy,
            "compact": _prepare_compact, "axes_fwd": _prepare_axes, "axes_bwd": _prepare_axes}


# ---- one pass --------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return _own(op, state) if own else _PLAIN[op](state)


def _own(op, st):
    B, c = st["B"], st["case"]
    if op == "attn":
        out, lse = B.cache_attention(st["cache"], st["q"], st["table"], st["lengths"], cu_q=st["cu"],
                                     causal=c["causal"], window=c["window"], lse=c["lse"])
        return [out, lse] if c["lse"] else [out]
    if op == "copy":
        B.cache_copy_pages(st["cache"], st["src"], st["dst"])
        return _values(st)
    if op == "fork":
        B.cache_free(st["refs"], st["table"], st["lengths"], st["children"])
        B.cache_fork(st["cache"], st["refs"], st["table"], st["lengths"], st["parents"], st["children"])
        return _values(st) + [st["refs"], st["table"], st["lengths"]]
    if op == "compact":
        live, refs, table = B.cache_compact(st["cache"], st["refs"], st["table"])
        return _values(st) + [live, refs, table]
    how = dict(positions=st["positions"], w_q=st["w_q"], w_k=st["w_k"], axes=st["layout"],
               interleaved=c["interleaved"], offset=c["offset"], magnitude=st["mag"])
    if op == "axes_fwd":
        got = B.rope_fwd(st["q"], st["k"], st["steps"], eps=st["eps"], **how)
    elif c["norm"]:
        got = B.rope_bwd(st["dq"], st["dk"], st["steps"], q=st["q"], k=st["k"], rstd_q=st["rstd_q"],
                         rstd_k=st["rstd_k"], **how)
    else:
        got = B.rope_bwd(st["dq"], st["dk"], st["steps"], **how)
    return [t for t in got if t is not None]


def _values(st):
    """The cache after the call (codes of 8 bits are read as what they stand for)."""
    if st["case"]["fmt"] == "e2m1":
        return list(_arrays(st))
    f8 = torch.float8_e4m3fn
    return [st["k_codes"].view(f8), st["k_scales"], st["v_codes"].view(f8), st["v_scales"]]


def _by_slot(st, name):
    """A cache array as [slots, heads, ...]."""
    t = st[name]
    return (t.transpose(1, 2) if st["case"]["heads_first"] else t).flatten(0, 1)


def _decoded(codes, scales, c):
    if c["fmt"] == "e4m3":
        f = codes.view(torch.float8_e4m3fn).float()
    else:
        i = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        f = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)[i.int()]
    return f * torch.exp2(scales.float() - 127).repeat_interleave(32, -1)[..., :c["D"]]


def _plain_attn(st):
    c, page = st["case"], st["case"]["page"]
    B, hk, G, D = c["B"], c["hk"], c["group"], c["D"]
    lens, cu = st["lengths"].long(), st["cu"].long()
    n = cu.diff()
    # every sequence's tokens side by side, up to the longest
    t = torch.arange(c["longest"], device=lens.device)
    held = t < lens[:, None]
    slots = torch.where(held, st["table"].long()[:, t // page] * page + t % page, 0)
    kv = [_decoded(_by_slot(st, x + "_codes")[slots], _by_slot(st, x + "_scales")[slots], c)
          .masked_fill_(~held[..., None, None], 0.0).permute(0, 2, 1, 3) for x in "kv"]
    # and its queries, up to the most: [B, hk, q * G, D]
    i = torch.arange(c["q"], device=lens.device)
    row = torch.where(i < n[:, None], cu[:-1, None] + i, 0)
    q = st["q"][row].float().unflatten(2, (hk, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = (q @ kv[0].transpose(-1, -2)) * D ** -0.5
    pos = (lens - n)[:, None] + i
    sees = held[:, None]
    if c["causal"]:
        sees = sees & (t <= pos[..., None])
    if c["window"]:
        sees = sees & (t > pos[..., None] - c["window"])
    sees = sees.expand(B, c["q"], -1).repeat_interleave(G, 1)[:, None]
    s.masked_fill_(~sees, float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s.sub_(m))
    z = p.sum(-1, keepdim=True)
    o = (p @ kv[1]) / torch.where(z > 0, z, 1.0)
    # back to the rows
    seq = torch.searchsorted(cu[1:].contiguous(), torch.arange(len(st["q"]), device=lens.device), right=True)
    at = torch.arange(len(st["q"]), device=lens.device) - cu[seq]

    def rows(x):
        return x.unflatten(2, (c["q"], G)).permute(0, 2, 1, 3, 4)[seq, at].flatten(1, 2)

    out = rows(o).to(st["q"].dtype)
    return [out, rows(m + torch.log(z))[..., 0]] if c["lse"] else [out]


def _plain_copy(st):
    some = st["src"] >= 0
    src, dst = st["src"][some].long(), st["dst"][some].long()
    for t in _arrays(st):
        t[dst] = t[src]
    return _values(st)


def _plain_fork(st):
    c, page = st["case"], st["case"]["page"]
    refs, table, lengths = st["refs"], st["table"], st["lengths"]
    children, parents = st["children"].long(), st["parents"].long()
    # the children's rows are freed
    named = table[children]
    refs.index_add_(0, named.clamp(min=0).flatten().long(), -(named >= 0).int().flatten())
    table[children] = -1
    lengths[children] = 0
    # full pages are shared, the last one is copied into the lowest free ones
    have = lengths[parents].long()
    part = have % page > 0
    lowest = torch.argsort((refs > 0).int(), stable=True)
    fresh = lowest[(part.cumsum(0) - 1).clamp(min=0)].to(torch.int32)
    col = torch.arange(table.shape[1], device=table.device)
    full = (have // page)[:, None]
    rows = torch.where(col < full, table[parents], -1)
    rows = torch.where((col == full) & part[:, None], fresh[:, None], rows)
    old = table[parents].gather(1, full)[:, 0]
    table[children] = rows
    lengths[children] = lengths[parents]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).int().flatten())
    src, dst = old[part].long(), fresh[part].long()
    mine = torch.arange(page, device=table.device) < (have % page)[part][:, None]
    mine = mine[:, None, :, None] if c["heads_first"] else mine[:, :, None, None]
    for t in _arrays(st):
        t[dst] = torch.where(mine, t[src], t[dst])
    return _values(st) + [refs, table, lengths]


def _plain_compact(st):
    refs, table = st["refs"], st["table"]
    used = refs > 0
    live = used.sum()
    p = torch.arange(len(refs), device=refs.device)
    src = torch.nonzero(used & (p >= live))[:, 0]
    dst = torch.nonzero(~used & (p < live))[:, 0]
    for t in _arrays(st):
        t[dst] = t[src]
    to = p.clone()
    to[src] = dst
    out = torch.zeros_like(refs)
    out[to[used]] = refs[used]
    moved = torch.where(table >= 0, to[table.clamp(min=0).long()], -1).to(torch.int32)
    return _values(st) + [live[None].to(torch.int32), out, moved]


def _turn(x, cos, sin, R, interleaved):
    """The rotation of the first R values of each head (32-bit)."""
    if interleaved:
        x1, x2 = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    else:
        x1, x2 = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    return torch.cat([turned, x[..., R:]], -1) if R < x.shape[-1] else turned


def _cos_sin(st):
    angle = st["positions"].double()[st["axis"]].T * st["inv"]
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _plain_axes_fwd(st):
    c = st["case"]
    cos, sin = _cos_sin(st)

    def one(x, w):
        f, a = x.float(), []
        if w is not None:
            a = [torch.rsqrt((f * f).mean(-1) + st["eps"])]
            f = f * a[0][..., None] * (c["offset"] + w.float())
        return [_turn(f, cos, sin, c["R"], c["interleaved"]).to(x.dtype)], a

    (q, a), (k, b) = one(st["q"], st["w_q"]), one(st["k"], st["w_k"])
    return q + k + a + b


def _plain_axes_bwd(st):
    c = st["case"]
    cos, sin = _cos_sin(st)

    def one(n):
        d, dw = _turn(st["d" + n].float(), cos, -sin, c["R"], c["interleaved"]), []
        if c["norm"]:
            a, w = st["rstd_" + n][..., None], c["offset"] + st["w_" + n].float()
            xhat = st[n].float() * a
            dw = [(d * xhat).sum((0, 1))]
            u = d * w
            d = a * (u - xhat * (u * xhat).mean(-1, keepdim=True))
        return [d.to(st["d" + n].dtype)], dw

    (dq, dwq), (dk, dwk) = one("q"), one("k")
    return dq + dk + dwq + dwk


_PLAIN = {"attn": _plain_attn, "copy": _plain_copy, "fork": _plain_fork, "compact": _plain_compact,
          "axes_fwd": _plain_axes_fwd, "axes_bwd": _plain_axes_bwd}


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    return _WORK[case["op"]](case)


def _token_bytes(case, heads):
    """Codes and scales of k and v of a token."""
    return 2 * heads * (_code_bytes(case) + _groups(case["D"]))


def _work_attn(case):
    held, queries = _lengths(case)
    hq, e, read, pairs = case["hk"] * case["group"], EB[case["dtype"]], 0, 0
    for have, n in zip(held, queries):
        low, seen = have, 0
        for p in range(have - n, have):  # a query's position
            last = p if case["causal"] else have - 1
            first = max(0, p - case["window"] + 1) if case["window"] else 0
            if last >= first:
                pairs += last - first + 1
                low, seen = min(low, first), max(seen, last + 1)
        read += max(0, seen - low)
    rows = sum(queries)
    return {"bytes": read * _token_bytes(case, case["hk"]) + 2 * rows * hq * case["D"] * e
            + 4 * (read // case["page"]) + 4 * rows * hq * case["lse"],
            "flops": 4 * pairs * hq * case["D"]}


def _work_pages(case):
    page = case["page"] * _token_bytes(case, case["heads"])
    if case["op"] == "copy":
        n = case["n"] * 97 // 100
        return {"bytes": 2 * n * page + 8 * n, "flops": n}
    if case["op"] == "fork":
        # half a page for each child, its row, and the counts
        entries = case["children"] * (case["longest"] // case["page"] // 2 + 1)
        return {"bytes": case["children"] * page + 24 * entries, "flops": entries}
    moved = case["used"] * (case["pages"] - case["used"]) // case["pages"]
    entries = case["used"] + 4 * case["rows"]
    return {"bytes": 2 * moved * page + 8 * case["pages"] + 8 * entries, "flops": entries}


def _work_axes(case):
    e, heads, D = EB[case["dtype"]], case["hq"] + case["hk"], case["D"]
    norm, fwd, n = int(case["norm"]), case["op"] == "axes_fwd", case["T"] * (case["hq"] + case["hk"])
    return {"bytes": e * n * D * (2 if fwd or not norm else 3) + 8 * case["axes"] * case["T"]
            + 4 * case["R"] + norm * (4 * n + 2 * e * D + (0 if fwd else 8 * D)),
            "flops": n * (3 * case["R"] + norm * (5 if fwd else 10) * D)}


_WORK = {"attn": _work_attn, "fork": _work_pages, "copy": _work_pages, "compact": _work_pages,
         "axes_fwd": _work_axes, "axes_bwd": _work_axes}


# ---- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _by_two(x, e):
    """x * 2^e, the power made from its bits."""
    return x * ((e.long() + 1023) << 52).view(torch.float64)


def _exact_tokens(case, st, n, pages, have):
    """The first `have` tokens behind a row of the table: [have, heads, D]."""
    at = torch.arange(have, device=DEV)
    codes, scales = st[n + "_codes"], st[n + "_scales"]
    if case["heads_first"]:
        codes, scales = codes.movedim(1, 2), scales.movedim(1, 2)
    where = pages[at // case["page"]].long(), at % case["page"]
    c, e = codes[where].long(), scales[where].long() - 127
    if case["fmt"] == "e2m1":
        c = torch.stack([c % 16, c // 16], -1).flatten(-2)
        x, m = (c >> 1) & 3, (c & 1).double()
        v = torch.where(x == 0, m / 2, _by_two(1 + m / 2, x - 1))
        sign = c >= 8
    else:
        x, m = (c >> 3) & 15, (c & 7).double()
        v = torch.where(x == 0, m / 512, _by_two(1 + m / 8, x - 7))
        sign = c >= 128
    v = torch.where(sign, -v, v)
    group = torch.arange(case["D"], device=DEV) // 32
    return _by_two(v, e[..., group])


def _exact_attn(case, st):
    held, queries = _lengths(case)
    G, D, row = case["group"], case["D"], 0
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    for b, (have, n) in enumerate(zip(held, queries)):
        k = _exact_tokens(case, st, "k", st["table"][b], have)
        v = _exact_tokens(case, st, "v", st["table"][b], have)
        for first in range(0, n, 512):
            i = torch.arange(first, min(n, first + 512), device=DEV)
            pos = have - n + i
            t = torch.arange(have, device=DEV)
            hidden = torch.zeros(len(i), have, dtype=torch.bool, device=DEV)
            if case["causal"]:
                hidden |= t[None] > pos[:, None]
            if case["window"]:
                hidden |= t[None] + case["window"] <= pos[:, None]
            for h in range(case["hk"]):
                for g in range(h * G, h * G + G):
                    z = st["q"][row + i, g].double() @ k[:, h].T / math.sqrt(D)
                    z[hidden] = -math.inf
                    total = torch.logsumexp(z, -1)
                    lse[row + i, g] = total
                    some = total > -math.inf
                    out[row + i[some], g] = torch.exp(z[some] - total[some, None]) @ v[:, h]
        row += n
    return [out, lse] if case["lse"] else [out]


def _exact_codes(case, arrays):
    """Codes of 8 bits as their values, the rest as it is held."""
    if case["fmt"] == "e2m1":
        return arrays
    f8 = torch.float8_e4m3fn
    return [arrays[0].view(f8).double(), arrays[1], arrays[2].view(f8).double(), arrays[3]]


def _exact_copy(case, st):
    out = [t.clone() for t in _arrays(st)]
    for t, old in zip(out, _arrays(st)):
        moves = [(s, d) for s, d in zip(st["src"].tolist(), st["dst"].tolist()) if s >= 0]
        s, d = torch.tensor(moves, device=DEV).T if moves else (st["src"][:0].long(),) * 2
        t.index_copy_(0, d, old.index_select(0, s))
    return _exact_codes(case, out)


def _exact_fork(case, st):
    page, out = case["page"], [t.clone() for t in _arrays(st)]
    refs, table, lengths = (st[n].tolist() for n in ("refs", "table", "lengths"))
    free = [p for p, r in enumerate(refs) if r == 0]
    for parent, child in zip(st["parents"].tolist(), st["children"].tolist()):
        have = lengths[parent]
        full, rest = divmod(have, page)
        row = table[parent][:full]
        if rest:
            new, old = free.pop(0), table[parent][full]
            row = row + [new]
            for t in out:
                if case["heads_first"]:
                    t[new, :, :rest] = t[old, :, :rest]
                else:
                    t[new, :rest] = t[old, :rest]
        for p in row:
            refs[p] += 1
        table[child] = row + [-1] * (len(table[child]) - len(row))
        lengths[child] = have
    return _exact_codes(case, out) + [torch.tensor(x, dtype=torch.int32, device=DEV)
                                      for x in (refs, table, lengths)]


def _exact_compact(case, st):
    refs, table, out = st["refs"].tolist(), st["table"].tolist(), [t.clone() for t in _arrays(st)]
    live = sum(r > 0 for r in refs)
    holes = iter([p for p in range(live) if refs[p] == 0])
    to = {p: next(holes) for p in range(live, len(refs)) if refs[p] > 0}
    new = refs[:live] + [0] * (len(refs) - live)
    for p, q in to.items():
        new[q] = refs[p]
    if to:
        s, d = (torch.tensor(list(x), device=DEV) for x in (to.keys(), to.values()))
        for t in out:
            t[d] = t[s]
    rows = [[to.get(p, p) for p in r] for r in table]
    return _exact_codes(case, out) + [torch.tensor(x, dtype=torch.int32, device=DEV)
                                      for x in ([live], new, rows)]


def _exact_turn(x, case, st, sign):
    """Pairs as complex numbers, turned by the angle of their axis's position."""
    R = case["R"]
    axes = torch.nn.functional.one_hot(st["axis"], case["axes"]).double()
    angle = sign * (axes @ st["positions"].double()).T[:, None] * st["inv"]
    head = x[..., :R]
    pairs = head.unflatten(-1, (R // 2, 2)) if case["interleaved"] else \
        head.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(angle), angle)
    pairs = torch.view_as_real(z)
    turned = pairs.flatten(-2) if case["interleaved"] else pairs.transpose(-1, -2).flatten(-2)
    return torch.cat([turned, x[..., R:]], -1)


def _exact_axes_fwd(case, st):
    outs, kept = [], []
    for n in "qk":
        x = st[n].double()
        if case["norm"]:
            d = torch.sqrt(torch.linalg.vector_norm(x, dim=-1).pow(2) / x.shape[-1] + st["eps"])
            kept.append(1 / d)
            x = x / d[..., None] * (case["offset"] + st["w_" + n].double())
        outs.append(_exact_turn(x, case, st, 1.0))
    return outs + kept


def _exact_axes_bwd(case, st):
    outs, dws = [], []
    for n in "qk":
        d = _exact_turn(st["d" + n].double(), case, st, -1.0)
        if case["norm"]:
            x, r = st[n].double(), st["rstd_" + n].double()[..., None]
            w = case["offset"] + st["w_" + n].double()
            dws.append((d * x * r).flatten(0, -2).sum(0))
            d = r * w * d - x * r.pow(3) * (w * d * x).sum(-1, keepdim=True) / x.shape[-1]
        outs.append(d)
    return outs + dws


_EXACT = {"attn": _exact_attn, "copy": _exact_copy, "fork": _exact_fork, "compact": _exact_compact,
          "axes_fwd": _exact_axes_fwd, "axes_bwd": _exact_axes_bwd}
