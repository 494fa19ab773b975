"""The quantised cache against the plain 64-bit encoder and decoder. Codes,
scale bytes and values read back are exact: they have to be equal, bit for bit.
"""
from __future__ import annotations

import pytest
import torch

import ops_util as U
from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _kv(T, heads, D, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, 2 * heads, D, generator=g) * scale
    x[..., ::17] *= 30
    x = x.to(U.DT[dtype]).to(DEV)
    return x[:, :heads], x[:, heads:]


def _expect(cache, k, v, slots):
    """The cache's four arrays after the write, on the CPU, from the plain encoder."""
    out = []
    for x, codes, scales in ((k, cache.k_codes, cache.k_scales), (v, cache.v_codes, cache.v_scales)):
        if codes is None:
            continue
        c, s = codes.cpu().clone(), scales.cpu().clone()
        if x is not None:
            code, byte = U.encode(x, cache.fmt)
            code = U.pack(code, cache.fmt)
            for t, slot in enumerate(slots.tolist()):
                if 0 <= slot < cache.pages * cache.page_size:
                    at = (slot // cache.page_size, slot % cache.page_size)
                    if cache.heads_first:
                        c[at[0], :, at[1]], s[at[0], :, at[1]] = code[t], byte[t]
                    else:
                        c[at], s[at] = code[t], byte[t]
        out += [c, s]
    return out


def _arrays(cache):
    return [t.cpu() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales) if t is not None]


def _same(cache, want):
    for got, w, name in zip(_arrays(cache), want, ("k_codes", "k_scales", "v_codes", "v_scales")):
        assert torch.equal(got, w), name


def _marked(*a, **kw):
    c = B.Cache(*a, **kw)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        if t is not None:
            t.fill_(0xA5)
    return c


def _token(cache, slot, which):
    """(codes, scales) of a slot's heads."""
    codes, scales = getattr(cache, which + "_codes"), getattr(cache, which + "_scales")
    p, i = slot // cache.page_size, slot % cache.page_size
    return (codes[p, :, i], scales[p, :, i]) if cache.heads_first else (codes[p, i], scales[p, i])


def _read_expect(cache, table, cu, starts, rows, dtype, fill):
    out = []
    for which in ("k", "v"):
        if getattr(cache, which + "_codes") is None:
            out.append(None)
            continue
        y = torch.full((rows, cache.heads, cache.head_dim), fill, dtype=dtype)
        for b in range(table.shape[0]):
            for i in range(cu[b], min(cu[b + 1], rows)):
                pos = i - cu[b] + (starts[b] if starts is not None else 0)
                col = pos // cache.page_size
                page = int(table[b, col]) if 0 <= col < table.shape[1] else -1
                if pos < 0 or not 0 <= page < cache.pages:
                    y[i] = 0
                    continue
                c, s = _token(cache, page * cache.page_size + pos % cache.page_size, which)
                y[i] = U.decode(c, s, cache.fmt, cache.head_dim, dtype)
        out.append(y)
    return out


def _equal_values(got, want):
    return torch.equal(torch.nan_to_num(got.cpu().float(), nan=12345.0), torch.nan_to_num(want.float(), nan=12345.0))


DIMS = [32, 64, 96, 128, 256, 512, 80, 33, 1, 7, 40]


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", DIMS)
def test_write_and_read_back(fmt, dtype, D):
    T, heads, page, pages = 45, 3, 8, 9
    k, v = _kv(T, heads, D, dtype, D)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(D))[:T].to(DEV)
    slots[::9] = -1
    for variant in ("auto", "generic"):
        for first in (False, True):
            c = _marked(pages, page, heads, D, fmt, heads_first=first)
            want = _expect(c, k, v, slots)
            B.cache_write(c, k, v, slots, variant=variant)
            _same(c, want)
            # a table of three ragged sequences, one empty, pages that end inside one
            table = torch.randperm(pages, generator=torch.Generator().manual_seed(1))[:8].view(4, 2).int()
            cu, starts = [0, 11, 11, 18, 27], [3, 0, 9, 0]
            ex = _read_expect(c, table, cu, starts, 30, U.DT[dtype], 9.0)
            ko, vo = (torch.full((30, heads, D), 9.0, dtype=U.DT[dtype], device=DEV) for _ in range(2))
            B.cache_read(c, table.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV), 30,
                         starts=torch.tensor(starts, dtype=torch.int32, device=DEV), k_out=ko, v_out=vo,
                         variant=variant)
            assert B.rmsnorm_check_device_status(0) == 0
            assert _equal_values(ko, ex[0]) and _equal_values(vo, ex[1])


@pytest.mark.parametrize("T,heads,D,page", [(1, 1, 32, 1), (1, 8, 128, 16), (64, 8, 128, 16), (1000, 5, 96, 24),
                                            (4097, 2, 64, 7), (300, 1, 512, 64)])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_sizes(T, heads, D, page, fmt):
    pages = -(-T // page) + 2
    k, v = _kv(T, heads, D, "bf16", T)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T].to(DEV)
    for opts in (dict(), dict(max_ctas=1)):
        c = _marked(pages, page, heads, D, fmt)
        B.cache_write(c, k, v, slots, **opts)
        code, byte = U.encode(k, fmt)
        at = slots.cpu()
        assert torch.equal(c.k_codes.cpu().flatten(0, 1)[at], U.pack(code, fmt))
        assert torch.equal(c.k_scales.cpu().flatten(0, 1)[at], byte)
        untouched = torch.ones(pages * page, dtype=torch.bool)
        untouched[at] = False
        assert bool((c.v_codes.cpu().flatten(0, 1)[untouched] == 0xA5).all())
        table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
        cu = torch.tensor([0, pages * page], dtype=torch.int32, device=DEV)
        c.k_codes.flatten(0, 1)[untouched.to(DEV)] = 0
        ko, vo = B.cache_read(c, table, cu, pages * page, **opts)
        want = U.decode(U.pack(code, fmt), byte, fmt, D, torch.bfloat16)
        assert torch.equal(ko.cpu()[at], want)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("variant", ["auto", "generic"])
def test_values_at_the_edges(fmt, dtype, variant):
    dt, D = U.DT[dtype], 64
    fi = torch.finfo(dt)
    rows = [torch.zeros(D), torch.full((D,), fi.max), torch.full((D,), -fi.max),
            torch.full((D,), fi.smallest_normal), torch.full((D,), fi.smallest_normal * fi.eps),
            torch.linspace(-6, 6, D), torch.linspace(-448, 448, D), torch.full((D,), 448.0),
            torch.full((D,), 449.0), torch.tensor([6.0] + [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] * 9),
            torch.tensor([448.0] + [2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 21.0, -17.0, -2.0 ** -10] * 9),
            -torch.zeros(D)]
    bad = torch.ones(D)
    bad[3] = float("inf")
    rows.append(bad)
    bad = torch.ones(D)
    bad[40] = float("nan")
    rows.append(bad)
    x = torch.stack(rows).to(dt).unsqueeze(1).to(DEV)
    c = _marked(4, 8, 1, D, fmt)
    slots = torch.arange(len(rows), device=DEV)
    want = _expect(c, x, x, slots)
    B.cache_write(c, x, x, slots, variant=variant)
    _same(c, want)
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4)
    cu = torch.tensor([0, len(rows)], dtype=torch.int32, device=DEV)
    ko, _ = B.cache_read(c, table, cu, len(rows), dtype=dt, variant=variant)
    ex = _read_expect(c, table.cpu(), [0, len(rows)], None, len(rows), dt, 0.0)[0]
    assert _equal_values(ko, ex)
    assert bool(ko[-2, 0, :32].isnan().all()) and bool((ko[-2, 0, 32:] == 1).all())
    assert bool(ko[-1, 0, 32:].isnan().all()) and bool((ko[-1, 0, :32] == 1).all())


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("variant", ["auto", "generic"])
def test_every_code_and_scale_reads_back(fmt, variant):
    c = B.Cache(1, 256, 1, 256, fmt)
    n = c.k_codes.shape[-1]
    c.k_codes.copy_(torch.arange(n, dtype=torch.uint8, device=DEV).expand(1, 256, 1, n))
    c.k_scales.copy_(torch.arange(256, dtype=torch.uint8, device=DEV).view(1, 256, 1, 1).expand(1, 256, 1, 8))
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 256], dtype=torch.int32, device=DEV)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        ko, _ = B.cache_read(c, table, cu, 256, dtype=dt, variant=variant)
        ex = _read_expect(c, table.cpu(), [0, 256], None, 256, dt, 0.0)[0]
        assert _equal_values(ko, ex), dt


@pytest.mark.parametrize("variant", ["auto", "generic"])
def test_a_cache_of_one_tensor_and_calls_for_one(variant):
    k, v = _kv(20, 2, 64, "bf16", 3)
    slots = torch.arange(20, device=DEV)
    c = _marked(2, 16, 2, 64, values=False)
    want = _expect(c, k, None, slots)
    B.cache_write(c, k, None, slots, variant=variant)
    _same(c, want)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 20], dtype=torch.int32, device=DEV)
    ko, vo = B.cache_read(c, table, cu, 20, variant=variant)
    assert vo is None and _equal_values(ko, _read_expect(c, table.cpu(), [0, 20], None, 20, torch.bfloat16, 0.0)[0])
    with pytest.raises(B.RMSNormError):
        B.cache_write(c, k, v, slots)
    c = _marked(2, 16, 2, 64)      # k alone into a cache of both: v stays
    want = _expect(c, k, None, slots)
    B.cache_write(c, k, None, slots, variant=variant)
    _same(c, want)


@pytest.mark.parametrize("variant", ["auto", "generic"])
def test_indices_out_of_range_are_skipped_and_reported(variant):
    k, v = _kv(6, 2, 64, "bf16", 4)
    c = _marked(2, 16, 2, 64)
    slots = torch.tensor([0, 32, -1, 1 << 40, 31, -(1 << 62)], device=DEV)
    want = _expect(c, k, v, slots)
    assert B.rmsnorm_check_device_status(0) == 0
    B.cache_write(c, k, v, slots, variant=variant)
    assert B.rmsnorm_check_device_status(0) == -12
    assert B.rmsnorm_check_device_status(0) == 0
    _same(c, want)
    table = torch.tensor([[1, 2], [-1, 0], [0, 1], [1, 0]], dtype=torch.int32)
    cu, starts = [0, 20, 25, 30, 40], [0, 12, 30, -4]
    ko, vo = (torch.full((45, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ex = _read_expect(c, table, cu, starts, 45, torch.bfloat16, 9.0)
    B.cache_read(c, table.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV), 45,
                 starts=torch.tensor(starts, dtype=torch.int32, device=DEV), k_out=ko, v_out=vo, variant=variant)
    assert B.rmsnorm_check_device_status(0) == -12
    assert _equal_values(ko, ex[0]) and _equal_values(vo, ex[1])
    assert bool((ko[40:] == 9.0).all()) and bool((ko[16:20] == 0).all())


@pytest.mark.parametrize("variant", ["auto", "generic"])
def test_rows_of_the_output_may_be_fewer_than_the_batch(variant):
    k, v = _kv(32, 1, 64, "bf16", 5)
    c = _marked(2, 16, 1, 64)
    B.cache_write(c, k, v, torch.arange(32, device=DEV))
    table = torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 16, 32], dtype=torch.int32, device=DEV)
    full = torch.full((32, 1, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    B.cache_read(c, table, cu, 20, k_out=full[:20], v_out=torch.empty_like(full[:20]), variant=variant)
    whole, _ = B.cache_read(c, table, cu, 32)
    assert torch.equal(full[:20], whole[:20]) and bool((full[20:] == 9.0).all())


@pytest.mark.parametrize("B_", [1, 2, 31, 32, 33, 1000, 1025, 5000])
def test_many_short_sequences(B_):
    # Every sequence's rows come from its own page; many are empty.
    g = torch.Generator().manual_seed(B_)
    lens = torch.randint(0, 3, (B_,), generator=g)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).int()
    rows = int(cu[-1])
    c = B.Cache(B_, 2, 1, 32)
    c.k_codes.random_(0, 120)
    c.k_scales.fill_(127)
    table = torch.randperm(B_, generator=g).int().view(B_, 1)
    ko, _ = B.cache_read(c, table.to(DEV), cu.to(DEV), rows)
    seq = torch.repeat_interleave(torch.arange(B_), lens)
    at = torch.arange(rows) - cu[seq].long()
    codes = c.k_codes.cpu()[table[seq, 0].long(), at, 0]
    assert torch.equal(ko.cpu()[:, 0], U.decode(codes, torch.full((rows, 1), 127), "e4m3", 32, torch.bfloat16))


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (1, 0), (0, 1), (4, 4)])
def test_strided_and_shifted_tensors(pad, shift):
    T, heads, D = 30, 3, 64
    k, v = _kv(T, heads, D, "bf16", 6)
    slots = torch.randperm(48, generator=torch.Generator().manual_seed(2))[:T].to(DEV)
    want = _expect(_marked(3, 16, heads, D), k, v, slots)

    def wide(t, fill=7.0):
        full = torch.full((T, heads, D + pad + shift), fill, dtype=torch.bfloat16, device=DEV)
        view = full[..., shift:shift + D]
        if t is not None:
            view.copy_(t)
        return full, view

    c = _marked(3, 16, heads, D)
    B.cache_write(c, wide(k)[1], wide(v)[1], slots)
    _same(c, want)
    # a whole-cache tensor at a shifted address
    n = c.k_codes.numel()
    raw = torch.full((n + 16,), 0xA5, dtype=torch.uint8, device=DEV)
    shifted = raw[shift:shift + n].view(c.k_codes.shape)
    c2 = B.Cache(3, 16, heads, D, tensors=(shifted, c.k_scales.clone(), c.v_codes.clone(), c.v_scales.clone()))
    B.cache_write(c2, k, v, slots)
    _same(c2, want)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    ex = _read_expect(c2, table.cpu(), [0, T], None, T, torch.bfloat16, 0.0)
    (fk, ko), (fv, vo) = wide(None), wide(None)
    B.cache_read(c2, table, cu, T, k_out=ko, v_out=vo)
    assert _equal_values(ko, ex[0]) and _equal_values(vo, ex[1])
    for f in (fk, fv):
        assert bool((f[..., :shift] == 7.0).all()) and bool((f[..., shift + D:] == 7.0).all())


@pytest.mark.slow
@pytest.mark.parametrize("fmt,first", [("e4m3", False), ("e2m1", True)])
def test_offsets_past_32_bits(fmt, first):
    # A cache whose codes pass 2^32 bytes: the last slots and the first ones.
    heads, D, page = 8, 256, 64
    per = page * heads * (D if fmt == "e4m3" else D // 2)
    pages = (1 << 32) // per + 3
    c = B.Cache(pages, page, heads, D, fmt, heads_first=first, values=False)
    k, _ = _kv(128, heads, D, "bf16", 7)
    slots = torch.cat([torch.arange(64), pages * page - 64 + torch.arange(64)]).to(DEV)
    B.cache_write(c, k, None, slots)
    code, byte = U.encode(k, fmt)
    code = U.pack(code, fmt)
    for page_at, part in ((0, slice(0, 64)), (pages - 1, slice(64, 128))):
        got, sc = c.k_codes[page_at].cpu(), c.k_scales[page_at].cpu()
        if first:
            got, sc = got.transpose(0, 1), sc.transpose(0, 1)
        assert torch.equal(got, code[part]) and torch.equal(sc, byte[part])
    assert int(c.k_codes[1:-1].any()) == 0
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 128], dtype=torch.int32, device=DEV)
    ko, _ = B.cache_read(c, table, cu, 128)
    want = U.decode(code, byte, fmt, D, torch.bfloat16)
    assert torch.equal(ko.cpu(), torch.cat([want[64:], want[:64]]))


def test_captured_and_replayed_and_on_another_stream():
    k, v = _kv(16, 2, 128, "bf16", 8)
    c, d = _marked(4, 16, 2, 128), _marked(4, 16, 2, 128)
    slots = torch.arange(16, device=DEV)
    table = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 0], dtype=torch.int32, device=DEV)
    out = torch.zeros(64, 2, 128, dtype=torch.bfloat16, device=DEV)
    vout = torch.zeros_like(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.cache_write(c, k, v, slots)
        slots += 16
        cu[1] += 16
        B.cache_read(c, table, cu, 64, k_out=out, v_out=vout)
    side = torch.cuda.Stream()
    for step in range(4):
        graph.replay()
        torch.cuda.synchronize()
        B.cache_write(d, k, v, torch.arange(16, device=DEV) + 16 * step, stream=side) if step == 0 else \
            B.cache_write(d, k, v, torch.arange(16, device=DEV) + 16 * step)
        torch.cuda.synchronize()
        _same(c, _arrays(d))
        ko, _ = B.cache_read(d, table, torch.tensor([0, 16 * step + 16], dtype=torch.int32, device=DEV),
                             16 * step + 16)
        assert torch.equal(out[:16 * step + 16], ko) and not bool(out[16 * step + 16:].any())


def test_refused_tensors():
    c = B.Cache(2, 16, 2, 64)
    k, v = _kv(4, 2, 64, "bf16", 9)
    slots = torch.arange(4, device=DEV)
    for bad in (dict(k=k[0]), dict(k=k[:, :1]), dict(v=v.half()), dict(slots=slots.int()), dict(slots=slots[:3]),
                dict(slots=slots.cpu()), dict(k=k.cpu()), dict(v=v[:3])):
        with pytest.raises(ValueError):
            B.cache_write(c, **{**dict(k=k, v=v, slots=slots), **bad})
    table = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    cu = torch.zeros(2, dtype=torch.int32, device=DEV)
    for bad in (dict(table=table[0]), dict(table=table.long()), dict(cu_rows=cu[:1]), dict(cu_rows=cu.long()),
                dict(starts=cu), dict(k_out=k[:, :1]), dict(cu_rows=cu.cpu())):
        with pytest.raises(ValueError):
            B.cache_read(c, **{**dict(table=table, cu_rows=cu, rows=4), **bad})
    for bad in (dict(fmt="int8"), dict(tensors=(c.k_codes,)), dict(tensors=(c.k_codes.cpu(),) * 4)):
        with pytest.raises(ValueError):
            B.Cache(2, 16, 2, 64, **bad)
