"""Rotary positions with several axes against the plain 64-bit implementation, and the run of the
serving operators together."""
from __future__ import annotations

import pytest
import torch

import ops_util as U
import serve_util as S
from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _axis_of(pairs, in_turn):
    n = len(pairs)
    if in_turn:
        return [i % n if i // n < pairs[i % n] else 0 for i in range(sum(pairs))]
    return [a for a in range(n) for _ in range(pairs[a])]


def _angles(steps, positions, axis):
    """[..., T, R / 2] from positions [axes, ..., T]."""
    per = torch.stack([U.rope_angles(steps, p) for p in positions.cpu()])
    return torch.stack([per[a][..., i] for i, a in enumerate(axis)], -1).to(DEV)


def _qk(lead, hq, hk, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*lead, hq + 2 * hk, D, generator=g).to(U.DT[dtype]).to(DEV)
    return x[..., :hq, :], x[..., hq:hq + hk, :]


CASES = [((8, 12, 12), False), ((14, 9, 9), True), ((12, 10, 10), True), ((0, 32, 0), False), ((32,), False),
         ((16, 16), True), ((1, 2, 3, 26), False), ((8, 8, 8, 8), True), ((30, 1, 1), True), ((32, 0), True)]


@pytest.mark.parametrize("pairs,in_turn", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,interleaved", [(64, False), (64, True), (96, False), (65, False), (65, True)])
def test_forward_and_backward(pairs, in_turn, dtype, D, interleaved):
    lead, hq, hk, R = (2, 9), 5, 2, 64
    axes = B.RopeAxes(pairs, in_turn)
    g = torch.Generator().manual_seed(len(pairs))
    pos = torch.randint(-5, 1 << 40, (len(pairs), *lead), generator=g).to(DEV)
    steps, mag = B.rope_steps(R, device=DEV, scaling=dict(kind="yarn", factor=4.0, length=2048))
    angle = _angles(steps, pos, _axis_of(pairs, in_turn))
    q, k = _qk(lead, hq, hk, D, dtype, 3)
    for weights in (False, True):
        w = (torch.rand(D, generator=g) + 0.5).to(U.DT[dtype]).to(DEV) if weights else None
        kw = dict(positions=pos, w_q=w, w_k=w, interleaved=interleaved, magnitude=mag, axes=axes, offset=0.0)
        outs = []
        for variant in ("auto", "generic"):
            oq, ok, rq, rk = B.rope_fwd(q, k, steps, variant=variant, **kw)
            for x, o, r in ((q, oq, rq), (k, ok, rk)):
                want, rstd, m = U.rope_fwd(x, angle, w, R, interleaved, 1e-6, 0.0, mag)
                U.check(o, want, m, U.DT[dtype], "out")
                if weights:
                    U.check(r, rstd, rstd, torch.float32, "rstd")
            dq, dk = _qk(lead, hq, hk, D, dtype, 4)
            got = B.rope_bwd(dq, dk, steps, q=q if weights else None, k=k if weights else None, rstd_q=rq,
                             rstd_k=rk, variant=variant, **kw)
            for d, x, r, gx, gw in ((dq, q, rq, got[0], got[2]), (dk, k, rk, got[1], got[3])):
                dx, dw, mdx, mdw = U.rope_bwd(d, x, r, angle, w, R, interleaved, 0.0, mag)
                U.check(gx, dx, mdx, U.DT[dtype], "dx")
                if weights:
                    U.check(gw, dw, mdw, torch.float32, "dw")
            outs.append((oq, ok))
        assert all(a.shape == b.shape for a, b in zip(*outs))


@pytest.mark.parametrize("interleaved", [False, True])
def test_same_positions_on_all_axes_give_the_bits_of_one(interleaved):
    q, k = _qk((50,), 4, 2, 128, "bf16", 1)
    steps, mag = B.rope_steps(128, device=DEV)
    pos = torch.arange(1000, 1050, device=DEV)
    one = B.rope_fwd(q, k, steps, positions=pos, interleaved=interleaved)
    for in_turn in (False, True):
        axes = B.RopeAxes((24, 20, 20), in_turn)
        # one row of positions for every axis: a stride of zero
        several = B.rope_fwd(q, k, steps, positions=pos.expand(3, 50), interleaved=interleaved, axes=axes)
        assert torch.equal(one[0], several[0]) and torch.equal(one[1], several[1])


def test_frequencies_of_the_axes_own():
    axes = B.RopeAxes((4, 6, 6))
    steps, mag = B.rope_steps(32, base=1000.0, device="cpu", axes=axes)
    parts = [B.rope_steps(2 * n, base=1000.0, device="cpu")[0] for n in (4, 6, 6)]
    assert torch.equal(steps, torch.cat(parts)) and mag == 1.0
    # an axis alone turns as a head of its pairs would
    q, _ = _qk((7,), 2, 1, 32, "fp32", 1)
    pos = torch.stack([torch.arange(7), torch.zeros(7, dtype=torch.int64), torch.arange(7) * 3]).to(DEV)
    got = B.rope_fwd(q, None, steps.to(DEV), positions=pos, axes=axes, interleaved=True)[0]
    for lo, n, p in ((0, 4, pos[0]), (8, 6, pos[1]), (20, 6, pos[2])):
        part = q[..., lo:lo + 2 * n]
        s, _ = B.rope_steps(2 * n, base=1000.0, device=DEV)
        assert torch.equal(got[..., lo:lo + 2 * n], B.rope_fwd(part, None, s, positions=p, interleaved=True)[0])


def test_positions_of_one_row_for_all_batches():
    q, k = _qk((3, 11), 4, 2, 64, "bf16", 1)
    steps, _ = B.rope_steps(64, device=DEV)
    axes = B.RopeAxes((12, 10, 10))
    pos = torch.randint(0, 5000, (3, 11), device=DEV)
    a = B.rope_fwd(q, k, steps, positions=pos, axes=axes)
    b = B.rope_fwd(q, k, steps, positions=pos[:, None].expand(3, 3, 11).contiguous(), axes=axes)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    none = B.rope_fwd(q[:, :0], k[:, :0], steps, positions=pos[:, :0], axes=axes)
    assert none[0].shape == (3, 0, 4, 64)


def test_gradient_against_differences():
    axes, steps = B.RopeAxes((3, 2, 3)), B.rope_steps(16, device=DEV)[0]
    q, _ = _qk((4,), 2, 1, 20, "fp32", 1)
    q = q.contiguous()
    w = torch.rand(20, device=DEV) + 0.5
    pos = torch.randint(0, 100, (3, 4), device=DEV)
    d = torch.randn(4, 2, 20, device=DEV)

    def loss(x, weight):
        y = B.rope_fwd(x, None, steps, positions=pos, w_q=weight, axes=axes)[0]
        return float((y.double() * d.double()).sum())

    _, _, r, _ = B.rope_fwd(q, None, steps, positions=pos, w_q=w, axes=axes)
    dq, _, dw, _ = B.rope_bwd(d, None, steps, positions=pos, q=q, rstd_q=r, w_q=w, axes=axes)
    # central differences of step h: their own error is about h^2 and 2^-24 / h of the values
    h = 2.0 ** -8
    for i in (0, 19, 37, 100, 159):
        e = torch.zeros_like(q).view(-1)
        e[i] = h
        e = e.view_as(q)
        assert abs((loss(q + e, w) - loss(q - e, w)) / (2 * h) - float(dq.flatten()[i])) < 2e-3
    for i in (0, 7, 19):
        e = torch.zeros_like(w)
        e[i] = h
        assert abs((loss(q, w + e) - loss(q, w - e)) / (2 * h) - float(dw[i])) < 2e-3


def test_backward_captured_next_to_eager_calls():
    q, k = _qk((40,), 4, 2, 128, "bf16", 1)
    steps, _ = B.rope_steps(128, device=DEV)
    axes = B.RopeAxes((24, 20, 20), True)
    pos = torch.randint(0, 5000, (3, 40), device=DEV)
    w = torch.rand(128, device=DEV).to(torch.bfloat16)
    kw = dict(positions=pos, w_q=w, w_k=w, axes=axes)
    oq, ok, rq, rk = B.rope_fwd(q, k, steps, **kw)
    eager = B.rope_bwd(oq, ok, steps, q=q, k=k, rstd_q=rq, rstd_k=rk, **kw)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = B.rope_bwd(oq, ok, steps, q=q, k=k, rstd_q=rq, rstd_k=rk, **kw)
    side = torch.cuda.Stream()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, got))
    pos.add_(3)
    side.wait_stream(torch.cuda.current_stream())
    other = B.rope_bwd(oq, ok, steps, q=q, k=k, rstd_q=rq, rstd_k=rk, stream=side, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, got))


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_served_together(fmt):
    """A step of a server: image tokens turned by three axes, written, forked, attended to, freed
    and compacted, against the plain forms of each on the same cache."""
    heads, G, D, page = 2, 3, 64, 8
    cache = B.Cache(40, page, heads, D, fmt)
    refs, lengths = torch.zeros(40, dtype=torch.int32, device=DEV), torch.zeros(6, dtype=torch.int32, device=DEV)
    table = torch.full((6, 5), -1, dtype=torch.int32, device=DEV)
    axes, steps = B.RopeAxes((12, 10, 10)), B.rope_steps(64, device=DEV)[0]
    # two prompts of 19 and 24 tokens on pages far back
    lens = [19, 24]
    for b, pages in enumerate(([30, 35, 39], [31, 37, 33])):
        table[b, :3] = torch.tensor(pages, dtype=torch.int32)
        refs[torch.tensor(pages, device=DEV)] = 1
        lengths[b] = lens[b]
    rows = sum(lens)
    qkv = torch.randn(rows, (G + 2) * heads, D, device=DEV).to(torch.bfloat16)
    q, k, v = qkv[:, :G * heads], qkv[:, G * heads:(G + 1) * heads], qkv[:, (G + 1) * heads:]
    pos = torch.randint(0, 64, (3, rows), device=DEV)
    qr, kr, _, _ = B.rope_fwd(q, k, steps, positions=pos, axes=axes)
    t = torch.cat([torch.arange(n) for n in lens]).to(DEV)
    seq = torch.tensor([0] * 19 + [1] * 24, device=DEV)
    slots = table[seq, t // page].long() * page + t % page
    B.cache_write(cache, kr, v, slots)
    cu = torch.tensor([0, 19, 43, 43, 43, 43, 43], dtype=torch.int32, device=DEV)
    out, lse = B.cache_attention(cache, qr, table, lengths, cu_q=cu, lse=True)
    want = S.attention(cache, qr, table.tolist(), lengths.tolist(), cu.tolist(), D ** -0.5, True, 0)
    S.check_attention(out, lse, want, torch.bfloat16, "prompt")
    # three answers to the first prompt, one to the second, each with a token of its own
    kids = torch.tensor([2, 3, 5, 4], dtype=torch.int32, device=DEV)
    B.cache_fork(cache, refs, table, lengths, torch.tensor([0, 0, 0, 1], dtype=torch.int32, device=DEV), kids)
    B.cache_free(refs, table, lengths, torch.tensor([1], dtype=torch.int32, device=DEV))
    live, refs, table = B.cache_compact(cache, refs, table)
    assert live.tolist() == [3 + 3 + 3] and bool((table < 9).all())
    assert refs.tolist()[:9].count(4) == 2 and sum(refs.tolist()) == 3 * 4 + 3
    some = torch.tensor([2, 3, 5], device=DEV)
    last = lengths[some].long()
    new = torch.randn(3, (G + 2) * heads, D, device=DEV).to(torch.bfloat16)
    npos = torch.full((3, 3), 70, device=DEV)
    nq, nk, _, _ = B.rope_fwd(new[:, :G * heads], new[:, G * heads:(G + 1) * heads], steps, positions=npos, axes=axes)
    B.cache_write(cache, nk, new[:, (G + 1) * heads:], table[some, last // page].long() * page + last % page)
    lengths[some] += 1
    rows3 = table[some].contiguous()
    out, lse = B.cache_attention(cache, nq, rows3, lengths[some].contiguous(), lse=True)
    want = S.attention(cache, nq, rows3.tolist(), lengths[some].tolist(), [0, 1, 2, 3], D ** -0.5, True, 0)
    S.check_attention(out, lse, want, torch.bfloat16, "answers")
    # the first prompt, whose pages two of them share, is what it was
    again, _ = B.cache_attention(cache, qr[:19], table[:1].contiguous(), lengths[:1].contiguous(),
                                 cu_q=torch.tensor([0, 19], dtype=torch.int32, device=DEV))
    first = S.attention(cache, qr[:19], table[:1].tolist(), [19], [0, 19], D ** -0.5, True, 0)
    S.check_attention(again, None, first, torch.bfloat16, "prompt again")
    assert B.rmsnorm_check_device_status(0) == 0
