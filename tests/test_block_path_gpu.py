"""The block, rope and cache operators together, as a block of a model uses them:
norm before the block, projections, head norms and rotation, the cache written
and read back, attention, projection, then the norm after the block with its
gate, residual and the next norm; forward and backward, against the same block in
64 bits with torch's own differentiation.
"""
from __future__ import annotations

import pytest
import torch

import ops_util as U
from memory_bound_normalization_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
S, N, HQ, HK, D = 48, 256, 4, 2, 64


def _weights(seed, dt):
    g = torch.Generator().manual_seed(seed)

    def rnd(*s, scale=1.0):
        return (torch.randn(*s, generator=g) * scale).to(dt).to(DEV)

    return dict(x=rnd(S, N), w_in=rnd(N, scale=0.1), w_qkv=rnd((HQ + 2 * HK) * D, N, scale=N ** -0.5),
                w_q=rnd(D, scale=0.1), w_k=rnd(D, scale=0.1), w_o=rnd(N, HQ * D, scale=(HQ * D) ** -0.5),
                w_post=rnd(N, scale=0.1), gate=rnd(N), w_pre=rnd(N, scale=0.1), dy=rnd(S, N), ds=rnd(S, N))


def _attend(q, k, v):
    k, v = (t.repeat_interleave(HQ // HK, 1) for t in (k, v))
    a = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
    a = a.masked_fill(torch.ones(S, S, dtype=torch.bool, device=DEV).triu(1), float("-inf")).softmax(-1)
    return torch.einsum("hij,jhd->ihd", a, v)


def _reference(w, angle):
    p = {k: v.double().requires_grad_() for k, v in w.items() if k not in ("dy", "ds")}
    rms = lambda t: t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    h = rms(p["x"]) * (1 + p["w_in"])
    qkv = (h @ p["w_qkv"].T).view(S, HQ + 2 * HK, D)
    q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:]
    q = U.turn(rms(q) * (1 + p["w_q"]), angle, D, False, 1.0, 1.0)
    k = U.turn(rms(k) * (1 + p["w_k"]), angle, D, False, 1.0, 1.0)
    o = _attend(q, k, v).reshape(S, HQ * D) @ p["w_o"].T
    s = p["x"] + 0.5 * p["gate"] * rms(o) * (1 + p["w_post"])
    y = rms(s) * (1 + p["w_pre"])
    loss = (y * w["dy"].double()).sum() + (s * w["ds"].double()).sum()
    return p, q, k, v, s, y, loss


def test_training_step_of_a_block_fp32():
    w = _weights(1, torch.float32)
    steps, _ = B.rope_steps(D, device=DEV)
    pos = torch.arange(S, device=DEV)
    p, _, _, _, s64, y64, loss = _reference(w, U.rope_angles(steps, pos))
    names = ["x", "w_in", "w_qkv", "w_q", "w_k", "w_o", "w_post", "gate", "w_pre"]
    want = dict(zip(names, torch.autograd.grad(loss, [p[n] for n in names])))

    h, r0 = B.fwd(w["x"], w["w_in"], offset=1.0)
    qkv = (h @ w["w_qkv"].T).view(S, HQ + 2 * HK, D)
    q0, k0, v = qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:]
    q, k, rq, rk = B.rope_fwd(q0, k0, steps, pos, w["w_q"], w["w_k"], offset=1.0)
    ql, kl, vl = (t.detach().clone().requires_grad_() for t in (q, k, v))
    att = _attend(ql, kl, vl).reshape(S, HQ * D)
    o = att.detach() @ w["w_o"].T
    s, y, rpost, rpre = B.block_fwd(o, w["x"], w["w_post"], w["w_pre"], w["gate"], offset=1.0, alpha=0.5)
    assert torch.allclose(s.double(), s64, rtol=1e-4, atol=1e-4)
    assert torch.allclose(y.double(), y64, rtol=1e-4, atol=1e-4)

    got = {}
    do, dr, got["gate"], got["w_post"], got["w_pre"] = B.block_bwd(
        o, s, rpost, rpre, w["dy"], w["ds"], w["w_post"], w["w_pre"], w["gate"], offset=1.0, alpha=0.5)
    got["w_o"] = do.T @ att.detach()
    dq, dk, dv = torch.autograd.grad(att, [ql, kl, vl], do @ w["w_o"])
    dqkv = torch.empty_like(qkv)
    dqkv[:, HQ + HK:] = dv
    _, _, got["w_q"], got["w_k"] = B.rope_bwd(dq.contiguous(), dk.contiguous(), steps, pos, q0, k0, rq, rk, w["w_q"], w["w_k"],
                                              offset=1.0, dq=dqkv[:, :HQ], dk=dqkv[:, HQ:HQ + HK])
    d2 = dqkv.view(S, -1)
    got["w_qkv"] = d2.T @ h
    dx, got["w_in"] = B.bwd(w["x"], w["w_in"], r0, d2 @ w["w_qkv"], offset=1.0)
    got["x"] = dx + dr
    for n in names:
        e = (got[n].double() - want[n]).norm() / want[n].norm()
        assert float(e) < 1e-5, (n, float(e))


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_decoding_from_the_cache_one_token_at_a_time(fmt):
    # A prompt of 40 tokens, then one token at a time: what the cache gives back is
    # the rounding of the same keys and values, whichever call wrote them.
    w = _weights(2, torch.bfloat16)
    steps, _ = B.rope_steps(D, device=DEV)
    h, _ = B.fwd(w["x"], w["w_in"], offset=1.0)
    qkv = (h @ w["w_qkv"].T).view(S, HQ + 2 * HK, D)
    cache = B.Cache(8, 16, HK, D, fmt)
    table = torch.tensor([[5, 0, 7]], dtype=torch.int32, device=DEV)
    pos = torch.arange(S, device=DEV)
    slots = table[0, pos // 16].long() * 16 + pos % 16
    keys = []
    for a, b in [(0, 40)] + [(i, i + 1) for i in range(40, S)]:
        part = qkv[a:b]
        q, k, _, _ = B.rope_fwd(part[:, :HQ], part[:, HQ:HQ + HK], steps, pos[a:b], w["w_q"], w["w_k"], offset=1.0)
        B.cache_write(cache, k, part[:, HQ + HK:], slots[a:b])
        keys.append(k)
        cu = torch.tensor([0, b], dtype=torch.int32, device=DEV)
        kr, vr = B.cache_read(cache, table, cu, b)
        for got, x in ((kr, torch.cat(keys)), (vr, qkv[:b, HQ + HK:])):
            code, byte = U.encode(x, fmt)
            assert torch.equal(got.cpu(), U.decode(U.pack(code, fmt), byte, fmt, D, torch.bfloat16))
    whole = B.rope_fwd(qkv[:, :HQ], qkv[:, HQ:HQ + HK], steps, pos, w["w_q"], w["w_k"], offset=1.0)[1]
    assert torch.equal(torch.cat(keys), whole)
    assert B.rmsnorm_check_device_status(0) == 0


def test_calls_from_several_threads_on_their_own_streams():
    # Four host threads, each with its stream, tensors and cache, all three operators
    # in turn: the results of the same calls one after another.
    import threading
    w = [_weights(10 + i, torch.bfloat16) for i in range(4)]
    steps, _ = B.rope_steps(D, device=DEV)
    pos = torch.arange(S, device=DEV)
    table = torch.arange(3, dtype=torch.int32, device=DEV).view(1, 3)
    cu = torch.tensor([0, S], dtype=torch.int32, device=DEV)

    def calls(x, stream):
        out = []
        cache = B.Cache(3, 16, HK, D)
        for _ in range(5):
            s, y, a, b = B.block_fwd(x["x"], x["ds"], x["w_post"], x["w_pre"], x["gate"], stream=stream)
            out += [s, y, a, b]
            out += B.block_bwd(x["x"], s, a, b, x["dy"], x["ds"], x["w_post"], x["w_pre"], x["gate"], stream=stream)
            qk = x["x"].view(S, 4, D)
            q, k, rq, rk = B.rope_fwd(qk[:, :2], qk[:, 2:], steps, pos, x["w_q"], x["w_k"], stream=stream)
            out += [q, k, rq, rk]
            out += B.rope_bwd(q, k, steps, pos, qk[:, :2], qk[:, 2:], rq, rk, x["w_q"], x["w_k"], stream=stream)
            B.cache_write(cache, k, q, pos, stream=stream)
            out += B.cache_read(cache, table, cu, S, stream=stream)
        stream.synchronize()
        return out

    streams = [torch.cuda.Stream() for _ in w]
    torch.cuda.synchronize()
    want = [calls(x, streams[0]) for x in w]
    got = [None] * len(w)

    def work(i):
        got[i] = calls(w[i], streams[i])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(w))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert b is not None and len(a) == len(b)
        for p, q in zip(a, b):
            assert torch.equal(p, q)


def test_two_captured_graphs_with_workspaces_of_their_own():
    # Two training steps captured with their own workspaces, replayed at once on two
    # streams: the results of each replayed alone.
    w = [_weights(20 + i, torch.bfloat16) for i in range(2)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in w]
    for x in w:
        s, _, a, b = B.block_fwd(x["x"], x["ds"], x["w_post"], x["w_pre"], x["gate"])
        ws = torch.empty(B.rmsnorm_block_bwd_workspace_size(S, N, B.BF16), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = B.block_bwd(x["x"], s, a, b, x["dy"], x["ds"], x["w_post"], x["w_pre"], x["gate"], workspace=ws)
        graphs.append((g, ws, s, a, b))
        outs.append(o)
    alone = []
    for (g, *_), o in zip(graphs, outs):
        g.replay()
        torch.cuda.synchronize()
        alone.append([t.clone() for t in o])
        for t in o:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, a in zip(outs, alone):
        for p, q in zip(o, a):
            assert torch.equal(p, q)
