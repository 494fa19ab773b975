"""Host-only checks of the block, rope and cache entry points: struct layouts
against the header, and refusals before any CUDA call. Pointers here are never
dereferenced: each case fails validation first.
"""
from __future__ import annotations

import ctypes
import os
import re
import shutil
import subprocess

import pytest

from memory_bound_normalization_fwd_gb300 import binding as B
from memory_bound_normalization_fwd_gb300 import build as BUILD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "rmsnorm.h")
STRUCTS = {"rmsnorm_block_args": (B.BlockArgs, B._BLOCK), "rmsnorm_block_grads": (B.BlockGrads, B._BLOCK_GRADS),
           "rmsnorm_heads": (B.Heads, B._HEADS), "rmsnorm_rope_args": (B.RopeArgs, B._ROPE),
           "rmsnorm_rope_grads": (B.RopeGrads, B._ROPE_GRADS), "rmsnorm_rope_scaling": (B.RopeScaling, None),
           "rmsnorm_cache": (B.CacheArgs, B._CACHE)}


@pytest.fixture(scope="module", autouse=True)
def lib():
    BUILD.build()
    return B.lib()


def test_struct_layouts_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not installed")
    lines = []
    for c, (cls, packed) in STRUCTS.items():
        if packed is not None:
            assert packed.size == ctypes.sizeof(cls), c
        lines.append(f'    printf("{c} size %zu\\n", sizeof({c}_t));')
        lines += [f'    printf("{c} {n} %zu\\n", offsetof({c}_t, {n}));' for n, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include "rmsnorm.h"\n#include <stddef.h>\n#include <stdio.h>\n'
                   "int main(void) {\n" + "\n".join(lines) + "\n    return 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = {tuple(l.split()[:2]): int(l.split()[2]) for l in out.splitlines() if l.strip()}
    for c, (cls, _) in STRUCTS.items():
        assert got[(c, "size")] == ctypes.sizeof(cls), c
        for n, _ in cls._fields_:
            assert got[(c, n)] == getattr(cls, n).offset, (c, n)


def test_every_field_of_the_header_is_in_the_binding():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for c, (cls, _) in STRUCTS.items():
        body = re.search(r"typedef struct " + c + r" \{(.*?)\} " + c + "_t;", text, re.S).group(1)
        fields = re.findall(r"(\w+);", body)
        assert fields == [n for n, _ in cls._fields_], c


# Addresses 1 GB apart, never dereferenced.
def A(i):
    return 0x100000000 + i * 0x40000000


def block_args(**kw):
    d = dict(struct_size=160, dtype=0, M=4, N=8, gate_rows=0, h=A(0), r=A(1), w_post=A(2), gate=None,
             w_pre=A(3), s=A(4), y=A(5), rstd_post=A(6), rstd_pre=A(7), ldh=8, ldr=8, ldg=8, lds=8, ldy=8,
             eps=1e-6, offset=0.0, alpha=1.0, beta=1.0)
    d.update(kw)
    return B.BlockArgs(**d)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=8), -9), (dict(dtype=3), -3), (dict(dtype=-1), -3),
    (dict(M=-1), -2), (dict(N=0), -2), (dict(N=(1 << 31) + 1), -2), (dict(M=1 << 47), -2),
    (dict(ldh=7), -2), (dict(ldr=0), -2), (dict(lds=-8), -2), (dict(ldy=7), -2),
    (dict(M=1 << 20, ldh=1 << 40), -2),
    (dict(gate_rows=1), -2),                       # rows per gate row without a gate
    (dict(gate=A(8)), -2),                         # a gate without rows
    (dict(gate=A(8), gate_rows=-1), -2), (dict(gate=A(8), gate_rows=2, ldg=7), -2),
    (dict(eps=-1.0), -4), (dict(eps=NAN), -4), (dict(offset=INF), -4), (dict(alpha=NAN), -4),
    (dict(beta=INF), -4),
    (dict(h=None), -1), (dict(r=None), -1), (dict(s=None), -1),
    (dict(w_post=None, w_pre=None, y=None), -1),   # no norm at all
    (dict(y=None), -1), (dict(w_pre=None), -1),    # y and w_pre go together
    (dict(h=A(0) + 1), -10), (dict(gate=A(8) + 1, gate_rows=4), -10), (dict(rstd_post=A(6) + 2), -10),
    (dict(dtype=2, y=A(5) + 2), -10),
    (dict(y=A(4)), -5),                            # s and y on one place
    (dict(s=A(0) + 2), -5), (dict(y=A(1) + 16), -5),   # over an input without being it
    (dict(s=A(0), lds=16), -5),                    # on h with another stride
    (dict(s=A(2)), -5), (dict(y=A(3)), -5), (dict(gate=A(4), gate_rows=1), -5),
    (dict(rstd_post=A(0)), -5), (dict(rstd_pre=A(6)), -5), (dict(rstd_pre=A(5) + 16), -5),
])
def test_block_fwd_refusals(kw, code):
    assert B.rmsnorm_block_fwd(block_args(**kw), None, 0) == code
    assert B.rmsnorm_last_error() != ""


def test_block_fwd_without_rows_is_ok():
    assert B.rmsnorm_block_fwd(block_args(M=0, h=None, r=None, s=None, y=None, rstd_post=None,
                                          rstd_pre=None), None, 0) == 0
    assert B.rmsnorm_block_fwd(None, None, 0) == -1


@pytest.mark.parametrize("variant", ["warp", "tma", "cluster"])
def test_variants_the_operators_do_not_have(variant):
    assert B.rmsnorm_block_fwd(block_args(), B.make_options(variant=variant), 0) == -8
    o = B.make_options()
    o.struct_size = 8
    assert B.rmsnorm_block_fwd(block_args(), o, 0) == -9


def block_grads(**kw):
    d = dict(struct_size=104, reserved=0, dy=A(10), ds=A(11), dh=A(12), dr=A(13), dgate=None, dw_post=A(14),
             dw_pre=A(15), lddy=8, ldds=8, lddh=8, lddr=8, lddg=8)
    d.update(kw)
    return B.BlockGrads(**d)


@pytest.mark.parametrize("a,g,ws,code", [
    ({}, dict(struct_size=8), A(20), -9), ({}, dict(reserved=1), A(20), -9),
    ({}, dict(dy=None), A(20), -1), (dict(w_pre=None), dict(dw_pre=None), A(20), -1),
    (dict(w_pre=None), dict(dw_pre=None, dy=None, ds=None), A(20), -1),
    ({}, dict(dw_post=None), A(20), -1), (dict(w_post=None), {}, A(20), -1),
    ({}, dict(dgate=A(16)), A(20), -1), (dict(gate=A(8), gate_rows=2), {}, A(20), -1),
    ({}, dict(dh=None), A(20), -1), ({}, dict(dr=None), A(20), -1), ({}, {}, 0, -1),
    (dict(s=None), {}, A(20), -1), (dict(rstd_pre=None), {}, A(20), -1), (dict(rstd_post=None), {}, A(20), -1),
    ({}, dict(lddy=7), A(20), -2), ({}, dict(ldds=0), A(20), -2), ({}, dict(lddr=7), A(20), -2),
    (dict(gate=A(8), gate_rows=2), dict(dgate=A(16), lddg=3), A(20), -2),
    ({}, {}, A(20) + 8, -10), ({}, dict(dy=A(10) + 1), A(20), -10), ({}, dict(dw_pre=A(15) + 2), A(20), -10),
    ({}, dict(dh=A(13)), A(20), -5), ({}, dict(dh=A(10) + 16), A(20), -5), ({}, dict(dr=A(2)), A(20), -5),
    ({}, dict(dw_post=A(15)), A(20), -5), ({}, dict(dw_post=A(6)), A(20), -5),
    (dict(gate=A(8), gate_rows=1), dict(dgate=A(8)), A(20), -5),
])
def test_block_bwd_refusals(a, g, ws, code):
    assert B.rmsnorm_block_bwd(block_args(**a), block_grads(**g), ws, 1 << 40, None, 0) == code
    assert B.rmsnorm_last_error() != ""


@pytest.mark.parametrize("args,code", [((-1, 8, 0), -2), ((4, 0, 0), -2), ((4, 8, 3), -3)])
def test_block_workspace_size_refusals(args, code):
    with pytest.raises(B.RMSNormError) as e:
        B.rmsnorm_block_bwd_workspace_size(*args)
    assert e.value.status == code


def heads(ptr, T=4, H=2, D=8, batch=0):
    return B.Heads(ptr, batch, H * D, D)


def rope_args(**kw):
    d = dict(struct_size=248, dtype=0, batch=1, seq=4, heads_q=2, heads_k=2, head_dim=8, rotary_dim=8,
             interleaved=0, reserved=0, positions=A(8), positions_stride=0, steps=A(9), w_q=A(2), w_k=A(3),
             rstd_q=A(6), rstd_k=A(7), eps=1e-6, offset=0.0, magnitude=1.0, reserved_f=0.0, q=heads(A(0)),
             k=heads(A(1)), out_q=heads(A(4)), out_k=heads(A(5)))
    d.update(kw)
    return B.RopeArgs(**d)


ROPE_SHAPES = [
    (dict(struct_size=4), -9), (dict(reserved=1), -9), (dict(dtype=4), -3), (dict(batch=-1), -2),
    (dict(seq=-1), -2), (dict(heads_q=0), -2), (dict(heads_k=-1), -2), (dict(head_dim=1), -2),
    (dict(rotary_dim=7), -2), (dict(rotary_dim=0), -2), (dict(rotary_dim=10), -2), (dict(head_dim=70000), -2),
    (dict(batch=1 << 41), -2), (dict(batch=1 << 21, seq=1 << 21), -2), (dict(interleaved=2), -9),
    (dict(offset=NAN), -4), (dict(magnitude=INF), -4), (dict(steps=None), -1), (dict(steps=A(9) + 4), -10),
    (dict(positions=A(8) + 4), -10), (dict(rstd_q=A(6) + 1), -10), (dict(w_q=A(2) + 1), -10),
    (dict(positions_stride=-1), -2), (dict(positions_stride=3), -2), (dict(heads_k=0), -1),
]


@pytest.mark.parametrize("kw,code", ROPE_SHAPES + [
    (dict(eps=-1.0), -4), (dict(q=heads(None)), -1), (dict(out_k=heads(None)), -1),
    (dict(q=B.Heads(A(0), 0, -16, 8)), -2), (dict(q=B.Heads(A(0), 0, 1 << 47, 8)), -2),
    (dict(q=heads(A(0) + 1)), -10),
    (dict(out_q=B.Heads(A(4), 0, 8, 8)), -5),       # an output that lies on itself
    (dict(out_q=heads(A(5))), -5),                  # both outputs on one place
    (dict(out_q=heads(A(0) + 16)), -5), (dict(out_k=heads(A(0) + 2)), -5),
    (dict(out_k=heads(A(0))), -5), (dict(out_q=heads(A(1))), -5),   # on the other tensor
    (dict(out_q=heads(A(8))), -5), (dict(out_q=heads(A(2))), -5), (dict(rstd_q=A(0)), -5),
    (dict(rstd_q=A(7)), -5), (dict(out_q=B.Heads(A(0), 0, 32, 8)), -5),
])
def test_rope_fwd_refusals(kw, code):
    assert B.rmsnorm_rope_fwd(rope_args(**kw), None, 0) == code
    assert B.rmsnorm_last_error() != ""


def test_rope_without_tokens_is_ok():
    assert B.rmsnorm_rope_fwd(rope_args(seq=0), None, 0) == 0
    assert B.rmsnorm_rope_fwd(rope_args(batch=0, q=heads(None)), None, 0) == 0
    assert B.rmsnorm_rope_fwd(None, None, 0) == -1


def rope_grads(**kw):
    d = dict(struct_size=152, reserved=0, dout_q=heads(A(10)), dout_k=heads(A(11)), dq=heads(A(12)),
             dk=heads(A(13)), dw_q=A(14), dw_k=A(15))
    d.update(kw)
    return B.RopeGrads(**d)


@pytest.mark.parametrize("a,g,ws,code", [(kw, {}, A(20), code) for kw, code in ROPE_SHAPES] + [
    ({}, dict(struct_size=1), A(20), -9), ({}, dict(reserved=2), A(20), -9),
    ({}, dict(dw_q=None), A(20), -1), (dict(w_k=None), {}, A(20), -1), ({}, {}, 0, -1),
    (dict(rstd_q=None), {}, A(20), -1), (dict(q=heads(None)), {}, A(20), -1),
    ({}, dict(dout_k=heads(None)), A(20), -1), ({}, dict(dq=heads(None)), A(20), -1),
    ({}, {}, A(20) + 4, -10), ({}, dict(dw_q=A(14) + 1), A(20), -10), ({}, dict(dq=heads(A(12) + 1)), A(20), -10),
    ({}, dict(dq=heads(A(0))), A(20), -5),           # dq on q, which is read for other values
    ({}, dict(dk=heads(A(10))), A(20), -5), ({}, dict(dq=heads(A(10) + 16)), A(20), -5), ({}, dict(dk=heads(A(12))), A(20), -5),
    ({}, dict(dw_q=A(15)), A(20), -5), ({}, dict(dq=B.Heads(A(12), 0, 0, 8)), A(20), -5),
])
def test_rope_bwd_refusals(a, g, ws, code):
    assert B.rmsnorm_rope_bwd(rope_args(**a), rope_grads(**g), ws, 1 << 40, None, 0) == code
    assert B.rmsnorm_last_error() != ""


def test_rope_workspace_size_refusals():
    for d in (1, 0, 65537):
        with pytest.raises(B.RMSNormError) as e:
            B.rmsnorm_rope_bwd_workspace_size(d)
        assert e.value.status == -2


def cache(**kw):
    d = dict(struct_size=64, format=0, pages=4, page_size=16, heads=2, head_dim=32, heads_first=0,
             k_codes=A(0), k_scales=A(1), v_codes=A(2), v_scales=A(3))
    d.update(kw)
    return B.CacheArgs(**d)


CACHE_SHAPES = [
    (dict(struct_size=5), -9), (dict(format=2), -3), (dict(pages=0), -2), (dict(page_size=0), -2),
    (dict(heads=0), -2), (dict(head_dim=0), -2), (dict(head_dim=65537), -2), (dict(heads_first=2), -2),
    (dict(pages=1 << 46), -2), (dict(k_codes=None), -1), (dict(k_scales=None), -1), (dict(v_codes=None), -1),
    (dict(v_scales=None), -1),
]


def kv(ptr, token=64, head=32):
    return B.Heads(ptr, 0, token, head)


@pytest.mark.parametrize("c,kw,code", [(c, {}, code) for c, code in CACHE_SHAPES] + [
    ({}, dict(dtype=3), -3), ({}, dict(T=-1), -2), ({}, dict(T=1 << 41), -2), ({}, dict(k=None), -1),
    ({}, dict(slots=0), -1), ({}, dict(slots=A(9) + 4), -10), ({}, dict(k=kv(None)), -1),
    ({}, dict(v=kv(A(6), token=-1)), -2), ({}, dict(k=kv(A(5) + 1)), -10),
    (dict(v_codes=None, v_scales=None), {}, -1),
    (dict(v_codes=A(0) + 64), {}, -5), (dict(k_scales=A(0)), {}, -5), ({}, dict(k=kv(A(0))), -5),
    ({}, dict(slots=A(1)), -5),
])
def test_cache_write_refusals(c, kw, code):
    d = dict(k=kv(A(5)), v=kv(A(6)), slots=A(9), T=3, dtype=0)
    d.update(kw)
    assert B.rmsnorm_cache_write(cache(**c), d["k"], d["v"], d["slots"], d["T"], d["dtype"], None, 0) == code
    assert B.rmsnorm_last_error() != ""


@pytest.mark.parametrize("c,kw,code", [(c, {}, code) for c, code in CACHE_SHAPES] + [
    ({}, dict(dtype=-1), -3), ({}, dict(rows=-1), -2), ({}, dict(rows=(1 << 31) + 1), -2),
    ({}, dict(sequences=-1), -2), ({}, dict(width=-1), -2), ({}, dict(width=1 << 47), -2),
    ({}, dict(k=None, v=None), -1), (dict(v_codes=None, v_scales=None), {}, -1), ({}, dict(table=0), -1),
    ({}, dict(cu=0), -1), ({}, dict(table=A(8) + 2), -10), ({}, dict(cu=A(9) + 1), -10),
    ({}, dict(starts=A(10) + 2), -10), ({}, dict(k=kv(A(5) + 1)), -10),
    ({}, dict(k=kv(A(5), token=16)), -5),         # rows of the output on one another
    ({}, dict(v=kv(A(5))), -5), ({}, dict(k=kv(A(0))), -5), ({}, dict(k=kv(A(8))), -5),
])
def test_cache_read_refusals(c, kw, code):
    d = dict(table=A(8), width=2, cu=A(9), starts=0, sequences=2, rows=5, k=kv(A(5)), v=kv(A(6)), dtype=0)
    d.update(kw)
    assert B.rmsnorm_cache_read(cache(**c), d["table"], d["width"], d["cu"], d["starts"], d["sequences"],
                                d["rows"], d["k"], d["v"], d["dtype"], None, 0) == code
    assert B.rmsnorm_last_error() != ""


def test_cache_calls_without_rows_are_ok():
    assert B.rmsnorm_cache_write(cache(), kv(None), None, 0, 0, 0, None, 0) == 0
    assert B.rmsnorm_cache_read(cache(), 0, 0, 0, 0, 0, 7, kv(A(5)), None, 0, None, 0) == 0
    assert B.rmsnorm_cache_read(cache(), 0, 0, 0, 0, 3, 0, kv(A(5)), None, 0, None, 0) == 0
