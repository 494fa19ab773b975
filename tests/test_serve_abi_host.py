"""Host-only checks of the entry points that serve from the cache: struct layouts against the
header, and refusals before any CUDA call. Pointers here are never dereferenced."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from memory_bound_normalization_fwd_gb300 import binding as B
from memory_bound_normalization_fwd_gb300 import build as BUILD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"rmsnorm_rope_axes": (B.RopeAxesArgs, B._AXES), "rmsnorm_cache_pages": (B.PagesArgs, B._PAGES),
           "rmsnorm_cache_attention_args": (B.AttentionArgs, B._ATTENTION)}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    BUILD.build()
    return B.lib()


def test_struct_layouts_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not installed")
    lines = []
    for c, (cls, packed) in STRUCTS.items():
        assert packed.size == ctypes.sizeof(cls), c
        lines.append(f'    printf("{c} size %zu\\n", sizeof({c}_t));')
        lines += [f'    printf("{c} {n} %zu\\n", offsetof({c}_t, {n}));' for n, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include "rmsnorm.h"\n#include <stddef.h>\n#include <stdio.h>\n'
                   "int main(void) {\n" + "\n".join(lines) + "\n    return 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out.splitlines() if line.strip()}
    for c, (cls, _) in STRUCTS.items():
        assert got[(c, "size")] == ctypes.sizeof(cls), c
        for n, _ in cls._fields_:
            assert got[(c, n)] == getattr(cls, n).offset, (c, n)


# Addresses 1 GB apart, never dereferenced.
def A(i):
    return 0x100000000 + i * 0x40000000


def cache(**kw):
    d = dict(struct_size=64, format=1, pages=10, page_size=16, heads=2, head_dim=64, heads_first=0,
             k_codes=A(0), k_scales=A(1), v_codes=A(2), v_scales=A(3))
    d.update(kw)
    return B.CacheArgs(**d)


def heads(i, token=512, head=64):
    return B.Heads(A(i), 0, token, head)


def attention(**kw):
    d = dict(struct_size=152, dtype=0, heads_q=8, causal=1, sequences=3, rows=3, table_width=4, window=0,
             table=A(4), lengths=A(5), cu_rows=A(6), lse=A(7), scale=0.1, reserved=0.0, q=heads(8), out=heads(9))
    d.update(kw)
    return B.AttentionArgs(**d)


BIG = 1 << 36


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=0), -9), (dict(reserved=1.0), -9), (dict(dtype=3), -3), (dict(heads_q=7), -2),
    (dict(heads_q=0), -2), (dict(heads_q=-2), -2), (dict(causal=2), -9), (dict(window=-1), -2),
    (dict(window=5, causal=0), -2), (dict(scale=NAN), -4), (dict(scale=INF), -4), (dict(sequences=-1), -2),
    (dict(rows=-1), -2), (dict(rows=1 << 40), -2), (dict(table_width=-1), -2), (dict(table_width=1 << 40), -2),
    (dict(cu_rows=None, rows=4), -2), (dict(lengths=None), -1), (dict(table=None), -1), (dict(table=A(4) + 2), -10),
    (dict(lengths=A(5) + 1), -10), (dict(cu_rows=A(6) + 2), -10), (dict(lse=A(7) + 2), -10),
    (dict(q=B.Heads(None, 0, 512, 64)), -1), (dict(out=B.Heads(None, 0, 512, 64)), -1),
    (dict(q=B.Heads(A(8) + 1, 0, 512, 64)), -10), (dict(q=heads(8, token=-512)), -2),
    (dict(out=heads(9, token=32, head=64)), -5),          # out's rows lie on one another
    (dict(out=heads(8)), -5), (dict(out=heads(0)), -5), (dict(lse=A(9)), -5), (dict(lse=A(5)), -5),
    (dict(out=heads(4)), -5),
])
def test_attention_refusals(kw, code):
    assert B.rmsnorm_cache_attention(cache(), attention(**kw), A(12), BIG, None, 0) == code


@pytest.mark.parametrize("kw,code", [
    (dict(struct_size=1), -9), (dict(format=2), -3), (dict(pages=0), -2), (dict(page_size=0), -2),
    (dict(heads=0), -2), (dict(head_dim=0), -2), (dict(head_dim=513), -2), (dict(v_codes=None, v_scales=None), -1),
    (dict(v_codes=None), -1), (dict(k_scales=None), -1), (dict(heads=3), -2), (dict(heads_first=2), -2),
])
def test_attention_refuses_the_cache(kw, code):
    assert B.rmsnorm_cache_attention(cache(**kw), attention(), A(12), BIG, None, 0) == code


def test_attention_of_nothing_is_taken():
    assert B.rmsnorm_cache_attention(cache(), attention(rows=0), 0, 0, None, 0) == 0
    assert B.rmsnorm_cache_attention(cache(), attention(sequences=0), 0, 0, None, 0) == 0
    assert B.rmsnorm_cache_attention(None, attention(), 0, 0, None, 0) == -1
    assert B.rmsnorm_cache_attention(cache(), None, 0, 0, None, 0) == -1


def pages(**kw):
    d = dict(struct_size=56, reserved=0, pages=10, sequences=4, table_width=5, refs=A(4), table=A(5), lengths=A(6))
    d.update(kw)
    return B.PagesArgs(**d)


PAGES = [(dict(struct_size=8), -9), (dict(reserved=1), -9), (dict(pages=0), -2), (dict(pages=(1 << 25) + 1), -2),
         (dict(sequences=-1), -2), (dict(sequences=(1 << 30) + 1), -2), (dict(table_width=-1), -2),
         (dict(refs=None), -1), (dict(table=None), -1), (dict(refs=A(4) + 1), -10), (dict(table=A(5) + 2), -10),
         (dict(refs=A(5)), -5)]


@pytest.mark.parametrize("kw,code", PAGES + [(dict(lengths=None), -1), (dict(lengths=A(6) + 2), -10),
                                             (dict(lengths=A(5)), -5), (dict(pages=11), -2)])
def test_fork_refusals(kw, code):
    assert B.rmsnorm_cache_fork(cache(), pages(**kw), A(7), A(8), 3, A(12), BIG, None, 0) == code


@pytest.mark.parametrize("kw,code", PAGES + [(dict(lengths=None), -1), (dict(lengths=A(5)), -5)])
def test_free_refusals(kw, code):
    assert B.rmsnorm_cache_free(pages(**kw), A(7), 3, None, 0) == code


@pytest.mark.parametrize("kw,code", [(k, c) for k, c in PAGES if k != dict(refs=A(5))] + [(dict(pages=11), -2)])
def test_compact_refusals(kw, code):
    assert B.rmsnorm_cache_compact(cache(), pages(**kw), A(9), A(10), A(11), A(12), BIG, None, 0) == code


def test_arguments_beside_the_structs():
    fork, free, comp = B.rmsnorm_cache_fork, B.rmsnorm_cache_free, B.rmsnorm_cache_compact
    assert fork(cache(), pages(), 0, A(8), 3, A(12), BIG, None, 0) == -1
    assert fork(cache(), pages(), A(7), 0, 3, A(12), BIG, None, 0) == -1
    assert fork(cache(), pages(), A(7), A(8), -1, A(12), BIG, None, 0) == -2
    assert fork(cache(), pages(), A(7) + 2, A(8), 3, A(12), BIG, None, 0) == -10
    assert fork(cache(), pages(), A(5), A(8), 3, A(12), BIG, None, 0) == -5      # parents in the table
    assert fork(cache(), pages(), A(7), A(8), 3, 0, BIG, None, 0) == -1
    assert fork(cache(), pages(), A(7), A(8), 3, A(12) + 8, BIG, None, 0) == -10
    assert fork(cache(), pages(), A(7), A(8), 3, A(12), 16, None, 0) == -11
    assert fork(cache(), pages(), A(7), A(8), 3, A(5), BIG, None, 0) == -5       # the workspace on the table
    assert fork(cache(), pages(), A(7), A(8), 3, A(7), BIG, None, 0) == -5
    assert fork(cache(), pages(), 0, 0, 0, 0, 0, None, 0) == 0
    assert free(pages(), 0, 2, None, 0) == -1 and free(pages(), A(7), -2, None, 0) == -2
    assert free(pages(), A(4), 2, None, 0) == -5 and free(pages(), 0, 0, None, 0) == 0
    assert comp(cache(), pages(), 0, A(10), A(11), A(12), BIG, None, 0) == -1
    assert comp(cache(), pages(), A(9), 0, A(11), A(12), BIG, None, 0) == -1
    assert comp(cache(), pages(), A(9), A(10), 0, A(12), BIG, None, 0) == -1
    assert comp(cache(), pages(), A(4) + 4, A(10), A(11), A(12), BIG, None, 0) == -5  # on refs, not equal to it
    assert comp(cache(), pages(), A(5), A(10), A(11), A(12), BIG, None, 0) == -5      # refs_out on the table
    assert comp(cache(), pages(), A(9), A(9), A(11), A(12), BIG, None, 0) == -5
    assert comp(cache(), pages(), A(9), A(10), A(11), A(12), 16, None, 0) == -11
    assert comp(cache(), pages(), A(9), A(10), A(11), A(9), BIG, None, 0) == -5
    copy = B.rmsnorm_cache_copy_pages
    assert copy(cache(), 0, A(5), 2, None, 0) == -1 and copy(cache(), A(4), 0, 2, None, 0) == -1
    assert copy(cache(), A(4), A(5), -1, None, 0) == -2 and copy(cache(), A(4) + 1, A(5), 2, None, 0) == -10
    assert copy(cache(), A(0), A(5), 2, None, 0) == -5 and copy(cache(), 0, 0, 0, None, 0) == 0
    assert copy(cache(k_codes=None), A(4), A(5), 2, None, 0) == -1
    assert copy(cache(k_codes=A(1)), A(4), A(5), 2, None, 0) == -5


def test_workspace_sizes_on_the_host():
    size = B.rmsnorm_cache_pages_workspace_size
    assert size(10, 4, 3) >= (2 * 3 + 4 + 3) * 4 and size(5000, 0, 0) >= 5000 // 8
    for args in ((0, 0, 0), ((1 << 25) + 1, 0, 0), (5, -1, 0), (5, 0, -1)):
        with pytest.raises(B.RMSNormError):
            size(*args)
    n = ctypes.c_int64()
    for args in ((2, 7, 64, 1, 1), (2, 8, 513, 1, 1), (0, 8, 64, 1, 1), (2, 8, 64, -1, 1)):
        assert B.lib().rmsnorm_cache_attention_workspace_size(*args, ctypes.byref(n)) == -2
    assert B.lib().rmsnorm_cache_attention_workspace_size(2, 8, 64, 1, 1, None) == -1


def rope(**kw):
    d = dict(struct_size=248, dtype=0, batch=2, seq=3, heads_q=4, heads_k=0, head_dim=64, rotary_dim=32,
             interleaved=0, reserved=0, positions=A(0), positions_stride=3, steps=A(1), w_q=None, w_k=None,
             rstd_q=None, rstd_k=None, eps=1e-6, offset=0.0, magnitude=1.0, reserved_f=0.0,
             q=B.Heads(A(2), 768, 256, 64), out_q=B.Heads(A(3), 768, 256, 64))
    d.update(kw)
    return B.RopeArgs(**d)


def axes(pairs=(6, 5, 5), **kw):
    d = dict(struct_size=40, axes=len(pairs), in_turn=0, reserved=0, axis_stride=6)
    d.update(kw)
    return B.RopeAxesArgs(pairs=(ctypes.c_int32 * 4)(*(pairs + (0,) * (4 - len(pairs)))), **d)


@pytest.mark.parametrize("x,kw,code", [
    (axes(struct_size=8), {}, -9), (axes(reserved=1), {}, -9), (axes(in_turn=2), {}, -9), (axes(axes=0), {}, -2),
    (axes(axes=5), {}, -2), (axes((6, 5, 4)), {}, -2), (axes((6, 5, 6)), {}, -2), (axes((18, -1, -1)), {}, -2),
    (axes((6, 5, 5), axes=2), {}, -2), (axes((1, 15), in_turn=1), {}, -2), (axes((4, 6, 6), in_turn=1), {}, -2),
    (axes(axis_stride=-1), {}, -2), (axes(axis_stride=1 << 50), {}, -2), (axes(), dict(positions=None), -1),
    (axes(), dict(out_q=B.Heads(A(0), 768, 256, 64)), -5),
    (axes(axis_stride=0x40000000 // 8 * 3), dict(positions=A(0)), -5),  # the second axis lies on the output
    (axes(), dict(struct_size=4), -9), (axes(), dict(rotary_dim=30), -2),
])
def test_axes_refusals(x, kw, code):
    assert B.rmsnorm_rope_axes_fwd(rope(**kw), x, None, 0) == code
    if code != -5:
        grads = B.RopeGrads(struct_size=152, reserved=0, dout_q=B.Heads(A(2), 768, 256, 64),
                            dq=B.Heads(A(3), 768, 256, 64))
        assert B.rmsnorm_rope_axes_bwd(rope(**kw), x, grads, 0, 0, None, 0) == code


def test_axes_that_are_not_given():
    assert B.rmsnorm_rope_axes_fwd(rope(), None, None, 0) == -1
    assert B.rmsnorm_rope_axes_bwd(rope(), None, None, 0, 0, None, 0) == -1
    assert B.rmsnorm_rope_axes_fwd(rope(seq=0, positions=None), axes(), None, 0) == 0
    for pairs in ((), (1, 2, 3, 4, 5), (3, -1)):
        with pytest.raises(ValueError):
            B.RopeAxes(pairs)
    for a, dim in ((B.RopeAxes((4, 4), True), 16), (B.RopeAxes((4, 4)), 20)):
        with pytest.raises(ValueError):
            B.rope_steps(dim, device="cpu", axes=a)
