"""Refusals of the prompt and cache operators without a GPU: the library's host
checks (fake device addresses, no CUDA call on these paths) and the binding's
checks of tensors."""

import ctypes
import subprocess

import pytest
import torch

from speculative_decoding_tree_sv_gb300 import binding as sv
from speculative_decoding_tree_sv_gb300 import build

A = 1 << 20  # a 16-byte aligned address that is never used


@pytest.fixture(scope="module")
def lib():
    build.build()
    return sv.load()


def chunk(**over):
    p = sv.sv_chunk_params()
    kw = dict(batch=2, num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16, num_pages=100, total_tokens=40,
              max_tokens=39, max_pages_per_seq=20, dtype=0, window_tokens=0, sink_tokens=0, sm_scale=0.0, flags=0,
              q_stride=0, out_stride=0, q=A, k_cache=A, v_cache=A, block_table=A, ctx_lens=A, cu_tokens=A, out=A,
              lse=None, workspace=A, workspace_bytes=1 << 40)
    kw.update(over)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,status", [
    (dict(q=None), 1), (dict(k_cache=None), 1), (dict(v_cache=None), 1), (dict(block_table=None), 1),
    (dict(ctx_lens=None), 1), (dict(cu_tokens=None), 1), (dict(out=None), 1),
    (dict(q=A + 8), 1), (dict(k_cache=A + 2), 1), (dict(out=A + 4), 1), (dict(workspace=A + 8), 1),
    (dict(batch=0), 1), (dict(batch=65536), 2), (dict(num_kv_heads=0), 1), (dict(num_q_heads=30), 1),
    (dict(num_q_heads=129, num_kv_heads=1), 2), (dict(head_dim=96), 2), (dict(head_dim=256), 2),
    (dict(page_size=32), 2), (dict(num_pages=0), 1), (dict(max_pages_per_seq=0), 1),
    (dict(max_pages_per_seq=1 << 27), 2), (dict(total_tokens=-1), 1), (dict(total_tokens=(1 << 30) + 1), 2), (dict(max_tokens=-1), 1),
    (dict(dtype=2), 2), (dict(dtype=-1), 2), (dict(window_tokens=-1), 1), (dict(sink_tokens=-1), 1),
    (dict(window_tokens=(1 << 28) + 1), 2), (dict(flags=1), 1), (dict(sm_scale=float("nan")), 1),
    (dict(sm_scale=float("inf")), 1), (dict(q_stride=4095), 1), (dict(q_stride=4096 + 4), 1),
    (dict(out_stride=4088), 1), (dict(workspace=None), 4), (dict(workspace_bytes=300), 4),
])
def test_chunk_attention_refuses(lib, over, status):
    assert lib.sv_chunk_attention(ctypes.byref(chunk(**over)), None) == status


def test_chunk_attention_nothing_to_do_and_null(lib):
    assert lib.sv_chunk_attention(None, None) == 1
    assert lib.sv_chunk_attention(ctypes.byref(chunk(total_tokens=0)), None) == 0
    assert lib.sv_chunk_attention(ctypes.byref(chunk(max_tokens=0)), None) == 0
    n = ctypes.c_size_t(0)
    assert lib.sv_chunk_attention_workspace_size(None, ctypes.byref(n)) == 1
    assert lib.sv_chunk_attention_workspace_size(ctypes.byref(chunk()), None) == 1


def test_chunk_workspace_holds_the_partials_of_each_kernel(lib):
    rows = 152 * 8 * 2 * 16 * (128 * 4 + 4)     # every warp: two pieces of 16 rows
    tiles = 152 * 2 * 256 * (128 * 4 + 4)       # every CTA: two pieces of 256 rows
    size = sv.sv_chunk_attention_workspace_size
    one = size(chunk(total_tokens=2, max_tokens=1))        # single tokens: the row kernel alone
    assert rows <= one <= rows + 8192
    mixed = size(chunk())
    assert rows + tiles <= mixed <= rows + tiles + 16384
    long = size(chunk(batch=1, total_tokens=39))           # one chunk: the tile kernel alone
    assert tiles <= long <= tiles + 16384
    # 32 rows per token: either kernel, by the size of the cache that the table's width allows
    either = size(chunk(num_q_heads=32, num_kv_heads=1, total_tokens=2, max_tokens=1))
    assert rows + tiles <= either <= rows + tiles + 16384
    assert size(chunk(num_q_heads=32, num_kv_heads=1, total_tokens=2, max_tokens=1, max_pages_per_seq=200000)) == either


def test_append_refuses(lib):
    def call(**over):
        kw = dict(k=A, v=A, ts=1024, ls=0, kc=A, vc=A, cs=0, layers=1, pages=10, bt=A, width=4, ctx=A, cu=A, batch=2,
                  total=5, heads=8, d=128, page=16, new=None, ws=None, wsb=0)
        kw.update(over)
        return lib.sv_kv_append(*kw.values(), None)

    for name in ("k", "v", "kc", "vc", "bt", "ctx", "cu"):
        assert call(**{name: None}) == 1
    for name in ("k", "v", "kc", "vc"):
        assert call(**{name: A + 8}) == 1
    for bad in (dict(layers=0), dict(pages=0), dict(width=0), dict(batch=0), dict(total=-1), dict(heads=0), dict(page=0),
                dict(ts=1016), dict(ts=1028), dict(ls=4), dict(ls=-8), dict(cs=4), dict(new=A)):
        assert call(**bad) == 1, bad          # (new: the context lengths themselves)
    assert call(d=12) == 2 and call(d=0) == 2 and call(layers=65536) == 2 and call(total=(1 << 30) + 1) == 2
    assert call(ws=A, wsb=255) == 4


def test_pages_refuse(lib):
    n = ctypes.c_size_t(0)
    assert lib.sv_pages_workspace_size(1, 1, ctypes.byref(n)) == 0 and n.value >= 256 + 7 * 4
    assert lib.sv_pages_workspace_size(0, 1, ctypes.byref(n)) == 1
    assert lib.sv_pages_workspace_size(1, 0, ctypes.byref(n)) == 1
    assert lib.sv_pages_workspace_size(1, 1, None) == 1
    assert lib.sv_pages_workspace_size(65536, 1, ctypes.byref(n)) == 2
    assert lib.sv_pages_workspace_size(1, (1 << 21) + 1, ctypes.byref(n)) == 2
    big = 1 << 40

    def release(**o):
        kw = {**dict(keep=A, rows=4, bt=A, width=8, held=A, refs=A, pages=10, page=16, ws=A, wsb=256), **o}
        return lib.sv_pages_release(*kw.values(), None)

    def fork(**o):
        kw = {**dict(pa=A, ch=A, n=2, bt=A, rows=4, width=8, ctx=A, held=A, refs=A, pages=10, page=16, ws=A, wsb=256), **o}
        return lib.sv_pages_fork(*kw.values(), None)

    def reserve(**o):
        kw = {**dict(ctx=A, new=A, rows=4, bt=A, width=8, held=A, refs=A, pages=10, page=16, src=A, dst=2 * A, count=A,
                     ws=A, wsb=big), **o}
        return lib.sv_pages_reserve(*kw.values(), None)

    def compact(**o):
        kw = {**dict(bt=A, held=A, rows=4, width=8, refs=A, pages=10, bto=A, refso=A, src=A, dst=2 * A, count=A, live=A,
                     ws=A, wsb=big), **o}
        return lib.sv_pages_compact(*kw.values(), None)

    for call, pointers in ((release, "keep bt held refs"), (fork, "pa ch bt ctx held refs"),
                           (reserve, "ctx new bt held refs src dst count"),
                           (compact, "bt held refs bto refso src dst count live")):
        for name in pointers.split():
            assert call(**{name: None}) == 1, (call, name)
        for bad in (dict(rows=0), dict(width=0), dict(pages=0)):
            assert call(**bad) == 1
        assert call(width=(1 << 30) + 1) == 2
        for bad in (dict(rows=65536), dict(pages=(1 << 21) + 1)):
            assert call(**bad) == 2
    assert release(page=0) == 1 and fork(page=0) == 1 and reserve(page=0) == 1
    assert fork(n=-1) == 1 and fork(n=65536) == 2 and fork(n=0) == 0
    assert release(wsb=255) == 4 and fork(wsb=255) == 4
    assert reserve(ws=None) == 4 and reserve(wsb=256) == 4 and compact(ws=None) == 4 and compact(wsb=256) == 4
    assert reserve(dst=A) == 1 and compact(dst=A) == 1    # one list for both

    def copy(**o):
        kw = {**dict(k=A, v=A, stride=0, layers=1, pages=10, elems=64, src=A, dst=A, count=A, most=3, ws=None, wsb=0), **o}
        return lib.sv_pages_copy(*kw.values(), None)

    for name in ("k", "src", "dst", "count"):
        assert copy(**{name: None}) == 1
    for bad in (dict(k=A + 8), dict(v=A + 8), dict(stride=4), dict(stride=-8), dict(layers=0), dict(pages=0),
                dict(elems=0), dict(elems=12), dict(most=-1)):
        assert copy(**bad) == 1, bad
    assert copy(layers=65536) == 2 and copy(elems=(1 << 26) + 8) == 2 and copy(ws=A, wsb=255) == 4
    assert copy(most=0) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    good = dict(q=h(5, 8, 64), k_cache=h(6, 2, 16, 64), v_cache=h(6, 2, 16, 64), block_table=i(2, 3), ctx_lens=i(2),
                cu_tokens=i(3), out=h(5, 8, 64), max_tokens=4)
    with pytest.raises(ValueError, match="device memory"):
        sv.make_chunk_params(**good)
    for bad, text in ((dict(q=h(5, 8, 64).float()), "bfloat16 or float16"), (dict(out=h(5, 8, 32)), "must both be"),
                      (dict(out=torch.zeros(5, 8, 64, dtype=torch.float16)), "out is"),
                      (dict(k_cache=h(6, 2, 16, 128), v_cache=h(6, 2, 16, 128)), "head_dim"),
                      (dict(v_cache=h(6, 2, 16, 32)), "same shape"), (dict(k_cache=h(6, 2, 64)), "a cache is"),
                      (dict(block_table=i(6)), r"\[batch, max_pages\]"), (dict(block_table=torch.zeros(2, 3)), "int32"),
                      (dict(block_table=i(3, 2).t()), "contiguous"), (dict(ctx_lens=i(3)), "2 elements"),
                      (dict(cu_tokens=i(2)), "3 elements"), (dict(lse=torch.zeros(5, 4)), "lse"),
                      (dict(q=h(5, 64, 8).transpose(1, 2)), "heads of q")):
        with pytest.raises(ValueError, match=text):
            sv.make_chunk_params(**{**good, **bad})
    with pytest.raises(ValueError, match="device memory"):
        sv.sv_kv_append(h(5, 2, 64), h(5, 2, 64), h(6, 2, 16, 64), h(6, 2, 16, 64), i(2, 3), i(2), i(3))
    with pytest.raises(ValueError, match="layers"):
        sv.sv_kv_append(h(2, 5, 2, 64), h(2, 5, 2, 64), h(3, 6, 2, 16, 64), h(3, 6, 2, 16, 64), i(2, 3), i(2), i(3))
    one = h(1, 6, 2, 16, 64).expand(3, 6, 2, 16, 64)
    with pytest.raises(ValueError, match="overlap"):
        sv.sv_kv_append(h(3, 5, 2, 64), h(3, 5, 2, 64), one, one, i(2, 3), i(2), i(3))
    with pytest.raises(ValueError, match="type"):
        sv.sv_kv_append(h(5, 2, 64).half(), h(5, 2, 64).half(), h(6, 2, 16, 64), h(6, 2, 16, 64), i(2, 3), i(2), i(3))
    with pytest.raises(ValueError, match="same shape and strides"):
        sv.sv_kv_append(h(5, 2, 64), h(6, 2, 64), h(6, 2, 16, 64), h(6, 2, 16, 64), i(2, 3), i(2), i(3))
    with pytest.raises(ValueError, match="device memory"):
        sv.sv_pages_release(i(2), i(2, 3), i(2), i(9))
    with pytest.raises(ValueError, match="device memory"):
        sv.sv_pages_fork(i(1), i(1), i(2, 3), i(2), i(2), i(9))
    with pytest.raises(ValueError, match="room for 2"):
        sv.sv_pages_reserve(i(2), i(2), i(2, 3), i(2), i(9), i(1), i(2), i(1))
    with pytest.raises(ValueError, match="room for 4"):
        sv.sv_pages_compact(i(2, 3), i(2), i(9), i(2, 3), i(9), i(4), i(3), i(1), i(1))
    with pytest.raises(ValueError, match="copy_count"):
        sv.sv_pages_copy(h(6, 2, 16, 64), None, i(3), i(3), i(2))
    with pytest.raises(ValueError, match="held_pages"):
        sv.sv_pages_release(i(2), i(2, 3), i(3), i(9))


STRIDED = r"""
#include "strided.h"
extern "C" int walk(unsigned block, unsigned blocks, unsigned thread, int length, int most, long long* out) {
  const sv::Strided s = sv::strided(block, blocks, 256, thread);
  int n = 0;
  for (long long b = s.first; b < length && n < most; b += s.step) out[n++] = b;
  return n;
}
"""


def test_append_takes_each_length_once_whatever_the_token_rows(tmp_path):
    """The lengths are dealt to the threads of a grid that the token rows size, up
    to 2^30 rows: every entry once, none outside the arrays, and no thread that
    never ends."""
    source, module = tmp_path / "walk.cpp", tmp_path / "walk.so"
    source.write_text(STRIDED)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, "-o", module, source], check=True)
    walk = ctypes.CDLL(str(module)).walk
    walk.argtypes = [ctypes.c_uint, ctypes.c_uint, ctypes.c_uint, ctypes.c_int, ctypes.c_int,
                     ctypes.POINTER(ctypes.c_longlong)]
    out = (ctypes.c_longlong * 4096)()
    for rows in (0, 1, 8, 9, 5000, (1 << 26) - 8, 1 << 26, (1 << 26) + 1, (1 << 27) - 1, 1 << 27, (1 << 28) + 9, 1 << 30):
        blocks = max(1, -(-rows // 8))
        for batch in (1, 255, 256, 257, 2000):
            near = set(range(min(blocks, 9))) | {blocks - 1, blocks // 2}
            near |= {b for at in (1 << 23, 1 << 24, 1 << 25, 1 << 26) for b in (at - 1, at, at + 1) if b < blocks}
            taken = []
            for block in near:
                for thread in range(256):
                    n = walk(block, blocks, thread, batch, len(out), out)
                    taken += out[:n]
            assert sorted(taken) == list(range(batch)), (rows, batch)


def chunk_tensors():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    return dict(q=h(5, 8, 64), k_cache=h(6, 2, 16, 64), v_cache=h(6, 2, 16, 64), block_table=i(2, 3), ctx_lens=i(2),
                cu_tokens=i(3), out=h(5, 8, 64), max_tokens=4)


@pytest.mark.parametrize("name", ["q", "out"])
def test_rows_that_overlap_are_refused(name):
    """A broadcast row has token stride 0, which the parameters read as dense."""
    good = chunk_tensors()
    rows = torch.zeros(5 * 512 + 512, dtype=torch.bfloat16)
    for stride in (0, 8, 504):
        with pytest.raises(ValueError, match=f"rows of {name} overlap"):
            sv.make_chunk_params(**{**good, name: rows.as_strided((5, 8, 64), (stride, 64, 1))})
    for t in (rows.as_strided((5, 8, 64), (520, 64, 1)), rows[:512].view(1, 8, 64).expand(1, 8, 64)):
        other = {k: torch.zeros_like(t) for k in ("q", "out")}
        with pytest.raises(ValueError, match="device memory"):   # (past the check of strides)
            sv.make_chunk_params(**{**good, **other, name: t})


def test_what_writes_the_context_signals_nothing_early():
    """sv.h says of SV_ATTN_EARLY_CONTEXT that the library's kernels never write
    tables, lengths or context pages behind an early signal: an attention that
    starts at the signal would read them half written."""
    for name in ("kv_append.cu", "pages.cu", "kv_commit.cu"):
        with open(f"{build.CSRC}/{name}") as f:
            source = f.read()
        assert "griddep_wait();" in source and "launch_dependents" not in source, name


@pytest.mark.parametrize("off", [1, 2, 3])
def test_workspaces_off_their_words_are_refused(lib, off):
    """The error word and the scratch are 32-bit words: a byte offset that is no
    multiple of four would be a misaligned access on the device."""
    size = 1 << 40
    append = lambda w: lib.sv_kv_append(A, A, 1024, 0, A, A, 0, 1, 10, A, 4, A, A, 2, 5, 8, 128, 16, None, w, size, None)  # noqa: E731
    release = lambda w: lib.sv_pages_release(A, 4, A, 8, A, A, 10, 16, w, size, None)  # noqa: E731
    fork = lambda w: lib.sv_pages_fork(A, A, 2, A, 4, 8, A, A, A, 10, 16, w, size, None)  # noqa: E731
    reserve = lambda w: lib.sv_pages_reserve(A, A, 4, A, 8, A, A, 10, 16, A, 2 * A, A, w, size, None)  # noqa: E731
    compact = lambda w: lib.sv_pages_compact(A, A, 4, 8, A, 10, A, A, A, 2 * A, A, A, w, size, None)  # noqa: E731
    copy = lambda w: lib.sv_pages_copy(A, A, 0, 1, 10, 64, A, A, A, 3, w, size, None)  # noqa: E731
    for call in (append, release, fork, reserve, compact, copy):
        assert call(A + off) == 1


def test_empty_tensors_have_no_address(lib):
    """A call without token rows, or with an empty list, is a call that has nothing
    to do, not a null pointer."""
    empty = chunk(total_tokens=0, q=None, out=None)
    n = ctypes.c_size_t(0)
    assert lib.sv_chunk_attention_workspace_size(ctypes.byref(empty), ctypes.byref(n)) == 0 and n.value >= 256
    assert lib.sv_chunk_attention(ctypes.byref(empty), None) == 0
    assert lib.sv_chunk_attention(ctypes.byref(chunk(max_tokens=0, q=None)), None) == 1
    copy = lambda src, dst, most: lib.sv_pages_copy(A, A, 0, 1, 10, 64, src, dst, A, most, None, 0, None)  # noqa: E731
    assert copy(None, None, 0) == 0 and copy(None, A, 1) == 1 and copy(A, None, 1) == 1
    if torch.cuda.is_available():
        return  # the append launches, for the lengths: with real tensors in the GPU tests
    append = lambda k, v, total: lib.sv_kv_append(k, v, 1024, 0, A, A, 0, 1, 10, A, 4, A, A, 2, total, 8, 128, 16, None,  # noqa: E731
                                                  None, 0, None)
    assert append(None, None, 0) == 3 and append(None, A, 1) == 1 and append(A, None, 1) == 1  # 3: no device to launch on


@pytest.mark.parametrize("name", ["max_tokens", "window_tokens", "sink_tokens"])
def test_counts_past_32_bits_are_refused(name):
    """ctypes would keep the low 32 bits: 2^32 + 5 would be a window of 5."""
    for value in (1 << 31, (1 << 32) + 5, -(1 << 31) - 1):
        with pytest.raises(ValueError, match=f"{name} does not fit 32 bits"):
            sv.make_chunk_params(**{**chunk_tensors(), name: value})
