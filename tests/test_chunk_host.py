"""Chunk attention without a GPU: argument checks of the C entry points, made before any CUDA
call."""
import ctypes
import math

import pytest

from test_dense_host import A, BAD_PAGES, INVALID, _pages


@pytest.fixture(scope="module")
def dhs():
    import hierarchical_sparse_kv_int8_gb300 as m
    m.build()
    return m


def _chunk(lib, p=None, q=A, st=None, n=4, cu=A, lens=A, table=A, width=3, seqs=2, hq=8, window=0,
           sinks=0, scale=0.0, out=A, lse=A, ws=A, nbytes=1 << 40, err=None, none=False):
    s = None if st is None else (ctypes.c_int64 * 2)(*st)
    return lib.dhs_page_chunk(None if none else ctypes.byref(p or _pages()), q, s, n, cu, lens, table, width,
                              seqs, hq, window, sinks, scale, out, lse, ws, nbytes, err, None)


def test_chunk_refusals(dhs):
    lib = dhs.load()
    for b in BAD_PAGES:
        assert _chunk(lib, _pages(**b)) == INVALID, b
        assert lib.dhs_page_chunk_workspace(ctypes.byref(_pages(**b)), 4, 2, 8) == -1
    for b in [dict(none=True), dict(q=None), dict(q=A + 8), dict(st=(-8, 128)), dict(st=(1028, 128)),
              dict(st=(1024, 64)), dict(st=(64, 128)), dict(st=(1 << 38, 128)), dict(n=-1),
              dict(n=(1 << 31) - 256), dict(cu=None), dict(cu=A + 2), dict(lens=None), dict(lens=A + 1),
              dict(table=None), dict(table=A + 2), dict(width=0), dict(width=-1), dict(seqs=-1),
              dict(seqs=(1 << 31) - 1024), dict(hq=0), dict(hq=7), dict(hq=2 * 129), dict(window=-1),
              dict(window=5, sinks=-1), dict(sinks=4), dict(scale=-1.0), dict(scale=math.nan),
              dict(scale=2e38), dict(out=None), dict(out=A + 8), dict(lse=A + 2), dict(ws=None),
              dict(ws=A + 8), dict(nbytes=-1), dict(err=A + 2)]:
        assert _chunk(lib, **b) == INVALID, b
    assert _chunk(lib, n=0, q=None, out=None) == 0
    assert _chunk(lib, seqs=0, cu=None, lens=None, table=None) == 0
    p = ctypes.byref(_pages())
    for bad in ((-1, 2, 8), (4, -1, 8), (4, 2, 0), (4, 2, 7), (4, 2, 258), ((1 << 31) - 256, 2, 8)):
        assert lib.dhs_page_chunk_workspace(p, *bad) == -1, bad


def _window(lib, p=None, q=A, ql=None, lens=A, table=A, width=3, seqs=2, q_len=2, hq=8, window=9, sinks=0,
            scale=0.0, out=A, lse=A, ws=A, nbytes=1 << 40, err=None):
    return lib.dhs_page_attend_window(ctypes.byref(p or _pages()), q, ql, lens, table, width, seqs, q_len, hq,
                                      window, sinks, scale, out, lse, ws, nbytes, err, None)


def test_window_refusals(dhs):
    lib = dhs.load()
    for b in BAD_PAGES:
        assert _window(lib, _pages(**b)) == INVALID, b
    for b in [dict(q=None), dict(q=A + 8), dict(ql=A + 2), dict(lens=None), dict(lens=A + 2),
              dict(table=None), dict(width=-1), dict(seqs=-1), dict(q_len=0), dict(q_len=9), dict(hq=7),
              dict(hq=0), dict(hq=2 * 65), dict(window=0), dict(window=-3), dict(sinks=-1),
              dict(scale=-1.0), dict(scale=math.nan), dict(out=None), dict(out=A + 8), dict(lse=A + 1),
              dict(ws=None), dict(ws=A + 8), dict(nbytes=-1), dict(err=A + 2)]:
        assert _window(lib, **b) == INVALID, b
    assert _window(lib, seqs=0, q=None, lens=None) == 0
