"""Rotation and append without a GPU: argument checks of the C entry points (made before any
CUDA call), frequencies in fixed point against exact arithmetic, and the binding's checks."""
import ctypes
import math

import numpy as np
import pytest

from test_dense_host import A, BAD_PAGES, CAPACITY, INVALID, _pages


@pytest.fixture(scope="module")
def dhs():
    import hierarchical_sparse_kv_int8_gb300 as m
    m.build()
    return m


def _heads(**kw):
    from hierarchical_sparse_kv_int8_gb300.dense import _Heads
    d = dict(x=A, out=A + (1 << 30), norm=A, x_token=256, x_head=128, out_token=256, out_head=128, heads=2)
    d.update(kw)
    return _Heads(*[d[n] for n, _ in _Heads._fields_])


def _rot(**kw):
    from hierarchical_sparse_kv_int8_gb300.dense import _Turns
    d = dict(turns=A, n_pairs=64, pairing=0, amplitude=1.0)
    d.update(kw)
    return _Turns(*[d[n] for n, _ in _Turns._fields_])


BAD_ROT = [dict(turns=None), dict(turns=A + 4), dict(n_pairs=0), dict(n_pairs=-4), dict(n_pairs=6),
           dict(n_pairs=68), dict(pairing=2), dict(pairing=-1), dict(amplitude=0.0),
           dict(amplitude=-1.0), dict(amplitude=math.nan), dict(amplitude=math.inf)]
BAD_HEADS = [dict(x=None), dict(x=A + 8), dict(out=A + 2), dict(norm=A + 4), dict(heads=0),
             dict(heads=-1), dict(heads=131073), dict(x_token=-256), dict(x_head=127),
             dict(out_token=252), dict(x_token=(1 << 40) + 8), dict(out_token=128), dict(out_head=0),
             dict(out=A, out_token=512),                   # in place with other strides
             dict(out=A + 64 * 2), dict(out=A + 256 * 2)]  # half a row, a token further on


def _rotate(lib, rot=None, q=None, k=None, eps=1e-6, d=128, n=3, pos=A, none=()):
    p = [None if name in none else ctypes.byref(x) for name, x in
         (("rot", rot or _rot()), ("q", q or _heads()), ("k", k or _heads()))]
    return lib.dhs_rotate(*p, eps, d, n, pos, None)


def test_rotate_refusals(dhs):
    lib = dhs.load()
    for b in BAD_ROT:
        assert _rotate(lib, rot=_rot(**b)) == INVALID, b
    for b in BAD_HEADS + [dict(out=None)]:
        assert _rotate(lib, q=_heads(**b)) == INVALID, b
        assert _rotate(lib, k=_heads(**b)) == INVALID, b
    for b in [dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(d=96), dict(d=0), dict(n=-1),
              dict(pos=None), dict(pos=A + 2), dict(none=("q", "k"))]:
        assert _rotate(lib, **b) == INVALID, b
    assert _rotate(lib, rot=_rot(n_pairs=36), d=64) == INVALID
    assert _rotate(lib, n=1 << 31) == CAPACITY
    assert _rotate(lib, n=0) == 0
    assert _rotate(lib, n=0, q=_heads(x=None)) == 0


def _append(lib, p=None, rot=None, q=None, k=None, v=A, st=(256, 128), eps=1e-6, n=4, pos=None, cu=A,
            lens=A, table=A, width=3, seqs=2, none=()):
    a = [None if name in none else ctypes.byref(x) for name, x in
         (("p", p or _pages()), ("rot", rot or _rot()), ("q", q or _heads()), ("k", k or _heads(out=None)))]
    s = None if st is None else (ctypes.c_int64 * 2)(*st)
    return lib.dhs_page_append(*a, v, s, eps, n, pos, cu, lens, table, width, seqs, None, None)


def test_append_refusals(dhs):
    lib = dhs.load()
    for b in BAD_PAGES:
        assert _append(lib, _pages(**b)) == INVALID, b
    for b in BAD_ROT:
        assert _append(lib, rot=_rot(**b)) == INVALID, b
    for b in BAD_HEADS + [dict(out=None)]:
        assert _append(lib, q=_heads(**b)) == INVALID, b
    for b in BAD_HEADS + [dict(heads=1), dict(heads=3)]:
        assert _append(lib, k=_heads(**b)) == INVALID, b
    for b in [dict(none=("p",)), dict(none=("k",)), dict(v=None), dict(v=A + 8), dict(st=(-8, 128)),
              dict(st=(256, 4)), dict(eps=-1.0), dict(eps=math.nan), dict(n=-1), dict(pos=A + 1),
              dict(cu=None), dict(cu=A + 2), dict(lens=None), dict(lens=A + 2), dict(table=None),
              dict(table=A + 1), dict(width=0), dict(width=-1), dict(seqs=-1), dict(seqs=(1 << 31) - 1024)]:
        assert _append(lib, **b) == INVALID, b
    assert _append(lib, n=1 << 31) == CAPACITY
    assert _append(lib, n=0, cu=None) == 0
    assert _append(lib, seqs=0, cu=None, lens=None, table=None) == 0


def test_turns_are_the_nearest_fixed_point_numbers(dhs):
    """round(f / 2 pi 2^64) mod 2^64; at most 2^-13 of a unit from the middle of two may go
    either way, which none of these is."""
    from fractions import Fraction as F
    from oracle import dense_oracle as oracle
    lib = dhs.load()
    rng = np.random.default_rng(1)
    f = np.concatenate([[0.0, -0.0, 1.0, -1.0, 2 * math.pi, math.pi, 4294967295.0, 2.0 ** 32 - 2.0 ** -21,
                         5e-324, 2.0 ** -64, 2.0 ** -62, 2.0 ** -60, 1e-300, 0.1, 1 / 3],
                        rng.standard_normal(200) * 10.0 ** rng.uniform(-20, 9, 200),
                        10000.0 ** (-np.arange(64) / 64)])
    f = f[np.abs(f) < 2.0 ** 32]
    got = np.zeros(len(f), np.uint64)
    assert lib.dhs_rotation_turns(f.ctypes.data, len(f), got.ctypes.data) == 0
    for x, t in zip(f, got):
        want = oracle.turns(x) * 2 ** 64
        off = (F(int(t)) - want) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        assert off <= F(1, 2) + F(1, 8192), (x, float(off))


def test_turns_refusals(dhs):
    lib = dhs.load()
    t = np.zeros(2, np.uint64)
    for bad in (math.inf, -math.inf, math.nan, 2.0 ** 32, -2.0 ** 32):
        f = np.array([1.0, bad])
        assert lib.dhs_rotation_turns(f.ctypes.data, 2, t.ctypes.data) == INVALID
        assert not t.any()
    assert lib.dhs_rotation_turns(None, 2, t.ctypes.data) == INVALID
    assert lib.dhs_rotation_turns(t.ctypes.data, 2, None) == INVALID
    assert lib.dhs_rotation_turns(t.ctypes.data, -1, t.ctypes.data) == INVALID
    assert lib.dhs_rotation_turns(None, 0, None) == 0


def test_binding_refuses_cpu_tensors(dhs):
    import torch
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dhs.rotate(x, None, None, None, x, None)
    with pytest.raises(ValueError):
        dhs.rotate(None, None, None, None, None, None)
    with pytest.raises(ValueError):
        dhs.Rotation(torch.zeros((2, 4), dtype=torch.float64), device="cpu")
    with pytest.raises(ValueError):
        dhs.Rotation(torch.zeros(4, dtype=torch.float64), pairing=2, device="cpu")
    with pytest.raises(ValueError):
        dhs.Rotation(torch.zeros(4, dtype=torch.float64), device="cpu")


@pytest.mark.parametrize("of", [list, tuple, np.asarray, lambda f: [np.float64(x) for x in f]])
def test_rotation_takes_frequencies_in_64_bits(dhs, of):
    """Python's numbers keep their 64 bits.  (Without a GPU a Rotation is refused after its turns
    are made.)"""
    import torch
    f = (10000.0 ** (-np.arange(32) / 32)).tolist()
    want, held = np.zeros(32, np.uint64), np.asarray(f)
    assert dhs.load().dhs_rotation_turns(held.ctypes.data, 32, want.ctypes.data) == 0
    rot = dhs.Rotation.__new__(dhs.Rotation)
    with pytest.raises(ValueError):
        rot.__init__(of(f), device="cpu")
    assert np.array_equal(rot.turns.numpy().view(np.uint64), want)
    # a tensor of fewer bits is taken as it is
    low = torch.tensor(f, dtype=torch.float32)
    with pytest.raises(ValueError):
        rot.__init__(low, device="cpu")
    held = low.double()
    assert dhs.load().dhs_rotation_turns(held.data_ptr(), 32, want.ctypes.data) == 0
    assert np.array_equal(rot.turns.numpy().view(np.uint64), want)
