"""Paged-cache and prompt operators without a GPU: argument checks of the C
entry points (made before any CUDA call), the binding's checks, and the oracle's
quantisation against brute force."""
import ctypes

import numpy as np
import pytest

INVALID, CAPACITY = 1, 3
A = 4096  # an aligned address nobody dereferences


@pytest.fixture(scope="module")
def dhs():
    import hierarchical_sparse_kv_int8_gb300 as m
    m.build()
    return m


def _pages(**kw):
    from hierarchical_sparse_kv_int8_gb300.dense import Pages
    d = dict(k=A, v=A, k_scale=A, v_scale=A, n_pages=8, page_rows=64, kv_heads=2, head_dim=128, kind=1)
    d.update(kw)
    return Pages(*[d[n] for n, _ in Pages._fields_])


BAD_PAGES = [dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 2), dict(k_scale=None),
             dict(v_scale=None), dict(n_pages=0), dict(n_pages=1 << 31), dict(page_rows=0), dict(kv_heads=0),
             dict(kv_heads=1025), dict(head_dim=96), dict(head_dim=0), dict(kind=3), dict(kind=-1)]


def _copy(lib, name, p=None, k=A, v=A, strides=None, n=4, cu=A, lens=A, table=A, width=3, seqs=2):
    p = p if p is not None else _pages()
    st = None if strides is None else (ctypes.c_int64 * 4)(*strides)
    return getattr(lib, name)(ctypes.byref(p), k, v, st, n, cu, lens, table, width, seqs, None, None)


@pytest.mark.parametrize("name", ["dhs_page_write", "dhs_page_read"])
def test_copy_refusals(dhs, name):
    lib = dhs.load()
    assert getattr(lib, name)(None, A, A, None, 4, A, A, A, 3, 2, None, None) == INVALID
    for b in BAD_PAGES:
        assert _copy(lib, name, _pages(**b)) == INVALID, b
    for b in [dict(k=None), dict(v=None), dict(k=A + 2), dict(v=A + 8), dict(cu=None), dict(lens=None),
              dict(table=None), dict(width=0), dict(width=-1), dict(n=-1), dict(seqs=-1),
              dict(strides=(-256, 128, 256, 128)), dict(strides=(256, 128, 256, 129)),
              dict(strides=(1 << 41, 128, 256, 128))]:
        assert _copy(lib, name, **b) == INVALID, b
    assert _copy(lib, name, n=1 << 31) == CAPACITY
    assert _copy(lib, name, n=0, k=None, v=None) == 0      # nothing to do
    assert _copy(lib, name, seqs=0, cu=None, lens=None, table=None) == 0


def test_read_refuses_overlapping_rows(dhs):
    lib = dhs.load()
    assert _copy(lib, "dhs_page_read", strides=(0, 128, 256, 128)) == INVALID
    assert _copy(lib, "dhs_page_read", strides=(256, 128, 256, 64)) == INVALID


def _rows_meet(first, second, d, same):
    """By every pair of rows (their first elements)."""
    return any(abs(a - b) < d for i, a in enumerate(first) for j, b in enumerate(second)
               if not (same and i == j))


def _starts(n, h, st, sh):
    return [i * st + j * sh for i in range(n) for j in range(h)]


@pytest.mark.parametrize("n,h,d", [(4, 2, 64), (3, 4, 64), (1, 3, 128), (5, 1, 128), (2, 2, 64)])
def test_read_refuses_rows_that_share_elements(dhs, n, h, d):
    """All layouts of a grid of strides in which two rows of k, two of v, or a row of
    each of the same strides meet: one of two heads over the next token, one token apart
    as heads are, and values among the keys."""
    lib = dhs.load()
    p = _pages(kv_heads=h, head_dim=d)
    seen = [0, 0]
    grid = [0, 8, d // 2, d - 8, d, d + 8, 2 * d - 8, 2 * d, 3 * d, h * d, h * d + 8, 8 * d]
    for st in grid:
        for sh in grid:
            own = _starts(n, h, st, sh)
            if _rows_meet(own, own, d, True):
                seen[0] += 1
                assert _copy(lib, "dhs_page_read", p, n=n, strides=(st, sh, 8 * d * h, 8 * d), v=A + (1 << 20)) == INVALID
                assert _copy(lib, "dhs_page_read", p, n=n, strides=(8 * d * h, 8 * d, st, sh), v=A + (1 << 20)) == INVALID
                continue
            for off in (0, 8, -8, d - 8, d, -d, 2 * d, st, -st, sh, st + sh - 8, st - sh, 2 * sh - st):
                if _rows_meet(own, [x + off for x in own], d, False):
                    seen[1] += 1
                    assert _copy(lib, "dhs_page_read", p, n=n, k=1 << 30, v=(1 << 30) + 2 * off,
                                 strides=(st, sh, st, sh)) == INVALID, (st, sh, off)
    assert (n * h == 1 or seen[0]) and seen[1]


def test_read_refuses_one_tensor_for_keys_and_values(dhs):
    assert _copy(dhs.load(), "dhs_page_read") == INVALID


def _attend(lib, p=None, q=A, lens=A, table=A, width=3, seqs=2, q_len=1, hq=8, scale=0.0, out=A, ws=A,
            nbytes=1 << 40):
    p = p if p is not None else _pages()
    return lib.dhs_page_attend(ctypes.byref(p), q, None, lens, table, width, seqs, q_len, hq, scale, out,
                               None, ws, nbytes, None, None)


def test_attend_refusals(dhs):
    lib = dhs.load()
    for b in BAD_PAGES:
        assert _attend(lib, _pages(**b)) == INVALID, b
    for b in [dict(q=None), dict(lens=None), dict(table=None), dict(out=None), dict(q=A + 8), dict(out=A + 2),
              dict(ws=A + 4), dict(ws=None), dict(width=-1), dict(seqs=-1), dict(q_len=0), dict(q_len=9), dict(hq=0),
              dict(hq=7), dict(hq=512), dict(q_len=8, hq=34), dict(scale=-1.0), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(nbytes=-1)]:
        assert _attend(lib, **b) == INVALID, b
    assert _attend(lib, seqs=0, q=None, ws=None) == 0


def test_attend_workspace_arguments(dhs):
    lib = dhs.load()
    for b in BAD_PAGES:
        assert lib.dhs_page_attend_workspace(ctypes.byref(_pages(**b)), 2, 1, 8) == -1, b
    p = ctypes.byref(_pages())
    for a in [(-1, 1, 8), (2, 0, 8), (2, 9, 8), (2, 1, 7), (2, 8, 34)]:
        assert lib.dhs_page_attend_workspace(p, *a) == -1, a


def _prompt(lib, q=A, k=A, v=A, strides=None, nq=4, nk=4, cq=A, ck=A, seqs=1, hq=8, hkv=2, d=128, scale=0.0,
            out=A, ws=A, nbytes=1 << 40):
    st = None if strides is None else (ctypes.c_int64 * 6)(*strides)
    return lib.dhs_prompt_attend(q, k, v, st, nq, nk, cq, ck, seqs, hq, hkv, d, scale, out, None, ws, nbytes,
                                 None, None)


def test_prompt_refusals(dhs):
    lib = dhs.load()
    for b in [dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cq=None), dict(ck=None),
              dict(q=A + 2), dict(k=A + 8), dict(v=A + 4), dict(out=A + 8), dict(ws=A + 8), dict(nq=-1),
              dict(nk=-1), dict(nq=1 << 31), dict(nk=1 << 31), dict(seqs=-1), dict(hq=7), dict(hq=0),
              dict(hkv=0), dict(hkv=1, hq=129), dict(d=96), dict(d=256), dict(scale=-0.5),
              dict(scale=float("nan")), dict(scale=float("inf")), dict(nbytes=-1),
              dict(strides=(-1024, 128, 256, 128, 256, 128)), dict(strides=(1024, 128, 252, 128, 256, 128))]:
        assert _prompt(lib, **b) == INVALID, b
    assert _prompt(lib, nq=0, q=None, out=None) == 0
    assert _prompt(lib, seqs=0, cq=None, ck=None) == 0
    for a in [(-1, 4, 1, 8, 2, 128), (4, -1, 1, 8, 2, 128), (4, 4, -1, 8, 2, 128), (4, 4, 1, 8, 3, 128),
              (4, 4, 1, 8, 2, 80)]:
        assert lib.dhs_prompt_attend_workspace(*a) == -1, a


def test_arrays_of_words_off_their_boundary(dhs):
    lib = dhs.load()
    good = ctypes.byref(_pages())
    for bad in (A + 1, A + 2, A + 3):
        for b in (dict(k_scale=bad), dict(v_scale=bad)):
            assert _copy(lib, "dhs_page_write", _pages(**b)) == INVALID
            assert _copy(lib, "dhs_page_read", _pages(**b), v=A << 20) == INVALID
            assert _attend(lib, _pages(**b)) == INVALID
            assert lib.dhs_page_attend_workspace(ctypes.byref(_pages(**b)), 2, 1, 8) == -1
        for i in range(4):
            cu, lens, table, err = (bad if x == i else A for x in range(4))
            for name in ("dhs_page_write", "dhs_page_read"):
                assert getattr(lib, name)(good, A, A << 20, None, 4, cu, lens, table, 3, 2, err, None) == INVALID
        for i in range(5):
            q_lens, lens, table, lse, err = (bad if x == i else A for x in range(5))
            assert lib.dhs_page_attend(good, A, q_lens, lens, table, 3, 2, 1, 8, 0.0, A, lse, A, 1 << 40, err,
                                       None) == INVALID
        for i in range(4):
            cq, ck, lse, err = (bad if x == i else A for x in range(4))
            assert lib.dhs_prompt_attend(A, A, A, None, 4, 4, cq, ck, 1, 8, 2, 128, 0.0, A, lse, A, 1 << 40, err,
                                         None) == INVALID


def test_limit_of_sequences(dhs):
    """Loops over the sequences and the search among them run past the last in 32 bits."""
    lib = dhs.load()
    p = ctypes.byref(_pages())
    for n in ((1 << 31) - 1, (1 << 31) - 1024):
        assert _copy(lib, "dhs_page_write", seqs=n) == INVALID
        assert _copy(lib, "dhs_page_read", seqs=n, v=A << 20) == INVALID
        assert _attend(lib, seqs=n) == INVALID
        assert lib.dhs_page_attend_workspace(p, n, 1, 8) == -1
        assert _prompt(lib, seqs=n) == INVALID
        assert lib.dhs_prompt_attend_workspace(4, 4, n, 8, 2, 128) == -1


def test_prompt_errors_refuses_no_place(dhs):
    assert dhs.load().dhs_prompt_errors(None, None) == INVALID


def test_limits_of_scale_and_tokens(dhs):
    """Larger scales are infinite once they are in log2 units; a tile's positions run past
    the last token in 32 bits."""
    lib = dhs.load()
    assert _attend(lib, scale=2e38) == INVALID and _prompt(lib, scale=2e38) == INVALID
    for n in ((1 << 31) - 1, (1 << 31) - 256):
        assert _prompt(lib, nq=n) == INVALID and _prompt(lib, nk=n) == INVALID
        assert lib.dhs_prompt_attend_workspace(n, 4, 1, 8, 2, 128) == -1


def test_binding_refuses_cpu_tensors_and_wrong_types(dhs):
    import torch
    x = torch.zeros((4, 2, 64, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dhs.PageCache(x, x)                                    # not on a GPU
    with pytest.raises(ValueError):
        dhs.PageCache(x.float(), x.float())
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    k = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    for bad in [dict(q=q.float()), dict(k=k[:, :, :64]), dict(v=k[:3]), dict(out=q[:, :, ::2]), dict(cu_q=cu.long()),
                dict()]:
        a = dict(q=q, k=k, v=k, cu_q=cu, cu_k=cu, out=torch.empty_like(q))
        a.update(bad)
        with pytest.raises(ValueError):
            dhs.prompt_attend(**a)


def test_oracle_quantisation_is_the_nearest_code():
    """Against every code: no other is nearer, and of two as near the even one is taken."""
    from oracle import dense_oracle as o
    rng = np.random.default_rng(3)
    for kind in ("int8", "e4m3"):
        every = (np.arange(-127, 128, dtype=np.int64) if kind == "int8"
                 else np.array([c for c in range(256) if c & 127 != 127]))
        for _ in range(6):
            x = (rng.standard_normal(64) * 2.0 ** rng.integers(-20, 20)).astype(np.float32)
            x[0], x[1] = np.abs(x).max(), np.abs(x).max() / 2
            codes, s = o.quantise(x, kind)
            got, grid = o.value(codes, s, kind), o.value(every, s, kind)
            best = np.abs(grid[None] - x.astype(np.float64)[:, None]).min(1)
            assert np.all(np.abs(got - x) <= best * (1 + 1e-12))
    assert o.quantise([0.0, -0.0], "int8")[1] == 0
    assert np.isnan(o.quantise([1.0, np.inf], "e4m3")[1])


def test_oracle_attention_matches_a_direct_sum():
    from oracle import dense_oracle as o
    rng = np.random.default_rng(4)
    q, k, v = (rng.standard_normal(s) for s in ((3, 4, 8), (5, 2, 8), (5, 2, 8)))
    out, lse, wt, _ = o.attend(q, k, v, 0.5)
    for u in range(3):
        for h in range(4):
            w = np.array([np.exp(0.5 * sum(q[u, h] * k[t, h // 2])) for t in range(3 + u)])
            assert np.allclose(out[u, h], (w[:, None] * v[:3 + u, h // 2]).sum(0) / w.sum(), atol=1e-12)
            assert np.isclose(lse[u, h], np.log(w.sum()))
    empty = o.attend(q, k[:1], v[:1], 0.5)
    assert np.all(empty[0][:2] == 0) and np.all(np.isneginf(empty[1][:2]))
