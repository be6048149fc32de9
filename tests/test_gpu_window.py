"""Attention of the newest tokens with a sliding window and first positions that stay visible,
on the GPU against the fp64 oracle (tolerances as for the attention without one)."""
import math

import numpy as np
import pytest

from test_gpu_chunk import _window_attend, give_away
from test_gpu_dense import BF16, E4M3, INT8, KINDS, Paged, _close, _np, dhs, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def _attend(torch, pc, kv, q_len, hq, window, sinks, q_lens=None, seed=5, qmul=1.0, q=None, workspace=None):
    from oracle import dense_oracle as oracle
    n, d = len(pc.lens), pc.d
    g = torch.Generator().manual_seed(seed)
    if q is None:
        q = (torch.randn((n, q_len, hq, d), generator=g) * qmul).bfloat16().cuda()
    out = torch.full_like(q, 77.0)
    lse = torch.full((n, q_len, hq), 77.0, dtype=torch.float32, device="cuda")
    ws = pc.cache.attend_workspace(n, q_len, hq) if workspace is None else workspace
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32).cuda()
    pc.cache.attend(q, pc.seq_lens, pc.table, out, ws, lse=lse, q_lens=ql, window=window, sinks=sinks)
    pc.cache.check()
    for i in range(n):
        nq = q_len if q_lens is None else q_lens[i]
        want = _window_attend(oracle, _np(q[i, :nq]), kv[i][0], kv[i][1], 1 / math.sqrt(d), window, sinks)
        vmax = np.nanmax(np.abs(kv[i][1])) if pc.kind != BF16 and pc.lens[i] else 0.0
        if nq:
            _close(_np(out[i, :nq]), _np(lse[i, :nq]), want, d, max(1, pc.lens[i]), vmax)
        assert torch.all(out[i, nq:] == 77) and torch.all(lse[i, nq:] == 77)
    return out, lse


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,d,rows,q_len", [
    (8, 1, 128, 64, 1), (16, 1, 128, 16, 4), (6, 2, 64, 7, 8), (5, 1, 64, 64, 8), (12, 1, 128, 100, 5),
    (64, 1, 128, 32, 2), (3, 3, 128, 1, 2)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (64, 4), (130, 0), (257, 65), (5000, 3)])
def test_window(torch, dhs, kind, hq, hkv, d, rows, q_len, window, sinks):
    lens = [0, 1, 5, 64, 130, 700, 1025]
    pc = Paged(torch, dhs, lens, rows, hkv, d, kind)
    kv = pc.fill()
    give_away(pc, [q_len] * len(lens), window, sinks)
    _attend(torch, pc, kv, q_len, hq, window, sinks)


@pytest.mark.parametrize("kind", KINDS)
def test_window_fewer_queries_than_room_and_many_sequences(torch, dhs, kind):
    lens = [(i * 37) % 400 for i in range(70)]
    q_lens = [i % 5 for i in range(70)]
    pc = Paged(torch, dhs, lens, 16, 2, 64, kind)
    kv = pc.fill()
    give_away(pc, [4] * 70, 50, 3)
    _attend(torch, pc, kv, 4, 8, 50, 3, q_lens=q_lens)


def test_window_of_a_long_sequence(torch, dhs):
    pc = Paged(torch, dhs, [70000, 33], 64, 1, 128, INT8)
    kv = pc.fill()
    _attend(torch, pc, kv, 1, 16, 2147483647, 2147483647)
    give_away(pc, [1, 1], 4096, 4)      # (from here on the rest is not there)
    _attend(torch, pc, kv, 1, 16, 4096, 4)


@pytest.mark.parametrize("window,sinks", [(3, 0), (3, 1), (70, 2), (128, 0)])
@pytest.mark.parametrize("q_len", [1, 4, 8])
def test_window_edges_hide_what_is_not_finite(torch, dhs, window, sinks, q_len):
    """bf16: every position around the window's edges and the sinks' end in turn holds infinities
    and NaN; the queries that see it get them, the others nothing."""
    from oracle import dense_oracle as oracle
    t, hq, d, rows = 300, 4, 64, 16
    first = t - q_len
    spots = sorted({p for p in list(range(first - window - 1, first - window + q_len + 2)) +
                    list(range(first - 1, t)) + [0, 1, 2, 3] if 0 <= p < t})
    for p in spots:
        pc = Paged(torch, dhs, [t], rows, 1, d, BF16)
        kv = pc.fill()
        page = int(pc.table[0, p // rows])
        for c, row in ((math.inf, 3), (-math.inf, 9), (math.nan, 20)):
            pc.cache.v[page, 0, p % rows, row] = c
            kv[0][1][p, 0, row] = c
        _attend(torch, pc, kv, q_len, hq, window, sinks)
        pc.cache.k[page, 0, p % rows] = math.nan     # now the scores as well
        kv[0][0][p] = math.nan
        q = torch.randn((1, q_len, hq, d), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
        out = torch.empty_like(q)
        pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(1, q_len, hq), window=window,
                        sinks=sinks)
        for j in range(q_len):
            pos = first + j
            seen = p <= pos and (p > pos - window or p < sinks)
            assert bool(torch.isnan(out[0, j]).all()) == seen, (p, j)
            if not seen:
                want = _window_attend(oracle, _np(q[0, :j + 1]), kv[0][0][:pos + 1], kv[0][1][:pos + 1],
                                      1 / math.sqrt(d), window, sinks)
                _close(_np(out[0, j:j + 1]), None, [x[j:j + 1] for x in want], d, t)


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("hq,d", [(2, 128), (8, 64), (16, 128)])
def test_window_large_scales_that_some_queries_do_not_see(torch, dhs, kind, hq, d):
    """A value's scale 2^20 times the others', or NaN, at either edge of the window: rows that do
    not see it keep their precision."""
    t, rows, q_len, window, sinks = 333, 16, 8, 100, 2
    first = t - q_len
    for p in (first - window, first - window + 1, first - window + 4, first - window + q_len - 1, t - window,
              first, first + 3, t - 1, 1):
        for s in (2.0 ** 14, math.nan):
            pc = Paged(torch, dhs, [t], rows, 1, d, kind)
            kv = pc.fill()
            page = int(pc.table[0, p // rows])
            if s == s:
                kv[0][1][p] *= s / float(pc.cache.v_scale[page, 0, p % rows])
            else:
                kv[0][1][p] = s
            pc.cache.v_scale[page, 0, p % rows] = s
            from oracle import dense_oracle as oracle
            q = torch.randn((1, q_len, hq, d), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
            out = torch.empty_like(q)
            pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(1, q_len, hq),
                            window=window, sinks=sinks)
            pc.cache.check()
            for j in range(q_len):
                pos = first + j
                keep = [x for x in range(pos + 1) if x > pos - window or x < sinks]
                want = oracle.attend(_np(q[0, j:j + 1]), kv[0][0][keep], kv[0][1][keep], 1 / math.sqrt(d))
                seen = p in keep
                if seen and s != s:
                    assert torch.isnan(out[0, j]).all(), (p, j)
                    continue
                vmax = np.abs(kv[0][1][keep]).max()
                _close(_np(out[0, j:j + 1]), None, want, d, t, vmax)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,hkv,window,sinks,q_len", [
    (33, 1, 2000, 3, 1), (40, 2, 500, 0, 4), (160, 2, 250, 4, 1), (255, 1, 600, 200, 1), (256, 2, 300, 4, 2),
    (257, 2, 300, 4, 1), (300, 1, 900, 1, 1), (520, 1, 260, 130, 2)])
def test_window_of_many_sequences(torch, dhs, kind, n, hkv, window, sinks, q_len):
    """CTAs' places among many items of some blocks each, empty sequences among them; twice the
    same bits."""
    lens = [0 if i % 11 == 5 else (i * 389) % 1400 + 1 for i in range(n)]
    pc = Paged(torch, dhs, lens, 32, hkv, 64, kind)
    kv = pc.fill()
    give_away(pc, [q_len] * n, window, sinks)
    out, lse = _attend(torch, pc, kv, q_len, 4 * hkv, window, sinks)
    again, lse2 = _attend(torch, pc, kv, q_len, 4 * hkv, window, sinks)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", [BF16, INT8])
def test_window_where_every_item_is_cut(torch, dhs, kind):
    """Few long items beside short ones: parts that begin in the units that an item counts for
    itself, and items of which a part has no block."""
    lens = [9000] * 9 + [1, 40, 200, 3000, 5000] * 7
    pc = Paged(torch, dhs, lens, 64, 1, 128, kind)
    kv = pc.fill()
    for window in (100000, 4096, 700):
        give_away(pc, [1] * len(lens), window, 2)
        _attend(torch, pc, kv, 1, 8, window, 2)


def _check_scaled(torch, pc, kv, q_len, hq, window, sinks, scaled, gone=()):
    """One sequence whose values at positions ``scaled`` {position: factor} are that much larger:
    every query against its own positions, without those of ``gone``."""
    from oracle import dense_oracle as oracle
    t, rows, d = pc.lens[0], pc.rows, pc.d
    kv = [(k, v.copy()) for k, v in kv]
    before = pc.cache.v_scale.clone()
    for p, s in scaled.items():
        pc.cache.v_scale[int(pc.table[0, p // rows]), 0, p % rows] *= s
        kv[0][1][p] *= s
    q = torch.randn((1, q_len, hq, d), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    out = torch.empty_like(q)
    pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(1, q_len, hq), window=window,
                    sinks=sinks)
    pc.cache.v_scale.copy_(before)
    for j in range(q_len):
        pos = t - q_len + j
        keep = [x for x in range(pos + 1) if (x > pos - window or x < sinks) and x not in gone]
        want = oracle.attend(_np(q[0, j:j + 1]), kv[0][0][keep], kv[0][1][keep], 1 / math.sqrt(d))
        _close(_np(out[0, j:j + 1]), None, want, d, t, np.abs(kv[0][1][keep]).max())


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("hq,d", [(2, 128), (8, 64), (16, 128)])
@pytest.mark.parametrize("q_len", [2, 4, 8])
def test_window_starts_at_a_tile_end(torch, dhs, kind, hq, d, q_len):
    """The tile in which the first query's window starts holds no position that all queries see:
    a scale that is large, at a position that the later ones do not see, costs them nothing."""
    window, rows = 100, 16
    for start in {128, 128 + q_len // 2}:          # the last query's first position
        pc = Paged(torch, dhs, [start + window], rows, 1, d, kind)
        kv = pc.fill()
        first = start - q_len + 1                  # the first query's
        for sinks in (0, 2):
            for p in sorted({first, first + 1, 127, start - 1, start}):
                for s in (2.0 ** 24, 2.0 ** 40):
                    _check_scaled(torch, pc, kv, q_len, hq, window, sinks, {p: s})
            # the first position that all see is small, or none at all
            _check_scaled(torch, pc, kv, q_len, hq, window, sinks, {start: 2.0 ** -40})
            _check_scaled(torch, pc, kv, q_len, hq, window, sinks, {start: 0.0, first: 2.0 ** 24})
        pc.cache.check()
        # its page is not there
        gone = range(start // rows * rows, start // rows * rows + rows)
        pc.table[0, start // rows] = -1
        _check_scaled(torch, pc, kv, q_len, hq, window, 0, {first: 1.0 if first in gone else 2.0 ** 24}, gone)
        with pytest.raises(dhs.DhsError):
            pc.cache.check()


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 0), (5, 0), (7, 1), (3, 2)])
@pytest.mark.parametrize("hq,d", [(2, 128), (16, 64)])
def test_window_of_fewer_positions_than_queries(torch, dhs, kind, window, sinks, hq, d):
    """No position but the first ones is seen by all queries: a large scale in any query's window
    costs the others nothing."""
    for t in (200, 196, 9, 8):
        pc = Paged(torch, dhs, [t], 16, 1, d, kind)
        kv = pc.fill()
        for p in range(max(0, t - 8 - window), t):
            _check_scaled(torch, pc, kv, 8, hq, window, sinks, {p: 2.0 ** 30})
        pc.cache.check()


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("q_len", [2, 8])
@pytest.mark.parametrize("hkv,d", [(256, 128), (600, 64)])
def test_window_starts_at_a_tile_end_and_goes_on(torch, dhs, kind, q_len, hkv, d):
    """The same where a group of warps goes on to later tiles of an item: they keep their precision
    after a scale that the first query alone sees."""
    from oracle import dense_oracle as oracle
    window, rows, start = 400, 16, 128
    t, first = start + window, start - q_len + 1
    pc = Paged(torch, dhs, [t], rows, hkv, d, kind)
    (k, v), = pc.fill()
    pc.cache.v_scale[int(pc.table[0, first // rows]), :, first % rows] *= 2.0 ** 30
    v[first] *= 2.0 ** 30
    q = torch.randn((1, q_len, hkv, d), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    out = torch.empty_like(q)
    pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(1, q_len, hkv), window=window)
    pc.cache.check()
    for j in range(q_len):
        seen = slice(first + j, first + j + window)
        for h in list(range(0, hkv, 41)) + [hkv - 1]:
            one = slice(h, h + 1)
            want = oracle.attend(_np(q[0, j:j + 1, one]), k[seen, one], v[seen, one], 1 / math.sqrt(d))
            _close(_np(out[0, j:j + 1, one]), None, want, d, t, np.abs(v[seen, one]).max())
