"""Chunk attention over a paged cache on the GPU against the fp64 oracle.

Tolerances are those of the other attention operators (half-steps of the output's and the
weights' rounding to bf16, and of the 32-bit scores and sums); weights of an 8-bit cache are
rounded once, times their value's scale, so the same terms hold, and nothing comes in for scales.
"""
import math

import numpy as np
import pytest

from test_gpu_dense import BF16, E4M3, INT8, KINDS, Paged, _close, _np, dhs, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def _window_attend(oracle, q, k, v, scale, window, sinks):
    """oracle.attend with a window: every query over the positions that it sees."""
    if not window:
        return oracle.attend(q, k, v, scale)
    parts = []
    for u in range(len(q)):
        p = len(k) - len(q) + u
        keep = [t for t in range(p + 1) if t > p - window or t < sinks]
        parts.append(oracle.attend(q[u:u + 1], k[keep], v[keep], scale) if keep
                     else oracle.attend(q[u:u + 1], k[:0], v[:0], scale))
    return tuple(np.concatenate([x[j] for x in parts]) if parts else oracle.attend(q, k, v, scale)[j]
                 for j in range(4))


def give_away(pc, new, window, sinks):
    """Pages of which no new token sees a position leave the table."""
    table = pc.table.cpu()
    for i, (a, t) in enumerate(zip(new, pc.lens)):
        for g in range(-(-t // pc.rows)):
            lo, hi = g * pc.rows, min(t, (g + 1) * pc.rows)   # its positions
            if lo >= sinks and hi - 1 <= t - a - window:
                table[i, g] = -9 if g % 2 else pc.n_pages + 5
    pc.table = table.cuda()


def _chunk(torch, dhs, pc, kv, new, hq, window=0, sinks=0, scale=0.0, seed=5, qmul=1.0, pad=(0, 0),
           strided=False, workspace=None, lse=True, check=True):
    from oracle import dense_oracle as oracle
    d = pc.d
    n = sum(new)
    cu = torch.tensor([pad[0]] + list(new)).cumsum(0).int().cuda()
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((pad[0] + n + pad[1], hq, d), generator=g) * qmul).bfloat16().cuda()
    if strided:
        q = torch.cat([q, torch.full_like(q[:, :1], math.nan)], 1)[:, :hq]
    out = torch.full(tuple(q.shape), 77.0, dtype=torch.bfloat16, device="cuda")
    lz = torch.full(tuple(q.shape[:2]), 77.0, dtype=torch.float32, device="cuda") if lse else None
    ws = pc.cache.chunk_workspace(q.shape[0], len(new), hq) if workspace is None else workspace
    pc.cache.attend_chunk(q, cu, pc.seq_lens, pc.table, out, ws, lse=lz, window=window, sinks=sinks, scale=scale)
    if not check:
        return q, cu, out, lz
    pc.cache.check()
    for i, a in enumerate(new):
        s = slice(int(cu[i]), int(cu[i]) + a)
        if not a:
            continue
        want = _window_attend(oracle, _np(q[s]), kv[i][0], kv[i][1], scale or 1 / math.sqrt(d), window, sinks)
        _close(_np(out[s]), None if lz is None else _np(lz[s]), want, d, max(1, pc.lens[i]))
    for s in (slice(0, pad[0]), slice(pad[0] + n, None)):
        assert torch.all(out[s] == 77) and (lz is None or torch.all(lz[s] == 77))
    return q, cu, out, lz


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 1, 128, 64), (6, 2, 64, 16), (7, 1, 128, 48), (3, 3, 64, 100),
                                           (4, 1, 128, 7), (2, 2, 64, 1), (5, 5, 128, 1)])
def test_chunk(torch, dhs, kind, hq, hkv, d, rows):
    lens, new = [0, 1, 5, 130, 300, 129, 260], [0, 1, 5, 3, 77, 129, 1]
    pc = Paged(torch, dhs, lens, rows, hkv, d, kind)
    _chunk(torch, dhs, pc, pc.fill(), new, hq, pad=(2, 3))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (5, 3), (64, 4), (128, 0), (129, 130),
                                          (200, 16), (1000, 4), (3, 1000)])
def test_chunk_window(torch, dhs, kind, window, sinks):
    lens, new = [600, 700, 1, 130, 300], [200, 1, 1, 130, 9]
    d, hkv, hq, rows = (128, 1, 8, 16) if window % 2 else (64, 2, 6, 48)
    pc = Paged(torch, dhs, lens, rows, hkv, d, kind)
    kv = pc.fill()
    give_away(pc, new, window, sinks)
    _chunk(torch, dhs, pc, kv, new, hq, window=window, sinks=sinks)
