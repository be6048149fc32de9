"""A dense layer's cache side as a serving loop uses it: rotated keys appended, chunks and
newest tokens attended over the pages, with and without a window, prompts, chunks and single
tokens in turn.  Each attention is held against the fp64 oracle on what the cache then holds
(the append has tests of its own), so that the order and the hand-over of the calls count."""
import math

import numpy as np
import pytest

from test_gpu_chunk import _window_attend
from test_gpu_dense import BF16, E4M3, INT8, KINDS, _close, _np, dhs, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def _cached(torch, cache, table, i, t):
    """Positions 0 .. t - 1 of sequence i as the cache holds them, in 64 bits."""
    rows = cache.page_rows
    pos = torch.arange(t, device="cuda")
    page, row = table[i].long()[pos // rows], pos % rows
    got = []
    for codes, scales in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = codes.view(torch.uint8)[page, :, row].view(codes.dtype) if codes.dtype == torch.float8_e4m3fn \
            else codes[page, :, row]
        x = x.double() if codes.dtype != torch.float8_e4m3fn else x.float().double()
        got.append((x if scales is None else x * scales[page, :, row].double()[..., None]).cpu().numpy())
    return got


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_prompt_chunks_and_decode(torch, dhs, kind, window, sinks):
    from oracle import dense_oracle as oracle
    d, hq, hkv, rows, n = 128, 8, 2, 16, 3
    g = torch.Generator().manual_seed(9)
    rot = dhs.Rotation(10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32))   # half of each head
    wq, wk = ((1 + 0.1 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    cache = dhs.PageCache.empty(60, rows, hkv, d, kind)
    table = torch.randperm(60, generator=g)[:57].view(n, 19).int().cuda()
    lens = [0, 0, 0]
    for step in ([200, 3, 70], [40, 90, 0], [1, 1, 1], [2, 0, 130], [1, 1, 1]):
        lens = [a + b for a, b in zip(lens, step)]
        cu = torch.tensor([0] + step).cumsum(0).int().cuda()
        seq = torch.tensor(lens, dtype=torch.int32).cuda()
        q, k, v = (torch.randn((sum(step), h, d), generator=g).bfloat16().cuda() for h in (hq, hkv, hkv))
        qo = torch.empty_like(q)
        cache.append(q, k, v, cu, seq, table, qo, rot, q_norm=wq, k_norm=wk)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        single = step == [1, 1, 1]
        if single:
            cache.attend(qo[:, None], seq, table, out[:, None], cache.attend_workspace(n, 1, hq), lse=lse[:, None],
                         window=window, sinks=sinks)
        else:
            cache.attend_chunk(qo, cu, seq, table, out, cache.chunk_workspace(len(q), n, hq), lse=lse,
                               window=window, sinks=sinks)
        cache.check()
        for i, a in enumerate(step):
            if not a:
                continue
            s = slice(int(cu[i]), int(cu[i]) + a)
            kv = _cached(torch, cache, table, i, lens[i])
            want = _window_attend(oracle, _np(qo[s]), *kv, 1 / math.sqrt(d), window, sinks)
            vmax = np.abs(kv[1]).max() if kind != BF16 and single else 0.0
            _close(_np(out[s]), _np(lse[s]), want, d, lens[i], vmax)


@pytest.mark.parametrize("kind", [BF16, INT8])
def test_a_captured_decode_step(torch, dhs, kind):
    """Append and windowed attention in one graph, replayed while the sequences grow."""
    from oracle import dense_oracle as oracle
    d, hq, hkv, rows, n, window, sinks = 64, 6, 2, 16, 4, 20, 2
    g = torch.Generator().manual_seed(1)
    rot = dhs.Rotation(10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32), dhs.ROTATE_NEIGHBOURS)
    cache = dhs.PageCache.empty(32, rows, hkv, d, kind)
    table = torch.randperm(32, generator=g).view(n, 8).int().cuda()
    cu = torch.arange(n + 1, dtype=torch.int32).cuda()
    seq = torch.zeros(n, dtype=torch.int32).cuda()
    q, k, v = (torch.zeros((n, h, d), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    qo, out = torch.empty_like(q), torch.empty((n, 1, hq, d), dtype=torch.bfloat16, device="cuda")
    lse, ws = torch.empty((n, 1, hq), device="cuda"), cache.attend_workspace(n, 1, hq)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(q, k, v, cu, seq, table, qo, rot)
        cache.attend(qo[:, None], seq, table, out, ws, lse=lse, window=window, sinks=sinks)
    for step in range(40):
        seq.copy_(torch.tensor([step + 1, step + 3, 2 * step + 1, step + 60], dtype=torch.int32))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        graph.replay()
        if step % 13 == 0:
            cache.check()
            for i in range(n):
                t = int(seq[i])
                kv = _cached(torch, cache, table, i, t)
                want = _window_attend(oracle, _np(qo[i:i + 1]), *kv, 1 / 8.0, window, sinks)
                _close(_np(out[i]), _np(lse[i]), want, d, t, np.abs(kv[1]).max() if kind else 0.0)
