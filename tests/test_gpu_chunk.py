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


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
def test_chunk_items_cut_between_ctas(torch, dhs, kind, window, sinks):
    """Long sequences of few rows, whose keys are shared out and joined, beside short ones."""
    lens, new = [5000, 40, 2600, 3, 900], [33, 40, 1, 1, 290]
    pc = Paged(torch, dhs, lens, 64, 1, 128, kind)
    _chunk(torch, dhs, pc, pc.fill(), new, 4, window=window, sinks=sinks)


@pytest.mark.parametrize("kind", KINDS)
def test_chunk_many_sequences_some_idle(torch, dhs, kind):
    lens = [(i * 53) % 300 for i in range(150)]
    new = [min(t, (0, 0, 1, 1, 7, 40)[i % 6]) for i, t in enumerate(lens)]
    pc = Paged(torch, dhs, lens, 16, 2, 64, kind)
    _chunk(torch, dhs, pc, pc.fill(), new, 6, pad=(1, 4))


@pytest.mark.parametrize("hq,hkv,d", [(128, 1, 128), (100, 1, 64), (9, 9, 128), (48, 16, 64)])
def test_chunk_head_layouts(torch, dhs, hq, hkv, d):
    pc = Paged(torch, dhs, [70, 300], 32, hkv, d, E4M3)
    _chunk(torch, dhs, pc, pc.fill(), [70, 21], hq)


@pytest.mark.parametrize("kind", KINDS)
def test_chunk_scale_large_scores_strides_and_alignment(torch, dhs, kind):
    pc = Paged(torch, dhs, [400, 90], 48, 2, 64, kind)
    kv = pc.fill(outlier=3.0)
    _chunk(torch, dhs, pc, kv, [150, 90], 4, qmul=30.0, strided=True)
    _chunk(torch, dhs, pc, kv, [150, 90], 4, scale=0.7, lse=False)
    # an output and a workspace on 16-byte boundaries only
    cu = torch.tensor([0, 150, 240], dtype=torch.int32).cuda()
    q = torch.randn((240, 4, 64), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    want = torch.empty_like(q)
    ws = pc.cache.chunk_workspace(240, 2, 4)
    pc.cache.attend_chunk(q, cu, pc.seq_lens, pc.table, want, ws)
    raw = torch.empty(q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    out = raw[8:].view(q.shape)
    assert out.data_ptr() % 32 == 16
    ws2 = torch.full((ws.numel() + 16,), 255, dtype=torch.uint8, device="cuda")[16:]
    pc.cache.attend_chunk(q, cu, pc.seq_lens, pc.table, out, ws2)
    assert torch.equal(out, want)
    with pytest.raises(dhs.DhsError):
        pc.cache.attend_chunk(q, cu, pc.seq_lens, pc.table, out, ws[:-16])


def test_chunk_agrees_with_the_prompt_and_the_decode(torch, dhs):
    """The same attention by the three calls, within two roundings of the output and of the
    weights (2^-7 of a value and of the weights' sum of magnitudes)."""
    lens = [513, 77]
    pc = Paged(torch, dhs, lens, 64, 2, 128, BF16)
    kv = pc.fill()
    q, cu, out, lse = _chunk(torch, dhs, pc, kv, lens, 8)
    k, v = (torch.cat([torch.from_numpy(x[j]) for x in kv]).bfloat16().cuda() for j in (0, 1))
    o2, l2 = torch.empty_like(q), torch.empty_like(lse)
    dhs.prompt_attend(q, k, v, cu, cu, o2, lse=l2, workspace=dhs.prompt_workspace(q, k, 2))
    mag = float(v.abs().max())
    assert (out.float() - o2.float()).abs().max() <= 2.0 ** -7 * 2 * mag
    assert (lse - l2).abs().max() <= 1e-5
    last = torch.stack([q[cu[1] - 1], q[cu[2] - 1]])[:, None].contiguous()
    o3 = torch.empty_like(last)
    pc.cache.attend(last, pc.seq_lens, pc.table, o3, pc.cache.attend_workspace(2, 1, 8))
    got = torch.stack([out[cu[1] - 1], out[cu[2] - 1]])[:, None]
    assert (got.float() - o3.float()).abs().max() <= 2.0 ** -7 * 2 * mag


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (70, 2), (128, 200)])
@pytest.mark.parametrize("hq,d", [(2, 128), (16, 64)])
def test_chunk_values_that_are_not_finite(torch, dhs, window, sinks, hq, d):
    """bf16: infinities and NaN among the values, at places that all tokens, some and none see,
    reach the tokens that see them and no other; and then keys of NaN."""
    t, new, rows = 420, 130, 16
    first = t - new
    for spots in ([first - 1, first + 5, t - 1], [first - window - 1, first - window, first - window + 1,
                                                  t - window - 1, t - window], [0, 1, 2, 199, 200, 128]):
        spots = sorted({p for p in spots if 0 <= p < t})
        pc = Paged(torch, dhs, [t, 200], rows, 1, d, BF16)
        kv = pc.fill()
        for j, p in enumerate(spots):
            page = int(pc.table[0, p // rows])
            for c, x in ((3, math.inf), (d - 1, -math.inf if j % 2 else math.inf), (20 + j, math.nan)):
                pc.cache.v[page, 0, p % rows, c] = x
                kv[0][1][p, 0, c] = x
        _chunk(torch, dhs, pc, kv, [new, 200], hq, window=window, sinks=sinks)
        p = spots[len(spots) // 2]
        pc.cache.k[int(pc.table[0, p // rows]), 0, p % rows] = math.nan
        _, cu, out, lse = _chunk(torch, dhs, pc, kv, [new, 200], hq, window=window, sinks=sinks, check=False)
        for u in range(new):
            pos = first + u
            seen = p <= pos and (not window or p > pos - window or p < sinks)
            assert bool(torch.isnan(lse[u]).all()) == seen and bool(torch.isnan(out[u]).all()) >= seen


@pytest.mark.parametrize("kind", [INT8, E4M3])
def test_chunk_scales_that_are_not_finite(torch, dhs, kind):
    """Rows with a scale of NaN, as stored for rows with an infinity, reach who sees them."""
    from oracle import dense_oracle as oracle
    t, new, rows, d, hq, window = 300, 100, 16, 64, 4, 60
    for side in (0, 1):
        for p in (150, 210, 250, 299):
            pc = Paged(torch, dhs, [t], rows, 1, d, kind)
            kv = pc.fill()
            (pc.cache.v_scale if side else pc.cache.k_scale)[int(pc.table[0, p // rows]), 0, p % rows] = math.nan
            for w in (0, window):
                q, cu, out, lse = _chunk(torch, dhs, pc, kv, [new], hq, window=w, check=False)
                pc.cache.check()
                for u in range(0, new, 7):
                    pos = t - new + u
                    seen = p <= pos and (not w or p > pos - w)
                    assert bool(torch.isnan(out[u]).all()) == seen
                    assert bool(torch.isnan(lse[u]).all()) == (seen and not side)
                    if not seen:
                        want = _window_attend(oracle, _np(q[u:u + 1]), kv[0][0][:pos + 1], kv[0][1][:pos + 1],
                                              1 / math.sqrt(d), w, 0)
                        _close(_np(out[u:u + 1]), _np(lse[u:u + 1]), want, d, t)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("rows", [16, 64])
def test_chunk_leaves_out_pages_that_are_not_there(torch, dhs, kind, window, rows):
    from oracle import dense_oracle as oracle
    t, new, d, hq = 500, 140, 128, 4
    pc = Paged(torch, dhs, [t, 90], rows, 1, d, kind)
    kv = pc.fill()
    gone = [p for g in (t // rows, 300 // rows, 420 // rows) for p in range(g * rows, min(t, (g + 1) * rows))]
    for j, g in enumerate((t // rows, 300 // rows, 420 // rows)):
        pc.table[0, g] = (-1, pc.n_pages, 2147483647)[j]
    q, cu, out, lse = _chunk(torch, dhs, pc, kv, [new, 90], hq, window=window, check=False)
    with pytest.raises(dhs.DhsError, match="dhs_page_chunk: a page"):
        pc.cache.check()
    pc.cache.check()
    for u in list(range(0, new, 9)) + [new - 1]:
        pos = t - new + u
        keep = [p for p in range(pos + 1) if p not in gone and (not window or p > pos - window)]
        want = oracle.attend(_np(q[u:u + 1]), kv[0][0][keep], kv[0][1][keep], 1 / math.sqrt(d))
        _close(_np(out[u:u + 1]), _np(lse[u:u + 1]), want, d, t)
    want = oracle.attend(_np(q[new:]), kv[1][0], kv[1][1], 1 / math.sqrt(d)) if not window else None
    if want:
        _close(_np(out[new:]), _np(lse[new:]), want, d, t)


def test_chunk_all_pages_gone(torch, dhs):
    pc = Paged(torch, dhs, [200, 50], 16, 2, 64, INT8)
    kv = pc.fill()
    pc.table[0] = -3
    q, cu, out, lse = _chunk(torch, dhs, pc, kv, [30, 50], 4, check=False)
    with pytest.raises(dhs.DhsError):
        pc.cache.check()
    assert torch.isneginf(lse[:30]).all() and torch.isnan(out[:30]).all()    # 0 / 0: positions, but no key
    assert torch.isfinite(out[30:]).all()


@pytest.mark.parametrize("what", ["length", "negative", "offset", "beyond"])
def test_chunk_bad_lengths_and_offsets(torch, dhs, what):
    lens, new = [60, 100, 40], [20, 33, 40]
    pc = Paged(torch, dhs, lens, 16, 1, 64, E4M3)
    kv = pc.fill()
    q, cu, want, wl = _chunk(torch, dhs, pc, kv, new, 4)
    ws = pc.cache.chunk_workspace(q.shape[0], 3, 4)
    seq, c2 = pc.seq_lens.clone(), cu.clone()
    left = slice(20, 53)
    if what == "length":
        seq[1] = pc.table.shape[1] * 16 + 1
    elif what == "negative":
        seq[1] = -5
    elif what == "offset":
        c2[2] = 10             # sequence 1 ends before it begins, sequence 2 starts at 10
        left = None
    else:
        c2[3] = q.shape[0] + 1
        left = slice(53, 93)
    out, lse = torch.full_like(want, 77), torch.full_like(wl, 77)
    pc.cache.attend_chunk(q, c2, seq, pc.table, out, ws, lse=lse)
    with pytest.raises(dhs.DhsError, match="dhs_page_chunk: a length"):
        pc.cache.check()
    pc.cache.check()
    if left is not None:
        assert torch.all(out[left] == 77) and torch.all(lse[left] == 77)
        keep = torch.ones(q.shape[0], dtype=torch.bool)
        keep[left] = False
        assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], wl[keep])


def test_chunk_positions_before_the_first(torch, dhs):
    """More new tokens than positions: the first of them see nothing."""
    pc = Paged(torch, dhs, [5, 300], 16, 1, 128, BF16)
    kv = pc.fill()
    _chunk(torch, dhs, pc, kv, [300, 300], 2)
    _chunk(torch, dhs, pc, kv, [300, 300], 2, window=7, sinks=2)


def test_chunk_same_result_again_beside_others_and_on_two_streams(torch, dhs):
    pc = Paged(torch, dhs, [3000, 500, 64], 64, 1, 128, INT8)
    kv = pc.fill()
    new = [200, 500, 1]
    q, cu, want, wl = _chunk(torch, dhs, pc, kv, new, 8)
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [pc.cache.chunk_workspace(q.shape[0], 3, 8) for _ in range(2)]
    outs = [torch.empty_like(want) for _ in range(2)]
    lses = [torch.empty_like(wl) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(6):
        for s, w, o, l in zip(streams, spaces, outs, lses):
            pc.cache.attend_chunk(q, cu, pc.seq_lens, pc.table, o, w, lse=l, stream=s)
    torch.cuda.synchronize()
    pc.cache.check()
    for o, l in zip(outs, lses):
        assert torch.equal(o, want) and torch.equal(l, wl)


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_chunk_captured_follows_lengths_and_pages(torch, dhs, kind):
    from oracle import dense_oracle as oracle
    lens = [400, 350]
    pc = Paged(torch, dhs, lens, 16, 1, 64, kind)
    kv = pc.fill()
    q = torch.randn((90, 4, 64), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    cu, seq = torch.zeros(3, dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    table = torch.zeros_like(pc.table)
    graphs, outs = [], []
    for _ in range(2):
        out, lse, ws = torch.empty_like(q), torch.empty((90, 4), device="cuda"), pc.cache.chunk_workspace(90, 2, 4)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pc.cache.attend_chunk(q, cu, seq, table, out, ws, lse=lse)
        graphs.append(g)
        outs.append((out, lse, ws))
    for a, b, x, y in ((60, 30, 400, 350), (1, 89, 70, 200), (90, 0, 333, 0), (1, 1, 399, 17)):
        cu.copy_(torch.tensor([0, a, a + b], dtype=torch.int32))
        seq.copy_(torch.tensor([x, y], dtype=torch.int32))
        table.copy_(pc.table)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        pc.cache.check()
        assert torch.equal(outs[0][0][:a + b], outs[1][0][:a + b])
        for i, (s, n, t) in enumerate(((0, a, x), (a, b, y))):
            if n:
                want = oracle.attend(_np(q[s:s + n]), kv[i][0][:t], kv[i][1][:t], 1 / 8.0)
                _close(_np(outs[0][0][s:s + n]), _np(outs[0][1][s:s + n]), want, 64, t)


@pytest.mark.parametrize("kind", [BF16, INT8])
def test_chunk_far_pages(torch, dhs, kind):
    """Pages whose elements lie beyond 2^31."""
    rows, hkv, d = 64, 2, 128
    huge = 2 ** 31 // (rows * hkv * d) + 9
    pc = Paged(torch, dhs, [300, 70], rows, hkv, d, kind, huge_pages=huge)
    assert int(pc.table.max()) * rows * hkv * d > 2 ** 31
    _chunk(torch, dhs, pc, pc.fill(), [100, 70], 4)
    _chunk(torch, dhs, pc, pc.fill(), [100, 70], 4, window=40, sinks=3)


def test_chunk_refuses_tensors_that_do_not_fit(torch, dhs):
    pc = Paged(torch, dhs, [64], 16, 2, 64, BF16)
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32).cuda()
    ws = pc.cache.chunk_workspace(4, 1, 4)
    call = pc.cache.attend_chunk
    for bad in (dict(q=q[..., :32]), dict(q=q.float()), dict(out=q[:3].clone()), dict(out=q.float()), dict(cu=cu.long()),
                dict(cu=cu[:1]), dict(lse=torch.zeros((4, 3), device="cuda")), dict(table=pc.table.long()),
                dict(q=q.cpu())):
        a = dict(q=q, cu=cu, out=torch.empty_like(q), lse=None, table=pc.table)
        a.update(bad)
        with pytest.raises(ValueError):
            call(a["q"], a["cu"], pc.seq_lens, a["table"], a["out"], ws, lse=a["lse"])
    with pytest.raises(dhs.DhsError):
        call(q, cu, pc.seq_lens, pc.table, torch.empty_like(q), ws, sinks=3)
    with pytest.raises(ValueError):
        pc.cache.chunk_workspace(4, 1, 3)


@pytest.mark.parametrize("kind", [INT8, E4M3])
def test_chunk_sequences_over_the_same_pages(torch, dhs, kind):
    """Sequences that share their pages, together longer than the cache."""
    n, t, new, hq, d = 14, 600, 300, 4, 64
    pc = Paged(torch, dhs, [t], 32, 1, d, kind)
    kv = pc.fill()
    pc.table = pc.table.expand(n, -1).contiguous()
    pc.seq_lens = pc.seq_lens.expand(n).contiguous()
    pc.lens = [t] * n
    _chunk(torch, dhs, pc, kv * n, [new] * n, hq)
    pc.seq_lens = (pc.seq_lens - torch.arange(n, dtype=torch.int32).cuda() * 7).contiguous()
    pc.lens = [t - 7 * i for i in range(n)]
    _chunk(torch, dhs, pc, [[x[:t - 7 * i] for x in kv[0]] for i in range(n)], [new - 9 * i for i in range(n)], hq,
           window=130, sinks=5)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("rows", [1, 2, 3, 12])
def test_chunk_small_pages_that_are_not_there(torch, dhs, kind, window, rows):
    """Pages of which more than 32 make a tile: one in every place of a tile's four 32s is gone."""
    from oracle import dense_oracle as oracle
    t, new, d, hq = 400, 150, 64, 4
    pc = Paged(torch, dhs, [t], rows, 1, d, kind)
    kv = pc.fill()
    pages = sorted({p // rows for p in (128 + 5, 128 + 40, 128 + 77, 255, 256, 300, 399)})
    for j, g in enumerate(pages):
        pc.table[0, g] = (-1, pc.n_pages, 2147483647)[j % 3]
    gone = {p for g in pages for p in range(g * rows, (g + 1) * rows)}
    q, cu, out, lse = _chunk(torch, dhs, pc, kv, [new], hq, window=window, check=False)
    with pytest.raises(dhs.DhsError, match="dhs_page_chunk: a page"):
        pc.cache.check()
    for u in list(range(0, new, 7)) + [new - 1]:
        pos = t - new + u
        keep = [p for p in range(pos + 1) if p not in gone and (not window or p > pos - window)]
        want = oracle.attend(_np(q[u:u + 1]), kv[0][0][keep], kv[0][1][keep], 1 / math.sqrt(d))
        _close(_np(out[u:u + 1]), _np(lse[u:u + 1]), want, d, t)


def _attend_64(torch, q, k, v, scale, window, sinks):
    """_window_attend for many rows: in 64 bits on the GPU, a head at a time."""
    n, hq, d = q.shape
    t, hkv, _ = k.shape
    q = q.double()
    k, v = (torch.from_numpy(x).cuda() for x in (k, v))
    at = torch.arange(t, device="cuda")
    p = (t - n + torch.arange(n, device="cuda"))[:, None]
    hide = at > p
    if window:
        hide |= (at <= p - window) & (at >= sinks)
    got = []
    for h in range(hq):
        kh, vh = k[:, h * hkv // hq], v[:, h * hkv // hq]
        s = (q[:, h] @ kh.T * scale).masked_fill_(hide, -math.inf)
        lse = torch.logsumexp(s, 1)
        s = s.sub_(lse[:, None]).exp_()
        reach = (q[:, h].abs() @ kh.abs().T).masked_fill_(hide, 0).amax(1) * scale
        got.append((s @ vh, lse, s @ vh.abs(), reach))
    return tuple(torch.stack([x[j] for x in got], 1).cpu().numpy() for j in range(4))


def _tiles_a_border_moves(torch, lens, new, hkv, group, window, sinks):
    """How far a border between two CTAs' shares is moved at most: an eighth of a share, in tiles
    of 128 positions, 2 to 8 (the kernel's rule, from the costs of its items)."""
    tpt = 128 // group
    cap = window + sinks + 2 * tpt + 256 if window else 1 << 31
    total = 0
    for t, a in zip(lens, new):
        for r in range(-(-a // (2 * tpt))):
            walked = min(t - a + (r + 1) * 2 * tpt, cap)
            total += hkv * (384 + (walked * 3 // 4 if a <= tpt else walked))
    share = total // torch.cuda.get_device_properties(0).multi_processor_count
    return max(2, min(8, share // 1024))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,new,d,window,sinks,least,most", [
    ([9000, 6000, 1200, 8000], [3000, 2500, 700, 1], 128, 0, 0, 8, 8),
    ([9000, 6000, 1200, 8000], [3000, 2500, 700, 1], 64, 6000, 130, 8, 8),
    ([9000, 6000, 1200], [3000, 2500, 700], 128, 2000, 5, 4, 7),
    ([5000, 2600] + [3000] * 8, [1500, 800] + [1] * 8, 64, 0, 0, 3, 6),
    ([12000, 9000], [12000, 9000], 64, 300, 4, 8, 8)])      # many short items to a CTA
def test_chunk_of_long_shares(torch, dhs, kind, lens, new, d, window, sinks, least, most):
    """Shares so long that borders are moved by more than two tiles, every row of every item: the
    CTAs on either side of a border and the join agree on it.  Twice the same bits."""
    hq, hkv = 16, 4
    assert least <= _tiles_a_border_moves(torch, lens, new, hkv, hq // hkv, window, sinks) <= most
    pc = Paged(torch, dhs, lens, 64, hkv, d, kind)
    kv = pc.fill()
    give_away(pc, new, window or 1 << 30, sinks)
    q, cu, out, lse = _chunk(torch, dhs, pc, kv, new, hq, window=window, sinks=sinks, pad=(3, 2), check=False)
    pc.cache.check()
    for i, a in enumerate(new):
        s = slice(int(cu[i]), int(cu[i]) + a)
        want = _attend_64(torch, q[s], *kv[i], 1 / math.sqrt(d), window, sinks)
        _close(_np(out[s]), _np(lse[s]), want, d, lens[i])
    for s in (slice(0, 3), slice(3 + sum(new), None)):
        assert torch.all(out[s] == 77) and torch.all(lse[s] == 77)
    _, _, again, lse2 = _chunk(torch, dhs, pc, kv, new, hq, window=window, sinks=sinks, pad=(3, 2), check=False)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (70, 2), (128, 200)])
@pytest.mark.parametrize("hq,d", [(2, 128), (16, 64)])
def test_chunk_keys_that_are_not_finite(torch, dhs, window, sinks, hq, d):
    """bf16: a key of NaN beside values that are not finite: tokens that do not see it have the
    outputs that they have without it."""
    from oracle import dense_oracle as oracle
    t, new, rows = 420, 130, 16
    first = t - new
    for p in sorted({first - 1, first + 5, t - 2, first - window + 40, t - window - 1, 1, 200} & set(range(t))):
        pc = Paged(torch, dhs, [t, 200], rows, 1, d, BF16)
        kv = pc.fill()
        page = int(pc.table[0, p // rows])
        for c, x in ((3, math.inf), (20, math.nan)):
            pc.cache.v[page, 0, p % rows, c] = x
            kv[0][1][p, 0, c] = x
        pc.cache.k[page, 0, p % rows] = math.nan
        kv[0][0][p] = math.nan
        q, cu, out, lse = _chunk(torch, dhs, pc, kv, [new, 200], hq, window=window, sinks=sinks, check=False)
        pc.cache.check()
        pos = torch.arange(first, t)
        seen = (p <= pos) & ((pos - p < window) if window and p >= sinks else torch.ones_like(pos, dtype=torch.bool))
        blind = (~seen).nonzero()[:, 0].tolist()
        assert torch.isnan(out[:new][seen]).all() and torch.isnan(lse[:new][seen]).all()
        kv[0][0][p] = kv[0][1][p] = 0.0      # (of no weight below: the oracle's masked places are left out)
        want = _window_attend(oracle, _np(q[:new]), *kv[0],
                              1 / math.sqrt(d), window, sinks)
        _close(_np(out[blind]), _np(lse[blind]), [x[blind] for x in want], d, t)
        want = _window_attend(oracle, _np(q[new:]), *kv[1],
                              1 / math.sqrt(d), window, sinks)
        _close(_np(out[new:]), _np(lse[new:]), want, d, 200)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(2147483647, 2147483647), (2147483647, 0), (1, 2147483647)])
def test_chunk_windows_and_sinks_of_any_size(torch, dhs, kind, window, sinks):
    pc = Paged(torch, dhs, [600, 40, 300], 16, 2, 64, kind)
    _chunk(torch, dhs, pc, pc.fill(), [150, 40, 1], 4, window=window, sinks=sinks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [0, 90])
def test_chunk_of_more_than_a_thousand_sequences(torch, dhs, kind, window):
    """Most of them decode one token, some have none, a few have a chunk."""
    n = 1100
    lens = [0 if i % 97 == 5 else (i * 131) % 260 + 1 for i in range(n)]
    new = [min(t, 0 if i % 13 == 2 else 150 if i % 200 == 77 else 1) for i, t in enumerate(lens)]
    pc = Paged(torch, dhs, lens, 16, 1, 64, kind)
    kv = pc.fill()
    give_away(pc, new, window or 1 << 30, 2 if window else 0)
    q, cu, out, lse = _chunk(torch, dhs, pc, kv, new, 4, window=window, sinks=2 if window else 0)
    _, _, again, lse2 = _chunk(torch, dhs, pc, kv, new, 4, window=window, sinks=2 if window else 0, check=False)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
