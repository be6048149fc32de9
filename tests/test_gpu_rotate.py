"""Head norms, rotation and append on the GPU against the fp64 oracle.

Tolerances.  The angle: its turns are cut to 32 bits (2^-32 of a turn), turned to 24 (2^-25 of
a half turn) and the frequency is off by 2^-65 a position, so under 2^-23 radians in all;
sine and cosine add 2 half-steps of 24 bits each way: 2^-22 of each.  The norm's factor: eight
products and sums in a lane and four sums of lanes (12 half-steps of a sum of squares, half of
that in its root), the reciprocal root 2^-22, two products: under 2^-20.5 of a value.  A
result a c - b s is so off by less than 2^-19.5 (|a| + |b|) before its rounding: half a step of
bf16, 2^-8; of int8, half a scale; of e4m3, 2^-4 or, below 2^-6 of a scale, 2^-10 scales.  A
scale is max|y| / Q, off by what the largest value is and half a step of fp32.
"""
import math

import numpy as np
import pytest

from test_gpu_dense import BF16, E4M3, INT8, KINDS, NAME, Paged, _np, _tokens, dhs, torch  # noqa: F401

pytestmark = pytest.mark.gpu
OFF = 2.0 ** -19.5


def _freqs(n, base=10000.0):
    return base ** (-np.arange(n) / max(1, n))


def _weight(torch, d, seed):
    return (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(seed))).float()


def _check(out, want, mag):
    # bf16 has no value from half a step above its largest, (2 - 2^-7) 2^127, on: infinity
    want = np.where(np.abs(want) >= (2 - 2.0 ** -8) * 2.0 ** 127, np.copysign(np.inf, want), want)
    tol = 2.0 ** -8 * np.abs(want) + OFF * mag + 1e-37
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(out), fine)
    assert np.array_equal(out[np.isinf(want)], want[np.isinf(want)])
    bad = fine & ~(np.abs(np.where(fine, out - want, 0)) <= np.where(fine, tol, 0))
    assert not bad.any(), (np.argwhere(bad)[0], out[bad][0], want[bad][0])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pairs,halves", [(0, True), (4, True), (12, True), (12, False), (32, True),
                                          (32, False), (64, True), (64, False)])
@pytest.mark.parametrize("norm", [False, True])
def test_rotate(torch, dhs, d, pairs, halves, norm):
    from oracle import dense_oracle as oracle
    if 2 * pairs > d:
        pairs = d // 2 - 8
    freqs = _freqs(pairs)
    rot = None if not pairs else dhs.Rotation(freqs, dhs.ROTATE_HALVES if halves else dhs.ROTATE_NEIGHBOURS,
                                              amplitude=1.25)
    for n, hq, hkv in ((1, 8, 1), (5, 3, 1), (37, 6, 2)):
        g = torch.Generator().manual_seed(n)
        q, k = (torch.randn((n, h, d), generator=g).mul(3).bfloat16() for h in (hq, hkv))
        pos = torch.randint(0, 200000, (n,), generator=g, dtype=torch.int32)
        pos[0] = 2147483647
        if n > 3:
            pos[1:4] = torch.tensor([-2147483648, 0, -5], dtype=torch.int32)
        wq, wk = (_weight(torch, d, s) if norm else None for s in (1, 2))
        qo, ko = torch.full_like(q, 7).cuda(), torch.full_like(k, 7).cuda()
        dhs.rotate(q.cuda(), k.cuda(), pos.cuda(), rot, qo, ko,
                   q_norm=None if wq is None else wq.cuda(), k_norm=None if wk is None else wk.cuda())
        for x, o, w in ((q, qo, wq), (k, ko, wk)):
            want, mag = oracle.rotate(_np(x), None if w is None else _np(w), 1e-6, pos.tolist(), freqs,
                                      halves, 1.25)
            _check(_np(o), want, mag)
            if not pairs and not norm:
                assert torch.equal(o.cpu(), x)


def test_rotate_one_of_both_strided_and_in_place(torch, dhs):
    d, hq, hkv, n = 128, 6, 2, 300
    rot = dhs.Rotation(_freqs(64))
    g = torch.Generator().manual_seed(4)
    packed = torch.randn((n, hq + 2 * hkv, d), generator=g).bfloat16().cuda()
    q, k = packed[:, :hq], packed[:, hq:hq + hkv]
    pos = torch.arange(n, dtype=torch.int32).cuda() * 331
    w = _weight(torch, d, 3).cuda()
    qo, ko = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty(
        (n, hkv, d), dtype=torch.bfloat16, device="cuda")
    dhs.rotate(q.contiguous(), k.contiguous(), pos, rot, qo, ko, q_norm=w, k_norm=w)
    one, two = torch.full_like(qo, 5), torch.full_like(ko, 5)
    dhs.rotate(q, None, pos, rot, one, None, q_norm=w)
    dhs.rotate(None, k, pos, rot, None, two, k_norm=w)
    assert torch.equal(one, qo) and torch.equal(two, ko)
    heads_first = torch.full((hq, n, d), 9, dtype=torch.bfloat16, device="cuda")
    dhs.rotate(q, k, pos, rot, heads_first.transpose(0, 1), two, q_norm=w, k_norm=w)
    assert torch.equal(heads_first.transpose(0, 1), qo)
    values = packed[:, hq + hkv:].clone()
    dhs.rotate(q, k, pos, rot, q, k, q_norm=w, k_norm=w)    # in place, between the values
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(packed[:, hq + hkv:], values)
    with pytest.raises(dhs.DhsError):
        dhs.rotate(q, k, pos, rot, packed[:, 1:hq + 1], two)   # one head further on
    with pytest.raises(dhs.DhsError):
        dhs.rotate(qo, None, pos, rot, qo[:1].expand(n, hq, d), None)


def test_rotate_values_that_are_not_finite_or_large(torch, dhs):
    from oracle import dense_oracle as oracle
    d, n = 64, 12
    rot, w = dhs.Rotation(_freqs(16)), _weight(torch, 64, 1)
    x = _tokens(torch, n, 1, d, 3)      # zeros, tiny, an infinity, a NaN, the largest among them
    x[8:] *= torch.tensor([2.0 ** 50, 2.0 ** -45, 2.0 ** -64, 2.0 ** 62])[:, None, None]
    pos = torch.arange(n, dtype=torch.int32)
    for norm in (None, w):
        out = torch.empty_like(x).cuda()
        dhs.rotate(x.cuda(), None, pos.cuda(), rot, out, None, q_norm=None if norm is None else norm.cuda())
        rows = [i for i in range(n) if i not in (2, 3)]
        want, mag = oracle.rotate(_np(x[rows]), None if norm is None else _np(norm), 1e-6,
                                  [int(pos[i]) for i in rows], _freqs(16), True)
        _check(_np(out[rows]), want, mag)
        if norm is not None:            # without an eps the smallest rows have a norm, too
            dhs.rotate(x.cuda(), None, pos.cuda(), rot, out, None, q_norm=norm.cuda(), eps=0.0)
            want, mag = oracle.rotate(_np(x[rows[1:]]), _np(norm), 0.0, [int(pos[i]) for i in rows[1:]],
                                      _freqs(16), True)
            _check(_np(out[rows[1:]]), want, mag)
            assert torch.isnan(out[0]).all()
        assert (~torch.isfinite(out[2:4])).any(-1).all()   # both rows say that something is wrong


def test_many_heads_and_tokens(torch, dhs):
    """More heads than a CTA has rows, and more tokens than CTAs: every row against one call
    per token."""
    d, n, h = 64, 2003, 40
    rot, w = dhs.Rotation(_freqs(32)), _weight(torch, 64, 5).cuda()
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn((n, h, d), generator=g, device="cuda").bfloat16()
    k = torch.randn((n, 3, d), generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 1 << 30, (n,), generator=g, device="cuda", dtype=torch.int32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    dhs.rotate(q, k, pos, rot, qo, ko, q_norm=w)
    q1, k1 = torch.empty_like(q), torch.empty_like(k)
    for t in list(range(0, n, 97)) + [n - 1]:
        dhs.rotate(q[t:t + 1], k[t:t + 1], pos[t:t + 1], rot, q1[t:t + 1], k1[t:t + 1], q_norm=w)
        assert torch.equal(q1[t], qo[t]) and torch.equal(k1[t], ko[t]), t


def _append_setup(torch, dhs, kind, d, hkv, rows, hq=6, lens=(0, 1, 40, 129, 5), new=(0, 1, 40, 3, 5)):
    pc = Paged(torch, dhs, list(lens), rows, hkv, d, kind)
    cu = torch.tensor([2] + list(new)).cumsum(0).int().cuda()  # two tokens of padding before, three after
    n = 2 + sum(new) + 3
    g = torch.Generator().manual_seed(3)
    q = torch.randn((n, hq, d), generator=g).bfloat16()
    return pc, cu, q, _tokens(torch, n, hkv, d, 1), _tokens(torch, n, hkv, d, 2)


def _bytes(c):
    return [None if t is None else t.clone().view(torch_uint8(t)) for t in (c.k, c.v, c.k_scale, c.v_scale)]


def torch_uint8(t):
    import torch
    return torch.uint8


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,hkv,rows,pairs,halves,norm", [
    (128, 1, 64, 64, True, True), (64, 3, 16, 32, False, False), (128, 8, 7, 16, True, False),
    (64, 2, 1, 0, True, True), (128, 2, 48, 0, True, False)])
def test_append(torch, dhs, kind, d, hkv, rows, pairs, halves, norm):
    from oracle import dense_oracle as oracle
    pc, cu, q, k, v = _append_setup(torch, dhs, kind, d, hkv, rows)
    c, lens, new = pc.cache, pc.lens, [0, 1, 40, 3, 5]
    freqs = _freqs(pairs)
    rot = None if not pairs else dhs.Rotation(freqs, dhs.ROTATE_HALVES if halves else dhs.ROTATE_NEIGHBOURS)
    wq, wk = (_weight(torch, d, s) if norm else None for s in (1, 2))
    gpu = lambda t: None if t is None else t.cuda()  # noqa: E731
    # the same without the cache, and the values (and keys that are not touched) by the write
    at = {}
    for i, (a, t) in enumerate(zip(new, lens)):
        for u in range(a):
            at[int(cu[i]) + u] = (i, t - a + u)
    pos = torch.tensor([at.get(t, (0, 0))[1] for t in range(len(q))], dtype=torch.int32)
    q1, k1 = torch.full_like(q, 9).cuda(), torch.full_like(k, 9).cuda()
    dhs.rotate(q.cuda(), k.cuda(), pos.cuda(), rot, q1, k1, q_norm=gpu(wq), k_norm=gpu(wk))
    other = Paged(torch, dhs, lens, rows, hkv, d, kind).cache
    other.write(k1, v.cuda(), cu, pc.seq_lens, pc.table)
    before = _bytes(c)
    qo, ko = torch.full_like(q, 9).cuda(), torch.full_like(k, 9).cuda()
    c.append(q.cuda(), k.cuda(), v.cuda(), cu, pc.seq_lens, pc.table, qo, rot, q_norm=gpu(wq),
             k_norm=gpu(wk), k_out=ko)
    c.check()
    inside = torch.tensor(sorted(at))
    outside = torch.tensor([t for t in range(len(q)) if t not in at])
    assert torch.equal(qo[inside].view(torch.int16), q1[inside].view(torch.int16))
    assert torch.equal(ko[inside].view(torch.int16), k1[inside].view(torch.int16))
    assert torch.all(qo[outside] == 9) and torch.all(ko[outside] == 9)
    assert torch.equal(c.v.view(torch.uint8), other.v.view(torch.uint8))
    if kind != BF16:
        assert torch.equal(c.v_scale.view(torch.int32), other.v_scale.view(torch.int32))
    if kind == BF16 or (not pairs and not norm):
        assert torch.equal(c.k.view(torch.uint8), other.k.view(torch.uint8))
        if kind != BF16:
            assert torch.equal(c.k_scale.view(torch.int32), other.k_scale.view(torch.int32))
        return
    table, touched = pc.table.cpu(), torch.zeros(c.k.shape[:3], dtype=torch.bool)
    for t, (i, p) in at.items():
        page, row = int(table[i, p // rows]), p % rows
        touched[page, :, row] = True
        want, mag = oracle.rotate(_np(k[t:t + 1]), None if wk is None else _np(wk), 1e-6, [p], freqs, halves)
        codes, scales = c.k[page, :, row].double().cpu().numpy(), _np(c.k_scale[page, :, row])
        for h in range(hkv):
            y, m = want[0, h], mag[0, h]
            if not (np.abs(y) < 2.0 ** 128).all():   # (in 32 bits an infinity, or a NaN)
                assert np.isnan(scales[h]) and not codes[h].any()
                continue
            if np.abs(y).max() < 2.0 ** -100 * (1 - 2.0 ** -18):
                assert scales[h] == 0 and not codes[h].any()
                continue
            Q = oracle.QMAX[NAME[kind]]
            s = np.abs(y).max() / Q
            assert abs(scales[h] - s) <= OFF * m.max() / Q + 2.0 ** -23 * s
            half = scales[h] * 0.5 if kind == INT8 else np.maximum(2.0 ** -4 * np.abs(y), scales[h] * 2.0 ** -10)
            # (the quotient's own half-steps: 2^-22 of a value)
            tol = half * (1 + 2.0 ** -20) + OFF * m + 2.0 ** -22 * np.abs(y) + OFF * m.max() * 2
            assert np.all(np.abs(codes[h] * scales[h] - y) <= tol), (t, h)
    for now, was in zip((c.k, c.k_scale), (before[0], before[2])):
        now, was = now.view(torch.uint8).cpu(), was.cpu()
        keep = ~touched
        assert torch.equal(now.reshape(*keep.shape, -1)[keep], was.reshape(*keep.shape, -1)[keep])


def test_append_without_queries_strided_and_other_positions(torch, dhs):
    pc, cu, q, k, v = _append_setup(torch, dhs, BF16, 64, 3, 16)
    rot = dhs.Rotation(_freqs(32))
    n = len(q)
    packed = torch.cat([q, k, v], 1).cuda()
    pos = (torch.arange(n, dtype=torch.int32) * 1001 - 7).cuda()
    qo, ko, k1 = torch.empty_like(q).cuda(), torch.empty_like(k).cuda(), torch.empty_like(k).cuda()
    dhs.rotate(q.cuda(), k.cuda(), pos, rot, qo, ko)
    other = Paged(torch, dhs, pc.lens, 16, 3, 64, BF16).cache
    other.write(ko, v.cuda(), cu, pc.seq_lens, pc.table)
    pc.cache.append(None, packed[:, 6:9], packed[:, 9:], cu, pc.seq_lens, pc.table, None, rot, positions=pos)
    pc.cache.check()
    for a, b in ((pc.cache.k, other.k), (pc.cache.v, other.v)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    # queries in place within the packed projections
    pc.cache.append(packed[:, :6], packed[:, 6:9], packed[:, 9:], cu, pc.seq_lens, pc.table, packed[:, :6], rot,
                    positions=pos, k_out=k1)
    inside = slice(2, n - 3)
    assert torch.equal(packed[inside, :6], qo[inside])
    assert torch.equal(k1[inside].view(torch.int16), ko[inside].view(torch.int16))
    assert torch.equal(packed[:2, :6].cpu(), q[:2])
    with pytest.raises(ValueError):
        pc.cache.append(q.cuda(), k.cuda(), v[:, :2].cuda(), cu, pc.seq_lens, pc.table, qo, rot)
    with pytest.raises(ValueError):
        pc.cache.append(q[:3].cuda(), k.cuda(), v.cuda(), cu, pc.seq_lens, pc.table, qo[:3], rot)


@pytest.mark.parametrize("what", ["page_high", "page_negative", "short", "long"])
def test_append_reports_and_skips(torch, dhs, what):
    """The tokens of sequence 2 that have no place leave everything as it was; the others land."""
    lens, new = [4, 20, 33], [4, 2, 3]
    pc, cu, q, k, v = _append_setup(torch, dhs, INT8, 64, 2, 16, lens=lens, new=new)
    rot = dhs.Rotation(_freqs(32))
    table, seq_lens = pc.table.clone(), pc.seq_lens.clone()
    bad = [2, 1, 0]                       # sequence 2's tokens are at 30, 31 and 32
    if what == "page_high":
        table[2, 2] = pc.n_pages
        bad = [2]
    elif what == "page_negative":
        table[2, 1] = -1
        bad = [0, 1]
    elif what == "short":
        seq_lens[2] = 2
        bad = [0]
    else:
        seq_lens[2] = table.shape[1] * 16 + 2
        bad = [1, 2]
        table[2, :] = table[2, 0]
    good = Paged(torch, dhs, lens, 16, 2, 64, INT8).cache
    qo, q1 = torch.full_like(q, 9).cuda(), torch.full_like(q, 9).cuda()
    pc.cache.append(q.cuda(), k.cuda(), v.cuda(), cu, seq_lens, table, qo, rot)
    with pytest.raises(dhs.DhsError, match="dhs_page_append"):
        pc.cache.check()
    pc.cache.check()
    good.append(q.cuda(), k.cuda(), v.cuda(), cu, pc.seq_lens, pc.table, q1, rot)
    t2 = int(cu[2])
    for u in range(3):
        if u in bad:
            assert torch.all(qo[t2 + u] == 9)
        elif what.startswith("page"):
            assert torch.equal(qo[t2 + u], q1[t2 + u])
    assert torch.equal(qo[2:t2], q1[2:t2])
    for i in (0, 1):
        pages = pc.table[i, :-(-lens[i] // 16)].long()
        assert torch.equal(pc.cache.k[pages], good.k[pages]) and torch.equal(pc.cache.v[pages], good.v[pages])


def test_append_captured_follows_lengths_and_on_another_stream(torch, dhs):
    lens, new = [5, 70], [1, 1]
    pc = Paged(torch, dhs, [80, 80], 16, 2, 128, E4M3)
    ref = Paged(torch, dhs, [80, 80], 16, 2, 128, E4M3)
    rot, w = dhs.Rotation(_freqs(64)), _weight(torch, 128, 1).cuda()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((2, h, 128), generator=g).bfloat16().cuda() for h in (8, 2, 2))
    seq_lens = torch.tensor(lens, dtype=torch.int32).cuda()
    qo, q1 = torch.empty_like(q), torch.empty_like(q)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pc.cache.append(q, k, v, cu, seq_lens, pc.table, qo, rot, q_norm=w, k_norm=w)
    for step in range(3):
        seq_lens.copy_(torch.tensor([5 + step, 70 + step], dtype=torch.int32))
        q.copy_(torch.randn(q.shape, generator=g).bfloat16())
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        ref.cache.append(q, k, v, cu, seq_lens, ref.table, q1, rot, q_norm=w, k_norm=w, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(qo, q1)
        for a, b in ((pc.cache.k, ref.cache.k), (pc.cache.v, ref.cache.v)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    pc.cache.check()


def test_append_far_pages_and_more_heads_than_a_launch_has_rows_of(torch, dhs):
    """Pages whose elements lie beyond 2^31, and 70000 heads of queries."""
    rows, hkv, d = 64, 2, 64
    pc = Paged(torch, dhs, [130], rows, hkv, d, INT8, huge_pages=2 ** 31 // (rows * hkv * d) + 9)
    ref = Paged(torch, dhs, [130], rows, hkv, d, INT8)
    rot = dhs.Rotation(_freqs(32))
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn((3, hkv, d), generator=g).bfloat16().cuda() for _ in range(2))
    cu = torch.tensor([0, 3], dtype=torch.int32).cuda()
    for p in (pc, ref):
        p.cache.append(None, k, v, cu, p.seq_lens, p.table, None, rot)
        p.cache.check()
    at, to = pc.table[0, :3].long(), ref.table[0, :3].long()
    assert int(at.max()) * rows * hkv * d > 2 ** 31
    for a, b in ((pc.cache.k, ref.cache.k), (pc.cache.v, ref.cache.v), (pc.cache.k_scale, ref.cache.k_scale)):
        assert torch.equal(a[at].view(torch.uint8), b[to].view(torch.uint8))
    q = torch.randn((2, 70000, d), generator=g).bfloat16().cuda()
    pos = torch.tensor([5, 100000], dtype=torch.int32).cuda()
    out, few = torch.empty_like(q), torch.empty((2, 7, d), dtype=torch.bfloat16, device="cuda")
    dhs.rotate(q, None, pos, rot, out, None)
    for h in (0, 35000, 69993):
        dhs.rotate(q[:, h:h + 7], None, pos, rot, few, None)
        assert torch.equal(out[:, h:h + 7], few)
